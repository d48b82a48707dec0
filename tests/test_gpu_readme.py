"""The serving example of README.md, run as it stands there."""
import os
import re

import pytest
import torch

from online_softmax_08_gb300 import fattn

pytestmark = pytest.mark.gpu

README = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "README.md")


def test_serving_example():
    """A prompt, single tokens, a cut, single tokens again and a second cut: no sequence is skipped,
    and every query's weight arrives at the keys."""
    text = open(README).read()
    code = [x for x in re.findall(r"```python\n(.*?)```", text, re.S) if "cache_evict" in x]
    assert len(code) == 1
    B, H, Hq, bs, keep = 2, 8, 32, 64, 2048
    space = {"torch": torch, "fattn": fattn}
    exec(code[0], space)  # a cache, a table, step() and cut()
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32, device="cuda")
    width = 40  # blocks of a sequence
    tables = [torch.arange(x, x + B * width, dtype=torch.int32, device="cuda").reshape(B, width)
              for x in (0, B * width)]
    g = torch.Generator(device="cuda").manual_seed(1)
    fattn.fattn_device_error()
    lens, weights, position, mass = [0, 0], None, [0, 0], 0.0
    batch = None
    for new in ([2200, 1800], [1, 1], "cut", [1, 1], [1, 1], [400, 1], "cut", [1, 1]):
        if new == "cut":
            batch, weights = space["cut"](batch, weights, tables[1])
            tables.reverse()
            lens = [min(x, keep) for x in lens]
            assert batch.lens.tolist() == lens and torch.equal(batch.block_table, tables[0])
            continue
        lens = [a + n for a, n in zip(lens, new)]
        total = sum(new)
        pos = torch.cat([torch.arange(p, p + n) for p, n in zip(position, new)]).int().cuda()
        position = [p + n for p, n in zip(position, new)]
        q, k, v = (torch.randn((total, h, 128), generator=g, device="cuda").bfloat16() for h in (Hq, H, H))
        batch = fattn.CacheBatch(tables[0], i32(*lens), i32(0, new[0], total), total, max(new))
        before = None if weights is None else weights.clone()
        o, weights = space["step"](q, k, v, pos, batch, weights)
        assert o.shape == (total, Hq, 128) and fattn.fattn_device_error() == 0
        for b in range(B):
            was = 0.0 if before is None else before[b, :, :lens[b] - new[b]].double().sum(dim=1)
            got = weights[b, :, :lens[b]].double().sum(dim=1) - was
            # each of the group's queries has a weight of one in all
            assert float((got - new[b] * Hq // H).abs().max()) <= 1e-4 * new[b] * Hq // H + 1e-3
    assert fattn.fattn_device_error() == 0

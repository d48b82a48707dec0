"""Argument checks of the 8-bit cache's entry points that need no GPU: each call
here fails validation before the library touches the device."""
import pytest
import torch

from online_softmax_08_gb300 import build as fbuild
from online_softmax_08_gb300 import fattn

# The descriptors are packed as the C structs are laid out (native alignment).
A = 1 << 20  # 256-byte aligned, never dereferenced
INVALID, UNSUPPORTED, CUDA, WORKSPACE = 1, 2, 3, 4


@pytest.fixture(scope="module")
def lib():
    fbuild.build()
    return fattn.load()


def _cache(**kw):
    f = dict(k=A, v=A, k_scale=A, v_scale=A, num_blocks=10, H=4, block_size=16, d=64, format=0)
    f.update(kw)
    return fattn._pack_cache(*f.values())


def _batch(**kw):
    f = dict(block_table=A, lens=A, cu_seqlens=A, B=2, table_width=4, total=8, max_seqlen=5)
    f.update(kw)
    return fattn._pack_batch(*f.values())


def _append(lib, c, b, k=A, kst=256, ksh=64, v=A, vst=256, vsh=64):
    return lib.fattn_cache_append(c, b, k, kst, ksh, v, vst, vsh, None)


def _read(lib, c, b, k=A, kst=256, ksh=64, v=A, vst=256, vsh=64):
    return lib.fattn_cache_read(c, b, k, kst, ksh, v, vst, vsh, None)


def _fwd(lib, c, b, q=A, qst=512, qsh=64, o=A, ost=512, osh=64, lse=A, Hq=8, scale=0.1, ws=A,
         nbytes=1 << 40):
    return lib.fattn_cache_fwd(c, b, q, qst, qsh, o, ost, osh, lse, Hq, scale, 1, ws, nbytes, None)


BAD_CACHE = [(dict(k=0), INVALID), (dict(v=A + 8), INVALID), (dict(k_scale=0), INVALID),
             (dict(v_scale=A + 2), INVALID), (dict(num_blocks=1 << 30), INVALID), (dict(num_blocks=0), INVALID), (dict(H=0), INVALID),
             (dict(H=1 << 17), INVALID), (dict(block_size=48), UNSUPPORTED),
             (dict(block_size=0), UNSUPPORTED), (dict(d=96), UNSUPPORTED),
             (dict(format=2), UNSUPPORTED)]
BAD_BATCH = [(dict(block_table=0), INVALID), (dict(lens=A + 2), INVALID),
             (dict(cu_seqlens=0), INVALID), (dict(B=0), INVALID), (dict(table_width=0), INVALID),
             (dict(total=-1), INVALID), (dict(max_seqlen=9), INVALID),
             (dict(max_seqlen=-1), INVALID), (dict(table_width=1 << 27), INVALID),
             (dict(table_width=(1 << 27) - 1), INVALID), (dict(table_width=(1 << 27) - 4095), INVALID),
             (dict(total=(1 << 31) - 1, max_seqlen=1), INVALID), (dict(B=1 << 25), INVALID)]


@pytest.mark.parametrize("call", [_append, _read, _fwd])
def test_bad_descriptors(lib, call):
    for kw, status in BAD_CACHE:
        assert call(lib, _cache(**kw), _batch()) == status, kw
    for kw, status in BAD_BATCH:
        assert call(lib, _cache(), _batch(**kw)) == status, kw
    assert call(lib, None, _batch()) == INVALID
    assert call(lib, _cache(), None) == INVALID
    # nothing to do: fine without touching the device
    assert call(lib, _cache(), _batch(total=0, max_seqlen=0)) == 0
    assert call(lib, _cache(), _batch(max_seqlen=0)) == 0


@pytest.mark.parametrize("call", [_append, _read])
def test_bad_tokens(lib, call):
    c, b = _cache(), _batch()
    for kw in (dict(k=None), dict(v=A + 2), dict(kst=260), dict(vsh=4), dict(kst=-256),
               dict(ksh=1 << 41), dict(vst=1 << 31)):
        assert call(lib, c, b, **kw) == INVALID, kw


def test_overlapping_outputs_are_refused(lib):
    c, b = _cache(), _batch()
    for st, sh in ((64, 64), (0, 64), (256, 0), (192, 64), (64, 448)):
        assert _read(lib, c, b, kst=st, ksh=sh) == INVALID, (st, sh)
        assert _fwd(lib, c, b, ost=st, osh=sh) == INVALID, (st, sh)
    if not torch.cuda.is_available():  # accepted: the calls go on to the device
        for st, sh in ((256, 64), (64, 512), (1024, 128)):
            assert _read(lib, c, b, kst=st, ksh=sh) == CUDA, (st, sh)
        assert _append(lib, c, b, kst=0, ksh=64) == CUDA  # inputs may be broadcast


def test_longest_table(lib):
    b = _batch(table_width=(1 << 27) - 4096)  # 2^31 - 65536 tokens
    if not torch.cuda.is_available():  # accepted: the calls go on to the device
        assert _append(lib, _cache(), b) == _read(lib, _cache(), b) == _fwd(lib, _cache(), b) == CUDA


def test_bad_attention_arguments(lib):
    c, b = _cache(), _batch()
    for kw in (dict(q=None), dict(o=A + 8), dict(lse=None), dict(Hq=6), dict(Hq=0), dict(scale=0.0),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(qst=-8), dict(qsh=12)):
        assert _fwd(lib, c, b, **kw) == INVALID, kw
    assert _fwd(lib, c, b, ws=None) == WORKSPACE
    assert _fwd(lib, c, b, ws=A + 128) == WORKSPACE
    assert lib.fattn_cache_fwd_workspace_bytes(_cache(d=80), b, 8) == 0
    assert lib.fattn_cache_fwd_workspace_bytes(c, b, 6) == 0


def test_binding_refuses_wrong_tensors():
    cache = fattn.new_cache(6, 2, 16, 64, device="cpu")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    batch = fattn.CacheBatch(i32([0, 1], [2, 3]), i32(20, 9), i32(0, 3, 5), 5, 3)
    x = torch.zeros((5, 2, 64), dtype=torch.bfloat16)
    bad = [
        (x, x, cache._replace(v=cache.v[:5]), batch),
        (x, x, cache._replace(k=cache.k.view(torch.uint8)), batch),
        (x, x, cache._replace(k_scale=cache.k_scale.double()), batch),
        (x, x, cache._replace(v_scale=cache.v_scale.t()), batch),
        (x, x, cache, batch._replace(lens=i32(1, 2, 3))),
        (x, x, cache, batch._replace(cu_seqlens=batch.cu_seqlens.long())),
        (x, x, cache, batch._replace(block_table=batch.block_table.t())),
        (x.float(), x, cache, batch),
        (x, x[:4], cache, batch),
        (x, x.transpose(1, 2).contiguous().transpose(1, 2), cache, batch),
    ]
    for k, v, c, b in bad:
        with pytest.raises(ValueError):
            fattn.cache_append(k, v, c, b)
    with pytest.raises(ValueError):
        fattn.cache_forward(x[0], cache, batch, 0.1, True)
    with pytest.raises(ValueError):
        fattn.new_cache(6, 2, 16, 64, dtype=torch.bfloat16, device="cpu")


def test_a_failed_workspace_query_is_not_remembered(monkeypatch):
    """0 bytes is the query's failure; the next call of the same sizes asks again."""
    class Lib:
        answers, calls = [0, 4096], []

        def fattn_cache_fwd_workspace_bytes(self, c, b, Hq):
            return self.answers.pop(0)

        def fattn_cache_fwd(self, *args):
            self.calls.append(args[13])
            return WORKSPACE if args[13] < 4096 else 0

    cache = fattn.new_cache(6, 2, 16, 64, device="cpu")
    i32 = lambda *a: torch.tensor(a, dtype=torch.int32)
    batch = fattn.CacheBatch(i32([0, 1], [2, 3]), i32(20, 9), i32(0, 3, 5), 5, 3)
    q = torch.zeros((5, 4, 64), dtype=torch.bfloat16)
    monkeypatch.setattr(fattn, "_cache_args", lambda c, b: (b"", b"", -1, 2, 64))
    monkeypatch.setattr(fattn, "_elsewhere", lambda dev, stream: False)
    monkeypatch.setattr(fattn, "_raw_stream", lambda dev: 0)
    monkeypatch.setattr(fattn, "_ws_bytes", {})
    monkeypatch.setattr(fattn, "_lib", Lib())
    with pytest.raises(fattn.FattnError):
        fattn.cache_forward(q, cache, batch, 0.1, True)
    for _ in range(2):  # the answer is asked for once
        fattn.cache_forward(q, cache, batch, 0.1, True)
    assert Lib.calls[1:] == [4096, 4096] and not Lib.answers

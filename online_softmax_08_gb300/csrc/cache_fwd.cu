// cache_fwd.cu -- attention over the paged 8-bit key/value cache.
//
// One warp per (query token, query head): lanes take 32 keys at a time, then
// the d columns of the values.
#include "cache.cuh"

namespace fattn {
namespace {

template <int D, bool E5M2>
__global__ void __launch_bounds__(128) cache_fwd_plain_kernel(const CacheFwdParams p) {
  __shared__ float sq[4][D];
  const CacheParams& c = p.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const long long row = (long long)blockIdx.x * 4 + warp;
  if (row >= (long long)c.total * p.Hq) return;
  const int t = (int)(row / p.Hq), hq = (int)(row % p.Hq);
  const int h = hq / (p.Hq / c.H);
  const int b = warp_search(c.B, t, [&](int i) { return (long long)c.cu_seqlens[i]; });
  CacheSeq s;
  if (!cache_seq(c, b, &s)) {
    if (lane == 0 && c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD);
    return;
  }
  if (t >= s.row0 + s.n) return;  // behind the last sequence
  const int limit = p.causal ? s.len - s.n + (t - s.row0) + 1 : s.len;  // keys [0, limit)
  const uint16_t* q = p.q.p + (long long)t * p.q.st + (long long)hq * p.q.sh;
  for (int i = lane; i < D; i += 32) sq[warp][i] = __uint_as_float((uint32_t)q[i] << 16);
  __syncwarp();
  float m = -INFINITY, l = 0.f, acc[D / 32];
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int j0 = 0; j0 < limit; j0 += 32) {
    const int j = j0 + lane;
    float x = -INFINITY, vs = 0.f;
    long long off = 0;
    if (j < limit) {
      const int page = c.block_table[(long long)b * c.table_width + j / c.block_size];
      if (page < 0 || page >= c.num_blocks) {
        if (c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD + 1);
      } else {
        const long long block = (long long)page * c.H + h;
        off = (block * c.block_size + j % c.block_size) * D;
        const uint16_t* k = reinterpret_cast<const uint16_t*>(c.k + off);
        float dot = 0.f;
        for (int i = 0; i < D / 2; ++i) {
          const float2 f = f16x2_to_f32(codes_to_f16x2<E5M2>(k[i]));
          dot = fmaf(f.x, sq[warp][2 * i], dot);
          dot = fmaf(f.y, sq[warp][2 * i + 1], dot);
        }
        x = dot * c.k_scale[block] * p.scale_log2;
        vs = c.v_scale[block];
      }
    }
    const bool seen = x != -INFINITY;
    float mb = x;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) mb = fmaxf(mb, __shfl_xor_sync(0xffffffffu, mb, w));
    const unsigned any = __ballot_sync(0xffffffffu, seen);
    if (any == 0u) continue;
    const float mn = fmaxf(m, mb);
    const float ref = mn == -INFINITY ? 0.f : mn;
    const float alpha = ex2(m - ref);
    const float pj = seen ? ex2(x - ref) : 0.f;
    float sum = pj;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, w);
    l = l * alpha + sum;
    m = mn;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) acc[i] *= alpha;
    for (int k = 0; k < 32; ++k) {
      if (!(any >> k & 1u)) continue;
      const float w = __shfl_sync(0xffffffffu, pj, k) * __shfl_sync(0xffffffffu, vs, k);
      const long long o = __shfl_sync(0xffffffffu, off, k);
#pragma unroll
      for (int i = 0; i < D / 32; ++i)
        acc[i] = fmaf(w, f16x2_to_f32(codes_to_f16x2<E5M2>(c.v[o + lane + 32 * i])).x, acc[i]);
    }
  }
  const bool has = limit > 0 && !(l == 0.f);
  const float inv = has ? 1.f / l : 0.f;
  uint16_t* o = p.o.p + (long long)t * p.o.st + (long long)hq * p.o.sh;
#pragma unroll
  for (int i = 0; i < D / 32; ++i)
    o[lane + 32 * i] = (uint16_t)(pack_bf16x2(has ? acc[i] * inv : 0.f, 0.f) & 0xffffu);
  if (lane == 0)
    p.lse[(long long)hq * c.total + t] =
        has ? (m + lg2(l)) * 0.6931471805599453f : -INFINITY;
}

}  // namespace

size_t cache_fwd_workspace(const CacheParams&, int, int) { return 256; }

cudaError_t launch_cache_fwd(const CacheFwdParams& p, int, cudaStream_t stream) {
  const long long ctas = ((long long)p.c.total * p.Hq + 3) / 4;
  if (p.c.d == 128) {
    if (p.c.format) cache_fwd_plain_kernel<128, true><<<(unsigned)ctas, 128, 0, stream>>>(p);
    else cache_fwd_plain_kernel<128, false><<<(unsigned)ctas, 128, 0, stream>>>(p);
  } else {
    if (p.c.format) cache_fwd_plain_kernel<64, true><<<(unsigned)ctas, 128, 0, stream>>>(p);
    else cache_fwd_plain_kernel<64, false><<<(unsigned)ctas, 128, 0, stream>>>(p);
  }
  return cudaGetLastError();
}

}  // namespace fattn

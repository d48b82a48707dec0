// cache4.cu -- the key/value cache in 4 bits: new tokens quantised into paged blocks, and
// tokens read back.
//
// A group of 16 neighbouring channels of a token shares an e5m2 scale s and has 16 codes c,
// value (c - 8) s, two to a byte, the even channel in the low half.  With a the largest
// magnitude of the group,
//   |s| = rn_e5m2(a / 8),  s < 0 if the group holds +a (which then gets the code 0) else s > 0,
//   c = 8 + clamp(rn(x / s), -8, 7).
// The largest value so takes the one level that has no opposite, -8, and a step is a / 8.
// Every token stands alone: nothing that was written before is read or changed.
//
// rn(x / s) is exact.  x has 8 significant bits and s 3, so x / s either is a tie n + 1/2
// (n below 13) or lies at least 2^-8 of its value away from one.  x times the rounded 1 / s
// is off by 2^-23 of it at most; rounded to fp16 (2^-11) a tie becomes what it is and
// nothing else becomes one; adding 1544 rounds that to the nearest whole number, ties to
// even, and leaves the code in the low four bits.
//
// The bound is memory.  A thread holds one group: 32 bytes of bf16 and 8 + 1 of the cache.
// A warp takes kIter x 32 groups of one head: the rows of 16 (d = 64: 32) packed tokens one
// behind another, so a prompt's codes and scales are written as whole lines.  The values are
// on their way while the tokens' places are looked up.  Bad entries of the batch are looked
// for by the first warps, so that one without tokens is found as well.
#include "cache.cuh"

namespace fattn {
namespace {

constexpr int kWarps4 = 4;
constexpr int kIter = 4;  // groups per thread

template <int D>
struct Quad {
  static constexpr int LPR = D / 16;        // lanes of a row: one per group
  static constexpr int RPI = 32 / LPR;      // rows that a warp takes at a time
  static constexpr int TOK = kIter * RPI;   // tokens of a warp
};

// Row of packed token `tok` in the pool, (block * H + h) * block_size + row; -1: no such
// token, -2: a token without a place.  Called by whole warps for tok0 + lane.
__device__ __forceinline__ long long place_of(const CacheParams& c, int h, int tok0, int count,
                                              uint32_t site) {
  const int lane = threadIdx.x & 31, tok = tok0 + lane;
  const int b0 = warp_search(c.B, (long long)tok0, [&](int b) { return (long long)c.cu_seqlens[b]; });
  // the sequences that start behind b0 and at or before this token: a window of 32, and
  // what lies behind it (rare) one by one
  const int next = c.cu_seqlens[min(b0 + 1 + lane, c.B)];
  int add = 0;
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) {
    const int x = __shfl_sync(0xffffffffu, next, (add + w - 1) & 31);
    if (b0 + add + w < c.B && x <= tok) add += w;
  }
  const int last = __shfl_sync(0xffffffffu, next, 31);
  if (lane >= count || tok >= c.total) return -1;
  int b = b0 + add;
  if (add == 31 && b0 + 32 < c.B && last <= tok) {
    b = b0 + 32;
    int hi = c.B;
    while (hi - b > 1) {
      const int mid = (b + hi) >> 1;
      if (c.cu_seqlens[mid] <= tok)
        b = mid;
      else
        hi = mid;
    }
  }
  CacheSeq seq;
  if (!cache_seq(c, b, &seq) || seq.len < seq.n) return -1;  // (reported by check_batch)
  const int i = tok - seq.row0;
  if (i < 0 || i >= seq.n) return -1;  // behind the last sequence
  const int pos = seq.len - seq.n + i;
  const int page = c.block_table[(long long)b * c.table_width + (pos >> c.block_log2)];
  if (page < 0 || page >= c.num_blocks) {
    if (c.err) atomicCAS(c.err, 0u, site + 1);
    return -2;
  }
  return (((long long)page * c.H + h) << c.block_log2) + (pos & (c.block_size - 1));
}

__device__ __forceinline__ void check_batch(const CacheParams& c, long long first, long long step,
                                            uint32_t site) {
  for (long long b = first; b < c.B; b += step) {
    CacheSeq seq;
    if (!cache_seq(c, (int)b, &seq) || seq.len < seq.n)
      if (c.err) atomicCAS(c.err, 0u, site);
  }
}

// The side, head and first token of a warp's work.
struct Work {
  bool value;
  int h, tok0, count;
};
template <int D>
__device__ __forceinline__ bool find_work(const CacheParams& c, Work* w) {
  long long i = (long long)blockIdx.x * kWarps4 + (threadIdx.x >> 5);
  const int side_head = (int)(i % (2 * c.H));
  i /= 2 * c.H;
  w->value = side_head >= c.H;
  w->h = side_head - (w->value ? c.H : 0);
  if (i * Quad<D>::TOK >= c.total) return false;
  w->tok0 = (int)i * Quad<D>::TOK;
  w->count = min(Quad<D>::TOK, c.total - w->tok0);
  return true;
}

// bf16 pairs with NaN as zero and magnitudes beyond 57344 as that
__device__ __forceinline__ void tame(uint32_t (&x)[8], uint32_t* mx) {
  *mx = 0u;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    uint32_t lo = x[i] & 0x7fffu, hi = (x[i] >> 16) & 0x7fffu;
    lo = lo > 0x7f80u ? 0u : min(lo, 0x4760u);
    hi = hi > 0x7f80u ? 0u : min(hi, 0x4760u);
    x[i] = (x[i] & 0x80008000u) | lo | hi << 16;
    *mx = max(*mx, max(lo, hi));
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps4)
    cache4_append_kernel(const CacheParams c, const TokenView kv, const TokenView vv) {
  using Q = Quad<D>;
  check_batch(c, (long long)blockIdx.x * blockDim.x + threadIdx.x,
              (long long)gridDim.x * blockDim.x, ERR_SITE_CACHE_APPEND);
  Work w;
  if (!find_work<D>(c, &w)) return;
  const int lane = threadIdx.x & 31, group = lane % Q::LPR;
  const TokenView& from = w.value ? vv : kv;
  const uint16_t* src = from.p + (long long)w.tok0 * from.st + (long long)w.h * from.sh + group * 16;
  uint32_t x[kIter][8];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int r = j * Q::RPI + lane / Q::LPR;
    uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
    if (r < w.count) {
      const uint4* at = reinterpret_cast<const uint4*>(src + (long long)r * from.st);
      a = __ldg(at);
      b = __ldg(at + 1);
    }
    x[j][0] = a.x, x[j][1] = a.y, x[j][2] = a.z, x[j][3] = a.w;
    x[j][4] = b.x, x[j][5] = b.y, x[j][6] = b.z, x[j][7] = b.w;
  }
  const long long place = place_of(c, w.h, w.tok0, w.count, ERR_SITE_CACHE_APPEND);
  uint8_t* codes = w.value ? c.v : c.k;
  uint8_t* scales = w.value ? c.v_scale4 : c.k_scale4;
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const long long at = __shfl_sync(0xffffffffu, place, j * Q::RPI + lane / Q::LPR);
    uint32_t m2 = 0u, s2 = 0x80008000u;  // largest magnitudes; largest values
#pragma unroll
    for (int i = 0; i < 8; ++i) m2 = __vmaxu2(m2, x[j][i] & 0x7fff7fffu);
    uint32_t mx = max(m2 & 0xffffu, m2 >> 16);
    if (mx > 0x4760u) tame(x[j], &mx);
#pragma unroll
    for (int i = 0; i < 8; ++i) s2 = __vmaxs2(s2, x[j][i]);
    const int top = max((int)(short)(s2 & 0xffffu), (int)(short)(s2 >> 16));
    const float a = __uint_as_float(mx << 16) * 0.125f;
    const float signed_a = top == (int)mx ? -a : a;
    const uint32_t s8 = f32_to_codes<true>(signed_a, 0.f) & 0xffu;
    // the scale's value: the upper byte of an fp16
    const float s = f16x2_to_f32(s8 << 8).x;
    const float inv = s == 0.f ? 0.f : __frcp_rn(s);
    uint32_t word[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      uint32_t bytes[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t v = x[j][k * 4 + i];
        uint32_t h, r;
        asm("cvt.rn.f16x2.f32 %0, %1, %2;"
            : "=r"(h)
            : "f"(__uint_as_float(v & 0xffff0000u) * inv), "f"(__uint_as_float(v << 16) * inv));
        asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(h), "r"(0x66086608u));  // 1544
        asm("max.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x66006600u));              // 1536
        asm("min.f16x2 %0, %0, %1;" : "+r"(r) : "r"(0x660f660fu));              // 1551
        bytes[i] = (r & 0xfu) | ((r >> 12) & 0xf0u);
      }
      word[k] = bytes[0] | bytes[1] << 8 | bytes[2] << 16 | bytes[3] << 24;
    }
    if (at >= 0) {
      *reinterpret_cast<uint2*>(codes + at * (D / 2) + group * 8) = make_uint2(word[0], word[1]);
      scales[at * (D / 16) + group] = (uint8_t)s8;
    }
  }
}

template <int D>
__global__ void __launch_bounds__(32 * kWarps4)
    cache4_read_kernel(const CacheParams c, const TokenView kv, const TokenView vv) {
  using Q = Quad<D>;
  check_batch(c, (long long)blockIdx.x * blockDim.x + threadIdx.x,
              (long long)gridDim.x * blockDim.x, ERR_SITE_CACHE_READ);
  Work w;
  if (!find_work<D>(c, &w)) return;
  const int lane = threadIdx.x & 31, group = lane % Q::LPR;
  const long long place = place_of(c, w.h, w.tok0, w.count, ERR_SITE_CACHE_READ);
  const uint8_t* codes = w.value ? c.v : c.k;
  const uint8_t* scales = w.value ? c.v_scale4 : c.k_scale4;
  long long at[kIter];
  uint2 x[kIter];
  uint32_t s8[kIter];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    at[j] = __shfl_sync(0xffffffffu, place, j * Q::RPI + lane / Q::LPR);
    x[j] = make_uint2(0x88888888u, 0x88888888u);
    s8[j] = 0u;  // a token without a block reads as zeros
    if (at[j] >= 0) {
      x[j] = __ldg(reinterpret_cast<const uint2*>(codes + at[j] * (D / 2) + group * 8));
      s8[j] = __ldg(scales + at[j] * (D / 16) + group);
    }
  }
  const TokenView& to = w.value ? vv : kv;
  uint16_t* dst = to.p + (long long)w.tok0 * to.st + (long long)w.h * to.sh + group * 16;
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    const int r = j * Q::RPI + lane / Q::LPR;
    if (at[j] == -1) continue;
    const float s = f16x2_to_f32(s8[j] << 8).x;
    uint32_t o[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const uint32_t b = (i < 4 ? x[j].x : x[j].y) >> (8 * (i & 3));
      o[i] = pack_bf16x2((float)((int)(b & 15u) - 8) * s, (float)((int)((b >> 4) & 15u) - 8) * s);
    }
    uint4* out = reinterpret_cast<uint4*>(dst + (long long)r * to.st);
    out[0] = make_uint4(o[0], o[1], o[2], o[3]);
    out[1] = make_uint4(o[4], o[5], o[6], o[7]);
  }
}

template <bool APPEND, int D>
cudaError_t start(const CacheParams& c, const TokenView& k, const TokenView& v,
                  cudaStream_t stream) {
  const long long warps = ((long long)c.total + Quad<D>::TOK - 1) / Quad<D>::TOK * 2 * c.H;
  const long long ctas = (warps + kWarps4 - 1) / kWarps4;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if constexpr (APPEND)
    cache4_append_kernel<D><<<(unsigned)ctas, 32 * kWarps4, 0, stream>>>(c, k, v);
  else
    cache4_read_kernel<D><<<(unsigned)ctas, 32 * kWarps4, 0, stream>>>(c, k, v);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache4_append(const CacheParams& c, const TokenView& k, const TokenView& v,
                                 cudaStream_t stream) {
  return c.d == 128 ? start<true, 128>(c, k, v, stream) : start<true, 64>(c, k, v, stream);
}

cudaError_t launch_cache4_read(const CacheParams& c, const TokenView& k, const TokenView& v,
                               cudaStream_t stream) {
  return c.d == 128 ? start<false, 128>(c, k, v, stream) : start<false, 64>(c, k, v, stream);
}

}  // namespace fattn

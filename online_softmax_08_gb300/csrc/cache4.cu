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
// The bound is memory, and next to it the logic pipe, which the quantising of a group takes
// 68 % of while it is written (measured: 32768 tokens of 16 heads, d = 128, 58.3 us written, 55.1
// read back, 87 and 92 % of the measured copy bandwidth).
// A thread holds one group: 32 bytes of bf16 and 8 + 1 of the cache.
// A warp takes kIter x 32 groups of one head: the rows of 16 (d = 64: 32) packed tokens one
// behind another, so a prompt's codes and scales are written as whole lines, then the same of
// its further heads, for which the tokens' places need not be looked up again.  The first
// values are on their way while they are.  Bad entries of the batch are looked for by the
// first warps, so that one without tokens is found as well.
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

// Row of packed token `tok` of head 0 in the pool, block * H * block_size + row; -1: no such
// token, -2: a token without a place.  Called by whole warps for tok0 + lane.
__device__ __forceinline__ long long place_of(const CacheParams& c, int tok0, int count,
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
  return (((long long)page * c.H) << c.block_log2) + (pos & (c.block_size - 1));
}

__device__ __forceinline__ void check_batch(const CacheParams& c, long long first, long long step,
                                            uint32_t site) {
  for (long long b = first; b < c.B; b += step) {
    CacheSeq seq;
    if (!cache_seq(c, (int)b, &seq) || seq.len < seq.n)
      if (c.err) atomicCAS(c.err, 0u, site);
  }
}

// A warp's work: the side, `heads` heads from h on, and the tokens.
struct Work {
  bool value;
  int h, h_end, tok0, count;
};
template <int D>
__device__ __forceinline__ bool find_work(const CacheParams& c, int heads, Work* w) {
  w->value = blockIdx.z != 0;
  w->h = ((int)blockIdx.y * kWarps4 + (int)(threadIdx.x >> 5)) * heads;
  w->h_end = min(c.H, w->h + heads);
  w->tok0 = (int)blockIdx.x * Quad<D>::TOK;
  w->count = min(Quad<D>::TOK, c.total - w->tok0);
  return w->h < c.H;
}
__device__ __forceinline__ void check_entries(const CacheParams& c, uint32_t site) {
  if (blockIdx.y == 0 && blockIdx.z == 0)
    check_batch(c, (long long)blockIdx.x * blockDim.x + threadIdx.x,
                (long long)gridDim.x * blockDim.x, site);
}

// 32 bytes, in one store (V8: 32-byte aligned) or two, each of which leaves half of every
// sector to the other (reading back the prompt above: 57 us and 61).
template <bool V8>
__device__ __forceinline__ void store32(uint16_t* p, const uint32_t (&x)[8]) {
  if constexpr (V8) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(p), "r"(x[0]),
                 "r"(x[1]), "r"(x[2]), "r"(x[3]), "r"(x[4]), "r"(x[5]), "r"(x[6]), "r"(x[7])
                 : "memory");
  } else {
    uint4* to = reinterpret_cast<uint4*>(p);
    to[0] = make_uint4(x[0], x[1], x[2], x[3]);
    to[1] = make_uint4(x[4], x[5], x[6], x[7]);
  }
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
    cache4_append_kernel(const CacheParams c, const TokenView kv, const TokenView vv, int heads) {
  using Q = Quad<D>;
  check_entries(c, ERR_SITE_CACHE_APPEND);
  Work w;
  if (!find_work<D>(c, heads, &w)) return;
  const int lane = threadIdx.x & 31, group = lane % Q::LPR;
  const TokenView& from = w.value ? vv : kv;
  const uint16_t* src = from.p + (long long)(w.tok0 + lane / Q::LPR) * from.st +
                        (long long)w.h * from.sh + group * 16;
  const long long step = Q::RPI * from.st;
  uint32_t x[kIter][8];
  auto load = [&]() {
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
      uint4 a = make_uint4(0u, 0u, 0u, 0u), b = a;
      if (j * Q::RPI + lane / Q::LPR < w.count) {
        const uint4* at = reinterpret_cast<const uint4*>(src + j * step);
        a = __ldg(at);
        b = __ldg(at + 1);
      }
      x[j][0] = a.x, x[j][1] = a.y, x[j][2] = a.z, x[j][3] = a.w;
      x[j][4] = b.x, x[j][5] = b.y, x[j][6] = b.z, x[j][7] = b.w;
    }
  };
  load();
  const long long place = place_of(c, w.tok0, w.count, ERR_SITE_CACHE_APPEND);
  uint8_t* codes = w.value ? c.v : c.k;
  uint8_t* scales = w.value ? c.v_scale4() : c.k_scale4();
  long long places[kIter];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    places[j] = __shfl_sync(0xffffffffu, place, j * Q::RPI + lane / Q::LPR);
    if (places[j] >= 0) places[j] += (long long)w.h << c.block_log2;
  }
  for (int h = w.h;;) {
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
      const long long at = places[j];
      if (at >= 0) places[j] += c.block_size;  // the next head's
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
        uint32_t r[4];  // 0x6600 + code in each half
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t v = x[j][k * 4 + i];
          uint32_t h;
          asm("cvt.rn.f16x2.f32 %0, %1, %2;"
              : "=r"(h)
              : "f"(__uint_as_float(v & 0xffff0000u) * inv), "f"(__uint_as_float(v << 16) * inv));
          asm("add.rn.f16x2 %0, %1, %2;" : "=r"(r[i]) : "r"(h), "r"(0x66086608u));  // 1544
          asm("max.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(0x66006600u));             // 1536
          asm("min.f16x2 %0, %0, %1;" : "+r"(r[i]) : "r"(0x660f660fu));             // 1551
        }
        // Codes 2 i and 2 i + 1 are the halves of r[i] and go to the nibbles of byte i.  Added up
        // with what the 0x6600 leave (no half overflows), which is taken off at the end.
        const uint32_t s01 = r[1] * 256u + r[0], s23 = r[3] * 256u + r[2];
        const uint32_t even = __byte_perm(s01, s23, 0x5410u), odd = __byte_perm(s01, s23, 0x7632u);
        word[k] = odd * 16u + even - (0x66666666u * 16u + 0x66006600u);
      }
      if (at >= 0) {
        *reinterpret_cast<uint2*>(codes + at * (D / 2) + group * 8) = make_uint2(word[0], word[1]);
        scales[at * (D / 16) + group] = (uint8_t)s8;
      }
    }
    if (++h >= w.h_end) break;
    src += from.sh;
    load();
  }
}

template <int D, bool V8>
__global__ void __launch_bounds__(32 * kWarps4)
    cache4_read_kernel(const CacheParams c, const TokenView kv, const TokenView vv, int heads) {
  using Q = Quad<D>;
  check_entries(c, ERR_SITE_CACHE_READ);
  Work w;
  if (!find_work<D>(c, heads, &w)) return;
  const int lane = threadIdx.x & 31, group = lane % Q::LPR;
  const long long place = place_of(c, w.tok0, w.count, ERR_SITE_CACHE_READ);
  const uint8_t* codes = w.value ? c.v : c.k;
  const uint8_t* scales = w.value ? c.v_scale4() : c.k_scale4();
  const TokenView& to = w.value ? vv : kv;
  uint16_t* dst = to.p + (long long)(w.tok0 + lane / Q::LPR) * to.st + (long long)w.h * to.sh +
                  group * 16;
  const long long step = Q::RPI * to.st;
  long long at[kIter];
#pragma unroll
  for (int j = 0; j < kIter; ++j) {
    at[j] = __shfl_sync(0xffffffffu, place, j * Q::RPI + lane / Q::LPR);
    if (at[j] >= 0) at[j] += (long long)w.h << c.block_log2;
  }
  for (int h = w.h; h < w.h_end; ++h, dst += to.sh) {
    uint2 x[kIter];
    uint32_t s8[kIter];
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
      x[j] = make_uint2(0x88888888u, 0x88888888u);
      s8[j] = 0u;  // a token without a block reads as zeros
      if (at[j] >= 0) {
        x[j] = __ldg(reinterpret_cast<const uint2*>(codes + at[j] * (D / 2) + group * 8));
        s8[j] = __ldg(scales + at[j] * (D / 16) + group);
      }
    }
#pragma unroll
    for (int j = 0; j < kIter; ++j) {
      if (at[j] == -1) continue;
      if (at[j] >= 0) at[j] += c.block_size;  // the next head's
      uint32_t o[8];
      const bool infinite = (s8[j] & 0x7fu) == 0x7cu;  // (which the multiply-add makes NaN of)
      const Bf16Scale s = bf16_scale(infinite ? 0x3cu : s8[j]);  // 1
      bf16_values(x[j].x, s, o);
      bf16_values(x[j].y, s, o + 4);
      if (__builtin_expect(infinite, 0)) {
        const uint32_t inf = (s8[j] & 0x80u) ? 0xff80ff80u : 0x7f807f80u;
#pragma unroll
        for (int i = 0; i < 8; ++i) asm("mul.rn.bf16x2 %0, %0, %1;" : "+r"(o[i]) : "r"(inf));
      }
      store32<V8>(dst + j * step, o);
    }
  }
}

template <bool APPEND, int D>
cudaError_t start(const CacheParams& c, const TokenView& k, const TokenView& v,
                  cudaStream_t stream) {
  // Append: up to 4 heads a warp while there are 64 warps for every SM, which saves 43 of a
  // group's 218 instructions (32768 tokens of 16 heads, d = 128: 66 us with one, 60 with four).
  // Read, which waits for memory: one (57 us; 59 with four).
  const long long groups = ((long long)c.total + Quad<D>::TOK - 1) / Quad<D>::TOK;
  int heads = 1;
  while (APPEND && heads < 4 && groups * 2 * c.H / (2 * heads) >= 64LL * c.n_sm) heads *= 2;
  const int per_cta = kWarps4 * heads;
  const dim3 grid((unsigned)groups, (unsigned)((c.H + per_cta - 1) / per_cta), 2);
  const dim3 block(32 * kWarps4);
  if constexpr (APPEND) {
    cache4_append_kernel<D><<<grid, block, 0, stream>>>(c, k, v, heads);
  } else {
    const auto wide = [](const TokenView& x) {
      return (reinterpret_cast<uintptr_t>(x.p) & 31u) == 0 && (x.st & 15) == 0 && (x.sh & 15) == 0;
    };
    if (wide(k) && wide(v))
      cache4_read_kernel<D, true><<<grid, block, 0, stream>>>(c, k, v, heads);
    else
      cache4_read_kernel<D, false><<<grid, block, 0, stream>>>(c, k, v, heads);
  }
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

// cache.cuh -- what the host API and the kernels of the key/value cache share: launch
// parameters, the formats' conversions and the search for a packed token's sequence.
#pragma once
#include "common.cuh"
#include "ptx.cuh"

namespace fattn {

// Codes of the device error word (see common.cuh).
enum : uint32_t {
  ERR_SITE_CACHE_APPEND = 0x440,  // + 0: bad sequence entry, + 1: bad block number
  ERR_SITE_CACHE_READ = 0x450,
  ERR_SITE_CACHE_FWD = 0x460,
};

// Division of 0 <= n < 2^31 by a fixed d >= 1 as a multiplication (Granlund and
// Montgomery, "Division by invariant integers using multiplication"):
// q = (n + floor(n mul / 2^32)) >> shift with 2^(shift - 1) < d <= 2^shift and
// mul = floor(2^32 (2^shift - d) / d) + 1.
struct FastDiv {
  unsigned d, mul, shift;
  FastDiv() = default;
  explicit FastDiv(unsigned divisor) : d(divisor), shift(0) {
    while ((1ull << shift) < d) ++shift;
    mul = (unsigned)((((1ull << shift) - d) << 32) / d) + 1u;
  }
#ifdef __CUDACC__
  __device__ __forceinline__ int div(int n) const {
    return (int)((__umulhi((unsigned)n, mul) + (unsigned)n) >> shift);
  }
  __device__ __forceinline__ int mod(int n) const { return n - div(n) * (int)d; }
#endif
};

// CacheParams::format and the kernels' template argument
enum : int { FMT_E4M3 = 0, FMT_E5M2 = 1, FMT_INT4 = 2 };

// The key/value cache: the pool of blocks and the tokens a call works on
// (fattn_cache and fattn_cache_batch, with the device's error word).
struct CacheParams {
  uint8_t* k;            // [num_blocks, H, block_size, d] codes (4 bits: d / 2 bytes)
  uint8_t* v;
  float* k_scale;        // [num_blocks, H]
  float* v_scale;
  int num_blocks, H, block_size, d, format;
  int block_log2;        // block_size = 1 << block_log2
  const int* block_table;
  const int* lens;
  const int* cu_seqlens;
  int B, table_width, total, max_seqlen;
  long long l2_bytes;    // of the device (append)
  unsigned int* err;
  int n_sm;              // of the device (append and read in 4 bits)
  // 4 bits: the scales are bytes, e5m2, [num_blocks, H, block_size, d / 16]
#ifdef __CUDACC__
  __device__ __forceinline__ uint8_t* k_scale4() const { return reinterpret_cast<uint8_t*>(k_scale); }
  __device__ __forceinline__ uint8_t* v_scale4() const { return reinterpret_cast<uint8_t*>(v_scale); }
#endif
};
// A packed [total, heads, d] tensor by element strides.
struct TokenView {
  uint16_t* p;
  long long st, sh;  // token and head stride
};
struct CacheFwdParams {
  CacheParams c;
  TokenView q, o;
  float* lse;        // [Hq, total]
  int Hq;
  int G;             // Hq / H, the query heads of a key/value head
  FastDiv by_G;
  int causal;
  float scale_log2;  // scale * log2(e)
  int narrow_rows;   // sequences with more query rows per key/value head (tokens x grouped heads)
                     // than this go to the 256-row tcgen05 kernel, the others to the split one
  int wide_tokens;   // tokens per row block of the 256-row kernel: 256 / G
  int wide_ctas;     // CTAs of it that run at a time: one per SM
  int wide_grid;     // CTAs of it
  void* workspace;   // of the split kernel
  void* wide_workspace;
};

// What an attention kernel leaves for the merge: a unit that was cut into `parts`
// pieces (0: none), its rows, and (256-row kernel) the place of its first piece.  A
// workspace holds one record per CTA (256-row kernel: per SM), then LSE [n, 2, R] and
// O [n, 2, R, d] of the pieces, fp32.
struct Record {
  int parts, rows, h, row0, first_row, place;
};

// Sequence b of a cache call: n tokens at packed rows [row0, row0 + n), the
// last ones of len.  False (and the error word set by the caller) for entries
// out of range.
struct CacheSeq {
  int row0, n, len;
};
__device__ __forceinline__ bool cache_seq(const CacheParams& c, int a, int e, int len,
                                          CacheSeq* s) {
  s->row0 = a;
  s->n = e - a;
  s->len = len;
  return a >= 0 && e >= a && e <= c.total && e - a <= c.max_seqlen && len >= 0 &&
         (long long)len <= (long long)c.table_width * c.block_size;
}
__device__ __forceinline__ bool cache_seq(const CacheParams& c, int b, CacheSeq* s) {
  return cache_seq(c, c.cu_seqlens[b], c.cu_seqlens[b + 1], c.lens[b], s);
}

// The cache in 8 bits and in 4: append, read back, attention over it.
cudaError_t launch_cache_append(const CacheParams& c, const TokenView& k, const TokenView& v,
                                cudaStream_t stream);
cudaError_t launch_cache_read(const CacheParams& c, const TokenView& k, const TokenView& v,
                              cudaStream_t stream);
cudaError_t launch_cache4_append(const CacheParams& c, const TokenView& k, const TokenView& v,
                                 cudaStream_t stream);
cudaError_t launch_cache4_read(const CacheParams& c, const TokenView& k, const TokenView& v,
                               cudaStream_t stream);
size_t cache_fwd_workspace(const CacheParams& c, int G, int n_sm);
// tk, tv: maps of the codes, {d, block_size, num_blocks * H}, boxes of 16 tokens (8 bits)
cudaError_t launch_cache_fwd(const CUtensorMap& tk, const CUtensorMap& tv, const CacheFwdParams& p,
                             int n_sm, cudaStream_t stream);
int cache_fwd_wide_rows();  // rows per unit of the 256-row kernel
// CTAs that the 256-row kernel is launched with for the sequences of more than
// narrow_rows rows, and the bytes of their pieces' descriptors
long long cache_fwd_wide_grid(const CacheParams& c, int G, int narrow_rows, int n_sm);
size_t cache_fwd_wide_plan_bytes(long long grid);
cudaError_t launch_cache_fwd_wide(const CacheFwdParams& p, cudaStream_t stream);

// Two 8-bit codes (low byte first) -> two fp16 values (low half first), exact.
template <bool E5M2>
__device__ __forceinline__ uint32_t codes_to_f16x2(uint16_t c) {
  uint32_t r;
  if constexpr (E5M2)
    asm("cvt.rn.f16x2.e5m2x2 %0, %1;" : "=r"(r) : "h"(c));
  else
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(c));
  return r;
}
// Four codes (low byte first) -> two pairs of fp16 values.
template <bool E5M2>
__device__ __forceinline__ void codes4_to_f16(uint32_t w, uint32_t& lo, uint32_t& hi) {
  if constexpr (E5M2)  // the upper byte of the fp16 value
    lo = __byte_perm(w, 0u, 0x1404u), hi = __byte_perm(w, 0u, 0x3424u);
  else
    asm("{\n\t.reg .b16 a, b;\n\t"
        "mov.b32 {a, b}, %2;\n\t"
        "cvt.rn.f16x2.e4m3x2 %0, a;\n\t"
        "cvt.rn.f16x2.e4m3x2 %1, b;\n\t}"
        : "=r"(lo), "=r"(hi)
        : "r"(w));
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t h) {
  float2 f;
  asm("{\n\t.reg .b16 lo, hi;\n\t"
      "mov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\t"
      "cvt.f32.f16 %1, hi;\n\t}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(h));
  return f;
}
// Two fp32 values -> two codes (lo in the low byte), to nearest even; NaN stays NaN.
template <bool E5M2>
__device__ __forceinline__ uint16_t f32_to_codes(float lo, float hi) {
  uint16_t r;
  if constexpr (E5M2)
    asm("cvt.rn.satfinite.e5m2x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  else
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---- 4 bits.  The value of code c with the e5m2 scale s is (c - 8) s: at most 7
// significant bits, exact in fp16 (and bf16).  The kernels form it times 2^-7, in one
// fused multiply-add per pair of codes: a code put into the mantissa of 1024 (0x6400) is
// 1024 + c, one four bits higher into that of 64 (0x5400) is 64 + c, and
//   (1024 + c) s' - 1032 s' = (64 + c) s' - 72 s' = (c - 8) s',   s' = 2^-7 s,
// with every term exact: 1032 s' has 10 bits and stays below 2^16 for |s| <= 7168, the
// largest scale that is written, and the smallest, 2^-16, leaves s' = 2^-23.
// (An e2m1 code takes four logic instructions where this takes 1.25, and with an e4m3
// scale it misses normal values by 0.0090 of their variance, this by 0.0066.)
constexpr float kInt4Unit = 128.f;    // 2^7, which the results are multiplied by
constexpr int kInt4UnitLog2 = 7;
constexpr uint32_t kInt4MaxScale = 0x6fu;  // 7168 as e5m2
struct Int4Scale {
  uint32_t s, lo, hi;  // pairs of fp16: s', -1032 s', -72 s'
};
__device__ __forceinline__ uint32_t fma_f16x2(uint32_t a, uint32_t b, uint32_t c) {
  uint32_t r;
  asm("fma.rn.f16x2 %0, %1, %2, %3;" : "=r"(r) : "r"(a), "r"(b), "r"(c));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// of two e5m2 scales in the upper bytes of the halves (an e5m2 value is the upper byte of
// the fp16 one)
__device__ __forceinline__ Int4Scale int4_scale(uint32_t e5m2_hi) {
  Int4Scale r;
  r.s = mul_f16x2(e5m2_hi, 0x20002000u);     // 2^-7
  r.lo = mul_f16x2(r.s, 0xe408e408u);        // -1032
  r.hi = mul_f16x2(r.s, 0xd480d480u);        // -72
  return r;
}
// The two constants, in registers and opaque to the compiler, which would load them at every
// use (an instruction takes one immediate operand; and of (w & mask) | magic it makes two).
struct Int4Magic {
  uint32_t m1024, m64;
  __device__ __forceinline__ Int4Magic() {
    asm volatile("mov.b32 %0, 0x64006400;" : "=r"(m1024));
    asm volatile("mov.b32 %0, 0x54005400;" : "=r"(m64));
  }
};
// The lowest (N = 0) or the second code of each half of w, put into the mantissas of `magic`.
template <int N>
__device__ __forceinline__ uint32_t nibbles(uint32_t w, uint32_t magic) {
  uint32_t r;  // (a & b) | c
  asm("lop3.b32 %0, %1, %2, %3, 0xea;"
      : "=r"(r)
      : "r"(w), "n"(N ? 0x00f000f0 : 0x000f000f), "r"(magic));
  return r;
}
// Eight codes, four in each half of w -> (c_i, c_i+4) of i = 0 ... 3 as pairs of fp16.
__device__ __forceinline__ void int4_values(uint32_t w, const Int4Scale& s, const Int4Magic& m,
                                            uint32_t (&o)[4]) {
  const uint32_t u = w >> 8;
  o[0] = fma_f16x2(nibbles<0>(w, m.m1024), s.s, s.lo);
  o[1] = fma_f16x2(nibbles<1>(w, m.m64), s.s, s.hi);
  o[2] = fma_f16x2(nibbles<0>(u, m.m1024), s.s, s.lo);
  o[3] = fma_f16x2(nibbles<1>(u, m.m64), s.s, s.hi);
}
// The same in bf16, eight codes of one scale in their order: a code in the mantissa of 128
// (0x4300) is 128 + c, and (128 + c) s - 136 s = (c - 8) s, every term exact for any finite scale.
struct Bf16Scale {
  uint32_t s, off;  // pairs: s, -136 s
};
__device__ __forceinline__ Bf16Scale bf16_scale(uint32_t e5m2) {
  const float s = f16x2_to_f32(e5m2 << 8).x;
  return Bf16Scale{pack_bf16x2(s, s), pack_bf16x2(-136.f * s, -136.f * s)};
}
__device__ __forceinline__ void bf16_values(uint32_t w, const Bf16Scale& s, uint32_t* o) {
  uint32_t v[4];  // (c_i, c_i+4)
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    asm("lop3.b32 %0, %1, %2, %3, 0xea;"  // (a & b) | c
        : "=r"(v[i])
        : "r"(w >> (4 * i)), "n"(0x000f000f), "r"(0x43004300u));
    asm("fma.rn.bf16x2 %0, %0, %1, %2;" : "+r"(v[i]) : "r"(s.s), "r"(s.off));
  }
  o[0] = __byte_perm(v[0], v[1], 0x5410u), o[1] = __byte_perm(v[2], v[3], 0x5410u);
  o[2] = __byte_perm(v[0], v[1], 0x7632u), o[3] = __byte_perm(v[2], v[3], 0x7632u);
}
// The scales of a word that append never writes (above 7168, infinite, NaN) as zeros.
__device__ __forceinline__ uint32_t int4_sane(uint32_t bytes) {
  const uint32_t m = ((bytes & 0x7f7f7f7fu) + (0x7fu - kInt4MaxScale) * 0x01010101u) & 0x80808080u;
  return bytes & ~(m | (m - (m >> 7)));
}

// 0x80 in the byte of each of four codes that stands for NaN (or, in e5m2, for
// infinity): the magnitudes from the first such code on carry into the sign bit.
template <bool E5M2>
__device__ __forceinline__ uint32_t nan_codes(uint32_t w) {
  return ((w & 0x7f7f7f7fu) + (E5M2 ? 0x04040404u : 0x01010101u)) & 0x80808080u;
}
// The four codes with zeros in the bytes that `m` (of nan_codes) marks.
__device__ __forceinline__ uint32_t clear_codes(uint32_t w, uint32_t m) {
  return w & ~(m | (m - (m >> 7)));
}

// The largest b in [0, B) with first(b) <= x, for a non-decreasing first() with
// first(0) <= x, found by the whole warp: 32 probes a step, so one step serves
// 32 sequences and two 1024 (a binary search would wait for 5 or 10 loads in
// turn).  Any values keep it inside [0, B).
template <typename First>
__device__ __forceinline__ int warp_search(int B, long long x, First first) {
  const int lane = threadIdx.x & 31;
  int lo = 0, hi = B;
  while (hi - lo > 1) {
    const int step = (hi - lo + 31) / 32;
    const int i = lo + lane * step;
    const unsigned yes = __ballot_sync(0xffffffffu, lane == 0 || (i < hi && first(i) <= x));
    const int last = yes == 0xffffffffu ? 31 : __ffs(~yes) - 2;  // the last probe that holds
    lo += last * step;
    hi = min(hi, lo + step);
  }
  return lo;
}

}  // namespace fattn

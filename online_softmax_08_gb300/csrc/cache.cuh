// cache.cuh -- what the host API and the kernels of the 8-bit key/value cache share:
// launch parameters, the 8-bit formats' conversions and the search for a packed
// token's sequence.
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

// The 8-bit key/value cache: the pool of blocks and the tokens a call works on
// (fattn_cache and fattn_cache_batch, with the device's error word).
struct CacheParams {
  uint8_t* k;            // [num_blocks, H, block_size, d] codes
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

// The 8-bit key/value cache (append, read back, attention over it).
cudaError_t launch_cache_append(const CacheParams& c, const TokenView& k, const TokenView& v,
                                cudaStream_t stream);
cudaError_t launch_cache_read(const CacheParams& c, const TokenView& k, const TokenView& v,
                              cudaStream_t stream);
size_t cache_fwd_workspace(const CacheParams& c, int G, int n_sm);
// tk, tv: maps of the codes, {d, block_size, num_blocks * H}, boxes of 16 tokens
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

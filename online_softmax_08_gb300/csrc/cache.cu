// cache.cu -- the 8-bit key/value cache: new tokens quantised into paged
// blocks, and tokens read back.
//
// A work item is one (block, head, key or value) that the call touches.  For
// sequence b with n tokens starting at position p, the blocks are p / bs ...
// (p + n - 1) / bs, at most n / bs + 2 of them, so item slots are laid out at
// cu_seqlens[b] / bs + 2 b: a flat grid of total / bs + 2 B slots holds every
// batch, however ragged, without the host knowing the lengths.  A slot's
// sequence is found by a search over cu_seqlens (warp_search).
//
// The quantisation of a block and head:
//   a = max |x| over the new tokens (finite values),
//   e = the smallest integer >= -100 with a <= MAX 2^e,   s = 2^e,
//   s = max(s, the block's scale) if it holds earlier tokens of the sequence,
//   code = rn8(x / s);  earlier codes become rn8(code * s_old / s) if s grew.
// A power of two costs a floating code no precision (its relative step does not
// depend on the scale), makes x / s and the growth of a block's scale exact,
// and lets the values be read back exactly as bf16.
//
// Memory-bound: the item's values stay in registers (64 per lane) between the
// maximum and the conversion, so every value is read once and written once.  Measured
// (d = 128): 32768 tokens of 16 heads written in 62.8 us, 95 % of the measured copy
// bandwidth; 16 sequences of 512 to 8192 tokens of 16 heads read back in 86 us, 97 %;
// one token of each of 256 sequences, 8 heads, 7 us, which is the search for the
// sequence, its block and its values one after the other.
#include "cache.cuh"

namespace fattn {
namespace {

constexpr int kMinExp = -100;
constexpr int kPerWarp = 2048;  // values a warp holds: 64 per lane

// 2^e for the smallest e >= kMinExp with a <= MAX 2^e, MAX = 1.75 * 2^TOP.
template <bool E5M2>
__device__ __forceinline__ float scale_for(float a) {
  constexpr int TOP = E5M2 ? 15 : 8;
  const uint32_t u = __float_as_uint(a);
  int e = (int)(u >> 23) - 127 - TOP + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  e = max(e, kMinExp);  // zero and subnormal a come out below it
  return __uint_as_float((uint32_t)(e + 127) << 23);
}

struct Item {
  int b, h;
  bool value;      // the value side (else the key side)
  CacheSeq seq;
  int row;         // first row of the block that belongs to the call
  int count;       // rows
  int token;       // packed row of the first one
  int page;        // block number; -1: out of range
};

// Item `i` of the grid; false when it has no work.  Warp-uniform.
__device__ __forceinline__ bool find_item(const CacheParams& c, long long i, uint32_t site,
                                          Item* it) {
  const int bs = c.block_size;
  it->h = (int)(i % c.H);
  i /= c.H;
  it->value = (i & 1) != 0;
  const long long slot = i >> 1;
  it->b = warp_search(c.B, slot, [&](int b) { return (long long)(c.cu_seqlens[b] / bs) + 2LL * b; });
  const int j = (int)(slot - (c.cu_seqlens[it->b] / bs + 2LL * it->b));
  if (j < 0) return false;
  const bool first = (threadIdx.x & 31) == 0;
  if (!cache_seq(c, it->b, &it->seq) || it->seq.len < it->seq.n) {
    if (first && c.err) atomicCAS(c.err, 0u, site);
    return false;
  }
  const int start = it->seq.len - it->seq.n;
  const int blk = start / bs + j;
  if (it->seq.n == 0 || blk > (it->seq.len - 1) / bs) return false;
  const int lo = max(start, blk * bs), hi = min(it->seq.len, (blk + 1) * bs);
  it->row = lo - blk * bs;
  it->count = hi - lo;
  it->token = it->seq.row0 + (lo - start);
  it->page = c.block_table[(long long)it->b * c.table_width + blk];
  if (it->page < 0 || it->page >= c.num_blocks) {
    if (first && c.err) atomicCAS(c.err, 0u, site + 1);
    it->page = -1;
  }
  return true;
}

// W warps per item: a CTA of W > 1 warps is one item, a CTA of 8 one-warp items
// otherwise.
template <int W>
struct Team {
  static constexpr int THREADS = W == 1 ? 256 : 32 * W;
  static constexpr int ITEMS = W == 1 ? 8 : 1;
  static __device__ __forceinline__ long long item() {
    return W == 1 ? (long long)blockIdx.x * 8 + (threadIdx.x >> 5) : (long long)blockIdx.x;
  }
  static __device__ __forceinline__ int lane() { return W == 1 ? threadIdx.x & 31 : threadIdx.x; }
};

// STREAM: loads and stores that do not stay in the caches.
template <int D, bool E5M2, int W, bool STREAM>
__global__ void __launch_bounds__(Team<W>::THREADS)
    cache_append_kernel(const CacheParams c, const TokenView kv, const TokenView vv,
                        long long items) {
  const long long i = Team<W>::item();
  Item it;
  if (i >= items || !find_item(c, i, ERR_SITE_CACHE_APPEND, &it) || it.page < 0) return;
  constexpr int PER_ROW = D / 8;  // 16-byte pieces of a row
  constexpr int LANES = 32 * W;
  constexpr int N = kPerWarp / 8 / 32;  // pieces per lane
  const int lane = Team<W>::lane();
  const TokenView& x = it.value ? vv : kv;
  const uint16_t* src = x.p + (long long)it.token * x.st + it.h * x.sh;
  const long long block = (long long)it.page * c.H + it.h;
  uint8_t* codes = (it.value ? c.v : c.k) + block * c.block_size * D;
  float* scale = (it.value ? c.v_scale : c.k_scale) + block;
  const int pieces = it.count * PER_ROW;

  uint4 v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = lane + j * LANES;
    v[j] = make_uint4(0u, 0u, 0u, 0u);
    if (q < pieces) {
      const uint4* from = reinterpret_cast<const uint4*>(src + (long long)(q / PER_ROW) * x.st +
                                                         q % PER_ROW * 8);
      v[j] = STREAM ? __ldcs(from) : *from;
    }
  }
  // an earlier token of the sequence in the block: its scale counts
  const float old = it.row > 0 ? *scale : 0.f;

  // largest magnitude, as bf16 bits (ordered like the values), two at a time
  uint32_t mx = 0u;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu),
                               __vmaxu2(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu)));
  }
  mx = max(mx & 0xffffu, mx >> 16);
  mx = __reduce_max_sync(0xffffffffu, mx);
  __shared__ uint32_t red[2][W];
  if constexpr (W > 1) {
    if ((threadIdx.x & 31) == 0) red[0][threadIdx.x >> 5] = mx;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) mx = max(mx, red[0][w]);
  }
  if (mx >= 0x7f80u) {  // item-uniform, rare: NaN or infinities, which become NaN and do not count
    mx = 0u;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      uint32_t* w = &v[j].x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t lo = w[k] & 0x7fffu, hi = (w[k] >> 16) & 0x7fffu;
        if (lo >= 0x7f80u) w[k] |= 0x7fffu, lo = 0u;
        if (hi >= 0x7f80u) w[k] |= 0x7fff0000u, hi = 0u;
        mx = max(mx, max(lo, hi));
      }
    }
    mx = __reduce_max_sync(0xffffffffu, mx);
    if constexpr (W > 1) {
      if ((threadIdx.x & 31) == 0) red[1][threadIdx.x >> 5] = mx;
      __syncthreads();
#pragma unroll
      for (int w = 0; w < W; ++w) mx = max(mx, red[1][w]);
    }
  }
  const float s = fmaxf(scale_for<E5M2>(__uint_as_float(mx << 16)), old);
  const float inv = 1.f / s;  // exact: a power of two

  if (old > 0.f && s > old) {  // item-uniform: the earlier rows move to the larger scale
    const float f = old * inv;
    uint4* rows = reinterpret_cast<uint4*>(codes);
    for (int q = lane; q < it.row * (D / 16); q += LANES) {
      uint4 r = rows[q];
      uint32_t* w = &r.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 a = f16x2_to_f32(codes_to_f16x2<E5M2>((uint16_t)(w[k] & 0xffffu)));
        const float2 b = f16x2_to_f32(codes_to_f16x2<E5M2>((uint16_t)(w[k] >> 16)));
        w[k] = (uint32_t)f32_to_codes<E5M2>(a.x * f, a.y * f) |
               (uint32_t)f32_to_codes<E5M2>(b.x * f, b.y * f) << 16;
      }
      rows[q] = r;
    }
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = lane + j * LANES;
    if (q < pieces) {
      const uint32_t* w = &v[j].x;
      uint16_t r[4];
#pragma unroll
      for (int k = 0; k < 4; ++k)
        r[k] = f32_to_codes<E5M2>(__uint_as_float(w[k] << 16) * inv,
                                  __uint_as_float(w[k] & 0xffff0000u) * inv);
      uint2* to = reinterpret_cast<uint2*>(codes + (long long)it.row * D + q * 8);
      const uint2 c8 = make_uint2((uint32_t)r[0] | (uint32_t)r[1] << 16,
                                  (uint32_t)r[2] | (uint32_t)r[3] << 16);
      if (STREAM)
        __stcs(to, c8);
      else
        *to = c8;
    }
  }
  // every lane has read the old scale by now (W > 1: the barrier above)
  __syncwarp();
  if (lane == 0) *scale = s;
}

template <int D, bool E5M2, int W>
__global__ void __launch_bounds__(Team<W>::THREADS)
    cache_read_kernel(const CacheParams c, const TokenView kv, const TokenView vv,
                      long long items) {
  const long long i = Team<W>::item();
  Item it;
  if (i >= items || !find_item(c, i, ERR_SITE_CACHE_READ, &it)) return;
  constexpr int PER_ROW = D / 8;  // 8 codes a piece
  constexpr int LANES = 32 * W;
  constexpr int N = kPerWarp / 8 / 32;
  const int lane = Team<W>::lane();
  const TokenView& x = it.value ? vv : kv;
  uint16_t* dst = x.p + (long long)it.token * x.st + it.h * x.sh;
  const bool ok = it.page >= 0;
  const long long block = (long long)(ok ? it.page : 0) * c.H + it.h;
  const uint8_t* codes = (it.value ? c.v : c.k) + (block * c.block_size + it.row) * D;
  const float s = (it.value ? c.v_scale : c.k_scale)[block];
  const int pieces = it.count * PER_ROW;
  uint2 v[N];
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = lane + j * LANES;
    v[j] = make_uint2(0u, 0u);
    if (ok && q < pieces) v[j] = *reinterpret_cast<const uint2*>(codes + q * 8);
  }
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int q = lane + j * LANES;
    if (q < pieces) {
      const uint32_t w[2] = {v[j].x, v[j].y};
      uint4 r;
      uint32_t* out = &r.x;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f =
            f16x2_to_f32(codes_to_f16x2<E5M2>((uint16_t)(w[k >> 1] >> (16 * (k & 1)))));
        out[k] = ok ? pack_bf16x2(f.x * s, f.y * s) : 0u;
      }
      *reinterpret_cast<uint4*>(dst + (long long)(q / PER_ROW) * x.st + q % PER_ROW * 8) = r;
    }
  }
}

// Launch of one of the two kernels with the warps per item that its largest
// item needs: a block's worth of tokens, or all of a sequence's new ones.
template <bool APPEND, int D, bool E5M2, int W>
cudaError_t start(const CacheParams& c, const TokenView& k, const TokenView& v, long long items,
                  cudaStream_t stream) {
  const long long ctas = (items + Team<W>::ITEMS - 1) / Team<W>::ITEMS;
  if (ctas > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  if constexpr (APPEND) {
    // Codes that fit in half of L2 are left there for the attention that follows.  More
    // than that would not survive: then nothing is kept, 62.3 us against 64.6 us for
    // 32768 tokens of 16 heads, d = 128 (one token of each of 256 sequences: 6.9 us
    // against 6.6 us).
    if (2LL * c.total * c.H * D > c.l2_bytes / 2) {
      cache_append_kernel<D, E5M2, W, true>
          <<<(unsigned)ctas, Team<W>::THREADS, 0, stream>>>(c, k, v, items);
      return cudaGetLastError();
    }
    cache_append_kernel<D, E5M2, W, false>
        <<<(unsigned)ctas, Team<W>::THREADS, 0, stream>>>(c, k, v, items);
  } else
    cache_read_kernel<D, E5M2, W><<<(unsigned)ctas, Team<W>::THREADS, 0, stream>>>(c, k, v, items);
  return cudaGetLastError();
}

template <bool APPEND, int D, bool E5M2>
cudaError_t start_sized(const CacheParams& c, const TokenView& k, const TokenView& v,
                        cudaStream_t stream) {
  const long long slots = c.total / c.block_size + 2LL * c.B;
  const long long items = slots * 2 * c.H;
  const int values = (c.max_seqlen < c.block_size ? c.max_seqlen : c.block_size) * D;
  if (values <= kPerWarp) return start<APPEND, D, E5M2, 1>(c, k, v, items, stream);
  if (values <= 2 * kPerWarp) return start<APPEND, D, E5M2, 2>(c, k, v, items, stream);
  if (values <= 4 * kPerWarp) return start<APPEND, D, E5M2, 4>(c, k, v, items, stream);
  return start<APPEND, D, E5M2, 8>(c, k, v, items, stream);
}

template <bool APPEND>
cudaError_t move(const CacheParams& c, const TokenView& k, const TokenView& v,
                 cudaStream_t stream) {
  if (c.d == 128)
    return c.format ? start_sized<APPEND, 128, true>(c, k, v, stream)
                    : start_sized<APPEND, 128, false>(c, k, v, stream);
  return c.format ? start_sized<APPEND, 64, true>(c, k, v, stream)
                  : start_sized<APPEND, 64, false>(c, k, v, stream);
}

}  // namespace

cudaError_t launch_cache_append(const CacheParams& c, const TokenView& k, const TokenView& v,
                                cudaStream_t stream) {
  return move<true>(c, k, v, stream);
}

cudaError_t launch_cache_read(const CacheParams& c, const TokenView& k, const TokenView& v,
                              cudaStream_t stream) {
  return move<false>(c, k, v, stream);
}

}  // namespace fattn

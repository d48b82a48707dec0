// cache_evict.cu -- the copy of a cache's most attended tokens into other blocks.
//
// Of a sequence of L > keep tokens every key/value head keeps its last `recent` tokens and,
// among the others, the keep - recent of the largest weight (NaN counts as the largest, of
// equal ones the first); their order stays.  Shorter sequences are copied whole.
//
// 1. Selection, a cluster of CTAs per (sequence, head).  Weights are taken as unsigned numbers of the
// same order.  The smallest kept one is found digit by digit, 11 + 11 + 10 bits from the top:
// a histogram in shared memory of the next digit among the weights that agree so far, and the
// bin in which the count from above reaches what is to be kept.  A last pass in the tokens'
// order numbers the kept ones.  The CTAs of a cluster add up their histograms and counts
// through distributed shared memory; one warp of each looks for the bin, in 32 groups of 64
// bins, then in one of them.  A thread keeps its weights in shared memory, up to 32768 in a CTA
// (longer rows are read anew by every pass); registers in place of it need every loop unrolled,
// code that runs once and takes longer to fetch than to execute (16384 weights, 8 CTAs: 19.3
// against 16.9 us for a call and the kept tokens read back).  What bounds it is the chain of
// passes: 8 x 8 rows of up to 32768 weights take 19 us with two CTAs a row (all weights in
// registers and all bins added up by every thread 22, with one CTA a row 31, every pass reading
// the weights anew, a thread one at a time, 54; four places for every bin of the first digit, so
// that fewer lanes meet at one, made no difference).
// 2. Copy.  The destination blocks are nobody's source, so every one is filled on its own: a
// CTA per (sequence, head, block).  In 4 bits a token's codes and scales move as they are; in
// 8 bits the block's scale is the largest of its tokens', and codes of a smaller one are
// rounded for it, as when append raises a block's scale.  8192 tokens of 8 x 8 rows, e4m3, d = 128:
// 46 us, 90 % of the measured copy bandwidth; the whole 63.5 us (one piece at a time instead of
// four on their way 66.0, eight 64.3).
#include <cooperative_groups.h>

#include <algorithm>
#include <type_traits>

#include "evict.cuh"

namespace fattn {
namespace {

constexpr int kSelect = 1024;  // threads of a selection
constexpr int kBins = 2048;
constexpr int kRun = 32;       // weights that a thread of it holds at a time
constexpr uint32_t kZero = 0x80000000u;  // a weight of zero, as an ordered number
constexpr int kCopy = 128;     // threads of a copy
constexpr int kAhead = 4;      // 16-byte pieces that each has on their way

__device__ __forceinline__ uint32_t order_of(float w) {
  const uint32_t u = __float_as_uint(w + 0.f);  // -0 as 0
  if ((u & 0x7fffffffu) > 0x7f800000u) return 0xffffffffu;
  return u ^ ((u >> 31) ? 0xffffffffu : 0x80000000u);
}

// Length of sequence b, or -1 (reported).
__device__ __forceinline__ int length_of(const EvictParams& p, int b) {
  const int len = p.c.lens[b];
  if (len < 0 || len > p.width || (long long)len > (long long)p.c.table_width * p.c.block_size) {
    if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_EVICT);
    return -1;
  }
  return len;
}

__device__ __forceinline__ float weight_of(uint32_t u) {  // any NaN, -0 as 0
  return __uint_as_float(u == 0xffffffffu ? 0x7fffffffu : u ^ ((u >> 31) ? 0x80000000u : 0xffffffffu));
}

// Sum of v over this lane and those before it.
__device__ __forceinline__ int sum_upto(int v) {
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const int o = __shfl_up_sync(0xffffffffu, v, w);
    if ((int)(threadIdx.x & 31) >= w) v += o;
  }
  return v;
}

// CS: CTAs of a cluster.
template <int CS>
__global__ void __launch_bounds__(kSelect) cache_select_kernel(const EvictParams p) {
  namespace cg = cooperative_groups;
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  __shared__ alignas(8) int hist[2][kBins];  // by turns: a neighbour may still read the last one
  __shared__ int groups[2][32];   // of 64 bins
  __shared__ int found_bin, found_above;
  // Of a segment's weights in a warp, in the CTA (at most 2^15): those larger than the smallest
  // kept one, times 2^16, and those equal to it
  __shared__ unsigned part[2][32], counts[2];
  const int unit = blockIdx.x / CS, rank = blockIdx.x % CS;
  const int b = unit / p.c.H, h = unit % p.c.H;
  const int t = threadIdx.x + rank * kSelect;  // of the cluster's threads
  constexpr int T = CS * kSelect;
  int* kept = p.kept + (long long)unit * p.keep;
  auto cluster_sync = [] {
    if constexpr (CS > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  auto of_rank = [](auto* x, int r) {
    if constexpr (CS > 1)
      return cg::this_cluster().map_shared_rank(x, r);
    else
      return x;
  };
  const int len = length_of(p, b);
  const int n = max(0, min(len, p.keep));
  if (h == 0 && t == 0) p.lens_out[b] = n;
  const float* w = p.in.p + b * p.in.sb + h * p.in.sh;
  float* w_out = p.out.p + b * p.out.sb + h * p.out.sh;
  // (unsigned: keep may be 2^31 - 1, and the last step goes past it)
  for (unsigned j = (unsigned)(n + t); j < (unsigned)p.keep; j += T) kept[j] = -1;
  if (len <= p.keep) {
    for (int j = t; j < n; j += T) {
      kept[j] = j;
      w_out[j] = w[j];
    }
    return;
  }
  const int old = len - p.recent;        // those that compete
  const int top = p.keep - p.recent;     // for so many places
  // A warp holds a run of `steps` x 32 neighbouring weights of a segment (kRun x kSelect of them;
  // a sequence that is no longer than that is read once), so the kept ones are numbered by
  // ballots, and the warps' totals by one sum over those before a segment.
  const int warp = t >> 5, lane = t & 31, cta_warp = threadIdx.x >> 5;
  const int steps = min(kRun, (old + T - 1) / T), segment = steps * T;
  extern __shared__ uint32_t held[];  // [kRun * kSelect], every thread its own
  uint32_t* const own = held + cta_warp * steps * 32 + lane;
  // (a place in a segment is compared with what is left from its start on: the number of the
  // weight behind a segment may pass 32 bits)
  auto index = [&](int i) { return (warp * steps + i) * 32 + lane; };
  auto load = [&](int seg) {
    const int left = old - seg;
    constexpr int N = 16;  // on their way at a time
#pragma unroll 1
    for (int i0 = 0; i0 < steps; i0 += N) {
      float x[N];
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const int j = index(i0 + i);
        x[i] = i0 + i < steps && j < left ? w[seg + j] : 0.f;
      }
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (i0 + i < steps) own[(i0 + i) * 32] = order_of(x[i]);
    }
  };
  if (top > 0) load(0);
  for (int j = t; j < p.recent; j += T) {  // (behind the loads of the others)
    kept[top + j] = old + j;
    w_out[top + j] = w[old + j];
  }
  if (top == 0) return;

  // ---------------------------------------------------------------- the smallest kept weight
  uint32_t prefix = 0u, mask = 0u;  // the digits found
  int need = top;                   // places for the weights that agree with them
#pragma unroll 1
  for (int digit = 0; digit < 3; ++digit) {
    const int shift = digit == 0 ? 21 : digit == 1 ? 10 : 0;
    const uint32_t low = digit == 2 ? 0x3ffu : 0x7ffu;
    int* bins = hist[digit & 1];
    for (int i = threadIdx.x; i < kBins; i += kSelect) bins[i] = 0;
    __syncthreads();
    int zeros = 0;  // many weights are zero, and would all add to one bin: counted apart
#pragma unroll 1
    for (int seg = 0;; seg += segment) {
      const int left = old - seg;
      if (old > segment) load(seg);
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        const uint32_t u = own[i * 32];
        const bool on = index(i) < left && (u & mask) == prefix, zero = u == kZero;
        zeros += on && zero;
        if (on && !zero) atomicAdd(&bins[u >> shift & low], 1);
      }
      if (left <= segment) break;
    }
    zeros = __reduce_add_sync(0xffffffffu, zeros);
    if (lane == 0 && zeros > 0) atomicAdd(&bins[kZero >> shift & low], zeros);
    __syncthreads();
    const int2 two = *reinterpret_cast<const int2*>(bins + 2 * threadIdx.x);
    const int group_sum = __reduce_add_sync(0xffffffffu, two.x + two.y);
    if (lane == 0) groups[digit & 1][cta_warp] = group_sum;
    cluster_sync();
    // From the top: the group of 64 bins, a lane each, then its bins, two a lane.  One warp looks
    // (all of them at all bins of 8 CTAs took 5000 clocks a digit, this takes 1300).
    if (cta_warp == 0) {
      int x = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) x += of_rank(groups[digit & 1], r)[31 - lane];
      int upto = sum_upto(x);
      const unsigned enough = __ballot_sync(0xffffffffu, upto >= need);
      const int hit = enough ? __ffs(enough) - 1 : 31;
      const int above_group = __shfl_sync(0xffffffffu, upto - x, hit);
      const int top_bin = (31 - hit) * 64 + 63 - 2 * lane;
      int h0 = 0, h1 = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        const int2 y = *reinterpret_cast<const int2*>(of_rank(bins, r) + top_bin - 1);
        h0 += y.y, h1 += y.x;
      }
      upto = sum_upto(h0 + h1);
      const int above = above_group + upto - h0 - h1;
      if (above < need && above + h0 >= need) found_bin = top_bin, found_above = above;
      if (above + h0 < need && above + h0 + h1 >= need)
        found_bin = top_bin - 1, found_above = above + h0;
    }
    __syncthreads();
    prefix |= (uint32_t)found_bin << shift;
    mask |= low << shift;
    need -= found_above;
  }

  // ---------------------------------------------------------------- the kept ones, in order
  int more0 = 0, ties0 = 0;  // in the segments before: larger than the smallest kept, equal to it
#pragma unroll 1
  for (int seg = 0, turn = 0;; seg += segment, turn ^= 1) {
    const int left = old - seg;
    if (old > segment) load(seg);
    int more = 0, ties = 0;  // of the lane, then of the warp
#pragma unroll 4
    for (int i = 0; i < steps; ++i) {
      const uint32_t u = own[i * 32];
      const bool in = index(i) < left;
      more += in && u > prefix;
      ties += in && u == prefix;
    }
    more = __reduce_add_sync(0xffffffffu, more);
    ties = __reduce_add_sync(0xffffffffu, ties);
    const bool any_ties = ties > 0;
    if (lane == 0) part[turn][cta_warp] = (unsigned)more << 16 | (unsigned)ties;
    __syncthreads();
    const unsigned of_warp = part[turn][lane];
    const unsigned all = __reduce_add_sync(0xffffffffu, of_warp);
    const unsigned front = __reduce_add_sync(0xffffffffu, lane < cta_warp ? of_warp : 0u);
    more = more0 + (int)(front >> 16), ties = ties0 + (int)(front & 0xffffu);
    int all_more = (int)(all >> 16), all_ties = (int)(all & 0xffffu);
    if constexpr (CS > 1) {  // and of the CTAs in front
      if (threadIdx.x == 0) counts[turn] = all;
      cluster_sync();
      all_more = all_ties = 0;
#pragma unroll
      for (int r = 0; r < CS; ++r) {
        const unsigned x = *of_rank(&counts[turn], r);
        const int m = (int)(x >> 16), e = (int)(x & 0xffffu);
        if (r < rank) more += m, ties += e;
        all_more += m, all_ties += e;
      }
    }
    // (places are below `top` unless the weights change meanwhile, which must not harm others)
    const unsigned before = (1u << lane) - 1u;
    if (!any_ties) {  // nearly always
      int at = more + min(ties, need);
#pragma unroll 4
      for (int i = 0; i < steps; ++i) {
        const uint32_t u = own[i * 32];
        const bool mine = index(i) < left && u > prefix;
        const unsigned m = __ballot_sync(0xffffffffu, mine);
        const int place = at + __popc(m & before);
        if (mine && (unsigned)place < (unsigned)top) {
          kept[place] = seg + index(i);
          w_out[place] = weight_of(u);
        }
        at += __popc(m);
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < steps; ++i) {
        const uint32_t u = own[i * 32];
        const bool in = index(i) < left;
        const unsigned m = __ballot_sync(0xffffffffu, in && u > prefix);
        const unsigned e = __ballot_sync(0xffffffffu, in && u == prefix);
        const int ties_here = ties + __popc(e & before);
        const int place = more + __popc(m & before) + min(ties_here, need);
        if (((m >> lane & 1u) || ((e >> lane & 1u) && ties_here < need)) &&
            (unsigned)place < (unsigned)top) {
          kept[place] = seg + index(i);
          w_out[place] = weight_of(u);
        }
        more += __popc(m), ties += __popc(e);
      }
    }
    more0 += all_more, ties0 += all_ties;
    if (left <= segment) break;
  }
  if constexpr (CS > 1) cluster_sync();  // nobody's shared memory goes while it is read
}

struct Source {
  long long row;  // (block * H + h) * block_size + row in the pool; -1: none
  float ks, vs;   // 8 bits: its block's scales
};

template <int D, int FMT>
__global__ void __launch_bounds__(kCopy) cache_copy_kernel(const EvictParams p, int blocks) {
  constexpr bool I4 = FMT == FMT_INT4, E5M2 = FMT == FMT_E5M2;
  const CacheParams& c = p.c;
  __shared__ long long row_of[128];
  __shared__ float ks_of[128], vs_of[128];
  __shared__ float part[2][kCopy / 32];
  const int t = threadIdx.x, bs = c.block_size;
  const int blk = (int)(blockIdx.x % (unsigned)blocks);
  const int bh = (int)(blockIdx.x / (unsigned)blocks);
  const int b = bh / c.H, h = bh % c.H;
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the selection
  const int n = p.lens_out[b];
  const int count = min(bs, n - blk * bs);  // tokens of this block
  if (count <= 0) return;
  const int page_out = p.table_out[(long long)b * p.table_out_width + blk];
  if (page_out < 0 || page_out >= c.num_blocks) {
    if (t == 0 && c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_EVICT + 1);
    return;
  }
  float ks_max = 0.f, vs_max = 0.f;
  if (t < count) {  // (a block has at most 128 tokens)
    const int pos = p.kept[(long long)bh * p.keep + blk * bs + t];
    // (no such token: its place was not written, as the weights changed under the selection)
    const bool there = (unsigned)pos < (unsigned)(c.table_width * bs);
    const int page =
        there ? c.block_table[(long long)b * c.table_width + (pos >> c.block_log2)] : -1;
    Source s{-1, 0.f, 0.f};
    if (page < 0 || page >= c.num_blocks) {
      if (c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_EVICT + 1);
    } else {
      const long long block = (long long)page * c.H + h;
      s.row = (block << c.block_log2) + (pos & (bs - 1));
      if constexpr (!I4) s.ks = c.k_scale[block], s.vs = c.v_scale[block];
    }
    row_of[t] = s.row;
    if constexpr (!I4) {
      ks_of[t] = s.ks, vs_of[t] = s.vs;
      ks_max = s.ks, vs_max = s.vs;
    }
  }
  const long long block_out = (long long)page_out * c.H + h;
  if constexpr (!I4) {
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) {
      ks_max = fmaxf(ks_max, __shfl_xor_sync(0xffffffffu, ks_max, w));
      vs_max = fmaxf(vs_max, __shfl_xor_sync(0xffffffffu, vs_max, w));
    }
    if ((t & 31) == 0) part[0][t >> 5] = ks_max, part[1][t >> 5] = vs_max;
  }
  __syncthreads();
  if constexpr (!I4) {
#pragma unroll
    for (int w = 0; w < kCopy / 32; ++w)
      ks_max = fmaxf(ks_max, part[0][w]), vs_max = fmaxf(vs_max, part[1][w]);
    if (!(ks_max > 0.f)) ks_max = 7.888609052210118e-31f;  // 2^-100: no token has a block
    if (!(vs_max > 0.f)) vs_max = 7.888609052210118e-31f;
    if (t == 0) c.k_scale[block_out] = ks_max, c.v_scale[block_out] = vs_max;
  }
  constexpr int RB = I4 ? D / 2 : D, PIECES = RB / 16;  // 16-byte pieces of a row
  const long long out0 = block_out << c.block_log2;
  const int pieces = count * PIECES;  // of the keys, and as many of the values
  for (int x0 = t; x0 < 2 * pieces; x0 += kAhead * kCopy) {
    uint4 v[kAhead];
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int x = x0 + n * kCopy;
      const bool value = x >= pieces;
      const int y = value ? x - pieces : x;
      v[n] = I4 ? make_uint4(0x88888888u, 0x88888888u, 0x88888888u, 0x88888888u)
                : make_uint4(0u, 0u, 0u, 0u);
      if (x >= 2 * pieces) continue;
      const long long row = row_of[y / PIECES];
      if (row >= 0)
        v[n] = *reinterpret_cast<const uint4*>((value ? c.v : c.k) + row * RB + y % PIECES * 16);
    }
#pragma unroll
    for (int n = 0; n < kAhead; ++n) {
      const int x = x0 + n * kCopy;
      if (x >= 2 * pieces) break;
      const bool value = x >= pieces;
      const int y = value ? x - pieces : x, r = y / PIECES;
      if constexpr (!I4) {
        const float from = value ? vs_of[r] : ks_of[r], to = value ? vs_max : ks_max;
        if (from != to && row_of[r] >= 0) {  // rounded for the larger scale
          const float f = from / to;
          uint32_t* w = &v[n].x;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float2 lo = f16x2_to_f32(codes_to_f16x2<E5M2>((uint16_t)(w[k] & 0xffffu)));
            const float2 hi = f16x2_to_f32(codes_to_f16x2<E5M2>((uint16_t)(w[k] >> 16)));
            // (infinities, which the conversion would bring to the largest value, stay)
            const uint32_t inf = E5M2 ? __vcmpeq4(w[k] & 0x7f7f7f7fu, 0x7c7c7c7cu) : 0u;
            const uint32_t r = (uint32_t)f32_to_codes<E5M2>(lo.x * f, lo.y * f) |
                               (uint32_t)f32_to_codes<E5M2>(hi.x * f, hi.y * f) << 16;
            w[k] = (w[k] & inf) | (r & ~inf);
          }
        }
      }
      *reinterpret_cast<uint4*>((value ? c.v : c.k) + (out0 + r) * RB + y % PIECES * 16) = v[n];
    }
  }
  if constexpr (I4) {
    using S = typename std::conditional<D == 128, uint2, uint32_t>::type;  // a token's scales
    for (int x = t; x < count * 2; x += kCopy) {
      const bool value = x >= count;
      const int r = value ? x - count : x;
      uint8_t* scales = value ? c.v_scale4() : c.k_scale4();
      S s{};
      if (row_of[r] >= 0) s = *reinterpret_cast<const S*>(scales + row_of[r] * (D / 16));
      *reinterpret_cast<S*>(scales + (out0 + r) * (D / 16)) = s;
    }
  }
}

template <int CS>
cudaError_t launch_select(const EvictParams& p, long long units, cudaStream_t stream) {
  constexpr int SMEM = kRun * kSelect * 4;
  static unsigned long long prepared[64];
  const cudaError_t e = prepare_once(prepared, [] {
    return cudaFuncSetAttribute(cache_select_kernel<CS>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, SMEM);
  });
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = CS;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(units * CS));
  cfg.blockDim = dim3(kSelect);
  cfg.dynamicSmemBytes = SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_select_kernel<CS>, p);
}

template <int D, int FMT>
cudaError_t start(const EvictParams& p, int n_sm, cudaStream_t stream) {
  const long long units = (long long)p.c.B * p.c.H;
  const long long most = std::min<long long>(p.keep, p.width);  // tokens of a sequence
  const int blocks = (int)((most + p.c.block_size - 1) / p.c.block_size);
  if (units * blocks > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
  // As many CTAs a row (up to 8) as leave none waiting for an SM, which one fills, and as have
  // two weights a thread.
  const auto fits = [&](int cs) { return units * cs <= n_sm && p.width >= 2 * cs * kSelect; };
  cudaError_t e = fits(8)   ? launch_select<8>(p, units, stream)
                  : fits(4) ? launch_select<4>(p, units, stream)
                  : fits(2) ? launch_select<2>(p, units, stream)
                            : launch_select<1>(p, units, stream);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(units * blocks));
  cfg.blockDim = dim3(kCopy);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_copy_kernel<D, FMT>, p, blocks);
}

}  // namespace

cudaError_t launch_cache_evict(const EvictParams& p, int n_sm, cudaStream_t stream) {
  const bool d128 = p.c.d == 128;
  switch (p.c.format) {
    case FMT_E4M3:
      return d128 ? start<128, FMT_E4M3>(p, n_sm, stream) : start<64, FMT_E4M3>(p, n_sm, stream);
    case FMT_E5M2:
      return d128 ? start<128, FMT_E5M2>(p, n_sm, stream) : start<64, FMT_E5M2>(p, n_sm, stream);
    default:
      return d128 ? start<128, FMT_INT4>(p, n_sm, stream) : start<64, FMT_INT4>(p, n_sm, stream);
  }
}

}  // namespace fattn

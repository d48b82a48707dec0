// cache_weights.cu -- the attention weight that every cached key receives from a batch's
// queries, for sequences with few query rows per key/value head.
//
// For sequence b and key/value head h, over its rows (token i, query head g of the group):
//   W_j (+)= sum_rows exp(scale q_row . k_j - lse_row),   row sees key j,
// with the log-sum-exp that the attention left.  A key's sum is formed by one warp in the
// rows' order, so the result does not depend on the launch.
//
// S^T = K Q^T on m16n8k16 mma.sync with the keys as the 16-row operand, as in the attention
// for few rows: codes exact in fp16 (4 bits: value times 2^-7), q as fp16 times a power of two
// per row.  A warp holds 32 keys as fp16 operands in registers, a CTA 128; the rows pass by in
// shared memory, 32 at a time.  The contraction's order follows the codes: a lane takes its
// quarter of a key's channels as 16-byte pieces of fp16, which are stored in the order in
// which four lanes and two rows read them without conflict.
//
// Work split.  A unit is (sequence, head, 128 keys); the units in that order are cut into equal
// contiguous shares, one per CTA, so a CTA goes through neighbouring keys of one sequence and,
// where the rows are at most 32, loads them once for all of them.
//
// Measured, one token of each of 32 sequences of 512 to 8192 tokens, 32 query and 8 key heads, 4 bits,
// d = 128: 20.5 us, 42 % of the measured copy bandwidth.  It is bound by issue, 520 instructions
// for 32 keys a warp at 2.0 a clock (168 registers: 12 warps an SM), and by the start of a
// share, 5000 of 39,000 clocks.  (With the next keys' codes loaded where they are needed 32 us, a block
// number for every 16 keys, zeroed registers for keys without a block and a key's sum
// stored by one lane of four 23.4; the rows staged ahead of the keys' conversion 21.8.)
#include <math.h>

#include "evict.cuh"

namespace fattn {
namespace {

constexpr int kWarpsW = 4;
constexpr int kKeys = 128;     // of a unit
constexpr int kRows = 32;      // staged at a time
constexpr int ctas_w(int d) { return d == 128 ? 3 : 4; }  // per SM: as the registers allow
constexpr float kLog2eW = 1.4426950408889634f;

template <int D>
struct Wt {
  static constexpr int PIECES = D / 8;            // 16-byte pieces of a row
  static constexpr int U = D / 32;                // of a lane's quarter
  static constexpr int STRIDE = D * 2 + 64;       // bytes: the next row starts 64 later, mod 128
};

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// First channel of piece u of quarter t: where the codes put the contraction index.
template <int D, bool I4>
__device__ __forceinline__ int piece_channel(int u, int t) {
  return I4 ? t * (D / 4) + u * 8 : (u >> 1) * 64 + t * 16 + (u & 1) * 8;
}

template <int D, int FMT>
__global__ void __launch_bounds__(32 * kWarpsW, ctas_w(D))
    cache_weights_kernel(const WeightParams p) {
  constexpr bool I4 = FMT == FMT_INT4, E5M2 = FMT == FMT_E5M2;
  using C = Wt<D>;
  constexpr int KS = D / 16;  // k16 steps
  __shared__ alignas(128) uint8_t rows_smem[kRows * C::STRIDE];
  __shared__ alignas(8) float row_scale[kRows], row_lse[kRows];
  __shared__ alignas(8) int row_lim[kRows];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const CacheParams& c = p.c;
  const uint32_t qs = smem_u32(rows_smem);

  // ---------------------------------------------------------------- this CTA's share
  auto units_of = [&](int b, CacheSeq* seq) -> long long {
    if (!cache_seq(c, b, seq) || seq->len > p.width) {
      if (c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_WEIGHTS);
      return 0;
    }
    // (more rows: the other kernel's)
    return seq->n == 0 || (long long)seq->n * p.G > p.narrow_rows
               ? 0
               : (long long)((seq->len + kKeys - 1) / kKeys) * c.H;
  };
  long long total = 0;
  CacheSeq seq;
  const long long n_first = lane < c.B ? units_of(lane, &seq) : 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    long long n = b0 == 0 ? n_first : b0 + lane < c.B ? units_of(b0 + lane, &seq) : 0;
#pragma unroll
    for (int w = 16; w > 0; w >>= 1) n += __shfl_xor_sync(0xffffffffu, n, w);
    total += n;
  }
  const long long share = (total + gridDim.x - 1) / gridDim.x;
  const long long lo = blockIdx.x * share, hi = min(total, lo + share);
  if (lo >= hi) return;
  long long before = 0;  // units of the sequences before b
  int b = 0;
  for (int b0 = 0; b0 < c.B; b0 += 32) {
    const long long n = b0 == 0 ? n_first : b0 + lane < c.B ? units_of(b0 + lane, &seq) : 0;
    long long upto = n;
#pragma unroll
    for (int w = 1; w < 32; w <<= 1) {
      const long long o = __shfl_up_sync(0xffffffffu, upto, w);
      if (lane >= w) upto += o;
    }
    const unsigned past = __ballot_sync(0xffffffffu, before + upto > lo);
    if (past) {
      const int src = __ffs(past) - 1;
      b = b0 + src;
      before += __shfl_sync(0xffffffffu, upto - n, src);
      break;
    }
    before += __shfl_sync(0xffffffffu, upto, 31);
  }
  const Int4Magic magic;
  const float factor = p.scale_log2 * (I4 ? kInt4Unit : 1.f);
  // A place in the list of units.  Three are alive: the one at hand, the next one, whose codes
  // are on their way, and the one behind it, whose block numbers are.
  struct At {
    long long left;  // units of the share from here on
    int b, h, key, keys;  // sequence, head, first key; keys of the sequence's units
    CacheSeq seq;
  };
  auto advance = [&](At* at) {
    if (--at->left <= 0 || (at->key += kKeys) < at->keys) return;
    at->key = 0;
    if (++at->h < c.H) return;
    at->h = 0;
    while (units_of(++at->b, &at->seq) == 0) {
    }
    at->keys = (at->seq.len + kKeys - 1) / kKeys * kKeys;
  };
  constexpr int RB = I4 ? D / 2 : D;      // bytes of a key's codes
  constexpr int RW = I4 ? C::U : D / 16;  // words of codes that a lane has of a key
  int pages[2];
  uint32_t codes[2][2][RW], scales[2][2];
  float ks_next[2] = {1.f, 1.f};
  bool live[2];
  const bool one_block = c.block_size >= 32;  // holds all of a warp's keys
  auto look_up = [&](const At& at) {
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && one_block) break;
      pages[m] = -1;
      if (at.left <= 0) continue;
      const int key = at.key + warp * 32 + 16 * m;
      if (key >= at.seq.len) continue;
      const int page = c.block_table[(long long)at.b * c.table_width + (key >> c.block_log2)];
      pages[m] = page == -1 ? -2 : page;  // (-1: no keys there)
    }
  };
  auto load = [&](const At& at) {  // from the pages looked up for it
    long long row = 0;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      if (m == 1 && one_block) {
        row += 16;
        live[1] = live[0];
        ks_next[1] = ks_next[0];
      } else {
        const int key = at.key + warp * 32 + 16 * m;
        int page = pages[m];
        live[m] = page >= 0 && page < c.num_blocks;
        if (!live[m]) {  // (block 0 is read instead, and what comes of it is not used)
          if (page != -1 && c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_WEIGHTS + 1);
          page = 0;
        }
        const long long block = (long long)page * c.H + at.h;
        if constexpr (!I4) ks_next[m] = c.k_scale[block];
        // (rows behind the sequence's end are read as well: they lie in its block)
        row = (block << c.block_log2) + (key & (c.block_size - 1)) + g;
      }
      const uint8_t* from = c.k + row * RB + t * (I4 ? D / 8 : 16);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t(&w)[RW] = codes[m][i];
        if constexpr (I4 && D == 128) {
          const uint4 x = __ldg(reinterpret_cast<const uint4*>(from + i * 8 * RB));
          w[0] = x.x, w[1] = x.y, w[RW - 2] = x.z, w[RW - 1] = x.w;
          scales[m][i] = __ldg(reinterpret_cast<const uint16_t*>(c.k_scale4() + row * 8 + t * 2 + i * 64));
        } else if constexpr (I4) {
          const uint2 x = __ldg(reinterpret_cast<const uint2*>(from + i * 8 * RB));
          w[0] = x.x, w[1] = x.y;
          scales[m][i] = __ldg(c.k_scale4() + row * 4 + t + i * 32);
        } else {
#pragma unroll
          for (int half = 0; half < D / 64; ++half) {
            const uint4 x = __ldg(reinterpret_cast<const uint4*>(from + i * 8 * RB + half * 64));
            w[half * 4] = x.x, w[half * 4 + 1] = x.y, w[half * 4 + 2] = x.z, w[half * 4 + 3] = x.w;
          }
        }
      }
    }
  };
  At now{hi - lo, b, 0, 0, 0, {}};
  {
    units_of(b, &now.seq);
    const int tiles = (now.seq.len + kKeys - 1) / kKeys;
    now.h = (int)((lo - before) / tiles);
    now.key = (int)((lo - before) % tiles) * kKeys;
    now.keys = tiles * kKeys;
  }
  At next = now;
  look_up(now);
  load(now);
  advance(&next);
  look_up(next);

  int staged_b = -1, staged_h = -1;  // whose rows (all of them) lie in shared memory
  while (now.left > 0) {
    const int b = now.b, h = now.h, cta_key0 = now.key, key0 = cta_key0 + warp * 32;
    const CacheSeq seq = now.seq;
    const int n_rows = seq.n * p.G;
    const int seen0 = p.causal ? seq.len - seq.n + 1 : seq.len;  // token 0's keys

    // ------------------------------------------------------------ the warp's keys
    uint32_t a[2][KS][4];
    const float ks[2] = {ks_next[0], ks_next[1]};
    const bool there[2] = {live[0], live[1]};
#pragma unroll
    for (int m = 0; m < 2; ++m) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if constexpr (I4) {
          const Int4Scale s0 = int4_scale(__byte_perm(scales[m][i], 0u, 0x0404u));
          const Int4Scale s1 = D == 128 ? int4_scale(__byte_perm(scales[m][i], 0u, 0x1414u)) : s0;
#pragma unroll
          for (int u = 0; u < C::U; ++u) {
            uint32_t o[4];
            int4_values(codes[m][i][u], u < 2 ? s0 : s1, magic, o);
            a[m][2 * u][i] = o[0], a[m][2 * u][i + 2] = o[1];
            a[m][2 * u + 1][i] = o[2], a[m][2 * u + 1][i + 2] = o[3];
          }
        } else {
#pragma unroll
          for (int w = 0; w < RW; ++w)
            codes4_to_f16<E5M2>(codes[m][i][w], a[m][w][i], a[m][w][i + 2]);
        }
      }
    }
    // A lane ends with the sum of one key, key0 + 8 t + g, and stores it
    const int mine = key0 + 8 * t + g;
    const bool kept = mine < seq.len;
    const float was = p.accumulate && mine < seq.len - seq.n
                          ? p.in.p[b * p.in.sb + h * p.in.sh + mine] : 0.f;
    load(next);
    now = next;
    advance(&next);
    look_up(next);

    // ------------------------------------------------------------ all rows that see some of them
    float sum[2][2] = {{0.f, 0.f}, {0.f, 0.f}};  // of keys g, g + 8 (+ 16 m), this lane's columns
    // (in 64 bits: a token's number times the group's size.)  Rows that are kept are all there
    const int r_first = p.causal && n_rows > kRows
                            ? (int)((long long)max(0, cta_key0 - (seq.len - seq.n)) * p.G / 8 * 8)
                            : 0;
    for (int r0 = r_first; r0 < n_rows; r0 += kRows) {
      if (!(staged_b == b && staged_h == h)) {
        __syncthreads();  // the rows before have been used
        // a row is taken by PIECES lanes, 16 bytes each
        constexpr int RPP = 32 * kWarpsW / C::PIECES;  // rows a pass
        const int staged = min(kRows, n_rows - r0);
#pragma unroll
        for (int pass = 0; pass < kRows / RPP; ++pass) {
          if (pass * RPP >= staged) break;
          const int r = pass * RPP + threadIdx.x / C::PIECES, piece = threadIdx.x % C::PIECES;
          const int i = r0 + r;
          const int u = piece % C::U, tt = piece / C::U;
          uint4 x = make_uint4(0u, 0u, 0u, 0u);
          long long token = 0;
          int hq = 0;
          if (i < n_rows) {
            token = (long long)seq.row0 + p.by_G.div(i);
            hq = h * p.G + p.by_G.mod(i);
            x = __ldg(reinterpret_cast<const uint4*>(p.q.p + token * p.q.st + (long long)hq * p.q.sh +
                                                     piece_channel<D, I4>(u, tt)));
          }
          uint32_t mx = __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                 __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu));
          mx = max(mx & 0xffffu, mx >> 16);
#pragma unroll
          for (int w = 1; w < C::PIECES; w <<= 1) mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, w));
          // the power of two that brings the row's largest element to [2^14, 2^15)
          int e = (int)(mx >> 7);
          e = (mx == 0u || e == 255) ? 0 : min(14 - (e - 127), 126);
          const float mul = __uint_as_float((uint32_t)(e + 127) << 23);
          uint32_t w[4] = {x.x, x.y, x.z, x.w}, o[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            // 4 bits: channels k and k + 4 of the eight side by side, as the keys have them
            const uint32_t v = I4 ? __byte_perm(w[k >> 1], w[2 + (k >> 1)], k & 1 ? 0x7632u : 0x5410u)
                                  : w[k];
            o[k] = pack_f16x2(__uint_as_float(v << 16) * mul, __uint_as_float(v & 0xffff0000u) * mul);
          }
          st_shared_v4(qs + r * C::STRIDE + (u * 4 + tt) * 16, o[0], o[1], o[2], o[3]);
          if (piece == 0) {
            const float l = i < n_rows ? p.lse[(long long)hq * c.total + token] : -INFINITY;
            row_scale[r] = __uint_as_float((uint32_t)(127 - e) << 23) * factor;
            row_lse[r] = l == -INFINITY ? INFINITY : l * kLog2eW;  // a row that saw nothing
            row_lim[r] = i < n_rows ? min(seq.len, p.causal ? seen0 + p.by_G.div(i) : seen0) : 0;
          }
        }
        __syncthreads();
        if (n_rows <= kRows) staged_b = b, staged_h = h;
      }
      const int n_tiles = (min(kRows, n_rows - r0) + 7) >> 3;
      for (int nt = 0; nt < n_tiles; ++nt) {
        float s[2][4];
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][i] = 0.f;
        const uint32_t at = qs + (nt * 8 + g) * C::STRIDE + t * 16;
#pragma unroll
        for (int u = 0; u < C::U; ++u) {
          uint32_t b0, b1, b2, b3;
          asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(b0), "=r"(b1), "=r"(b2), "=r"(b3)
                       : "r"(at + u * 64));
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_f16(s[m], a[m][2 * u][0], a[m][2 * u][1], a[m][2 * u][2], a[m][2 * u][3], b0, b1);
            mma_f16(s[m], a[m][2 * u + 1][0], a[m][2 * u + 1][1], a[m][2 * u + 1][2],
                    a[m][2 * u + 1][3], b2, b3);
          }
        }
        // columns 2 t, 2 t + 1
        const float2 f2 = *reinterpret_cast<const float2*>(&row_scale[nt * 8 + 2 * t]);
        const float2 l2 = *reinterpret_cast<const float2*>(&row_lse[nt * 8 + 2 * t]);
        const float f[2] = {f2.x, f2.y}, l[2] = {l2.x, l2.y};
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 4; ++i) s[m][i] = ex2(fmaf(s[m][i], I4 ? f[i & 1] : ks[m] * f[i & 1], -l[i & 1]));
        if (key0 + 32 > seen0) {  // some row may not see all of them
          const int2 lim2 = *reinterpret_cast<const int2*>(&row_lim[nt * 8 + 2 * t]);
          const int lim[2] = {lim2.x, lim2.y};
#pragma unroll
          for (int m = 0; m < 2; ++m)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (key0 + 16 * m + g + 8 * (i >> 1) >= lim[i & 1]) s[m][i] = 0.f;
        }
#pragma unroll
        for (int m = 0; m < 2; ++m)
#pragma unroll
          for (int i = 0; i < 2; ++i) sum[m][i] += s[m][2 * i] + s[m][2 * i + 1];
      }
    }
    // over the four lanes of a key; lane t goes on with keys 8 t + g alone
    float half[2];
#pragma unroll
    for (int m = 0; m < 2; ++m)
      half[m] = (t & 1 ? sum[m][1] : sum[m][0]) +
                __shfl_xor_sync(0xffffffffu, t & 1 ? sum[m][0] : sum[m][1], 1);
    const float x = (t & 2 ? half[1] : half[0]) +
                    __shfl_xor_sync(0xffffffffu, t & 2 ? half[0] : half[1], 2);
    // (no block there: nothing from the queries)
    if (kept) p.out.p[b * p.out.sb + h * p.out.sh + mine] = was + ((t & 2 ? there[1] : there[0]) ? x : 0.f);
  }
}

template <int D, int FMT>
cudaError_t start(const WeightParams& p, int n_sm, cudaStream_t stream) {
  cache_weights_kernel<D, FMT><<<(unsigned)(n_sm * ctas_w(D)), 32 * kWarpsW, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_weights(const WeightParams& p, int n_sm, cudaStream_t stream) {
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

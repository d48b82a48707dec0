// cache_weights_wide.cu -- the attention weight that every cached key receives, for sequences
// with many query rows (pieces of prompts): tcgen05 + TMEM.
//
// S^T = K Q^T with the keys as the 128 lanes of a TMEM tile and 256 query rows as its columns,
// so a thread owns a key and adds exp(s f - lse) over the columns it reads, in their order.
// Both operands are bf16 without a rounding: codes and 4-bit values have at most 7 significant
// bits, q is what it is (a block's scale and the softmax scale make f, by key).
//
// A CTA (one per SM) goes through its share of the units, each 128 keys of one (sequence,
// key/value head), against all rows that see some of them:
//   warps 0-15      exponentials and sums, four warps each a quarter of the columns of every S
//                   tile.  They also load the next unit's codes while they work on one, and
//                   store them as bf16, in the 128-byte-swizzled layout that a TMA load would
//                   leave, ahead of its last rows, into the other of two places
//   warp 16         Q, 256 rows at a time, by TMA straight from the caller's tensor: a tile is
//                   tb = 256 / G tokens of the group's G heads, which a box {64, G, tb} leaves as
//                   rows
//   warps 17, 19    the MMAs, a thread each for the tiles of one of two S buffers
//   warp 18         the rows' log-sum-exp, a place for each S buffer
// Two units are needed about equally: 128 x 256 exponentials take 1024 clocks of the
// special-function unit at the 32 a clock that were measured, and the products of that tile keep
// the tensor pipe busy for 1015 (its counter; A and B alone, read from shared memory at 128 bytes a
// clock, would take 768).  One thread that issued all MMAs was the bound before: its waits, 8
// instructions and commits take 1500 clocks a tile, as it shares its issue slots with the
// exponentials.  (Built and measured before this, 512 queries behind 16384 tokens, 32 query and
// 8 key heads, d = 128: mma.sync 457 us; 256 keys a unit, 8 warps, tiles of 128 rows 127 us, 16
// warps 94 us; tiles of 256 rows, S in one buffer for each 128 keys, 88 us; S in two, 32
// columns loaded at a time, 76 us; the next 16 on their way while 16 are worked on 74; one
// barrier for S and the log-sum-exp instead of two 70; whole tiles without the mask's arithmetic
// and units found by counting 68.5.)  Now 68.5 us, 1018 TFLOP/s.  The warps of exponentials are the
// bound: a warp's 64 columns take 1500 clocks, the four warps of a scheduler at once, its arrival
// and the next wait 300, a change of unit 2000.  (Work for the next unit moved into a tile, another
// for every quarter of the columns: 73.  With half of Q loaded, to see what its way from L2
// costs, 73 where the whole took 74; without the loads of the log-sum-exp 70; without the
// exponentials 64.)
#define FATTN_INLINE_WAIT_SLOW_PATH
#include <math.h>

#include <algorithm>
#include <type_traits>

#include "evict.cuh"

namespace fattn {
namespace {

constexpr float kLog2eV = 1.4426950408889634f;

template <int D>
struct Ww {
  static constexpr int BM = 128, BN = 256;
  static constexpr int HALF = BM * 128;      // 64 channels of the keys (bytes)
  static constexpr int TILE = BM * D * 2;
  static constexpr int Q_HALF = BN * 128, Q_TILE = BN * D * 2;
  static constexpr int ST = D == 128 ? 2 : 4;
  static constexpr int SUMS = 4;             // units
  static constexpr int OFF_K = 0;            // [2]
  static constexpr int OFF_Q = 2 * TILE;
  static constexpr int OFF_INFO = OFF_Q + ST * Q_TILE;      // [2][BN] -lse log2(e)
  static constexpr int OFF_SUM = OFF_INFO + 2 * BN * 4;  // [SUMS][3][BM] of the later columns
  static constexpr int OFF_BAR = OFF_SUM + SUMS * 3 * BM * 4;
  static constexpr int SMEM = OFF_BAR + 512 + 1024;
  static constexpr int W_LOAD = 16, W_MMA = 17, W_INFO = 18, W_MMA2 = 19, THREADS = 640;
  static constexpr uint32_t IDESC = idesc_bf16_f32(128, BN, false, false);
  static constexpr uint32_t IDESC_128 = idesc_bf16_f32(128, 128, false, false);
  static_assert(SMEM <= 232448, "shared memory budget");
};
enum {
  X_K_FULL = 0,    // [2] keys in shared memory (512 threads)
  X_S_FULL = 2,    // [2] S, and the log-sum-exp of its rows
  X_S_EMPTY = 4,   // [2], 16 warps
  X_DONE = 6,      // [2]
  X_SUM = 8,       // [SUMS] the sums of the later columns (384 threads)
  X_I_FULL = 12,   // [2] the rows' log-sum-exp
  X_Q_FULL = 14,   // [ST], then q_empty [ST]
};

__device__ __forceinline__ void fma_x2(float a0, float a1, float b, float c0, float c1, float& r0,
                                       float& r1) {
  asm("{\n\t.reg .b64 a, b, c, r;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %4};\n\t"
      "mov.b64 c, {%5, %6};\n\t"
      "fma.rn.f32x2 r, a, b, c;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c0), "f"(c1));
}
__device__ __forceinline__ void add_x2(float& s0, float& s1, float a0, float a1) {
  asm("{\n\t.reg .b64 s, a;\n\t"
      "mov.b64 s, {%0, %1};\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "add.rn.f32x2 s, s, a;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "+f"(s0), "+f"(s1)
      : "f"(a0), "f"(a1));
}
__device__ __forceinline__ void tmem_ld16(uint32_t at, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, "
      "%12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
        "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]),
        "=r"(r[15])
      : "r"(at));
}
__device__ __forceinline__ void tmem_wait_ld16(uint32_t (&r)[16]) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]),
                 "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]),
                 "+r"(r[13]), "+r"(r[14]), "+r"(r[15])::"memory");
}
__device__ __forceinline__ float4 ld_shared_f4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(a));
  return v;
}

// A unit of this CTA's share, found alike by every warp.  The units of a sequence count as many
// row tiles as it has; a share is an equal part of all, to which the units belong that begin in it.
// (The causal mask is not counted: of a prompt without tokens before it, the shares with a head's
// first keys have up to twice the mean to do; and a unit is one CTA's, however many rows it has.
// 8192 such tokens, 32 query and 8 key heads, d = 128, take 468 us, 587 TFLOP/s.)
template <int KEYS>
struct Walk {
  const WeightParams& p;
  long long before, hi;  // cost of the sequences before; end of the share
  long long rest;        // units of the sequence that are the share's, from this one on
  int b, h, tile;        // sequence, head, tile of keys
  CacheSeq seq;
  int tiles, row_tiles;  // of keys, of rows
  __device__ __forceinline__ long long cost_of(int b) {
    row_tiles = tiles = 0;
    if (!cache_seq(p.c, b, &seq) || seq.len > p.width) return 0;  // (reported by the other kernel)
    if ((long long)seq.n * p.G <= p.narrow_rows) return 0;
    tiles = (seq.len + KEYS - 1) / KEYS;
    row_tiles = (seq.n + p.tile_tokens - 1) / p.tile_tokens;
    return (long long)tiles * p.c.H * row_tiles;
  }
  __device__ __forceinline__ explicit Walk(const WeightParams& p_) : p(p_) {
    const int lane = threadIdx.x & 31;
    long long total = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      long long n = b0 + lane < p.c.B ? cost_of(b0 + lane) : 0;
#pragma unroll
      for (int w = 16; w > 0; w >>= 1) n += __shfl_xor_sync(0xffffffffu, n, w);
      total += n;
    }
    const long long share = (total + gridDim.x - 1) / gridDim.x, lo = blockIdx.x * share;
    hi = min(total, lo + share);
    b = p.c.B, rest = 0, h = tile = 0, before = total;
    if (lo >= hi) return;
    before = 0;
    for (int b0 = 0; b0 < p.c.B; b0 += 32) {
      const long long n = b0 + lane < p.c.B ? cost_of(b0 + lane) : 0;
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
    const long long n = cost_of(b), u = (lo - before + row_tiles - 1) / row_tiles;
    h = (int)(u / tiles);
    tile = (int)(u % tiles);
    rest = of_share() - u;
    if (u * row_tiles >= n)
      enter(n);
    else if (rest <= 0)
      b = p.c.B;
  }
  __device__ __forceinline__ long long of_share() const {  // units that begin before its end
    return min((long long)tiles * p.c.H, (hi - before + row_tiles - 1) / row_tiles);
  }
  __device__ __forceinline__ void enter(long long n) {  // the sequence after b, whose cost is n
    h = tile = 0;
    do {
      before += n;
      if (before >= hi || ++b >= p.c.B) {
        b = p.c.B;
        return;
      }
      n = cost_of(b);
    } while (n == 0);
    rest = of_share();
  }
  __device__ __forceinline__ bool valid() const { return b < p.c.B; }
  __device__ __forceinline__ void next() {
    if (--rest <= 0) return enter((long long)tiles * p.c.H * row_tiles);
    if (++tile == tiles) tile = 0, ++h;
  }
  __device__ __forceinline__ int key0() const { return tile * KEYS; }
  // the first tile of rows that see some of the unit's keys
  __device__ __forceinline__ int first_rows() const {
    return p.causal ? p.by_tile.div(max(0, key0() - (seq.len - seq.n))) : 0;
  }
};

template <int D, int FMT>
__global__ void __launch_bounds__(Ww<D>::THREADS, 1)
    cache_weights_wide_kernel(const __grid_constant__ CUtensorMap tm_q, const WeightParams p) {
  using C = Ww<D>;
  constexpr bool I4 = FMT == FMT_INT4, E5M2 = FMT == FMT_E5M2;
  constexpr int ST = C::ST;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const CacheParams& c = p.c;
  auto bar = [&](int i) { return sbase + C::OFF_BAR + 8u * (uint32_t)i; };
  const uint32_t q_full0 = bar(X_Q_FULL), q_empty0 = bar(X_Q_FULL + ST);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * (X_Q_FULL + 2 * ST));
  volatile uint32_t* abort_flag = tmem_slot + 1;
  const WaitCtx wctx{abort_flag, c.err};
  static_assert(8 * (X_Q_FULL + 2 * ST) + 8 <= 512, "barrier block");
  static_assert(X_I_FULL - X_SUM == C::SUMS, "barriers");

  if (threadIdx.x == 0) {
    for (int i = 0; i < 2; ++i) {
      mbar_init(bar(X_K_FULL + i), 512);
      mbar_init(bar(X_S_FULL + i), 2);
      mbar_init(bar(X_S_EMPTY + i), 16);
      mbar_init(bar(X_DONE + i), 1);
      mbar_init(bar(X_I_FULL + i), 1);
    }
    for (int i = 0; i < C::SUMS; ++i) mbar_init(bar(X_SUM + i), 384);
    for (int i = 0; i < ST; ++i) {
      mbar_init(q_full0 + 8u * i, 1);
      mbar_init(q_empty0 + 8u * i, 1);
    }
    *abort_flag = 0u;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  Walk<C::BM> walk(p);

  if (warp == C::W_LOAD) {
    // ---------------------------------------------------------------- Q (one thread)
    if (lane == 0) {
      int i = 0;  // tiles of rows so far
      bool ok = true;
      for (; ok && walk.valid(); walk.next()) {
        const int h = walk.h, row0 = walk.seq.row0;
        for (int j = walk.first_rows(); j < walk.row_tiles; ++j, ++i) {
          const int stage = i % ST, use = i / ST;
          ok = use == 0 || mbar_wait(q_empty0 + 8u * stage, (use - 1) & 1, wctx,
                                     ERR_SITE_CACHE_WEIGHTS + 2);
          if (!ok) break;
          const uint32_t dst = sbase + C::OFF_Q + stage * C::Q_TILE;
          // (what lies outside of the tensor counts as loaded zeros)
          mbar_arrive_expect_tx(q_full0 + 8u * stage, (uint32_t)(p.tile_tokens * p.G * D * 2));
#pragma unroll
          for (int x = 0; x < D / 64; ++x)
            tma_load_3d(dst + x * C::Q_HALF, &tm_q, q_full0 + 8u * stage, x * 64, h * p.G,
                        row0 + j * p.tile_tokens);
        }
      }
      // copies in flight land before the CTA ends (only after a wait that ran out)
      for (int k = max(0, i - ST); k < i; ++k)
        mbar_drain(q_full0 + 8u * (k % ST), (k / ST) & 1, wctx, ERR_SITE_CACHE_WEIGHTS + 3);
    }
    __syncwarp();
  } else if (warp == C::W_INFO) {
    // ---------------------------------------------------------------- log-sum-exp
    int i = 0;
    bool ok = true;
    for (; ok && walk.valid(); walk.next()) {
      const int h = walk.h, n = walk.seq.n, row0 = walk.seq.row0;
      for (int j = walk.first_rows(); j < walk.row_tiles; ++j, ++i) {
        const int buf = i & 1, use = i >> 1;
        const int tok0 = j * p.tile_tokens;
        const int rows = min(p.tile_tokens, n - tok0) * p.G;
        float l[C::BN / 32];
#pragma unroll
        for (int k = 0; k < C::BN / 32; ++k) {
          const int r = k * 32 + lane;
          l[k] = -INFINITY;
          if (r < rows)
            l[k] = p.lse[(long long)(h * p.G + p.by_G.mod(r)) * c.total + row0 + tok0 + p.by_G.div(r)];
        }
        ok = use == 0 || __all_sync(0xffffffffu, mbar_wait(bar(X_S_EMPTY + buf), (use - 1) & 1, wctx,
                                                           ERR_SITE_CACHE_WEIGHTS + 11));
        if (!ok) break;
#pragma unroll
        for (int k = 0; k < C::BN / 32; ++k)  // a row that saw nothing adds nothing
          reinterpret_cast<float*>(smem + C::OFF_INFO)[buf * C::BN + k * 32 + lane] =
              l[k] == -INFINITY ? -INFINITY : -l[k] * kLog2eV;
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(X_I_FULL + buf));
      }
    }
    __syncwarp();
  } else if (warp == C::W_MMA || warp == C::W_MMA2) {
    // ---------------------------------------------------------------- MMA issuers (a thread each:
    // electing one of a warp for every instruction took longer)
    if (lane == 0) {
      const int buf = warp == C::W_MMA ? 0 : 1;  // this one's tiles of rows: the even, the odd ones
      int i = 0, units = 0;
      const uint64_t ka0 = sdesc_sw128(sbase + C::OFF_K, 16, 1024);
      const uint64_t qb0 = sdesc_sw128(sbase + C::OFF_Q, 16, 1024);
      bool ok = true;
      for (; ok && walk.valid(); walk.next(), ++units) {
        bool keys = false;  // this unit's have been waited for
        for (int j = walk.first_rows(); ok && j < walk.row_tiles; ++j, ++i) {
          if ((i & 1) != buf) continue;
          const int stage = i % ST, use = i >> 1;
          const bool half = (walk.seq.n - j * p.tile_tokens) * p.G <= 128;
          ok = mbar_wait(q_full0 + 8u * stage, (i / ST) & 1, wctx, ERR_SITE_CACHE_WEIGHTS + 5) &&
               (keys || mbar_wait(bar(X_K_FULL + (units & 1)), (units >> 1) & 1, wctx,
                                  ERR_SITE_CACHE_WEIGHTS + 4)) &&
               (use == 0 || mbar_wait(bar(X_S_EMPTY + buf), (use - 1) & 1, wctx,
                                      ERR_SITE_CACHE_WEIGHTS + 6));
          if (!ok) break;
          keys = true;
          tc_fence_after();
          const uint64_t ka = ka0 + (uint32_t)((units & 1) * C::TILE >> 4);
          const uint64_t qb = qb0 + (uint32_t)(stage * C::Q_TILE >> 4);
          const uint32_t idesc = half ? C::IDESC_128 : C::IDESC;
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk)
            mma_bf16_ss(tmem + buf * C::BN,
                        ka + (uint32_t)(((kk >> 2) * C::HALF + (kk & 3) * 32) >> 4),
                        qb + (uint32_t)(((kk >> 2) * C::Q_HALF + (kk & 3) * 32) >> 4), idesc, kk > 0);
          mma_commit(bar(X_S_FULL + buf));
          mma_commit(q_empty0 + 8u * stage);
          // on behalf of the log-sum-exp: one wait less for 16 warps
          ok = mbar_wait(bar(X_I_FULL + buf), use & 1, wctx, ERR_SITE_CACHE_WEIGHTS + 8);
          if (ok) mbar_arrive(bar(X_S_FULL + buf));
        }
      }
      mma_commit(bar(X_DONE + buf));  // drain before TMEM is freed
      mbar_drain(bar(X_DONE + buf), 0, wctx, ERR_SITE_CACHE_WEIGHTS + 7);
    }
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- keys, exponentials, sums
    const int part = warp >> 2, t = threadIdx.x & 127;
    constexpr int RB = I4 ? D / 2 : D, PPR = RB / 16;  // bytes, 16-byte pieces of a row
    constexpr int RPI = 512 / PPR < 128 ? 512 / PPR : 128;  // rows of a load by all threads
    constexpr int LD = 128 / RPI;
    const int prow = (int)threadIdx.x / PPR, piece = threadIdx.x % PPR;
    const bool loads = prow < RPI;
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    uint4 raw_codes[LD];
    uint32_t raw_scale[LD];
    float ks = 0.f;     // of key t; 0: it has no block
    auto checked = [&](int page) {
      if (page == -1 || (page >= 0 && page < c.num_blocks)) return page;
      if (c.err) atomicCAS(c.err, 0u, (unsigned)ERR_SITE_CACHE_WEIGHTS + 1);
      return -1;
    };
    // The codes of the unit that `walk` is at: block numbers first, the rest once they are there
    int pages[LD], page_k = -1;
    auto look_up = [&]() {
      auto entry = [&](int key) {  // (-1: no key there)
        if (key >= walk.seq.len) return -1;
        const int page = c.block_table[(long long)walk.b * c.table_width + (key >> c.block_log2)];
        return page == -1 ? -2 : page;
      };
#pragma unroll
      for (int x = 0; x < LD; ++x) pages[x] = loads ? entry(walk.key0() + x * RPI + prow) : -1;
      page_k = entry(walk.key0() + t);
    };
    auto load = [&]() {
      const int h = walk.h, key0 = walk.key0();
#pragma unroll
      for (int x = 0; x < LD; ++x) {
        const int key = key0 + x * RPI + prow;
        const int page = checked(pages[x]);
        raw_codes[x] = make_uint4(0u, 0u, 0u, 0u);
        raw_scale[x] = 0u;
        if (page < 0) continue;
        const long long row = (((long long)page * c.H + h) << c.block_log2) + (key & (c.block_size - 1));
        raw_codes[x] = __ldg(reinterpret_cast<const uint4*>(c.k + row * RB + piece * 16));
        if constexpr (I4)
          raw_scale[x] =
              __ldg(reinterpret_cast<const uint16_t*>(c.k_scale4() + row * (D / 16) + piece * 2));
      }
      const int page = checked(page_k);
      ks = page < 0 ? 0.f : I4 ? 1.f : c.k_scale[(long long)page * c.H + h];
    };
    auto store = [&](int u) {  // unit u's, as bf16, rows of 128 bytes, 16-byte columns swizzled
      // by row & 7; the MMAs of unit u - 2, whose place it is, are done: its last S was read
      const uint32_t tile = sbase + C::OFF_K + (u & 1) * C::TILE;
#pragma unroll
      for (int x = 0; x < LD; ++x) {
        if (!loads) break;
        const int row = x * RPI + prow;
        const uint32_t w[4] = {raw_codes[x].x, raw_codes[x].y, raw_codes[x].z, raw_codes[x].w};
        auto put = [&](int ch, const uint32_t (&o)[4]) {  // eight channels from ch on
          const uint32_t at = tile + (ch >> 6) * C::HALF + row * 128 +
                              ((((ch >> 3) & 7) ^ (row & 7)) << 4);
          st_shared_v4(at, o[0], o[1], o[2], o[3]);
        };
        if constexpr (I4) {
#pragma unroll
          for (int y = 0; y < 4; ++y) {  // a word: eight codes
            uint32_t o[4];
            bf16_values(w[y], bf16_scale(raw_scale[x] >> (8 * (y >> 1)) & 0xffu), o);
            put(piece * 32 + y * 8, o);
          }
        } else {
#pragma unroll
          for (int y = 0; y < 2; ++y) {  // two words: eight codes
            uint32_t o[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              const float2 v = f16x2_to_f32(
                  codes_to_f16x2<E5M2>((uint16_t)(w[2 * y + (k >> 1)] >> (16 * (k & 1)) & 0xffffu)));
              o[k] = pack_bf16x2(v.x, v.y);
            }
            put(piece * 16 + y * 8, o);
          }
        }
      }
      fence_proxy_async_smem();
      mbar_arrive(bar(X_K_FULL + (u & 1)));
    };
    const bool whole = part * 64 + 64 <= p.tile_tokens * p.G;  // of a tile without its last rows
    int i = 0;      // tiles of rows so far
    int units = 0;
    bool ok = true;
    if (walk.valid()) {
      look_up();
      load();
      store(0);
    }
    while (ok && walk.valid()) {
      const float k_scale = ks, f = ks * p.scale_log2;
      // the unit at hand; `walk` goes on to the next one
      const int b = walk.b, h = walk.h, len = walk.seq.len, n = walk.seq.n;
      const int key = walk.key0() + t, key_last = walk.key0() + C::BM - 1;
      const int first = walk.first_rows(), row_tiles = walk.row_tiles;
      walk.next();
      const bool more = walk.valid();
      if (more) {
        look_up();
        load();
      }
      const bool older = part == 0 && p.accumulate && key < len - n;
      const float was = older ? p.in.p[b * p.in.sb + h * p.in.sh + key] : 0.f;
      float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f;
      // rows of tokens from here on see all of the unit's keys
      const int all_seen = p.causal ? key_last - (len - n) : 0;
      int tok0 = first * p.tile_tokens;
      for (int j = first; ok && j < row_tiles; ++j, ++i, tok0 += p.tile_tokens) {
        if (more && j == row_tiles - 1) store(units + 1);
        const int buf = i & 1;
        ok = __all_sync(0xffffffffu, mbar_wait(bar(X_S_FULL + buf), (i >> 1) & 1, wctx,
                                               ERR_SITE_CACHE_WEIGHTS + 9));
        if (!ok) break;
        tc_fence_after();
        int rows = 0, from = 0;
        bool masked = false, some = true;
        if (tok0 < all_seen || tok0 + p.tile_tokens > n || !whole) {
          rows = min(p.tile_tokens, n - tok0) * p.G;
          // this key is seen by rows from `from` on
          const int ahead = p.causal ? key - (len - n) - tok0 : 0;
          from = ahead >= p.tile_tokens ? C::BN : max(0, ahead) * p.G;
          masked = tok0 < all_seen || part * 64 + 64 > rows;
          some = part * 64 < rows;
        }
        const uint32_t info = sbase + C::OFF_INFO + (uint32_t)(buf * C::BN + part * 64) * 4u;
        const uint32_t tS = tmem + lane_off + buf * C::BN + part * 64;
        // 16 columns at a time, the next ones on their way; the exponents of two at a time
        uint32_t v[2][16];
        auto columns = [&](auto with_mask) {
          tmem_ld16(tS, v[0]);
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            uint32_t(&y)[16] = v[x & 1];
            tmem_wait_ld16(y);
            if (x < 3) tmem_ld16(tS + (x + 1) * 16, v[(x + 1) & 1]);
#pragma unroll
            for (int k = 0; k < 16; k += 4) {
              const float4 l = ld_shared_f4(info + (x * 16 + k) * 4u);
              float e[4];
              fma_x2(__uint_as_float(y[k]), __uint_as_float(y[k + 1]), f, l.x, l.y, e[0], e[1]);
              fma_x2(__uint_as_float(y[k + 2]), __uint_as_float(y[k + 3]), f, l.z, l.w, e[2], e[3]);
#pragma unroll
              for (int z = 0; z < 4; ++z) {
                e[z] = ex2(e[z]);
                const int col = part * 64 + x * 16 + k + z;
                if (with_mask && (col < from || col >= rows)) e[z] = 0.f;
              }
              add_x2(s0, s1, e[0], e[1]);
              add_x2(s2, s3, e[2], e[3]);
            }
          }
        };
        if (!masked && some)
          columns(std::false_type());
        else if (some)
          columns(std::true_type());
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(bar(X_S_EMPTY + buf));
      }
      // The other columns' sums join the first quarter's.  A unit can have one tile of rows, and
      // S has two buffers: the later quarters may be two units ahead, hence the four places.
      float w = (s0 + s1) + (s2 + s3);
      const int place = units % C::SUMS, turn = units / C::SUMS;
      float* sums = reinterpret_cast<float*>(smem + C::OFF_SUM) + place * 3 * C::BM + t;
      ++units;
      if (part > 0) {
        sums[(part - 1) * C::BM] = w;
        mbar_arrive(bar(X_SUM + place));
        continue;
      }
      ok = ok && __all_sync(0xffffffffu, mbar_wait(bar(X_SUM + place), turn & 1, wctx,
                                                   ERR_SITE_CACHE_WEIGHTS + 10));
      if (ok && key < len) {
        w = k_scale == 0.f ? 0.f : (w + sums[0]) + (sums[C::BM] + sums[2 * C::BM]);
        p.out.p[b * p.out.sb + h * p.out.sh + key] = was + w;
      }
    }
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, int FMT>
cudaError_t start(const CUtensorMap& tq, const WeightParams& p, int n_sm, cudaStream_t stream) {
  using C = Ww<D>;
  static unsigned long long prepared[64];
  const cudaError_t e = prepare_once(prepared, [] {
    return cudaFuncSetAttribute(cache_weights_wide_kernel<D, FMT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  cache_weights_wide_kernel<D, FMT><<<(unsigned)n_sm, C::THREADS, C::SMEM, stream>>>(tq, p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_weights_wide(const CUtensorMap& tq, const WeightParams& p, int n_sm,
                                      cudaStream_t stream) {
  const bool d128 = p.c.d == 128;
  switch (p.c.format) {
    case FMT_E4M3:
      return d128 ? start<128, FMT_E4M3>(tq, p, n_sm, stream) : start<64, FMT_E4M3>(tq, p, n_sm, stream);
    case FMT_E5M2:
      return d128 ? start<128, FMT_E5M2>(tq, p, n_sm, stream) : start<64, FMT_E5M2>(tq, p, n_sm, stream);
    default:
      return d128 ? start<128, FMT_INT4>(tq, p, n_sm, stream) : start<64, FMT_INT4>(tq, p, n_sm, stream);
  }
}

}  // namespace fattn

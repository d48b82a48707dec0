// cache_fwd_wide.cu -- attention over the paged 8-bit key/value cache, many query
// rows per key/value head (pieces of prompts): tcgen05 + TMEM.
//
// A unit is up to 256 rows of one (sequence, key/value head), in two 128-row
// subtiles.  A row is a (token, query head of the group), token-major, so all heads
// that share a key/value head share the unit's keys.  A CTA (one per SM) owns one
// piece of a unit: at most max(8, all tiles of 128 keys / SMs) of its tiles.  So one
// long sequence is spread over the machine, while units that are short against the
// machine's share are not cut and pay for no merge.  (A persistent grid with equal
// shares, built and measured: the loop over pieces cost the MMA warp and the
// registers more than the better balance gave, 371 us against 250 us for 2048 tokens
// behind 8192 with 32 query and 8 key heads, d = 128.)  Per piece the structure is
// that of the dense forward kernel: keys and values of 128 tokens at a time pass
// through a ring of shared-memory slots, S_s = Q_s K^T lives in TMEM, the softmax
// warps turn it into P_s (at d = 128 in place), and O_s += P_s V accumulates in TMEM.
//
// What differs is how a slot is filled.  The codes cannot feed the tensor core as
// they are (q and P need more than 8 bits), so four warps load them from their
// blocks, convert them to fp16 (exact) and store them into the slot in the
// 128-byte-swizzled layout that a TMA load would leave.  Each warp owns 32 rows of
// every tile, two pieces of 16 tokens (a piece lies in one block), and has the next
// tile's codes in flight; block numbers are read 16 to 32 tiles ahead, scales 8 to 24.
//
// The scales are applied by the softmax, per piece, as in the kernel for few rows:
// y = s * ks + log2 vs - b, p = 2^(y - r) (fp16), l += w p with w = 2^(b - log2 vs),
// O = 2^b acc / l.  r is the running maximum of y less 8, moved only when a y
// exceeds it by more than 15 (p stays below 2^16); where |y| >= 2^22 it is the
// maximum itself, as 8 is then too near its rounding.
// b is the smallest exponent of the piece's value scales, which three warps look up
// while the others start.  fp16 weights hold scales up to 2^20 above it.  Where they
// differ more, the piece's tiles are gone through two or three times, each time with
// the keys of 21 exponents, the smallest first: O and r go on, so what is there when
// larger values come is scaled down in fp32, and each pass's l joins the log-sum-exp.
// Scales more than 2^60 below the largest (blocks of zeros) are taken as 2^(b - 60).
// With one block in eight 2^30 smaller the case measured below takes 490 us, with one in
// eight of zeros no longer than without.  (Relative to the first block's scale alone, as
// once, a first block of zeros made O zero or NaN.  The look-up costs 1 us a piece: 16
// sequences of 70 to 128 tokens behind 300 to 7000, 16 heads, 62 us instead of 59 at
// d = 64, 81 instead of 79 at d = 128.)
//
// Warps: 0-3 softmax of subtile 0, 4-7 of subtile 1 (thread t owns row t; they also
// load Q and write O), 8-11 fill the slots, 12 issues the MMAs, 13-15 look up the value
// scales.  TMEM: S_0, S_1, O_0, O_1 (d = 64: P_0, P_1).
//
// Measured, 2048 tokens behind 8192 (32 query, 8 key heads, d = 128): 255 us, 1212
// TFLOP/s, tensor pipe 51 % active.  256 units on 152 SMs are two rounds where 1.7
// would do (16 %); a tile of 128 keys takes 3100 clocks against the MMAs' 2048, the
// MMA warp's own issue (1750) and its waits for P (1350) alternating; the start and
// end of a piece take 11,000 and 5,000 clocks of 250,000.  At d = 64 (16 sequences of
// 1 to 1000 tokens behind 300 to 7000, 16 heads) a tile takes 2200 to 2900 clocks,
// bound by the softmax, and the starts and ends are a fifth of the time.
#define FATTN_INLINE_WAIT_SLOW_PATH
#include <math.h>

#include <algorithm>

#include "cache.cuh"

namespace fattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kOff = 8.f;    // the reference lies this far below the running maximum
constexpr float kRoom = 15.f;  // and moves when a y exceeds it by more
constexpr float kFar = 4194304.f;
constexpr int kWindow = 20;        // exponents of the value scales that share a pass: b ... b + 20
constexpr float kNothing = -60.f;  // log2 vs - b of blocks far below the others
constexpr int kMaxPasses = 3;      // 61 exponents, 21 at a time

template <int N>
__device__ __forceinline__ void regs_inc() {
  asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N));
}
template <int N>
__device__ __forceinline__ void regs_dec() {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N));
}
// (r0, r1) = (a0, a1) * (b, b) + (c, c)
__device__ __forceinline__ void fma_x2(float a0, float a1, float b, float c, float& r0, float& r1) {
  asm("{\n\t.reg .b64 a, b, c, r;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %4};\n\t"
      "mov.b64 c, {%5, %5};\n\t"
      "fma.rn.f32x2 r, a, b, c;\n\t"
      "mov.b64 {%0, %1}, r;\n\t}"
      : "=f"(r0), "=f"(r1)
      : "f"(a0), "f"(a1), "f"(b), "f"(c));
}
// (s0, s1) = (a0, a1) + (b0, b1)
__device__ __forceinline__ void add_x2(float a0, float a1, float b0, float b1, float& s0,
                                       float& s1) {
  asm("{\n\t.reg .b64 s, a, b;\n\t"
      "mov.b64 a, {%2, %3};\n\t"
      "mov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 s, a, b;\n\t"
      "mov.b64 {%0, %1}, s;\n\t}"
      : "=f"(s0), "=f"(s1)
      : "f"(a0), "f"(a1), "f"(b0), "f"(b1));
}

// r + log2 l of a positive l, whose exponent meets r before either is rounded
__device__ __forceinline__ float add_log2(float r, float l) {
  const uint32_t u = __float_as_uint(l);
  if (!(l < INFINITY)) return r + l;  // NaN stays
  return (r + (float)((int)(u >> 23) - 127)) + lg2(__uint_as_float((u & 0x7fffffu) | 0x3f800000u));
}

// log2(2^a + 2^b)
__device__ __forceinline__ float log2_add(float a, float b) {
  const float m = fmaxf(a, b), mm = m == -INFINITY ? 0.f : m;
  return m == -INFINITY ? a + b : add_log2(mm, ex2(a - mm) + ex2(b - mm));
}

// 16 bytes to shared memory, or zeros
__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 x;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
               : "r"(a));
  return x;
}

template <int D>
struct Wide {
  static constexpr int BM = 128;                // rows per subtile
  static constexpr int ROWS = 2 * BM;           // rows per CTA
  static constexpr int BN = 128;                // keys per tile
  static constexpr int PIECES = BN / 16;
  static constexpr int HALF = BM * 128;         // 64 columns of 128 rows (bytes)
  static constexpr int TILE = BM * D * 2;       // fp16
  // With at most 7 slots V of tile j + 3, and K of tile j + 4 behind it, are filled only
  // after all PV of tile j, hence after the softmax read tile j's scales: a ring of four
  // tiles' scales needs no barrier for its reuse
  static constexpr int STAGES = D == 128 ? 5 : 6;
  static constexpr int SCALE_TILES = 4;
  static constexpr int OFF_Q = 0;
  static constexpr int OFF_KV = OFF_Q + 2 * TILE;
  static constexpr int OFF_SCALE = OFF_KV + STAGES * TILE;  // [SCALE_TILES][PIECES] float4
  static constexpr int OFF_BAR = OFF_SCALE + SCALE_TILES * PIECES * 16;
  static constexpr int OFF_SCAN = OFF_BAR + 256;  // Scan
  static constexpr int OFF_LSE = OFF_SCAN + 32;   // [ROWS], used by units of several passes
  static constexpr int SMEM = OFF_LSE + ROWS * 4 + 1024;
  static constexpr int THREADS = 512;
  static constexpr int W_FILL = 8, N_FILL = 4, W_MMA = 12;
  static constexpr int REG_LAUNCH = 128, REG_SOFTMAX = 184, REG_FILL = 104, REG_CTRL = 40;
  static_assert((2 * REG_SOFTMAX + REG_FILL + REG_CTRL) * 128 <= THREADS * REG_LAUNCH,
                "register split");
  static_assert(SMEM <= 232448, "shared memory budget");
  static constexpr uint32_t TM_S = 0, TM_O = 256;
  // At d = 64 the columns behind O_1 hold P_0 and P_1, so S_s of the next tile can be
  // issued as soon as the softmax holds this tile's in registers; at d = 128 P_s takes
  // the place of S_s.
  static constexpr bool DEC = D == 64;
  static constexpr uint32_t TM_P = DEC ? TM_O + 2 * D : TM_S, P_STRIDE = DEC ? 64 : 128;
  static constexpr uint32_t TMEM_COLS = 512;
  // fp16 operands, fp32 result: as idesc_bf16_f32 with the formats' fields zero
  static constexpr uint32_t kFormats = (1u << 7) | (1u << 10);
  static constexpr uint32_t IDESC_S = idesc_bf16_f32(128, BN, false, false) & ~kFormats;
  static constexpr uint32_t IDESC_PV = idesc_bf16_f32(128, D, false, true) & ~kFormats;
};

enum {
  B_Q = 0,        // softmax threads -> MMA: Q in shared memory
  B_S_FULL = 1,   // [2] MMA -> softmax
  B_P_FULL = 3,   // [2] softmax -> MMA: P_s in TMEM
  B_PV_DONE = 5,  // [2] MMA -> epilogue
  B_P_HALF = 7,   // [2] softmax -> MMA: keys 0-63 of P_s in TMEM and O_s rescaled
  B_MMA_DONE = 9,
  B_SCALE = 10,    // [SCALE_TILES] slot filling -> softmax: the scales of a tile
  B_S_READ = 14,   // [2] softmax -> MMA (d = 64): S_s is in registers
  B_SCAN = 16,     // the scan of the value scales -> all
  B_KV_FULL = 17,  // [STAGES], then kv_empty [STAGES]
};
static_assert(8 * (B_KV_FULL + 2 * Wide<64>::STAGES) + 16 <= 256, "barrier block");
static_assert(Wide<64>::STAGES <= 7 && Wide<128>::STAGES <= 7, "reuse of the scales' ring");

// A piece of a unit: tiles [t0, t0 + max(c0, c1)) of it, of which subtile s sees the
// first c_s.
struct __align__(16) Segment {
  int row0, n, len, b;  // the sequence
  int h, rb;            // head, row block (tb tokens each)
  int t0, c0, c1;
  int part;             // -1: the whole unit; else where its rows go in the workspace
  int unused[2];
};
static_assert(sizeof(Segment) == 48, "three 16-byte loads");

// What the idle warps find out about the value scales of a piece's blocks: their largest
// and smallest (biased) exponent, and the passes over its tiles that they ask for.
struct Scan {
  int hi, lo;
  unsigned set[2];  // bit i: there are blocks of exponent hi - i (only where hi - lo is large)
  int passes;
  int b[kMaxPasses];
};
static_assert(sizeof(Scan) == 32, "room in shared memory");

// Where the rows of pieces go: LSE [places, ROWS], then O [places, ROWS, d], behind the
// records.
struct PieceView {
  float* lse;
  float* o;
};
__device__ __forceinline__ PieceView piece_view(const CacheFwdParams& p) {
  float* lse = reinterpret_cast<float*>(static_cast<char*>(p.wide_workspace) +
                                        (((size_t)p.wide_ctas * sizeof(Record) + 255) & ~(size_t)255));
  return PieceView{lse, lse + (size_t)p.wide_ctas * 2 * Wide<128>::ROWS};
}

// Behind them: the number of pieces (256 bytes), then the pieces.
struct PlanView {
  int* pieces;
  Segment* seg;
};
__device__ __forceinline__ PlanView plan_view(const CacheFwdParams& p, int d) {
  char* at = reinterpret_cast<char*>(piece_view(p).o + (size_t)p.wide_ctas * 2 * Wide<128>::ROWS * d);
  return PlanView{reinterpret_cast<int*>(at), reinterpret_cast<Segment*>(at + 256)};
}

constexpr int kMinTiles = 8;  // a piece of fewer tiles would not repay its start and merge

// The plan: one CTA writes a descriptor for each piece, in about 4 us, behind which a
// piece starts 0.7 us after its CTA.  (With every CTA of the attention finding its own
// piece that took 3 to 5 us each time: 16 sequences of 1 to 1000 tokens, two rounds of
// CTAs, 81.5 us against 79.0; 116 of 1320 tokens, one head of two, nine rounds, 192 us
// against 165.  With 1024 threads instead of 256 the plan took 1.5 us longer.)
// Sequences (up to 256 of them) are taken from the longest to the shortest, so that the
// last pieces to start are short ones: 16 sequences of 70 to 128 tokens behind 300 to 7000,
// 16 heads, d = 128, 99 us as they come and 80 us so.  Row blocks are taken from the last,
// which sees the most keys, to the first, a block's pieces head by head; 256 sequences at a time, then 256 of their
// row blocks.  Two passes: all tiles, which give the pieces' size, and the pieces.
struct Plan {
  static constexpr int T = 256;
  long long part[T / 32];
  long long start[T];            // row blocks of the sequences before
  int row0[T], n[T], len[T], b[T], blocks[T];
  alignas(16) unsigned key[T];
  long long first[T];            // pieces of the row blocks before
  int seq[T], rb[T], tiles[T];   // of a row block
};

// the sum of v over the threads before this one, and over all
__device__ __noinline__ long long sum_before(long long v, long long* part, long long* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long upto = v;
#pragma unroll
  for (int w = 1; w < 32; w <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, upto, w);
    if (lane >= w) upto += o;
  }
  if (lane == 31) part[warp] = upto;
  __syncthreads();
  long long all = lane < Plan::T / 32 ? part[lane] : 0, low = lane < warp ? all : 0;
#pragma unroll
  for (int w = Plan::T / 64; w > 0; w >>= 1) {
    all += __shfl_xor_sync(0xffffffffu, all, w);
    low += __shfl_xor_sync(0xffffffffu, low, w);
  }
  __syncthreads();
  *total = __shfl_sync(0xffffffffu, all, 0);
  return upto - v + __shfl_sync(0xffffffffu, low, 0);
}
// the last i < n with at[i] <= x, of ascending at with at[0] <= x
__device__ __forceinline__ int last_at_most(const long long* at, int n, long long x) {
  int lo = 0;
  while (n - lo > 1) {
    const int mid = (lo + n) >> 1;
    if (at[mid] <= x)
      lo = mid;
    else
      n = mid;
  }
  return lo;
}

__global__ void __launch_bounds__(Plan::T) cache_fwd_plan_kernel(const CacheFwdParams p) {
  constexpr int BN = Wide<128>::BN, BM = Wide<128>::BM;
  static_assert(Wide<64>::BN == BN && Wide<64>::BM == BM, "tile");
  extern __shared__ uint8_t smem_raw[];
  Plan& plan = *reinterpret_cast<Plan*>(smem_raw);
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const int B = p.c.B, H = p.c.H, G = p.G, tb = p.wide_tokens, T = Plan::T, t = threadIdx.x;
  const PlanView out = plan_view(p, p.c.d);
  Record* records = reinterpret_cast<Record*>(p.wide_workspace);
  for (int i = t; i < p.wide_ctas; i += T) records[i] = Record{0, 0, 0, 0, 0, 0};
  long long tiles = 0, blocks = 0, pieces = 0, most = 0, ng = 0;
  bool room = true;
  int mine = 0;  // tiles of this thread's row block
#pragma unroll 1
  for (int pass = 0; pass < 2; ++pass) {
    blocks = 0;
#pragma unroll 1
    for (int c0 = 0; c0 < B; c0 += T) {
      if (pass == 0 || B > T) {
        CacheSeq x{};
        int nb = 0;
        if (c0 + t < B) {
          if (!cache_seq(p.c, B - 1 - c0 - t, &x)) {
            if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD);
          } else if (x.n * G > p.narrow_rows) {
            nb = (x.n + tb - 1) / tb;
          }
        }
        __syncthreads();  // the last ones have been read
        int at = t;
        if (B > 1 && B <= T) {
          // tiles, then the place (a length is below 2^31): no two are alike
          const unsigned key = (nb > 0 ? ((unsigned)x.len + BN - 1) / BN << 8 : 0u) | (T - 1 - t);
          plan.key[t] = t < B ? key : 0u;
          __syncthreads();
          if (t < B) {
            at = 0;
#pragma unroll 4
            for (int i = 0; i < B; i += 4) {
              const uint4 k = *reinterpret_cast<const uint4*>(&plan.key[i]);
              at += (k.x > key) + (k.y > key) + (k.z > key) + (k.w > key);
            }
          }
        }
        plan.row0[at] = x.row0, plan.n[at] = x.n, plan.len[at] = x.len;
        plan.b[at] = B - 1 - c0 - t, plan.blocks[at] = nb;
        __syncthreads();
        plan.start[t] = sum_before(plan.blocks[t], plan.part, &ng);
      }
#pragma unroll 1
      for (long long g0 = 0; g0 < ng; g0 += T) {
        const bool on = g0 + t < ng;
        if (pass == 0 || B > T || ng > T) {
          __syncthreads();
          mine = 0;
        }
        if (on && (pass == 0 || B > T || ng > T)) {
          const int seq = last_at_most(plan.start, min(T, B - c0), g0 + t);
          const int n = plan.n[seq], len = plan.len[seq];
          const int rb = (n + tb - 1) / tb - 1 - (int)(g0 + t - plan.start[seq]);
          const int limit = max(1, p.causal ? len - n + min(n, (rb + 1) * tb) : len);
          // (one that sees nothing counts as one tile, to be written)
          mine = (limit + BN - 1) / BN;
          plan.seq[t] = seq, plan.rb[t] = rb, plan.tiles[t] = mine;
        }
        if (pass == 0) {
          tiles += mine;
          continue;
        }
        // parts of a unit: at most one more than the SMs, so the products below stay
        // below 2^32
        auto parts_of = [&](int n) {
          return n <= most ? 1 : (int)(((unsigned)n + (unsigned)most - 1) / (unsigned)most);
        };
        long long all;
        plan.first[t] = sum_before(on ? (long long)parts_of(mine) * H : 0, plan.part, &all);
        __syncthreads();
        // the grid has room for every batch whose offsets ascend
        room = room && pieces + all <= p.wide_grid;
        if (!room) {
          if (t == 0 && p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD);
          all = 0;
        }
        for (int i = t; i < all; i += T) {
          const int x = last_at_most(plan.first, (int)min((long long)T, ng - g0), i);
          const int seq = plan.seq[x], rb = plan.rb[x], n_tiles = plan.tiles[x];
          const int k = parts_of(n_tiles);
          int h = i - (int)plan.first[x], part = 0, take = n_tiles;
          const int n = plan.n[seq], len = plan.len[seq];
          Segment g{};
          g.row0 = plan.row0[seq], g.n = n, g.len = len, g.b = plan.b[seq];
          if (k > 1) {
            part = h % k, h /= k;
            g.t0 = (int)((unsigned)part * (unsigned)n_tiles / (unsigned)k);
            take = (int)((unsigned)(part + 1) * (unsigned)n_tiles / (unsigned)k) - g.t0;
          }
          g.h = h, g.rb = rb;
          // tiles that the subtiles see: up to their last row's limit
          const int rows = min(tb, n - rb * tb) * G;
          auto sees = [&](int last_row) {
            const int j = rb * tb + p.by_G.div(last_row);
            return (max(0, p.causal ? len - n + j + 1 : len) + BN - 1) / BN;
          };
          g.c0 = max(0, min(take, sees(min(rows, BM) - 1) - g.t0));
          g.c1 = rows > BM ? max(0, min(take, sees(rows - 1) - g.t0)) : 0;
          // A unit of k > 1 pieces owns k - 1 records and 2 (k - 1) >= k places for rows,
          // counted over the units before it: at most one record and two places per SM
          const long long place =
              pieces + plan.first[x] + (long long)h * k - ((blocks + g0 + x) * H + h);
          g.part = -1;
          if (k > 1) {
            g.part = (int)(2 * place) + part;
            if (part == 0 && place < p.wide_ctas)
              records[place] = Record{k, rows, h, g.row0, rb * tb * G, (int)(2 * place)};
          }
          out.seg[pieces + i] = g;
        }
        pieces += all;
      }
      blocks += ng;
    }
    if (pass == 0) {
      sum_before(tiles, plan.part, &tiles);
      tiles *= H;
      // (a 64-bit division takes ten times as long)
      const long long share = tiles < 0x7fffffff
                                  ? ((unsigned)tiles + p.wide_ctas - 1) / (unsigned)p.wide_ctas
                                  : (tiles + p.wide_ctas - 1) / p.wide_ctas;
      most = max((long long)kMinTiles, share);
    }
  }
  if (t == 0) *out.pieces = (int)pieces;
}

template <int D, bool E5M2>
__global__ void __launch_bounds__(Wide<D>::THREADS, 1)
    cache_fwd_wide_kernel(const CacheFwdParams p) {
  using C = Wide<D>;
  constexpr int ST = C::STAGES;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int G = p.G;

  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  asm volatile("griddepcontrol.wait;" ::: "memory");  // the plan
  const PlanView plan = plan_view(p, D);
  Segment seg;
  {
    const int4* from = reinterpret_cast<const int4*>(plan.seg + blockIdx.x);
    const int4 x = __ldcg(from), y = __ldcg(from + 1), z = __ldcg(from + 2);
    seg = Segment{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w, z.x, z.y, {}};
  }
  if ((int)blockIdx.x >= __ldcg(plan.pieces)) return;
  const uint32_t bar0 = sbase + C::OFF_BAR;
  auto bar = [&](int i) { return bar0 + 8u * (uint32_t)i; };
  const uint32_t kv_full0 = bar(B_KV_FULL), kv_empty0 = bar(B_KV_FULL + ST);
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + 8 * (B_KV_FULL + 2 * ST));
  volatile uint32_t* abort_flag = tmem_slot + 1;
  volatile uint32_t* poison = tmem_slot + 2;        // a NaN was kept out of some rows' sums
  volatile Scan* scan = reinterpret_cast<volatile Scan*>(smem + C::OFF_SCAN);
  const WaitCtx wctx{abort_flag, p.c.err};
  float4* scales = reinterpret_cast<float4*>(smem + C::OFF_SCALE);

  if (threadIdx.x == 32) {
    mbar_init(bar(B_Q), 256);
    for (int s = 0; s < 2; ++s) {
      mbar_init(bar(B_S_FULL + s), 1);
      mbar_init(bar(B_P_FULL + s), 128);
      mbar_init(bar(B_P_HALF + s), 128);
      mbar_init(bar(B_PV_DONE + s), 1);
      mbar_init(bar(B_S_READ + s), 128);
    }
    mbar_init(bar(B_MMA_DONE), 1);
    mbar_init(bar(B_SCAN), 1);
    scan->hi = 0, scan->lo = 255;
    scan->set[0] = scan->set[1] = 0u;
    for (int i = 0; i < C::SCALE_TILES; ++i) mbar_init(bar(B_SCALE + i), C::PIECES);
    for (int i = 0; i < ST; ++i) {
      mbar_init(kv_full0 + 8u * i, C::N_FILL);
      mbar_init(kv_empty0 + 8u * i, 1);
    }
    *abort_flag = 0u;
    *poison = 0u;
    fence_mbar_init();
  }
  if (warp == C::W_MMA) {
    tmem_alloc(smem_u32(tmem_slot), C::TMEM_COLS);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const int b = seg.b, h = seg.h, t0 = seg.t0, rb = seg.rb;
  const int len = seg.len, n_new = seg.n, row0 = seg.row0, part = seg.part;
  const int n_rows = min(p.wide_tokens, n_new - rb * p.wide_tokens) * G;  // of the unit
  // keys seen by row r of the unit
  const int seen0 = p.causal ? len - n_new + rb * p.wide_tokens + 1 : len;
  auto limit_of = [&](int r) {
    return max(0, min(len, p.causal ? seen0 + p.by_G.div(r) : seen0));
  };
  const int n_tiles = max(seg.c0, seg.c1);
  const int lim_lo = limit_of(0), lim_hi = limit_of(n_rows - 1);
  // Several passes run through all of the tiles, one after the other
  auto scanned = [&]() {
    return mbar_wait(bar(B_SCAN), 0, wctx, ERR_SITE_CACHE_FWD + 15);
  };
  auto tiles_of = [&](int c) {  // of a subtile, over all passes
    const int passes = scan->passes;
    return passes == 1 || c == 0 ? c : passes * n_tiles;
  };

  if (warp > C::W_MMA) {
    regs_dec<C::REG_CTRL>();
    // ---------------------------------------------------------------- scan of the value scales
    constexpr int N = 96;
    const int me = (int)threadIdx.x - (C::W_MMA + 1) * 32;
    const int end = min(lim_hi, (t0 + n_tiles) * C::BN);
    const int past = end > 0 ? ((end - 1) >> p.c.block_log2) + 1 : 0;
    int hi = 0, lo = 255;
    for (int again = 0;; ++again) {  // the second time (rare) for the set
      unsigned set0 = 0u, set1 = 0u;
      int most = 0, least = 255;
#pragma unroll 1
      for (int i0 = ((t0 * C::BN) >> p.c.block_log2) + me; i0 < past; i0 += 2 * N) {
        int page[2];
        float vs[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
          page[k] = i0 + k * N < past
                        ? p.c.block_table[(long long)b * p.c.table_width + i0 + k * N]
                        : -1;
#pragma unroll
        for (int k = 0; k < 2; ++k)
          vs[k] = page[k] >= 0 && page[k] < p.c.num_blocks
                      ? p.c.v_scale[(long long)page[k] * p.c.H + h]
                      : -1.f;
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          if (!(vs[k] > 0.f)) continue;
          const int e = (int)(__float_as_uint(vs[k]) >> 23), i = hi - e;
          most = max(most, e), least = min(least, e);
          const unsigned bit = 1u << (i & 31);
          if (i < 32)
            set0 |= bit;
          else if (i <= -(int)kNothing)
            set1 |= bit;
        }
      }
      if (again) {
        atomicOr(const_cast<unsigned*>(&scan->set[0]), set0);
        atomicOr(const_cast<unsigned*>(&scan->set[1]), set1);
      } else {
        atomicMax(const_cast<int*>(&scan->hi), most);
        atomicMin(const_cast<int*>(&scan->lo), least);
      }
      named_bar_sync(1, N);
      hi = scan->hi, lo = scan->lo;
      if (again || hi - lo <= kWindow) break;
    }
    if (me == 0) {
      int passes = 1;
      scan->b[0] = lo <= hi ? lo : 127;
      if (hi - lo > kWindow) {  // from the smallest on
        passes = 0;
        unsigned long long set = (unsigned long long)scan->set[1] << 32 | scan->set[0];
        while (set != 0ull && passes < kMaxPasses) {
          const int i = 63 - __clzll((long long)set);
          scan->b[passes++] = hi - i;
          set = i > kWindow ? set & ((1ull << (i - kWindow)) - 1ull) : 0ull;
        }
      }
      scan->passes = passes;
      mbar_arrive(bar(B_SCAN));
    }
  } else if (warp >= C::W_FILL && warp < C::W_FILL + C::N_FILL) {
    regs_dec<C::REG_FILL>();
    // ---------------------------------------------------------------- slot filling
    // Warp w fills rows [32 w, 32 w + 32) of every slot: two pieces of 16 tokens.
    const int bs = p.c.block_size;
    const int me = warp - C::W_FILL;
    // lane i of a set of 16 tiles holds the place and scales of this warp's piece i & 1 of
    // tile i / 2.  They are fetched in steps, none of which waits for its own loads (in one
    // step: 16 sequences of 1 to 1000 tokens 82.5 us, against 81.5).
    struct Info {
      int piece;        // number of its 16 tokens in the pool (-1: nothing visible there)
      float ks, lv, w;  // as the softmax takes them
    };
    auto pass_of = [&](int j) { return (j >= n_tiles ? 1 : 0) + (j >= 2 * n_tiles ? 1 : 0); };
    auto key_of = [&](int j0) {
      const int j = j0 + (lane >> 1);
      return (t0 + j - pass_of(j) * n_tiles) * C::BN + me * 32 + (lane & 1) * 16;
    };
    auto page_of = [&](int j0) {
      const int key = key_of(j0);
      return key < lim_hi ? p.c.block_table[(long long)b * p.c.table_width + (key >> p.c.block_log2)]
                          : 0;
    };
    auto scales_of = [&](int j0, int page) {  // ks, lv: the scales themselves
      Info r{-1, 1.f, 0.f, 0.f};
      const int key = key_of(j0);
      if (key >= lim_hi) return r;
      if (page < 0 || page >= p.c.num_blocks) {
        if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD + 1);
        return r;
      }
      const int slice = page * p.c.H + h;
      r.piece = (slice << (p.c.block_log2 - 4)) + ((key & (bs - 1)) >> 4);  // 1 KB or more each
      r.ks = p.c.k_scale[slice];
      r.lv = p.c.v_scale[slice];
      return r;
    };
    auto finish = [&](Info r, int j0) {  // the scales as the softmax takes them
      const int pass = pass_of(j0 + (lane >> 1));
      const int e = (int)(__float_as_uint(r.lv) >> 23), base = scan->b[pass];
      // of this pass; or of none, as the values are next to nothing
      const bool in = e >= base && e <= base + kWindow;
      const bool nothing = pass == 0 && e < scan->hi + (int)kNothing;
      float lv = -INFINITY;
      if (r.piece >= 0) lv = nothing ? kNothing : in ? lg2(r.lv) - (float)(base - 127) : lv;
      r.ks = r.piece < 0 ? 1.f : r.ks * p.scale_log2;
      r.lv = lv;
      r.w = lv == -INFINITY ? 0.f : ex2(-lv);
      return r;
    };
    constexpr int LD = D / 32;  // 16-byte loads per lane and piece
    // a load instruction covers whole rows; eight lanes of a store phase hold the
    // same four 16-byte columns of two neighbouring rows, which the swizzle puts
    // into different banks
    const int row4 = D == 128 ? (lane >> 4) * 2 + ((lane >> 2) & 1) : lane >> 2;
    const int col16 = D == 128 ? ((lane >> 3) & 1) * 4 + (lane & 3) : lane & 3;
    constexpr int ROWS_LD = D == 128 ? 4 : 8;  // rows per load instruction
    const int lane_src = row4 * D + col16 * 16;
    // a lane's 16 codes become 32 bytes: two neighbouring 16-byte columns of its row
    const uint32_t lane_dst = (uint32_t)((col16 >> 2) * C::HALF + (me * 32 + row4) * 128);
    uint4 buf[2][2][LD];  // [K, V][piece]
    int at[2];  // the pieces of the next tile
    auto load = [&](int value) {
#pragma unroll
      for (int pc = 0; pc < 2; ++pc) {
        const uint8_t* src = (value ? p.c.v : p.c.k) + (long long)at[pc] * (16 * D) + lane_src;
#pragma unroll
        for (int i = 0; i < LD; ++i)
          buf[value][pc][i] = at[pc] < 0 ? make_uint4(0u, 0u, 0u, 0u)
                                         : __ldg(reinterpret_cast<const uint4*>(src + i * ROWS_LD * D));
      }
    };
    auto look_up = [&](int j, const Info& set) {
#pragma unroll
      for (int pc = 0; pc < 2; ++pc) at[pc] = __shfl_sync(0xffffffffu, set.piece, (j & 15) * 2 + pc);
    };
    Info now{-1, 1.f, -INFINITY, 0.f}, next = now;
    int page = 0;
    bool ok = true;
    if (n_tiles > 0) {
      now = scales_of(0, page_of(0));
      look_up(0, now);
      load(0);
      load(1);
      ok = __all_sync(0xffffffffu, scanned());
      now = finish(now, 0);
    }
    int first = t0;  // of tile 0, less the tiles of the passes before
    const int n_max = ok && n_tiles > 0 ? scan->passes * n_tiles : 0;
    for (int j = 0; ok && j < n_max; ++j) {
      if (first + j == t0 + n_tiles) first -= n_tiles;
      {  // the tile's scales
        // the slot of K_j is free: with it, the scales' (see SCALE_TILES)
        const int i = 2 * j, use = i / ST;
        ok = use == 0 ||
             __all_sync(0xffffffffu, mbar_wait(kv_empty0 + 8u * (i % ST), (use - 1) & 1, wctx,
                                               ERR_SITE_CACHE_FWD + 4));
        if (!ok) break;
        const int ring = j % C::SCALE_TILES;
        if ((lane >> 1) == (j & 15)) {
          scales[ring * C::PIECES + me * 2 + (lane & 1)] = make_float4(now.ks, now.lv, now.w, 0.f);
          mbar_arrive(bar(B_SCALE + ring));
        }
      }
      if ((j & 15) == 0) page = page_of(j + 16);
      if ((j & 15) == 8) next = scales_of(j + 8, page);
      if ((j & 15) == 15) now = finish(next, j + 1);  // the loads below are for its first tile
      look_up(j + 1, now);
#pragma unroll
      for (int value = 0; value < 2; ++value) {
        const int i = 2 * j + value, use = i / ST;
        const int kv_slot = i % ST;
        if (value) {
          ok = use == 0 ||
               __all_sync(0xffffffffu, mbar_wait(kv_empty0 + 8u * kv_slot, (use - 1) & 1, wctx,
                                                 ERR_SITE_CACHE_FWD + 4));
          if (!ok) break;
          const int key0 = (first + j) * C::BN + me * 32 + row4;
          if ((first + j) * C::BN + me * 32 + 32 > lim_lo) {  // some row does not see all of it
            bool nan = false;
#pragma unroll
            for (int pc = 0; pc < 2; ++pc)
#pragma unroll
              for (int x = 0; x < LD; ++x) {
                uint32_t* w = &buf[1][pc][x].x;
#pragma unroll
                for (int y = 0; y < 4; ++y) {
                  if (key0 + pc * 16 + x * ROWS_LD >= lim_hi) w[y] = 0u;  // stale, whatever it is
                  const uint32_t m = nan_codes<E5M2>(w[y]);
                  nan |= m != 0u;
                  w[y] = clear_codes(w[y], m);
                }
              }
            if (nan) *poison = 1u;
          }
        }
        const uint32_t dst = sbase + C::OFF_KV + kv_slot * C::TILE + lane_dst;
#pragma unroll
        for (int pc = 0; pc < 2; ++pc)
#pragma unroll
          for (int x = 0; x < LD; ++x) {
            const uint32_t* w = &buf[value][pc][x].x;
            const int row = pc * 16 + x * ROWS_LD;  // + 32 me + row4; the swizzle takes it mod 8
            const uint32_t line = dst + row * 128;
#pragma unroll
            for (int y = 0; y < 2; ++y) {
              const uint32_t c = (uint32_t)(((col16 & 3) * 2 + y) ^ ((row + row4) & 7));
              uint32_t o[4];
              codes4_to_f16<E5M2>(w[2 * y], o[0], o[1]);
              codes4_to_f16<E5M2>(w[2 * y + 1], o[2], o[3]);
              st_shared_v4(line + (c << 4), o[0], o[1], o[2], o[3]);
            }
          }
        fence_proxy_async_smem();  // the MMAs read through the async proxy
        __syncwarp();
        if (lane == 0) mbar_arrive(kv_full0 + 8u * kv_slot);
        if (j + 1 < n_max) load(value);
      }
    }
    __syncwarp();
  } else if (warp == C::W_MMA) {
    regs_dec<C::REG_CTRL>();
    // ---------------------------------------------------------------- MMA issuer (whole warp)
    auto kv_wait = [&](int i) {
      return __all_sync(0xffffffffu, mbar_wait(kv_full0 + 8u * (i % ST), (i / ST) & 1, wctx,
                                               ERR_SITE_CACHE_FWD + 5));
    };
    auto issue_s = [&](int s, int j) {  // S_s = Q_s K_j^T
      const uint32_t a = sbase + C::OFF_Q + s * C::TILE;
      const uint32_t bk = sbase + C::OFF_KV + ((2 * j) % ST) * C::TILE;
#pragma unroll
      for (int kk = 0; kk < D / 16; ++kk) {
        const uint32_t off = (kk >> 2) * C::HALF + (kk & 3) * 32;
        mma_bf16_ss_w(tmem + C::TM_S + s * 128, sdesc_sw128(a + off, 16, 1024),
                      sdesc_sw128(bk + off, 16, 1024), C::IDESC_S, kk > 0);
      }
      mma_commit_w(bar(B_S_FULL + s));
    };
    auto issue_pv = [&](int s, int j, int half) {  // O_s += P_s V_j over 64 keys
      const uint32_t bv = sbase + C::OFF_KV + ((2 * j + 1) % ST) * C::TILE;
#pragma unroll
      for (int k = 0; k < C::BN / 32; ++k) {
        const int kk = half * (C::BN / 32) + k;
        mma_bf16_ts_w(tmem + C::TM_O + s * D, tmem + C::TM_P + s * C::P_STRIDE + kk * 8,
                      sdesc_sw128(bv + kk * 16 * 128, C::HALF, 1024), C::IDESC_PV,
                      (j > 0 || kk > 0));
      }
      if (half == 1) mma_commit_w(bar(B_PV_DONE + s));
    };
    bool ok = __all_sync(0xffffffffu, mbar_wait(bar(B_Q), 0, wctx, ERR_SITE_CACHE_FWD + 6) &&
                                          scanned());
    const int nt0 = ok ? tiles_of(seg.c0) : 0, nt1 = ok ? tiles_of(seg.c1) : 0;
    const int n_max = max(nt0, nt1);
    if (ok && n_max > 0) {
      ok = kv_wait(0);
      if (ok) {
        tc_fence_after();
        if (nt0 > 0) issue_s(0, 0);
        if (nt1 > 0) issue_s(1, 0);
        mma_commit_w(kv_empty0);
      }
    }
    for (int j = 0; C::DEC && ok && j < n_max; ++j) {
      // S_s(j + 1) once the softmax holds S_s(j) in registers; O_s += P_s V_j once P_s(j)
      // is in its own columns.  The pipe runs them in issue order.
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (ok && j + 1 < (s ? nt1 : nt0)) {
          ok = kv_wait(2 * (j + 1)) &&
               __all_sync(0xffffffffu, mbar_wait(bar(B_S_READ + s), j & 1, wctx,
                                                 ERR_SITE_CACHE_FWD + 13));
          if (ok) {
            tc_fence_after();
            issue_s(s, j + 1);
          }
        }
      }
      if (!ok) break;
      if (j + 1 < n_max) mma_commit_w(kv_empty0 + 8u * ((2 * (j + 1)) % ST));
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        if (ok && j < (s ? nt1 : nt0)) {
          ok = kv_wait(2 * j + 1) &&
               __all_sync(0xffffffffu, mbar_wait(bar(B_P_HALF + s), j & 1, wctx,
                                                 ERR_SITE_CACHE_FWD + 7));
          if (ok) {
            tc_fence_after();
            issue_pv(s, j, 0);
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_P_FULL + s), j & 1, wctx,
                                                   ERR_SITE_CACHE_FWD + 8));
          }
          if (ok) {
            tc_fence_after();
            issue_pv(s, j, 1);
          }
        }
      }
      if (!ok) break;
      mma_commit_w(kv_empty0 + 8u * ((2 * j + 1) % ST));
    }
    for (int j = 0; !C::DEC && ok && j < n_max; ++j) {
      const bool next = j + 1 < n_max;
      bool k_next = false;
      ok = kv_wait(2 * j + 1);
#pragma unroll
      for (int s = 0; s < 2; ++s) {
        const int nts = s ? nt1 : nt0;
        if (ok && j < nts) {
          ok = __all_sync(0xffffffffu, mbar_wait(bar(B_P_HALF + s), j & 1, wctx,
                                                 ERR_SITE_CACHE_FWD + 7));
          if (ok) {
            tc_fence_after();
            issue_pv(s, j, 0);
            ok = __all_sync(0xffffffffu, mbar_wait(bar(B_P_FULL + s), j & 1, wctx,
                                                   ERR_SITE_CACHE_FWD + 8));
          }
          if (ok) {
            tc_fence_after();
            issue_pv(s, j, 1);
          }
        }
        if (ok && j + 1 < nts) {  // after the PV above: S_s is overwritten in pipe order
          if (!k_next) {
            ok = kv_wait(2 * (j + 1));
            k_next = true;
          }
          if (ok) issue_s(s, j + 1);
        }
      }
      if (!ok) break;
      if (next) mma_commit_w(kv_empty0 + 8u * ((2 * (j + 1)) % ST));
      mma_commit_w(kv_empty0 + 8u * ((2 * j + 1) % ST));
    }
    // drain: every MMA issued has finished before TMEM is freed
    mma_commit_w(bar(B_MMA_DONE));
    mbar_drain(bar(B_MMA_DONE), 0, wctx, ERR_SITE_CACHE_FWD + 9);
    __syncwarp();
  } else {
    // ---------------------------------------------------------------- softmax (warps 0-7)
    regs_inc<C::REG_SOFTMAX>();
    const int s = warp >> 2;
    const int t = threadIdx.x & 127;  // row in the subtile == TMEM lane
    const int row = s * C::BM + t;  // of the unit
    const bool valid = row < n_rows;
    const int lim = valid ? limit_of(row) : 0;
    const int my_c = s ? seg.c1 : seg.c0;
    const int my_lo = limit_of(s * C::BM);  // keys that every row of the subtile sees
    const uint32_t lane_off = (uint32_t)((warp & 3) * 32) << 16;
    const uint32_t tS = tmem + lane_off + C::TM_S + s * 128;
    const uint32_t tO = tmem + lane_off + C::TM_O + s * D;
    const uint32_t tP = tmem + lane_off + C::TM_P + s * C::P_STRIDE;
    // A row of q and o is LPR pieces of 16 bytes; a warp moves RPI of its 32 rows at a
    // time, piece by lane (a thread that moved its own row would touch 32 lines with
    // every instruction).
    constexpr int LPR = D / 8, RPI = 32 / LPR, IT = 32 / RPI;
    const int sub = lane / LPR, piece = lane % LPR;
    // offsets of this thread's row in q, o and lse (-1: no such row); the lanes that
    // move the row take them from here
    long long q_off = -1, o_off = -1, lse_off = 0;
    if (valid) {
      const long long token = (long long)row0 + rb * p.wide_tokens + p.by_G.div(row);
      const long long hq = h * G + p.by_G.mod(row);
      q_off = token * p.q.st + hq * p.q.sh;
      o_off = token * p.o.st + hq * p.o.sh;
      lse_off = hq * p.c.total + token;
    }
    const uint32_t rows_smem = sbase + C::OFF_Q + s * C::TILE + (piece >> 3) * C::HALF;
    auto row_piece = [&](int i) {  // where piece `piece` of the warp's row i RPI + sub lies
      const int r = (warp & 3) * 32 + i * RPI + sub;
      return rows_smem + r * 128 + (((piece & 7) ^ (r & 7)) << 4);
    };
    // Q: copied as it is, then each thread multiplies its row by the power of two that
    // brings its largest element to [2^14, 2^15), as fp16 in place (exact down to 2^-29 of
    // that element, the quantum below it 2^-39).
    // (Loops that run once per piece are kept short: straight-line code of their length
    // is bound by its instruction fetches.)
#pragma unroll 4
    for (int i = 0; i < IT; ++i) {
      const long long off = __shfl_sync(0xffffffffu, q_off, i * RPI + sub);
      copy16_async(row_piece(i), p.q.p + (off >= 0 ? off + 8 * piece : 0), off >= 0);
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncwarp();
    auto own_piece = [&](int k) {
      return sbase + C::OFF_Q + s * C::TILE + (k >> 3) * C::HALF + t * 128 +
             (((k & 7) ^ (t & 7)) << 4);
    };
    uint32_t m2 = 0u;  // the largest elements in the halves of the words
#pragma unroll 4
    for (int k = 0; k < D / 8; ++k) {
      const uint4 x = ld_shared_v4(own_piece(k));
      m2 = __vmaxu2(m2, __vmaxu2(__vmaxu2(x.x & 0x7fff7fffu, x.y & 0x7fff7fffu),
                                 __vmaxu2(x.z & 0x7fff7fffu, x.w & 0x7fff7fffu)));
    }
    const uint32_t mx = max(m2 & 0xffffu, m2 >> 16);
    int e = (int)(mx >> 7);
    e = (mx == 0u || e == 255) ? 0 : min(14 - (e - 127), 126);
    const float mul = __uint_as_float((uint32_t)(e + 127) << 23);
    const float back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll 2
    for (int k = 0; k < D / 8; ++k) {
      const uint4 x = ld_shared_v4(own_piece(k));
      const uint32_t* w = &x.x;
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        asm("cvt.rn.f16x2.f32 %0, %1, %2;"
            : "=r"(o[i])
            : "f"(__uint_as_float(w[i] & 0xffff0000u) * mul), "f"(__uint_as_float(w[i] << 16) * mul));
      st_shared_v4(own_piece(k), o[0], o[1], o[2], o[3]);
    }
    fence_proxy_async_smem();
    mbar_arrive(bar(B_Q));
    const int my_nt = scanned() ? tiles_of(my_c) : 0;

    float r_run = -INFINITY, l_run = 0.f;  // the reference r, and l
    int first = t0;  // of tile 0, less the tiles of the passes before
    for (int j = 0;;) {
      const int stop = my_nt > my_c ? j + n_tiles : my_nt;  // the pass's
      for (; j < stop; ++j) {
        mbar_wait(bar(B_S_FULL + s), j & 1, wctx, ERR_SITE_CACHE_FWD + 10);
        mbar_wait(bar(B_SCALE + j % C::SCALE_TILES), (j / C::SCALE_TILES) & 1, wctx,
                  ERR_SITE_CACHE_FWD + 11);
        tc_fence_after();
        uint32_t u[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(tS + c * 32, u[c]);
        tmem_wait_ld();
#pragma unroll
        for (int c = 0; c < 4; ++c) reg_fence32(u[c]);
        const float4* sc = scales + (j % C::SCALE_TILES) * C::PIECES;
        float sv[128];
#pragma unroll
        for (int k = 0; k < 128; ++k) sv[k] = __uint_as_float(u[k >> 5][k & 31]);
        if (C::DEC) {  // its columns may take S_s(j + 1)
          tc_fence_before();
          mbar_arrive(bar(B_S_READ + s));
        }
        const int c0 = (first + j) * C::BN;
        if (c0 + C::BN > my_lo) {
          const int n = lim - c0;
#pragma unroll
          for (int k = 0; k < 128; ++k)
            if (k >= n) sv[k] = -INFINITY;
        }
        // the largest y: of each piece the largest product, then its scale (positive)
        float ks[C::PIECES], top[C::PIECES];
#pragma unroll
        for (int g = 0; g < C::PIECES; ++g) {
          const float* x = sv + g * 16;
          float m = fmax3(fmax3(x[0], x[1], x[2]), fmax3(x[3], x[4], x[5]), fmax3(x[6], x[7], x[8]));
          m = fmax3(m, fmax3(x[9], x[10], x[11]), fmax3(x[12], x[13], x[14]));
          const float2 kl = *reinterpret_cast<const float2*>(&sc[g]);
          ks[g] = fmaxf(kl.x * back, 1.17549435e-38f);
          top[g] = fmaf(fmaxf(m, x[15]), ks[g], kl.y);
        }
        const float m_blk = fmax3(fmax3(top[0], top[1], top[2]), fmax3(top[3], top[4], top[5]),
                                  fmaxf(top[6], top[7]));
        // (-inf) - (-inf) is NaN, which moves nothing
        const bool rescale = m_blk - r_run > kRoom;
        const float r_new = rescale ? (fabsf(m_blk) < kFar ? m_blk - kOff : m_blk) : r_run;
        const float shift = r_new == -INFINITY ? 0.f : -r_new;
        const float alpha = rescale ? ex2(r_run + shift) : 1.f;
        // p = 2^(s ks + (log2 vs - r)).  Far from zero, the rounding of y that the check
        // above saw is itself large: there p is formed from the rounded y
        const bool far = __any_sync(0xffffffffu, fabsf(shift) >= kFar);
        if (far) {  // warp-uniform, rare
#pragma unroll
          for (int g = 0; g < C::PIECES; ++g) {
            const float lv = sc[g].y;
#pragma unroll
            for (int i = 0; i < 16; ++i) sv[g * 16 + i] = fmaf(sv[g * 16 + i], ks[g], lv) + shift;
            ks[g] = 1.f;
          }
        }
        float lw = 0.f;
#pragma unroll
        for (int hh = 0; hh < 2; ++hh) {
          uint32_t pk[32];
#pragma unroll
          for (int g = 0; g < 4; ++g) {
            float l0 = 0.f, l1 = 0.f, l2 = 0.f, l3 = 0.f;
            const float c = far ? 0.f : sc[hh * 4 + g].y + shift;
#pragma unroll
            for (int i = 0; i < 16; i += 4) {
              const int k = g * 16 + i, kk = hh * 64 + k;
              float p0, p1, p2, p3;
              fma_x2(sv[kk], sv[kk + 1], ks[hh * 4 + g], c, p0, p1);
              fma_x2(sv[kk + 2], sv[kk + 3], ks[hh * 4 + g], c, p2, p3);
              p0 = ex2(p0);
              p1 = ex2(p1);
              p2 = ex2(p2);
              p3 = ex2(p3);
              add_x2(l0, l1, p0, p1, l0, l1);
              add_x2(l2, l3, p2, p3, l2, l3);
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[k / 2]) : "f"(p1), "f"(p0));
              asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(pk[k / 2 + 1]) : "f"(p3), "f"(p2));
            }
            lw = fmaf((l0 + l1) + (l2 + l3), sc[hh * 4 + g].z, lw);
          }
          if (C::DEC && hh == 0 && j > 0) {
            // O_s += P_s V_{j-1} has finished: P_s's columns are free and O_s complete
            mbar_wait(bar(B_PV_DONE + s), (j - 1) & 1, wctx, ERR_SITE_CACHE_FWD + 14);
            tc_fence_after();
          }
          tmem_st32(tP + hh * 32, pk);
          if (hh == 0) {
            if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll
              for (int c = 0; c < D / 32; ++c) {
                uint32_t o[32];
                tmem_ld32(tO + c * 32, o);
                tmem_wait_ld(o);
#pragma unroll
                for (int i = 0; i < 32; ++i) o[i] = __float_as_uint(__uint_as_float(o[i]) * alpha);
                tmem_st32(tO + c * 32, o);
              }
            }
            tmem_wait_st();
            tc_fence_before();
            mbar_arrive(bar(B_P_HALF + s));
          }
        }
        l_run = l_run * alpha + lw;
        r_run = r_new;
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(bar(B_P_FULL + s));
      }
      if (j == my_nt) break;
      // (rare) another pass, from another b
      first -= n_tiles;
      const int pass = j / n_tiles;
      float* lse_part = reinterpret_cast<float*>(smem + C::OFF_LSE) + threadIdx.x;
      const float more = l_run == 0.f ? -INFINITY : add_log2(r_run, l_run);
      *lse_part = pass == 1 ? more : log2_add(*lse_part, more);
      l_run = 0.f;
      r_run += (float)(scan->b[pass - 1] - scan->b[pass]);
    }

    // ------------------------------------------------------------ epilogue
    bool has = my_nt > 0 && !(l_run == 0.f);
    float inv = has ? 1.f / l_run : 0.f, up = ex2((float)(scan->b[0] - 127));
    float lse = has ? add_log2(r_run, l_run) : -INFINITY;
    if (__builtin_expect(my_nt > my_c, 0)) {  // several passes: O = 2^(r + b - LSE) acc
      const float more = lse, b_last = (float)(scan->b[scan->passes - 1] - 127);
      lse = log2_add(reinterpret_cast<float*>(smem + C::OFF_LSE)[threadIdx.x], more);
      has = !(lse == -INFINITY);
      inv = up = ex2(0.5f * (r_run + b_last - lse));
    }
    lse *= kLn2;
    if (my_nt > 0) {
      mbar_wait(bar(B_PV_DONE + s), (my_nt - 1) & 1, wctx, ERR_SITE_CACHE_FWD + 12);
      tc_fence_after();
    }
    // a whole unit's rows go to o as bf16, a piece's to the workspace as fp32
    const PieceView out = piece_view(p);
    const size_t place = (size_t)max(part, 0) * C::ROWS + row;
#pragma unroll 1
    for (int c = 0; c < D / 32; ++c) {
      uint32_t o[32];
      if (my_nt > 0) {  // subtile-uniform
        tmem_ld32(tO + c * 32, o);
        tmem_wait_ld(o);
      }
#pragma unroll
      for (int i = 0; i < 32; ++i)
        o[i] = has ? __float_as_uint(__uint_as_float(o[i]) * inv * up) : 0u;
      if (part < 0) {  // into Q_s's place, which no MMA reads any more
#pragma unroll
        for (int q4 = 0; q4 < 4; ++q4) {
          const int k = c * 4 + q4;
          uint32_t x[4];
#pragma unroll
          for (int e = 0; e < 4; ++e)
            x[e] = pack_bf16x2(__uint_as_float(o[q4 * 8 + 2 * e]),
                               __uint_as_float(o[q4 * 8 + 2 * e + 1]));
          st_shared_v4(own_piece(k), x[0], x[1], x[2], x[3]);
        }
      } else if (valid) {
#pragma unroll
        for (int q4 = 0; q4 < 8; ++q4)
          *reinterpret_cast<uint4*>(out.o + place * D + c * 32 + q4 * 4) =
              make_uint4(o[q4 * 4], o[q4 * 4 + 1], o[q4 * 4 + 2], o[q4 * 4 + 3]);
      }
    }
    if (part < 0) {
      __syncwarp();
#pragma unroll 4
      for (int i = 0; i < IT; ++i) {
        const uint4 x = ld_shared_v4(row_piece(i));
        const long long off = __shfl_sync(0xffffffffu, o_off, i * RPI + sub);
        if (off >= 0) *reinterpret_cast<uint4*>(p.o.p + off + 8 * piece) = x;
      }
    }
    if (valid) {
      if (part < 0)
        p.lse[lse_off] = lse;
      else
        out.lse[place] = lse;
    }
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  if (warp == C::W_MMA) {
    tc_fence_after();
    tmem_dealloc(tmem, C::TMEM_COLS);
  }
  if (*poison && warp < 8) {
    // rare: values that were NaN in keys that some rows see and others do not; they
    // were left out of the sums, and here reach the rows that do see them
    const int row = (int)threadIdx.x;
    if (row < n_rows) {
      const int bs = p.c.block_size;
      const long long at = (long long)row0 + rb * p.wide_tokens + p.by_G.div(row);
      uint16_t* o_row = p.o.p + at * p.o.st + (long long)(h * G + p.by_G.mod(row)) * p.o.sh;
      float* part_row = piece_view(p).o + ((size_t)max(part, 0) * C::ROWS + row) * D;
      const int from = max(t0 * C::BN, lim_lo & ~31);  // whole 32-row pieces were cleared
      const int to = min(limit_of(row), (t0 + n_tiles) * C::BN);
      for (int key = from; key < to; ++key) {
        const int page = p.c.block_table[(long long)b * p.c.table_width + (key >> p.c.block_log2)];
        if (page < 0 || page >= p.c.num_blocks) continue;
        const uint8_t* v = p.c.v + (((long long)page * p.c.H + h) * bs + (key & (bs - 1))) * D;
        for (int c = 0; c < D; ++c)
          if ((v[c] & 0x7fu) >= (E5M2 ? 0x7cu : 0x7fu)) {
            if (part < 0)
              o_row[c] = 0x7fffu;
            else
              part_row[c] = __uint_as_float(0x7fffffffu);
          }
      }
    }
  }
}

template <int D, bool E5M2>
cudaError_t launch(const CacheFwdParams& p, cudaStream_t stream) {
  using C = Wide<D>;
  static unsigned long long prepared[64];
  const cudaError_t e = prepare_once(prepared, [] {
    cudaError_t r = cudaFuncSetAttribute(cache_fwd_wide_kernel<D, E5M2>,
                                         cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
    if (r != cudaSuccess) return r;
    // the setmaxnreg split hands out at most the launch's registers
    cudaFuncAttributes fa;
    r = cudaFuncGetAttributes(&fa, cache_fwd_wide_kernel<D, E5M2>);
    if (r != cudaSuccess) return r;
    return fa.numRegs >= C::REG_LAUNCH ? cudaSuccess : cudaErrorInvalidConfiguration;
  });
  if (e != cudaSuccess) return e;
  cache_fwd_plan_kernel<<<1, Plan::T, sizeof(Plan), stream>>>(p);
  const cudaError_t r = cudaGetLastError();
  if (r != cudaSuccess) return r;
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)p.wide_grid);
  cfg.blockDim = dim3(C::THREADS);
  cfg.dynamicSmemBytes = C::SMEM;
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, cache_fwd_wide_kernel<D, E5M2>, p);
}

}  // namespace

int cache_fwd_wide_rows() { return Wide<128>::ROWS; }

// Room for every unit, and for the cuts: a unit of t tiles has at most
// 1 + t / (all tiles / SMs) pieces.  A sequence of n > narrow_rows / G tokens has
// ceil(n / tb) <= n / tb + 1 row blocks, which is also at most n / least for n <= tb and
// 2 n / (tb + 1) for n > tb.  (A CTA without a piece costs about 1 us of an SM.)
long long cache_fwd_wide_grid(const CacheParams& c, int G, int narrow_rows, int n_sm) {
  const long long total = c.total, tb = cache_fwd_wide_rows() / G, least = narrow_rows / G + 1;
  const long long blocks = std::min(total / tb + c.B, std::max(total / least, 2 * total / (tb + 1)));
  return blocks * c.H + n_sm;
}
size_t cache_fwd_wide_plan_bytes(long long grid) { return 256 + (size_t)grid * sizeof(Segment); }

cudaError_t launch_cache_fwd_wide(const CacheFwdParams& p, cudaStream_t stream) {
  if (p.c.d == 128) return p.c.format ? launch<128, true>(p, stream) : launch<128, false>(p, stream);
  return p.c.format ? launch<64, true>(p, stream) : launch<64, false>(p, stream);
}

}  // namespace fattn

// cache_fwd.cu -- attention over the paged 8-bit key/value cache, few query rows
// per key/value head (decoding, drafted tokens).
//
// The mathematics.  With codes k, v and scales ks, vs of key j's block, in base 2:
//   x_j = scale log2(e) ks_j (q . k_j),   O = sum_j 2^x_j vs_j v_j / sum_j 2^x_j.
// The value scale is folded into the exponent: y_j = x_j + log2 vs_j - b, b the log2 vs
// of the first block, and with a reference r carried along the keys (the running
// maximum of the online softmax, less 8, moved when a y exceeds it by more than 15)
//   acc = sum_j p_j v_j,  p_j = 2^(y_j - r),   l = sum_j p_j 2^(b - log2 vs_j):
// O = 2^b acc / l and LSE = ln2 (r + log2 l).  So blocks of different scales need no
// rescale of acc, and the weights p_j can be held in fp16: they lie at or below 2^15, the
// largest at or above 2^8, so weights down to 2^-22 of it keep 11 bits and what is
// flushed lies below 2^-33 of it.  (Where |y| >= 2^22 r is the maximum itself, as 8
// is then too near its rounding.)
// As a scale takes its part of that range, only blocks whose log2 vs lies within 10 of
// b share sums.  At another one the warp puts its sums aside, joins them with what is
// there by their log-sum-exp, and starts again from that block's scale.  A scale more
// than 2^60 below 2^b is taken as 2^(b - 60), which needs no new start: a block of zeros
// has the scale 2^-100.  With one block in eight 2^30 smaller the first case below takes
// 14 % longer, with one in eight of zeros 3 %.
// Codes are exact in fp16; q is down to 2^-29 of its row's largest element (each row is
// multiplied by the power of two that brings that to [2^14, 2^15)), sums and statistics
// are fp32.
//
// The bound is memory: every code is read once.  At the measured copy
// bandwidth an SM gets about 24 codes a clock, and a 16-key tile of keys and
// values (4 KB at d = 128) costs 174 clocks, of which the arithmetic below takes
// about half of the issue slots.  Measured: 4 sequences of 32768 tokens, 32 heads,
// d = 128 (1.07 GB) 163 us, 97 % of the measured copy bandwidth; 32 sequences of 512
// to 8192 tokens, 32 query and 8 key heads (185 MB) 41.5 us, 66 %: the start of a share
// (offsets, block table, first codes, one after the other) takes 3 us, its end and
// the merge 3 us; one sequence of 1000 tokens 8.6 us.  Three CTAs per SM and three ring
// slots a warp: with four CTAs the registers spilled (221 us for the first case), with
// two the loads in flight fell short (211 us).  With 1 to 16 rows per key/value head the
// tensor work is far too small for a 128-row tcgen05 tile and its trip through
// shared memory and TMEM; m16n8k16 mma.sync with the keys as the 16-row operand
// takes the codes straight from shared memory into registers:
//   S^T = K Q^T:   A = 16 keys x d codes, B = d x 8 query rows
//   O^T += V^T P^T: A = d x 16 keys,      B = 16 keys x 8 query rows
// The contraction index may be permuted at will (q is loaded to match), so a
// lane's share of a key is 16 consecutive bytes; P goes from the first
// product's layout to the second's by movmatrix.
//
// Work split.  A unit is (sequence, key/value head, block of R query rows); its
// keys come in chunks, one tile of 16 keys (d = 64: 32) for each of the CTA's four
// warps.
// The chunks of all units, in order, are cut into equal contiguous shares, one
// per CTA of a grid that fills the machine once, so ragged batches load every
// SM alike and no length is needed on the host.  A unit that lies inside one
// share is finished by its CTA; the pieces of one that does not are merged by a
// second kernel (at most two pieces per CTA, so the workspace does not depend
// on the lengths).  Each warp runs its own ring of TMA loads (box: 16 tokens of
// one block), addressed through page numbers and scales that its lanes fetch
// 32 tiles at a time.
#include <math.h>

#include <algorithm>

#include "cache_split.cuh"

namespace fattn {
namespace {

constexpr float kWindow = 10.f;    // log2 vs - b of the blocks that share sums
constexpr float kNothing = -60.f;  // what lies below it is taken as it

template <int D, int NT_>
struct Dec {
  static constexpr int NT = NT_;
  static constexpr int R = split_rows(NT);        // query rows per unit
  static constexpr int PARTS = D == 128 ? 1 : 2;  // of 16 keys in a warp's tile (4 KB with values)
  static constexpr int KEYS = 16 * PARTS;
  static constexpr int CHUNK = kWarps * KEYS;     // keys per CTA step
  static constexpr int PART = 16 * D;             // bytes of 16 keys or values: one TMA box
  static constexpr int TILE = KEYS * D;
  static constexpr int STAGE = 2 * TILE;          // keys and values
  // ring slots per warp, CTAs per SM: as much as the shared memory and registers take
  static constexpr int ST = D == 64 && NT == 1 ? 4 : D == 128 && NT == 2 ? 4 : 3;
  static constexpr int OFF_RED = kWarps * ST * STAGE;
  static constexpr int OFF_SCL = OFF_RED + kWarps * R * D * 4;  // [warps][ST] scales of a tile
  static constexpr int OFF_STAT = OFF_SCL + kWarps * ST * 16;
  static constexpr int OFF_BAR = OFF_STAT + kWarps * R * 4;
  static constexpr int SMEM = OFF_BAR + kWarps * ST * 8 + 16 + 1024;
  static constexpr int CTAS = split_ctas(D, NT);  // per SM
};

constexpr int kWideMerge = 8;  // merge blocks per CTA of the 256-row kernel

template <int D, bool E5M2, int NT>
__global__ void __launch_bounds__(128, Dec<D, NT>::CTAS)
    cache_fwd_kernel(const __grid_constant__ CUtensorMap tm_k,
                     const __grid_constant__ CUtensorMap tm_v, const CacheFwdParams p) {
  using C = Dec<D, NT>;
  constexpr int R = C::R;
  constexpr int KW = D / 16;   // 4-byte words of a key that a lane holds (16 values per step)
  constexpr int VW = D / 32;   // 4-byte words of a value row that a lane holds
  constexpr int MT = D / 16;   // 16-row tiles of O^T
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 1023u) & ~1023u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);    // [warps][R][D]
  float* stat = reinterpret_cast<float*>(smem + C::OFF_STAT);  // [warps][R]
  const uint32_t bar0 = sbase + C::OFF_BAR + 8u * (uint32_t)(warp * C::ST);
  volatile uint32_t* abort_flag =
      reinterpret_cast<uint32_t*>(smem + C::OFF_BAR + kWarps * C::ST * 8);
  const uint32_t red_bar = sbase + C::OFF_BAR + kWarps * C::ST * 8 + 8;  // `red` has been read
  const WaitCtx wctx{abort_flag, p.c.err};
  const uint32_t ring = sbase + (uint32_t)(warp * C::ST * C::STAGE);

  // this lane's sequence of the first group of 32, on its way during the set-up
  int first_row0 = 0, first_end = 0, first_len = 0;
  if (lane < p.c.B) {
    first_row0 = p.c.cu_seqlens[lane];
    first_end = p.c.cu_seqlens[lane + 1];
    first_len = p.c.lens[lane];
  }
  if (lane == 0) {
    for (int i = 0; i < C::ST; ++i) mbar_init(bar0 + 8u * i, 1);
    if (warp == 0) {
      mbar_init(red_bar, kWarps);
      *abort_flag = 0u;
    }
    fence_mbar_init();
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }

  // ---------------------------------------------------------------- this CTA's share
  const int G = p.G;
  Cursor cur;
  long long share;
  const int F = find_share<C>(p, first_row0, first_end, first_len, &cur, &share);
  Record* records = reinterpret_cast<Record*>(p.workspace);
  float* part_lse = reinterpret_cast<float*>(static_cast<char*>(p.workspace) +
                                             (((size_t)gridDim.x * sizeof(Record) + 255) & ~255u));
  float* part_o = part_lse + (((size_t)gridDim.x * 2 * R + 63) & ~(size_t)63);
  Record rec{0, 0, 0, 0, 0, 0};
  __syncthreads();  // barriers initialised
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");

  // ---------------------------------------------------------------- tile info, 32 at a time
  // Lane i holds tile i of a set of 32: the blocks of its parts of 16 keys (-1: no keys
  // there) and their scales.
  struct Info {
    int slice[2];  // page * H + h, of each part
    int row;       // of the first key in its block
    float ks[2], vs[2];
  };
  const int bs = p.c.block_size;
  auto fetch = [&](Cursor at, int f0) {  // tiles f0 .. f0 + 31, `at` being tile f0
    Info r{{-1, -1}, 0, {0.f, 0.f}, {0.f, 0.f}};
    if (f0 + lane >= F) return r;
    advance<C>(p, &at, lane);
    const int key = at.ch * C::CHUNK + warp * C::KEYS;
    r.row = key & (bs - 1);
    const int* table = p.c.block_table + (long long)at.b * p.c.table_width;
#pragma unroll
    for (int i = 0; i < C::PARTS; ++i)
      if (key + 16 * i < at.seq.len) {
        const int page = table[(key + 16 * i) >> p.c.block_log2];
        if (page < 0 || page >= p.c.num_blocks) {
          if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD + 1);
        } else {
          r.slice[i] = page * p.c.H + at.h;
          r.ks[i] = p.c.k_scale[r.slice[i]];  // not waited for here
          r.vs[i] = p.c.v_scale[r.slice[i]];
        }
      }
    return r;
  };
  Cursor ahead = cur;
  int set = 0;  // the one that `info` holds
  Info info = fetch(ahead, 0);
  unsigned live0 = __ballot_sync(0xffffffffu, info.slice[0] >= 0);
  unsigned live1 = C::PARTS == 2 ? __ballot_sync(0xffffffffu, info.slice[1] >= 0) : 0u;
  unsigned now0 = live0, now1 = live1;  // of the set being consumed
  auto next_set = [&]() {
    advance<C>(p, &ahead, 32);
    ++set;
    info = fetch(ahead, 32 * set);
    live0 = __ballot_sync(0xffffffffu, info.slice[0] >= 0);
    if (C::PARTS == 2) live1 = __ballot_sync(0xffffffffu, info.slice[1] >= 0);
  };

  int fi = 0;                     // next tile to load
  uint32_t issued = 0, done = 0;  // live tiles loaded and consumed
  const uint32_t scl0 = sbase + C::OFF_SCL + (uint32_t)(warp * C::ST) * 16u;
  auto issue = [&](int f, bool more) {  // keep the ring full while consuming tile f
    while (fi < F && issued - done < (uint32_t)C::ST) {
      if ((fi >> 5) > set) {
        if (!more || set > (f >> 5)) break;  // at most one set ahead
        next_set();
      }
      const unsigned bit = 1u << (fi & 31);
      if ((live0 | live1) & bit) {
        if (lane == (fi & 31)) {
          const uint32_t slot = issued % C::ST;
          const uint32_t bar = bar0 + 8u * slot, dst = ring + slot * C::STAGE;
          const bool l0 = info.slice[0] >= 0, l1 = C::PARTS == 2 && info.slice[1] >= 0;
          uint32_t v0 = __float_as_uint(info.vs[0]), v1 = __float_as_uint(info.vs[1]);
          if (!l1) v1 = v0;  // a part without keys takes the other one's value scale
          if (!l0) v0 = v1;
          st_shared_v4(scl0 + slot * 16u, __float_as_uint(info.ks[0]), __float_as_uint(info.ks[1]),
                       v0, v1);
          mbar_arrive_expect_tx(bar, (uint32_t)(l0 + l1) * 2u * C::PART);
          if (l0) {
            tma_load_3d(dst, &tm_k, bar, 0, info.row, info.slice[0]);
            tma_load_3d(dst + C::TILE, &tm_v, bar, 0, info.row, info.slice[0]);
          }
          if (l1) {
            const int row = (info.row + 16) & (bs - 1);
            tma_load_3d(dst + C::PART, &tm_k, bar, 0, row, info.slice[1]);
            tma_load_3d(dst + C::TILE + C::PART, &tm_v, bar, 0, row, info.slice[1]);
          }
        }
        ++issued;
      }
      ++fi;
    }
  };
  bool ok = true;

  // ---------------------------------------------------------------- per-segment state
  uint32_t qf[NT][KW][2];        // B operand of S^T: query row g (+ 8 nt)
  float acc[MT][NT][4];          // O^T
  float ref[NT][2], lsum[NT][2], qinv[NT][2];  // columns (query rows) 2t, 2t + 1 (+ 8 nt)
  int lim[NT][2];                // keys visible to those rows
  int lim_lo = 0, lim_hi = 0;    // least and most over the unit's rows
  float lvb = 0.f;               // b
  bool first_live = true;
  bool parked = false;           // sums of another b are in shared memory
  uint32_t ended = 0;            // units

  // Lane layout of the operands.  d = 128: rows of 128 bytes, 16-byte pieces
  // swizzled by row & 7; matrix row i stands for key (i & 1) * 4 + i / 2 (so the
  // two rows of a load phase lie four apart and touch different banks), and a
  // lane's value columns are piece (g & 1) * 4 + g / 2.  d = 64: rows of 64 bytes,
  // pieces swizzled by (row / 2) & 3; keys in order, and lanes of odd t load the
  // odd one of a pair of value rows first.
  const int krow = D == 128 ? ((g & 1) << 2 | g >> 1) : g;
  const int vcol = D == 128 ? ((g & 1) << 2 | g >> 1) * 16 : g * 8;  // first column

  // Sums that are put aside (rare): a normalised O in the warp's part of `red`, each lane its
  // own elements, and a log2-sum-exp in `stat`.  Joined with the running sums, row by row:
  // O = keep O_aside + add acc, and the result's log2-sum-exp.
  float* aside = red + warp * R * D + lane;
  auto join = [&](float (&keep)[NT][2], float (&add)[NT][2], float (&lse)[NT][2]) {
    const float up = ex2(lvb);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float l = lsum[nt][i];
#pragma unroll
        for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
        const float a = parked ? stat[warp * R + nt * 8 + 2 * t + i] : -INFINITY;
        const float c = l == 0.f ? -INFINITY : ref[nt][i] + lg2(l);
        const float m = fmaxf(a, c), mm = m == -INFINITY ? 0.f : m;
        const float wa = ex2(a - mm), wc = ex2(c - mm), z = wa + wc;
        keep[nt][i] = z == 0.f ? 0.f : wa / z;
        add[nt][i] = z == 0.f || l == 0.f ? 0.f : wc / z / l * up;
        lse[nt][i] = z == 0.f ? -INFINITY : mm + lg2(z);
      }
    __syncwarp();
  };
  auto park = [&]() {
    if (ended > 0)  // the other warps have read the last unit's results
      mbar_wait(red_bar, (ended - 1) & 1u, wctx, ERR_SITE_CACHE_FWD + 15);
    float keep[NT][2], add[NT][2], lse[NT][2];
    join(keep, add, lse);
#pragma unroll
    for (int mt = 0; mt < MT; ++mt)
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float* at = aside + ((mt * NT + nt) * 4 + i) * 32;
          *at = (parked ? *at : 0.f) * keep[nt][i & 1] + acc[mt][nt][i] * add[nt][i & 1];
          acc[mt][nt][i] = 0.f;
        }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (g == 0) stat[warp * R + nt * 8 + 2 * t + i] = lse[nt][i];
        lsum[nt][i] = 0.f;
        ref[nt][i] = -INFINITY;
      }
    __syncwarp();
    parked = true;
  };

  int f = 0;             // the tile (of all warps) that comes next
  bool resumed = false;  // in the middle of a unit
  bool calm = false;     // that tile's scale is settled:
  float calm_lv = 0.f;   // its log2 vs - b
  int only = 0;          // 1, 2: only the first, the second part of it
  while (f < F) {
    const int h = cur.h, rb = cur.rb;
    const int rows = min(R, cur.seq.n * G - rb * R);
    const int last = f + min(cur.nch - cur.ch, F - f) - 1;  // of this unit in the share
    uint4 qraw[NT][D / 32];  // bf16: 16 of d = 128's first half, 16 of its second (d = 64: 16)
    if (!resumed) {  // a unit (or piece) begins
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
#pragma unroll
        for (int j = 0; j < D / 32; ++j) qraw[nt][j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int i = rb * R + r;
          const uint16_t* q = p.q.p + (long long)(cur.seq.row0 + p.by_G.div(i)) * p.q.st +
                              (long long)(h * G + p.by_G.mod(i)) * p.q.sh;
#pragma unroll
          for (int j = 0; j < D / 32; ++j)
            qraw[nt][j] = *reinterpret_cast<const uint4*>(q + (j >> 1) * 64 + t * 16 + (j & 1) * 8);
        }
      }
      if (f == 0) issue(0, false);  // while q is on its way
      const int seen0 = p.causal ? cur.seq.len - cur.seq.n + 1 : cur.seq.len;  // token 0's keys
      auto limit_of = [&](int r) {
        return p.causal ? seen0 + p.by_G.div(rb * R + r) : seen0;
      };
      lim_lo = limit_of(0);
      lim_hi = min(cur.seq.len, limit_of(rows - 1));
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const uint4* v = qraw[nt];
        uint32_t mx = 0u;
#pragma unroll
        for (int j = 0; j < D / 32; ++j)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu),
                                     __vmaxu2(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu)));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^(14 - exponent of the largest element); rows of zeros or with inf or NaN stay
        int e = (int)(mx >> 7);  // biased exponent
        e = (mx == 0u || e == 255) ? 0 : min(14 - (e - 127), 126);
        const float mul = __uint_as_float((uint32_t)(e + 127) << 23);
        const float back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int w = 0; w < KW; ++w) {
          const uint32_t* x = &v[w >> 1].x + (w & 1) * 2;
          qf[nt][w][0] = pack_f16x2(__uint_as_float(x[0] << 16) * mul,
                                    __uint_as_float(x[0] & 0xffff0000u) * mul);
          qf[nt][w][1] = pack_f16x2(__uint_as_float(x[1] << 16) * mul,
                                    __uint_as_float(x[1] & 0xffff0000u) * mul);
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 2 * t + i;
          qinv[nt][i] = __shfl_sync(0xffffffffu, back, col * 4) * p.scale_log2;
          lim[nt][i] = nt * 8 + col < rows ? min(cur.seq.len, limit_of(nt * 8 + col)) : 0;
          ref[nt][i] = -INFINITY;
          lsum[nt][i] = 0.f;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
      first_live = true;
      lvb = 0.f;
      parked = false;
    }

    // ---------------------------------------------------------------- its tiles
    bool event = false;  // a block whose scale is too far from b
    while (true) {
      const int key0 = cur.ch * C::CHUNK + warp * C::KEYS;
      bool on[2] = {(now0 >> (f & 31) & 1u) != 0u, (now1 >> (f & 31) & 1u) != 0u};
      if ((on[0] || on[1]) && ok) {
        const uint32_t slot = done % C::ST;
        ok = __all_sync(0xffffffffu, mbar_wait(bar0 + 8u * slot, (done / C::ST) & 1u, wctx,
                                               ERR_SITE_CACHE_FWD + 2));
        if (ok) {
          const uint4 sc = ld_shared_v4(scl0 + slot * 16u);
          const float ks[2] = {__uint_as_float(sc.x), __uint_as_float(sc.y)};
          float lv[2] = {lg2(__uint_as_float(sc.z)), lg2(__uint_as_float(sc.w))};
          if (first_live) lvb = lv[0];
          first_live = false;
          lv[0] -= lvb, lv[1] -= lvb;
          const float far = C::PARTS == 2 ? fmaxf(fabsf(lv[0]), fabsf(lv[1])) : fabsf(lv[0]);
          if (__builtin_expect(far > kWindow || (C::PARTS == 2 && only != 0), 0)) {
            if (!calm) {  // rare, warp-uniform
              event = true;
              break;
            }
            if (only == 1) on[1] = false;
            if (only == 2) on[0] = false;
            lv[0] = lv[1] = calm_lv;
          }
          const uint32_t ka = ring + slot * C::STAGE, va = ka + C::TILE;
          const bool masked = key0 + C::KEYS > lim_lo;  // some row does not see all of it
          // S^T, 16 keys at a time; y = x + log2 vs - b, masked keys before the maximum
          float s[C::PARTS][NT][4];
#pragma unroll
          for (int pt = 0; pt < C::PARTS; ++pt) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i) s[pt][nt][i] = on[pt] ? 0.f : -INFINITY;
            if (!on[pt]) continue;
#pragma unroll
            for (int half = 0; half < D / 64; ++half) {
              uint32_t a[2][4];  // keys krow and krow + 8: 16 bytes
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const int row = krow + 8 * i;
                const int piece = half * 4 + t;
                const uint32_t at = ka + pt * C::PART;
                const uint32_t addr = D == 128 ? at + row * 128 + ((piece ^ (row & 7)) << 4)
                                               : at + row * 64 + ((piece ^ ((row >> 1) & 3)) << 4);
                const uint4 x = ld_shared_v4(addr);
                a[i][0] = x.x, a[i][1] = x.y, a[i][2] = x.z, a[i][3] = x.w;
              }
#pragma unroll
              for (int w = 0; w < 4; ++w) {
                uint32_t a0, a1, a2, a3;
                codes4_to_f16<E5M2>(a[0][w], a0, a2);
                codes4_to_f16<E5M2>(a[1][w], a1, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(s[pt][nt], a0, a1, a2, a3, qf[nt][half * 4 + w][0],
                          qf[nt][half * 4 + w][1]);
              }
            }
            const int k0 = key0 + pt * 16 + krow, k1 = k0 + 8;
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[pt][nt][i] = fmaf(s[pt][nt][i], ks[pt] * qinv[nt][i & 1], lv[pt]);
            if (masked) {
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if ((i < 2 ? k0 : k1) >= lim[nt][i & 1]) s[pt][nt][i] = -INFINITY;
            }
          }
          float top[NT][2];  // this lane's largest y
          bool move = false;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              top[nt][i] = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
              if (C::PARTS == 2)
                top[nt][i] = fmaxf(top[nt][i], fmaxf(s[C::PARTS - 1][nt][i],
                                                     s[C::PARTS - 1][nt][i + 2]));
              move |= top[nt][i] - ref[nt][i] > kRoom;  // (-inf) - (-inf) moves nothing
            }
          if (__any_sync(0xffffffffu, move)) {
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float alpha[2];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                float m = top[nt][i];
#pragma unroll
                for (int w = 4; w < 32; w <<= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, w));
                const float r = fabsf(m) < kFar ? m - kOff : m;
                const float to = fmaxf(r, ref[nt][i]);
                alpha[i] = to == -INFINITY ? 1.f : ex2(ref[nt][i] - to);
                ref[nt][i] = to;
                lsum[nt][i] *= alpha[i];
              }
#pragma unroll
              for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int i = 0; i < 4; ++i) acc[mt][nt][i] *= alpha[i & 1];
            }
          }
          const int odd = D == 64 ? (t & 1) : 0;
#pragma unroll
          for (int pt = 0; pt < C::PARTS; ++pt) {
            if (!on[pt]) continue;
            const float w = ex2(-lv[pt]);
            uint32_t pf[NT][2];  // B operand of O^T
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float pr[4];
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const float r = ref[nt][i] == -INFINITY ? 0.f : ref[nt][i];
                pr[i] = ex2(s[pt][nt][i] - r);
                pr[i + 2] = ex2(s[pt][nt][i + 2] - r);
                lsum[nt][i] = fmaf(pr[i] + pr[i + 2], w, lsum[nt][i]);
              }
              pf[nt][0] = movmatrix(pack_f16x2(pr[0], pr[1]));
              pf[nt][1] = movmatrix(pack_f16x2(pr[2], pr[3]));
            }
            // value rows of this lane: keys of matrix rows 2t, 2t + 1, 2t + 8, 2t + 9
            const int first = key0 + pt * 16;
            auto value_row = [&](int i) {
              return D == 128 ? t + 4 * i : 2 * t + ((i & 1) ^ odd) + 8 * (i >> 1);
            };
            auto load_values = [&](uint32_t (&v)[4][VW]) {
              const uint32_t at = va + pt * C::PART;
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int row = value_row(i);
                if constexpr (D == 128) {
                  const uint4 x = ld_shared_v4(at + row * 128 + (((vcol >> 4) ^ (row & 7)) << 4));
                  v[i][0] = x.x, v[i][1] = x.y, v[i][2] = x.z, v[i][3] = x.w;
                } else {
                  const uint2 x = ld_shared_v2(at + row * 64 +
                                               (((vcol >> 4) ^ ((row >> 1) & 3)) << 4) + (vcol & 15));
                  v[i][0] = x.x, v[i][1] = x.y;
                }
              }
              if (masked) {  // stale rows, whatever they hold
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (first + value_row(i) >= lim_hi) {
#pragma unroll
                    for (int j = 0; j < VW; ++j) v[i][j] = 0u;
                  }
              }
            };
            uint32_t v[4][VW];
            load_values(v);
            // keys that some rows see and others do not: a NaN there must reach the former
            // only, and a weight of zero does not keep it out of the product
            bool poison = false;
            if (masked && lim_lo < min(first + 16, lim_hi)) {
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VW; ++j) {
                  const uint32_t m = nan_codes<E5M2>(v[i][j]);
                  poison |= m != 0u;
                  v[i][j] = clear_codes(v[i][j], m);
                }
              poison = __any_sync(0xffffffffu, poison);
            }
            // O^T: bytes 2 mt, 2 mt + 1 of the lane's columns are rows g, g + 8 of tile mt
            const uint32_t sel_lo = odd ? 0x1504u : 0x5140u, sel_hi = odd ? 0x3726u : 0x7362u;
#pragma unroll
            for (int j = 0; j < VW; ++j) {
#pragma unroll
              for (int m = 0; m < 2; ++m) {
                uint32_t a0, a1, a2, a3;
                codes4_to_f16<E5M2>(__byte_perm(v[0][j], v[1][j], m ? sel_hi : sel_lo), a0, a1);
                codes4_to_f16<E5M2>(__byte_perm(v[2][j], v[3][j], m ? sel_hi : sel_lo), a2, a3);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(acc[2 * j + m][nt], a0, a1, a2, a3, pf[nt][0], pf[nt][1]);
              }
            }
            if (poison) {  // rare: NaN for the rows that see it
              load_values(v);
#pragma unroll
              for (int i = 0; i < 4; ++i)
#pragma unroll
                for (int j = 0; j < VW; ++j) v[i][j] = nan_codes<E5M2>(v[i][j]);
#pragma unroll
              for (int j = 0; j < 4 * VW; ++j) {
                uint32_t bad = 0u;  // the part's keys whose value in this column is NaN
#pragma unroll
                for (int i = 0; i < 4; ++i)
                  if (v[i][j >> 2] >> (8 * (j & 3)) & 0x80u) bad |= 1u << value_row(i);
                bad |= __shfl_xor_sync(0xffffffffu, bad, 1);
                bad |= __shfl_xor_sync(0xffffffffu, bad, 2);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int i = 0; i < 2; ++i)
                    if (bad & ((1u << max(0, min(16, lim[nt][i] - first))) - 1u))
                      acc[j >> 1][nt][(j & 1) * 2 + i] = __uint_as_float(0x7fffffffu);
              }
            }
          }
          calm = false;
          if (C::PARTS == 2 && only == 1) {
            only = 2;
            continue;
          }
          only = 0;
          __syncwarp();  // the slot may be loaded again
          ++done;
        }
      }
      const bool ends = f == last;
      if (++f < F) {
        if ((f & 31) == 0) {
          if (set < (f >> 5)) next_set();
          now0 = live0, now1 = live1;
        }
        if (ok) issue(f, true);
      }
      if (ends) break;
      ++cur.ch;
    }
    resumed = event;
    if (__builtin_expect(event, 0)) {
      const uint32_t slot = done % C::ST;
      const uint4 sc = ld_shared_v4(scl0 + slot * 16u);
      const bool on0 = (now0 >> (f & 31) & 1u) != 0u, on1 = (now1 >> (f & 31) & 1u) != 0u;
      if (C::PARTS == 2 && only == 0 && on0 && on1) only = 1;
      const bool second = C::PARTS == 2 && (only == 2 || !on0);
      const float lvs = lg2(__uint_as_float(second ? sc.w : sc.z));
      calm = true;
      calm_lv = lvs - lvb;
      if (calm_lv < kNothing) {
        calm_lv = kNothing;
      } else if (fabsf(calm_lv) > kWindow) {
        park();
        lvb = lvs;
        calm_lv = 0.f;
      }
      continue;
    }

    // ---------------------------------------------------------------- the unit (or piece) ends
    if (__builtin_expect(parked, 0)) {  // rare: all of it as if it were one key's
      float keep[NT][2], add[NT][2];
      join(keep, add, ref);
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i)
            acc[mt][nt][i] = aside[((mt * NT + nt) * 4 + i) * 32] * keep[nt][i & 1] +
                             acc[mt][nt][i] * add[nt][i & 1];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int i = 0; i < 2; ++i) lsum[nt][i] = g == 0 && ref[nt][i] != -INFINITY ? 1.f : 0.f;
      lvb = 0.f;
    }
    end_unit<C, D>(p, cur, f, share, rows, acc, ref, lsum, lvb, vcol, red, stat, part_lse, part_o, h,
                   rb, G, &rec);
    __syncwarp();
    if (lane == 0) mbar_arrive(red_bar);
    ++ended;
    advance<C>(p, &cur, 1);
  }
  // loads in flight land before the CTA ends (only after a wait that ran out)
  for (; done < issued; ++done)
    mbar_drain(bar0 + 8u * (done % C::ST), (done / C::ST) & 1u, wctx, ERR_SITE_CACHE_FWD + 3);
  if (threadIdx.x == 0) records[blockIdx.x] = rec;
  // launched behind the 256-row kernel, this one may overtake it; the merge must not
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Joins the pieces of the unit that CTA blockIdx.x of an attention kernel began and
// did not finish: its own second slot, then the first slots of the CTAs behind.
// The first narrow_ctas blocks serve the kernel above, the others the 256-row one,
// kWideMerge of them each of its CTAs.
// Latency counts: the weights of 32 pieces are read by one instruction, and eight
// pieces' rows are in flight at a time.
template <int D>
__global__ void __launch_bounds__(256)
    cache_merge_kernel(const CacheFwdParams p, int narrow_ctas, int narrow_R, int wide_ctas,
                       int wide_R) {
  constexpr float kLog2e = 1.4426950408889634f;
  constexpr int C4 = D / 4;  // 16-byte columns: one per lane (d = 64: two rows per warp)
  constexpr int RPW = 32 / C4;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int behind = (int)blockIdx.x - narrow_ctas;
  const bool wide = behind >= 0;
  const int ctas = wide ? wide_ctas : narrow_ctas, R = wide ? wide_R : narrow_R;
  const int cta = wide ? behind % wide_ctas : blockIdx.x;
  const char* ws = static_cast<const char*>(wide ? p.wide_workspace : p.workspace);
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const Record rec = reinterpret_cast<const Record*>(ws)[cta];
  const float* part_lse =
      reinterpret_cast<const float*>(ws + (((size_t)ctas * sizeof(Record) + 255) & ~255u));
  const float4* part_o =
      reinterpret_cast<const float4*>(part_lse + (((size_t)ctas * 2 * R + 63) & ~(size_t)63));
  // piece i of row r: slot 1 of this CTA, slot 0 of the next ones; wide: one behind another
  auto at = [&](int i, int r) {
    return (wide ? (size_t)rec.place + i : (size_t)(cta + i) * 2 + (i == 0 ? 1 : 0)) * R + r;
  };
  if (rec.parts == 0) return;
  const int first = wide ? behind / wide_ctas * 8 + warp : warp;
  const int step = wide ? kWideMerge * 8 : 8;
  for (int r0 = first * RPW; r0 < rec.rows; r0 += step * RPW) {
    const int r = r0 + lane / C4, c4 = lane % C4;
    const bool on = r < rec.rows;
    float m = -INFINITY, sum = 0.f;
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int i0 = 0; i0 < rec.parts; i0 += C4) {  // as many pieces as a row has lanes
      const float l = on && i0 + c4 < rec.parts ? part_lse[at(i0 + c4, r)] * kLog2e : -INFINITY;
      float top = l;
#pragma unroll
      for (int w = C4 / 2; w > 0; w >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, w));
      top = fmaxf(top, m);
      const float mm = top == -INFINITY ? 0.f : top;
      const float alpha = ex2(m - mm);
      m = top;
      const float w = ex2(l - mm);  // 0 behind the last piece
      float z = w;
#pragma unroll
      for (int k = C4 / 2; k > 0; k >>= 1) z += __shfl_xor_sync(0xffffffffu, z, k);
      sum = sum * alpha + z;
      o.x *= alpha, o.y *= alpha, o.z *= alpha, o.w *= alpha;
      const int n = min(C4, rec.parts - i0);
      for (int i = 0; i < n; i += 8) {
        float4 v[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
          v[k] = on && i + k < n ? part_o[at(i0 + i + k, r) * C4 + c4] : make_float4(0, 0, 0, 0);
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const float x = __shfl_sync(0xffffffffu, w, (lane / C4) * C4 + ((i + k) & (C4 - 1)));
          o.x = fmaf(x, v[k].x, o.x), o.y = fmaf(x, v[k].y, o.y);
          o.z = fmaf(x, v[k].z, o.z), o.w = fmaf(x, v[k].w, o.w);
        }
      }
    }
    if (!on) continue;
    const bool any = !(sum == 0.f);
    const float inv = any ? 1.f / sum : 0.f;
    const int i0 = rec.first_row + r;
    const long long token = rec.row0 + p.by_G.div(i0);
    const int hq = rec.h * p.G + p.by_G.mod(i0);
    *reinterpret_cast<uint2*>(p.o.p + token * p.o.st + hq * p.o.sh + c4 * 4) = make_uint2(
        pack_bf16x2(o.x * inv, o.y * inv), pack_bf16x2(o.z * inv, o.w * inv));
    if (c4 == 0)
      p.lse[(long long)hq * p.c.total + token] =
          any ? (m + lg2(sum)) * kLn2 : -INFINITY;
  }
}

// Joins the pieces that the kernel for few rows (`grid` CTAs, R rows per unit) and the
// 256-row kernel left.
cudaError_t launch_merge(const CacheFwdParams& p, int grid, int R, int n_sm, bool wide,
                         cudaStream_t stream) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(grid + (wide ? kWideMerge * n_sm : 0)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return p.c.d == 128
             ? cudaLaunchKernelEx(&cfg, cache_merge_kernel<128>, p, grid, R, n_sm, cache_fwd_wide_rows())
             : cudaLaunchKernelEx(&cfg, cache_merge_kernel<64>, p, grid, R, n_sm, cache_fwd_wide_rows());
}

template <int D, bool E5M2, int NT>
cudaError_t launch(const CUtensorMap& tk, const CUtensorMap& tv, const CacheFwdParams& p, int n_sm,
                   bool wide, cudaStream_t stream) {
  using C = Dec<D, NT>;
  static_assert(C::CTAS * (C::SMEM + 1024) <= 233472, "shared memory of the CTAs sharing an SM");
  static unsigned long long prepared[64];
  const cudaError_t e = prepare_once(prepared, [] {
    return cudaFuncSetAttribute(cache_fwd_kernel<D, E5M2, NT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  const int grid = n_sm * C::CTAS;
  const cudaError_t r =
      launch_split(cache_fwd_kernel<D, E5M2, NT>, grid, C::SMEM, wide, stream, tk, tv, p);
  return r != cudaSuccess ? r : launch_merge(p, grid, C::R, n_sm, wide, stream);
}

template <int D, bool E5M2>
cudaError_t launch_rows(const CUtensorMap& tk, const CUtensorMap& tv, const CacheFwdParams& p,
                        int n_sm, bool wide, cudaStream_t stream) {
  const long long rows = (long long)p.c.max_seqlen * p.G;
  return rows <= 8 ? launch<D, E5M2, 1>(tk, tv, p, n_sm, wide, stream)
                   : launch<D, E5M2, 2>(tk, tv, p, n_sm, wide, stream);
}

// Bytes of the records, LSE and O of `ctas` CTAs with R rows per unit.
size_t pieces_bytes(size_t ctas, int R, int d) {
  return ((ctas * sizeof(Record) + 255) & ~(size_t)255) +
         ((ctas * 2 * R + 63) & ~(size_t)63) * 4 + ctas * 2 * R * d * 4;
}
size_t narrow_bytes(int d, int n_sm) {  // the largest variant's, in 8 and in 4 bits
  return std::max(pieces_bytes((size_t)n_sm * split_ctas(128, 1), split_rows(1), d),
                  pieces_bytes((size_t)n_sm * split_ctas(64, 2), split_rows(2), d));
}
// The most query rows per key/value head (tokens x grouped heads) of a sequence that
// stays with the kernel above.  From 33 rows on it reads the keys three times and
// more, and the 256-row kernel costs less of the machine, but finishes a small batch
// later.  Measured with limits of 32 and 64 rows: 16 sequences of 1 to 1000 tokens, 16
// key heads, d = 64, 79 and 102 us; 150 of 50 to 100 tokens, 4 heads, d = 128, 84 and
// 154 us; 24 of 5 tokens, 2 key heads of 8 query heads, d = 64, 24 and 17 us.  (Many
// sequences of very few keys lose by it, 134 of 7 keys, 8 heads of 7, 61 and 35 us: their
// lengths are not known on the host.)
int narrow_limit(const CacheParams& c, int n_sm) {
  return (long long)c.B * c.H >= n_sm ? 32 : 64;
}
// Whether a call may have sequences for the 256-row kernel (whose row blocks hold
// whole tokens: groups of more than 256 heads stay with the other one).
bool takes_wide(const CacheParams& c, int G, int n_sm) {
  return (long long)c.max_seqlen * G > narrow_limit(c, n_sm) && G <= cache_fwd_wide_rows();
}

}  // namespace

size_t cache_fwd_workspace(const CacheParams& c, int G, int n_sm) {
  return narrow_bytes(c.d, n_sm) +
         (takes_wide(c, G, n_sm) ? pieces_bytes((size_t)n_sm, cache_fwd_wide_rows(), c.d) +
                                       cache_fwd_wide_plan_bytes(cache_fwd_wide_grid(
                                           c, G, narrow_limit(c, n_sm), n_sm))
                                 : 0);
}

cudaError_t launch_cache_fwd(const CUtensorMap& tk, const CUtensorMap& tv,
                             const CacheFwdParams& params, int n_sm, cudaStream_t stream) {
  CacheFwdParams p = params;
  const bool wide = takes_wide(p.c, p.G, n_sm);
  p.narrow_rows = wide ? narrow_limit(p.c, n_sm) : 0x7fffffff;
  if (wide) {
    p.wide_tokens = cache_fwd_wide_rows() / p.G;
    p.wide_ctas = n_sm;
    const long long grid = cache_fwd_wide_grid(p.c, p.G, p.narrow_rows, n_sm);
    if (grid > 0x7fffffffLL) return cudaErrorInvalidConfiguration;
    p.wide_grid = (int)grid;
    p.wide_workspace = static_cast<char*>(p.workspace) + narrow_bytes(p.c.d, n_sm);
    const cudaError_t e = launch_cache_fwd_wide(p, stream);
    if (e != cudaSuccess) return e;
  }
  if (p.c.format == FMT_INT4) {
    int grid, R;
    const cudaError_t e = launch_cache4_fwd(p, n_sm, wide, stream, &grid, &R);
    return e != cudaSuccess ? e : launch_merge(p, grid, R, n_sm, wide, stream);
  }
  if (p.c.d == 128)
    return p.c.format ? launch_rows<128, true>(tk, tv, p, n_sm, wide, stream)
                      : launch_rows<128, false>(tk, tv, p, n_sm, wide, stream);
  return p.c.format ? launch_rows<64, true>(tk, tv, p, n_sm, wide, stream)
                    : launch_rows<64, false>(tk, tv, p, n_sm, wide, stream);
}

}  // namespace fattn

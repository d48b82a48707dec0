// cache4_fwd.cu -- attention over the paged 4-bit key/value cache, few query rows per
// key/value head (decoding, drafted tokens).
//
// The mathematics is that of the 8-bit kernel without the blocks' scales: in base 2, with a
// reference r carried along the keys (the running maximum less 8, moved when a score exceeds
// it by more than 15),
//   x_j = scale log2(e) (q . k_j),   acc = sum_j p_j v_j,  l = sum_j p_j,  p_j = 2^(x_j - r),
//   O = acc / l,  LSE = ln2 (r + log2 l).
// Weights are held in fp16, at or below 2^15, the largest at or above 2^8.  Keys and values
// are exact in fp16 as (c - 8) s 2^-7; q is as in the 8-bit kernel.  (Where |x| >= 2^22, r is the
// maximum itself and p is formed from the rounded x, whose rounding the maximum has seen.)
//
// The products are those of the 8-bit kernel, m16n8k16 mma.sync with the keys (S^T = K Q^T) or
// the value channels (O^T += V^T P^T) as the 16-row operand; a lane's share of a key is a quarter
// of its channels, of a value row an eighth, all of one or two groups of 16, so it applies few
// scales: one fused multiply-add makes two codes two values (see cache.cuh).
//
// The bound: a token's keys and values are 144 bytes at d = 128, which an SM gets in 6.5 clocks at
// the measured copy bandwidth; two codes cost 2.25 instructions, so the conversions alone take
// 9 of the 26 issue slots of that time.  So the kernel is built around few instructions per
// tile of 32 keys: loads by cp.async, 9 for a tile, whose addresses are one multiplication each
// (bulk copies and their barriers took 40 more), scores scaled inside the exponent's
// multiply-add, constants held in registers, codes put into fp16 by one lop3 a pair.
//
// Measured, 4 x 32768 keys, 32 heads, d = 128, one token each: 120 us, 5040 GB/s, 74 % of the
// measured copy bandwidth, bound by issue: 308 instructions for 16 keys a warp, 144 of them
// the conversions, at 2.3 of 4 a clock, as the 168 registers that they are kept in leave
// room for 12 warps an SM.  (The 8-bit kernel with this format took 177 us, this one with
// two lop3 a pair 141.  Against 117 at their time: four CTAs an SM 131, two 130, row sums by
// a product with ones 121, two chains for each score 121, both parts' products interleaved
// 124, values loaded before the softmax 121, the value products in a loop 126.)  d = 64, tiles of
// 64 keys: 73 us, with 32 keys 81.
#include <math.h>

#include <algorithm>

#include "cache_split.cuh"

namespace fattn {
namespace {

template <int D, int NT_>
struct Dec4 {
  static constexpr int NT = NT_;
  static constexpr int R = split_rows(NT);
  static constexpr int PARTS = D == 128 || NT == 2 ? 2 : 4;  // of 16 keys in a warp's tile
  static constexpr int KEYS = 16 * PARTS;
  static constexpr int CHUNK = kWarps * KEYS;
  static constexpr int ROW = D / 2;             // bytes of a key's or value's codes
  static constexpr int TILE = KEYS * ROW;
  static constexpr int PART_SCL = D;            // bytes of the scales of 16 keys
  static constexpr int TILE_SCL = PARTS * PART_SCL;
  static constexpr int STAGE = 2 * TILE + 2 * TILE_SCL;  // keys, values, their scales
  static constexpr int ST = D == 64 && NT == 2 ? 6 : NT == 1 ? 3 : 4;  // ring slots per warp
  static constexpr int CTAS = split_ctas(D, NT);  // per SM
  static constexpr int OFF_RED = kWarps * ST * STAGE;
  static constexpr int OFF_STAT = OFF_RED + kWarps * R * D * 4;
  static constexpr int SMEM = OFF_STAT + kWarps * R * 4 + 128;
};

__device__ __forceinline__ void copy16_async(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
template <int N>
__device__ __forceinline__ void copies_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

template <int D, int NT>
__global__ void __launch_bounds__(32 * kWarps, Dec4<D, NT>::CTAS)
    cache4_fwd_kernel(const CacheFwdParams p) {
  using C = Dec4<D, NT>;
  constexpr int R = C::R, ST = C::ST;
  constexpr int KW = D / 16;  // k16 steps of S^T
  constexpr int MT = D / 16;  // 16-row tiles of O^T
  constexpr int W = D / 32;   // words of eight codes: a quarter of a key
  constexpr int VW = D / 64;  // and an eighth of a value row
  extern __shared__ uint8_t smem_raw[];
  const uint32_t raw = smem_u32(smem_raw);
  const uint32_t sbase = (raw + 127u) & ~127u;
  uint8_t* smem = smem_raw + (sbase - raw);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int g = lane >> 2, t = lane & 3;
  float* red = reinterpret_cast<float*>(smem + C::OFF_RED);
  float* stat = reinterpret_cast<float*>(smem + C::OFF_STAT);
  const uint32_t ring = sbase + (uint32_t)(warp * ST * C::STAGE);
  const int G = p.G;

  int first_row0 = 0, first_end = 0, first_len = 0;
  if (lane < p.c.B) {
    first_row0 = p.c.cu_seqlens[lane];
    first_end = p.c.cu_seqlens[lane + 1];
    first_len = p.c.lens[lane];
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  Cursor cur;
  long long share;
  const int F = find_share<C>(p, first_row0, first_end, first_len, &cur, &share);
  Record* records = reinterpret_cast<Record*>(p.workspace);
  float* part_lse = reinterpret_cast<float*>(static_cast<char*>(p.workspace) +
                                             (((size_t)gridDim.x * sizeof(Record) + 255) & ~255u));
  float* part_o = part_lse + (((size_t)gridDim.x * 2 * R + 63) & ~(size_t)63);
  Record rec{0, 0, 0, 0, 0, 0};

  // ---------------------------------------------------------------- blocks, 32 tiles at a time
  // Lane i holds tile i of a set of 32.  The next set's entries of the block table are on their
  // way while this one's are used.
  struct Pages {
    int page[C::PARTS];  // of each part: as the table has it; -1: no keys there
    int h, row16;  // head; place of the first key in its block, in units of 16
  };
  const int bs = p.c.block_size;
  Cursor ahead = cur;
  auto look_up = [&](int f0) {  // `ahead` being tile f0
    Pages r{};
#pragma unroll
    for (int i = 0; i < C::PARTS; ++i) r.page[i] = -1;
    if (f0 + lane >= F) return r;
    Cursor at = ahead;
    advance<C>(p, &at, lane);
    const int key = at.ch * C::CHUNK + warp * C::KEYS;
    const int* table = p.c.block_table + (long long)at.b * p.c.table_width;
    r.h = at.h;
    r.row16 = (key & (bs - 1)) >> 4;
#pragma unroll
    for (int i = 0; i < C::PARTS; ++i)
      if (key + 16 * i < at.seq.len) {
        const int page = table[(key + 16 * i) >> p.c.block_log2];
        // (a bad number that means "no keys" is one that may be reported here)
        r.page[i] = page == -1 ? -2 : page;
      }
    return r;
  };
  // Place of the part's 16 keys in the pool, in units of 16 (-1: no keys): a lane's own
  int place[C::PARTS];
  auto settle = [&](const Pages& s) {
#pragma unroll
    for (int i = 0; i < C::PARTS; ++i) {
      place[i] = -1;
      if (s.page[i] == -1) continue;
      if (s.page[i] < 0 || s.page[i] >= p.c.num_blocks) {
        if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD + 1);
        continue;
      }
      // (a unit is 512 bytes of codes or more: their number stays below 2^31)
      place[i] = ((s.page[i] * p.c.H + s.h) << (p.c.block_log2 - 4)) +
                 ((s.row16 + i) & ((bs >> 4) - 1));
    }
  };
  Pages next = look_up(0);
  settle(next);
  advance<C>(p, &ahead, 32);
  next = look_up(32);

  // ---------------------------------------------------------------- loads
  // A lane's 16 bytes of each 512 of codes; d = 128: rows of 64 bytes, 16-byte pieces swizzled
  // by (row / 2) & 3; d = 64: of 32, by (row / 4) & 1.  The scales of keys and values are one
  // more instruction, behind the codes.
  constexpr int LD = C::ROW / 32;  // 512-byte loads of a part's codes: 2, 1
  const int crow = lane * 16 / C::ROW;  // row within such a load
  const uint32_t cdst =
      D == 128 ? (uint32_t)(crow * 64 + (((lane & 3) ^ ((crow >> 1) & 3)) << 4))
               : (uint32_t)(crow * 32 + (((lane & 1) ^ ((crow >> 2) & 1)) << 4));
  constexpr int LP = D / 16;  // lanes that copy a part's scales
  const int sside = lane / (C::PARTS * LP), spart = lane / LP % C::PARTS;
  static_assert(2 * C::PARTS * LP == 32 || NT == 2, "all lanes");
  const uint32_t sdst = 2 * C::TILE + sside * C::TILE_SCL + spart * C::PART_SCL + lane % LP * 16;
  const uint8_t* sfrom = (sside ? p.c.v_scale4() : p.c.k_scale4()) + lane % LP * 16;
  uint32_t live[C::PARTS] = {};  // bit i: whether tile (issued - 1 - i) has keys in that part
  int fi = 0;                   // next tile to load
  uint32_t fill = ring;         // its slot
  auto issue = [&]() {
#pragma unroll
    for (int i = 0; i < C::PARTS; ++i) live[i] <<= 1;
    if (fi < F) {
      if ((fi & 31) == 0 && fi > 0) {
        settle(next);
        advance<C>(p, &ahead, 32);
        next = look_up(fi + 32);
      }
      int at[C::PARTS], sat = -1;
#pragma unroll
      for (int i = 0; i < C::PARTS; ++i) {
        at[i] = __shfl_sync(0xffffffffu, place[i], fi & 31);
        if (spart == i) sat = at[i];
        if (at[i] >= 0) {
          live[i] |= 1u;
          const long long off = (long long)at[i] * (16 * C::ROW) + lane * 16;
          const uint8_t* k = p.c.k + off;
          const uint8_t* v = p.c.v + off;
#pragma unroll
          for (int x = 0; x < LD; ++x) {
            const uint32_t dst = fill + cdst + (i * LD + x) * 512;
            copy16_async(dst, k + x * 512);
            copy16_async(dst + C::TILE, v + x * 512);
          }
        }
      }
      if (sside < 2 && sat >= 0)
        copy16_async(fill + sdst, sfrom + (long long)sat * C::PART_SCL);
      ++fi;
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    fill = fill == ring + (ST - 1) * C::STAGE ? ring : fill + C::STAGE;
  };

  // ---------------------------------------------------------------- per-unit state
  uint32_t qf[NT][KW][2];
  float acc[MT][NT][4];
  float ref[NT][2], nref[NT][2], bound[NT][2];  // r; -r (0 before any key); r + 15
  float lsum[NT][2], fac[NT][2];                // fac: of a product to x
  int lim[NT][2];
  int lim_lo = 0, lim_hi = 0;
  bool far = false;  // some |r| is too large for a fused multiply-add

  // matrix row 2 i + e stands for key krow4(i, e) of 16: the rows of a load phase touch
  // different banks, those of the keys' products (two or four g, all t) and those of the
  // values' (one e, all t) alike
  auto krow4 = [](int i, int e) {
    return D == 128 ? ((i ^ e) & 1) | e << 1 | (i >> 1) << 2 : (i ^ e << 1) | e << 2;
  };
  const int krow = krow4(g >> 1, g & 1);
  const int vcol = g * (D / 8);
  // this lane's places in a slot
  const uint32_t ka0 = D == 128 ? (uint32_t)(krow * 64 + ((t ^ ((krow >> 1) & 3)) << 4))
                                : (uint32_t)(krow * 32 + (((t >> 1) ^ ((krow >> 2) & 1)) << 4) +
                                             (t & 1) * 8);
  const uint32_t ks0 = 2 * C::TILE + (D == 128 ? krow * 8 + t * 2 : krow * 4 + t);
  uint32_t va0[2], vs0[2];
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const int row = krow4(t, e);
    va0[e] = C::TILE +
             (D == 128 ? (uint32_t)(row * 64 + (((g >> 1) ^ ((row >> 1) & 3)) << 4) + (g & 1) * 8)
                       : (uint32_t)(row * 32 + (((g >> 2) ^ ((row >> 2) & 1)) << 4) + (g & 3) * 4));
    vs0[e] = 2 * C::TILE + C::TILE_SCL + (D == 128 ? row * 8 + g : row * 4 + (g >> 1));
  }
  const Int4Magic magic;

  for (int i = 0; i < ST - 1; ++i) issue();
  uint32_t slot = ring;
  int f = 0;
  while (f < F) {
    const int h = cur.h, rb = cur.rb;
    const int rows = min(R, cur.seq.n * G - rb * R);
    const int last = f + min(cur.nch - cur.ch, F - f) - 1;  // of this unit in the share
    {  // a unit (or piece) begins
      uint4 qraw[NT][W];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        const int r = nt * 8 + g;
#pragma unroll
        for (int j = 0; j < W; ++j) qraw[nt][j] = make_uint4(0u, 0u, 0u, 0u);
        if (r < rows) {
          const int i = rb * R + r;
          const uint16_t* q = p.q.p + (long long)(cur.seq.row0 + p.by_G.div(i)) * p.q.st +
                              (long long)(h * G + p.by_G.mod(i)) * p.q.sh + t * (D / 4);
#pragma unroll
          for (int j = 0; j < W; ++j) qraw[nt][j] = *reinterpret_cast<const uint4*>(q + j * 8);
        }
      }
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
        for (int j = 0; j < W; ++j)
          mx = __vmaxu2(mx, __vmaxu2(__vmaxu2(v[j].x & 0x7fff7fffu, v[j].y & 0x7fff7fffu),
                                     __vmaxu2(v[j].z & 0x7fff7fffu, v[j].w & 0x7fff7fffu)));
        mx = max(mx & 0xffffu, mx >> 16);
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = max(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        // 2^(14 - exponent of the largest element); rows of zeros or with inf or NaN stay
        int e = (int)(mx >> 7);
        e = (mx == 0u || e == 255) ? 0 : min(14 - (e - 127), 126);
        const float mul = __uint_as_float((uint32_t)(e + 127) << 23);
        const float back = __uint_as_float((uint32_t)(127 - e) << 23);
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const uint32_t* x = &v[w].x;
#pragma unroll
          for (int m = 0; m < 2; ++m) {  // channels i and i + 4 of eight, as int4_values gives them
            qf[nt][2 * w + m][0] = pack_f16x2(__uint_as_float(x[m] << 16) * mul,
                                              __uint_as_float(x[m + 2] << 16) * mul);
            qf[nt][2 * w + m][1] = pack_f16x2(__uint_as_float(x[m] & 0xffff0000u) * mul,
                                              __uint_as_float(x[m + 2] & 0xffff0000u) * mul);
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          const int col = 2 * t + i;
          fac[nt][i] = fmaxf(__shfl_sync(0xffffffffu, back, col * 4) * (p.scale_log2 * kInt4Unit),
                             1.17549435e-38f);  // positive: -inf stays what it is
          lim[nt][i] = nt * 8 + col < rows ? min(cur.seq.len, limit_of(nt * 8 + col)) : 0;
          ref[nt][i] = bound[nt][i] = -INFINITY;
          nref[nt][i] = 0.f;
          lsum[nt][i] = 0.f;
        }
      }
#pragma unroll
      for (int mt = 0; mt < MT; ++mt)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[mt][nt][i] = 0.f;
      far = false;
    }

    // ---------------------------------------------------------------- its tiles
    int key0 = cur.ch * C::CHUNK + warp * C::KEYS;
    cur.ch += last - f;
    for (;; ++f, key0 += C::CHUNK) {
      issue();
      copies_wait<ST - 1>();
      __syncwarp();
      bool on[C::PARTS], any = false, all = true;
#pragma unroll
      for (int pt = 0; pt < C::PARTS; ++pt) {
        on[pt] = (live[pt] >> (ST - 1) & 1u) != 0u;
        any |= on[pt], all &= on[pt];
      }
      if (any) {
        float s[C::PARTS][NT][4];
#pragma unroll
        for (int pt = 0; pt < C::PARTS; ++pt) {
          uint32_t a[2][W];         // keys krow and krow + 8
          Int4Scale sc[2][W / 2];   // of their groups of 16
          const uint32_t at = slot + ka0 + pt * (16 * C::ROW);
          const uint32_t sa = slot + ks0 + pt * C::PART_SCL;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            if constexpr (D == 128) {
              const uint4 x = ld_shared_v4(at + i * 8 * C::ROW);
              a[i][0] = x.x, a[i][1] = x.y, a[i][W - 2] = x.z, a[i][W - 1] = x.w;
              const uint32_t s2 = ld_shared_u16(sa + i * 64);
              sc[i][0] = int4_scale(__byte_perm(s2, 0u, 0x0404u));
              sc[i][W / 2 - 1] = int4_scale(__byte_perm(s2, 0u, 0x1414u));
            } else {
              const uint2 x = ld_shared_v2(at + i * 8 * C::ROW);
              a[i][0] = x.x, a[i][1] = x.y;
              sc[i][0] = int4_scale(__byte_perm(ld_shared_u8(sa + i * 32), 0u, 0x0404u));
            }
          }
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int i = 0; i < 4; ++i) s[pt][nt][i] = 0.f;
#pragma unroll
          for (int w = 0; w < W; ++w) {
            uint32_t lo[4], hi[4];
            int4_values(a[0][w], sc[0][w >> 1], magic, lo);
            int4_values(a[1][w], sc[1][w >> 1], magic, hi);
#pragma unroll
            for (int m = 0; m < 2; ++m)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt)
                mma_f16(s[pt][nt], lo[2 * m], hi[2 * m], lo[2 * m + 1], hi[2 * m + 1],
                        qf[nt][2 * w + m][0], qf[nt][2 * w + m][1]);
          }
        }
        // some row does not see all of it, or a part has no keys (and its slot holds anything)
        const bool masked = key0 + C::KEYS > lim_lo || !all;
        if (masked) {
#pragma unroll
          for (int pt = 0; pt < C::PARTS; ++pt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                if (!on[pt] || key0 + pt * 16 + krow + 8 * (i >> 1) >= lim[nt][i & 1])
                  s[pt][nt][i] = -INFINITY;
        }
        float top[NT][2];  // this lane's largest x
        bool move = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float m = fmaxf(s[0][nt][i], s[0][nt][i + 2]);
#pragma unroll
            for (int pt = 1; pt < C::PARTS; ++pt) m = fmax3(m, s[pt][nt][i], s[pt][nt][i + 2]);
            top[nt][i] = m * fac[nt][i];
            move |= top[nt][i] > bound[nt][i];
          }
        if (__any_sync(0xffffffffu, move)) {
          bool wide = false;
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
              nref[nt][i] = to == -INFINITY ? 0.f : -to;
              bound[nt][i] = to + kRoom;
              wide |= fabsf(nref[nt][i]) >= kFar;
              lsum[nt][i] *= alpha[i];
            }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[mt][nt][i] *= alpha[i & 1];
          }
          far = __any_sync(0xffffffffu, wide);
        }
        if (__builtin_expect(far, 0)) {
#pragma unroll
          for (int pt = 0; pt < C::PARTS; ++pt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[pt][nt][i] = __fadd_rn(__fmul_rn(s[pt][nt][i], fac[nt][i & 1]), nref[nt][i & 1]);
        } else {
#pragma unroll
          for (int pt = 0; pt < C::PARTS; ++pt)
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int i = 0; i < 4; ++i)
                s[pt][nt][i] = fmaf(s[pt][nt][i], fac[nt][i & 1], nref[nt][i & 1]);
        }
#pragma unroll
        for (int pt = 0; pt < C::PARTS; ++pt) {
          uint32_t pf[NT][2];
#pragma unroll
          for (int nt = 0; nt < NT; ++nt) {
            float pr[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) pr[i] = ex2(s[pt][nt][i]);
#pragma unroll
            for (int i = 0; i < 2; ++i) lsum[nt][i] += pr[i] + pr[i + 2];
            pf[nt][0] = movmatrix(pack_f16x2(pr[0], pr[1]));
            pf[nt][1] = movmatrix(pack_f16x2(pr[2], pr[3]));
          }
          uint32_t v[4][VW], sv[4];  // keys 2t, 2t + 1, 2t + 8, 2t + 9 of the matrix
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const uint32_t at = slot + va0[i & 1] + pt * (16 * C::ROW) + (i >> 1) * 8 * C::ROW;
            if constexpr (D == 128) {
              const uint2 x = ld_shared_v2(at);
              v[i][0] = x.x, v[i][VW - 1] = x.y;
            } else {
              v[i][0] = ld_shared_u32(at);
            }
            sv[i] = ld_shared_u8(slot + vs0[i & 1] + pt * C::PART_SCL + (i >> 1) * (D / 2));
          }
          if (masked) {
            // rows that no query sees hold anything; a scale that is none must not reach the
            // queries that do not see its row
#pragma unroll
            for (int i = 0; i < 4; ++i)
              sv[i] = !on[pt] || key0 + pt * 16 + krow4(t, i & 1) + 8 * (i >> 1) >= lim_hi
                          ? 0u
                          : int4_sane(sv[i]);
          }
          const Int4Scale s0 = int4_scale(__byte_perm(sv[0], sv[1], 0x4101u));
          const Int4Scale s1 = int4_scale(__byte_perm(sv[2], sv[3], 0x4101u));
#pragma unroll
          for (int j = 0; j < VW; ++j)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              uint32_t lo[4], hi[4];
              int4_values(__byte_perm(v[0][j], v[1][j], half ? 0x7632u : 0x5410u), s0, magic, lo);
              int4_values(__byte_perm(v[2][j], v[3][j], half ? 0x7632u : 0x5410u), s1, magic, hi);
#pragma unroll
              for (int m = 0; m < 2; ++m)
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
                  mma_f16(acc[j * 4 + half * 2 + m][nt], lo[2 * m], lo[2 * m + 1], hi[2 * m],
                          hi[2 * m + 1], pf[nt][0], pf[nt][1]);
            }
        }
      }
      slot = slot == ring + (ST - 1) * C::STAGE ? ring : slot + C::STAGE;
      __syncwarp();  // the slot may be loaded again
      if (f == last) break;
    }
    ++f;
    end_unit<C, D>(p, cur, f, share, rows, acc, ref, lsum, (float)kInt4UnitLog2, vcol, red, stat,
                   part_lse, part_o, h, rb, G, &rec);
    advance<C>(p, &cur, 1);
  }
  copies_wait<0>();
  if (threadIdx.x == 0) records[blockIdx.x] = rec;
  // launched behind the 256-row kernel, this one may overtake it; the merge must not
  asm volatile("griddepcontrol.wait;" ::: "memory");
}

template <int D, int NT>
cudaError_t launch(const CacheFwdParams& p, int n_sm, bool wide, cudaStream_t stream, int* grid,
                   int* R) {
  using C = Dec4<D, NT>;
  static_assert(C::CTAS * (C::SMEM + 1024) <= 233472, "shared memory of the CTAs sharing an SM");
  static unsigned long long prepared[64];
  const cudaError_t e = prepare_once(prepared, [] {
    return cudaFuncSetAttribute(cache4_fwd_kernel<D, NT>,
                                cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM);
  });
  if (e != cudaSuccess) return e;
  *grid = n_sm * C::CTAS;
  *R = C::R;
  return launch_split(cache4_fwd_kernel<D, NT>, *grid, C::SMEM, wide, stream, p);
}

}  // namespace

cudaError_t launch_cache4_fwd(const CacheFwdParams& p, int n_sm, bool wide, cudaStream_t stream,
                              int* grid, int* R) {
  const bool one = (long long)p.c.max_seqlen * p.G <= 8;
  if (p.c.d == 128)
    return one ? launch<128, 1>(p, n_sm, wide, stream, grid, R)
               : launch<128, 2>(p, n_sm, wide, stream, grid, R);
  return one ? launch<64, 1>(p, n_sm, wide, stream, grid, R)
             : launch<64, 2>(p, n_sm, wide, stream, grid, R);
}

}  // namespace fattn

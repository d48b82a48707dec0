// cache_split.cuh -- what the cache attention kernels for few query rows share (8 and 4 bits):
// the cut of all units' chunks of keys into one equal share per CTA, and the end of a unit
// or of its piece in a share.  A kernel's traits C give D's tile: CHUNK, the keys that its
// kWarps warps take together, R = 8 NT, the query rows of a unit.
#pragma once
#include <math.h>

#include "cache.cuh"

namespace fattn {
namespace {

constexpr float kLn2 = 0.6931471805599453f;
constexpr float kOff = 8.f;    // the reference lies this far below the running maximum
constexpr float kRoom = 15.f;  // and moves when a y exceeds it by more
constexpr float kFar = 4194304.f;
constexpr int kWarps = 4;
// Of the kernels, for 8 nt query rows a unit: rows of a unit and CTAs per SM, by which the
// workspace is sized.
constexpr int split_rows(int nt) { return 8 * nt; }
constexpr int split_ctas(int d, int nt) { return nt == 1 || d == 64 ? 3 : 2; }

// A position in the list of all chunks: chunk ch of unit (sequence b, head h, row
// block rb).  Sequence b has H x nrb units of nch chunks (none: nch = 0).
struct Cursor {
  int b, h, rb, ch;
  int nch, nrb;
  CacheSeq seq;
};
template <typename C>
__device__ __forceinline__ void set_seq(const CacheFwdParams& p, int b, int row0, int end,
                                        int len, Cursor* c) {
  c->b = b;
  c->nch = c->nrb = 0;
  if (!cache_seq(p.c, row0, end, len, &c->seq)) {
    if (p.c.err) atomicCAS(p.c.err, 0u, (unsigned)ERR_SITE_CACHE_FWD);
    return;
  }
  const int rows = c->seq.n * p.G;
  if (rows == 0 || rows > p.narrow_rows) return;  // (the other kernel's)
  c->nch = max(1, (c->seq.len + C::CHUNK - 1) / C::CHUNK);
  c->nrb = (rows + C::R - 1) / C::R;
}
template <typename C>
__device__ __forceinline__ void load_seq(const CacheFwdParams& p, int b, Cursor* c) {
  set_seq<C>(p, b, p.c.cu_seqlens[b], p.c.cu_seqlens[b + 1], p.c.lens[b], c);
}
template <typename C>
__device__ __forceinline__ void advance(const CacheFwdParams& p, Cursor* c, int by) {
  c->ch += by;
  while (c->ch >= c->nch) {
    c->ch -= c->nch;
    if (++c->rb < c->nrb) continue;
    c->rb = 0;
    if (++c->h < p.c.H) continue;
    c->h = 0;
    int b = c->b;
    do {
      if (++b >= p.c.B) {
        c->b = b;
        c->nch = 0x7fffffff;  // behind the last chunk
        return;
      }
      load_seq<C>(p, b, c);
    } while (c->nch == 0);
  }
}

// The place where this CTA's share of all chunks begins, its number of chunks (the return
// value) and that of a share.  first_*: the entries of sequence `lane`.
template <typename C>
__device__ __forceinline__ int find_share(const CacheFwdParams& p, int first_row0, int first_end,
                                          int first_len, Cursor* at, long long* chunks_each) {
  const int B = p.c.B, lane = threadIdx.x & 31;
  Cursor& cur = *at;
  auto chunks = [&](const Cursor& c) { return (long long)c.nch * c.nrb * p.c.H; };
  cur = Cursor{};
  long long mine = 0, total = 0;  // chunks of sequence `lane` of the last group, and of all
  for (int b0 = 0; b0 < B; b0 += 32) {
    mine = 0;
    if (b0 + lane < B) {
      if (b0 == 0)
        set_seq<C>(p, lane, first_row0, first_end, first_len, &cur);
      else
        load_seq<C>(p, b0 + lane, &cur);
      mine = chunks(cur);
    }
    total += mine;
  }
#pragma unroll
  for (int w = 16; w > 0; w >>= 1) total += __shfl_xor_sync(0xffffffffu, total, w);
  // (a 64-bit division takes ten times as long)
  const long long share = total < 0x7fffffff ? ((unsigned)total + gridDim.x - 1) / gridDim.x
                                   : (total + gridDim.x - 1) / gridDim.x;
  const long long lo = blockIdx.x * share;
  *chunks_each = share;
  const int F = (int)max(0LL, min(share, total - lo));  // chunks of this CTA
  if (F > 0) {
    long long before = 0;
    for (int b0 = 0; b0 < B; b0 += 32) {
      if (B > 32) {
        mine = 0;
        if (b0 + lane < B) {
          load_seq<C>(p, b0 + lane, &cur);
          mine = chunks(cur);
        }
      }
      long long upto = mine;
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const long long o = __shfl_up_sync(0xffffffffu, upto, d);
        if (lane >= d) upto += o;
      }
      const unsigned past = __ballot_sync(0xffffffffu, before + upto > lo);
      if (past) {
        const int src = __ffs(past) - 1;
        const long long pos = lo - __shfl_sync(0xffffffffu, before + upto - mine, src);
        cur.b = b0 + src;
        cur.nch = __shfl_sync(0xffffffffu, cur.nch, src);
        cur.nrb = __shfl_sync(0xffffffffu, cur.nrb, src);
        cur.seq.row0 = __shfl_sync(0xffffffffu, cur.seq.row0, src);
        cur.seq.n = __shfl_sync(0xffffffffu, cur.seq.n, src);
        cur.seq.len = __shfl_sync(0xffffffffu, cur.seq.len, src);
        const unsigned unit = pos < 0x7fffffff ? (unsigned)pos / (unsigned)cur.nch
                                               : (unsigned)(pos / cur.nch);
        cur.ch = (int)(pos - (long long)unit * cur.nch);
        cur.h = (int)(unit / (unsigned)cur.nrb);
        cur.rb = (int)(unit % (unsigned)cur.nrb);
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
    }
  }
  return F;
}

__device__ __forceinline__ void mma_f16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                        uint32_t a3, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t movmatrix(uint32_t x) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(x));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(a));
  return v;
}
__device__ __forceinline__ uint2 ld_shared_v2(uint32_t a) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u32(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u16(uint32_t a) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(a));
  return v;
}
__device__ __forceinline__ uint32_t ld_shared_u8(uint32_t a) {
  uint32_t v;
  asm volatile("ld.shared.u8 %0, [%1];" : "=r"(v) : "r"(a));
  return v;
}

// A unit (or its piece in this share) ends in front of tile f: the four warps' sums are
// joined, and the rows go to o and lse or, of a piece, to the workspace.  Lane (g, t) holds
// the columns vcol + 2 mt, + 1 (acc[mt][nt][i], [i + 2]) of rows 8 nt + 2 t + i.  O = 2^lvb acc /
// l.  `red` [warps][R][D] and `stat` [warps][R] are the CTA's; h, rb, G are the unit's.
template <typename C, int D, int NT>
__device__ __forceinline__ void end_unit(const CacheFwdParams& p, const Cursor& cur, int f,
                                         long long share, int rows,
                                         const float (&acc)[D / 16][NT][4],
                                         const float (&ref)[NT][2], float (&lsum)[NT][2],
                                         float lvb, int vcol, float* red, float* stat,
                                         float* part_lse, float* part_o, int h, int rb, int G,
                                         Record* rec) {
  constexpr int R = C::R, VW = D / 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int ch = cur.ch;
  const bool unit_ends = ch == cur.nch - 1;
  // this warp's rows: normalised result and log2-sum-exp
  float mine[NT][2], fac[NT][2];
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      float l = lsum[nt][i];
#pragma unroll
      for (int w = 4; w < 32; w <<= 1) l += __shfl_xor_sync(0xffffffffu, l, w);
      lsum[nt][i] = l;
      mine[nt][i] = l == 0.f ? -INFINITY : ref[nt][i] + lg2(l);
      if (g == 0) stat[warp * R + nt * 8 + 2 * t + i] = mine[nt][i];
    }
  __syncthreads();
  float top[NT][2], sum[NT][2];
  const float up = ex2(lvb);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = nt * 8 + 2 * t + i;
      float m = -INFINITY, z = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) m = fmaxf(m, stat[w * R + r]);
      const float mm = m == -INFINITY ? 0.f : m;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) z += ex2(stat[w * R + r] - mm);
      top[nt][i] = m;
      sum[nt][i] = z;
      fac[nt][i] = lsum[nt][i] == 0.f ? 0.f : ex2(mine[nt][i] - mm) / (z * lsum[nt][i]);
    }
  // the warps' results side by side; 16-byte columns are permuted so that the lanes
  // of a store phase (two g, four t) touch different banks
  auto column = [&](int r, int c4) {
    const int k = r >> 1;  // t of the lane that holds row r
    return D == 128 ? c4 ^ (((c4 >> 4) & 1) << 2 | (k & 3))
                    : c4 ^ ((k & 1) << 2 | ((k >> 1) & 1));
  };
  float4* red4 = reinterpret_cast<float4*>(red);
#pragma unroll
  for (int nt = 0; nt < NT; ++nt)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = nt * 8 + 2 * t + i;
#pragma unroll
      for (int j = 0; j < VW; ++j)
        red4[(warp * R + r) * (D / 4) + column(r, vcol / 4 + j)] = make_float4(
            acc[2 * j][nt][i] * fac[nt][i] * up, acc[2 * j][nt][i + 2] * fac[nt][i] * up,
            acc[2 * j + 1][nt][i] * fac[nt][i] * up,
            acc[2 * j + 1][nt][i + 2] * fac[nt][i] * up);
    }
  __syncthreads();
  const bool starts_here = f > ch;  // the unit's chunk 0 is in this share
  const bool whole = starts_here && unit_ends;
  const int slot = starts_here ? 1 : 0;
  if (warp == 0 && g == 0) {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = nt * 8 + 2 * t + i;
        const float L = top[nt][i] == -INFINITY && sum[nt][i] == 0.f
                            ? -INFINITY
                            : (top[nt][i] + lg2(sum[nt][i])) * kLn2;
        if (r < rows) {
          if (whole) {
            const int i0 = rb * R + r;
            p.lse[(long long)(h * G + p.by_G.mod(i0)) * p.c.total + cur.seq.row0 +
                  p.by_G.div(i0)] = L;
          } else {
            part_lse[((size_t)blockIdx.x * 2 + slot) * R + r] = L;
          }
        }
      }
  }
  for (int x = threadIdx.x; x < rows * (D / 4); x += 128) {
    const int r = x / (D / 4), c4 = x % (D / 4);
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kWarps; ++w) {
      const float4 y = red4[(w * R + r) * (D / 4) + column(r, c4)];
      o.x += y.x, o.y += y.y, o.z += y.z, o.w += y.w;
    }
    if (whole) {
      const int i0 = rb * R + r;
      *reinterpret_cast<uint2*>(p.o.p + (long long)(cur.seq.row0 + p.by_G.div(i0)) * p.o.st +
                                (long long)(h * G + p.by_G.mod(i0)) * p.o.sh + c4 * 4) =
          make_uint2(pack_bf16x2(o.x, o.y), pack_bf16x2(o.z, o.w));
    } else {
      reinterpret_cast<float4*>(part_o)[(((size_t)blockIdx.x * 2 + slot) * R + r) * (D / 4) +
                                        c4] = o;
    }
  }
  if (starts_here && !unit_ends) {  // later CTAs hold the rest
    rec->parts = 1 + (cur.nch - 1 - ch + (int)share - 1) / (int)share;
    rec->rows = rows;
    rec->h = h;
    rec->row0 = cur.seq.row0;
    rec->first_row = rb * R;
  }
}

// Launch of one of the kernels.  Behind the 256-row kernel it may start while that one's
// last CTAs finish; what depends on its results is waited for on the device.
template <typename... P, typename... A>
cudaError_t launch_split(void (*kernel)(P...), int grid, int smem, bool wide, cudaStream_t stream,
                         const A&... args) {
  cudaLaunchConfig_t cfg{};
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3(32 * kWarps);
  cfg.dynamicSmemBytes = (size_t)smem;
  cfg.stream = stream;
  if (wide) {
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
  }
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

}  // namespace

// The 4-bit kernel; gives the CTAs and the rows per unit that the merge is to know.
cudaError_t launch_cache4_fwd(const CacheFwdParams& p, int n_sm, bool wide, cudaStream_t stream,
                              int* grid, int* R);

}  // namespace fattn

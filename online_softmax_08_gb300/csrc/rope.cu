// rope.cu -- rotary positions of queries and keys.
//
// A pair of channels (a, b) of a token at position p turns by the angle p w_i:
//   a' = m (a cos - b sin),  b' = m (a sin + b cos),
// w_i the pair's frequency and m one magnitude for all (1 but for scaled contexts).  The
// gradient is the transpose, which turns the other way.
//
// The angle is formed without rounding: w_i / 2 pi is given as a 64-bit fraction of a turn, so
// p times it, modulo 2^64, is the angle's fraction of a turn at any 32-bit position; its upper
// 32 bits, taken as a signed number, are what sincospi gets.  (In fp32, p w_i at p = 10^6 is
// off by 0.03 radians.)
//
// The bound is memory: every value is read and written once.  A thread holds 8 pairs, so
// eight sines and cosines, and takes them through the heads of its token, queries and keys:
// 32 bytes of a row, as two 16-byte pieces.  kUnroll heads' loads are in flight at a time.
// Measured: 16384 tokens of 32 + 8 heads, d = 128, 53 us, 6340 GB/s, 93 % of the measured copy
// bandwidth; 64 tokens 2.9 us.
#include "rope.cuh"

namespace fattn {
namespace {

constexpr int kUnroll = 4;
constexpr int kThreads = 128;

// D / 16 lanes take a row, 512 / D rows a warp at a time.  A warp's heads: passes [y, y + 1) x
// `passes` of its token, kUnroll of them at once.
template <int D, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const RopeParams p) {
  constexpr int LPR = D / 16, RPW = 32 / LPR;
  const int lane = threadIdx.x & 31, c = lane % LPR;
  const int tok = (int)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
  if (tok >= p.T) return;
  const int half = p.rot >> 1, turning = p.rot >> 4;  // lanes that turn their channels
  // first channels of the thread's two pieces
  const int c0 = c >= turning || INTERLEAVED ? c * 16 : c * 8;
  const int c1 = c >= turning || INTERLEAVED ? c0 + 8 : c0 + half;
  const int rows = p.Hq + p.Hk;
  const int first = (int)blockIdx.y * p.passes * RPW;
  const int last = min(rows, first + p.passes * RPW);
  if (first >= rows) return;

  uint4 x[kUnroll][2];
  auto load = [&](int r0) {
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * RPW + lane / LPR;
      if (r >= last) continue;
      const TokenView& v = r < p.Hq ? p.q : p.k;
      const uint16_t* at = v.p + (long long)tok * v.st + (long long)(r < p.Hq ? r : r - p.Hq) * v.sh;
      x[u][0] = *reinterpret_cast<const uint4*>(at + c0);
      x[u][1] = *reinterpret_cast<const uint4*>(at + c1);
    }
  };
  load(first);
  float cs[8], sn[8];
  if (c < turning) {
    const long long pos = p.positions[tok];
    const unsigned long long* w = p.turns + c * 8;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int frac = (int)(((unsigned long long)pos * w[i]) >> 32);
      sincospif((float)frac * 4.656612873077393e-10f, &sn[i], &cs[i]);  // 2^-31: in half turns
      cs[i] *= p.magnitude;
      sn[i] *= p.back ? -p.magnitude : p.magnitude;
    }
  }
  for (int r0 = first; r0 < last; r0 += kUnroll * RPW) {
    if (r0 > first) load(r0);
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const int r = r0 + u * RPW + lane / LPR;
      if (r >= last) continue;
      if (c < turning) {
        uint32_t* a = &x[u][0].x;
        uint32_t* b = &x[u][1].x;
        if (INTERLEAVED) {
#pragma unroll
          for (int i = 0; i < 8; ++i) {  // word i: one pair
            uint32_t& v = i < 4 ? a[i] : b[i - 4];
            const float lo = __uint_as_float(v << 16), hi = __uint_as_float(v & 0xffff0000u);
            v = pack_bf16x2(lo * cs[i] - hi * sn[i], lo * sn[i] + hi * cs[i]);
          }
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) {  // word i of the two pieces: two pairs
            const float a0 = __uint_as_float(a[i] << 16), a1 = __uint_as_float(a[i] & 0xffff0000u);
            const float b0 = __uint_as_float(b[i] << 16), b1 = __uint_as_float(b[i] & 0xffff0000u);
            a[i] = pack_bf16x2(a0 * cs[2 * i] - b0 * sn[2 * i],
                               a1 * cs[2 * i + 1] - b1 * sn[2 * i + 1]);
            b[i] = pack_bf16x2(a0 * sn[2 * i] + b0 * cs[2 * i],
                               a1 * sn[2 * i + 1] + b1 * cs[2 * i + 1]);
          }
        }
      }
      const TokenView& v = r < p.Hq ? p.q_out : p.k_out;
      uint16_t* at = v.p + (long long)tok * v.st + (long long)(r < p.Hq ? r : r - p.Hq) * v.sh;
      *reinterpret_cast<uint4*>(at + c0) = x[u][0];
      *reinterpret_cast<uint4*>(at + c1) = x[u][1];
    }
  }
}

template <int D, bool INTERLEAVED>
cudaError_t start(RopeParams p, int n_sm, cudaStream_t stream) {
  constexpr int RPW = 512 / D, WARPS = kThreads / 32;
  // One warp a token, unless there are too few tokens for 16 warps on every SM: then a token's
  // heads are spread over several, each of which forms the sines again.
  const int all = (p.Hq + p.Hk + RPW - 1) / RPW;  // passes of a warp over a token
  const int want = std::max(1, 16 * n_sm / p.T);
  p.passes = std::max(1, (all + want - 1) / want);
  const dim3 grid((unsigned)((p.T + WARPS - 1) / WARPS), (unsigned)((all + p.passes - 1) / p.passes));
  rope_kernel<D, INTERLEAVED><<<grid, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeParams& p, int d, bool interleaved, int n_sm,
                        cudaStream_t stream) {
  if (d == 128)
    return interleaved ? start<128, true>(p, n_sm, stream) : start<128, false>(p, n_sm, stream);
  return interleaved ? start<64, true>(p, n_sm, stream) : start<64, false>(p, n_sm, stream);
}

}  // namespace fattn

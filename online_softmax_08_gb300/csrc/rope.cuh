// rope.cuh -- launch parameters of the rotary positions.
#pragma once
#include <algorithm>

#include "cache.cuh"

namespace fattn {

struct RopeParams {
  TokenView q, k, q_out, k_out;  // [T, heads, d]
  int T, Hq, Hk;
  int rot;                          // channels that turn
  const int* positions;             // [T]
  const unsigned long long* turns;  // [rot / 2], in 2^-64 turns per position
  float magnitude;
  int back;                         // the gradient: turns the other way
  int passes;                       // of a warp over the heads of its token
};
cudaError_t launch_rope(const RopeParams& p, int d, bool interleaved, int n_sm,
                        cudaStream_t stream);

}  // namespace fattn

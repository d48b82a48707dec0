// evict.cuh -- launch parameters of the cached keys' attention weights and of the eviction
// that goes by them.
#pragma once
#include "cache.cuh"

namespace fattn {

// Codes of the device error word: + 0 bad sequence entry, + 1 bad block number
enum : uint32_t { ERR_SITE_CACHE_WEIGHTS = 0x470, ERR_SITE_CACHE_EVICT = 0x480 };

// Weights of a batch's keys, fp32 by element strides, `width` of each sequence and head.
struct WeightView {
  float* p;
  long long sb, sh;
};

struct WeightParams {
  CacheParams c;
  TokenView q;
  const float* lse;  // [Hq, total]
  WeightView in, out;
  int accumulate;    // whether `in` is read
  int width;
  int G;
  FastDiv by_G;
  int causal;
  float scale_log2;
  int narrow_rows;   // sequences with more query rows per key/value head go to the tcgen05 kernel
  int tile_tokens;   // of its tiles of rows: 256 / G
  FastDiv by_tile;
};
cudaError_t launch_cache_weights(const WeightParams& p, int n_sm, cudaStream_t stream);
// tq: map of q, {d, Hq, total}, boxes {64, G, tile_tokens}
cudaError_t launch_cache_weights_wide(const CUtensorMap& tq, const WeightParams& p, int n_sm,
                                      cudaStream_t stream);

struct EvictParams {
  CacheParams c;       // cu_seqlens, total and max_seqlen are not used
  WeightView in, out;
  int width;
  const int* table_out;
  int table_out_width;
  int keep, recent;
  int* lens_out;
  int* kept;           // [B, H, keep]
};
cudaError_t launch_cache_evict(const EvictParams& p, int n_sm, cudaStream_t stream);

}  // namespace fattn

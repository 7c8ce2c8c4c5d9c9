// scored_prefill.h -- the scored chunked prefill (scored_prefill.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace rswa {

struct ScoredPrefillLaunch {
  int B, H, n, T;
  int64_t cap;
  const void* q;
  const void* k_out;
  const void* v_out;
  const void* pk;  // pk, pv, prefix_len: not read when cap == 0
  const void* pv;
  const int32_t* prefix_len;
  const void* ring_k;  // NULL: no previous chunk
  const void* ring_v;
  const int32_t* wp;
  const int32_t* fill;
  float scale, softcap;
  const float* slopes;
  const int32_t* pos;
  const int2* ranges;
  void* out;
  float* lse;
  int write_ring;
  void* ring_k_w;  // the same buffers as ring_k / ring_v / wp / fill
  void* ring_v_w;
  int32_t* wp_w;
  int32_t* fill_w;
  int32_t* status;
  uint64_t wait_limit_ns;  // as in BalancedArgs; the tile: the key tile of the first CTA
  int drop_tile;
};
cudaError_t launch_scored_prefill(const ScoredPrefillLaunch& L, cudaStream_t stream);

}  // namespace rswa

// shared.h -- the shared part of shared-prefix decode (shared.cu).
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

#include "balanced.h"

namespace rswa {

constexpr int kMaxShared = 8192;  // prefixes of a call (the grouping's shared-memory table)

// Offsets of the tables and records in launch_shared's scratch.
struct SharedPlan {
  size_t head, tiles, order, seqs, records, bytes;
};
SharedPlan plan_shared(int B, int H, int P);

struct SharedLaunch {
  int B, H, P;
  int64_t cap;
  const uint16_t* q;
  const void* sk;
  const void* sv;
  const int32_t* shared_len;
  const int32_t* share_of;
  float scale;
  int32_t* status;
  uint64_t wait_limit_ns;  // as in BalancedArgs; the tile: the key tile of the first CTA
  int drop_tile;
};
// Groups the sequences and attends to the shared prefixes; *tables is for launch_balanced.
cudaError_t launch_shared(const SharedLaunch& L, void* scratch, SharedTables* tables, cudaStream_t stream);

}  // namespace rswa

// balanced.h -- the evenly cut single-token attention (balanced.cu) and the tables and records
// that the shared part of shared-prefix decode (shared.cu) hands to it.
#pragma once

#include <cstddef>
#include <cstdint>
#include <cuda_runtime.h>

namespace rswa {

constexpr int kMaxPos = 1 << 30;       // largest query position of a distance bias
constexpr int kRecordFloats = 4 + 128;  // max, sum of the weights that met V, sum of the weights, -, accumulator
constexpr int kSharedRows = 256;        // sequences that one pass over a shared prefix serves

// Up to kSharedRows sequences over one shared prefix. Units of the shared part: key tiles of 128,
// a tile's heads one after the other. (The entry point keeps the units of a call below 2^31.)
struct SharedTile {
  int first_unit;
  int first_seq;  // its sequences: order[first_seq .. first_seq + rows)
  int rows;
  int prefix;
  int len;        // rows of the prefix
  int key_tiles;
  int pad[2];
};

// Where a sequence's shared part is: row `row` (-1: it has none) of a tile with these fields.
struct SharedSeq {
  int row, first_seq, rows, key_tiles, first_unit;
  int pad[3];
};

struct SharedHead {
  int units;  // of all tiles and heads
  int per;    // units a CTA takes: CTA c has [c per, (c + 1) per)
  int tiles;
  int pad;
};

struct SharedTables {
  SharedHead* head;     // null: no shared part
  SharedTile* tiles;
  int32_t* order;       // sequences, grouped by prefix
  SharedSeq* seqs;      // by sequence
  float* records;       // [B * H + CTAs * kSharedRows][kRecordFloats]
};

struct BalancedArgs {
  int B, H, n;
  int64_t cap;
  const uint16_t* q;
  const uint16_t* pk;
  const uint16_t* pv;
  const int32_t* prefix_len;  // not read when cap == 0
  const uint16_t* ring_k;
  const uint16_t* ring_v;
  const int32_t* wp;
  const int32_t* fill;
  float scale;
  void* out;  // f32; bf16 with a shared part
  float* lse;
  int32_t* status;
  // scored decode
  float softcap;           // 0: none
  const float* slopes;     // [H] or null
  const int32_t* pos;      // [B], with slopes
  const int2* ranges;      // [B] or null: the whole prefix
  SharedTables shared;
  // as in DecodeArgs: the limit of every wait, and a test's dropped unit of CTA 0 (-1: none)
  uint64_t wait_limit_ns;
  int drop_tile;
  // set by launch_balanced
  int32_t* counters;
  float* records;
};

int balanced_grid();
size_t balanced_scratch_bytes();  // of launch_balanced's zero-filled scratch
cudaError_t launch_balanced(BalancedArgs a, void* scratch, cudaStream_t stream);

}  // namespace rswa

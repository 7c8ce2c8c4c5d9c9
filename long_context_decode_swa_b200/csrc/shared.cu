// shared.cu -- the shared part of shared-prefix decode: many sequences, each with one query a
// head, over few long prefixes that they have in common.
//
// Each shared key / value row is read once for up to 256 sequences instead of once a sequence:
// the queries of a prefix's sequences are gathered into 128-row tiles and the products run on
// the tensor cores (tcgen05, accumulators in TMEM), scores S = Q K^T and O += P V, P = exp(S - max)
// rounded to bf16. What bounds it: at up to about 128 sequences a prefix the K / V bytes (64 KiB a
// key tile of 128 rows, some 2,700 cycles of one SM's share of HBM, against 1,024 cycles of MMA
// and as many of exponentials a tile of queries); above that the exponentials' chain of latencies.
// Measured: 64 sequences over 102,400 rows 167 to 177 us (138 at the copy rate), 512 over 64 times 2,592
// 311 to 350 (290).
//
// Grouping sorts the sequences by prefix and lays the tables out: a launch of one CTA (group_kernel), or,
// with at most 384 sequences and prefixes, by every CTA of the attention for itself, which saves the
// launch (3 us of a call's host time; eight sequences over one page 10.7 -> 10.0 us on the GPU).
// shared_kernel: one CTA an SM;
// the work is a line of units (a key tile of one head of one tile of sequences) cut evenly over the
// CTAs, so few long prefixes fill the chip as well as many short ones. A CTA walks its run in
// segments, one per (tile, head), with roles as in the chunked prefill:
//   warp 0 / warp 2, lane 0 : TMA producers of the K / V tiles, running ahead across segments
//   warp 1, one thread      : issues the MMAs, and nothing else (the tensor core's queue is shallow:
//                             what it does between two MMAs is idle time)
//   warp 3                  : zeroes V rows past the prefix's end (0 * NaN)
//   warps 4-7, 8-11         : softmax groups A and B; thread r owns TMEM lane r of its group
// With more than 128 sequences in the tile the groups take 128 rows each and read the same keys;
// with fewer, both take the same rows and every other key tile, so that one group's exponentials
// run under the other's MMAs, and meet at the segment's end. A segment leaves one record a row
// (max, sum of the rounded weights, sum of the weights, f32 accumulator), which the launch that
// attends to the private rows joins. Every wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>

#include "balanced.h"
#include "common.cuh"
#include "internal.h"
#include "shared.h"
#include "tcgen05.cuh"

namespace rswa {

namespace {

constexpr int kRows = 128;                 // rows of a query tile, keys of a key tile
constexpr int kRegionBytes = kRows * 128;  // one 64-column 128-byte-swizzled region
constexpr int kTileBytes = 2 * kRegionBytes;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kLazyRescaleLog2 = 8.f;
constexpr int kGroupThreads = 1024;

// ---------------------------------------------------------------------------------------------
// grouping
// ---------------------------------------------------------------------------------------------

struct GroupArgs {
  int B, H, P;
  int64_t cap;
  int ctas;  // of the attention
  const int32_t* shared_len;
  const int32_t* share_of;
  SharedTables t;
  int32_t* status;
};

struct Counts {
  int seqs, tiles, units;
};

__device__ __forceinline__ Counts plus(const Counts& a, const Counts& b) {
  return Counts{a.seqs + b.seqs, a.tiles + b.tiles, a.units + b.units};
}

__device__ __forceinline__ Counts warp_scan(Counts v, int lane) {  // inclusive
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Counts t = Counts{__shfl_up_sync(0xffffffffu, v.seqs, o), __shfl_up_sync(0xffffffffu, v.tiles, o),
                            __shfl_up_sync(0xffffffffu, v.units, o)};
    if (lane >= o) v = plus(v, t);
  }
  return v;
}

// Exclusive scan of v over the block (warps: 32 entries of shared memory); total over all threads.
__device__ Counts block_scan(const Counts& v, Counts* warps, Counts& total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, n = blockDim.x >> 5;
  const Counts inc = warp_scan(v, lane);
  if (lane == 31) warps[warp] = inc;
  __syncthreads();
  const Counts sums = warp_scan(lane < n ? warps[lane] : Counts{0, 0, 0}, lane);
  total = Counts{__shfl_sync(0xffffffffu, sums.seqs, 31), __shfl_sync(0xffffffffu, sums.tiles, 31),
                 __shfl_sync(0xffffffffu, sums.units, 31)};
  const int from = warp > 0 ? warp - 1 : 0;
  Counts before = Counts{__shfl_sync(0xffffffffu, sums.seqs, from), __shfl_sync(0xffffffffu, sums.tiles, from),
                         __shfl_sync(0xffffffffu, sums.units, from)};
  if (warp == 0) before = Counts{0, 0, 0};
  __syncthreads();  // warps[] is written again
  return plus(before, Counts{inc.seqs - v.seqs, inc.tiles - v.tiles, inc.units - v.units});
}

// blockDim.x: a multiple of 32, at most 1,024.
__global__ void __launch_bounds__(kGroupThreads) group_kernel(const GroupArgs a) {
  extern __shared__ int tab[];
  int* count = tab;            // sequences of prefix p
  int* first = tab + a.P;      // its first place in order[]
  int* tile0 = tab + 2 * a.P;  // its first tile (-1: no rows, or nobody reads it)
  __shared__ Counts scan[kGroupThreads / 32];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, threads = blockDim.x;
  for (int p = tid; p < a.P; p += threads) count[p] = 0;
  griddep_wait();
  griddep_launch_dependents();
  __syncthreads();
  // Each sequence's rank among its prefix's. A row's arithmetic does not depend on its place in a
  // tile, so any order will do while a prefix's sequences fit one tile; where they do not, ranks go by the
  // sequences' order, so that their cut, and with it the rounding, is the same in every call.
  bool more = false;
  for (int base = 0; base < a.B; base += threads) {
    const int b = base + tid;
    int p = b < a.B ? a.share_of[b] : -1;
    if (p < -1 || p >= a.P) {
      set_status(a.status, RSWA_DEVICE_BAD_SHARE);
      p = -1;
    }
    const unsigned same = __match_any_sync(0xffffffffu, p);
    const int leader = __ffs(same) - 1;
    int rank = 0;
    if (lane == leader && p >= 0) rank = atomicAdd(&count[p], __popc(same));
    rank = __shfl_sync(0xffffffffu, rank, leader) + __popc(same & ((1u << lane) - 1));
    more |= p >= 0 && rank >= kSharedRows;
    if (b < a.B) {
      a.t.seqs[b].first_seq = p;  // until the end: prefix and rank
      a.t.seqs[b].row = rank;
    }
  }
  if (__syncthreads_or(more)) {
    for (int p = tid; p < a.P; p += threads) count[p] = 0;
    __syncthreads();
    for (int base = 0; base < a.B; base += threads) {
      const int b = base + tid;
      const int p = b < a.B ? a.t.seqs[b].first_seq : -1;
      const unsigned same = __match_any_sync(0xffffffffu, p);
      const int leader = __ffs(same) - 1;
      int rank = 0;
      for (int w = 0; w < threads / 32; ++w) {
        if (warp == w && lane == leader && p >= 0) {
          rank = count[p];
          count[p] = rank + __popc(same);
        }
        __syncthreads();
      }
      rank = __shfl_sync(0xffffffffu, rank, leader) + __popc(same & ((1u << lane) - 1));
      if (b < a.B) a.t.seqs[b].row = rank;
    }
  }
  Counts sum{0, 0, 0};  // so far
  for (int base = 0; base < a.P; base += threads) {
    const int p = base + tid;
    int n = p < a.P ? count[p] : 0;
    int len = 0;
    if (n > 0) {
      len = a.shared_len[p];
      if (len < 0 || len > a.cap) {
        set_status(a.status, RSWA_DEVICE_BAD_PREFIX_LEN);
        len = 0;
      }
      if (len == 0) n = 0;
    }
    const int nt = (n + kSharedRows - 1) / kSharedRows;
    const int keys = (len + kRows - 1) / kRows;
    const int each = keys * a.H;
    Counts total;
    const Counts at = plus(sum, block_scan(Counts{n, nt, nt * each}, scan, total));
    if (p < a.P) {
      first[p] = at.seqs;
      tile0[p] = nt > 0 ? at.tiles : -1;
      for (int i = 0; i < nt; ++i) {
        SharedTile t = {};
        t.first_unit = at.units + i * each;
        t.first_seq = at.seqs + i * kSharedRows;
        t.rows = min(kSharedRows, n - i * kSharedRows);
        t.prefix = p;
        t.len = len;
        t.key_tiles = keys;
        a.t.tiles[at.tiles + i] = t;
      }
    }
    sum = plus(sum, total);
  }
  if (tid == 0) {
    a.t.head->units = sum.units;
    a.t.head->per = max(1, (sum.units + a.ctas - 1) / a.ctas);
    a.t.head->tiles = sum.tiles;
  }
  __syncthreads();
  for (int b = tid; b < a.B; b += threads) {  // the rows this thread wrote above
    const int p = a.t.seqs[b].first_seq, rank = a.t.seqs[b].row;
    SharedSeq q = {};
    q.row = -1;
    if (p >= 0 && tile0[p] >= 0) {
      a.t.order[first[p] + rank] = b;
      const SharedTile t = a.t.tiles[tile0[p] + rank / kSharedRows];
      q.row = rank % kSharedRows;
      q.first_seq = t.first_seq;
      q.rows = t.rows;
      q.key_tiles = t.key_tiles;
      q.first_unit = t.first_unit;
    }
    a.t.seqs[b] = q;
  }
}

// ---------------------------------------------------------------------------------------------
// attention
// ---------------------------------------------------------------------------------------------

constexpr int kSmallGroup = kThreads;  // sequences and prefixes that a CTA's threads take one each
static_assert(5 * kSmallGroup * 4 + (kSmallGroup / 32) * 12 <= 8192, "group_small's scratch");

struct SharedSmem {
  uint8_t q[2][kTileBytes];
  uint8_t k[kKStages][kTileBytes];
  uint8_t v[kVStages][kTileBytes];
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_ready[kVStages], v_empty[kVStages];
  uint64_t s_full[2], p_full[2], o_done[2];
  uint64_t drain;
  uint64_t wait_limit_ns;  // of every wait
  uint32_t tmem_base;
  int abort_flag;
  float stat_m[2][kRows];              // at a segment's end: both groups' maxima,
  float stat_l[kRows], stat_lu[kRows];  // group B's sums
};
// the swizzled tiles need the struct at a 1,024-byte boundary, and there is no room to move it
static_assert(sizeof(SharedSmem) <= 227 * 1024, "shared memory");

struct AttnArgs {
  int B, H;
  int64_t cap;
  const uint16_t* q;
  float scale_log2;
  SharedTables t;
  int32_t* status;
  uint64_t wait_limit_ns;
  int drop_tile;           // a wait-timeout test: key tile that CTA 0 leaves out (-1: none)
  int group;     // 1: the tables are laid out in this launch, by group_small
  GroupArgs g;
};

// group_kernel's tables for at most kSmallGroup sequences and prefixes, by the whole CTA. Every CTA
// writes the same values and reads its own. scratch: 8 KiB of shared memory.
__device__ void group_small(const GroupArgs& a, int* scratch) {
  int* share = scratch;
  int* first = scratch + kSmallGroup;      // of a prefix: its first place in order[],
  int* tile0 = first + kSmallGroup;        // its first tile (-1: no rows, or nobody reads it),
  int* unit0 = tile0 + kSmallGroup;        // its first unit
  int* keys_of = unit0 + kSmallGroup;      // and its key tiles
  Counts* sums = reinterpret_cast<Counts*>(keys_of + kSmallGroup);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  int p = tid < a.B ? a.share_of[tid] : -1;
  int len = tid < a.P ? a.shared_len[tid] : 0;
  if (p < -1 || p >= a.P) {
    if (blockIdx.x == 0) set_status(a.status, RSWA_DEVICE_BAD_SHARE);
    p = -1;
  }
  share[tid] = p;
  __syncthreads();
  int rank = 0, n = 0;  // of sequence tid among its prefix's; sequences of prefix tid
  for (int j = 0; j < a.B; j += 4) {
    const int4 s4 = *reinterpret_cast<const int4*>(share + j);  // past B: -1
    const int s[4] = {s4.x, s4.y, s4.z, s4.w};
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      rank += s[u] == p && j + u < tid;
      n += s[u] == tid;
    }
  }
  if (n > 0 && (len < 0 || len > a.cap)) {
    if (blockIdx.x == 0) set_status(a.status, RSWA_DEVICE_BAD_PREFIX_LEN);
    len = 0;
  }
  if (len <= 0) n = 0;
  const int nt = (n + kSharedRows - 1) / kSharedRows;
  const int keys = n > 0 ? (len + kRows - 1) / kRows : 0;
  const Counts mine{n, nt, nt * keys * a.H};
  const Counts inc = warp_scan(mine, lane);
  if (lane == 31) sums[warp] = inc;
  __syncthreads();
  Counts at{inc.seqs - mine.seqs, inc.tiles - mine.tiles, inc.units - mine.units}, total{0, 0, 0};
  for (int w = 0; w < kSmallGroup / 32; ++w) {
    if (w < warp) at = plus(at, sums[w]);
    total = plus(total, sums[w]);
  }
  first[tid] = at.seqs;
  tile0[tid] = nt > 0 ? at.tiles : -1;
  unit0[tid] = at.units;
  keys_of[tid] = keys;
  for (int i = 0; i < nt; ++i) {
    SharedTile t = {};
    t.first_unit = at.units + i * keys * a.H;
    t.first_seq = at.seqs + i * kSharedRows;
    t.rows = min(kSharedRows, n - i * kSharedRows);
    t.prefix = tid;
    t.len = len;
    t.key_tiles = keys;
    a.t.tiles[at.tiles + i] = t;
  }
  if (tid == 0) {
    a.t.head->units = total.units;
    a.t.head->per = max(1, (total.units + a.ctas - 1) / a.ctas);
    a.t.head->tiles = total.tiles;
  }
  __syncthreads();
  if (tid < a.B) {
    SharedSeq q = {};
    q.row = -1;
    if (p >= 0 && tile0[p] >= 0) {
      const int i = rank / kSharedRows;
      a.t.order[first[p] + rank] = tid;
      q.row = rank % kSharedRows;
      q.first_seq = first[p] + i * kSharedRows;
      q.key_tiles = keys_of[p];
      q.first_unit = unit0[p] + i * keys_of[p] * a.H;
      q.rows = a.t.tiles[tile0[p] + i].rows;  // written by this CTA, before the barrier
    }
    a.t.seqs[tid] = q;
  }
  fence_async_smem();  // the scratch is a TMA destination next
  __syncthreads();
}

__device__ __forceinline__ bool wait_or_abort(SharedSmem& sm, uint64_t* bar, uint32_t parity, int32_t* status) {
  if (mbar_try_wait(bar, parity)) return true;
  const uint64_t t0 = global_timer_ns();
  while (true) {
#pragma unroll 1
    for (int i = 0; i < 32; ++i)
      if (mbar_try_wait(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sm.abort_flag)) return false;
    if (global_timer_ns() - t0 > *reinterpret_cast<volatile uint64_t*>(&sm.wait_limit_ns)) break;
  }
  sm.abort_flag = 1;
  set_status(status, RSWA_DEVICE_WAIT_TIMEOUT);
  return false;
}

// A CTA's run of units as segments: key tiles [k0, k1) of head h of one tile of sequences.
struct Walk {
  int u, end;
  int ti, h, k0, k1;
  SharedTile t;

  __device__ __forceinline__ bool begin(const SharedTables& tab) {
    const SharedHead head = *tab.head;
    if ((int64_t)blockIdx.x * head.per >= head.units) return false;
    u = (int)blockIdx.x * head.per;
    end = head.units - u > head.per ? u + head.per : head.units;
    int lo = 0, hi = head.tiles - 1;  // the last tile whose first unit is at or before u
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (tab.tiles[mid].first_unit <= u)
        lo = mid;
      else
        hi = mid - 1;
    }
    ti = lo;
    t = tab.tiles[ti];
    h = (u - t.first_unit) / t.key_tiles;
    k0 = (u - t.first_unit) % t.key_tiles;
    k1 = min(t.key_tiles, k0 + (end - u));
    return true;
  }
  __device__ __forceinline__ bool next(const SharedTables& tab, int H) {
    u += k1 - k0;
    if (u >= end) return false;
    if (++h == H) {
      h = 0;
      t = tab.tiles[++ti];
    }
    k0 = 0;
    k1 = min(t.key_tiles, end - u);
    return true;
  }
  __device__ __forceinline__ bool two() const { return t.rows > kRows; }  // a group takes its own rows
  __device__ __forceinline__ int events() const { return two() ? 2 * (k1 - k0) : k1 - k0; }
};

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

// Both softmax groups meet; true for all of them if any thread gives up, so that they leave together.
__device__ __forceinline__ bool softmax_barrier_or(bool stop) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, 1, 256, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(stop ? 1u : 0u)
      : "memory");
  return any != 0;
}

__global__ void __launch_bounds__(kThreads, 1)
    shared_kernel(const __grid_constant__ AttnArgs a, const __grid_constant__ CUtensorMap tm_k,
                  const __grid_constant__ CUtensorMap tm_v) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  SharedSmem& sm = *reinterpret_cast<SharedSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if ((smem_addr(smem_raw) & 1023u) != 0) {  // it is, with no other shared memory in the kernel
    if (tid == 0) set_status(a.status, RSWA_DEVICE_PIPELINE);
    return;
  }
  if (tid == 0) {
    sm.abort_flag = 0;
    sm.wait_limit_ns = a.wait_limit_ns;
    mbar_init(&sm.q_full, 256);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_ready[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int x = 0; x < 2; ++x) {
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 4);  // one arrival a warp
      mbar_init(&sm.o_done[x], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = sm.tmem_base;
  griddep_wait();  // the tables come from the grouping launch, or are laid out here
  if (a.group) group_small(a.g, reinterpret_cast<int*>(sm.k[0]));
  griddep_launch_dependents();

  Walk w;
  bool more = w.begin(a.t);
  int issued = 0;  // by a producer: key tiles up to here
  if (warp == 0 || warp == 2) {
    // ---------------- producers: K tiles (warp 0), V tiles (warp 2) ----------------
    if (lane == 0) {
      const bool is_k = warp == 0;
      const int stages = is_k ? kKStages : kVStages;
      uint64_t* full = is_k ? sm.k_full : sm.v_full;
      uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
      const CUtensorMap* map = is_k ? &tm_k : &tm_v;
      bool ok = true;
      for (; ok && more; more = w.next(a.t, a.H)) {
        const int row0 = (int)(((int64_t)w.t.prefix * a.H + w.h) * a.cap);
        for (int k = w.k0; k < w.k1; ++k, ++issued) {
          const int n = issued, s = n % stages;
          if (n >= stages && !wait_or_abort(sm, &empty[s], ((n / stages) - 1) & 1, a.status)) {
            ok = false;
            break;
          }
          if (is_k && n == a.drop_tile && blockIdx.x == 0) continue;  // a wait-timeout test
          uint8_t* dst = is_k ? sm.k[s] : sm.v[s];
          mbar_arrive_expect_tx(&full[s], kTileBytes);
          tma_load_2d(dst, map, 0, row0 + k * kRows, &full[s]);
          tma_load_2d(dst + kRegionBytes, map, 64, row0 + k * kRows, &full[s]);
        }
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer: one thread ----------------
    if (elect_one()) {
      constexpr uint32_t kIdescQK = idesc_bf16_m128_n128(0);
      constexpr uint32_t kIdescPV = idesc_bf16_m128_n128(1);
      const uint64_t q_desc = smem_desc_sw128(smem_addr(sm.q[0]), 16, 1024);
      const uint64_t k_desc = smem_desc_sw128(smem_addr(sm.k[0]), 16, 1024);
      const uint64_t v_desc = smem_desc_sw128(smem_addr(sm.v[0]), kRegionBytes, 1024);
      int ks = 0, vs = 0;
      uint32_t k_phase = 0, v_phase = 0, q_phase = 0, p_phase[2] = {0, 0};
      auto issue_s = [&](int x, int q) {  // S_x = Q K^T, key tile in stage ks
        const uint64_t qd = q_desc + (uint64_t)(q * (kTileBytes >> 4)), kd = k_desc + (uint64_t)(ks * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint64_t off = (uint64_t)(((kk >> 2) * kRegionBytes + (kk & 3) * 32) >> 4);
          tc_mma_ss(tmem + (uint32_t)x * 128u, qd + off, kd + off, kIdescQK, kk > 0);
        }
        tc_commit(&sm.s_full[x]);
      };
      auto issue_pv = [&](int x, bool more_v) {  // O_x += P_x V, value tile in stage vs
        const uint64_t vd = v_desc + (uint64_t)(vs * (kTileBytes >> 4));
#pragma unroll
        for (int kk = 0; kk < 8; ++kk)
          tc_mma_ts(tmem + kColO + (uint32_t)x * 128u, tmem + (uint32_t)x * 128u + (uint32_t)kk * 8u,
                    vd + (uint64_t)(kk * (2048 >> 4)), kIdescPV, (more_v || kk > 0) ? 1u : 0u);
        tc_commit(&sm.o_done[x]);
      };
      auto take_k = [&]() {
        if (!wait_or_abort(sm, &sm.k_full[ks], k_phase, a.status)) return false;
        tc_fence_after();
        return true;
      };
      auto free_k = [&]() {
        tc_commit(&sm.k_empty[ks]);
        if (++ks == kKStages) {
          ks = 0;
          k_phase ^= 1;
        }
      };
      auto take_p = [&](int x) {
        if (!wait_or_abort(sm, &sm.p_full[x], p_phase[x], a.status)) return false;
        p_phase[x] ^= 1;
        tc_fence_after();
        return true;
      };
      bool ok = true;
      for (; ok && more; more = w.next(a.t, a.H)) {
        const int n = w.k1 - w.k0;
        if (!(ok = wait_or_abort(sm, &sm.q_full, q_phase, a.status))) break;
        q_phase ^= 1;
        tc_fence_after();
        if (w.two()) {
          if ((ok = take_k())) {
            issue_s(0, 0);
            issue_s(1, 1);
            free_k();
          }
        } else {
          for (int t = 0; ok && t < min(2, n); ++t)
            if ((ok = take_k())) {
              issue_s(t, 0);
              free_k();
            }
        }
        for (int t = 0; ok && t < n; ++t) {
          if (!(ok = wait_or_abort(sm, &sm.v_ready[vs], v_phase, a.status))) break;
          if (w.two()) {
            const bool next = t + 1 < n;
            if (!(ok = take_p(0))) break;
            issue_pv(0, t > 0);
            if (next) {
              if (!(ok = take_k())) break;
              issue_s(0, 0);
            }
            if (!(ok = take_p(1))) break;
            issue_pv(1, t > 0);
            tc_commit(&sm.v_empty[vs]);
            if (next) {
              issue_s(1, 1);
              free_k();
            }
          } else {
            const int x = t & 1;
            if (!(ok = take_p(x))) break;
            issue_pv(x, t > 1);
            tc_commit(&sm.v_empty[vs]);
            if (t + 2 < n) {
              if (!(ok = take_k())) break;
              issue_s(x, 0);
              free_k();
            }
          }
          if (++vs == kVStages) {
            vs = 0;
            v_phase ^= 1;
          }
        }
      }
      tc_commit(&sm.drain);  // fires once every issued MMA is done
    }
    __syncwarp();
  } else if (warp == 3) {
    // ---------------- V rows past the prefix's end: zeroed ----------------
    int n = 0;
    bool ok = true;
    for (; ok && more; more = w.next(a.t, a.H)) {
      for (int k = w.k0; ok && k < w.k1; ++k, ++n) {
        const int s = n % kVStages;
        ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.v_full[s], (n / kVStages) & 1, a.status));
        if (!ok) break;
        const int left = w.t.len - k * kRows;  // rows of the prefix in this tile
        if (left < kRows) {
          for (int r = left + lane; r < kRows; r += 32) {
            uint4* row0 = reinterpret_cast<uint4*>(sm.v[s] + r * 128);
            uint4* row1 = reinterpret_cast<uint4*>(sm.v[s] + kRegionBytes + r * 128);
#pragma unroll
            for (int i = 0; i < 8; ++i) {
              row0[i] = make_uint4(0, 0, 0, 0);
              row1[i] = make_uint4(0, 0, 0, 0);
            }
          }
          fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sm.v_ready[s]);
      }
    }
  } else if (warp >= kSoftmaxWarp0) {
    // ---------------- softmax groups ----------------
    const int x = (warp - kSoftmaxWarp0) / 4;
    const int r = tid - (kSoftmaxWarp0 + 4 * x) * 32;
    const uint32_t lane_base = (uint32_t)(((warp - kSoftmaxWarp0) & 3) * 32) << 16;
    const uint32_t s_cols = tmem + lane_base + (uint32_t)x * 128u;
    const uint32_t o_cols = tmem + lane_base + kColO;  // O of group A; B's is 128 columns on
    uint32_t seen = 0;  // scores of this group so far, over all segments
    bool ok = true;
    for (; ok && more; more = w.next(a.t, a.H)) {
      const bool two = w.two();
      const int row = two ? x * kRows + r : r;
      const bool live = row < w.t.rows;
      const bool warp_live = (two ? x * kRows : 0) + (r & ~31) < w.t.rows;
      {  // this segment's queries into shared memory, 128-byte swizzled
        uint4 z = make_uint4(0, 0, 0, 0);
        const uint4* src = nullptr;
        if (live)
          src = reinterpret_cast<const uint4*>(a.q + ((int64_t)a.t.order[w.t.first_seq + row] * a.H + w.h) * kHeadDim);
        // two tiles: a thread copies its row; one tile: groups A and B copy a row's halves
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          if (!two && half != x) continue;
          uint8_t* dst = sm.q[two ? x : 0] + half * kRegionBytes + r * 128;
          uint4 buf[8];
#pragma unroll
          for (int i = 0; i < 8; ++i) buf[i] = src != nullptr ? src[half * 8 + i] : z;
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(dst + ((i ^ (r & 7)) << 4)) = buf[i];
        }
        fence_async_smem();
        tc_fence_before();
        mbar_arrive(&sm.q_full);
      }
      float m_used = -INFINITY, l = 0.f, lu = 0.f;
      const int events = w.events();
      for (int e = x; e < events; e += 2) {
        const int t = two ? e >> 1 : e;
        ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.s_full[x], seen & 1, a.status));
        if (!ok) break;
        tc_fence_after();
        ++seen;
        if (warp_live) {
          const int left = w.t.len - (w.k0 + t) * kRows;
          const bool full = left >= kRows;
          float m0 = -INFINITY, m1 = -INFINITY;
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t rr[32];
            tmem_ld32(s_cols + (uint32_t)ch * 32u, rr);
            tmem_wait_ld();
            if (full) {
#pragma unroll
              for (int i = 0; i < 32; i += 4) {
                m0 = max3(m0, __uint_as_float(rr[i]), __uint_as_float(rr[i + 1]));
                m1 = max3(m1, __uint_as_float(rr[i + 2]), __uint_as_float(rr[i + 3]));
              }
            } else {
#pragma unroll
              for (int i = 0; i < 32; ++i)
                if (ch * 32 + i < left) m0 = fmaxf(m0, __uint_as_float(rr[i]));
            }
          }
          const float tmax = fmaxf(m0, m1) * a.scale_log2;
          const bool rescale = tmax > m_used + kLazyRescaleLog2;
          float alpha = 1.f;
          if (rescale) {
            alpha = ex2(m_used - tmax);
            l *= alpha;
            lu *= alpha;
            m_used = tmax;
          }
          // the previous P V of this group is done (the commit that completed S covers it)
          if (e >= 2 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
            for (int ch = 0; ch < 4; ++ch) {
              uint32_t rr[32];
              tmem_ld32(o_cols + (uint32_t)(x * 128 + ch * 32), rr);
              tmem_wait_ld();
#pragma unroll
              for (int i = 0; i < 32; ++i) rr[i] = __float_as_uint(__uint_as_float(rr[i]) * alpha);
              tmem_st32(o_cols + (uint32_t)(x * 128 + ch * 32), rr);
            }
          }
          const float m_sub = m_used == -INFINITY ? 0.f : m_used;
          float2 ls = make_float2(0.f, 0.f), lus = make_float2(0.f, 0.f);
          const float2 neg_m = make_float2(-m_sub, -m_sub);
          const float2 scale2 = make_float2(a.scale_log2, a.scale_log2);
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t rr[32];
            tmem_ld32(s_cols + (uint32_t)ch * 32u, rr);
            tmem_wait_ld();
            uint32_t pk[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) {
              const float2 z2 = __ffma2_rn(make_float2(__uint_as_float(rr[2 * i]), __uint_as_float(rr[2 * i + 1])), scale2,
                                           neg_m);
              float2 p2 = make_float2(ex2(z2.x), ex2(z2.y));
              if (!full) {
                if (ch * 32 + 2 * i >= left) p2.x = 0.f;
                if (ch * 32 + 2 * i + 1 >= left) p2.y = 0.f;
              }
              const __nv_bfloat162 pb = __floats2bfloat162_rn(p2.x, p2.y);
              pk[i] = *reinterpret_cast<const uint32_t*>(&pb);
              ls = __fadd2_rn(ls, make_float2(__uint_as_float(pk[i] << 16), __uint_as_float(pk[i] & 0xffff0000u)));
              lus = __fadd2_rn(lus, p2);
            }
            tmem_st16(s_cols + (uint32_t)ch * 16u, pk);
          }
          l += ls.x + ls.y;
          lu += lus.x + lus.y;
          tmem_wait_st();
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[x]);
      }
      // ---- the segment's records ----
      const bool any = x < events;
      if (ok && any) ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.o_done[x], (seen - 1) & 1, a.status));
      // Group B without a score of its own writes nothing: it has waited for nothing in this segment, and group A
      // may still be reading the statistics of the segment before. (A group with a score has waited for scores,
      // which were issued when all threads of both groups had brought this segment's queries, past their reads.)
      if (!two && any) {
        sm.stat_m[x][r] = m_used;
        if (x == 1) {
          sm.stat_l[r] = l;
          sm.stat_lu[r] = lu;
        }
      }
      tc_fence_before();
      if (softmax_barrier_or(!ok)) break;
      tc_fence_after();
      if (warp_live) {
        // the run that holds the tile's first keys, or this CTA's (it began inside)
        float* rec = a.t.records + (w.k0 == 0 ? (int64_t)w.t.first_seq * a.H + (int64_t)w.h * w.t.rows + row
                                              : (int64_t)a.B * a.H + (int64_t)blockIdx.x * kSharedRows + row) *
                                       kRecordFloats;
        if (two) {
          if (live) *reinterpret_cast<float4*>(rec) = make_float4(m_used, l, lu, 0.f);
#pragma unroll 1
          for (int ch = 0; ch < 4; ++ch) {
            uint32_t rr[32];
            tmem_ld32(o_cols + (uint32_t)(x * 128 + ch * 32), rr);
            tmem_wait_ld();
            if (live)
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(rec + 4 + ch * 32 + i) =
                    make_float4(__uint_as_float(rr[i]), __uint_as_float(rr[i + 1]), __uint_as_float(rr[i + 2]),
                                __uint_as_float(rr[i + 3]));
          }
        } else {
          // the two groups' halves of the keys meet; each writes half of the columns
          const bool both = events > 1;
          const float ma = sm.stat_m[0][r], mb = both ? sm.stat_m[1][r] : -INFINITY;
          const float M = fmaxf(ma, mb), m_sub = M == -INFINITY ? 0.f : M;
          const float fa = ex2(ma - m_sub), fb = both ? ex2(mb - m_sub) : 0.f;
          if (live && x == 0)
            *reinterpret_cast<float4*>(rec) = make_float4(M, both ? fmaf(sm.stat_l[r], fb, l * fa) : l * fa,
                                                          both ? fmaf(sm.stat_lu[r], fb, lu * fa) : lu * fa, 0.f);
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            const uint32_t col = (uint32_t)(x * 64 + ch * 32);
            uint32_t ra[32], rb[32];
            tmem_ld32(o_cols + col, ra);
            if (both) tmem_ld32(o_cols + 128u + col, rb);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) {
              float o = __uint_as_float(ra[i]) * fa;
              if (both) o = fmaf(__uint_as_float(rb[i]), fb, o);
              ra[i] = __float_as_uint(o);
            }
            if (live)
#pragma unroll
              for (int i = 0; i < 32; i += 4)
                *reinterpret_cast<float4*>(rec + 4 + col + i) =
                    make_float4(__uint_as_float(ra[i]), __uint_as_float(ra[i + 1]), __uint_as_float(ra[i + 2]),
                                __uint_as_float(ra[i + 3]));
          }
        }
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  // After a give-up, which may have come long after the last copy was issued: the copies in flight land
  // (bounded) before the CTA's shared memory goes away.
  if ((warp == 0 || warp == 2) && lane == 0 && sm.abort_flag)
    land_copies(warp == 0 ? sm.k_full : sm.v_full, warp == 0 ? kKStages : kVStages, issued,
                warp == 0 && blockIdx.x == 0 ? a.drop_tile : -1, a.wait_limit_ns);
  if (warp == 1) {
    if (lane == 0) mbar_wait(&sm.drain, 0);  // bounded; the MMAs drain before their TMEM is freed
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

size_t align256(size_t x) { return (x + 255) / 256 * 256; }

int64_t most_tiles(int B, int P) {
  // every prefix can leave one tile part full, and each tile has at least one sequence
  const int64_t t = (int64_t)P + B / kSharedRows;
  return t < B ? t : B;
}

}  // namespace

SharedPlan plan_shared(int B, int H, int P) {
  SharedPlan p;
  size_t off = 0;
  auto take = [&](size_t bytes) {
    const size_t at = off;
    off += align256(bytes);
    return at;
  };
  p.head = take(sizeof(SharedHead));
  p.tiles = take((size_t)most_tiles(B, P) * sizeof(SharedTile));
  p.order = take((size_t)B * 4);
  p.seqs = take((size_t)B * sizeof(SharedSeq));
  p.records = take(((size_t)B * H + (size_t)device_sm_count() * kSharedRows) * kRecordFloats * 4);
  p.bytes = off;
  return p;
}

cudaError_t launch_shared(const SharedLaunch& L, void* scratch, SharedTables* tables, cudaStream_t stream) {
  const SharedPlan p = plan_shared(L.B, L.H, L.P);
  uint8_t* base = static_cast<uint8_t*>(scratch);
  const int ctas = device_sm_count();
  GroupArgs g;
  g.B = L.B;
  g.H = L.H;
  g.P = L.P;
  g.cap = L.cap;
  g.ctas = ctas;
  g.shared_len = L.shared_len;
  g.share_of = L.share_of;
  g.t.head = reinterpret_cast<SharedHead*>(base + p.head);
  g.t.tiles = reinterpret_cast<SharedTile*>(base + p.tiles);
  g.t.order = reinterpret_cast<int32_t*>(base + p.order);
  g.t.seqs = reinterpret_cast<SharedSeq*>(base + p.seqs);
  g.t.records = reinterpret_cast<float*>(base + p.records);
  g.status = L.status;
  static unsigned long long done[2] = {};
  cudaError_t e;
  const bool small = L.B <= kSmallGroup && L.P <= kSmallGroup;
  if (!small) {
    const size_t tab = (size_t)L.P * 12;
    if ((e = ensure_smem_limit(group_kernel, (size_t)kMaxShared * 12, &done[0])) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    const int want = ((L.B > L.P ? L.B : L.P) + 31) / 32 * 32;
    fill_launch_config(cfg, attr, dim3(1), dim3(want < kGroupThreads ? want : kGroupThreads), tab, stream);
    if ((e = cudaLaunchKernelEx(&cfg, group_kernel, g)) != cudaSuccess) return e;
  }

  *tables = g.t;
  AttnArgs a;
  a.B = L.B;
  a.H = L.H;
  a.cap = L.cap;
  a.q = L.q;
  a.scale_log2 = L.scale * 1.4426950408889634f;
  a.t = *tables;
  a.status = L.status;
  a.wait_limit_ns = L.wait_limit_ns;
  a.drop_tile = L.drop_tile;
  a.group = small;
  a.g = g;
  CUtensorMap tk, tv;
  const int64_t rows = (int64_t)L.P * L.H * L.cap;
  if ((e = make_rows_map(&tk, L.sk, rows)) != cudaSuccess) return e;
  if ((e = make_rows_map(&tv, L.sv, rows)) != cudaSuccess) return e;
  const size_t smem = sizeof(SharedSmem);
  if ((e = ensure_smem_limit(shared_kernel, smem, &done[1])) != cudaSuccess) return e;
  cudaLaunchConfig_t cfg2 = {};
  cudaLaunchAttribute attr2[1];
  fill_launch_config(cfg2, attr2, dim3(ctas), dim3(kThreads), smem, stream);
  return cudaLaunchKernelEx(&cfg2, shared_kernel, a, tk, tv);
}

}  // namespace rswa

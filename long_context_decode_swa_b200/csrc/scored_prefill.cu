// scored_prefill.cu -- chunked R-SWA prefill whose scores are capped, biased by distance and
// limited to each query's own document, on the sm_100a tensor cores (tcgen05 + TMEM).
//
// Query i of a chunk attends to the prefix rows [lo_i, hi_i) of its document, to the outputs j with
// i - n < j <= i and, for j < 0, to the previous chunk's last outputs in the ring, with
//   s = cap tanh(scale q.k / cap) - slope_h (pos_q - pos_k).
//
// A CTA owns two 128-row query tiles (A and B) of one (sequence, head) and walks the key tiles (128
// keys) that any of its rows sees; the roles are those of the plain prefill (prefill.cu): TMA
// producers in warps 0 (Q, K) and 2 (V), the MMA issuer in warp 1, softmax of tile A in warps 4-7
// and of tile B in warps 8-11, thread r owning row r; P (bf16) replaces S in TMEM and is the A
// operand of P V.
//
// Documents: the union of the 256 rows' ranges, as up to four runs of rows, gives the prefix tiles;
// rows of a tile that none of them sees are zeroed in V (0 * NaN would reach O). A chunk over packed
// documents so costs what its documents cost, not what the prefix does.
//
// Scores: tanh(u) = 1 - 2 / (e^2u + 1), by one ex2 and one rcp of the special-function unit (16 a
// cycle and SM); with the softmax's own ex2 that is three a score, 3,072 cycles a tile against 512
// of MMA. The cancellation at small u costs 2^-23 of the cap, not of the score: 1e-5 at cap 50.
#include <cuda.h>
#include <cuda_bf16.h>

#include <cmath>

#include "balanced.h"
#include "common.cuh"
#include "internal.h"
#include "scored_prefill.h"
#include "tcgen05.cuh"

namespace rswa {

namespace {

constexpr int kRows = 128;                 // query rows per tile, keys per key tile
constexpr int kQTiles = 2;                 // query tiles per CTA
constexpr int kCtaRows = kQTiles * kRows;
constexpr int kRegionBytes = kRows * 128;  // one 64-column SW128 region of a 128-row tile
constexpr int kTileBytes = 2 * kRegionBytes;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kThreads = 384;
constexpr int kSoftmaxWarp0 = 4;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kColO = 256;
constexpr float kLazyRescaleLog2 = 8.f;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kRuns = 4;  // disjoint runs of prefix rows that a CTA tells apart

struct Ctx {
  int m, n, fill, wp, T, i0;
  int lo[kRuns], hi[kRuns];        // runs of prefix rows some query sees, ascending
  int tile0[kRuns], first[kRuns];  // first key tile of run r, and its number among the CTA's tiles
  int runs;
  int exact;                       // every row of the runs is seen (else the last run has gaps)
  int row_lo[kQTiles], row_hi[kQTiles];  // hull of each query tile's ranges
  int np, nr, jt0, total;
};

struct __align__(1024) Smem {
  uint8_t q[kQTiles][kTileBytes];
  uint8_t k[kKStages][kTileBytes];
  uint8_t v[kVStages][kTileBytes];
  uint64_t q_full;
  uint64_t k_full[kKStages], k_empty[kKStages];
  uint64_t v_full[kVStages], v_empty[kVStages];
  uint64_t s_full[kQTiles], p_full[kQTiles], o_done[kQTiles];
  uint64_t drain;
  uint32_t tmem_base;
  int abort_flag;
  int skip;
  Ctx ctx;
};

struct Args {
  int B, H, n, T;
  int64_t cap;
  const int32_t* prefix_len;
  const int32_t* wp;
  const int32_t* fill;
  int has_ring;
  const int2* ranges;     // [B][T] or null
  const float* slopes;    // [H], with pos [B], or null
  const int32_t* pos;
  float softcap, scale;
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
};

enum Kind { kPrefix = 0, kRing = 1, kBand = 2 };

// Key tile t of the CTA: prefix rows, ring slots or the chunk's outputs [start, start + 128).
__device__ __forceinline__ void tile_kind(const Ctx& c, int t, int& kind, int& start) {
  if (t < c.np) {
    kind = kPrefix;
    int tile = c.tile0[0] + t;
#pragma unroll
    for (int r = 1; r < kRuns; ++r)
      if (r < c.runs && t >= c.first[r]) tile = c.tile0[r] + t - c.first[r];
    start = tile * kRows;
  } else if (t < c.np + c.nr) {
    kind = kRing;
    start = (t - c.np) * kRows;
  } else {
    kind = kBand;
    start = (c.jt0 + t - c.np - c.nr) * kRows;
  }
}

__device__ __forceinline__ int ring_age(const Ctx& c, int slot) {
  int a = c.wp - 1 - slot;
  if (a < 0) a += c.n;
  return a + 1;
}

// Does query tile X see anything of the tile?
__device__ __forceinline__ bool tile_visible(const Ctx& c, int X, int kind, int start) {
  const int ilo = c.i0 + X * kRows;
  if (ilo >= c.T) return false;
  const int ihi = min(ilo + kRows - 1, c.T - 1);
  if (kind == kPrefix) return start < c.row_hi[X] && start + kRows > c.row_lo[X];
  if (kind == kRing) return ilo <= c.n - 2;
  const int jhi = min(start + kRows - 1, c.T - 1);
  return start <= ihi && jhi >= ilo - c.n + 1;
}

__device__ __forceinline__ bool tile_visible(const Ctx& c, int X, int t) {
  int kind, start;
  tile_kind(c, t, kind, start);
  return tile_visible(c, X, kind, start);
}

// The prefix rows query i of sequence b sees (empty: 0, 0).
__device__ __forceinline__ int2 range_of(const Args& a, int m, int b, int i, bool report) {
  if (i >= a.T) return make_int2(0, 0);
  if (a.ranges == nullptr) return make_int2(0, m);
  const int2 r = a.ranges[(int64_t)b * a.T + i];
  if (r.x >= r.y) return make_int2(0, 0);
  if (r.x < 0 || r.y > m) {
    if (report) set_status(a.status, RSWA_DEVICE_BAD_RANGE);
    return make_int2(0, 0);
  }
  return r;
}

__device__ __forceinline__ bool wait_or_abort(Smem& sm, uint64_t* bar, uint32_t parity, int32_t* status) {
  if (*reinterpret_cast<volatile int*>(&sm.abort_flag)) return false;
  if (mbar_wait(bar, parity)) return true;
  sm.abort_flag = 1;
  set_status(status, RSWA_DEVICE_WAIT_TIMEOUT);
  return false;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// What a row does to its raw scores. In the log2 domain: s = mul raw (no cap), or
// cap2 - 2 cap2 / (2^(mul raw) + 1), plus slope2 (column - away0).
struct RowScore {
  float mul, cap2, slope2;
};

template <bool kCap>
__device__ __forceinline__ float scored(const RowScore& s, float raw) {
  if (!kCap) return raw * s.mul;
  return fmaf(-2.f * s.cap2, rcp(ex2(raw * s.mul) + 1.f), s.cap2);
}

// The scores of one 32-column chunk: masked columns -inf. fbase: the distance of the tile's column 0
// (less the row's reference distance).
template <bool kCap, bool kBias>
__device__ __forceinline__ void score_chunk(const Ctx& c, const RowScore& rs, int kind, int start, int col0, int lo, int hi,
                                            int i, int base, bool full, const uint32_t (&r)[32], float (&x)[32]) {
  if (kind == kRing) {
#pragma unroll
    for (int e = 0; e < 32; ++e) {
      const int slot = start + col0 + e, age = ring_age(c, slot);
      float s = scored<kCap>(rs, __uint_as_float(r[e]));
      if (kBias) s = fmaf(-rs.slope2, (float)(base + age), s);
      x[e] = (slot < c.n && age <= c.fill && age < c.n - i) ? s : -INFINITY;
    }
    return;
  }
  const float b0 = kBias ? rs.slope2 * (float)(col0 - base) : 0.f;
#pragma unroll
  for (int e = 0; e < 32; ++e) {
    float s = scored<kCap>(rs, __uint_as_float(r[e]));
    if (kBias) s += fmaf(rs.slope2, (float)e, b0);
    x[e] = (full || (col0 + e >= lo && col0 + e < hi)) ? s : -INFINITY;
  }
}

template <bool kCap, bool kBias>
__global__ void __launch_bounds__(kThreads, 1)
    scored_prefill_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_ko, const __grid_constant__ CUtensorMap tm_vo,
                          const __grid_constant__ CUtensorMap tm_pk, const __grid_constant__ CUtensorMap tm_pv,
                          const __grid_constant__ CUtensorMap tm_rk, const __grid_constant__ CUtensorMap tm_rv) {
  extern __shared__ uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  const int qt = blockIdx.x, h = blockIdx.y, b = blockIdx.z;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int64_t bh = (int64_t)b * a.H + h;
  griddep_wait();
  griddep_launch_dependents();
  if (tid == 0) {
    // a CTA of this launch already gave up on a wait: skip the work (the output is flagged invalid)
    sm.skip = (*reinterpret_cast<volatile int32_t*>(a.status) & RSWA_DEVICE_WAIT_TIMEOUT) != 0;
    sm.abort_flag = 0;
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int x = 0; x < kQTiles; ++x) {
      mbar_init(&sm.s_full[x], 1);
      mbar_init(&sm.p_full[x], 128);
      mbar_init(&sm.o_done[x], 1);
    }
    mbar_init(&sm.drain, 1);
    fence_mbar_init();
  }
  __syncthreads();
  if (sm.skip) return;
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_addr(&sm.tmem_base)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  } else if (warp == 0) {
    // ---- the CTA's key tiles ----
    const bool first = qt == 0 && h == 0 && lane == 0;
    int m = a.cap > 0 ? a.prefix_len[b] : 0;
    if (m < 0 || m > a.cap) {
      if (first) set_status(a.status, RSWA_DEVICE_BAD_PREFIX_LEN);
      m = 0;
    }
    if (kBias) {
      const int p = a.pos[b];
      if (p < 0 || p > kMaxPos) {
        if (first) set_status(a.status, RSWA_DEVICE_BAD_POS);
        m = 0;
      }
    }
    const int i0 = qt * kCtaRows;
    int2 rg[kCtaRows / 32];  // lane's rows: 32 u + lane
#pragma unroll
    for (int u = 0; u < kCtaRows / 32; ++u) rg[u] = range_of(a, m, b, i0 + 32 * u + lane, h == 0);
    Ctx& c = sm.ctx;
    for (int x = 0; x < kQTiles; ++x) {
      int lo = INT32_MAX, hi = 0;
#pragma unroll
      for (int u = 0; u < kCtaRows / 32; ++u)
        if (u / (kRows / 32) == x && rg[u].y > rg[u].x) {
          lo = min(lo, rg[u].x);
          hi = max(hi, rg[u].y);
        }
      lo = __reduce_min_sync(0xffffffffu, lo);
      hi = __reduce_max_sync(0xffffffffu, hi);
      if (lane == 0) {
        c.row_lo[x] = lo;
        c.row_hi[x] = hi;
      }
    }
    int runs = 0, np = 0, cur = 0, next_tile = 0;
    bool exact = true;
    while (runs < kRuns) {
      int s = INT32_MAX, top = 0;
#pragma unroll
      for (int u = 0; u < kCtaRows / 32; ++u)
        if (rg[u].y > rg[u].x && rg[u].y > cur) {
          s = min(s, max(rg[u].x, cur));
          top = max(top, rg[u].y);
        }
      s = __reduce_min_sync(0xffffffffu, s);
      top = __reduce_max_sync(0xffffffffu, top);
      if (s == INT32_MAX) break;
      int e = s;
      while (true) {  // ranges that overlap or touch join the run
        int e2 = e;
#pragma unroll
        for (int u = 0; u < kCtaRows / 32; ++u)
          if (rg[u].y > rg[u].x && rg[u].x <= e) e2 = max(e2, rg[u].y);
        e2 = __reduce_max_sync(0xffffffffu, e2);
        if (e2 == e) break;
        e = e2;
      }
      if (runs == kRuns - 1 && e < top) {  // the rest in one run, gaps and all
        e = top;
        exact = false;
      }
      const int t0 = max(next_tile, s / kRows), t1 = (e + kRows - 1) / kRows;
      if (lane == 0) {
        c.lo[runs] = s;
        c.hi[runs] = e;
        c.tile0[runs] = t0;
        c.first[runs] = np;
      }
      np += max(0, t1 - t0);
      next_tile = max(next_tile, t1);
      cur = e;
      ++runs;
    }
    if (lane == 0) {
      c.m = m;
      c.n = a.n;
      c.T = a.T;
      c.i0 = i0;
      c.runs = runs;
      c.exact = exact;
      c.wp = c.fill = 0;
      if (runs == 0) c.tile0[0] = 0;
      if (a.has_ring) {
        const int w = a.wp[b], f = a.fill[b];
        if (w < 0 || w >= a.n || f < 0 || f > a.n) {
          if (first) set_status(a.status, RSWA_DEVICE_BAD_RING_STATE);
        } else {
          c.wp = w;
          c.fill = f;
        }
      }
      c.np = np;
      c.nr = c.fill > 0 && i0 <= a.n - 2 ? (a.n + kRows - 1) / kRows : 0;
      const int jlo = i0 - a.n + 1;
      c.jt0 = jlo > 0 ? jlo / kRows : 0;
      c.total = np + c.nr + min(i0 + kCtaRows - 1, a.T - 1) / kRows - c.jt0 + 1;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Ctx& c = sm.ctx;
  const uint32_t tmem = sm.tmem_base;
  const int total = c.total;

  if (warp == 0 || warp == 2) {
    // ---------------- producers: Q and K tiles (warp 0), V tiles (warp 2) ----------------
    if (lane == 0) {
      const bool is_k = warp == 0;
      if (is_k) {
        const int qrow = (int)(bh * a.T) + c.i0;
        mbar_arrive_expect_tx(&sm.q_full, kQTiles * kTileBytes);
        for (int x = 0; x < kQTiles; ++x) {
          tma_load_2d(sm.q[x], &tm_q, 0, qrow + x * kRows, &sm.q_full);
          tma_load_2d(sm.q[x] + kRegionBytes, &tm_q, 64, qrow + x * kRows, &sm.q_full);
        }
      }
      const int stages = is_k ? kKStages : kVStages;
      uint64_t* full = is_k ? sm.k_full : sm.v_full;
      uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
      int t = 0;
      for (; t < total; ++t) {
        const int s = t % stages;
        if (t >= stages && !wait_or_abort(sm, &empty[s], ((t / stages) - 1) & 1, a.status)) break;
        int kind, start;
        tile_kind(c, t, kind, start);
        const CUtensorMap* map = is_k ? (kind == kPrefix ? &tm_pk : (kind == kRing ? &tm_rk : &tm_ko))
                                      : (kind == kPrefix ? &tm_pv : (kind == kRing ? &tm_rv : &tm_vo));
        const int64_t rows = kind == kPrefix ? a.cap : (kind == kRing ? a.n : a.T);
        const int row = (int)(bh * rows) + start;
        uint8_t* dst = is_k ? sm.k[s] : sm.v[s];
        mbar_arrive_expect_tx(&full[s], kTileBytes);
        tma_load_2d(dst, map, 0, row, &full[s]);
        tma_load_2d(dst + kRegionBytes, map, 64, row, &full[s]);
      }
      if (sm.abort_flag) {  // let the copies in flight land before shared memory is released
        if (is_k) mbar_wait(&sm.q_full, 0);
        for (int i = max(0, t - stages); i < t; ++i) mbar_wait(&full[i % stages], (i / stages) & 1);
      }
    }
  } else if (warp == 1) {
    // ---------------- MMA issuer (lane 0) + V-row zeroing (whole warp) ----------------
    constexpr uint32_t kIdescQK = idesc_bf16_m128_n128(0);
    constexpr uint32_t kIdescPV = idesc_bf16_m128_n128(1);
    int n_pv[kQTiles] = {0, 0};
    bool ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.q_full, 0, a.status));
    auto issue_s = [&](int x, int t) {  // S_x = Q_x K_t^T
      if (lane == 0) {
        const uint32_t q_addr = smem_addr(sm.q[x]);
        const uint32_t k_addr = smem_addr(sm.k[t % kKStages]);
#pragma unroll
        for (int kk = 0; kk < 8; ++kk) {
          const uint32_t off = (uint32_t)(kk >> 2) * kRegionBytes + (uint32_t)(kk & 3) * 32u;
          tc_mma_ss(tmem + (uint32_t)x * 128u, smem_desc_sw128(q_addr + off, 16, 1024),
                    smem_desc_sw128(k_addr + off, 16, 1024), kIdescQK, kk > 0);
        }
        tc_commit(&sm.s_full[x]);
      }
      __syncwarp();
    };
    auto wait_k = [&](int t) {
      const bool w = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.k_full[t % kKStages], (t / kKStages) & 1, a.status));
      tc_fence_after();
      return w;
    };
    if (ok) {
      ok = wait_k(0);
      if (ok) {
        for (int x = 0; x < kQTiles; ++x)
          if (tile_visible(c, x, 0)) issue_s(x, 0);
        if (lane == 0) tc_commit(&sm.k_empty[0]);
        __syncwarp();
      }
    }
    for (int t = 0; ok && t < total; ++t) {
      const int vs = t % kVStages;
      ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.v_full[vs], (t / kVStages) & 1, a.status));
      if (!ok) break;
      int kind, start;
      tile_kind(c, t, kind, start);
      bool zeroed = false;
      // a prefix tile inside one run is seen whole
      bool whole = kind == kBand && start + kRows <= c.T;
      if (kind == kPrefix)
        for (int r = 0; r < c.runs; ++r)
          whole |= start >= c.lo[r] && start + kRows <= c.hi[r] && (c.exact || r < kRuns - 1);
      if (!whole) {
        for (int r = lane; r < kRows; r += 32) {
          const int x = start + r;
          bool some = false;
          if (kind == kBand) {
            some = x < c.T;
          } else if (kind == kRing) {
            some = x < c.n && ring_age(c, x) <= c.fill;
          } else if (c.exact) {
            for (int u = 0; u < c.runs; ++u) some |= x >= c.lo[u] && x < c.hi[u];
          } else {
            for (int i = c.i0; !some && i < min(c.i0 + kCtaRows, c.T); ++i) {
              const int2 g = range_of(a, c.m, b, i, false);
              some = x >= g.x && x < g.y;
            }
          }
          if (!some) {
            uint4* row0 = reinterpret_cast<uint4*>(sm.v[vs] + r * 128);
            uint4* row1 = reinterpret_cast<uint4*>(sm.v[vs] + kRegionBytes + r * 128);
#pragma unroll
            for (int e = 0; e < 8; ++e) {
              row0[e] = make_uint4(0, 0, 0, 0);
              row1[e] = make_uint4(0, 0, 0, 0);
            }
            zeroed = true;
          }
        }
        if (__any_sync(0xffffffffu, zeroed)) fence_async_smem();
        __syncwarp();
      }
      const bool next = t + 1 < total;
      bool k_next = false;
      for (int x = 0; ok && x < kQTiles; ++x) {
        if (tile_visible(c, x, kind, start)) {
          ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.p_full[x], n_pv[x] & 1, a.status));
          if (!ok) break;
          tc_fence_after();
          if (lane == 0) {
            const uint32_t v_addr = smem_addr(sm.v[vs]);
            const uint32_t p_tmem = tmem + (uint32_t)x * 128u;
            const uint32_t o_tmem = tmem + kColO + (uint32_t)x * 128u;
#pragma unroll
            for (int kk = 0; kk < 8; ++kk)
              tc_mma_ts(o_tmem, p_tmem + (uint32_t)kk * 8u, smem_desc_sw128(v_addr + (uint32_t)kk * 2048u, kRegionBytes, 1024),
                        kIdescPV, (n_pv[x] > 0 || kk > 0) ? 1u : 0u);
            tc_commit(&sm.o_done[x]);
          }
          __syncwarp();
          ++n_pv[x];
        }
        if (next && tile_visible(c, x, t + 1)) {
          if (!k_next) {
            ok = wait_k(t + 1);
            if (!ok) break;
            k_next = true;
          }
          issue_s(x, t + 1);
        }
      }
      if (!ok) break;
      if (lane == 0) tc_commit(&sm.v_empty[vs]);
      if (next) {
        if (!k_next) {  // no query tile needed it: still let the copy land before freeing the stage
          ok = wait_k(t + 1);
          if (!ok) break;
        }
        if (lane == 0) tc_commit(&sm.k_empty[(t + 1) % kKStages]);
      }
      __syncwarp();
    }
    if (lane == 0) tc_commit(&sm.drain);  // fires once every issued MMA is done
  } else if (warp >= kSoftmaxWarp0) {
    // ---------------- softmax: thread r owns row r of its tile ----------------
    const int x = (warp - kSoftmaxWarp0) / 4;
    const int r = tid - (kSoftmaxWarp0 + 4 * x) * 32;
    const int i = c.i0 + x * kRows + r;
    const uint32_t lane_base = (uint32_t)(((warp - kSoftmaxWarp0) & 3) * 32) << 16;
    const uint32_t s_cols = tmem + lane_base + (uint32_t)x * 128u;
    const uint32_t o_cols = tmem + lane_base + kColO + (uint32_t)x * 128u;
    const int2 range = range_of(a, c.m, b, i, false);
    RowScore rs;
    rs.mul = kCap ? a.scale / a.softcap * 2.f * kLog2e : a.scale * kLog2e;
    rs.cap2 = a.softcap * kLog2e;
    rs.slope2 = 0.f;
    int pos = 0, ref = 0;  // ref: the distance of the row's most favoured key, taken off all of them
    if (kBias) {
      const float slope = a.slopes[h];
      rs.slope2 = slope * kLog2e;
      pos = a.pos[b] + i;
      const bool pre = range.y > range.x;
      if (slope >= 0.f)
        ref = pre ? min(0, pos - (range.y - 1)) : 0;
      else
        ref = max(min(i + c.fill, c.n - 1), pre ? pos - range.x : 0);
    }
    // l normalises O with the same bf16-rounded weights the MMA used; lu gives lse
    float m_used = -INFINITY, l = 0.f, lu = 0.f;
    int j = 0;  // key tiles this query tile has seen
    bool ok = true;
    for (int t = 0; t < total; ++t) {
      int kind, start;
      tile_kind(c, t, kind, start);
      if (!tile_visible(c, x, kind, start)) continue;
      ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.s_full[x], j & 1, a.status));
      if (!ok) break;
      tc_fence_after();
      // this row's visible columns of the tile
      int lo = 0, hi = 0, base = 0;
      if (kind == kPrefix) {
        lo = range.x - start;
        hi = range.y - start;
        base = pos - start - ref;
      } else if (kind == kBand) {
        lo = i - c.n + 1 - start;
        hi = min(i, c.T - 1) + 1 - start;
        base = i - start - ref;
      } else {
        base = i - ref;
      }
      const bool full = kind != kRing && __all_sync(0xffffffffu, lo <= 0 && hi >= kRows);
      // pass 1: the row's maximum
      float m0 = -INFINITY, m1 = -INFINITY;
      const bool raw_max = full && !kBias;  // the scale and the cap keep the order
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t rr[32];
        tmem_ld32(s_cols + (uint32_t)ch * 32u, rr);
        tmem_wait_ld();
        if (raw_max) {
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = max3(m0, __uint_as_float(rr[e]), __uint_as_float(rr[e + 1]));
            m1 = max3(m1, __uint_as_float(rr[e + 2]), __uint_as_float(rr[e + 3]));
          }
        } else {
          float xv[32];
          score_chunk<kCap, kBias>(c, rs, kind, start, ch * 32, lo, hi, i, base, full, rr, xv);
#pragma unroll
          for (int e = 0; e < 32; e += 4) {
            m0 = max3(m0, xv[e], xv[e + 1]);
            m1 = max3(m1, xv[e + 2], xv[e + 3]);
          }
          // pass 2 finds them scored
#pragma unroll
          for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(xv[e]);
          tmem_st32(s_cols + (uint32_t)ch * 32u, rr);
        }
      }
      float tmax = fmaxf(m0, m1);
      if (raw_max) tmax = scored<kCap>(rs, tmax);
      else tmem_wait_st();
      const bool rescale = tmax > m_used + kLazyRescaleLog2;
      float alpha = 1.f;
      if (rescale) {
        alpha = ex2(m_used - tmax);
        l *= alpha;
        lu *= alpha;
        m_used = tmax;
      }
      if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
        for (int ch = 0; ch < 4; ++ch) {
          uint32_t rr[32];
          tmem_ld32(o_cols + (uint32_t)ch * 32u, rr);
          tmem_wait_ld();
#pragma unroll
          for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
          tmem_st32(o_cols + (uint32_t)ch * 32u, rr);
        }
      }
      const float m_sub = m_used == -INFINITY ? 0.f : m_used;
      float2 lsum = make_float2(0.f, 0.f), lusum = make_float2(0.f, 0.f);
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t rr[32];
        tmem_ld32(s_cols + (uint32_t)ch * 32u, rr);
        tmem_wait_ld();
        uint32_t pk[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          float2 s2 = make_float2(__uint_as_float(rr[2 * e]), __uint_as_float(rr[2 * e + 1]));
          if (raw_max) s2 = make_float2(scored<kCap>(rs, s2.x), scored<kCap>(rs, s2.y));
          const float2 p2 = make_float2(ex2(s2.x - m_sub), ex2(s2.y - m_sub));
          const __nv_bfloat162 pb = __floats2bfloat162_rn(p2.x, p2.y);
          pk[e] = *reinterpret_cast<const uint32_t*>(&pb);
          lsum = __fadd2_rn(lsum, make_float2(__uint_as_float(pk[e] << 16), __uint_as_float(pk[e] & 0xffff0000u)));
          lusum = __fadd2_rn(lusum, p2);
        }
        tmem_st16(s_cols + (uint32_t)ch * 16u, pk);
      }
      l += lsum.x + lsum.y;
      lu += lusum.x + lusum.y;
      tmem_wait_st();
      tc_fence_before();
      mbar_arrive(&sm.p_full[x]);
      ++j;
    }
    if (ok && j > 0) ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.o_done[x], (j - 1) & 1, a.status));
    if (ok && j > 0) {
      tc_fence_after();
      const float inv = l == 0.f ? 0.f : 1.f / l;  // (a NaN sum stays one)
      uint4* orow = reinterpret_cast<uint4*>(a.out + (bh * a.T + i) * kHeadDim);
#pragma unroll 1
      for (int ch = 0; ch < 4; ++ch) {
        uint32_t rr[32];
        tmem_ld32(o_cols + (uint32_t)ch * 32u, rr);
        tmem_wait_ld();
        if (i < c.T) {
#pragma unroll
          for (int e = 0; e < 32; e += 8) {
            uint32_t w[4];
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const __nv_bfloat162 o2 = __floats2bfloat162_rn(__uint_as_float(rr[e + 2 * u]) * inv,
                                                              __uint_as_float(rr[e + 2 * u + 1]) * inv);
              w[u] = *reinterpret_cast<const uint32_t*>(&o2);
            }
            orow[ch * 4 + e / 8] = make_uint4(w[0], w[1], w[2], w[3]);
          }
        }
      }
      if (i < c.T && a.lse)
        a.lse[bh * a.T + i] = lu == 0.f ? -INFINITY : (m_used + log2f(lu) - rs.slope2 * (float)ref) * kLn2;
    }
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) {
    if (lane == 0) mbar_wait(&sm.drain, 0);  // bounded; the MMAs drain before their TMEM is freed
    __syncwarp();
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
  }
}

// Leaves the ring as if the chunk's outputs had been appended in order: a CTA a (sequence, head)
// copies the last min(T, n) rows; the launch after it moves wp and fill, which these CTAs read.
__global__ void __launch_bounds__(256) ring_rows_kernel(int H, int n, int T, const uint4* __restrict__ k_out,
                                                        const uint4* __restrict__ v_out, uint4* __restrict__ ring_k,
                                                        uint4* __restrict__ ring_v, const int32_t* wp,
                                                        const int32_t* fill) {
  constexpr int kVec = kHeadDim / 8;
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const int w = wp[b], f = fill[b];
  if (w < 0 || w >= n || f < 0 || f > n) return;  // flagged by the attention
  const int64_t bh = (int64_t)b * H + blockIdx.x;
  const int keep = min(T, n);
  for (int idx = threadIdx.x; idx < keep * kVec; idx += blockDim.x) {
    const int tok = T - keep + idx / kVec, e = idx % kVec;
    const int slot = (int)(((int64_t)w + tok) % n);
    ring_k[(bh * n + slot) * kVec + e] = k_out[(bh * T + tok) * kVec + e];
    ring_v[(bh * n + slot) * kVec + e] = v_out[(bh * T + tok) * kVec + e];
  }
}

__global__ void __launch_bounds__(256) ring_state_kernel(int B, int n, int T, int32_t* wp, int32_t* fill) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.x * blockDim.x + threadIdx.x;
  if (b >= B) return;
  const int w = wp[b], f = fill[b];
  if (w < 0 || w >= n || f < 0 || f > n) return;
  wp[b] = (int)(((int64_t)w + T) % n);
  fill[b] = (int)min((int64_t)f + T, (int64_t)n);
}

}  // namespace

cudaError_t launch_scored_prefill(const ScoredPrefillLaunch& L, cudaStream_t stream) {
  CUtensorMap tq, tko, tvo, tpk, tpv, trk, trv;
  const int64_t bh = (int64_t)L.B * L.H;
  const bool ring = L.ring_k != nullptr, prefix = L.cap > 0;
  cudaError_t e;
  // without a prefix or a ring their maps are never used and stand on q
  if ((e = make_rows_map(&tq, L.q, bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&tko, L.k_out, bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&tvo, L.v_out, bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&tpk, prefix ? L.pk : L.q, prefix ? bh * L.cap : bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&tpv, prefix ? L.pv : L.q, prefix ? bh * L.cap : bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&trk, ring ? L.ring_k : L.q, ring ? bh * L.n : bh * L.T)) != cudaSuccess) return e;
  if ((e = make_rows_map(&trv, ring ? L.ring_v : L.q, ring ? bh * L.n : bh * L.T)) != cudaSuccess) return e;
  Args a;
  a.B = L.B;
  a.H = L.H;
  a.n = L.n;
  a.T = L.T;
  a.cap = L.cap;
  a.prefix_len = L.prefix_len;
  a.wp = L.wp;
  a.fill = L.fill;
  a.has_ring = ring ? 1 : 0;
  a.ranges = L.ranges;
  a.slopes = L.slopes;
  a.pos = L.pos;
  a.softcap = L.softcap;
  a.scale = L.scale;
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.lse = L.lse;
  a.status = L.status;
  const bool cap = L.softcap > 0.f, bias = L.slopes != nullptr;
  auto kernel = cap ? (bias ? scored_prefill_kernel<true, true> : scored_prefill_kernel<true, false>)
                    : (bias ? scored_prefill_kernel<false, true> : scored_prefill_kernel<false, false>);
  static unsigned long long done[4] = {};
  const size_t smem = sizeof(Smem) + 1024;
  if ((e = ensure_smem_limit(kernel, smem, &done[2 * cap + bias])) != cudaSuccess) return e;
  const dim3 grid((L.T + kCtaRows - 1) / kCtaRows, L.H, L.B);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  fill_launch_config(cfg, attr, grid, dim3(kThreads), smem, stream);
  if ((e = cudaLaunchKernelEx(&cfg, kernel, a, tq, tko, tvo, tpk, tpv, trk, trv)) != cudaSuccess) return e;
  if (!L.write_ring) return cudaSuccess;
  fill_launch_config(cfg, attr, dim3(L.H, L.B), dim3(256), 0, stream);
  if ((e = cudaLaunchKernelEx(&cfg, ring_rows_kernel, L.H, L.n, L.T, static_cast<const uint4*>(L.k_out),
                              static_cast<const uint4*>(L.v_out), static_cast<uint4*>(L.ring_k_w),
                              static_cast<uint4*>(L.ring_v_w), L.wp, L.fill)) != cudaSuccess)
    return e;
  fill_launch_config(cfg, attr, dim3((L.B + 255) / 256), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&cfg, ring_state_kernel, L.B, L.n, L.T, L.wp_w, L.fill_w);
}

}  // namespace rswa

// scored_prefill.cu -- chunked R-SWA prefill whose scores are capped, biased by distance and
// limited to each query's own document, on the sm_100a tensor cores (tcgen05 + TMEM).
//
// Query i of a chunk attends to the prefix rows [lo_i, hi_i) of its document, to the outputs j with
// i - n < j <= i and, for j < 0, to the previous chunk's last outputs in the ring, with
//   s = cap tanh(scale q.k / cap) - slope_h (pos_q - pos_k).
//
// A CTA has two streams of work, A and B, each a 128-row query tile against key tiles of 128 rows:
//   paired (many queries): A and B are neighbouring query tiles and walk the same key tiles, so a
//     key tile is fetched once for 256 queries;
//   split (few queries): A and B are the same query tile and take every other key tile, and a
//     cluster of up to 8 CTAs deals the key tiles out among its CTAs; the parts meet through shared
//     memory, the CTAs' through distributed shared memory.
// While one stream's softmax runs, the tensor core works on the other's products. Roles: warp 0 TMA
// producer of Q and K, warp 2 of V, warp 3 cleans V, one thread of warp 1 issues the MMAs, warps 4-11 /
// 12-19 softmax of stream A / B, two threads a row; P (bf16) goes back over S as the A operand of P V.
//
// Documents: the union of the rows' ranges, as up to four runs of rows, gives the prefix tiles;
// rows of a tile that no query of the CTA sees are zeroed in V (0 * NaN would reach O). A chunk over
// packed documents so costs what its documents cost, not what the prefix does, while a CTA's queries
// see at most four runs. What lies past the third run is taken as one run with its gaps, whose
// unseen rows are found query by query: 16 heads x 2304 queries, each 256 of them over eight documents of
// 300 rows, take 65 us where the documents touch and 6,600 us with gaps of 300 rows between them.
//
// What bounds it: a tile's MMAs take 1,024 cycles, and one ex2 a score as many of the special-function
// unit (16 a cycle and SM); a stream's chain of scores, maximum, exponentials and P V takes some 5,000, of which
// the two streams' overlap leaves the tensor pipe 40 to 49% busy. 2 x 16 heads x 4096 capped queries over 10272
// rows take 870 to 890 us (430 at the measured tensor rate) and run into the power limit there (820 in a burst).
//
// Scores: tanh(u) = 1 - 2 / (e^2u + 1) would cost two more special-function operations; where a warp's
// scores all have |u| = |scale q.k| / cap <= 0.4 (or 1), tanh is u times a minimax polynomial in u^2
// instead, on the packed FMA pipe. Scores against 64 bits, in units of the cap, at 12,288 points each: within
// 6.3e-8 (|u| up to 0.4), 1.4e-7 (up to 1) and 2.9e-7 (any, by the two operations).
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
constexpr int kQTiles = 2;                 // query tiles of a paired CTA, streams of any
constexpr int kMaxRows = kQTiles * kRows;
constexpr int kRegionBytes = kRows * 128;  // one 64-column SW128 region of a 128-row tile
constexpr int kTileBytes = 2 * kRegionBytes;
constexpr int kKStages = 3;
constexpr int kVStages = 2;
constexpr int kThreads = 640;
constexpr int kSoftmaxWarp0 = 4;           // warps 4-11: stream A, 12-19: stream B
constexpr int kHalf = kRows / 2;           // key columns of a softmax thread
constexpr int kMaxCluster = 8;
constexpr int kPartStride = kHeadDim + 4;  // floats of a row's part in shared memory (keeps rows off one bank)
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
  uint64_t v_full[kVStages], v_ready[kVStages], v_empty[kVStages];
  uint64_t s_full[kQTiles], p_full[kQTiles][2], o_done[kQTiles];
  uint64_t drain;
  uint64_t wait_limit_ns;  // of every wait (as a kernel parameter it cost 0.5 us of 52)
  uint32_t tmem_base;
  int abort_flag;
  int seen_by[kKStages];  // with a key tile: the streams that see it, as bits
  Ctx ctx;
  float half[2][2][kRows];  // what the two halves of a stream's columns tell each other
};
static_assert(sizeof(Smem) <= 227 * 1024, "shared memory");

// Split: a row's values on their way to the cluster, over the query tile that a split CTA does not have.
struct RowStats {
  float m[kRows], l[kRows], lse_ref[kRows];
};
static_assert((kKStages + kVStages) * kTileBytes >= kRows * kPartStride * 4, "parts lie over the K / V stages");

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
  float small_u;          // |u| up to which the short polynomial is taken (negative: never)
  int cluster;            // split: CTAs that share a query tile's key tiles
  int first;              // split: the first pair of query tiles that is this launch's
  int late;               // the launch before this one is its own first part: waited for at the end
  __nv_bfloat16* out;
  float* lse;
  int32_t* status;
  uint64_t wait_limit_ns;
  int drop_tile;           // a wait-timeout test: key tile that CTA 0 leaves out (-1: none)
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

// The prefix rows query i of sequence b sees (empty: 0, 0).
__device__ __forceinline__ int2 range_of(const Args& a, int m, int b, int i, bool report) {
  if (i >= a.T) return make_int2(0, 0);
  if (a.ranges == nullptr) return make_int2(0, m);
  const int2 r = __ldcg(a.ranges + (int64_t)b * a.T + i);
  if (r.x >= r.y) return make_int2(0, 0);
  if (r.x < 0 || r.y > m) {
    if (report) set_status(a.status, RSWA_DEVICE_BAD_RANGE);
    return make_int2(0, 0);
  }
  return r;
}

__device__ __forceinline__ bool wait_or_abort(Smem& sm, uint64_t* bar, uint32_t parity, int32_t* status) {
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

__device__ __forceinline__ float min3(float a, float b, float c) {
  float d;
  asm("min.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}

__device__ __forceinline__ float rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred P;\n\telect.sync _|P, 0xffffffff;\n\tselp.b32 %0, 1, 0, P;\n\t}" : "=r"(p));
  return p != 0;
}

__device__ __forceinline__ float2 splat(float x) { return make_float2(x, x); }

__device__ __forceinline__ float max_nan(float a, float b) {
  float d;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(d) : "f"(a), "f"(b));
  return d;
}

// 2^z of a pair without the special-function unit: z to the nearest integer (the low bits of z + 1.5 2^23) and a
// rest f in [-1/2, 1/2], 2^f as a minimax polynomial of degree 4 (relative error 2.6e-6, a 700th of the
// rounding to bf16 that follows), times 2 to the integer. z <= 2^8; NaN: NaN. An integer of -127 has the bits of
// 0 as its power: z below -126.5, -inf too, gives 0 (as ex2 with flush-to-zero does below -126).
__device__ __forceinline__ float2 ex2_pair(float2 z) {
  z = make_float2(max_nan(z.x, -127.f), max_nan(z.y, -127.f));
  const float2 t = __fadd2_rn(z, splat(12582912.f));
  const float2 n = __fadd2_rn(t, splat(-12582912.f));
  const float2 f = __ffma2_rn(n, splat(-1.f), z);
  float2 p = __ffma2_rn(splat(0.00957009898f), f, splat(0.0559178601f));
  p = __ffma2_rn(p, f, splat(0.240247449f));
  p = __ffma2_rn(p, f, splat(0.693121815f));
  p = __ffma2_rn(p, f, splat(0.999999261f));
  return __fmul2_rn(p, make_float2(__uint_as_float((__float_as_uint(t.x) << 23) + 0x3f800000u),
                                   __uint_as_float((__float_as_uint(t.y) << 23) + 0x3f800000u)));
}
// Of plain scores' exponentials every kPolyPairs-th pair goes there: with one in four 16 heads x 2304 queries
// x 10272 rows take 185 us instead of 188, and x 1152 queries 102 instead of 108. (Capped ones keep the FMA pipe busy.)
constexpr int kPolyPairs = 4;

// tanh(u) = u p(u^2): minimax polynomials, within 2e-8 (f32 rounding of their evaluation aside) for |u| up to 0.4 and
// up to 1 (four and seven terms).
constexpr float kTanhSmall = 0.4f, kTanhMid = 1.f;
__host__ __device__ constexpr float tanh_small_coef(int i) {
  constexpr float c[4] = {0.999999573f, -0.333297261f, 0.132505672f, -0.0468257397f};
  return c[i];
}
struct TanhMid {
  static constexpr int kTerms = 7;
  static __device__ __forceinline__ float coef(int i) {
    constexpr float c[kTerms] = {0.999999693f,  -0.333321293f,   0.133195837f,  -0.0532658353f,
                                 0.0199732827f, -0.00595128048f, 0.000963772187f};
    return c[i];
  }
};

// The short polynomial with the scores' factors in its coefficients: cap2 tanh(raw k) = raw q(raw^2),
// q_i = c_i cap2 k^(2 i + 1). A multiplication less a pair (889 -> 865 us at 2 x 16 heads x 4096 queries x
// 10272 rows, capped); taken where the coefficients stay well inside the f32 range (Args.small_u).
struct TanhFolded {
  float q[4];
};

__device__ __forceinline__ TanhFolded fold_tanh(float k, float cap2) {
  TanhFolded t;
  float f = cap2 * k;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    t.q[i] = tanh_small_coef(i) * f;
    f *= k * k;
  }
  return t;
}

__device__ __forceinline__ float2 capped_pair(float2 raw, const TanhFolded& t, float2 add) {
  const float2 w = __fmul2_rn(raw, raw);
  float2 p = __ffma2_rn(splat(t.q[3]), w, splat(t.q[2]));
  p = __ffma2_rn(p, w, splat(t.q[1]));
  p = __ffma2_rn(p, w, splat(t.q[0]));
  return __ffma2_rn(raw, p, add);
}

// cap2 tanh(raw k) + add, for a pair.
template <typename Poly>
__device__ __forceinline__ float2 capped_pair(float2 raw, float k, float cap2, float2 add) {
  const float2 u = __fmul2_rn(raw, splat(k));
  const float2 w = __fmul2_rn(u, u);
  float2 p = splat(Poly::coef(Poly::kTerms - 1) * cap2);
#pragma unroll
  for (int i = Poly::kTerms - 2; i >= 0; --i) p = __ffma2_rn(p, w, splat(Poly::coef(i) * cap2));
  return __ffma2_rn(u, p, add);
}

__device__ __forceinline__ float capped_exact(float raw, float k, float cap2) {
  return fmaf(-2.f * cap2, rcp(ex2(raw * (k * 2.f * kLog2e)) + 1.f), cap2);
}

// Visible columns [lo, hi) of a tile as bits of its w-th 32 columns.
__device__ __forceinline__ uint32_t column_bits(int lo, int hi, int w) {
  const int a = min(max(lo - 32 * w, 0), 32), b = min(max(hi - 32 * w, 0), 32);
  const uint32_t below_b = b == 32 ? 0xffffffffu : (1u << b) - 1, below_a = a == 32 ? 0xffffffffu : (1u << a) - 1;
  return below_b & ~below_a;
}

// A row's view of one key tile: columns [lo, hi) and [lo2, hi2) are visible; column e is at distance
// base - e (less the row's reference distance), and n further on from column cut (the ring's wrap).
struct RowTile {
  int lo, hi, lo2, hi2;
  int base, cut;
};

__device__ __forceinline__ RowTile row_tile(const Ctx& c, int kind, int start, int i, const int2& range, int pos, int ref) {
  RowTile t;
  t.lo2 = t.hi2 = 0;
  t.cut = kRows;
  if (kind == kPrefix) {
    t.lo = range.x - start;
    t.hi = range.y - start;
    t.base = pos - start - ref;
  } else if (kind == kBand) {
    t.lo = i - c.n + 1 - start;
    t.hi = min(i, c.T - 1) + 1 - start;
    t.base = i - start - ref;
  } else {
    // slots of ages 1 .. left: wp - 1 down to wp - left, round the ring's end
    const int left = min(c.fill, c.n - 1 - i);
    t.lo = max(c.wp - left, 0) - start;
    t.hi = (left > 0 ? c.wp : 0) - start;
    if (left > c.wp) {
      t.lo2 = c.n + c.wp - left - start;
      t.hi2 = c.n - start;
    }
    t.base = i + c.wp - start - ref;
    t.cut = c.wp - start;
  }
  return t;
}

// How a warp takes the tanh of some scores: by the largest |u| among its rows'.
enum Tanh { kSmall, kMid, kExact };

__device__ __forceinline__ Tanh tanh_of(float lowest, float highest, float k, float small_u) {
  const float u = fmaxf(highest, -lowest) * k;
  if (__all_sync(0xffffffffu, u <= small_u)) return kSmall;
  return __all_sync(0xffffffffu, u <= kTanhMid) ? kMid : kExact;
}

__device__ __forceinline__ float highest_of(const float (&x)[32], float a) {
  float b = a;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    a = max3(a, x[e], x[e + 1]);
    b = max3(b, x[e + 2], x[e + 3]);
  }
  return fmaxf(a, b);
}

__device__ __forceinline__ float lowest_of(const float (&x)[32], float a) {
  float b = a;
#pragma unroll
  for (int e = 0; e < 32; e += 4) {
    a = min3(a, x[e], x[e + 1]);
    b = min3(b, x[e + 2], x[e + 3]);
  }
  return fminf(a, b);
}

// Raw scores of a tile's columns [col0, col0 + 32) -> scores in the log2 domain, masked ones -inf.
// k: scale / cap, or scale log2(e) without a cap; full (uniform over the warp): nothing is masked.
template <bool kCap, bool kBias>
__device__ __forceinline__ void score_chunk(float (&x)[32], const RowTile& t, int col0, bool full, float k, float cap2,
                                            float small_u, float slope2, int n) {
  // -slope (base - e) = slope e + c0: exact integers, one rounding of the bias
  const float c0 = kBias ? -slope2 * (float)(t.base - col0) : 0.f;
  auto bias = [&](int e) {
    // (not paired: a pair of constants would take two moves, one is an immediate operand)
    return kBias ? make_float2(fmaf(slope2, (float)e, c0), fmaf(slope2, (float)(e + 1), c0)) : make_float2(0.f, 0.f);
  };
  const Tanh how = kCap ? tanh_of(lowest_of(x, INFINITY), highest_of(x, -INFINITY), k, small_u) : kSmall;
  if (kCap && how == kExact) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 b = bias(e);
      x[e] = capped_exact(x[e], k, cap2) + b.x;
      x[e + 1] = capped_exact(x[e + 1], k, cap2) + b.y;
    }
  } else if (kCap && how == kMid) {
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      const float2 s2 = capped_pair<TanhMid>(make_float2(x[e], x[e + 1]), k, cap2, bias(e));
      x[e] = s2.x;
      x[e + 1] = s2.y;
    }
  } else {
    const TanhFolded folded = fold_tanh(k, cap2);  // (without a cap not used)
#pragma unroll
    for (int e = 0; e < 32; e += 2) {
      float2 s2 = make_float2(x[e], x[e + 1]);
      if (kCap)
        s2 = capped_pair(s2, folded, bias(e));
      else
        s2 = kBias ? __ffma2_rn(s2, splat(k), bias(e)) : __fmul2_rn(s2, splat(k));
      x[e] = s2.x;
      x[e + 1] = s2.y;
    }
  }
  if (kBias && t.cut < kRows) {  // the ring's wrap
    const float wrap = -slope2 * (float)n;
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] += col0 + e < t.cut ? 0.f : wrap;
  }
  if (!full) {
    const int w = col0 / 32;
    const uint32_t bits = column_bits(t.lo, t.hi, w) | column_bits(t.lo2, t.hi2, w);
#pragma unroll
    for (int e = 0; e < 32; ++e) x[e] = (bits >> e) & 1 ? x[e] : -INFINITY;
  }
}

__device__ __forceinline__ void cluster_sync() {
  asm volatile("barrier.cluster.arrive.release;\n\tbarrier.cluster.wait.acquire;" ::: "memory");
}

__device__ __forceinline__ uint32_t cluster_rank() {
  uint32_t r;
  asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
  return r;
}

// The address of the same shared-memory place in CTA `rank` of the cluster.
__device__ __forceinline__ uint32_t peer_smem(const void* p, uint32_t rank) {
  uint32_t a;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_addr(p)), "r"(rank));
  return a;
}

__device__ __forceinline__ float peer_f32(uint32_t a) {
  float v;
  asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ float4 peer_f32x4(uint32_t a) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a) : "memory");
  return v;
}

__device__ __forceinline__ uint4 to_bf16x8(const float* o) {
  uint32_t w[4];
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const __nv_bfloat162 o2 = __floats2bfloat162_rn(o[2 * u], o[2 * u + 1]);
    w[u] = *reinterpret_cast<const uint32_t*>(&o2);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// The two warps that share 32 rows of a stream meet (barrier 1 + pair); whether any thread of them says so.
__device__ __forceinline__ bool pair_any(int pair, bool v) {
  uint32_t any;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "barrier.cta.red.or.pred q, %2, 64, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}"
      : "=r"(any)
      : "r"(v ? 1u : 0u), "r"(1 + pair)
      : "memory");
  return any != 0;
}
__device__ __forceinline__ void stream_barrier(int x) { asm volatile("barrier.cta.sync %0, 256;" ::"r"(9 + x) : "memory"); }
// Both streams meet.
__device__ __forceinline__ void softmax_barrier() { asm volatile("barrier.cta.sync 11, 512;" ::: "memory"); }

template <bool kCap, bool kBias, bool kSplit>
__global__ void __launch_bounds__(kThreads, 1)
    scored_prefill_kernel(const __grid_constant__ Args a, const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_ko, const __grid_constant__ CUtensorMap tm_vo,
                          const __grid_constant__ CUtensorMap tm_pk, const __grid_constant__ CUtensorMap tm_pv,
                          const __grid_constant__ CUtensorMap tm_rk, const __grid_constant__ CUtensorMap tm_rv) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
  constexpr int kCtaRows = kSplit ? kRows : kMaxRows;
  // P goes to the MMAs in two parts, so that the first 64 keys' products run under the exponentials of the
  // others: 202 -> 196 us at 16 heads x 2304 queries x 10272 rows of plain scores; capped ones without a bias,
  // whose exponentials wait on the FMA pipe, took 879 us whole and 889 in parts (2 x 16 heads x 4096 queries).
  constexpr bool kInParts = !kCap || kBias;
  const int cluster = kSplit ? a.cluster : 1;
  const int rank = kSplit ? (int)cluster_rank() : 0;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  // pairs of query tiles in order: a (sequence, head)'s side by side
  const int pairs = (a.T + kMaxRows - 1) / kMaxRows;
  const int unit = kSplit ? blockIdx.x / cluster : blockIdx.x;
  const int pair = kSplit ? a.first + unit / 2 : unit;
  const int64_t bh = pair / pairs;
  const int b = (int)(bh / a.H), h = (int)(bh - (int64_t)b * a.H);
  const int qt = kSplit ? pair % pairs * 2 + (unit & 1) : pair % pairs;
  if ((smem_addr(smem_raw) & 1023u) != 0) {  // it is, with no other shared memory in the kernel
    if (tid == 0) set_status(a.status, RSWA_DEVICE_PIPELINE);
    return;
  }
  // A late launch's CTAs start when the last of the first part's have (they have waited for what came
  // before both), and run beside them; what follows waits for this launch, so it waits for them.
  if (!a.late) griddep_wait();
  griddep_launch_dependents();
  if (kSplit && qt * kRows >= a.T) {  // the chunk ends in the first tile of the pair
    if (a.late) griddep_wait();
    return;
  }
  if (tid == 0) {
    sm.abort_flag = 0;
    sm.wait_limit_ns = a.wait_limit_ns;
    mbar_init(&sm.q_full, 1);
    for (int s = 0; s < kKStages; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    for (int s = 0; s < kVStages; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_ready[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    for (int x = 0; x < kQTiles; ++x) {
      mbar_init(&sm.s_full[x], 1);
      for (int u = 0; u < 2; ++u) mbar_init(&sm.p_full[x][u], 8);  // one arrival a warp
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
  } else if (warp == 0) {
    // ---- the CTA's key tiles ----
    const bool first = qt == 0 && rank == 0 && h == 0 && lane == 0;
    // (inputs through L2: a late launch starts while its first part runs, past no launch boundary
    // that would have cleared what an L1 holds since they were written)
    int m = a.cap > 0 ? __ldcg(a.prefix_len + b) : 0;
    if (m < 0 || m > a.cap) {
      if (first) set_status(a.status, RSWA_DEVICE_BAD_PREFIX_LEN);
      m = 0;
    }
    if (kBias) {
      const int p = __ldcg(a.pos + b);
      if (p < 0 || p > kMaxPos) {
        if (first) set_status(a.status, RSWA_DEVICE_BAD_POS);
        m = 0;
      }
    }
    const int i0 = qt * kCtaRows;
    int2 rg[kCtaRows / 32];  // lane's rows: 32 u + lane
#pragma unroll
    for (int u = 0; u < kCtaRows / 32; ++u) rg[u] = range_of(a, m, b, i0 + 32 * u + lane, h == 0 && rank == 0);
    Ctx& c = sm.ctx;
#pragma unroll
    for (int x = 0; x < kCtaRows / kRows; ++x) {
      int lo = INT32_MAX, hi = 0;
#pragma unroll
      for (int u = 0; u < kRows / 32; ++u) {
        const int2 g = rg[x * (kRows / 32) + u];
        if (g.y > g.x) {
          lo = min(lo, g.x);
          hi = max(hi, g.y);
        }
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
        const int w = __ldcg(a.wp + b), f = __ldcg(a.fill + b);
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
      const int all = np + c.nr + min(i0 + kCtaRows - 1, a.T - 1) / kRows - c.jt0 + 1;
      c.total = kSplit ? (all - rank + cluster - 1) / cluster : all;  // key tiles rank, rank + cluster, ...
      // a CTA of this launch gave up on a wait: no work (the output is flagged invalid)
      if (*reinterpret_cast<volatile int32_t*>(a.status) & RSWA_DEVICE_WAIT_TIMEOUT) c.total = 0;
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const Ctx& c = sm.ctx;
  const uint32_t tmem = sm.tmem_base;
  const int total = c.total;
  // this CTA's t-th key tile
  auto tile_of = [&](int t, int& kind, int& start) { tile_kind(c, kSplit ? t * cluster + rank : t, kind, start); };
  if (warp < kSoftmaxWarp0) {
    int issued = 0;  // by a producer: key tiles up to here
    if (warp == 0 || warp == 2) {
      // ---------------- producers: Q and K tiles (warp 0), V tiles (warp 2) ----------------
      if (lane == 0) {
        const bool is_k = warp == 0;
        if (is_k) {
          const int qrow = (int)(bh * a.T) + c.i0;
          mbar_arrive_expect_tx(&sm.q_full, kCtaRows / kRows * kTileBytes);
          for (int x = 0; x < kCtaRows / kRows; ++x) {
            tma_load_2d(sm.q[x], &tm_q, 0, qrow + x * kRows, &sm.q_full);
            tma_load_2d(sm.q[x] + kRegionBytes, &tm_q, 64, qrow + x * kRows, &sm.q_full);
          }
        }
        const int stages = is_k ? kKStages : kVStages;
        uint64_t* full = is_k ? sm.k_full : sm.v_full;
        uint64_t* empty = is_k ? sm.k_empty : sm.v_empty;
        for (int t = 0; t < total; issued = ++t) {
          const int s = t % stages;
          if (t >= stages && !wait_or_abort(sm, &empty[s], ((t / stages) - 1) & 1, a.status)) break;
          int kind, start;
          tile_of(t, kind, start);
          const CUtensorMap* map = is_k ? (kind == kPrefix ? &tm_pk : (kind == kRing ? &tm_rk : &tm_ko))
                                        : (kind == kPrefix ? &tm_pv : (kind == kRing ? &tm_rv : &tm_vo));
          const int64_t rows = kind == kPrefix ? a.cap : (kind == kRing ? a.n : a.T);
          const int row = (int)(bh * rows) + start;
          uint8_t* dst = is_k ? sm.k[s] : sm.v[s];
          if (is_k && !kSplit)  // released by the arrival below
            sm.seen_by[s] = (tile_visible(c, 0, kind, start) ? 1 : 0) | (tile_visible(c, 1, kind, start) ? 2 : 0);
          if (is_k && t == a.drop_tile && blockIdx.x == 0) continue;  // a wait-timeout test
          mbar_arrive_expect_tx(&full[s], kTileBytes);
          tma_load_2d(dst, map, 0, row, &full[s]);
          tma_load_2d(dst + kRegionBytes, map, 64, row, &full[s]);
        }
      }
    } else if (warp == 1) {
      // ---------------- MMA issuer: one thread ----------------
      // The tensor core's queue is two or three MMAs deep: issuing blocks for about as long as they
      // run, and whatever else this thread does leaves the tensor core idle. So it waits, issues and
      // commits, and others look tiles up (warp 0) and clean V (warp 3).
      if (elect_one()) {
        constexpr uint32_t kIdescQK = idesc_bf16_m128_n128(0);
        constexpr uint32_t kIdescPV = idesc_bf16_m128_n128(1);
        const uint64_t q_desc = smem_desc_sw128(smem_addr(sm.q[0]), 16, 1024);
        const uint64_t k_desc = smem_desc_sw128(smem_addr(sm.k[0]), 16, 1024);
        const uint64_t v_desc = smem_desc_sw128(smem_addr(sm.v[0]), kRegionBytes, 1024);
        auto issue_s = [&](int x, int ks) {  // S_x = Q K^T
          const uint64_t q = q_desc + (uint64_t)((kSplit ? 0 : x) * (kTileBytes >> 4)), k = k_desc + (uint64_t)(ks * (kTileBytes >> 4));
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            const uint64_t off = (uint64_t)(((kk >> 2) * kRegionBytes + (kk & 3) * 32) >> 4);
            tc_mma_ss(tmem + (uint32_t)x * 128u, q + off, k + off, kIdescQK, kk > 0);
          }
          tc_commit(&sm.s_full[x]);
        };
        auto issue_pv = [&](int x, int vs, uint32_t phase, bool more) {  // O_x += P_x V, P in two parts as it comes
          const uint64_t v = v_desc + (uint64_t)(vs * (kTileBytes >> 4));
#pragma unroll
          for (int e = 0; e < 8; ++e) {
            const int kk = (e & 1) + (e >> 1 & 1) * 4 + (e >> 2) * 2;  // both halves' first 32 columns, then their last
            if (e == 0 || (kInParts && e == 4)) {
              if (!wait_or_abort(sm, &sm.p_full[x][kInParts ? e / 4 : 1], phase, a.status)) return false;
              tc_fence_after();
            }
            tc_mma_ts(tmem + kColO + (uint32_t)x * 128u, tmem + (uint32_t)x * 128u + (uint32_t)((kk >> 2) * kHalf + (kk & 3) * 8),
                      v + (uint64_t)(kk * (2048 >> 4)), kIdescPV, (more || e > 0) ? 1u : 0u);
          }
          tc_commit(&sm.o_done[x]);
          return true;
        };
        bool ok = wait_or_abort(sm, &sm.q_full, 0, a.status);
        uint32_t p_phase[kQTiles] = {0, 0};
        bool more[kQTiles] = {false, false};
        int ks = 0, vs = 0;
        uint32_t k_phase = 0, v_phase = 0;
        auto take_k = [&](int& seen) {  // the next key tile has landed
          if (!wait_or_abort(sm, &sm.k_full[ks], k_phase, a.status)) return false;
          tc_fence_after();
          if (!kSplit) seen = *reinterpret_cast<volatile int*>(&sm.seen_by[ks]);
          return true;
        };
        auto free_k = [&]() {
          tc_commit(&sm.k_empty[ks]);
          if (++ks == kKStages) {
            ks = 0;
            k_phase ^= 1;
          }
        };
        int seen = 0, seen_next = 0;
        if (kSplit) {
          for (int t = 0; ok && t < min(2, total); ++t)
            if ((ok = take_k(seen))) {
              issue_s(t, ks);
              free_k();
            }
        } else if (ok && total > 0 && (ok = take_k(seen))) {  // (no tile: a CTA after a give-up)
          if (seen & 1) issue_s(0, ks);
          if (seen & 2) issue_s(1, ks);
          free_k();
        }
        if (kSplit) {
          // The streams' tiles in order. V stage x is stream x's; a key tile's stage and phase go by its number.
          // With a bias, whose tiles cost unlike (masked, whole), a stream whose P is there goes ahead of the
          // other's one tile earlier: 3 x 16 heads x 333 queries over documents 55 -> 52 us, over 2592 rows each
          // 58.5 -> 56.3. Alike tiles keep each other in step better than this does: 16 heads x 1152 capped queries
          // over 10272 rows took 122 us in order, 130 so.
          static_assert(kVStages == 2, "a V stage a stream");
          int at[2] = {0, 1};  // each stream's next tile
          while (ok && min(at[0], at[1]) < total) {
            int x = at[1] < at[0];
            const int y = x ^ 1, ty = at[y];
            if (kBias && ty == at[x] + 1 && ty < total) {
              constexpr int kFirst = kInParts ? 0 : 1;
              for (int i = 0; i < 4096; ++i) {  // then it waits for the earlier one
                if (mbar_try_wait(&sm.p_full[x][kFirst], (at[x] >> 1) & 1)) break;
                if (mbar_try_wait(&sm.p_full[y][kFirst], (ty >> 1) & 1) && mbar_try_wait(&sm.v_ready[y], (ty >> 1) & 1) &&
                    (ty + 2 >= total || mbar_try_wait(&sm.k_full[(ty + 2) % kKStages], ((ty + 2) / kKStages) & 1))) {
                  x = y;
                  break;
                }
              }
            }
            const int t = at[x];
            if (!(ok = wait_or_abort(sm, &sm.v_ready[x], (t >> 1) & 1, a.status))) break;
            if (!(ok = issue_pv(x, x, (t >> 1) & 1, t > 1))) break;
            tc_commit(&sm.v_empty[x]);
            if (t + 2 < total) {
              const int k = (t + 2) % kKStages;
              if (!(ok = wait_or_abort(sm, &sm.k_full[k], ((t + 2) / kKStages) & 1, a.status))) break;
              tc_fence_after();
              issue_s(x, k);
              tc_commit(&sm.k_empty[k]);
            }
            at[x] += 2;
          }
        }
        for (int t = 0; !kSplit && ok && t < total; ++t) {
          if (!(ok = wait_or_abort(sm, &sm.v_ready[vs], v_phase, a.status))) break;
          const bool next = t + 1 < total;
#pragma unroll
          for (int x = 0; x < kQTiles; ++x) {
            if (seen >> x & 1) {
              if (!(ok = issue_pv(x, vs, p_phase[x], more[x]))) break;
              p_phase[x] ^= 1;
              more[x] = true;
            }
            if (x == 0 && next && !(ok = take_k(seen_next))) break;
            if (x == 1) tc_commit(&sm.v_empty[vs]);
            if (next && (seen_next >> x & 1)) issue_s(x, ks);
          }
          if (!ok) break;
          if (next) free_k();
          seen = seen_next;
          if (++vs == kVStages) {
            vs = 0;
            v_phase ^= 1;
          }
        }
        tc_commit(&sm.drain);  // fires once every issued MMA is done
      }
    } else {
      // ---------------- V rows that no query of the CTA sees: zeroed (whole warp) ----------------
      bool ok = true;
      for (int t = 0; ok && t < total; ++t) {
        const int vs = t % kVStages;
        int kind, start;
        tile_of(t, kind, start);
        // a prefix tile inside one run is seen whole
        bool whole = kind == kBand && start + kRows <= c.T;
        if (kind == kPrefix)
          for (int r = 0; r < c.runs; ++r)
            whole |= start >= c.lo[r] && start + kRows <= c.hi[r] && (c.exact || r < kRuns - 1);
        ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.v_full[vs], (t / kVStages) & 1, a.status));
        if (!ok) break;
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
            }
          }
          fence_async_smem();
          __syncwarp();
        }
        if (lane == 0) mbar_arrive(&sm.v_ready[vs]);
      }
    }
    __syncwarp();
    if (kSplit && cluster > 1) {
      cluster_sync();
      cluster_sync();
    }
    __syncthreads();
    if (a.late) griddep_wait();
    // After a give-up, which may have come long after the last copy was issued: the copies in flight land
    // (bounded) before the CTA's shared memory goes away.
    if ((warp == 0 || warp == 2) && lane == 0 && sm.abort_flag) {
      if (warp == 0) {
        land_copies(&sm.q_full, 1, 1, -1, a.wait_limit_ns);
        land_copies(sm.k_full, kKStages, issued, blockIdx.x == 0 ? a.drop_tile : -1, a.wait_limit_ns);
      } else {
        land_copies(sm.v_full, kVStages, issued, -1, a.wait_limit_ns);
      }
    }
    if (warp == 1) {
      tc_fence_after();
      if (lane == 0) mbar_wait(&sm.drain, 0);  // bounded; the MMAs drain before their TMEM is freed
      __syncwarp();
      asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
  } else {
    // ---------------- softmax: two threads a row of a stream's tile, 64 key columns each ----------------
    const int sw = warp - kSoftmaxWarp0;
    const int x = sw >> 3, half = sw >> 2 & 1;
    const int r = (sw & 3) * 32 + lane;
    const int row = (kSplit ? 0 : x * kRows) + r;  // row of the CTA
    const int i = c.i0 + row;
    const int col0 = half * kHalf;
    const int rows32 = 4 * x + (sw & 3);  // its 32 rows of the CTA's, which one other warp has too
    const uint32_t lane_base = (uint32_t)((sw & 3) * 32) << 16;
    const uint32_t s_cols = tmem + lane_base + (uint32_t)(x * 128 + col0);  // its scores; its P goes over their first half
    const uint32_t o_cols = tmem + lane_base + kColO;                       // O of stream A; B's is 128 columns on
    const int2 range = range_of(a, c.m, b, i, false);
    const float mul = kCap ? a.scale / a.softcap : a.scale * kLog2e;
    const float cap2 = a.softcap * kLog2e;
    float slope2 = 0.f;
    int pos = 0, ref = 0;  // ref: the distance of the row's most favoured key, taken off all of them
    if (kBias) {
      const float slope = __ldcg(a.slopes + h);
      slope2 = slope * kLog2e;
      pos = __ldcg(a.pos + b) + i;
      const bool pre = range.y > range.x;
      if (slope >= 0.f)
        ref = pre ? min(0, pos - (range.y - 1)) : 0;
      else
        ref = max(min(i + c.fill, c.n - 1), pre ? pos - range.x : 0);
    }
    // Where the bias changes by at most 2^60 along 32 columns, their largest raw score and their largest bias
    // bound the row's maximum closely enough: its weights stay above 2^-69, far from f32's least. (Paired only:
    // 382 -> 358 us at 16 heads x 2368 queries x 10272 rows, capped, by 64 columns and 334 -> 326 later by 32; a split
    // chunk of 3 x 333 queries over documents, whose tiles wait for the slowest of 8 warps, often a masked one, took
    // 55 us without it and 59 with.)
    const bool gentle = fabsf(slope2) * 31.f <= 60.f;
    // l sums the unrounded weights, for O and lse alike: where one key dominates, O is off by the
    // rounding of its weight (at most half a bf16 step, as the output's own rounding); summing the
    // rounded ones too cost three more instructions a score pair
    float m_used = -INFINITY, l = 0.f;  // m_used is the same in both threads of a row
    int j = 0;                          // key tiles this stream has seen
    bool ok = true;
    for (int t = kSplit ? x : 0; t < total; t += kSplit ? 2 : 1) {
      int kind, start;
      tile_of(t, kind, start);
      if (!kSplit && !tile_visible(c, x, kind, start)) continue;
      ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.s_full[x], j & 1, a.status));
      tc_fence_after();
      const RowTile rt = row_tile(c, kind, start, i, range, pos, ref);
      // does any row of this warp see one of its columns; do all rows see all of them
      const int from = max(rt.lo, col0), from2 = max(rt.lo2, col0), to = col0 + kHalf;
      const bool none = __all_sync(0xffffffffu, from >= min(rt.hi, to) && from2 >= min(rt.hi2, to));
      const bool full = __all_sync(0xffffffffu, rt.lo <= col0 && rt.hi >= to);
      // The passes over the row's scores go 32 columns at a time, through TMEM, in loops that are not
      // unrolled: holding all of them in registers made straight-line code of 20 to 40 KB a tile, which
      // the instruction cache did not feed (a biased tile took 8,000 cycles instead of 4,000). 16 columns at
      // a time took 236 us where this takes 224 (16 heads x 2304 capped queries x 10272 rows).
      auto load = [&](int ch, float(&v)[32]) {
        uint32_t raw[32];
        tmem_ld32(s_cols + (uint32_t)ch * 32u, raw);
        tmem_wait_ld();
#pragma unroll
        for (int e = 0; e < 32; ++e) v[e] = __uint_as_float(raw[e]);
      };
      Tanh how = kExact;
      bool fused = false;
      float tmax = -INFINITY;
      if (ok && !none) {
        if (full && (!kBias || (!kSplit && gentle && rt.cut >= kRows))) {
          float lowest = INFINITY;
          float2 top = splat(-INFINITY);  // with a bias of each 32 columns, else of all
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            float v[32];
            load(ch, v);
            if (kBias) top.x = top.y;
            top.y = highest_of(v, kBias ? -INFINITY : top.y);
            if (kCap) lowest = lowest_of(v, lowest);
          }
          if (!kBias) top.x = top.y;
          if (kCap) how = tanh_of(lowest, fmaxf(top.x, top.y), mul, a.small_u);
          // without a mask the raw maxima give the maximum (a bound of it, where a bias is added), and the
          // scoring joins the exponentials' loop
          fused = !kCap || how != kExact;
          if (!kCap)
            top = __fmul2_rn(top, splat(mul));
          else if (how == kSmall)
            top = capped_pair(top, fold_tanh(mul, cap2), splat(0.f));
          else if (how == kMid)
            top = capped_pair<TanhMid>(top, mul, cap2, splat(0.f));
          if (kBias) {
            const float b0 = fmaf(fmaxf(slope2, 0.f), 31.f, -slope2 * (float)(rt.base - col0));
            top = make_float2(top.x + b0, top.y + fmaf(slope2, 32.f, b0));
          }
          tmax = fmaxf(top.x, top.y);
        }
        if (!fused) {
          tmax = -INFINITY;
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            float v[32];
            load(ch, v);
            score_chunk<kCap, kBias>(v, rt, col0 + ch * 32, full, mul, cap2, a.small_u, slope2, c.n);
            tmax = highest_of(v, tmax);
            uint32_t w[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) w[e] = __float_as_uint(v[e]);
            tmem_st32(s_cols + (uint32_t)ch * 32u, w);
          }
          tmem_wait_st();
        }
      }
      // Both warps of the rows meet here, also after a give-up. The running maximum only moves when
      // it grows by more than 2^8 (the exponentials stay below 256): then the halves agree on it.
      if (pair_any(rows32, !ok || tmax > m_used + kLazyRescaleLog2)) {
        sm.half[x][half][r] = tmax;
        if (pair_any(rows32, !ok)) {
          ok = false;
          break;
        }
        tmax = fmaxf(tmax, sm.half[x][half ^ 1][r]);
        const bool rescale = tmax > m_used + kLazyRescaleLog2;
        float alpha = 1.f;
        if (rescale) {
          alpha = ex2(m_used - tmax);
          l *= alpha;
          m_used = tmax;
        }
        // the previous P V of this stream is done (the commit that completed S covers it)
        if (j > 0 && __any_sync(0xffffffffu, rescale)) {
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            uint32_t rr[32];
            tmem_ld32(o_cols + (uint32_t)(x * 128 + col0 + ch * 32), rr);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e) rr[e] = __float_as_uint(__uint_as_float(rr[e]) * alpha);
            tmem_st32(o_cols + (uint32_t)(x * 128 + col0 + ch * 32), rr);
          }
        }
      }
      auto given = [&](int part) {  // of P
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.p_full[x][part]);
      };
      if (none) {
        const uint32_t zero[16] = {};
#pragma unroll
        for (int ch = 0; ch < 2; ++ch) tmem_st16(s_cols + (uint32_t)ch * 16u, zero);
        if (kInParts) given(0);
      } else {
        const float2 minus_m = splat(m_used == -INFINITY ? 0.f : -m_used);
        float2 sum0 = make_float2(0.f, 0.f), sum1 = make_float2(0.f, 0.f);
        auto weights = [&](auto&& less_m) {  // less_m: a pair of s, what is added to it -> score - m
#pragma unroll 1
          for (int ch = 0; ch < 2; ++ch) {
            float v[32];
            load(ch, v);
            uint32_t pk[16];
            const float c0 = kBias && !kSplit ? fmaf(-slope2, (float)(rt.base - col0 - ch * 32), minus_m.x) : 0.f;
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const float2 add = kBias && !kSplit && fused ? make_float2(fmaf(slope2, (float)(2 * e), c0), fmaf(slope2, (float)(2 * e + 1), c0)) : minus_m;
              const float2 z2 = less_m(make_float2(v[2 * e], v[2 * e + 1]), add);
              const bool poly = !kCap && !kBias && e % kPolyPairs == 1;
              const float2 p2 = poly && fused ? ex2_pair(z2) : make_float2(ex2(z2.x), ex2(z2.y));
              const __nv_bfloat162 pb = __floats2bfloat162_rn(p2.x, p2.y);
              pk[e] = *reinterpret_cast<const uint32_t*>(&pb);
              if (e & 1)
                sum1 = __fadd2_rn(sum1, p2);
              else
                sum0 = __fadd2_rn(sum0, p2);
            }
            tmem_st16(s_cols + (uint32_t)ch * 16u, pk);
            if (kInParts && ch == 0) given(0);
          }
        };
        if (!fused)  // (a split biased chunk's only way)
          weights([&](float2 z, float2) { return __fadd2_rn(z, minus_m); });
        else if (!kCap)
          weights([&](float2 z, float2 add) { return __ffma2_rn(z, splat(mul), add); });
        else if (how == kSmall)
          weights([&, folded = fold_tanh(mul, cap2)](float2 z, float2 add) { return capped_pair(z, folded, add); });
        else
          weights([&](float2 z, float2 add) { return capped_pair<TanhMid>(z, mul, cap2, add); });
        l += (sum0.x + sum0.y) + (sum1.x + sum1.y);
      }
      given(1);
      ++j;
    }
    if (ok && j > 0) ok = __all_sync(0xffffffffu, wait_or_abort(sm, &sm.o_done[x], (j - 1) & 1, a.status));
    const float lse_ref = kBias ? slope2 * (float)ref : 0.f;
    sm.half[x][half][r] = l;
    if (!kSplit) {
      stream_barrier(x);  // all 256 threads of the stream come here, also after a give-up
      if (ok && j > 0) {
        tc_fence_after();
        const float L = sm.half[x][0][r] + sm.half[x][1][r];
        const float inv = L == 0.f ? 0.f : 1.f / L;  // (a NaN sum stays one)
        uint4* orow = reinterpret_cast<uint4*>(a.out + (bh * a.T + i) * kHeadDim + col0);
#pragma unroll 1
        for (int ch = 0; ch < 2; ++ch) {
          uint32_t rr[32];
          tmem_ld32(o_cols + (uint32_t)(x * 128 + col0 + ch * 32), rr);
          tmem_wait_ld();
          if (i < c.T) {
            float o[32];
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __uint_as_float(rr[e]) * inv;
#pragma unroll
            for (int e = 0; e < 4; ++e) orow[ch * 4 + e] = to_bf16x8(o + 8 * e);
          }
        }
        if (half == 0 && i < c.T && a.lse)
          a.lse[bh * a.T + i] = L == 0.f ? -INFINITY : (m_used + log2f(L) - lse_ref) * kLn2;
      }
    } else {
      // ---- the two streams' parts of the row meet; each of the four groups takes 32 columns ----
      RowStats* own = reinterpret_cast<RowStats*>(sm.q[1]);
      if (half == 0) own[x].m[r] = m_used;
      tc_fence_before();
      softmax_barrier();  // all 512 threads come here, also after a give-up
      tc_fence_after();
      const float ma = own[0].m[r], mb = own[1].m[r];
      const float M = fmaxf(ma, mb), m_sub = M == -INFINITY ? 0.f : M;
      const bool empty = total < 1, one = total < 2;  // streams without a key tile have no O
      const float fa = empty ? 0.f : ex2(ma - m_sub), fb = one ? 0.f : ex2(mb - m_sub);
      const float L = fmaf(sm.half[1][0][r] + sm.half[1][1][r], fb, (sm.half[0][0][r] + sm.half[0][1][r]) * fa);
      const float inv = cluster > 1 ? 1.f : (L == 0.f ? 0.f : 1.f / L);
      float* part = reinterpret_cast<float*>(sm.k[0]) + r * kPartStride;  // every copy and MMA of the CTA is done
      {
        const int col = (2 * x + half) * 32;
        uint32_t ra[32], rb[32];
        if (!empty) tmem_ld32(o_cols + (uint32_t)col, ra);
        if (!one) tmem_ld32(o_cols + 128u + (uint32_t)col, rb);
        tmem_wait_ld();
        float o[32];
#pragma unroll
        for (int e = 0; e < 32; ++e) {
          o[e] = empty ? 0.f : __uint_as_float(ra[e]) * fa;
          if (!one) o[e] = fmaf(__uint_as_float(rb[e]), fb, o[e]);
          o[e] *= inv;
        }
        if (cluster > 1) {
#pragma unroll
          for (int e = 0; e < 32; e += 4)
            *reinterpret_cast<float4*>(part + col + e) = make_float4(o[e], o[e + 1], o[e + 2], o[e + 3]);
        } else if (i < c.T) {
          uint4* orow = reinterpret_cast<uint4*>(a.out + (bh * a.T + i) * kHeadDim + col);
#pragma unroll
          for (int e = 0; e < 4; ++e) orow[e] = to_bf16x8(o + 8 * e);
        }
      }
      if (cluster == 1) {
        if (x == 0 && half == 0 && i < c.T && a.lse)
          a.lse[bh * a.T + i] = L == 0.f ? -INFINITY : (M + log2f(L) - lse_ref) * kLn2;
      } else {
        RowStats& all = own[2];
        if (x == 0 && half == 0) {
          all.m[r] = M;
          all.l[r] = L;
          all.lse_ref[r] = lse_ref;
        }
        // ---- the cluster's parts meet: CTA `rank` joins rows [rank, rank + 1) * 128 / cluster ----
        cluster_sync();  // every CTA of the cluster comes here, also after a give-up
        const int rows = kRows / cluster;
        for (int v = tid - kSoftmaxWarp0 * 32; v < rows * (kHeadDim / 8); v += kThreads - kSoftmaxWarp0 * 32) {
          const int r2 = rank * rows + v / (kHeadDim / 8), d = v % (kHeadDim / 8) * 8, i2 = c.i0 + r2;
          if (i2 >= c.T) continue;
          float ms[kMaxCluster], Mc = -INFINITY;
#pragma unroll
          for (int u = 0; u < kMaxCluster; ++u) {
            ms[u] = u < cluster ? peer_f32(peer_smem(&all.m[r2], u)) : -INFINITY;
            Mc = fmaxf(Mc, ms[u]);
          }
          const float mc_sub = Mc == -INFINITY ? 0.f : Mc;
          float o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f}, Lc = 0.f;
#pragma unroll
          for (int u = 0; u < kMaxCluster; ++u) {
            if (u >= cluster) break;
            const float f = exp2f(ms[u] - mc_sub);
            Lc = fmaf(peer_f32(peer_smem(&all.l[r2], u)), f, Lc);
            const uint32_t at = peer_smem(reinterpret_cast<const float*>(sm.k[0]) + r2 * kPartStride + d, u);
            const float4 p = peer_f32x4(at), q = peer_f32x4(at + 16);
            o[0] = fmaf(p.x, f, o[0]), o[1] = fmaf(p.y, f, o[1]), o[2] = fmaf(p.z, f, o[2]), o[3] = fmaf(p.w, f, o[3]);
            o[4] = fmaf(q.x, f, o[4]), o[5] = fmaf(q.y, f, o[5]), o[6] = fmaf(q.z, f, o[6]), o[7] = fmaf(q.w, f, o[7]);
          }
          const float inv_c = Lc == 0.f ? 0.f : 1.f / Lc;
#pragma unroll
          for (int e = 0; e < 8; ++e) o[e] *= inv_c;
          reinterpret_cast<uint4*>(a.out + (bh * a.T + i2) * kHeadDim)[d / 8] = to_bf16x8(o);
          if (d == 0 && a.lse)
            a.lse[bh * a.T + i2] = Lc == 0.f ? -INFINITY : (Mc + log2f(Lc) - all.lse_ref[r2]) * kLn2;
        }
        __syncwarp();
        cluster_sync();  // no CTA's shared memory goes away while another reads it
      }
    }
    tc_fence_before();
    __syncthreads();
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
  a.small_u = -1.f;
  if (L.softcap > 0.f) {
    const double k = (double)L.scale / L.softcap, cap2 = (double)L.softcap * kLog2e;
    const double least = std::fabs(tanh_small_coef(3)) * cap2 * std::pow(k, 7), most = std::fmax(cap2 * k, cap2 * std::pow(k, 7));
    if (least > 1e-36 && most < 1e36) a.small_u = kTanhSmall;
  }
  a.out = static_cast<__nv_bfloat16*>(L.out);
  a.lse = L.lse;
  a.status = L.status;
  a.wait_limit_ns = L.wait_limit_ns;
  a.drop_tile = L.drop_tile;
  // Paired CTAs (each an SM, a key tile fetched once for 256 queries) in whole waves of the SMs; what is
  // left, split into 128-row tiles, in clusters as large as the SMs and the key tiles allow. A rest
  // whose tiles would not fit one wave goes paired too: two waves of half the length each.
  const int sms = device_sm_count();
  const int64_t per_row = (L.T + kMaxRows - 1) / kMaxRows;  // pairs of a (sequence, head)
  const int64_t pairs = per_row * bh, over = pairs % sms;
  // 128-row tiles of the last `over` pairs: a chunk of an odd number of them leaves one a row out
  const int64_t over_tiles = 2 * over - ((L.T + kRows - 1) / kRows % 2 ? bh - (pairs - over) / per_row : 0);
  const int64_t whole = over_tiles > sms ? pairs : pairs - over, rest = pairs - whole;
  const int64_t keys = (L.cap + kRows - 1) / kRows + (L.n + kRows - 1) / kRows;  // at most, for a query tile
  const bool cap = L.softcap > 0.f, bias = L.slopes != nullptr;
  static unsigned long long done[8] = {};
  for (int split = 0; split < 2; ++split) {
    const int64_t units = split ? 2 * rest : whole;
    if (units == 0) continue;
    a.first = split ? (int)whole : 0;
    a.late = split && whole > 0 && pdl_enabled();
    a.cluster = 1;
    while (split && a.cluster < kMaxCluster && over_tiles * a.cluster * 2 <= sms && keys >= 4 * a.cluster) a.cluster *= 2;
    auto kernel = split ? (cap ? (bias ? scored_prefill_kernel<true, true, true> : scored_prefill_kernel<true, false, true>)
                               : (bias ? scored_prefill_kernel<false, true, true> : scored_prefill_kernel<false, false, true>))
                        : (cap ? (bias ? scored_prefill_kernel<true, true, false> : scored_prefill_kernel<true, false, false>)
                               : (bias ? scored_prefill_kernel<false, true, false> : scored_prefill_kernel<false, false, false>));
    const int which = 4 * split + 2 * cap + bias;
    const size_t smem = sizeof(Smem);
    if ((e = ensure_smem_limit(kernel, smem, &done[which])) != cudaSuccess) return e;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[2];
    fill_launch_config(cfg, attr, dim3((unsigned)(units * a.cluster)), dim3(kThreads), smem, stream);
    attr[cfg.numAttrs].id = cudaLaunchAttributeClusterDimension;
    attr[cfg.numAttrs].val.clusterDim.x = a.cluster;
    attr[cfg.numAttrs].val.clusterDim.y = attr[cfg.numAttrs].val.clusterDim.z = 1;
    ++cfg.numAttrs;
    if ((e = cudaLaunchKernelEx(&cfg, kernel, a, tq, tko, tvo, tpk, tpv, trk, trv)) != cudaSuccess) return e;
  }
  if (!L.write_ring) return cudaSuccess;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  fill_launch_config(cfg, attr, dim3(L.H, L.B), dim3(256), 0, stream);
  if ((e = cudaLaunchKernelEx(&cfg, ring_rows_kernel, L.H, L.n, L.T, static_cast<const uint4*>(L.k_out),
                              static_cast<const uint4*>(L.v_out), static_cast<uint4*>(L.ring_k_w),
                              static_cast<uint4*>(L.ring_v_w), L.wp, L.fill)) != cudaSuccess)
    return e;
  fill_launch_config(cfg, attr, dim3((L.B + 255) / 256), dim3(256), 0, stream);
  return cudaLaunchKernelEx(&cfg, ring_state_kernel, L.B, L.n, L.T, L.wp_w, L.fill_w);
}

}  // namespace rswa

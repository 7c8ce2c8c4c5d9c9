// balanced.cu -- single-token attention over each sequence's own rows (a range of its prefix,
// and its ring), cut evenly over the CTAs by the lengths found on the device.
//
// Two uses: scored decode, whose scores are capped by a tanh and biased by distance,
//   s = cap tanh(scale q.k / cap) - slope_h (pos_q - pos_k),
// over prefix rows [lo, hi) and the ring; and the private part of shared-prefix decode, which
// joins the records that the shared part left (shared.cu).
//
// HBM-bound: about one multiply-add per byte. The work of a call is a line of units, one unit a
// tile of up to 32 K/V rows of one (sequence, head); a sequence's heads and a head's tiles lie
// side by side. Every CTA sums the tile counts of all sequences (they are device values:
// prefix_len, ranges, fill), takes an equal share of the line and walks it, so a short document
// among long ones, or a range of 2,000 rows in a capacity of 100,000, leaves no CTA idle. A plan
// by the capacity (the plan of rswa_decode) would cut every sequence alike and leave the CTAs of
// its empty splits without work. Within a CTA unit i belongs to warp i mod 6, which streams it
// through its own 16 KiB shared-memory stage by bulk copies and issues the next unit's copy as
// soon as the stage is read, across (sequence, head) borders.
//
// A CTA's share can begin and end inside a (sequence, head): such a part leaves a record
// (max, sum, sum, accumulator) and the last CTA to finish one joins them; a CTA has at most two.
#include <cuda_bf16.h>

#include "balanced.h"
#include "common.cuh"
#include "internal.h"

namespace rswa {

namespace {

constexpr int kWarps = 6;
constexpr int kThreads = kWarps * 32;
constexpr int kTileBytes = kBlock * kRowBytes;  // 8 KiB
constexpr int kCtasPerSm = 2;                   // by shared memory
// The thresholds of the cut (where it is made says what they mean), with what the values beside
// them measured, in us:
constexpr int kSoloItems = 4;    // 1: 144 instead of 134 at 256 x 16 items of 416 rows; 16: 324 instead of 311 with 512 x 16
                                 // items of 128 rows over shared prefixes (but 184 instead of 190 at 512 x 16 of 288)
constexpr int kWholeItems = 3;   // 1: 64 instead of 55 at 37 x 12 ragged items of up to 2,099 rows; 12: 44 instead of 40 at
                                 // 64 x 16 items of 416 rows
constexpr int kWholeRounds = 3;  // 1: 9.9 instead of 8.0 at 16 items of 416 rows; 9: as 3
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// A sequence's rows: prefix rows [lo, hi) and the ring's valid slots in up to two runs.
struct SeqRows {
  int lo, hi;
  int a0, len0, len1;  // slots [a0, a0 + len0) and [0, len1)
  int wp;
  int n_pre, n_r0;
  int tiles;  // >= 1: a sequence without rows still owns one (empty) unit, which writes its output
};

struct BalancedSmem {
  uint8_t stage[kWarps][2][kTileBytes];
  uint64_t full[kWarps];
  float wm[kWarps], wl[kWarps], wlu[kWarps];
  float wacc[kWarps][kHeadDim];
  int scan[kWarps];
  int most[kWarps];
  SeqRows start_rows[kWarps];  // of the sequence that the team's share starts in,
  int start_b[kWarps];
  int start_base[kWarps];      // and the units before it
  int is_last;
};

// (Inputs are read through L2: with a shared part this launch starts while the one before it runs, so
// that no launch boundary has cleared what an L1 holds since the inputs were written.)
template <bool kScored>
__device__ __forceinline__ SeqRows rows_of(const BalancedArgs& a, int b, bool report) {
  SeqRows s;
  int m = a.cap > 0 ? __ldcg(a.prefix_len + b) : 0;
  if (m < 0 || m > a.cap) {
    if (report) set_status(a.status, RSWA_DEVICE_BAD_PREFIX_LEN);
    m = 0;
  }
  s.lo = 0;
  s.hi = m;
  if (kScored && a.ranges != nullptr) {
    const int2 r = __ldcg(a.ranges + b);
    if (r.x >= r.y) {
      s.hi = 0;
    } else if (r.x < 0 || r.y > m) {
      if (report) set_status(a.status, RSWA_DEVICE_BAD_RANGE);
      s.hi = 0;
    } else {
      s.lo = r.x;
      s.hi = r.y;
    }
  }
  if (kScored && a.slopes != nullptr) {
    const int p = __ldcg(a.pos + b);
    if (p < 0 || p > kMaxPos) {
      if (report) set_status(a.status, RSWA_DEVICE_BAD_POS);
      s.lo = s.hi = 0;
    }
  }
  int w = __ldcg(a.wp + b), f = __ldcg(a.fill + b);
  if (w < 0 || w >= a.n || f < 0 || f > a.n) {
    if (report) set_status(a.status, RSWA_DEVICE_BAD_RING_STATE);
    w = f = 0;
  }
  s.wp = w;
  s.a0 = f == a.n ? 0 : w - f;  // a full ring is one run
  if (s.a0 < 0) s.a0 += a.n;
  s.len0 = min(f, a.n - s.a0);
  s.len1 = f - s.len0;
  s.n_pre = (s.hi - s.lo + kBlock - 1) / kBlock;
  s.n_r0 = (s.len0 + kBlock - 1) / kBlock;
  s.tiles = max(1, s.n_pre + s.n_r0 + (s.len1 + kBlock - 1) / kBlock);
  return s;
}

// A team's share of the line: a CTA's, or with `solo` a warp's. Units [0, units) of it; with `whole` it
// is the items (the (sequence, head)s) that start there, to their ends.
struct Share {
  int units;
  bool whole, solo;
};

// One warp's place in its share: units [first, first + s.tiles) (first may be negative: the share
// starts inside) belong to (b, h).
struct Cursor {
  int b, h;
  int first;
  SeqRows s;
};

template <bool kScored>
__device__ __forceinline__ void advance(const BalancedArgs& a, Cursor& c) {
  c.first += c.s.tiles;
  if (++c.h == a.H) {
    c.h = 0;
    ++c.b;
    c.s = rows_of<kScored>(a, min(c.b, a.B - 1), false);
  }
}

struct Tile {
  int rows;  // 0: empty, nothing was copied
  bool armed;  // its copy was issued (all but the tile that a wait-timeout test drops)
  int row0;  // first prefix row (>= 0), or ~ of the first ring slot
};

// Issues unit u of the share (if it has it) into this warp's stage.
template <bool kScored>
__device__ __forceinline__ Tile issue(const BalancedArgs& a, BalancedSmem& sm, int u, const Share& share, Cursor& c,
                                      int warp, int lane) {
  Tile t;
  t.rows = 0;
  t.row0 = 0;
  t.armed = false;
  if (!share.whole && u >= share.units) return t;
  while (c.first < share.units && u >= c.first + c.s.tiles) advance<kScored>(a, c);
  if (c.first >= share.units) return t;
  int i = u - c.first;
  const int64_t bh = (int64_t)c.b * a.H + c.h;
  const uint16_t *k, *v;
  if (i < c.s.n_pre) {
    t.row0 = c.s.lo + i * kBlock;
    t.rows = min(kBlock, c.s.hi - t.row0);
    const int64_t off = (bh * a.cap + t.row0) * kHeadDim;
    k = a.pk + off;
    v = a.pv + off;
  } else {
    i -= c.s.n_pre;
    int slot, len;
    if (i < c.s.n_r0) {
      slot = c.s.a0 + i * kBlock;
      len = c.s.len0 - i * kBlock;
    } else {
      slot = (i - c.s.n_r0) * kBlock;
      len = c.s.len1 - slot;
    }
    t.row0 = ~slot;
    t.rows = max(0, min(kBlock, len));
    const int64_t off = (bh * a.n + slot) * kHeadDim;
    k = a.ring_k + off;
    v = a.ring_v + off;
  }
  // a wait-timeout test: CTA 0 neither arms nor fills the stage of its unit drop_tile
  if (a.drop_tile >= 0 && blockIdx.x == 0 && u == a.drop_tile) return t;
  t.armed = t.rows > 0;
  if (t.rows > 0 && lane == 0) {
    const uint32_t bytes = (uint32_t)t.rows * kRowBytes;
    mbar_arrive_expect_tx(&sm.full[warp], 2 * bytes);
    bulk_copy_g2s(sm.stage[warp][0], k, bytes, &sm.full[warp]);
    bulk_copy_g2s(sm.stage[warp][1], v, bytes, &sm.full[warp]);
  }
  return t;
}

__device__ __forceinline__ float2 bf16x2_f2(uint32_t w) { return make_float2(bf16lo(w), bf16hi(w)); }

// A (sequence, head)'s softmax state in one warp. In the tile loop lane (g, c) accumulates dims
// 8c..8c+7 of rows of parity g, l is per lane; after fold() every lane c holds dims 8c..8c+7 and
// l, lu are uniform. l weighs the accumulator, lu the log-sum-exp (they differ only for records of
// the tensor-core part, whose weights were rounded to bf16 before they met V).
struct State {
  float m, l, lu;
  float2 acc[4];
};

__device__ __forceinline__ void clear(State& s) {
  s.m = -INFINITY;
  s.l = s.lu = 0.f;
#pragma unroll
  for (int e = 0; e < 4; ++e) s.acc[e] = make_float2(0.f, 0.f);
}

// Scoring of an item in the log2 domain: dot (of the query scaled by qmul) -> score.
struct Score {
  float cap_log2;    // cap log2(e), or 0: no cap
  float slope_log2;  // slope log2(e)
  int ref;           // distance taken off every distance: the item's most favoured one
  int pos;
  int wp, n;
};

// Dots of the tile's 32 rows, reduce-scattered: lane (g, c) returns row 2c + g's.
__device__ __forceinline__ float tile_dots(const uint8_t* kt, const float2 (&q2)[4], int g, int c) {
  float pd[16];
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const uint4 w = *reinterpret_cast<const uint4*>(kt + (2 * j + g) * kRowBytes + c * 16);
    float2 d = __fmul2_rn(q2[0], bf16x2_f2(w.x));
    d = __ffma2_rn(q2[1], bf16x2_f2(w.y), d);
    d = __ffma2_rn(q2[2], bf16x2_f2(w.z), d);
    d = __ffma2_rn(q2[3], bf16x2_f2(w.w), d);
    pd[j] = d.x + d.y;
  }
#pragma unroll
  for (int half = 8; half > 0; half >>= 1) {
    const bool up = c & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float send = up ? pd[i] : pd[i + half];
      const float keep = up ? pd[i + half] : pd[i];
      pd[i] = keep + __shfl_xor_sync(0xffffffffu, send, half);
    }
  }
  return pd[0];
}

template <bool kScored, bool kFull>
__device__ __forceinline__ void consume(const uint8_t* kt, const uint8_t* vt, const Tile& t, const Score& sc,
                                        const float2 (&q2)[4], int g, int c, State& s) {
  float x = tile_dots(kt, q2, g, c);
  const int row = 2 * c + g;
  if (kScored) {
    if (sc.cap_log2 > 0.f) x = sc.cap_log2 * tanhf(x);
    int away;
    if (t.row0 >= 0) {
      away = sc.pos - (t.row0 + row);
    } else {  // a ring slot's age, counted back from the newest
      away = sc.wp - 1 - (~t.row0 + row);
      if (away < 0) away += sc.n;
    }
    x = fmaf(-sc.slope_log2, (float)(away - sc.ref), x);
  }
  if (!kFull && row >= t.rows) x = -INFINITY;
  const float m_new = fmaxf(s.m, warp_max(x));
  // a tile whose scores are all -inf (a -inf key row) leaves m at -inf: nothing to weigh yet
  const float base = m_new == -INFINITY ? 0.f : m_new;
  const float alpha = exp2f(s.m - base);
  const float p = exp2f(x - base);
  s.l = fmaf(s.l, alpha, p);
  const float2 a2 = make_float2(alpha, alpha);
#pragma unroll
  for (int e = 0; e < 4; ++e) s.acc[e] = __fmul2_rn(s.acc[e], a2);
  s.m = m_new;
#pragma unroll
  for (int j = 0; j < 16; ++j) {
    const float pj = __shfl_sync(0xffffffffu, p, (g << 4) | j);
    if (kFull || 2 * j + g < t.rows) {
      const uint4 w = *reinterpret_cast<const uint4*>(vt + (2 * j + g) * kRowBytes + c * 16);
      const float2 p2 = make_float2(pj, pj);
      s.acc[0] = __ffma2_rn(p2, bf16x2_f2(w.x), s.acc[0]);
      s.acc[1] = __ffma2_rn(p2, bf16x2_f2(w.y), s.acc[1]);
      s.acc[2] = __ffma2_rn(p2, bf16x2_f2(w.z), s.acc[2]);
      s.acc[3] = __ffma2_rn(p2, bf16x2_f2(w.w), s.acc[3]);
    }
  }
}

__device__ __forceinline__ void fold(State& s) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    s.acc[e].x += __shfl_xor_sync(0xffffffffu, s.acc[e].x, 16);
    s.acc[e].y += __shfl_xor_sync(0xffffffffu, s.acc[e].y, 16);
  }
  s.l = s.lu = warp_sum(s.l);
}

// Joins a record into a folded state.
__device__ __forceinline__ void join(State& s, const float* rec, int c) {
  const float4 head = __ldcg(reinterpret_cast<const float4*>(rec));
  if (head.x == -INFINITY && head.y == 0.f) return;  // nothing seen
  const float4 r0 = __ldcg(reinterpret_cast<const float4*>(rec + 4 + 8 * c));
  const float4 r1 = __ldcg(reinterpret_cast<const float4*>(rec + 8 + 8 * c));
  const float m = fmaxf(s.m, head.x);
  const float fs = exp2f(s.m - m), fr = exp2f(head.x - m);
  s.m = m;
  s.l = fmaf(s.l, fs, head.y * fr);
  s.lu = fmaf(s.lu, fs, head.z * fr);
  s.acc[0] = make_float2(fmaf(s.acc[0].x, fs, r0.x * fr), fmaf(s.acc[0].y, fs, r0.y * fr));
  s.acc[1] = make_float2(fmaf(s.acc[1].x, fs, r0.z * fr), fmaf(s.acc[1].y, fs, r0.w * fr));
  s.acc[2] = make_float2(fmaf(s.acc[2].x, fs, r1.x * fr), fmaf(s.acc[2].y, fs, r1.y * fr));
  s.acc[3] = make_float2(fmaf(s.acc[3].x, fs, r1.z * fr), fmaf(s.acc[3].y, fs, r1.w * fr));
}

// The records that the shared part left for (b, h): one for each CTA that had a run of its keys.
struct SharedRecords {
  int count;
  const float* first;  // the run that holds the first key tile
  const float* next;   // the others, kSharedRows records apart
  __device__ __forceinline__ const float* at(int r) const {
    return r == 0 ? first : next + (int64_t)(r - 1) * kSharedRows * kRecordFloats;
  }
};

__device__ __forceinline__ SharedRecords shared_records(const BalancedArgs& a, const SharedSeq& t, int per, int h) {
  SharedRecords r;
  r.count = 0;
  r.first = r.next = nullptr;
  if (t.row < 0) return r;
  const int u = t.first_unit + h * t.key_tiles;
  const int c0 = u / per, c1 = (u + t.key_tiles - 1) / per;
  r.count = c1 - c0 + 1;
  r.first = a.shared.records + ((int64_t)t.first_seq * a.H + (int64_t)h * t.rows + t.row) * kRecordFloats;
  r.next = a.shared.records + ((int64_t)a.B * a.H + (int64_t)(c0 + 1) * kSharedRows + t.row) * kRecordFloats;
  return r;
}

template <bool kScored, bool kShared>
__global__ void __launch_bounds__(kThreads, kCtasPerSm) balanced_kernel(const __grid_constant__ BalancedArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  BalancedSmem& sm = *reinterpret_cast<BalancedSmem*>(smem_raw);
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int g = lane >> 4, c = lane & 15;
  if (tid == 0) {
    for (int s = 0; s < kWarps; ++s) mbar_init(&sm.full[s], 1);
    fence_mbar_init();
  }
  // With a shared part, its launch is the one before: its records are waited for where they are
  // joined, and until then this launch runs beside it (on the SMs that it leaves free, or leaves).
  // What came before the shared part has ended: this launch started after all CTAs of that one had
  // waited for it.
  if (!kShared) griddep_wait();
  griddep_launch_dependents();

  // ---- this CTA's share of the line of units (fewer than 2^31, as the entry points see to) ----
  const int per_thread = (a.B + kThreads - 1) / kThreads;
  const int b0 = min(a.B, tid * per_thread), b1 = min(a.B, b0 + per_thread);
  int mine = 0;
  int most = 0;  // tiles of the longest item
  SeqRows rows0;  // of sequence b0
  for (int b = b0; b < b1; ++b) {
    const SeqRows r = rows_of<kScored>(a, b, blockIdx.x == 0);
    if (b == b0) rows0 = r;
    mine += r.tiles;
    most = max(most, r.tiles);
  }
  most = __reduce_max_sync(0xffffffffu, most);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int t = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += t;
  }
  if (lane == 31) {
    sm.scan[warp] = inc;
    sm.most[warp] = most;
  }
  __syncthreads();
  int before = inc - mine, total = 0;
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    before += w < warp ? sm.scan[w] : 0;
    total += sm.scan[w];
    most = max(most, sm.most[w]);
  }
  before *= a.H;
  mine *= a.H;
  total *= a.H;
  // How the line is cut. Items that are short against a share go whole: to a warp each where every
  // warp gets at least kSoloItems of them (no barrier at an item's end, next to no imbalance), to a CTA
  // where a CTA gets that many, and, where there are no more items than CTAs, one to a CTA as long
  // as it is done in a few rounds of the six warps (records to join cost more). Else shares cut
  // through items.
  const int grid = gridDim.x;
  int per = (total - 1) / grid + 1;
  Share share;
  share.solo = per >= kSoloItems * kWarps * most;
  share.whole = share.solo || per >= kWholeItems * most || (per <= most && most <= kWholeRounds * kWarps);
  if (share.solo)
    per = (total - 1) / (grid * kWarps) + 1;
  else
    per = max(per, share.whole ? most : kWarps);  // fewer units than warps: idle warps, more records
  const int step = share.solo ? 1 : kWarps;
  const int slot = share.solo ? warp : 0;  // this warp's team in the CTA
  const int team0 = (int)blockIdx.x * (share.solo ? kWarps : 1);
  for (int w = 0; w < (share.solo ? kWarps : 1); ++w) {
    const int64_t u = (int64_t)(team0 + w) * per;
    if (mine > 0 && u >= before && u < (int64_t)before + mine) {
      int base = before, b = b0;
      SeqRows r = rows0;
      while (u >= base + r.tiles * a.H) {
        base += r.tiles * a.H;
        r = rows_of<kScored>(a, ++b, false);
      }
      sm.start_rows[w] = r;
      sm.start_b[w] = b;
      sm.start_base[w] = base;
    }
  }
  __syncthreads();
  if ((int64_t)(team0 + slot) * per >= total) return;  // a whole team: no barrier follows for it
  const int u0 = (team0 + slot) * per;
  share.units = min(per, total - u0);

  Cursor ahead;  // where this warp issues copies
  ahead.b = sm.start_b[slot];
  ahead.s = sm.start_rows[slot];
  ahead.h = (u0 - sm.start_base[slot]) / ahead.s.tiles;
  ahead.first = sm.start_base[slot] + ahead.h * ahead.s.tiles - u0;
  if (share.whole && ahead.first < 0) {  // that item is another team's
    if (u0 + ahead.first + ahead.s.tiles >= total) return;
    advance<kScored>(a, ahead);
    if (ahead.first >= share.units) return;
  }
  Cursor at = ahead;  // the (sequence, head) being read
  int u = at.first > 0 ? at.first : 0;  // with `whole`, units before its first item are another team's
  u += share.solo ? 0 : warp;
  Tile tile = issue<kScored>(a, sm, u, share, ahead, warp, lane);
  SharedSeq seq;
  int seq_b = -1, shared_per = 1;
  uint4 q_next = __ldcg(reinterpret_cast<const uint4*>(a.q + ((int64_t)at.b * a.H + at.h) * kHeadDim + c * 8));
  uint32_t phase = 0;
  bool ok = true;

  while (true) {
    const int end = share.whole ? at.first + at.s.tiles : min(share.units, at.first + at.s.tiles);
    const int64_t bh = (int64_t)at.b * a.H + at.h;
    Score sc;
    sc.cap_log2 = sc.slope_log2 = 0.f;
    sc.ref = sc.pos = sc.wp = sc.n = 0;
    float qmul = a.scale * kLog2e;
    if (kScored) {
      if (a.softcap > 0.f) {
        qmul = a.scale / a.softcap;
        sc.cap_log2 = a.softcap * kLog2e;
      }
      sc.wp = at.s.wp;
      sc.n = a.n;
      if (a.slopes != nullptr) {
        const float slope = __ldcg(a.slopes + at.h);
        sc.slope_log2 = slope * kLog2e;
        sc.pos = __ldcg(a.pos + at.b);
        // distances are taken from the favoured end of the rows seen, an integer, so that far
        // documents keep the bias small where it counts; the log-sum-exp adds it back
        const int ring = at.s.len0 + at.s.len1;
        const bool pre = at.s.hi > at.s.lo;
        if (slope >= 0.f)
          sc.ref = ring > 0 ? (pre ? min(0, sc.pos - (at.s.hi - 1)) : 0) : (pre ? sc.pos - (at.s.hi - 1) : 0);
        else
          sc.ref = ring > 0 ? (pre ? max(ring - 1, sc.pos - at.s.lo) : ring - 1) : (pre ? sc.pos - at.s.lo : 0);
      }
    }
    float2 q2[4];
    {
      const uint32_t ws[4] = {q_next.x, q_next.y, q_next.z, q_next.w};
#pragma unroll
      for (int e = 0; e < 4; ++e) q2[e] = make_float2(bf16lo(ws[e]) * qmul, bf16hi(ws[e]) * qmul);
    }
    if (bh + 1 < (int64_t)a.B * a.H)  // the next item's query, while this one streams
      q_next = __ldcg(reinterpret_cast<const uint4*>(a.q + (bh + 1) * kHeadDim + c * 8));
    State st;
    clear(st);
    for (; ok && u < end; u += step) {
      const Tile cur = tile;
      if (cur.rows > 0) {
        if (!__all_sync(0xffffffffu, mbar_wait(&sm.full[warp], phase, a.wait_limit_ns))) {
          if (lane == 0) set_status(a.status, RSWA_DEVICE_WAIT_TIMEOUT);
          ok = false;
          break;
        }
        phase ^= 1;
        if (cur.rows == kBlock)
          consume<kScored, true>(sm.stage[warp][0], sm.stage[warp][1], cur, sc, q2, g, c, st);
        else
          consume<kScored, false>(sm.stage[warp][0], sm.stage[warp][1], cur, sc, q2, g, c, st);
      }
      __syncwarp();  // every lane has read the stage before it is filled again
      tile = issue<kScored>(a, sm, u + step, share, ahead, warp, lane);
    }
    fold(st);
    const bool starts = at.first >= 0, ends = share.whole || at.first + at.s.tiles <= share.units;
    SharedRecords sr;
    sr.count = 0;
    if (kShared) {
      if (seq_b < 0) {  // the first item: the shared part has to be done now
        griddep_wait();
        shared_per = a.shared.head->per;
      }
      if (seq_b != at.b) {
        seq = a.shared.seqs[at.b];
        seq_b = at.b;
      }
      sr = shared_records(a, seq, shared_per, at.h);
      if (starts && ends)  // the whole item is here: the shared part's records join its warps
        for (int r = share.solo ? 0 : warp; r < sr.count; r += step) join(st, sr.at(r), c);
    }

    if (share.solo) {
      if (g == 0 && ok) {
        const float inv = st.l == 0.f ? 0.f : 1.f / st.l;  // no row seen: zero (a NaN sum stays one)
        float o[8];
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[2 * e] = st.acc[e].x * inv;
          o[2 * e + 1] = st.acc[e].y * inv;
        }
        if (kShared) {
          uint32_t w[4];
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const __nv_bfloat162 o2 = __floats2bfloat162_rn(o[2 * e], o[2 * e + 1]);
            w[e] = *reinterpret_cast<const uint32_t*>(&o2);
          }
          reinterpret_cast<uint4*>(a.out)[bh * (kHeadDim / 8) + c] = make_uint4(w[0], w[1], w[2], w[3]);
        } else {
          float4* out = reinterpret_cast<float4*>(a.out) + bh * (kHeadDim / 4) + 2 * c;
          out[0] = make_float4(o[0], o[1], o[2], o[3]);
          out[1] = make_float4(o[4], o[5], o[6], o[7]);
        }
        if (c == 0 && a.lse)
          a.lse[bh] = st.lu == 0.f ? -INFINITY : (st.m + log2f(st.lu) - sc.slope_log2 * (float)sc.ref) * kLn2;
      }
      if (!ok || end >= share.units) break;
      advance<kScored>(a, at);
      continue;
    }

    // ---- the warps' states meet; `joined` says that st holds records of the whole item ----
    for (bool joined = starts && ends;; joined = true) {
      if (g == 0) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          sm.wacc[warp][c * 8 + 2 * e] = st.acc[e].x;
          sm.wacc[warp][c * 8 + 2 * e + 1] = st.acc[e].y;
        }
      }
      if (lane == 0) {
        sm.wm[warp] = st.m;
        sm.wl[warp] = st.l;
        sm.wlu[warp] = st.lu;
      }
      __syncthreads();
      float M = -INFINITY;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) M = fmaxf(M, sm.wm[w]);
      float fw[kWarps], L = 0.f, LU = 0.f;
#pragma unroll
      for (int w = 0; w < kWarps; ++w) {
        fw[w] = M > -INFINITY ? exp2f(sm.wm[w] - M) : 0.f;
        L = fmaf(sm.wl[w], fw[w], L);
        LU = fmaf(sm.wlu[w], fw[w], LU);
      }
      float A = 0.f;
      if (tid < kHeadDim) {
#pragma unroll
        for (int w = 0; w < kWarps; ++w) A = fmaf(sm.wacc[w][tid], fw[w], A);
      }
      if (joined) {
        if (tid < kHeadDim) {
          const float o = L == 0.f ? 0.f : A / L;  // no row seen: zero (a NaN sum stays one)
          if (kShared)
            static_cast<__nv_bfloat16*>(a.out)[bh * kHeadDim + tid] = __float2bfloat16_rn(o);
          else
            static_cast<float*>(a.out)[bh * kHeadDim + tid] = o;
        }
        if (tid == 0 && a.lse)
          a.lse[bh] = LU == 0.f ? -INFINITY : (M + log2f(LU) - sc.slope_log2 * (float)sc.ref) * kLn2;
        break;
      }
      float* rec = a.records + (int64_t)(2 * blockIdx.x + (starts ? 1 : 0)) * kRecordFloats;
      if (tid < kHeadDim) rec[4 + tid] = A;
      if (tid == 0) {
        rec[0] = M;
        rec[1] = L;
        rec[2] = LU;
      }
      __threadfence();
      __syncthreads();
      // CTAs c0..c1 hold a part of this item; c0, where it starts, keeps its counter
      const int s0 = u0 + at.first, c0 = s0 / per, c1 = (s0 + at.s.tiles - 1) / per;
      if (tid == 0) sm.is_last = atomicAdd(&a.counters[c0], 1) == c1 - c0;
      __syncthreads();
      if (!sm.is_last) break;
      __threadfence();
      if (tid == 0) a.counters[c0] = 0;
      clear(st);
      for (int r = warp; r <= c1 - c0 + sr.count; r += kWarps) {
        const int k = r - (c1 - c0 + 1);
        join(st, k < 0 ? a.records + (int64_t)(2 * (c0 + r) + (r == 0 ? 1 : 0)) * kRecordFloats : sr.at(k), c);
      }
    }
    // the merge buffers are written again by the next item; a warp that gave up ends the CTA
    if (__syncthreads_or(!ok) || !ends || end >= share.units) break;
    advance<kScored>(a, at);
  }
  // after a give-up, this warp's or another's of its CTA, the copy issued last may be in flight: let it
  // land (bounded) before the shared memory goes away (after a normal end none is)
  if (tile.armed) mbar_wait(&sm.full[warp], phase, a.wait_limit_ns);
}

}  // namespace

int balanced_grid() { return device_sm_count() * kCtasPerSm; }

size_t balanced_scratch_bytes() {
  const size_t grid = (size_t)balanced_grid();
  return (grid * 4 + 255) / 256 * 256 + grid * 2 * kRecordFloats * 4;
}

cudaError_t launch_balanced(BalancedArgs a, void* scratch, cudaStream_t stream) {
  static unsigned long long done[2] = {};
  const int grid = balanced_grid();
  a.counters = static_cast<int32_t*>(scratch);
  a.records = reinterpret_cast<float*>(static_cast<uint8_t*>(scratch) + ((size_t)grid * 4 + 255) / 256 * 256);
  const bool shared = a.shared.head != nullptr;
  auto kernel = shared ? balanced_kernel<false, true> : balanced_kernel<true, false>;
  cudaError_t e = ensure_smem_limit(kernel, sizeof(BalancedSmem), &done[shared ? 1 : 0]);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  fill_launch_config(cfg, attr, dim3(grid), dim3(kThreads), sizeof(BalancedSmem), stream);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace rswa

// rope1d.cu -- rotary position encoding with one position per token.
//
// Pair i of a head's first rot dims turns by pos * inv_freq[i]; the dims from rot on pass
// through. "Half" pairs are dims (i, i + rot/2), "interleaved" ones dims (2i, 2i + 1). With
// (c, s) = mscale (cos, sin) of the angle a pair (x, y) becomes (x c - y s, y c + x s); the
// transpose, which turns gradients back, is the same with -s.
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: the host gives
// frac(inv_freq / 2 pi) * 2^64 (its lowest bit 0), the kernel multiplies by the integer position
// modulo 2^64 (whole turns fall off the top) and keeps the 32 leading bits: exact to
// |pos| * 2^-63 + 2^-32 turns for every int32 position without fp64 arithmetic, whose rate
// on this chip would bound the kernel (the page2d kernel's fp64 sincos is its second cost).
// The 32 bits are rounded to f32 (by at most 2^-26 turns) for sincospif, of f32 rows; of bf16
// rows they are taken times 2 pi / 2^32 (3.1e-7 in all, at most) for __sincosf.
//
// HBM-bound: every element is read once and written once. A warp takes the rows of a few
// consecutive tokens (four at 128 bf16 dims: 1 KiB runs) in up to 8 heads, four heads at a time in
// flight; a lane keeps its place in the row, so that the cos and sin of its pairs stay in its registers
// for all heads, with no table and no barrier (a CTA-wide table in shared memory, filled behind the loads
// of 4 or 16 tokens, measured 77 to 90 us where this takes 42, as a plain copy does: the loads waited for it).
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace rswa {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;       // heads of a row in flight
constexpr int kMaxHeads = 8;    // heads of a warp
constexpr int kMaxPairs = 128;  // rot <= 256

struct RowStrides {
  int64_t b, h, t;  // elements
};

struct Rope1dArgs {
  int64_t rows;  // batch * tokens
  int T, Hq, H;  // H = Hq + Hk
  int units;     // D / (2 vectors): units of one row
  int rot_units; // of them rotated
  int half;      // rot / 2
  int tokens;    // of a warp: 32 / units
  int heads;     // of a warp
  int copy;      // the dims past rot have to be copied (not in place)
  const void* q;
  void* q_out;
  const void* k;
  void* k_out;
  RowStrides qs, qos, ks, kos;
  const int32_t* pos;
  float mscale, sign;
  uint64_t turns[kMaxPairs];
};

template <typename E>
struct Vec;  // 16 bytes of E as floats
template <>
struct Vec<uint16_t> {
  static constexpr int kN = 8;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = bf16lo(w[i]);
      f[2 * i + 1] = bf16hi(w[i]);
    }
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec<float> {
  static constexpr int kN = 4;
  static __device__ __forceinline__ void get(const uint4& v, float (&f)[4]) {
    f[0] = __uint_as_float(v.x), f[1] = __uint_as_float(v.y), f[2] = __uint_as_float(v.z), f[3] = __uint_as_float(v.w);
  }
  static __device__ __forceinline__ uint4 put(const float (&f)[4]) {
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
  }
};

// Rotates the unit's two vectors: half layout: x's of N pairs, then their y's; interleaved:
// N / 2 pairs in each vector. cs: the unit's N pairs.
template <typename E, bool kInterleaved>
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2 (&cs)[Vec<E>::kN]) {
  constexpr int N = Vec<E>::kN;
  float x[N], y[N];
  Vec<E>::get(a, x);
  Vec<E>::get(b, y);
  if (kInterleaved) {
#pragma unroll
    for (int i = 0; i < N; i += 2) {
      const float2 c0 = cs[i / 2], c1 = cs[N / 2 + i / 2];
      const float x0 = x[i], y0 = y[i];
      x[i] = fmaf(x0, c0.x, -x[i + 1] * c0.y);
      x[i + 1] = fmaf(x[i + 1], c0.x, x0 * c0.y);
      y[i] = fmaf(y0, c1.x, -y[i + 1] * c1.y);
      y[i + 1] = fmaf(y[i + 1], c1.x, y0 * c1.y);
    }
  } else {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float2 c = cs[i];
      const float x0 = x[i];
      x[i] = fmaf(x0, c.x, -y[i] * c.y);
      y[i] = fmaf(y[i], c.x, x0 * c.y);
    }
  }
  a = Vec<E>::put(x);
  b = Vec<E>::put(y);
}

template <typename E, bool kInterleaved>
__global__ void __launch_bounds__(kThreads, 3) rope1d_kernel(const __grid_constant__ Rope1dArgs a) {
  constexpr int N = Vec<E>::kN;
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int64_t group = (int64_t)blockIdx.x * (blockDim.x >> 5) + (threadIdx.x >> 5);
  // this lane's unit c of the rows of token r
  const int g = lane / a.units, c = lane - g * a.units;
  const int64_t r = group * a.tokens + g;
  const bool turned = c < a.rot_units;
  if (g >= a.tokens || r >= a.rows || !(turned || a.copy)) return;
  const int first = (turned && !kInterleaved) ? c * N : 2 * c * N;
  const int second = (turned && !kInterleaved) ? a.half : N;  // from the first vector to the second
  const int pos = a.pos[r];
  int64_t b;
  if (a.rows <= 0x7fffffff)
    b = (unsigned)r / (unsigned)a.T;
  else
    b = r / a.T;
  const int64_t t = r - b * a.T;
  const E* q = static_cast<const E*>(a.q) + b * a.qs.b + t * a.qs.t + first;
  E* q_out = static_cast<E*>(a.q_out) + b * a.qos.b + t * a.qos.t + first;
  const E* k = static_cast<const E*>(a.k) + b * a.ks.b + t * a.ks.t + first - a.Hq * a.ks.h;
  E* k_out = static_cast<E*>(a.k_out) + b * a.kos.b + t * a.kos.t + first - a.Hq * a.kos.h;
  const int h0 = blockIdx.y * a.heads, h1 = min(h0 + a.heads, a.H);
  float2 cs[N];
  for (int hb = h0; hb < h1; hb += kBatch) {
    uint4 va[kBatch], vb[kBatch];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h < h1) {
        const E* src = h < a.Hq ? q + h * a.qs.h : k + h * a.ks.h;
        va[j] = *reinterpret_cast<const uint4*>(src);
        vb[j] = *reinterpret_cast<const uint4*>(src + second);
      }
    }
    if (hb == h0 && turned) {  // this lane's cos / sin, while its loads are in flight
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const uint64_t turn = (uint64_t)(int64_t)pos * a.turns[c * N + i];
        const float part = (float)(int32_t)(turn >> 32);  // of a turn, times 2^32: half a turn either way
        float s, co;
        if (sizeof(E) == 2)  // its own error is at most 2^-21.2 up to pi, far below a bf16 step
          __sincosf(part * 1.4629180792671596e-9f, &s, &co);  // 2 pi / 2^32
        else
          sincospif(part * 4.656612873077393e-10f, &s, &co);  // 2^-31
        cs[i] = make_float2(co * a.mscale, s * a.sign);
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int h = hb + j;
      if (h < h1) {
        if (turned) rotate<E, kInterleaved>(va[j], vb[j], cs);
        E* dst = h < a.Hq ? q_out + h * a.qos.h : k_out + h * a.kos.h;
        *reinterpret_cast<uint4*>(dst) = va[j];
        *reinterpret_cast<uint4*>(dst + second) = vb[j];
      }
    }
  }
}

}  // namespace

cudaError_t launch_rope1d(const Rope1dLaunch& L, cudaStream_t stream) {
  Rope1dArgs a;
  const int vec = L.f32 ? 4 : 8;
  a.rows = (int64_t)L.B * L.T;
  a.T = L.T;
  a.Hq = L.Hq;
  a.H = L.Hq + L.Hk;
  a.units = L.D / (2 * vec);
  a.rot_units = L.rot / (2 * vec);
  a.half = L.rot / 2;
  a.copy = L.copy_rest;
  a.q = L.q;
  a.q_out = L.q_out;
  a.k = L.k;
  a.k_out = L.k_out;
  auto strides = [](const int64_t* s) { return RowStrides{s[0], s[1], s[2]}; };
  a.qs = strides(L.q_stride);
  a.qos = strides(L.q_out_stride);
  a.ks = strides(L.k_stride);
  a.kos = strides(L.k_out_stride);
  a.pos = L.pos;
  a.mscale = L.mscale;
  a.sign = L.inverse ? -L.mscale : L.mscale;
  for (int i = 0; i < a.half; ++i) a.turns[i] = L.turns[i];
  a.tokens = 32 / a.units;
  // few rows: fewer heads a warp and smaller CTAs, until every SM has one
  const int sms = device_sm_count();
  const int64_t groups = (a.rows + a.tokens - 1) / a.tokens;
  a.heads = a.H < kMaxHeads ? a.H : kMaxHeads;
  int warps = kThreads / 32;
  auto ctas = [&]() { return (groups + warps - 1) / warps * ((a.H + a.heads - 1) / a.heads); };
  while (a.heads > kBatch && ctas() < 4 * sms) a.heads = (a.heads + 1) / 2;
  while (warps > 1 && ctas() < sms) warps /= 2;
  while (a.heads > 1 && ctas() < sms) a.heads = (a.heads + 1) / 2;
  if ((groups + warps - 1) / warps > 0x7fffffff) return cudaErrorInvalidValue;
  const dim3 grid((unsigned)((groups + warps - 1) / warps), (a.H + a.heads - 1) / a.heads);
  auto kernel = L.f32 ? (L.interleaved ? rope1d_kernel<float, true> : rope1d_kernel<float, false>)
                      : (L.interleaved ? rope1d_kernel<uint16_t, true> : rope1d_kernel<uint16_t, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  fill_launch_config(cfg, attr, grid, dim3(warps * 32), 0, stream);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace rswa

// rope1d.cu -- rotary position encoding with one position per token.
//
// Pair i of a head's first rot dims turns by pos * inv_freq[i]; the dims from rot on pass
// through. "Half" pairs are dims (i, i + rot/2), "interleaved" ones dims (2i, 2i + 1). With
// (c, s) = mscale (cos, sin) of the angle a pair (x, y) becomes (x c - y s, y c + x s); the
// transpose, which turns gradients back, is the same with -s.
//
// The angle is kept as a fraction of a turn in 64-bit fixed point: the host gives
// frac(inv_freq / 2 pi) * 2^64, the kernel multiplies by the integer position modulo 2^64
// (whole turns fall off the top), and the 32 leading bits go to sincospif. That is exact to
// |pos| * 2^-65 + 2^-32 turns for every int32 position without fp64 arithmetic, whose rate
// on this chip would bound the kernel (the page2d kernel's fp64 sincos is its second cost).
//
// HBM-bound: every element is read once and written once. A CTA takes a group of tokens and
// all their heads, so that one table of cos / sin serves every head; a thread holds up to
// four units (two 16-byte vectors each) in flight while the CTA fills the table.
#include <cuda_bf16.h>

#include "common.cuh"
#include "internal.h"

namespace rswa {

namespace {

constexpr int kThreads = 256;
constexpr int kUnits = 4;       // units a thread holds per pass
constexpr int kMaxGroup = 16;   // tokens per CTA
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
  int group;
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
__device__ __forceinline__ void rotate(uint4& a, uint4& b, const float2* cs) {
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
__global__ void __launch_bounds__(kThreads) rope1d_kernel(const __grid_constant__ Rope1dArgs a) {
  constexpr int N = Vec<E>::kN;
  __shared__ float2 cs[kMaxGroup * kMaxPairs];
  __shared__ int2 at[kMaxGroup];  // (sequence, token) of each row of the group
  griddep_wait();
  griddep_launch_dependents();
  const int64_t r0 = (int64_t)blockIdx.x * a.group;
  const int g_rows = (int)min((int64_t)a.group, a.rows - r0);
  if ((int)threadIdx.x < g_rows) {
    const int64_t r = r0 + threadIdx.x;
    const int b = (int)(r / a.T);
    at[threadIdx.x] = make_int2(b, (int)(r - (int64_t)b * a.T));
  }
  __syncthreads();
  const int per_head = g_rows * a.units;
  const int total = per_head * a.H;
  for (int u0 = 0; u0 < total; u0 += kUnits * kThreads) {
    uint4 va[kUnits], vb[kUnits];
    E* dst[kUnits];
    int ci[kUnits];
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      const int u = u0 + j * kThreads + (int)threadIdx.x;
      dst[j] = nullptr;
      ci[j] = 0;
      if (u >= total) continue;
      // consecutive threads walk a head's rows of consecutive tokens
      const int h = u / per_head, rem = u - h * per_head;
      const int g = rem / a.units, c = rem - g * a.units;
      const bool turned = c < a.rot_units;
      if (!turned && !a.copy) continue;
      const int2 bt = at[g];
      const bool is_q = h < a.Hq;
      const int hh = is_q ? h : h - a.Hq;
      const RowStrides& si = is_q ? a.qs : a.ks;
      const RowStrides& so = is_q ? a.qos : a.kos;
      const E* src = static_cast<const E*>(is_q ? a.q : a.k) + bt.x * si.b + hh * si.h + bt.y * si.t;
      const int first = (turned && !kInterleaved) ? c * N : 2 * c * N;
      const int second = (turned && !kInterleaved) ? a.half + c * N : first + N;
      va[j] = *reinterpret_cast<const uint4*>(src + first);
      vb[j] = *reinterpret_cast<const uint4*>(src + second);
      dst[j] = static_cast<E*>(is_q ? a.q_out : a.k_out) + bt.x * so.b + hh * so.h + bt.y * so.t + first;
      ci[j] = turned ? g * a.half + c * N : -1;
    }
    if (u0 == 0) {  // the group's cos / sin, while its loads are in flight
      for (int p = threadIdx.x; p < g_rows * a.half; p += kThreads) {
        const int g = p / a.half, i = p - g * a.half;
        const uint64_t turn = (uint64_t)(int64_t)a.pos[r0 + g] * a.turns[i];
        float s, c;
        sincospif((float)(int32_t)(turn >> 32) * 4.656612873077393e-10f, &s, &c);  // 2^-31 half turns
        cs[p] = make_float2(c * a.mscale, s * a.sign);
      }
      __syncthreads();
    }
#pragma unroll
    for (int j = 0; j < kUnits; ++j) {
      if (dst[j] == nullptr) continue;
      int second = N;
      if (ci[j] >= 0) {
        rotate<E, kInterleaved>(va[j], vb[j], cs + ci[j]);
        if (!kInterleaved) second = a.half;
      }
      *reinterpret_cast<uint4*>(dst[j]) = va[j];
      *reinterpret_cast<uint4*>(dst[j] + second) = vb[j];
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
  // tokens of a CTA: one pass of four units a thread where the rows are few enough
  const int per_row = a.H * a.units;
  int group = kUnits * kThreads / per_row;
  group = group < 1 ? 1 : (group > kMaxGroup ? kMaxGroup : group);
  // a call of few tokens is spread over the SMs instead
  while (group > 1 && (a.rows + group - 1) / group < device_sm_count()) --group;
  a.group = group;
  const int64_t grid = (a.rows + group - 1) / group;
  if (grid > 0x7fffffff) return cudaErrorInvalidValue;
  auto kernel = L.f32 ? (L.interleaved ? rope1d_kernel<float, true> : rope1d_kernel<float, false>)
                      : (L.interleaved ? rope1d_kernel<uint16_t, true> : rope1d_kernel<uint16_t, false>);
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  fill_launch_config(cfg, attr, dim3((unsigned)grid), dim3(kThreads), 0, stream);
  return cudaLaunchKernelEx(&cfg, kernel, a);
}

}  // namespace rswa

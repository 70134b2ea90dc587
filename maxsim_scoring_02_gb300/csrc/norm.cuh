// norm.cuh -- what both directions of the root-mean-square norm share: their
// parameters, a team's sums, and the row's statistics.
#pragma once

#include "rows.cuh"

namespace msim {

struct NormParams {
  const void *x, *res;  // forward: x and the residual; backward: dy and h
  const void* more;     // backward: the gradient that reaches the sum from elsewhere, or null
  const void* weight;   // or null
  void *sum, *out;      // forward: sum, result; backward: the residual's gradient, dx
  float* scale;         // of 8-bit rows
  float* parts;         // backward: [blocks, d] partial sums of the weight's gradient, or null
  int64_t x_stride, res_stride, more_stride, sum_stride, out_stride;
  int T, d, weight_fp32, format;
  float eps;
  Drop drop;
};

// Sums of two values over a team of kTeam threads: parts of a warp by shuffles, a
// block's warps through shared memory, added in the same order by every thread.
// `at` alternates between calls, so that one barrier a call is enough.
template <int kTeam, typename V, typename Op>
__device__ __forceinline__ void team_all(V& a, V& b, Op op, int at) {
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o; o >>= 1) op(a, b, __shfl_xor_sync(~0u, a, o), __shfl_xor_sync(~0u, b, o));
  if constexpr (kTeam > 32) {
    __shared__ V s[2][kTeam / 32][2];
    if ((threadIdx.x & 31) == 0) s[at][threadIdx.x >> 5][0] = a, s[at][threadIdx.x >> 5][1] = b;
    __syncthreads();
    a = s[at][0][0], b = s[at][0][1];
#pragma unroll
    for (int w = 1; w < kTeam / 32; ++w) op(a, b, s[at][w][0], s[at][w][1]);
  }
}

// Whether a flag that a team's threads agree on is set for a team of this warp:
// what follows is then done by whole warps.
template <int kTeam>
__device__ __forceinline__ bool any_of_team(bool flag) {
  if constexpr (kTeam < 32) return __any_sync(~0u, flag);
  return flag;
}

struct AddBoth {
  template <typename V>
  __device__ __forceinline__ void operator()(V& a, V& b, V c, V d) const { a += c, b += d; }
};
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
struct AddAndMax {
  __device__ __forceinline__ void operator()(float& a, float& b, float c, float d) const { a += c, b = max_nan(b, d); }
};

// Eight weights of the thread's columns.
template <typename T, bool kWhole>
__device__ __forceinline__ void load_weights(const NormParams& p, const Cols<kWhole>& c, float (&w)[8]) {
  if (!p.weight) {
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = 1.f;
  } else if (p.weight_fp32) {
    alignas(16) float v[8];
    load8<float, kWhole>(static_cast<const float*>(p.weight), c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = v[j];
  } else {
    alignas(16) T v[8];
    load8<T, kWhole>(static_cast<const T*>(p.weight), c, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = up(v[j]);
  }
}

constexpr int kMaxNormWidth = 16384;

}  // namespace msim

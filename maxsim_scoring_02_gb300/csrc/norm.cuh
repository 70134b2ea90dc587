// norm.cuh -- what both directions of the root-mean-square norm share: their
// parameters, a team's sums, and the row's statistics.
#pragma once

#include "ptx.cuh"
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
  float per;            // 1 / d
  float eps;
  Drop drop;
};

// Two values of all threads of a team joined: a warp's by shuffles, a block's warps'
// through shared memory, in the same order by every thread. `at` alternates between
// calls, so that one barrier a call is enough.
template <int kTeam, typename V, typename Op>
__device__ __forceinline__ void team_all(V& a, V& b, Op op, int at) {
#pragma unroll
  for (int o = (kTeam < 32 ? kTeam : 32) / 2; o; o >>= 1) op(a, b, __shfl_xor_sync(~0u, a, o), __shfl_xor_sync(~0u, b, o));
  if constexpr (kTeam > 32) {
    __shared__ alignas(16) V s[2][kTeam / 32][2];
    if ((threadIdx.x & 31) == 0) s[at][threadIdx.x >> 5][0] = a, s[at][threadIdx.x >> 5][1] = b;
    __syncthreads();
    if constexpr (kTeam <= 256 && sizeof(V) == 4) {
      const float4* v = reinterpret_cast<const float4*>(s[at]);
      float4 q = v[0];
      a = q.x, b = q.y;
      op(a, b, q.z, q.w);
#pragma unroll
      for (int w = 1; w < kTeam / 64; ++w) {
        q = v[w];
        op(a, b, q.x, q.y);
        op(a, b, q.z, q.w);
      }
    } else {
      const int lane = threadIdx.x & 31;
      a = s[at][lane % (kTeam / 32)][0], b = s[at][lane % (kTeam / 32)][1];
#pragma unroll
      for (int o = kTeam / 64; o; o >>= 1) op(a, b, __shfl_xor_sync(~0u, a, o), __shfl_xor_sync(~0u, b, o));
    }
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
__device__ __forceinline__ float max_nan(float a, float b, float c) {  // NaN if one of them is
  float r;
  asm("max.NaN.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
struct AddAndMax {
  __device__ __forceinline__ void operator()(float& a, float& b, float c, float d) const { a += c, b = max_nan(b, d, d); }
};

// Eight weights of the thread's columns, 0 past the end.
template <typename T, bool kWhole>
__device__ __forceinline__ Eight load_weights(const NormParams& p, const Cols<kWhole>& c) {
  if (!p.weight) {
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i) o.p[i] = Pair(1.f, 1.f);
    return o;
  }
  if (p.weight_fp32) return up8<float>(load8<float, kWhole>(static_cast<const float*>(p.weight), c));
  return up8<T>(load8<T, kWhole>(static_cast<const T*>(p.weight), c));
}

// The rows that a thread will work on next, its own columns of them: copied to shared
// memory kStages - 1 rows ahead, each by the thread that reads it, so no thread waits
// for another one's and no register holds them. Loads into registers were in flight
// only until the row's sums: with as many threads as fit, half of the time.
// Rows that are not whole, or of which two do not fit, are loaded into registers as
// they come (one stage).
// kDeep: bytes of a block up to which there are three stages. Forward 75000 (a million
// rows of 128 to e4m3: three 67 us, two 117); backward 40000, beyond which more blocks are
// worth more (30011 x 4096: two stages 178 us, three 195; others alike). 0, fp32: none. A
// thread then has as much in flight in registers, and copies of 16 of every 32 bytes are
// worse than loads, whose other half L1 has (50000 x 2048 forward 244 us, with stages 330;
// backward 248 and 413).
__host__ __device__ constexpr int queue_stages(int row_bytes, int deep, bool whole) {
  return !whole || deep == 0 || 2 * row_bytes > 200000 ? 1 : 3 * row_bytes <= deep ? 3 : 2;
}
template <typename T, int kBlock, int kGroups, int kStreams, int kDeep, bool kWhole>
struct Queue {
  static constexpr int kParts = sizeof(T) / 2;  // 16-byte parts of eight elements
  static constexpr int kRowBytes = kStreams * kGroups * kParts * kBlock * 16;
  static constexpr int kStages = queue_stages(kRowBytes, kDeep, kWhole);
  static constexpr bool kAhead = kStages > 1;
  static constexpr int kBytes = kAhead ? kStages * kRowBytes : 0;
  uint4* mine;
  Raw<T> held[kAhead ? 1 : kStreams][kGroups];
  __device__ __forceinline__ explicit Queue(uint4* smem) : mine(smem + threadIdx.x) {}
  __device__ __forceinline__ uint4* slot(int stage, int stream, int g) const {
    return mine + ((stage * kStreams + stream) * kGroups + g) * kParts * kBlock;
  }
  // `row` is not read where it is not there.
  __device__ __forceinline__ void fetch(int stage, int stream, int g, const T* row, const Cols<kWhole>& c, bool there) {
    if constexpr (kAhead) {
      const bool in = there && c.in(0);
      const uint4* from = reinterpret_cast<const uint4*>(row + c.first);
#pragma unroll
      for (int i = 0; i < kParts; ++i) cp_async16(smem_u32(slot(stage, stream, g) + i * kBlock), from + i, in ? 16 : 0);
    } else {
      held[stream][g] = load8<T, kWhole>(row, c, there);
    }
  }
  __device__ __forceinline__ Raw<T> get(int stage, int stream, int g) const {
    Raw<T> r;
    if constexpr (kAhead) {
#pragma unroll
      for (int i = 0; i < kParts; ++i) r.v[i] = slot(stage, stream, g)[i * kBlock];
    } else {
      r = held[stream][g];
    }
    return r;
  }
};

// 1 / sqrt(x), x > 0: the hardware's value and one step of Newton's method.
__device__ __forceinline__ float root_of(float x) {
  const float r = rsqrtf(x);
  return r * fmaf(-0.5f * x * r, r, 1.5f);
}

constexpr int kMaxNormWidth = 16384;

}  // namespace msim

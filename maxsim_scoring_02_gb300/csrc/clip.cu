// clip.cu -- the global norm of many gradient tensors, and their clipping.
//
//   norm = sqrt(sum over all tensors of g^2);  g *= min(1, max_norm / (norm + 1e-6))
//
// Two kernels read the tensors' table from their launch parameters. The first
// sums squares: every block walks over 32 KB chunks, a thread adds its own
// squares in fp32 within a chunk and in fp64 across chunks, and each block
// writes one partial. Squares that leave fp32's range (a chunk whose sum is
// not finite, or tiny with something nonzero in it) are added again in fp64.
// In the second every block adds all partials in the same order, so the
// factor is the same everywhere and does not depend on scheduling, and scales
// chunks from the last to the first: what the first kernel read last is still
// in L2. Bound by HBM: one read for the norm, one read and one write: 264 M fp32
// elements 497 us for both (6.4 TB/s), 516 with six blocks an SM and streaming
// accesses, 562 with four and 64 KB chunks. An output that lies differently from
// its input against 16-byte boundaries is written element by element: 196 tensors,
// 132.8 M bf16 elements 304 us for both where vectors take 140.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace msim {
namespace {

constexpr int kThreads = 256;
constexpr int kVecs = 8;                                 // 16-byte vectors of a thread in a chunk
constexpr int kChunkBytes = kThreads * kVecs * 16;       // 32 KB
constexpr int kBlocksPerSm = 8;
constexpr int kMaxClipBlocks = 2048;                     // partials of one launch

template <int N>
struct ClipTable {
  const void* in[N];
  void* out[N];
  int64_t n[N];
  int first[N + 1];   // first chunk of each tensor
  int8_t dtype[N];
  int tensors;
};

struct ClipArgs {
  double* partials;   // of this launch
  const double* all;  // of every launch
  float* norm;
  int count;          // of all partials
  float max_norm;
  int writes_norm;
};

template <typename T>
__device__ __forceinline__ float up(T x) { return static_cast<float>(x); }

// One chunk of one tensor: elements [a, b), the vectors in it start at the
// first 16-byte boundary `head` of the tensor.
struct Chunk {
  int tensor;
  int64_t a, b, body;
};

template <int N>
__device__ __forceinline__ Chunk find_chunk(const ClipTable<N>& t, int c) {
  int lo = 0, hi = t.tensors;
  while (hi - lo > 1) {
    const int m = (lo + hi) / 2;
    if (t.first[m] <= c) lo = m; else hi = m;
  }
  Chunk k;
  k.tensor = lo;
  const int esize = t.dtype[lo] == MAXSIM_FP32 ? 4 : 2;
  const int64_t n = t.n[lo];
  const int64_t head = min(n, static_cast<int64_t>(((16 - (reinterpret_cast<uintptr_t>(t.in[lo]) & 15)) & 15) / esize));
  const int64_t per = kChunkBytes / esize, j = c - t.first[lo];
  k.body = head + j * per;
  k.a = j == 0 ? 0 : k.body;
  k.b = min(n, k.body + per);
  return k;
}

__device__ __forceinline__ double block_sum(double v) {
  __shared__ double s[kThreads / 32];
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(~0u, v, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = 0.;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) r += s[w];
  __syncthreads();
  return r;
}

template <typename T>
__device__ __forceinline__ double chunk_squares(const T* g, const Chunk& k) {
  constexpr int E = 16 / sizeof(T);
  const int64_t vecs = (k.b - k.body) / E;
  float s[4] = {};
  uint32_t any = 0;
  const uint4* v = reinterpret_cast<const uint4*>(g + k.body);
#pragma unroll 8
  for (int u = 0; u < kVecs; ++u) {
    const int64_t i = u * kThreads + threadIdx.x;
    if (i < vecs) {
      const uint4 w = __ldg(v + i);
      any |= w.x | w.y | w.z | w.w;
      const T* e = reinterpret_cast<const T*>(&w);
#pragma unroll
      for (int x = 0; x < E; ++x) s[x % 4] = fmaf(up(e[x]), up(e[x]), s[x % 4]);
    }
  }
  float sum = (s[0] + s[1]) + (s[2] + s[3]);
  double total = sum;
  if (any && !(sum > 1e-25f && sum < 3e38f)) {  // out of fp32's range, or not finite: once more in fp64
    total = 0.;
    for (int64_t i = threadIdx.x; i < vecs; i += kThreads)
      for (int x = 0; x < E; ++x) {
        const double y = up(g[k.body + i * E + x]);
        total += y * y;
      }
  }
  // elements before the first boundary and after the last whole vector
  const int64_t tail = k.body + vecs * E, loose = (k.body > k.b ? k.b : k.body) - k.a;
  for (int64_t i = threadIdx.x; i < loose; i += kThreads) {
    const double y = up(g[k.a + i]);
    total += y * y;
  }
  for (int64_t i = tail + threadIdx.x; i < k.b; i += kThreads) {
    const double y = up(g[i]);
    total += y * y;
  }
  return total;
}

template <int N>
__global__ void __launch_bounds__(kThreads) norm_kernel(const __grid_constant__ ClipTable<N> t, const ClipArgs a) {
  double total = 0.;
  for (int c = blockIdx.x; c < t.first[t.tensors]; c += gridDim.x) {
    const Chunk k = find_chunk(t, c);
    const void* g = t.in[k.tensor];
    switch (t.dtype[k.tensor]) {
      case MAXSIM_BF16: total += chunk_squares(static_cast<const __nv_bfloat16*>(g), k); break;
      case MAXSIM_FP16: total += chunk_squares(static_cast<const __half*>(g), k); break;
      default: total += chunk_squares(static_cast<const float*>(g), k);
    }
  }
  total = block_sum(total);
  if (threadIdx.x == 0) a.partials[blockIdx.x] = total;
}

template <typename T>
__device__ __forceinline__ void scale_chunk(const T* g, T* o, const Chunk& k, float f) {
  constexpr int E = 16 / sizeof(T);
  int64_t from = k.a;
  if (((reinterpret_cast<uintptr_t>(g) ^ reinterpret_cast<uintptr_t>(o)) & 15) == 0 && k.body < k.b) {
    const int64_t vecs = (k.b - k.body) / E;
    const uint4* v = reinterpret_cast<const uint4*>(g + k.body);
    uint4* d = reinterpret_cast<uint4*>(o + k.body);
#pragma unroll 8
    for (int u = 0; u < kVecs; ++u) {
      const int64_t i = u * kThreads + threadIdx.x;
      if (i < vecs) {
        uint4 w = v[i];
        T* e = reinterpret_cast<T*>(&w);
#pragma unroll
        for (int x = 0; x < E; ++x) e[x] = static_cast<T>(up(e[x]) * f);
        d[i] = w;
      }
    }
    for (int64_t i = k.a + threadIdx.x; i < k.body; i += kThreads) o[i] = static_cast<T>(up(g[i]) * f);
    from = k.body + vecs * E;
  }
  for (int64_t i = from + threadIdx.x; i < k.b; i += kThreads) o[i] = static_cast<T>(up(g[i]) * f);
}

template <int N>
__global__ void __launch_bounds__(kThreads) scale_kernel(const __grid_constant__ ClipTable<N> t, const ClipArgs a) {
  double s = 0.;
  for (int i = threadIdx.x; i < a.count; i += kThreads) s += a.all[i];
  const double norm = sqrt(block_sum(s));
  const double ratio = static_cast<double>(a.max_norm) / (norm + 1e-6);
  const float f = ratio >= 1. ? 1.f : static_cast<float>(ratio);  // a norm that is not a number stays one
  if (a.writes_norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = static_cast<float>(norm);
  const int chunks = t.first[t.tensors];
  for (int c = chunks - 1 - static_cast<int>(blockIdx.x); c >= 0; c -= gridDim.x) {
    const Chunk k = find_chunk(t, c);
    const void* g = t.in[k.tensor];
    void* o = t.out[k.tensor];
    if (f == 1.f && g == o) continue;  // in place and within the limit: nothing changes
    switch (t.dtype[k.tensor]) {
      case MAXSIM_BF16:
        scale_chunk(static_cast<const __nv_bfloat16*>(g), static_cast<__nv_bfloat16*>(o), k, f);
        break;
      case MAXSIM_FP16: scale_chunk(static_cast<const __half*>(g), static_cast<__half*>(o), k, f); break;
      default: scale_chunk(static_cast<const float*>(g), static_cast<float*>(o), k, f);
    }
  }
}

struct ClipCall {
  const void* const* in;
  void* const* out;
  const int64_t* n;
  const int32_t* dtype;
};

template <int N>
bool fill(ClipTable<N>& t, const ClipCall& call, int from, int to) {
  int64_t chunks = 0;
  t.tensors = to - from;
  for (int i = from; i < to; ++i) {
    const int j = i - from, esize = call.dtype[i] == MAXSIM_FP32 ? 4 : 2;
    const int64_t head = ((16 - (reinterpret_cast<uintptr_t>(call.in[i]) & 15)) & 15) / esize;
    const int64_t per = kChunkBytes / esize, body = call.n[i] > head ? call.n[i] - head : 0;
    t.in[j] = call.in[i];
    t.out[j] = call.out[i];
    t.n[j] = call.n[i];
    t.dtype[j] = static_cast<int8_t>(call.dtype[i]);
    t.first[j] = static_cast<int>(chunks);
    chunks += call.n[i] == 0 ? 0 : (body + per - 1) / per > 1 ? (body + per - 1) / per : 1;
    if (chunks > INT_MAX / 2) return false;
  }
  t.first[t.tensors] = static_cast<int>(chunks);
  return true;
}

template <int N>
maxsim_status launch_group(const ClipCall& call, int from, int to, int blocks, ClipArgs a, bool scale,
                           cudaStream_t stream) {
  ClipTable<N> t;
  if (!fill(t, call, from, to)) return MAXSIM_ERR_UNSUPPORTED;
  const int chunks = t.first[t.tensors];
  if (scale) {
    const int grid = chunks < 1 ? 1 : chunks < blocks ? chunks : blocks;
    scale_kernel<N><<<grid, kThreads, 0, stream>>>(t, a);
  } else {
    norm_kernel<N><<<blocks, kThreads, 0, stream>>>(t, a);
  }
  return cudaGetLastError() == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

// The table travels in the launch parameters (at most 32,764 bytes): longer
// lists take several launches, short ones a small table.
constexpr int kGroup = 1024;

}  // namespace

size_t clip_workspace_bytes(int tensors) {
  const int groups = tensors < 1 ? 1 : (tensors + kGroup - 1) / kGroup;
  return static_cast<size_t>(groups) * kMaxClipBlocks * sizeof(double);
}

maxsim_status launch_clip(const void* const* grads, void* const* outs, const int64_t* sizes, const int32_t* dtypes,
                          int tensors, float max_norm, float* norm, void* workspace, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  const ClipCall call{grads, outs, sizes, dtypes};
  int64_t bytes = 0;
  for (int i = 0; i < tensors; ++i) bytes += sizes[i] * (dtypes[i] == MAXSIM_FP32 ? 4 : 2);
  int64_t most = bytes / kChunkBytes + tensors;  // no more blocks than chunks
  int blocks = dev->sm_count * kBlocksPerSm;
  if (blocks > kMaxClipBlocks) blocks = kMaxClipBlocks;
  if (most < blocks) blocks = most < 1 ? 1 : static_cast<int>(most);
  const int groups = tensors < 1 ? 1 : (tensors + kGroup - 1) / kGroup;
  ClipArgs a;
  a.all = static_cast<const double*>(workspace);
  a.norm = norm;
  a.count = groups * blocks;
  a.max_norm = max_norm;
  for (int scale = 0; scale < 2; ++scale)
    for (int g = 0; g < groups; ++g) {
      a.partials = static_cast<double*>(workspace) + static_cast<int64_t>(g) * blocks;
      a.writes_norm = g == 0;
      const int from = g * kGroup, to = tensors < from + kGroup ? tensors : from + kGroup;
      maxsim_status st;
      if (to - from <= 32) st = launch_group<32>(call, from, to, blocks, a, scale, stream);
      else if (to - from <= 256) st = launch_group<256>(call, from, to, blocks, a, scale, stream);
      else st = launch_group<kGroup>(call, from, to, blocks, a, scale, stream);
      if (st != MAXSIM_OK) return st;
    }
  return MAXSIM_OK;
}

}  // namespace msim

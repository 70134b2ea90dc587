// rotary.cu -- rotary positions on [T, heads, d] views, forward and gradient.
//
// Pair i of a head is turned by position * theta_i:
//   y1 = a (x1 cos - x2 sin),  y2 = a (x2 cos + x1 sin)
// with (x1, x2) = (x[i], x[i + r/2]) or (x[2i], x[2i + 1]); the gradient is the
// same with the sine's sign turned. Dimensions from r on are copied.
//
// theta_i comes as turns per position in units of 2^-64, so position *
// theta_i in 64-bit integers, which drops whole turns, is exact to 2^-32 of a
// turn for positions up to 2^31: an fp32 product would be off by 5e-3 rad at
// position 10^5. The upper 32 bits become the argument of sincospif.
//
// A thread owns V pairs of one token and walks over heads, so the sine and
// cosine are made once per token and pair, not once per head. The kernel moves
// every byte once and is bound by HBM: 96 x 1024 tokens, 20 heads of 128 in
// bf16 160 us (6.3 TB/s); 131071 tokens, 64 of 128 dimensions of 10 heads turned
// in fp16 119 us (5.6 TB/s), 160 while turning and copying threads ran apart.
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace msim {
namespace {

constexpr int kThreads = 256;

struct RotaryParams {
  const void* x;
  void* out;
  int64_t x_token, x_head, o_token, o_head;
  const uint64_t* freq;
  const int64_t* offsets;
  const int32_t* positions;
  unsigned* status;
  int64_t B;
  int T, heads, d, r;
  int per_token;      // threads of one token: V pairs each, then up to 2 V copied elements each
  int heads_each;     // heads walked by one thread
  float amplitude, sign;
};

template <typename T>
__device__ __forceinline__ float up(T x) { return static_cast<float>(x); }
template <typename T>
__device__ __forceinline__ T down(float x) { return static_cast<T>(x); }

template <typename T, int V>
struct alignas(sizeof(T) * V) Vec {
  T e[V];
};

__device__ __forceinline__ int position_of(const RotaryParams& p, int t) {
  if (p.positions) return p.positions[t];
  if (!p.offsets) return t;
  int64_t lo = 0, hi = p.B;
  while (hi - lo > 1) {
    const int64_t m = lo + (hi - lo) / 2;
    if (p.offsets[m] <= t) lo = m; else hi = m;
  }
  const int64_t s = p.offsets[lo], e = p.offsets[lo + 1];
  if (s < 0 || s > t || e <= t || e > p.T) {
    atomicOr(p.status, kDevErrBadInput);
    return 0;
  }
  return t - static_cast<int>(s);
}

// V: pairs of a thread. Half layout: two vectors of V elements r/2 apart.
// Interleaved: two neighbouring vectors that hold V pairs.
template <typename T, int V, bool kInterleaved, bool kCopies>
__global__ void __launch_bounds__(kThreads) rotary_kernel(const RotaryParams p) {
  const int64_t id = blockIdx.x * static_cast<int64_t>(kThreads) + threadIdx.x;
  const int t = static_cast<int>(id / p.per_token), part = static_cast<int>(id % p.per_token);
  if (t >= p.T) return;
  const int h0 = blockIdx.y * p.heads_each, h1 = min(p.heads, h0 + p.heads_each);
  const T* src = static_cast<const T*>(p.x) + t * p.x_token;
  T* dst = static_cast<T*>(p.out) + t * p.o_token;
  using W = Vec<T, V>;
  const int rotating = p.r / 2 / V;
  const bool turns = !kCopies || part < rotating;  // else two vectors that are only copied
  float cs[V], sn[V];
  if (turns) {
    const uint64_t pos = static_cast<uint64_t>(static_cast<int64_t>(position_of(p, t)));
#pragma unroll
    for (int k = 0; k < V; ++k) {
      const int turn = static_cast<int>(static_cast<uint32_t>((pos * p.freq[part * V + k]) >> 32));
      sincospif(static_cast<float>(turn) * (1.f / 2147483648.f), &sn[k], &cs[k]);
      cs[k] *= p.amplitude;
      sn[k] *= p.amplitude * p.sign;
    }
  } else {
#pragma unroll
    for (int k = 0; k < V; ++k) cs[k] = 1.f, sn[k] = 0.f;
  }
  const int c0 = !turns ? p.r + (part - rotating) * 2 * V : kInterleaved ? part * 2 * V : part * V;
  const int c1 = !turns || kInterleaved ? c0 + V : c0 + p.r / 2;
  const bool second = turns || c1 < p.d;  // the copied vectors may be odd in number
  // Rotating and copying threads of a warp run the same loop: two vectors a
  // head each, so loads and stores of both are in flight together.
#pragma unroll 4
  for (int h = h0; h < h1; ++h) {
    W a = *reinterpret_cast<const W*>(src + h * p.x_head + c0);
    W b = *reinterpret_cast<const W*>(src + h * p.x_head + (second ? c1 : c0));
    const W a0 = a, b0 = b;
    if constexpr (kInterleaved) {
#pragma unroll
      for (int k = 0; k < V; ++k) {  // pair k sits at elements 2k, 2k + 1 of a and b
        T& e1 = 2 * k < V ? a.e[(2 * k) % V] : b.e[(2 * k) % V];
        T& e2 = 2 * k + 1 < V ? a.e[(2 * k + 1) % V] : b.e[(2 * k + 1) % V];
        const float x1 = up(e1), x2 = up(e2);
        e1 = down<T>(x1 * cs[k] - x2 * sn[k]);
        e2 = down<T>(x2 * cs[k] + x1 * sn[k]);
      }
    } else {
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float x1 = up(a.e[k]), x2 = up(b.e[k]);
        a.e[k] = down<T>(x1 * cs[k] - x2 * sn[k]);
        b.e[k] = down<T>(x2 * cs[k] + x1 * sn[k]);
      }
    }
    *reinterpret_cast<W*>(dst + h * p.o_head + c0) = turns ? a : a0;
    if (second) *reinterpret_cast<W*>(dst + h * p.o_head + c1) = turns ? b : b0;
  }
}

template <typename T, int V>
void launch_v(RotaryParams& p, int interleaved, int copied, int sm_count, cudaStream_t stream) {
  p.per_token = p.r / 2 / V + (copied / V + 1) / 2;
  const int64_t blocks = (static_cast<int64_t>(p.T) * p.per_token + kThreads - 1) / kThreads;
  // few tokens: the heads are split over blocks until every SM has a few
  const int64_t want = (4 * static_cast<int64_t>(sm_count) + blocks - 1) / blocks;
  const int parts = static_cast<int>(want < p.heads ? want : p.heads);
  p.heads_each = (p.heads + parts - 1) / parts;
  const dim3 grid(static_cast<unsigned>(blocks), (p.heads + p.heads_each - 1) / p.heads_each);
  if (interleaved && copied) rotary_kernel<T, V, true, true><<<grid, kThreads, 0, stream>>>(p);
  else if (interleaved) rotary_kernel<T, V, true, false><<<grid, kThreads, 0, stream>>>(p);
  else if (copied) rotary_kernel<T, V, false, true><<<grid, kThreads, 0, stream>>>(p);
  else rotary_kernel<T, V, false, false><<<grid, kThreads, 0, stream>>>(p);
}

}  // namespace

maxsim_status launch_rotary(const maxsim_heads& x, int64_t T, int heads, int d, int rot_dim, const uint64_t* freq,
                            const int64_t* offsets, int64_t B, const int32_t* positions, int interleaved,
                            float amplitude, int inverse, int dtype, const maxsim_heads& out, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  RotaryParams p;
  p.x = x.data;
  p.out = out.data;
  p.x_token = x.token_stride;
  p.x_head = x.head_stride;
  p.o_token = out.token_stride;
  p.o_head = out.head_stride;
  p.freq = freq;
  p.offsets = offsets;
  p.positions = positions;
  p.status = dev->status;
  p.B = B;
  p.T = static_cast<int>(T);
  p.heads = heads;
  p.d = d;
  p.r = rot_dim;
  p.amplitude = amplitude;
  p.sign = inverse ? -1.f : 1.f;
  const int copied = x.data == out.data ? 0 : d - rot_dim;  // in place, the other dimensions are there already
  const int esize = dtype == MAXSIM_FP32 ? 4 : 2;
  // widest vector (at most 16 bytes) that every address is a multiple of
  const uint64_t all = static_cast<uint64_t>(p.x_token) | p.x_head | p.o_token | p.o_head | (rot_dim / 2) | copied |
                       (reinterpret_cast<uintptr_t>(p.x) / esize) | (reinterpret_cast<uintptr_t>(p.out) / esize);
  int V = 16 / esize;
  while (V > 1 && all % V) V /= 2;
  const int n = dev->sm_count;
#define MSIM_ROTARY(T_)                                              \
  do {                                                               \
    if (V == 8 && sizeof(T_) == 2) launch_v<T_, 8>(p, interleaved, copied, n, stream); \
    else if (V == 4) launch_v<T_, 4>(p, interleaved, copied, n, stream);               \
    else if (V == 2) launch_v<T_, 2>(p, interleaved, copied, n, stream);               \
    else launch_v<T_, 1>(p, interleaved, copied, n, stream);                           \
  } while (0)
  if (dtype == MAXSIM_BF16) MSIM_ROTARY(__nv_bfloat16);
  else if (dtype == MAXSIM_FP16) MSIM_ROTARY(__half);
  else MSIM_ROTARY(float);
#undef MSIM_ROTARY
  return cudaGetLastError() == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

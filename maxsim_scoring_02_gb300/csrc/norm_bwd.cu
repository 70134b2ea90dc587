// norm_bwd.cu -- gradients of the root-mean-square norm (norm.cu), of the residual's
// addition and of the dropout before it.
//
//   g = dy w,  c = mean(g h) rstd^2,  dsum = rstd (g - h c) + more
//   dx = dropped(dsum),  dw = sum over rows of dy h rstd
//
// One pass over dy, h and what reaches the sum from elsewhere; rstd is made again
// from h, which is read anyway, so the forward keeps nothing but its sum. A thread
// has the same columns in all of its team's rows and adds their part of dw in
// registers; a block's teams are added in order, each block writes one row of
// partial sums, and a second kernel adds those in order: no atomics, and results
// depend on the number of SMs alone. Bound by HBM.
#include "norm.cuh"

namespace msim {
namespace {

constexpr int kMaxBlocks = 8 * 160;

template <typename T, int kTeam, int kGroups, bool kWhole>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : 256) norm_bwd_kernel(const NormParams p) {
  constexpr int kTeams = kTeam > 32 ? 1 : 256 / kTeam;
  const int t = threadIdx.x % kTeam, lane = threadIdx.x & 31, team = threadIdx.x / kTeam;
  const Key key = load_key(p.drop);
  const auto cols = [&](int g) {
    return Cols<kWhole>(kWhole ? g * kTeam + t : g * (kTeam / 32) + (kTeam > 32 ? t >> 5 : 0), lane, p.d);
  };
  float acc[kGroups][8] = {};
  int at = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kTeams; first < p.T;
       first += static_cast<int64_t>(gridDim.x) * kTeams) {
    const bool live = first + team < p.T;
    const int r = live ? static_cast<int>(first + team) : p.T - 1;
    alignas(16) T dy[kGroups][8], hh[kGroups][8], more[kGroups][8];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      load8<T, kWhole>(static_cast<const T*>(p.x) + r * p.x_stride, cols(g), dy[g]);
      load8<T, kWhole>(static_cast<const T*>(p.res) + r * p.res_stride, cols(g), hh[g]);
      if (p.more) load8<T, kWhole>(static_cast<const T*>(p.more) + r * p.more_stride, cols(g), more[g]);
    }
    float ss = 0.f, gh = 0.f, w[kGroups][8];
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      load_weights<T, kWhole>(p, cols(g), w[g]);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = up(hh[g][j]);
        w[g][j] *= up(dy[g][j]);
        ss = fmaf(h, h, ss);
        gh = fmaf(w[g][j], h, gh);
      }
    }
    team_all<kTeam>(ss, gh, AddBoth(), at);
    const bool fits = ss < 3e38f && fabsf(gh) < 3e38f;
    float rstd = 1.f / sqrtf(ss / p.d + p.eps), c = gh / p.d * rstd * rstd;
    if (any_of_team<kTeam>(!fits)) {  // out of fp32's range: once more in fp64
      double a = 0., b = 0.;
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const double h = up(hh[g][j]);
          a += h * h;
          b += w[g][j] * h;
        }
      team_all<kTeam>(a, b, AddBoth(), at);
      if (!fits) {
        const double wide = 1. / sqrt(a / p.d + p.eps);
        rstd = static_cast<float>(wide), c = static_cast<float>(b / p.d * wide * wide);
      }
    }
    at ^= 1;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> cc = cols(g);
      float back[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float h = up(hh[g][j]);
        back[j] = fmaf(rstd, w[g][j] - h * c, p.more ? up(more[g][j]) : 0.f);
        if (live) acc[g][j] = fmaf(up(dy[g][j]), h * rstd, acc[g][j]);
      }
      if (p.sum && live) store8<T, kWhole>(static_cast<T*>(p.sum) + r * p.sum_stride, cc, back);
      if (p.drop.limit) {
        const uint32_t keep = kept<kWhole>(key, cc, r, p.drop.limit);
#pragma unroll
        for (int j = 0; j < 8; ++j) back[j] = keep >> j & 1 ? back[j] * p.drop.factor : 0.f;
      }
      if (p.out && live) store8<T, kWhole>(static_cast<T*>(p.out) + r * p.out_stride, cc, back);
    }
  }
  if (!p.parts) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * p.d;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> c = cols(g);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c.in(j)) part[c.at(j)] = acc[g][j];
    }
  } else {
    __shared__ float s[kTeam * kGroups * 8];
    for (int k = 0; k < kTeams; ++k) {
      if (team == k)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const Cols<kWhole> c = cols(g);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c.in(j)) s[c.at(j)] = k ? s[c.at(j)] + acc[g][j] : acc[g][j];
        }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < p.d; i += 256) part[i] = s[i];
  }
}

// dw: the blocks' partial sums of 32 columns, 32 warps each adding every 32nd block.
template <typename W>
__global__ void __launch_bounds__(1024) fold_kernel(const float* parts, int blocks, int d, W* dw) {
  __shared__ float s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, col = blockIdx.x * 32 + lane;
  float a = 0.f;
  if (col < d)
#pragma unroll 8
    for (int b = warp; b < blocks; b += 32) a += parts[static_cast<int64_t>(b) * d + col];
  s[warp][lane] = a;
  __syncthreads();
  a = s[lane][warp];
#pragma unroll
  for (int o = 16; o; o >>= 1) a += __shfl_xor_sync(~0u, a, o);
  if (lane == 0 && blockIdx.x * 32 + warp < d) dw[blockIdx.x * 32 + warp] = static_cast<W>(a);
}

template <typename T, int kTeam, int kGroups, bool kWhole>
cudaError_t go(const NormParams& p, int sms, int* blocks, cudaStream_t stream) {
  constexpr int kTeams = kTeam > 32 ? 1 : 256 / kTeam, kBlock = kTeam > 32 ? kTeam : 256;
  int fit = 0;
  cudaError_t e =
      cudaOccupancyMaxActiveBlocksPerMultiprocessor(&fit, norm_bwd_kernel<T, kTeam, kGroups, kWhole>, kBlock, 0);
  if (e != cudaSuccess) return e;
  int grid = sms * (fit < 8 ? fit : 8);
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  const int64_t need = (static_cast<int64_t>(p.T) + kTeams - 1) / kTeams;
  if (need < grid) grid = static_cast<int>(need);
  norm_bwd_kernel<T, kTeam, kGroups, kWhole><<<grid, kBlock, 0, stream>>>(p);
  *blocks = grid;
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const NormParams& p, bool whole, int sms, int* blocks, cudaStream_t stream) {
  if (whole) {
    if (p.d <= 128) return go<T, 16, 1, true>(p, sms, blocks, stream);
    if (p.d <= 256) return go<T, 32, 1, true>(p, sms, blocks, stream);
    if (p.d <= 512) return go<T, 32, 2, true>(p, sms, blocks, stream);
    if (p.d <= 1024) return go<T, 128, 1, true>(p, sms, blocks, stream);
    if (p.d <= 2048) return go<T, 256, 1, true>(p, sms, blocks, stream);
    if (p.d <= 4096) return go<T, 512, 1, true>(p, sms, blocks, stream);
    if (p.d <= 8192) return go<T, 512, 2, true>(p, sms, blocks, stream);
    return go<T, 1024, 2, true>(p, sms, blocks, stream);
  }
  if (p.d <= 256) return go<T, 32, 1, false>(p, sms, blocks, stream);
  if (p.d <= 1024) return go<T, 128, 1, false>(p, sms, blocks, stream);
  if (p.d <= 4096) return go<T, 512, 1, false>(p, sms, blocks, stream);
  return go<T, 1024, 2, false>(p, sms, blocks, stream);
}

template <typename W>
cudaError_t fold(const float* parts, int blocks, int d, void* dw, cudaStream_t stream) {
  fold_kernel<W><<<(d + 31) / 32, 1024, 0, stream>>>(parts, blocks, d, static_cast<W*>(dw));
  return cudaGetLastError();
}

}  // namespace

size_t norm_bwd_workspace_bytes(int T, int d) {
  const int64_t blocks = T < kMaxBlocks ? T : kMaxBlocks;
  return static_cast<size_t>(blocks) * d * sizeof(float);
}

maxsim_status launch_norm_bwd(const NormParams& p, int dtype, bool whole, void* dweight, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  int blocks = 0;
  cudaError_t e = dtype == MAXSIM_BF16   ? pick<__nv_bfloat16>(p, whole, dev->sm_count, &blocks, stream)
                  : dtype == MAXSIM_FP16 ? pick<__half>(p, whole, dev->sm_count, &blocks, stream)
                                         : pick<float>(p, whole, dev->sm_count, &blocks, stream);
  if (e == cudaSuccess && dweight)
    e = p.weight_fp32          ? fold<float>(p.parts, blocks, p.d, dweight, stream)
        : dtype == MAXSIM_BF16 ? fold<__nv_bfloat16>(p.parts, blocks, p.d, dweight, stream)
        : dtype == MAXSIM_FP16 ? fold<__half>(p.parts, blocks, p.d, dweight, stream)
                               : fold<float>(p.parts, blocks, p.d, dweight, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

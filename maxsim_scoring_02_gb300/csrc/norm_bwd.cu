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
// depend on the sizes and the number of SMs alone. Bound by HBM: 24576 x 2048 bf16 with
// dropout and both gradients 94 us and 5 for the second kernel (5.3 TB/s), 30011 x 4096
// without 150 for both (6.5), a million rows of 128 124 (6.2). By instructions where rows are not whole
// (74962 x 2001 bf16 480, 2.5 TB/s), and by spilled registers where fp32 rows take four groups
// (146484 x 1024 502, 4.8; bf16 208, 5.8; 195312 x 768 394, 6.1; 187, 6.4).
#include "after.cuh"
#include "norm.cuh"

namespace msim {
namespace {

constexpr int kMaxBlocks = 1280;  // partial sums; each block has its rows from the start, so that their order is fixed

template <typename T, int kTeam, int kGroups, bool kWhole>
struct Shape {
  static constexpr int kBlock = kTeam > 32 ? kTeam : 256, kTeams = kBlock / kTeam;
  using Rows = Queue<T, kBlock, kGroups, 3, sizeof(T) == 4 ? 0 : 40000, kWhole>;
  // blocks of an SM that the registers have to allow (24576 x 2048: 512 threads 99 us, 768 103)
  static constexpr int kFit = kTeam > 256 ? 1 : 512 / kBlock;
};

template <typename T, int kTeam, int kGroups, bool kWhole>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : 256, Shape<T, kTeam, kGroups, kWhole>::kFit) rms_norm_bwd_kernel(const NormParams p) {
  using S = Shape<T, kTeam, kGroups, kWhole>;
  let_next_begin();
  constexpr int kTeams = S::kTeams, kStages = S::Rows::kStages, kAhead = kStages - 1;
  extern __shared__ uint4 smem[];
  const int t = threadIdx.x % kTeam, lane = threadIdx.x & 31, team = threadIdx.x / kTeam;
  const Key key = load_key(p.drop);
  const auto cols = [&](int g) {
    return Cols<kWhole>(kWhole ? g * kTeam + t : g * (kTeam / 32) + (kTeam > 32 ? t >> 5 : 0), lane, p.d);
  };
  Eight acc[kGroups];
#pragma unroll
  for (int g = 0; g < kGroups; ++g)
#pragma unroll
    for (int i = 0; i < 4; ++i) acc[g].p[i] = Pair(0.f, 0.f);
  Eight w[kGroups];  // in registers: read from L1 twice a row they cost a fifth of the time
#pragma unroll
  for (int g = 0; g < kGroups; ++g) w[g] = load_weights<T, kWhole>(p, cols(g));
  typename S::Rows rows(smem);  // dy, h, and what reaches the sum from elsewhere
  const int64_t step = static_cast<int64_t>(gridDim.x) * kTeams;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kTeams + team;
  const auto fetch = [&](int stage, int64_t r) {
    const bool there = r < p.T;  // else all of it is 0, and adds 0
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      rows.fetch(stage, 0, g, static_cast<const T*>(p.x) + r * p.x_stride, cols(g), there);
      rows.fetch(stage, 1, g, static_cast<const T*>(p.res) + r * p.res_stride, cols(g), there);
      if (p.more) rows.fetch(stage, 2, g, static_cast<const T*>(p.more) + r * p.more_stride, cols(g), there);
    }
    if constexpr (kAhead > 0) cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i, row + i * step);
  int at = 0, stage = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kTeams; first < p.T;
       first += step, at ^= 1, row += step, stage = stage + 1 < kStages ? stage + 1 : 0) {
    const bool live = row < p.T;
    fetch(stage + kAhead < kStages ? stage + kAhead : stage + kAhead - kStages, row + kAhead * step);
    if constexpr (kAhead > 0) cp_async_wait<kAhead>();
    Pair squares(0.f, 0.f), cross(0.f, 0.f);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Eight y = up8<T>(rows.get(stage, 0, g)), v = up8<T>(rows.get(stage, 1, g));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        squares = fma2(v.p[i], v.p[i], squares);
        cross = fma2(mul2(w[g].p[i], y.p[i]), v.p[i], cross);
      }
    }
    float ss, gh, odd;
    squares.get(ss, odd);
    ss += odd;
    cross.get(gh, odd);
    gh += odd;
    team_all<kTeam>(ss, gh, AddBoth(), at);
    asm volatile("" ::: "memory");  // elements are read and unpacked again, not held in 4 registers each
    const bool fits = ss < 3e38f && fabsf(gh) < 3e38f;
    float rstd = root_of(fmaf(ss, p.per, p.eps)), c = gh * p.per * rstd * rstd;
    if (any_of_team<kTeam>(!fits)) {  // out of fp32's range: once more in fp64
      double a = 0., b = 0.;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const Eight y = up8<T>(rows.get(stage, 0, g)), v = up8<T>(rows.get(stage, 1, g));
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float v0, v1, g0, g1;
          v.p[i].get(v0, v1);
          mul2(w[g].p[i], y.p[i]).get(g0, g1);
          a += static_cast<double>(v0) * v0 + static_cast<double>(v1) * v1;
          b += static_cast<double>(g0) * v0 + static_cast<double>(g1) * v1;
        }
      }
      team_all<kTeam>(a, b, AddBoth(), at);
      if (!fits) {
        const double wide = 1. / sqrt(a / p.d + p.eps);
        rstd = static_cast<float>(wide), c = static_cast<float>(b / p.d * wide * wide);
      }
    }
    const Pair r2(rstd, rstd), c2(-c, -c);
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> cc = cols(g);
      const Eight y = up8<T>(rows.get(stage, 0, g)), v = up8<T>(rows.get(stage, 1, g));
      Eight back;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        back.p[i] = mul2(r2, fma2(v.p[i], c2, mul2(w[g].p[i], y.p[i])));
        acc[g].p[i] = fma2(y.p[i], mul2(v.p[i], r2), acc[g].p[i]);
      }
      if (p.more) {
        const Eight m = up8<T>(rows.get(stage, 2, g));
#pragma unroll
        for (int i = 0; i < 4; ++i) back.p[i] = add2(back.p[i], m.p[i]);
      }
      if (p.sum && live) store8<T, kWhole>(static_cast<T*>(p.sum) + row * p.sum_stride, cc, down8<T>(back));
      if (p.drop.limit) {
        const Kept<kWhole> keep(key, cc, static_cast<uint32_t>(row), p.drop.limit);
        back = keep.of(back, p.drop.factor, back, false);
      }
      if (p.out && live) store8<T, kWhole>(static_cast<T*>(p.out) + row * p.out_stride, cc, down8<T>(back));
    }
  }
  if (!p.parts) return;
  float* part = p.parts + static_cast<int64_t>(blockIdx.x) * p.d;
  if constexpr (kTeams == 1) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> c = cols(g);
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[g].p[i].get(v[2 * i], v[2 * i + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c.in(j)) part[c.at(j)] = v[j];
    }
  } else {
    __shared__ float s[kTeam * kGroups * 8];
    for (int k = 0; k < kTeams; ++k) {
      if (team == k)
#pragma unroll
        for (int g = 0; g < kGroups; ++g) {
          const Cols<kWhole> c = cols(g);
          float v[8];
#pragma unroll
          for (int i = 0; i < 4; ++i) acc[g].p[i].get(v[2 * i], v[2 * i + 1]);
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c.in(j)) s[c.at(j)] = k ? s[c.at(j)] + v[j] : v[j];
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
  wait_for_previous();
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
cudaError_t go(const NormParams& p, const DeviceInfo& dev, int* blocks, cudaStream_t stream) {
  using S = Shape<T, kTeam, kGroups, kWhole>;
  const auto kernel = rms_norm_bwd_kernel<T, kTeam, kGroups, kWhole>;
  static Fits known;
  int fit = 1;
  const cudaError_t e = blocks_that_fit(known, dev, kernel, S::kBlock, S::Rows::kBytes, &fit);
  if (e != cudaSuccess) return e;
  int grid = dev.sm_count * (fit < 8 ? fit : 8);
  const int64_t need = (static_cast<int64_t>(p.T) + S::kTeams - 1) / S::kTeams;
  if (grid > kMaxBlocks) grid = kMaxBlocks;
  if (need < grid) grid = static_cast<int>(need);
  kernel<<<grid, S::kBlock, S::Rows::kBytes, stream>>>(p);
  *blocks = grid;
  return cudaGetLastError();
}

// Threads and groups of a row as in the forward, but for widths that are measured to be better
// otherwise (one gradient, with what reaches the sum; us, bf16 and fp32, this form first):
//   195312 x 768 three groups of a warp 187, 394; four 229, 565
//   9155 x 16383 1024 threads 483, 785; 512 with four groups 508, 785; 16664 x 9001 707, 1134; 750, 1003
// and as in the forward: 9155 x 16384 512 threads 191, 647; 1024 with two groups 190, 722; 74962 x 2001
// 256 threads 480, 630; 512 with one group 961, 750; 37490 x 4001 388, 419; 554, 504.
// fp32 rows of two groups or more, rows of four groups of a warp, and rows of 1024 threads spill.
template <typename T>
cudaError_t pick(const NormParams& p, bool whole, const DeviceInfo& dev, int* blocks, cudaStream_t stream) {
  if (whole) {
    if (p.d <= 64) return go<T, 8, 1, true>(p, dev, blocks, stream);
    if (p.d <= 128) return go<T, 8, 2, true>(p, dev, blocks, stream);
    if (p.d <= 256) return go<T, 16, 2, true>(p, dev, blocks, stream);
    if (p.d <= 512) return go<T, 32, 2, true>(p, dev, blocks, stream);
    if (p.d <= 768) return go<T, 32, 3, true>(p, dev, blocks, stream);
    if (p.d <= 1024) return go<T, 32, 4, true>(p, dev, blocks, stream);
    if (p.d <= 2048) return go<T, 128, 2, true>(p, dev, blocks, stream);
    if (p.d <= 4096) return go<T, 256, 2, true>(p, dev, blocks, stream);
    if (p.d <= 8192) return go<T, 512, 2, true>(p, dev, blocks, stream);
    return go<T, 512, 4, true>(p, dev, blocks, stream);
  }
  if (p.d <= 256) return go<T, 32, 1, false>(p, dev, blocks, stream);
  if (p.d <= 1024) return go<T, 128, 1, false>(p, dev, blocks, stream);
  if (p.d <= 4096) return go<T, 256, 2, false>(p, dev, blocks, stream);
  return go<T, 1024, 2, false>(p, dev, blocks, stream);
}

template <typename W>
cudaError_t fold(const float* parts, int blocks, int d, void* dw, cudaStream_t stream) {
  return launch_after(fold_kernel<W>, (d + 31) / 32, 1024, 0, stream, parts, blocks, d, static_cast<W*>(dw));
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
  cudaError_t e = dtype == MAXSIM_BF16   ? pick<__nv_bfloat16>(p, whole, *dev, &blocks, stream)
                  : dtype == MAXSIM_FP16 ? pick<__half>(p, whole, *dev, &blocks, stream)
                                         : pick<float>(p, whole, *dev, &blocks, stream);
  if (e == cudaSuccess && dweight)
    e = p.weight_fp32          ? fold<float>(p.parts, blocks, p.d, dweight, stream)
        : dtype == MAXSIM_BF16 ? fold<__nv_bfloat16>(p.parts, blocks, p.d, dweight, stream)
        : dtype == MAXSIM_FP16 ? fold<__half>(p.parts, blocks, p.d, dweight, stream)
                               : fold<float>(p.parts, blocks, p.d, dweight, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

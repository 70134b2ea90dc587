// norm.cu -- root-mean-square norm of rows, with dropout and the residual's addition
// before it, and with output in the rows' type or in 8 bits.
//
//   h = round(residual + dropped(x)),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   8 bits: scale = max(max |y|, 1e-30) / top,  code = round(y / scale)
//
// One pass: a team of threads holds its row in registers, so x and the residual are
// read once. With 8-bit output the sum of squares and the largest |h w| are found
// together, and y / scale = h w (top / max |h w|) needs no second look at the row.
// Teams are a warp or half of one where a row fits four groups of eight columns a
// lane, else a block. Bound by HBM.
#include <cuda_fp8.h>

#include "norm.cuh"

namespace msim {
namespace {

constexpr float kLeast = 1e-30f;

template <typename T, int kTeam, int kGroups, bool kWhole>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : 256) norm_kernel(const NormParams p) {
  constexpr int kRows = kTeam > 32 ? 1 : 256 / kTeam;
  const int t = threadIdx.x % kTeam, lane = threadIdx.x & 31;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTeam;
  const bool live = row < p.T;
  const int r = live ? static_cast<int>(row) : p.T - 1;
  const Key key = load_key(p.drop);
  const auto cols = [&](int g) {
    return Cols<kWhole>(kWhole ? g * kTeam + t : g * (kTeam / 32) + (kTeam > 32 ? t >> 5 : 0), lane, p.d);
  };
  alignas(16) T x[kGroups][8], add[kGroups][8];
#pragma unroll
  for (int g = 0; g < kGroups; ++g) load8<T, kWhole>(static_cast<const T*>(p.x) + r * p.x_stride, cols(g), x[g]);
  if (p.res)
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
      load8<T, kWhole>(static_cast<const T*>(p.res) + r * p.res_stride, cols(g), add[g]);
  float h[kGroups][8], ss = 0.f, most = 0.f;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const Cols<kWhole> c = cols(g);
    const uint32_t keep = p.drop.limit ? kept<kWhole>(key, c, r, p.drop.limit) : 0xFFu;
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float a = p.res ? up(add[g][j]) : 0.f;
      const float v = keep >> j & 1 ? fmaf(up(x[g][j]), p.drop.factor, a) : a;
      h[g][j] = up(static_cast<T>(v));  // the norm is that of the sum as it is kept
      ss = fmaf(h[g][j], h[g][j], ss);
    }
    if (p.sum && live) store8<T, kWhole>(static_cast<T*>(p.sum) + r * p.sum_stride, c, h[g]);
    if (p.format != MAXSIM_NORM_SAME) {
      float w[8];
      load_weights<T, kWhole>(p, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float u = h[g][j] * w[j];
        most = max_nan(most, c.in(j) ? fabsf(u) : 0.f);
      }
    }
  }
  team_all<kTeam>(ss, most, AddAndMax(), 0);
  const float rstd = [&] {
    const bool fits = ss < 3e38f;
    const float usual = 1.f / sqrtf(ss / p.d + p.eps);
    if (!any_of_team<kTeam>(!fits)) return usual;
    double wide = 0., none = 0.;  // squares out of fp32's range: once more in fp64
#pragma unroll
    for (int g = 0; g < kGroups; ++g)
#pragma unroll
      for (int j = 0; j < 8; ++j) wide += static_cast<double>(h[g][j]) * h[g][j];
    team_all<kTeam>(wide, none, AddBoth(), 1);
    return fits ? usual : static_cast<float>(1. / sqrt(wide / p.d + p.eps));
  }();
  if (p.format == MAXSIM_NORM_SAME) {
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> c = cols(g);
      float w[8];
      load_weights<T, kWhole>(p, c, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) w[j] *= h[g][j] * rstd;
      if (live) store8<T, kWhole>(static_cast<T*>(p.out) + r * p.out_stride, c, w);
    }
    return;
  }
  const float top = p.format == MAXSIM_NORM_INT8 ? 127.f : 448.f;
  float reach = most * rstd;
  reach = reach < kLeast ? kLeast : reach;  // NaN stays
  const float factor = top * rstd / reach;
  if (t == 0 && live) p.scale[r] = reach / top;
  uint8_t* out = static_cast<uint8_t*>(p.out) + r * p.out_stride;
#pragma unroll
  for (int g = 0; g < kGroups; ++g) {
    const Cols<kWhole> c = cols(g);
    float w[8];
    load_weights<T, kWhole>(p, c, w);
    uint32_t code[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float v = h[g][j] * w[j] * factor;
      if (p.format == MAXSIM_NORM_INT8) {
        const int q = __float2int_rn(v);
        code[j] = static_cast<uint32_t>(max(-127, min(127, q))) & 0xFFu;
      } else {
        code[j] = __nv_cvt_float_to_fp8(v, __NV_SATFINITE, __NV_E4M3);
      }
    }
    if (!live) continue;
    if constexpr (kWhole) {
      if (c.in(0))
        *reinterpret_cast<uint2*>(out + c.first) =
            make_uint2(code[0] | code[1] << 8 | code[2] << 16 | code[3] << 24,
                       code[4] | code[5] << 8 | code[6] << 16 | code[7] << 24);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c.in(j)) out[c.at(j)] = static_cast<uint8_t>(code[j]);
    }
  }
}

template <typename T, int kTeam, int kGroups, bool kWhole>
cudaError_t go(const NormParams& p, cudaStream_t stream) {
  constexpr int kRows = kTeam > 32 ? 1 : 256 / kTeam;
  const int grid = static_cast<int>((static_cast<int64_t>(p.T) + kRows - 1) / kRows);
  norm_kernel<T, kTeam, kGroups, kWhole><<<grid, kTeam > 32 ? kTeam : 256, 0, stream>>>(p);
  return cudaGetLastError();
}

template <typename T>
cudaError_t pick(const NormParams& p, bool whole, cudaStream_t stream) {
  if (whole) {
    if (p.d <= 128) return go<T, 16, 1, true>(p, stream);
    if (p.d <= 256) return go<T, 32, 1, true>(p, stream);
    if (p.d <= 512) return go<T, 32, 2, true>(p, stream);
    if (p.d <= 1024) return go<T, 32, 4, true>(p, stream);
    if (p.d <= 2048) return go<T, 128, 2, true>(p, stream);
    if (p.d <= 4096) return go<T, 256, 2, true>(p, stream);
    if (p.d <= 8192) return go<T, 512, 2, true>(p, stream);
    return go<T, 512, 4, true>(p, stream);
  }
  if (p.d <= 256) return go<T, 32, 1, false>(p, stream);
  if (p.d <= 1024) return go<T, 32, 4, false>(p, stream);
  if (p.d <= 4096) return go<T, 256, 2, false>(p, stream);
  return go<T, 512, 4, false>(p, stream);
}

}  // namespace

maxsim_status launch_norm(const NormParams& p, int dtype, bool whole, cudaStream_t stream) {
  const cudaError_t e = dtype == MAXSIM_BF16   ? pick<__nv_bfloat16>(p, whole, stream)
                        : dtype == MAXSIM_FP16 ? pick<__half>(p, whole, stream)
                                               : pick<float>(p, whole, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

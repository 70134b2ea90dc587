// norm.cu -- root-mean-square norm of rows, with dropout and the residual's addition
// before it, and with output in the rows' type or in 8 bits.
//
//   h = round(residual + dropped(x)),  rstd = 1 / sqrt(mean(h^2) + eps),  y = h rstd w
//   8 bits: scale = max(max |y|, 1e-30) / top,  code = round(y / scale)
//
// One pass: x and the residual are read once, and the sum stays in registers as it is
// kept. With 8-bit output the sum of squares and the largest |h w| are found together:
// max |y| = rstd max |h w| needs no second look at the row, and y / scale = (h w rstd) (top / max |y|).
// A team of threads has a row, eight neighbouring columns a thread and group: part of
// a warp up to 256 columns, a warp up to 1024, a block beyond. Its next rows are on
// their way to shared memory (norm.cuh). Bound by HBM: 98304 x 2048 bf16 with residual
// and sum 235 us (6.9 TB/s), 30011 x 4096 to e4m3 130 (6.6), a million rows of 128 to
// e4m3 68 (5.6; issue slots 71 % busy), to int8 74 (5.2). With loads into registers e4m3 took 151
// and 169. Rows that are not whole: 200011 x 1001 bf16 200 us (4.0 TB/s), 2 bytes an access.
#include <cuda_fp8.h>

#include "norm.cuh"

namespace msim {
namespace {

constexpr float kLeast = 1e-30f;

template <typename T, int kTeam, int kGroups, bool kWhole>
struct Shape {
  static constexpr int kBlock = kTeam > 32 ? kTeam : 256, kRows = kBlock / kTeam;
  using Rows = Queue<T, kBlock, kGroups, 2, sizeof(T) == 4 ? 0 : 75000, kWhole>;
  // Blocks of an SM that the registers have to allow; rows of a team, where a row takes a
  // warp or more, or of fp32: blocks that come and go even out what SMs do, fixed ones (a
  // million rows of 128 to e4m3: 68 us, 75 with 32 rows a team) wait for the slowest (98304 x
  // 2048: 262 us, 235). fp32: 512 threads 244 us for 50000 x 2048, 1024 259.
  static constexpr int kFit = kTeam > 256 ? 1 : sizeof(T) == 4 ? 512 / kBlock : kTeam > 32 ? 1024 / kTeam : 2;
  static constexpr int kRounds = 8;
  static constexpr bool kComeAndGo = kTeam > 16 || sizeof(T) == 4;
};

template <typename T, int kTeam, int kGroups, bool kWhole, bool k8>
__global__ void __launch_bounds__(kTeam > 32 ? kTeam : 256, Shape<T, kTeam, kGroups, kWhole>::kFit) rms_norm_kernel(const NormParams p) {
  using S = Shape<T, kTeam, kGroups, kWhole>;
  constexpr int kRows = S::kRows, kStages = S::Rows::kStages, kAhead = kStages - 1;
  constexpr bool kHold = kGroups <= 2;  // weights stay in registers
  extern __shared__ uint4 smem[];
  const int t = threadIdx.x % kTeam, lane = threadIdx.x & 31;
  const Key key = load_key(p.drop);
  const auto cols = [&](int g) {
    return Cols<kWhole>(kWhole ? g * kTeam + t : g * (kTeam / 32) + (kTeam > 32 ? t >> 5 : 0), lane, p.d);
  };
  Eight held[kHold ? kGroups : 1];
  if constexpr (kHold)
#pragma unroll
    for (int g = 0; g < kGroups; ++g) held[g] = load_weights<T, kWhole>(p, cols(g));
  const auto weights = [&](int g) -> Eight {
    if constexpr (kHold) return held[g];
    else return load_weights<T, kWhole>(p, cols(g));
  };
  typename S::Rows rows(smem);
  const int64_t step = static_cast<int64_t>(gridDim.x) * kRows;
  int64_t row = static_cast<int64_t>(blockIdx.x) * kRows + threadIdx.x / kTeam;
  const auto fetch = [&](int stage, int64_t r) {
    const bool there = r < p.T;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) rows.fetch(stage, 0, g, static_cast<const T*>(p.x) + r * p.x_stride, cols(g), there);
    if (p.res)
#pragma unroll
      for (int g = 0; g < kGroups; ++g)
        rows.fetch(stage, 1, g, static_cast<const T*>(p.res) + r * p.res_stride, cols(g), there);
    if constexpr (kAhead > 0) cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) fetch(i, row + i * step);
  int at = 0, stage = 0;
  for (int64_t first = static_cast<int64_t>(blockIdx.x) * kRows; first < p.T;
       first += step, at ^= 1, row += step, stage = stage + 1 < kStages ? stage + 1 : 0) {
    const bool live = row < p.T;
    fetch(stage + kAhead < kStages ? stage + kAhead : stage + kAhead - kStages, row + kAhead * step);
    if constexpr (kAhead > 0) cp_async_wait<kAhead>();
    Raw<T> in[kGroups];  // becomes the sum
#pragma unroll
    for (int g = 0; g < kGroups; ++g) in[g] = rows.get(stage, 0, g);
    Pair squares(0.f, 0.f);
    float most = 0.f;
#pragma unroll
    for (int g = 0; g < kGroups; ++g) {
      const Cols<kWhole> c = cols(g);
      Eight v = up8<T>(in[g]);
      if (p.drop.limit || p.res) {
        Eight a;
        if (p.res) a = up8<T>(rows.get(stage, 1, g));
        if (p.drop.limit) {
          const Kept<kWhole> keep(key, c, static_cast<uint32_t>(row), p.drop.limit);
          v = keep.of(v, p.drop.factor, a, p.res != nullptr);
        } else {
#pragma unroll
          for (int i = 0; i < 4; ++i) v.p[i] = add2(v.p[i], a.p[i]);
        }
        in[g] = down8<T>(v);
        v = up8<T>(in[g]);  // the norm is that of the sum as it is kept
      }
      if (p.sum && live) store8<T, kWhole>(static_cast<T*>(p.sum) + row * p.sum_stride, c, in[g]);
#pragma unroll
      for (int i = 0; i < 4; ++i) squares = fma2(v.p[i], v.p[i], squares);
      if constexpr (k8) {  // columns past the end are 0
        const Eight w = weights(g);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          mul2(v.p[i], w.p[i]).get(a, b);
          most = max_nan(most, fabsf(a), fabsf(b));
        }
      }
    }
#pragma unroll
    for (int g = 0; g < kGroups; ++g) forget<T>(in[g]);
    float ss, odd;
    squares.get(ss, odd);
    ss += odd;
    team_all<kTeam>(ss, most, AddAndMax(), at);
    const bool fits = ss < 3e38f;
    float rstd = root_of(fmaf(ss, p.per, p.eps));
    if (any_of_team<kTeam>(!fits)) {  // squares out of fp32's range: once more in fp64
      double wide = 0., none = 0.;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const Eight h = up8<T>(in[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          h.p[i].get(a, b);
          wide += static_cast<double>(a) * a + static_cast<double>(b) * b;
        }
      }
      team_all<kTeam>(wide, none, AddBoth(), at);
      if (!fits) rstd = static_cast<float>(1. / sqrt(wide / p.d + p.eps));
    }
    if constexpr (!k8) {
      const Pair r2(rstd, rstd);
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        Eight y = weights(g);
        const Eight h = up8<T>(in[g]);
#pragma unroll
        for (int i = 0; i < 4; ++i) y.p[i] = mul2(y.p[i], mul2(h.p[i], r2));
        if (live) store8<T, kWhole>(static_cast<T*>(p.out) + row * p.out_stride, cols(g), down8<T>(y));
      }
    } else {
      const bool whole_numbers = p.format == MAXSIM_NORM_INT8;
      const float top = whole_numbers ? 127.f : 448.f;
      float reach = most * rstd;
      reach = reach < kLeast ? kLeast : reach;  // NaN stays
      const float steps = __fdividef(0.25f * top, 0.25f * reach);  // whose divisors end at 2^126
      // y first: its product with steps stays in range, while top rstd / reach and top / max |h w|
      // leave it for small rows where eps is small
      const Pair r2(rstd, rstd), s2(steps, steps);
      if (t == 0 && live) p.scale[row] = reach / top;
      uint8_t* out = static_cast<uint8_t*>(p.out) + row * p.out_stride;
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        const Cols<kWhole> c = cols(g);
        const Eight w = weights(g), h = up8<T>(in[g]);
        uint32_t two[4];  // codes of two columns each
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          float a, b;
          mul2(mul2(mul2(h.p[i], w.p[i]), r2), s2).get(a, b);
          if (whole_numbers) {  // |a| <= 127 (1 + 2^-21): no code is -128
            int q, s;
            asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(q) : "f"(a));
            asm("cvt.rni.sat.s8.f32 %0, %1;" : "=r"(s) : "f"(b));
            two[i] = __byte_perm(q, s, 0x7740);  // the upper half is not used
          } else {
            two[i] = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
          }
        }
        if (!live) continue;
        if constexpr (kWhole) {
          if (c.in(0))
            *reinterpret_cast<uint2*>(out + c.first) =
                make_uint2(__byte_perm(two[0], two[1], 0x5410), __byte_perm(two[2], two[3], 0x5410));
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (c.in(j)) out[c.at(j)] = static_cast<uint8_t>(two[j / 2] >> (8 * (j & 1)));
        }
      }
    }
  }
}

template <typename T, int kTeam, int kGroups, bool kWhole>
cudaError_t go(const NormParams& p, const DeviceInfo& dev, cudaStream_t stream) {
  using S = Shape<T, kTeam, kGroups, kWhole>;
  const auto launch = [&](auto kernel, Fits& known) {
    int fit = 1;
    const cudaError_t e = blocks_that_fit(known, dev, kernel, S::kBlock, S::Rows::kBytes, &fit);
    if (e != cudaSuccess) return e;
    const int64_t need = (static_cast<int64_t>(p.T) + S::kRows - 1) / S::kRows;
    int64_t most = static_cast<int64_t>(dev.sm_count) * fit;
    if (S::kComeAndGo && need / S::kRounds > most) most = need / S::kRounds;
    kernel<<<static_cast<int>(need < most ? need : most), S::kBlock, S::Rows::kBytes, stream>>>(p);
    return cudaGetLastError();
  };
  static Fits known[2];
  return p.format == MAXSIM_NORM_SAME ? launch(rms_norm_kernel<T, kTeam, kGroups, kWhole, false>, known[0])
                                      : launch(rms_norm_kernel<T, kTeam, kGroups, kWhole, true>, known[1]);
}

template <typename T>
cudaError_t pick(const NormParams& p, bool whole, const DeviceInfo& dev, cudaStream_t stream) {
  if (whole) {
    if (p.d <= 64) return go<T, 8, 1, true>(p, dev, stream);
    if (p.d <= 128) return go<T, 8, 2, true>(p, dev, stream);
    if (p.d <= 256) return go<T, 16, 2, true>(p, dev, stream);
    if (p.d <= 512) return go<T, 32, 2, true>(p, dev, stream);
    if (p.d <= 1024) return go<T, 32, 4, true>(p, dev, stream);
    if (p.d <= 2048) return go<T, 128, 2, true>(p, dev, stream);
    if (p.d <= 4096) return go<T, 256, 2, true>(p, dev, stream);
    if (p.d <= 8192) return go<T, 512, 2, true>(p, dev, stream);
    return go<T, 512, 4, true>(p, dev, stream);
  }
  if (p.d <= 256) return go<T, 32, 1, false>(p, dev, stream);
  if (p.d <= 1024) return go<T, 128, 1, false>(p, dev, stream);
  if (p.d <= 4096) return go<T, 256, 2, false>(p, dev, stream);
  return go<T, 512, 4, false>(p, dev, stream);
}

}  // namespace

maxsim_status launch_norm(const NormParams& p, int dtype, bool whole, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  const cudaError_t e = dtype == MAXSIM_BF16   ? pick<__nv_bfloat16>(p, whole, *dev, stream)
                        : dtype == MAXSIM_FP16 ? pick<__half>(p, whole, *dev, stream)
                                               : pick<float>(p, whole, *dev, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

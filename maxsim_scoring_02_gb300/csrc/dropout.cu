// dropout.cu -- dropout of rows from a counter-based generator, and the residual's
// addition; its gradient is the same call on the gradient.
//
//   out = residual + (lot >= limit ? x * factor : 0)
//
// The mask is never stored: rows.cuh makes an element's lot from its place, ten rounds
// of integer products for eight elements, which hide behind their loads (issue slots 58 %
// busy). Bound by HBM with a residual: 98304 x 2048 bf16 179 us (6.8 TB/s), without one 138
// (5.8, instructions and loads alike). Rows that are not whole: 20011 x 1001 fp32 31 us (5.1
// TB/s), 200011 x 1001 bf16 255 (3.1), 2 bytes an access.
#include "rows.cuh"

namespace msim {
namespace {

constexpr int kThreads = 256;
// Groups of eight columns of a thread, and blocks of an SM that the registers have to
// allow. 98304 x 2048 bf16 with a residual, and without: four and four 179 and 138 us,
// three with as many registers as asked for 187 and 150, six 186 and 142. 50000 x 2048
// fp32: three 173 and 133, four and four 231 and 169. Rows that are not whole, 200011 x 1001
// bf16: one 255, two 310.
template <typename T, bool kWhole>
constexpr int kUnits = !kWhole ? 1 : sizeof(T) == 4 ? 3 : 4;
template <typename T, bool kWhole>
constexpr int kFit = kWhole && sizeof(T) == 4 ? 1 : 4;

struct DropoutParams {
  const void *x, *res;
  void* out;
  int64_t x_stride, res_stride, out_stride;
  Drop drop;
  Divisor parts;   // groups (whole) or runs of 256 columns (else) of a row
  uint32_t count;  // of them in this launch
  int row0, d;
};

template <typename T, bool kWhole>
__global__ void __launch_bounds__(kThreads, kFit<T, kWhole>) dropout_kernel(const DropoutParams p) {
  const Key key = load_key(p.drop);
  const int lane = threadIdx.x & 31;
  // a warp's lanes share a run of 256 columns where rows are not whole
  const uint32_t per = kWhole ? kThreads : kThreads / 32, mine = kWhole ? threadIdx.x : threadIdx.x >> 5;
  constexpr int N = kUnits<T, kWhole>;
  // whole groups stay packed until their turn
  std::conditional_t<kWhole, Raw<T>, Eight> x[N], r[N];
  uint32_t row[N], part[N];
  bool live[N];
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const uint32_t n = (blockIdx.x * N + u) * per + mine;
    live[u] = n < p.count;
    const uint32_t q = p.parts.of(live[u] ? n : 0);
    part[u] = (live[u] ? n : 0) - q * p.parts.d;
    row[u] = p.row0 + q;
    const Cols<kWhole> c(part[u], lane, p.d);
    const T *from = static_cast<const T*>(p.x) + row[u] * p.x_stride, *res = static_cast<const T*>(p.res) + row[u] * p.res_stride;
    if constexpr (kWhole) x[u] = load8<T, true>(from, c);
    else x[u] = load_up8<T, false>(from, c);
    if (p.res) {
      if constexpr (kWhole) r[u] = load8<T, true>(res, c);
      else r[u] = load_up8<T, false>(res, c);
    }
  }
#pragma unroll
  for (int u = 0; u < N; ++u) {
    const Cols<kWhole> c(part[u], lane, p.d);
    Eight v, add;
    if constexpr (kWhole) v = up8<T>(x[u]);
    else v = x[u];
    if (p.res) {
      if constexpr (kWhole) add = up8<T>(r[u]);
      else add = r[u];
    }
    if (p.drop.limit) {
      const Kept<kWhole> keep(key, c, row[u], p.drop.limit);
      v = keep.of(v, p.drop.factor, add, p.res != nullptr);
    } else if (p.res) {
#pragma unroll
      for (int i = 0; i < 4; ++i) v.p[i] = add2(v.p[i], add.p[i]);
    }
    if (live[u]) store_down8<T, kWhole>(static_cast<T*>(p.out) + row[u] * p.out_stride, c, v);
  }
}

template <typename T>
maxsim_status run(DropoutParams p, int T_, bool whole, cudaStream_t stream) {
  const uint32_t parts = whole ? p.d / 8 : (p.d + 255) / 256, per = whole ? kThreads : kThreads / 32;
  const int most = static_cast<int>((INT_MAX - 8192) / parts);  // rows of a launch: its parts are counted in 31 bits
  for (int64_t row0 = 0; row0 < T_; row0 += most) {
    const int rows = T_ - row0 < most ? static_cast<int>(T_ - row0) : most;
    p.row0 = static_cast<int>(row0);
    p.count = static_cast<uint32_t>(rows) * parts;
    const uint32_t each = per * (whole ? kUnits<T, true> : kUnits<T, false>);
    const int grid = static_cast<int>((p.count + each - 1) / each);
    if (whole) dropout_kernel<T, true><<<grid, kThreads, 0, stream>>>(p);
    else dropout_kernel<T, false><<<grid, kThreads, 0, stream>>>(p);
    if (cudaGetLastError() != cudaSuccess) return MAXSIM_ERR_CUDA;
  }
  return MAXSIM_OK;
}

}  // namespace

maxsim_status launch_dropout(const maxsim_rows& x, const maxsim_rows* residual, int T, int d, const Drop& drop, int dtype,
                             const maxsim_rows& out, cudaStream_t stream) {
  const int e = dtype == MAXSIM_FP32 ? 4 : 2;
  const bool whole = whole_rows(&x, d, e) && whole_rows(residual, d, e) && whole_rows(&out, d, e);
  DropoutParams p = {x.data, residual ? residual->data : nullptr, out.data, x.row_stride,
                     residual ? residual->row_stride : 0, out.row_stride, drop,
                     Divisor(whole ? d / 8 : (d + 255) / 256), 0, 0, d};
  switch (dtype) {
    case MAXSIM_BF16: return run<__nv_bfloat16>(p, T, whole, stream);
    case MAXSIM_FP16: return run<__half>(p, T, whole, stream);
    default: return run<float>(p, T, whole, stream);
  }
}

}  // namespace msim

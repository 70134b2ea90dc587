// api_layer.cu -- the extern "C" entry points of the operators on rows of hidden
// states: dropout, root-mean-square norms, cross entropy over a vocabulary.
// Argument checks on the host.
#include <climits>
#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "loss.cuh"
#include "norm.cuh"

using namespace msim;

namespace {

constexpr int64_t kMaxStride = int64_t(1) << 38;

bool multiple(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }
bool known(maxsim_dtype t) { return t == MAXSIM_BF16 || t == MAXSIM_FP16 || t == MAXSIM_FP32; }
int size_of(maxsim_dtype t) { return t == MAXSIM_FP32 ? 4 : 2; }

// A view of T rows of d elements of e bytes.
struct View {
  const maxsim_rows* v;
  int64_t T, d;
  int e;
  bool given() const { return v && v->data; }
  // Readable: aligned to its elements, any stride from 0 on (rows may coincide).
  bool readable() const {
    return given() && multiple(v->data, e) && v->row_stride >= 0 && v->row_stride < kMaxStride;
  }
  // Written: no two rows share an element.
  bool writable() const { return readable() && (T <= 1 || v->row_stride >= d); }
  int64_t stride() const { return v->row_stride * e; }
  uintptr_t first() const { return reinterpret_cast<uintptr_t>(v->data); }
  uintptr_t last() const { return first() + ((T - 1) * v->row_stride + d) * e; }  // one past
};

// Whether a view that is written leaves another one alone: it is the same rows of
// elements of the same size (each is read by the thread that writes it, before),
// lies elsewhere, or has other columns of the same rows.
bool apart(const View& a, const View& b, bool may_be_same = true) {
  if (!a.given() || !b.given()) return true;
  if (may_be_same && a.first() == b.first() && a.e == b.e && (a.T <= 1 || a.stride() == b.stride())) return true;
  if (a.last() <= b.first() || b.last() <= a.first()) return true;
  if (a.T <= 1 || a.stride() != b.stride()) return false;
  const int64_t step = a.stride();
  int64_t off = static_cast<int64_t>(b.first() - a.first()) % step;
  if (off < 0) off += step;
  return off >= a.d * a.e && off + b.d * b.e <= step;
}

// The same for n elements of e bytes in a row: no byte between the view's first and last.
bool apart(const View& a, const void* p, int64_t n, int e) {
  const uintptr_t first = reinterpret_cast<uintptr_t>(p);
  return !a.given() || !p || a.last() <= first || first + n * e <= a.first();
}

// The same for other memory that the call reads or writes: `size` bytes at p.
struct Bytes {
  const void* p;
  size_t size;
  uintptr_t first() const { return reinterpret_cast<uintptr_t>(p); }
};
bool apart(const Bytes& a, const Bytes& b) {
  return !a.p || !b.p || a.first() + a.size <= b.first() || b.first() + b.size <= a.first();
}
// Whether a workspace, or a row of results, leaves all views and all other memory of its call alone.
bool alone(const Bytes& a, std::initializer_list<const View*> views, std::initializer_list<Bytes> others) {
  for (const View* v : views)
    if (!apart(*v, a.p, static_cast<int64_t>(a.size), 1)) return false;
  for (const Bytes& b : others)
    if (!apart(a, b)) return false;
  return true;
}

// The chance of being dropped as a limit of 16-bit lots.
bool drop_of(float p, const int64_t* rng, Drop& drop) {
  drop = {rng, 0, 1.f};
  if (!(p >= 0.f && p < 1.f)) return false;
  const long limit = std::lrint(static_cast<double>(p) * 65536.);
  if (limit > 65535) return false;
  drop.limit = static_cast<uint32_t>(limit);
  drop.factor = static_cast<float>(65536. / (65536. - limit));
  return limit == 0 || (rng && multiple(rng, 8));
}

maxsim_status check_norm(const maxsim_norm_spec* s, Drop& drop) {
  if (!s || s->T < 0 || s->d < 1 || !known(s->dtype) || !multiple(s->weight, 2)) return MAXSIM_ERR_INVALID_ARG;
  if (s->weight && s->weight_dtype != MAXSIM_FP32 && s->weight_dtype != s->dtype) return MAXSIM_ERR_INVALID_ARG;
  if (s->weight && !multiple(s->weight, size_of(s->weight_dtype))) return MAXSIM_ERR_INVALID_ARG;
  if (s->format != MAXSIM_NORM_SAME && s->format != MAXSIM_NORM_INT8 && s->format != MAXSIM_NORM_E4M3)
    return MAXSIM_ERR_INVALID_ARG;
  if (!(s->eps >= 0x1p-60f && s->eps <= 0x1p60f)) return MAXSIM_ERR_INVALID_ARG;
  if (!drop_of(s->p, s->rng, drop)) return MAXSIM_ERR_INVALID_ARG;
  if (s->T >= INT_MAX - 256 || s->d > kMaxNormWidth) return MAXSIM_ERR_UNSUPPORTED;
  return MAXSIM_OK;
}

maxsim_status check_loss(const maxsim_loss_spec* s, LossShape& shape) {
  if (!s || s->T < 0 || s->V < 1 || s->d < 1 || !known(s->dtype)) return MAXSIM_ERR_INVALID_ARG;
  if (!(s->scale > 0.f) || !std::isfinite(s->scale)) return MAXSIM_ERR_INVALID_ARG;
  if (s->dtype == MAXSIM_FP32 || s->d % 8 != 0 || s->d > 65536 || s->T >= INT_MAX - 256 || s->V >= INT_MAX - 256 ||
      s->scale > 0x1p60f || s->scale < 0x1p-60f)
    return MAXSIM_ERR_UNSUPPORTED;
  if (s->T > 0 && (!s->targets || !multiple(s->targets, 8))) return MAXSIM_ERR_INVALID_ARG;
  shape = {s->V, static_cast<int>(s->T), s->d, s->dtype == MAXSIM_BF16, s->scale};
  return MAXSIM_OK;
}

// A view that TMA can address.
bool fits(const maxsim_rows* v, int64_t rows, int64_t d) {
  return v && v->data && multiple(v->data, 16) && v->row_stride % 8 == 0 && v->row_stride > 0 &&
         v->row_stride < kMaxStride && (rows <= 1 || v->row_stride >= d);
}

}  // namespace

extern "C" {

maxsim_status maxsim_dropout(const maxsim_rows* x, const maxsim_rows* residual, int64_t T, int32_t d, float p,
                             const int64_t* rng, maxsim_dtype dtype, const maxsim_rows* out, void* stream) {
  Drop drop;
  if (T < 0 || d < 1 || !known(dtype) || !drop_of(p, rng, drop)) return MAXSIM_ERR_INVALID_ARG;
  if (T >= INT_MAX - 256 || d >= INT_MAX - 256) return MAXSIM_ERR_UNSUPPORTED;
  if (T == 0) return MAXSIM_OK;
  const int e = size_of(dtype);
  const View vx{x, T, d, e}, vr{residual, T, d, e}, vo{out, T, d, e};
  if (!vx.readable() || (residual && !vr.readable()) || !vo.writable()) return MAXSIM_ERR_INVALID_ARG;
  if (!apart(vo, vx) || !apart(vo, vr) || (drop.limit && !apart(vo, rng, 2, 8))) return MAXSIM_ERR_INVALID_ARG;
  return launch_dropout(*x, residual, static_cast<int>(T), d, drop, dtype, *out, static_cast<cudaStream_t>(stream));
}

maxsim_status maxsim_rms_norm(const maxsim_norm_spec* spec, const maxsim_rows* x, const maxsim_rows* residual,
                              const maxsim_rows* sum, const maxsim_rows* out, float* scale, void* stream) {
  Drop drop;
  const maxsim_status st = check_norm(spec, drop);
  if (st != MAXSIM_OK || spec->T == 0) return st;
  const int e = size_of(spec->dtype), eo = spec->format == MAXSIM_NORM_SAME ? e : 1, d = spec->d;
  const int64_t T = spec->T;
  const View vx{x, T, d, e}, vr{residual, T, d, e}, vs{sum, T, d, e}, vo{out, T, d, eo};
  if (!vx.readable() || (residual && !vr.readable()) || (sum && !vs.writable()) || !vo.writable())
    return MAXSIM_ERR_INVALID_ARG;
  if (!apart(vo, vx) || !apart(vo, vr) || !apart(vo, vs, false) || !apart(vs, vx) || !apart(vs, vr))
    return MAXSIM_ERR_INVALID_ARG;
  if (spec->format == MAXSIM_NORM_SAME) scale = nullptr;
  else if (!scale || !multiple(scale, 4)) return MAXSIM_ERR_INVALID_ARG;
  for (const View* v : {&vx, &vr, &vs, &vo})
    if (!apart(*v, scale, T, 4)) return MAXSIM_ERR_INVALID_ARG;
  const Bytes weight{spec->weight, static_cast<size_t>(d) * size_of(spec->weight_dtype)}, rng{drop.limit ? spec->rng : nullptr, 16};
  if (!alone(weight, {&vs, &vo}, {}) || !alone(rng, {&vs, &vo}, {}) || !alone({scale, static_cast<size_t>(T) * 4}, {}, {weight, rng}))
    return MAXSIM_ERR_INVALID_ARG;
  NormParams p = {};
  p.x = x->data, p.x_stride = x->row_stride;
  if (residual) p.res = residual->data, p.res_stride = residual->row_stride;
  if (sum) p.sum = sum->data, p.sum_stride = sum->row_stride;
  p.out = out->data, p.out_stride = out->row_stride;
  p.weight = spec->weight;
  p.weight_fp32 = spec->weight_dtype == MAXSIM_FP32;
  p.scale = scale;
  p.T = static_cast<int>(T), p.d = d, p.per = 1.f / d, p.format = spec->format, p.eps = spec->eps, p.drop = drop;
  const bool whole = whole_rows(x, d, e) && whole_rows(residual, d, e) && whole_rows(sum, d, e) &&
                     whole_rows(out, d, eo) && multiple(spec->weight, 16);
  return launch_norm(p, spec->dtype, whole, static_cast<cudaStream_t>(stream));
}

size_t maxsim_rms_norm_backward_workspace_size(const maxsim_norm_spec* spec) {
  Drop drop;
  if (check_norm(spec, drop) != MAXSIM_OK || !spec->weight) return 0;
  return norm_bwd_workspace_bytes(static_cast<int>(spec->T), spec->d);
}

maxsim_status maxsim_rms_norm_backward(const maxsim_norm_spec* spec, const maxsim_rows* dy, const maxsim_rows* h,
                                       const maxsim_rows* dsum, const maxsim_rows* dx, const maxsim_rows* dresidual,
                                       void* dweight, void* workspace, size_t workspace_bytes, void* stream) {
  Drop drop;
  const maxsim_status st = check_norm(spec, drop);
  if (st != MAXSIM_OK) return st;
  if (spec->format != MAXSIM_NORM_SAME || (dweight && !spec->weight)) return MAXSIM_ERR_INVALID_ARG;
  const int ew = size_of(spec->weight_dtype);
  if (!multiple(dweight, ew)) return MAXSIM_ERR_INVALID_ARG;
  const cudaStream_t s = static_cast<cudaStream_t>(stream);
  if (spec->T == 0)  // no rows: their sum is 0
    return dweight && cudaMemsetAsync(dweight, 0, static_cast<size_t>(spec->d) * ew, s) != cudaSuccess ? MAXSIM_ERR_CUDA
                                                                                                      : MAXSIM_OK;
  const int e = size_of(spec->dtype), d = spec->d;
  const int64_t T = spec->T;
  const View vy{dy, T, d, e}, vh{h, T, d, e}, vm{dsum, T, d, e}, vx{dx, T, d, e}, vr{dresidual, T, d, e};
  if (!vy.readable() || !vh.readable() || (dsum && !vm.readable()) || (dx && !vx.writable()) ||
      (dresidual && !vr.writable()))
    return MAXSIM_ERR_INVALID_ARG;
  for (const View* w : {&vx, &vr})
    if (!apart(*w, vy) || !apart(*w, vh) || !apart(*w, vm) || !apart(*w, spec->weight, d, ew) || !apart(*w, dweight, d, ew))
      return MAXSIM_ERR_INVALID_ARG;
  const Bytes weight{spec->weight, static_cast<size_t>(d) * ew}, sums{dweight, static_cast<size_t>(d) * ew},
      rng{drop.limit ? spec->rng : nullptr, 16};
  if (!apart(vx, vr, false) || !alone(rng, {&vx, &vr}, {sums})) return MAXSIM_ERR_INVALID_ARG;
  const size_t need = norm_bwd_workspace_bytes(static_cast<int>(T), d);
  if (dweight && (!workspace || !multiple(workspace, 16) || workspace_bytes < need)) return MAXSIM_ERR_WORKSPACE;
  if (dweight && !alone({workspace, need}, {&vy, &vh, &vm, &vx, &vr}, {weight, sums, rng})) return MAXSIM_ERR_INVALID_ARG;
  NormParams p = {};
  p.x = dy->data, p.x_stride = dy->row_stride;
  p.res = h->data, p.res_stride = h->row_stride;
  if (dsum) p.more = dsum->data, p.more_stride = dsum->row_stride;
  if (dresidual) p.sum = dresidual->data, p.sum_stride = dresidual->row_stride;
  if (dx) p.out = dx->data, p.out_stride = dx->row_stride;
  p.weight = spec->weight;
  p.weight_fp32 = spec->weight_dtype == MAXSIM_FP32;
  p.parts = dweight ? static_cast<float*>(workspace) : nullptr;
  p.T = static_cast<int>(T), p.d = d, p.per = 1.f / d, p.eps = spec->eps, p.drop = drop;
  const bool whole = whole_rows(dy, d, e) && whole_rows(h, d, e) && whole_rows(dsum, d, e) && whole_rows(dx, d, e) &&
                     whole_rows(dresidual, d, e) && multiple(spec->weight, 16);
  return launch_norm_bwd(p, spec->dtype, whole, dweight, s);
}

size_t maxsim_cross_entropy_workspace_size(const maxsim_loss_spec* spec) {
  LossShape s;
  return check_loss(spec, s) != MAXSIM_OK || s.T == 0 ? 0 : loss_workspace_bytes(s);
}

maxsim_status maxsim_cross_entropy(const maxsim_loss_spec* spec, const maxsim_rows* x, const maxsim_rows* weight,
                                   float* loss, float* lse, void* workspace, size_t workspace_bytes, void* stream) {
  LossShape s;
  const maxsim_status st = check_loss(spec, s);
  if (st != MAXSIM_OK || s.T == 0) return st;
  if (!fits(x, s.T, s.d) || !fits(weight, s.V, s.d) || !loss || !lse || !multiple(loss, 4) || !multiple(lse, 4))
    return MAXSIM_ERR_INVALID_ARG;
  const View vx{x, s.T, s.d, 2}, vw{weight, s.V, s.d, 2};
  const maxsim_rows first{loss, 0}, second{lse, 0}, labels{const_cast<int64_t*>(spec->targets), 0};
  const View vl{&first, 1, s.T, 4}, ve{&second, 1, s.T, 4}, vt{&labels, 1, s.T, 8};
  for (const View* v : {&vl, &ve})
    if (!apart(*v, vx, false) || !apart(*v, vw, false) || !apart(*v, vt, false)) return MAXSIM_ERR_INVALID_ARG;
  if (!apart(vl, ve, false)) return MAXSIM_ERR_INVALID_ARG;
  const size_t need = loss_workspace_bytes(s);
  if (!workspace || !multiple(workspace, 16) || workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
  if (!alone({workspace, need}, {&vx, &vw, &vl, &ve, &vt}, {})) return MAXSIM_ERR_INVALID_ARG;
  return launch_loss(s, *x, *weight, spec->targets, loss, lse, workspace, static_cast<cudaStream_t>(stream));
}

size_t maxsim_cross_entropy_backward_workspace_size(const maxsim_loss_spec* spec) {
  LossShape s;
  return check_loss(spec, s) != MAXSIM_OK || s.T == 0 ? 0 : loss_bwd_workspace_bytes(s);
}

maxsim_status maxsim_cross_entropy_backward(const maxsim_loss_spec* spec, const float* dloss, const maxsim_rows* x,
                                            const maxsim_rows* weight, const float* lse, const maxsim_rows* dx,
                                            const maxsim_rows* dweight, void* workspace, size_t workspace_bytes,
                                            void* stream) {
  LossShape s;
  const maxsim_status st = check_loss(spec, s);
  if (st != MAXSIM_OK) return st;
  if (dweight && !fits(dweight, s.V, s.d)) return MAXSIM_ERR_INVALID_ARG;
  const cudaStream_t on = static_cast<cudaStream_t>(stream);
  if (s.T == 0)  // no rows: their sum is 0
    return dweight && cudaMemset2DAsync(dweight->data, static_cast<size_t>(dweight->row_stride) * 2, 0,
                                        static_cast<size_t>(s.d) * 2, static_cast<size_t>(s.V), on) != cudaSuccess
               ? MAXSIM_ERR_CUDA
               : MAXSIM_OK;
  if (!fits(x, s.T, s.d) || !fits(weight, s.V, s.d) || (dx && !fits(dx, s.T, s.d)) || !dloss || !lse ||
      !multiple(dloss, 4) || !multiple(lse, 4))
    return MAXSIM_ERR_INVALID_ARG;
  // operands are read by several blocks: a gradient may lie in none of them
  const View vx{x, s.T, s.d, 2}, vw{weight, s.V, s.d, 2}, vdx{dx, s.T, s.d, 2}, vdw{dweight, s.V, s.d, 2};
  for (const View* a : {&vdx, &vdw})
    if (!apart(*a, vx, false) || !apart(*a, vw, false) || !apart(*a, dloss, s.T, 4) || !apart(*a, lse, s.T, 4) ||
        !apart(*a, spec->targets, s.T, 8))
      return MAXSIM_ERR_INVALID_ARG;
  if (!apart(vdx, vdw, false)) return MAXSIM_ERR_INVALID_ARG;
  if (!dx && !dweight) return MAXSIM_OK;
  const size_t need = loss_bwd_workspace_bytes(s), row = static_cast<size_t>(s.T) * 4;
  if (!workspace || !multiple(workspace, 256) || workspace_bytes < need) return MAXSIM_ERR_WORKSPACE;
  if (!alone({workspace, need}, {&vx, &vw, &vdx, &vdw}, {{dloss, row}, {lse, row}, {spec->targets, 2 * row}}))
    return MAXSIM_ERR_INVALID_ARG;
  return launch_loss_bwd(s, dloss, *x, *weight, spec->targets, lse, dx, dweight, workspace, on);
}

}  // extern "C"

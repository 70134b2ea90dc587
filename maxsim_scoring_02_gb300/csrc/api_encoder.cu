// api_encoder.cu -- the extern "C" entry points of the token-encoder
// operators (rotary positions, packed attention, gradient clipping): argument
// checks on the host, and the frequency table.
#include <climits>
#include <cmath>
#include <cstdint>

#include "attn_common.cuh"
#include "internal.h"

using namespace msim;

namespace {

constexpr double kTwoPi = 6.283185307179586476925286766559;
constexpr int64_t kMaxStride = int64_t(1) << 39;
constexpr float kLargest = 0x1p60f;  // of scale and cap, and of their reciprocals: the kernels' constants made of them
                                     // (scale / cap, cap log2(e)) then neither overflow nor lose bits

bool multiple(const void* p, uintptr_t bytes) { return reinterpret_cast<uintptr_t>(p) % bytes == 0; }

bool known(maxsim_dtype t) { return t == MAXSIM_BF16 || t == MAXSIM_FP16 || t == MAXSIM_FP32; }

// A view whose rows the TMA can address.
bool fits(const maxsim_heads* v) {
  return v && v->data && multiple(v->data, 16) && v->token_stride > 0 && v->head_stride > 0 &&
         v->token_stride % 8 == 0 && v->head_stride % 8 == 0 && v->token_stride < kMaxStride &&
         v->head_stride < kMaxStride;
}

// No two rows of a view that is written share an element: the longer stride
// steps over all that the shorter one reaches.
bool apart(const maxsim_heads* v, int64_t T, int heads, int d) {
  if ((heads > 1 && v->head_stride < d) || (T > 1 && v->token_stride < d)) return false;
  if (heads == 1 || T == 1) return true;
  const bool tokens_outside = v->head_stride <= v->token_stride;
  const int64_t near = tokens_outside ? v->head_stride : v->token_stride, n = tokens_outside ? heads : T;
  const int64_t far = tokens_outside ? v->token_stride : v->head_stride;
  return (far - d) / near >= n - 1;  // far >= (n - 1) * near + d
}

// Checks of a spec that both directions share. MAXSIM_OK with T == 0 means that
// there is nothing to do.
maxsim_status check_spec(const maxsim_attention_spec* s) {
  if (!s || s->T < 0 || s->B < 0 || s->heads < 1 || s->kv_heads < 1 || s->d < 1 || !known(s->dtype))
    return MAXSIM_ERR_INVALID_ARG;
  if (s->mask != MAXSIM_MASK_FULL && s->mask != MAXSIM_MASK_CAUSAL && s->mask != MAXSIM_MASK_PREFIX)
    return MAXSIM_ERR_INVALID_ARG;
  if (!(s->scale > 0.f) || !std::isfinite(s->scale) || !std::isfinite(s->cap)) return MAXSIM_ERR_INVALID_ARG;
  if (s->heads % s->kv_heads != 0) return MAXSIM_ERR_INVALID_ARG;
  if (s->dtype == MAXSIM_FP32 || s->d % 8 != 0 || s->d > 128 || s->heads > 65535 || s->T >= INT_MAX - 256 ||
      s->B >= INT_MAX)
    return MAXSIM_ERR_UNSUPPORTED;
  if (s->scale > kLargest || s->scale < 1.f / kLargest || (s->cap > 0.f && (s->cap > kLargest || s->cap < 1.f / kLargest)))
    return MAXSIM_ERR_UNSUPPORTED;
  if (s->T == 0) return MAXSIM_OK;
  if (s->B == 0) return MAXSIM_ERR_INVALID_ARG;  // tokens, and no document that holds them
  if (!s->offsets || !multiple(s->offsets, 8) || !multiple(s->key_len, 4) || !multiple(s->prefix_len, 4) ||
      !multiple(s->slopes, 4) || (s->mask == MAXSIM_MASK_PREFIX && !s->prefix_len))
    return MAXSIM_ERR_INVALID_ARG;
  return MAXSIM_OK;
}

AttnParams params_of(const maxsim_attention_spec* s) {
  AttnParams p = {};
  p.offsets = s->offsets;
  p.key_len = s->key_len;
  p.prefix_len = s->prefix_len;
  p.slopes = s->slopes;
  p.B = s->B;
  p.T = static_cast<int>(s->T);
  p.heads = s->heads;
  p.kv_heads = s->kv_heads;
  p.d = s->d;
  p.mask = s->mask;
  p.scale = s->scale;
  p.cap = s->cap > 0.f ? s->cap : 0.f;
  return p;
}

size_t delta_bytes(const maxsim_attention_spec* s) {
  return static_cast<size_t>(s->T) * s->heads * 2 * sizeof(float);
}

}  // namespace

extern "C" {

maxsim_status maxsim_rotary_frequencies(int rot_dim, double base, maxsim_rotary_scaling scaling, double factor,
                                        int64_t original_length, uint64_t* freq_host, float* amplitude) {
  if (rot_dim < 2 || rot_dim % 2 != 0 || !(base > 1.) || !std::isfinite(base) || !freq_host || !amplitude)
    return MAXSIM_ERR_INVALID_ARG;
  if (scaling != MAXSIM_ROTARY_NONE && (!(factor >= 1.) || !std::isfinite(factor))) return MAXSIM_ERR_INVALID_ARG;
  double low = 0., high = 0.;
  *amplitude = 1.f;
  switch (scaling) {
    case MAXSIM_ROTARY_NONE:
    case MAXSIM_ROTARY_LINEAR: break;
    case MAXSIM_ROTARY_NTK:
      if (rot_dim < 4) return MAXSIM_ERR_INVALID_ARG;
      base *= std::pow(factor, rot_dim / (rot_dim - 2.));
      break;
    case MAXSIM_ROTARY_YARN: {
      if (original_length < 1) return MAXSIM_ERR_INVALID_ARG;
      // the pair that turns `turns` times within the original length
      const auto pair = [&](double turns) {
        return rot_dim * std::log(original_length / (turns * kTwoPi)) / (2. * std::log(base));
      };
      low = std::fmax(0., std::floor(pair(32.)));
      high = std::fmin(rot_dim - 1., std::ceil(pair(1.)));
      *amplitude = static_cast<float>(0.1 * std::log(factor) + 1.);
      break;
    }
    default: return MAXSIM_ERR_INVALID_ARG;
  }
  for (int i = 0; i < rot_dim / 2; ++i) {
    double theta = std::pow(base, -2. * i / rot_dim);
    if (scaling == MAXSIM_ROTARY_LINEAR) theta /= factor;
    if (scaling == MAXSIM_ROTARY_YARN) {
      const double ramp = std::fmin(1., std::fmax(0., (i - low) / std::fmax(high - low, 1e-3)));
      theta = theta * (1. - ramp) + theta / factor * ramp;
    }
    freq_host[i] = static_cast<uint64_t>(std::ldexp(theta / kTwoPi, 64));  // theta <= 1: below 2^62
  }
  return MAXSIM_OK;
}

maxsim_status maxsim_rotary(const maxsim_heads* x, int64_t T, int heads, int d, int rot_dim, const uint64_t* freq,
                            const int64_t* offsets, int64_t B, const int32_t* positions, int interleaved,
                            float amplitude, int inverse, maxsim_dtype dtype, const maxsim_heads* out, void* stream) {
  if (!x || !out || T < 0 || B < 0 || heads < 1 || d < 1 || rot_dim < 2 || rot_dim % 2 != 0 || rot_dim > d ||
      !known(dtype) || !std::isfinite(amplitude))
    return MAXSIM_ERR_INVALID_ARG;
  if (offsets && positions) return MAXSIM_ERR_INVALID_ARG;
  if (d > 4096 || heads > 65535 || T >= INT_MAX || B >= INT_MAX) return MAXSIM_ERR_UNSUPPORTED;
  if (T == 0) return MAXSIM_OK;
  if (offsets && B == 0) return MAXSIM_ERR_INVALID_ARG;  // tokens, and no document that holds them
  const uintptr_t e = dtype == MAXSIM_FP32 ? 4 : 2;
  if (!x->data || !out->data || !freq || !multiple(x->data, e) || !multiple(out->data, e) || !multiple(freq, 8) ||
      !multiple(offsets, 8) || !multiple(positions, 4))
    return MAXSIM_ERR_INVALID_ARG;
  if (x->token_stride < 0 || x->head_stride < 0 || out->token_stride < 0 || out->head_stride < 0 ||
      x->token_stride >= kMaxStride || x->head_stride >= kMaxStride || out->token_stride >= kMaxStride ||
      out->head_stride >= kMaxStride)
    return MAXSIM_ERR_INVALID_ARG;
  if (!apart(out, T, heads, d)) return MAXSIM_ERR_INVALID_ARG;
  if (x->data == out->data && (x->token_stride != out->token_stride || x->head_stride != out->head_stride))
    return MAXSIM_ERR_INVALID_ARG;
  return launch_rotary(*x, T, heads, d, rot_dim, freq, offsets, B, positions, interleaved, amplitude, inverse, dtype,
                       *out, static_cast<cudaStream_t>(stream));
}

maxsim_status maxsim_attention(const maxsim_attention_spec* spec, const maxsim_heads* q, const maxsim_heads* k,
                               const maxsim_heads* v, const maxsim_heads* out, float* lse, void* stream) {
  maxsim_status st = check_spec(spec);
  if (st != MAXSIM_OK || spec->T == 0) return st;
  if (!fits(q) || !fits(k) || !fits(v) || !fits(out) || !multiple(lse, 4)) return MAXSIM_ERR_INVALID_ARG;
  if (!apart(out, spec->T, spec->heads, spec->d)) return MAXSIM_ERR_INVALID_ARG;
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  AttnParams p = params_of(spec);
  p.status = dev->status;
  p.q = *q;
  p.k = *k;
  p.v = *v;
  p.out = *out;
  p.lse = lse;
  return launch_attn_fwd(p, spec->dtype == MAXSIM_BF16, static_cast<cudaStream_t>(stream));
}

size_t maxsim_attention_backward_workspace_size(const maxsim_attention_spec* spec) {
  if (check_spec(spec) != MAXSIM_OK) return 0;
  return delta_bytes(spec) + (spec->dtype == MAXSIM_FP16 ? static_cast<size_t>(spec->T) * sizeof(float2) : 0);
}

maxsim_status maxsim_attention_backward(const maxsim_attention_spec* spec, const maxsim_heads* dO,
                                        const maxsim_heads* q, const maxsim_heads* k, const maxsim_heads* v,
                                        const maxsim_heads* out, const float* lse, const maxsim_heads* dq,
                                        const maxsim_heads* dk, const maxsim_heads* dv, void* workspace,
                                        size_t workspace_bytes, void* stream) {
  maxsim_status st = check_spec(spec);
  if (st != MAXSIM_OK || spec->T == 0) return st;
  if (!fits(dO) || !fits(q) || !fits(k) || !fits(v) || !fits(out) || !fits(dq) || !fits(dk) || !fits(dv) || !lse ||
      !multiple(lse, 4))
    return MAXSIM_ERR_INVALID_ARG;
  if (!apart(dq, spec->T, spec->heads, spec->d) || !apart(dk, spec->T, spec->kv_heads, spec->d) ||
      !apart(dv, spec->T, spec->kv_heads, spec->d))
    return MAXSIM_ERR_INVALID_ARG;
  if (!workspace || !multiple(workspace, 16) || workspace_bytes < maxsim_attention_backward_workspace_size(spec))
    return MAXSIM_ERR_WORKSPACE;
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  AttnParams p = params_of(spec);
  p.status = dev->status;
  p.dO = *dO;
  p.q = *q;
  p.k = *k;
  p.v = *v;
  p.out = *out;
  p.lse = const_cast<float*>(lse);
  p.dq = *dq;
  p.dk = *dk;
  p.dv = *dv;
  p.delta = static_cast<float*>(workspace);
  if (spec->dtype == MAXSIM_FP16) p.shifts = reinterpret_cast<float2*>(static_cast<char*>(workspace) + delta_bytes(spec));
  return launch_attn_bwd(p, spec->dtype == MAXSIM_BF16, static_cast<cudaStream_t>(stream));
}

size_t maxsim_clip_grad_norm_workspace_size(int n_tensors) {
  return n_tensors < 0 ? 0 : clip_workspace_bytes(n_tensors);
}

maxsim_status maxsim_clip_grad_norm(const void* const* grads, void* const* outs, const int64_t* sizes,
                                    const int32_t* dtypes, int n_tensors, float max_norm, float* norm,
                                    void* workspace, size_t workspace_bytes, void* stream) {
  if (n_tensors < 0 || !norm || !multiple(norm, 4) || !(max_norm >= 0.f)) return MAXSIM_ERR_INVALID_ARG;
  if (n_tensors > 0 && (!grads || !outs || !sizes || !dtypes)) return MAXSIM_ERR_INVALID_ARG;
  for (int i = 0; i < n_tensors; ++i) {
    if (sizes[i] < 0 || sizes[i] > (int64_t(1) << 46) || !known(static_cast<maxsim_dtype>(dtypes[i])))
      return MAXSIM_ERR_INVALID_ARG;
    const uintptr_t e = dtypes[i] == MAXSIM_FP32 ? 4 : 2;
    if (sizes[i] > 0 && (!grads[i] || !outs[i] || !multiple(grads[i], e) || !multiple(outs[i], e)))
      return MAXSIM_ERR_INVALID_ARG;
  }
  if (!workspace || !multiple(workspace, 16) || workspace_bytes < clip_workspace_bytes(n_tensors))
    return MAXSIM_ERR_WORKSPACE;
  return launch_clip(grads, outs, sizes, dtypes, n_tensors, max_norm, norm, workspace,
                     static_cast<cudaStream_t>(stream));
}

}  // extern "C"

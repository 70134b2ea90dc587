// attn_common.cuh -- what the packed-attention kernels share: the parameters
// of a call, the document that a token belongs to, and which keys a row sees.
//
// Documents are CSR-packed: document b owns tokens offsets[b] ..
// offsets[b+1]-1 of the T packed ones. With i and j counted within the
// document, row i sees key j when j < key_len[b] and
//   full:    always
//   causal:  j <= i
//   prefix:  j <= i or j < prefix_len[b]
// so the keys that a row sees are always the interval [0, row_end(i)).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "internal.h"
#include "ptx.cuh"

namespace msim {

using HeadsView = maxsim_heads;

struct AttnParams {
  HeadsView q, k, v, out, dO, dq, dk, dv;
  float* lse;    // [heads, T] natural log of the softmax denominators, or null
  float* delta;  // [heads, T] rowsum(dO * out), backward only
  const int64_t* offsets;
  const int32_t* key_len;
  const int32_t* prefix_len;
  const float* slopes;
  unsigned* status;
  int64_t B;
  int T, heads, kv_heads, d, mask;
  float scale, cap;
};

struct Doc {
  int start, len, keys, prefix;  // keys: how many of the document's keys are not hidden
};

// The document's extent, with everything clamped into range. A document whose
// offsets are inconsistent is empty; `bad` reports it.
__device__ __forceinline__ Doc load_doc(const AttnParams& p, int64_t b, bool& bad) {
  const int64_t s = p.offsets[b], e = p.offsets[b + 1];
  Doc r;
  bad = s < 0 || e < s || e > p.T || (b > 0 && p.offsets[b - 1] > s);
  r.start = bad ? 0 : static_cast<int>(s);
  r.len = bad ? 0 : static_cast<int>(e - s);
  r.keys = r.len;
  r.prefix = 0;
  if (p.key_len) {
    const int n = p.key_len[b];
    bad |= n < 0 || n > r.len;
    r.keys = n < 0 ? 0 : min(n, r.len);
  }
  if (p.mask == MAXSIM_MASK_PREFIX) {
    const int n = p.prefix_len[b];
    bad |= n < 0;
    r.prefix = max(0, min(n, r.keys));
  }
  return r;
}

// Every document is looked at once by one of a kernel's threads, also those
// that no tile leads to.
__device__ __forceinline__ void check_docs(const AttnParams& p, int64_t thread, int64_t threads) {
  for (int64_t b = thread; b < p.B; b += threads) {
    bool bad;
    load_doc(p, b, bad);
    bad |= b == 0 && p.offsets[0] != 0;
    bad |= b == p.B - 1 && p.offsets[p.B] != p.T;
    if (bad) atomicOr(p.status, kDevErrBadInput);
  }
}

// Row i of the document sees keys [0, row_end).
__device__ __forceinline__ int row_end(const Doc& c, int mask, int i) {
  if (mask == MAXSIM_MASK_FULL) return c.keys;
  return min(c.keys, max(i + 1, c.prefix));
}
// Key j (< keys) is seen by rows [key_begin, len).
__device__ __forceinline__ int key_begin(const Doc& c, int mask, int j) {
  return mask == MAXSIM_MASK_FULL || j < c.prefix ? 0 : j;
}

}  // namespace msim

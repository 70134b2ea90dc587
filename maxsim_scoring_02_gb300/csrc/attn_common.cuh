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
#include "attn_ptx.cuh"
#include "pair.cuh"

namespace msim {

using HeadsView = maxsim_heads;

struct AttnParams {
  HeadsView q, k, v, out, dO, dq, dk, dv;
  float* lse;    // [heads, T] natural log of the softmax denominators, or null
  float* delta;  // [heads, T] pairs (-lse in log2 units, -<dO, out>), backward only
  float2* shifts;  // [T] (shift, 2^-shift): P and dS are held times 2^shift; backward in fp16 only
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

// ------------------------------------------------ tiles for the tensor cores
//
// Work is cut into slots of R rows. Document b owns the slots from
// offsets[b] / R + b on: as many as its rows can touch, so the slots of all
// documents are known without a sum over their lengths (T / R + B in all). A
// slot past its document's last row is empty.
__device__ __forceinline__ int64_t slot_base(const AttnParams& p, int64_t b, int rows) {
  const int64_t s = p.offsets[b];
  return (s < 0 ? 0 : s > p.T ? p.T : s) / rows + b;
}

// The last document whose slots begin at or before `slot`, for each lane's own
// slot: 32 places are looked at together, the rest of the way alone.
__device__ __forceinline__ int64_t slot_doc(const AttnParams& p, int64_t slot, int rows) {
  const int lane = threadIdx.x & 31;
  int64_t lo = 0, hi = p.B;
  const int64_t step = (hi + 31) / 32;
  const int64_t mine = lane * step < p.B ? slot_base(p, lane * step, rows) : INT64_MAX;
  int at = 0;
#pragma unroll
  for (int k = 16; k; k >>= 1)
    if (__shfl_sync(0xffffffffu, mine, at + k) <= slot) at += k;
  lo = at * step;
  hi = lo + step < hi ? lo + step : hi;
  while (hi - lo > 1) {
    const int64_t m = lo + (hi - lo) / 2;
    if (slot_base(p, m, rows) <= slot) lo = m;
    else hi = m;
  }
  return lo;
}

// One block's next piece of work, and what it needs to know of its document.
struct Work {
  int start, len, keys, prefix;  // Doc
  int row0;                      // first row (or key) of the slot, within the document
  int head;
  int live;                      // 0: no work is left
};

// A piece of work read from shared memory, known to be the same in all lanes.
__device__ __forceinline__ Work uniform_work(const Work& a) {
  Work w;
  w.start = __shfl_sync(0xffffffffu, a.start, 0);
  w.len = __shfl_sync(0xffffffffu, a.len, 0);
  w.keys = __shfl_sync(0xffffffffu, a.keys, 0);
  w.prefix = __shfl_sync(0xffffffffu, a.prefix, 0);
  w.row0 = __shfl_sync(0xffffffffu, a.row0, 0);
  w.head = __shfl_sync(0xffffffffu, a.head, 0);
  w.live = __shfl_sync(0xffffffffu, a.live, 0);
  return w;
}

constexpr int kRing = 4;  // pieces of work that are planned ahead

// One warp finds the block's pieces of work, 32 at a time, since each takes a
// chain of dependent reads, and hands them to the other roles through a ring.
// Block c of G takes (slot, head) pairs c, 2G - 1 - c, 2G + c, ..., so that
// early (heavy) and late (light) ones of a document even out; with `reverse`
// the last rows, which see most keys, come first.
template <class Smem>
__device__ void plan_work(const AttnParams& p, const Smem& sm, int rows, int heads, int reverse) {
  const int lane = threadIdx.x & 31;
  const int64_t slots = p.T / rows + p.B, items = slots * heads, G = gridDim.x;
  uint32_t n = 0;
  const auto put = [&](const Work& w, bool me) -> bool {
    const int r = n % kRing;
    if (!mbar_wait_warp(sm.info_empty(r), ((n / kRing) & 1) ^ 1, sm.abort_flag, p.status))
      return false;
    if (me) {
      sm.info[r] = w;
      mbar_arrive_a(sm.info_full(r));  // releases the write
    }
    __syncwarp();
    ++n;
    return true;
  };
  Work w;
  for (int64_t round0 = 0; round0 * G < items; round0 += 32) {
    const int64_t round = round0 + lane;
    int64_t item = round * G + ((round & 1) ? G - 1 - static_cast<int64_t>(blockIdx.x) : blockIdx.x);
    w.live = item < items;
    if (!w.live) item = items - 1;
    const int64_t s = item / heads, slot = reverse ? slots - 1 - s : s;
    const int64_t b = slot_doc(p, slot, rows);
    bool bad;
    const Doc c = load_doc(p, b, bad);
    const int64_t row0 = (slot - slot_base(p, b, rows)) * rows;
    w.start = c.start;
    w.len = c.len;
    w.keys = c.keys;
    w.prefix = c.prefix;
    w.row0 = static_cast<int>(row0);
    w.head = static_cast<int>(item - s * heads);
    w.live = w.live && row0 >= 0 && row0 < c.len;  // else the slot is empty
    for (unsigned set = __ballot_sync(0xffffffffu, w.live != 0); set; set &= set - 1)
      if (!put(w, lane == __ffs(set) - 1)) return;
  }
  w.live = 0;
  put(w, lane == 0);
}

__device__ __forceinline__ int row_end(const Work& c, int mask, int i) {
  if (mask == MAXSIM_MASK_FULL) return c.keys;
  return min(c.keys, max(i + 1, c.prefix));
}

// 2^x and 1/x in hardware (2 ulp, 1 ulp).
__device__ __forceinline__ float fast_exp2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ __forceinline__ float fast_rcp(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// tanh(x) = 1 - 2 / (1 + e^2x); `x2` is 2 x log2(e). Off by 2^-22 absolutely,
// for any x: e^2x may overflow to infinity or vanish.
__device__ __forceinline__ float fast_tanh(float x2) { return fmaf(-2.f, fast_rcp(1.f + fast_exp2(x2)), 1.f); }

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// tanh(x) = x p(x^2) for |x| <= 0.7, with p of degree 5, fitted to tanh on that
// interval by least squares reweighted towards equal errors: off by 1.3e-8
// relatively, 7e-8 in fp32 arithmetic.
constexpr float kTanhReach = 0.7f;
__device__ __forceinline__ constexpr float tanh_fit(int i) {
  constexpr float c[6] = {1.0f, -0.3333314061164856f, 0.13328571617603302f, -0.05353494733572006f,
                          0.02004525437951088f, -0.005105282180011272f};
  return c[i];
}

// How scores are capped. fast_tanh may be off by 2^-22, so all scores by that part
// of the cap: up to 3e-5 for caps of 128. Beyond, where scores are small against
// their cap and that error would reach them, the tangent is made right relatively,
// to 2^-20 (kWide, in kernels of their own: in those for usual caps the additional
// code cost 2 %; 24 documents of 1024 tokens, 16 heads of 128: forward 433 us where
// narrow caps take 308, backward 1022 and 876).
enum Cap { kNoCap, kNarrow, kWide };
constexpr float kWideCap = 128.f;

// Both forms are made and one is taken: a branch for each value took four times as long.
__device__ __forceinline__ float close_tanh(float x) {
  const float w = x * x, far = fast_tanh(2.f * 1.4426950408889634f * x);
  float r = tanh_fit(5);
#pragma unroll
  for (int i = 4; i >= 0; --i) r = fmaf(r, w, tanh_fit(i));
  float y;
  asm("{\n\t.reg .pred p;\n\tsetp.le.f32 p, %1, %2;\n\tselp.f32 %0, %3, %4, p;\n\t}"
      : "=f"(y)
      : "f"(fabsf(x)), "f"(kTanhReach), "f"(x * r), "f"(far));
  return y;
}

// u = tanh(k u) for 32 values of each lane. `whole`: the same for the warp, all
// 32 are scores; `live`: this lane's are (others hold what was left there, and
// must not decide how the rest is rounded). Through exp2 and a reciprocal a value
// costs two of the special function unit's slots, and the softmax of capped
// scores waits for that unit: where no value of the warp exceeds 0.7 (scores up
// to 0.7 cap) the polynomial makes all of them.
template <bool kClose>
__device__ __forceinline__ void tanh_group(uint32_t (&u)[32], float k, bool whole, bool live) {
  float top = 0.f;
#pragma unroll
  for (int x = 0; x < 32; x += 2) top = max3(top, fabsf(__uint_as_float(u[x])), fabsf(__uint_as_float(u[x + 1])));
  if (__all_sync(0xffffffffu, whole && (!live || top * k <= kTanhReach))) {
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const Pair v = mul2(Pair(__uint_as_float(u[x]), __uint_as_float(u[x + 1])), Pair(k, k)), w = mul2(v, v);
      Pair r(tanh_fit(5), tanh_fit(5));
#pragma unroll
      for (int i = 4; i >= 0; --i) r = fma2(r, w, Pair(tanh_fit(i), tanh_fit(i)));
      float a, b;
      mul2(v, r).get(a, b);
      u[x] = __float_as_uint(a);
      u[x + 1] = __float_as_uint(b);
    }
  } else {
    const float k2 = 2.f * 1.4426950408889634f * k;
#pragma unroll
    for (int x = 0; x < 32; ++x) {
      const float z = __uint_as_float(u[x]);
      u[x] = __float_as_uint(kClose ? close_tanh(z * k) : fast_tanh(z * k2));
    }
  }
}

// Two values as 16-bit ones in a word, `lo` in its low half.
template <bool kBf16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  uint32_t r;
  if constexpr (kBf16) asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  else asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// A warp's 32 rows of kCols columns of 16-bit values (kCols / 2 words a lane,
// one row each) to memory. Written as they are, each store would touch 32 lines,
// 16 bytes of each; through shared memory it touches a few, kCols * 2 bytes of
// each. Rows lie 80 bytes apart, or 128 with their 16-byte parts exchanged by
// the row's number: no bank conflicts either way. base: the first row's head.
template <int kCols>
constexpr uint32_t kStageBytes = 32 * (kCols == 32 ? 80 : 128);
template <int kCols>
__device__ __forceinline__ void store_rows(uint32_t stage, const uint32_t (&v)[kCols / 2], uint16_t* base,
                                           int64_t stride, int rows, int col0, int d) {
  constexpr int kParts = kCols / 8, kPitch = kCols == 32 ? 80 : 128;
  const int lane = threadIdx.x & 31;
  const auto at = [&](int r, int part) -> uint32_t { return stage + r * kPitch + (kCols == 32 ? part : part ^ (r & 7)) * 16; };
#pragma unroll
  for (int x = 0; x < kParts; ++x)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at(lane, x)), "r"(v[x * 4]), "r"(v[x * 4 + 1]),
                 "r"(v[x * 4 + 2]), "r"(v[x * 4 + 3])
                 : "memory");
  __syncwarp();
  const int part = lane % kParts, col = col0 + part * 8;
  uint4 y[kParts];
#pragma unroll
  for (int i = 0; i < kParts; ++i)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(y[i].x), "=r"(y[i].y), "=r"(y[i].z), "=r"(y[i].w)
                 : "r"(at(i * (32 / kParts) + lane / kParts, part))
                 : "memory");
#pragma unroll
  for (int i = 0; i < kParts; ++i) {
    const int r = i * (32 / kParts) + lane / kParts;
    if (r < rows && col < d) *reinterpret_cast<uint4*>(base + r * stride + col) = y[i];
  }
  __syncwarp();
}

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

// Tensor map of a view: 64 elements of one head (128 bytes, 128-byte swizzle)
// by `box_rows` tokens. Elements past d and tokens past T read as zeros.
bool attn_tmap(void* map, const HeadsView& v, int64_t T, int heads, int d, int is_bf16, int box_rows);

}  // namespace msim

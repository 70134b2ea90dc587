// rows.cuh -- what the operators on rows of hidden states share: eight columns of
// a row at a time, and the generator that decides which of them dropout keeps.
//
// Random numbers come from Philox4x32-10 (J. Salmon, M. Moraes, R. Dror, D. Shaw,
// "Parallel random numbers: as easy as 1, 2, 3", 2011): a bijection of a 128-bit
// counter under a 64-bit key, ten rounds of two 32 x 32 -> 64 bit products. The
// key is the seed, the counter (column / 8, row, call's number): an element's lot
// depends on its place alone, so the mask is made again wherever it is needed.
// The four words are eight lots of 16 bits, in the order of the columns, low half
// first: half the products of a word an element, and chances are multiples of 2^-16.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <climits>
#include <cstdint>
#include <type_traits>

#include "internal.h"
#include "pair.cuh"

namespace msim {

// Dropout as the kernels take it: lots below `limit` are dropped (0: none), and
// what stays is multiplied by `factor`.
struct Drop {
  const int64_t* rng;  // seed, call's number
  uint32_t limit;
  float factor;
};

struct Key {
  uint32_t k0, k1, c2, c3;
};
__device__ __forceinline__ Key load_key(const Drop& d) {
  Key k = {};
  if (d.limit) {
    const uint64_t seed = static_cast<uint64_t>(__ldg(d.rng)), call = static_cast<uint64_t>(__ldg(d.rng + 1));
    k = {static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(call),
         static_cast<uint32_t>(call >> 32)};
  }
  return k;
}

// The four words of a group of eight columns.
struct Lots {
  uint32_t w[4];
  // Whether column j of the group stays; `high` is the limit in the upper half of a
  // word: a word's lower bits never change how its upper half compares with it.
  __device__ __forceinline__ bool stays(int j, uint32_t high) const {
    return (j & 1 ? w[j >> 1] : w[j >> 1] << 16) >= high;
  }
};
__device__ __forceinline__ Lots draw_lots(const Key& key, uint32_t group, uint32_t row) {
  uint32_t c0 = group, c1 = row, c2 = key.c2, c3 = key.c3;
#pragma unroll
  for (uint32_t i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ (key.k0 + i * 0x9E3779B9u);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ (key.k1 + i * 0xBB67AE85u);
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
  }
  return {{c0, c1, c2, c3}};
}

// Eight elements of a thread, as they lie in memory and as fp32 pairs.
template <typename T>
struct Raw {
  uint4 v[sizeof(T) / 2];
};
struct Eight {
  Pair p[4];
};

template <typename T>
__device__ __forceinline__ Eight up8(const Raw<T>& r) {
  Eight o;
  if constexpr (sizeof(T) == 4) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      o.p[2 * i] = Pair(__uint_as_float(r.v[i].x), __uint_as_float(r.v[i].y));
      o.p[2 * i + 1] = Pair(__uint_as_float(r.v[i].z), __uint_as_float(r.v[i].w));
    }
  } else {
    const uint32_t w[4] = {r.v[0].x, r.v[0].y, r.v[0].z, r.v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (std::is_same<T, __nv_bfloat16>::value) {
        o.p[i] = Pair(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xFFFF0000u));
      } else {
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
        o.p[i] = Pair(f.x, f.y);
      }
    }
  }
  return o;
}
template <typename T>
__device__ __forceinline__ Raw<T> down8(const Eight& e) {
  Raw<T> r;
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float a, b;
    e.p[i].get(a, b);
    if constexpr (sizeof(T) == 4) {
      if (i & 1) r.v[i / 2].z = __float_as_uint(a), r.v[i / 2].w = __float_as_uint(b);
      else r.v[i / 2].x = __float_as_uint(a), r.v[i / 2].y = __float_as_uint(b);
    } else if constexpr (std::is_same<T, __nv_bfloat16>::value) {
      asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    } else {
      asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(b), "f"(a));
    }
  }
  if constexpr (sizeof(T) == 2) r.v[0] = make_uint4(w[0], w[1], w[2], w[3]);
  return r;
}

// The compiler is kept from holding on to what it made of these elements: they are
// unpacked again where they are needed again (an instruction each, half the registers).
template <typename T>
__device__ __forceinline__ void forget(Raw<T>& r) {
#pragma unroll
  for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
    asm volatile("" : "+r"(r.v[i].x), "+r"(r.v[i].y), "+r"(r.v[i].z), "+r"(r.v[i].w));
}

// How a team of threads divides a row. Whole: a thread has eight neighbouring
// columns, moved as 16-byte vectors; every row then begins on a 16-byte boundary
// and the width is a multiple of 8. Else a warp has 256 neighbouring columns, of
// which a lane has every 32nd, so that single elements are moved by whole lines.
template <bool kWhole>
struct Cols {
  int first, d;
  __device__ __forceinline__ Cols(int part, int lane, int d_) : d(d_) {
    // part: the thread's (whole) or the warp's number among the row's
    first = kWhole ? part * 8 : part * 256 + lane;
  }
  __device__ __forceinline__ int at(int j) const { return first + j * (kWhole ? 1 : 32); }
  __device__ __forceinline__ bool in(int j) const { return kWhole ? first < d : at(j) < d; }
};

// Zeros where the row ends, or is not there.
template <typename T, bool kWhole>
__device__ __forceinline__ Raw<T> load8(const T* row, const Cols<kWhole>& c, bool there = true) {
  Raw<T> r;
  if constexpr (kWhole) {
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i)
      r.v[i] = there && c.in(0) ? reinterpret_cast<const uint4*>(row + c.first)[i] : make_uint4(0, 0, 0, 0);
  } else {
    alignas(16) T e[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) e[j] = there && c.in(j) ? row[c.at(j)] : static_cast<T>(0.f);
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) r.v[i] = reinterpret_cast<uint4*>(e)[i];
  }
  return r;
}
template <typename T, bool kWhole>
__device__ __forceinline__ void store8(T* row, const Cols<kWhole>& c, const Raw<T>& r) {
  if constexpr (kWhole) {
    if (c.in(0))
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(row + c.first)[i] = r.v[i];
  } else {
    alignas(16) T e[8];
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(e)[i] = r.v[i];
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = e[j];
  }
}
// The same as fp32 pairs at once: single elements need no packing.
template <typename T, bool kWhole>
__device__ __forceinline__ Eight load_up8(const T* row, const Cols<kWhole>& c, bool there = true) {
  if constexpr (kWhole) return up8<T>(load8<T, kWhole>(row, c, there));
  float v[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) v[j] = there && c.in(j) ? static_cast<float>(row[c.at(j)]) : 0.f;
  Eight o;
#pragma unroll
  for (int i = 0; i < 4; ++i) o.p[i] = Pair(v[2 * i], v[2 * i + 1]);
  return o;
}
template <typename T, bool kWhole>
__device__ __forceinline__ void store_down8(T* row, const Cols<kWhole>& c, const Eight& e) {
  if constexpr (kWhole) {
    store8<T, kWhole>(row, c, down8<T>(e));
  } else {
    float v[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) e.p[i].get(v[2 * i], v[2 * i + 1]);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = static_cast<T>(v[j]);
  }
}

// Which of the thread's eight elements stay. Where a warp's columns are
// interleaved, each lane draws for eight neighbouring ones, and what it found is
// passed on: all lanes have to be there.
template <bool kWhole>
struct Kept {
  Lots lots;
  uint32_t high, bits;
  __device__ __forceinline__ Kept(const Key& key, const Cols<kWhole>& c, uint32_t row, uint32_t limit) : high(limit << 16) {
    if constexpr (kWhole) {
      lots = draw_lots(key, static_cast<uint32_t>(c.first) >> 3, row);
    } else {
      const uint32_t lane = threadIdx.x & 31;
      const Lots mine = draw_lots(key, ((static_cast<uint32_t>(c.first) - lane) >> 3) + lane, row);
      // column j * 32 + lane is element lane % 8 of group j * 4 + lane / 8
      bits = 0;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const uint32_t all = __ballot_sync(~0u, mine.stays(j, high));
        if ((lane & 7) == j) bits = all;
      }
      bits >>= lane >> 3;
    }
  }
  __device__ __forceinline__ bool operator()(int j) const {
    if constexpr (kWhole) return lots.stays(j, high);
    return bits >> (4 * j) & 1;
  }
  // add + (stays ? x * factor : 0), the sum rounded once; without `add`, 0 or the product.
  __device__ __forceinline__ Eight of(const Eight& x, float factor, const Eight& add, bool adds) const {
    Eight o;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a, b, c = 0.f, d = 0.f;
      x.p[i].get(a, b);
      if (adds) add.p[i].get(c, d);
      o.p[i] = Pair((*this)(2 * i) ? (adds ? fmaf(a, factor, c) : a * factor) : c,
                    (*this)(2 * i + 1) ? (adds ? fmaf(b, factor, d) : b * factor) : d);
    }
    return o;
  }
};

// Quotients of numbers below 2^31 by one divisor, without a division (T. Granlund,
// P. Montgomery, "Division by invariant integers using multiplication", 1994).
struct Divisor {
  uint32_t d, m, s;
  explicit Divisor(uint32_t d_) : d(d_), m(0), s(0) {
    while (s < 31 && (1u << s) < d) ++s;
    m = static_cast<uint32_t>(((uint64_t(1) << 32) * ((uint64_t(1) << s) - d)) / d + 1);
  }
  __device__ __forceinline__ uint32_t of(uint32_t n) const { return (__umulhi(n, m) + n) >> s; }
};

inline bool whole_rows(const maxsim_rows* v, int d, int esize) {
  return !v || !v->data || (d % 8 == 0 && reinterpret_cast<uintptr_t>(v->data) % (esize == 1 ? 8 : 16) == 0 &&
                            v->row_stride * esize % (esize == 1 ? 8 : 16) == 0);
}

}  // namespace msim

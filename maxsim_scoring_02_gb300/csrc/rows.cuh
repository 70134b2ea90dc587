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

#include "internal.h"

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

// Bit e is set where column 8 * group + e of the row stays.
__device__ __forceinline__ uint32_t kept8(const Key& key, uint32_t group, uint32_t row, uint32_t limit) {
  uint32_t c0 = group, c1 = row, c2 = key.c2, c3 = key.c3, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int i = 0; i < 10; ++i) {
    const uint64_t a = static_cast<uint64_t>(c0) * 0xD2511F53u, b = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  const uint32_t w[4] = {c0, c1, c2, c3};
  uint32_t bits = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    bits |= (w[i] & 0xFFFFu) >= limit ? 1u << (2 * i) : 0u;
    bits |= w[i] >> 16 >= limit ? 2u << (2 * i) : 0u;
  }
  return bits;
}

template <typename T>
__device__ __forceinline__ float up(T x) { return static_cast<float>(x); }

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

template <typename T, bool kWhole>
__device__ __forceinline__ void load8(const T* row, const Cols<kWhole>& c, T (&v)[8]) {
  if constexpr (kWhole) {
    if (c.in(0)) {
      const uint4* s = reinterpret_cast<const uint4*>(row + c.first);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) reinterpret_cast<uint4*>(v)[i] = s[i];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = static_cast<T>(0.f);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c.in(j) ? row[c.at(j)] : static_cast<T>(0.f);
  }
}
template <typename T, bool kWhole>
__device__ __forceinline__ void store8(T* row, const Cols<kWhole>& c, const float (&v)[8]) {
  if constexpr (kWhole) {
    if (c.in(0)) {
      alignas(16) T o[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] = static_cast<T>(v[j]);
      uint4* s = reinterpret_cast<uint4*>(row + c.first);
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(T)) / 2; ++i) s[i] = reinterpret_cast<uint4*>(o)[i];
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (c.in(j)) row[c.at(j)] = static_cast<T>(v[j]);
  }
}
// Which of the thread's eight elements stay. Where a warp's columns are
// interleaved, each lane makes the lots of eight neighbouring ones, and they are
// passed on: all lanes have to be there.
template <bool kWhole>
__device__ __forceinline__ uint32_t kept(const Key& key, const Cols<kWhole>& c, uint32_t row, uint32_t limit) {
  if constexpr (kWhole) return kept8(key, static_cast<uint32_t>(c.first) >> 3, row, limit);
  const uint32_t lane = threadIdx.x & 31;
  const uint32_t mine = kept8(key, ((static_cast<uint32_t>(c.first) - lane) >> 3) + lane, row, limit);
  uint32_t bits = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j)
    bits |= (__shfl_sync(~0u, mine, j * 4 + (lane >> 3)) >> (lane & 7) & 1u) << j;
  return bits;
}

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

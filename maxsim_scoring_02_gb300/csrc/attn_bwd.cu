// attn_bwd.cu -- packed attention, backward, on tcgen05.
//
// Three kernels (and a small one in fp16). The first makes, for each row and head, its lse in log2 units
// and delta = <dO, out>. The other two make each score again and own what they
// write, so there are no atomics and results do not depend on scheduling:
//
//   dQ:  128 rows of one document and head, walking over the keys:
//       S = Q K^T, dP = dO V^T               (both operands in shared memory)
//       P = 2^(S c - lse2), dS = P (dP - delta) bend
//       dQ += dS K, R += P bend K            (A from TMEM, B as it lies in memory)
//   dK and dV:  128 keys of one document and key-value head, walking over the
//     query heads that share it and over the rows that see the keys:
//       S^T = K Q^T, dP^T = V dO^T, P^T and dS^T as above
//       dV += P^T dO, dK += dS^T Q
//
// delta made from `out` carries that tensor's rounding to 16 bits, which would
// add as much error to dQ and dK as all other roundings together. Its exact
// value is sum_j P_ij dP_ij, known at the end of a row: the dQ kernel gathers
// off = sum_j P_ij (dP_ij - delta) in fp32 on the way, takes off * R from dQ
// (the same as if delta + off had been used all along) and leaves delta + off
// for the other kernel. (Error against fp64 on capped pages of 1024 tokens:
// 0.0032 without, 0.0024 with.)
//
// Eight products of 128 x 128 x d for a tile where five would do if dQ were
// added up in memory by all key blocks, in an order that changes results, and
// delta were taken as it is.
//
// Measured: 24 documents of 1024 tokens, 16 heads of 128: 0.65 ms (0.79 PFLOP/s
// of the five products, 1.27 of the eight made); 64 documents, 12 heads of 64: 0.91
// ms. Bound by the arithmetic phases beside the products: 960 to 1180 cycles
// for P and 750 to 850 for dS of a tile whose eight products, in both kernels,
// take 4130.
//
// A tile passes through two phases of the arithmetic warps, P and dS. While
// they are at dS of tile i the tensor cores make the product with P of tile i and S of tile
// i + 1, while they are at P of tile i + 1 that with dS of tile i and dP of
// tile i + 1: single buffers of S and dP are enough, because the tensor cores
// run in order. P lies over S and dS over dP, each warpgroup's half in its own
// columns. P and dS are rounded to the inputs' type for their products, as the
// tensor cores take nothing wider at this rate; sums are fp32. `scale` is
// applied to the sums.
//
// fp16 holds 2^-14 to 2^16 in full, but a weight among 16K keys is 2^-14 on
// average and dS less by dO's size (dO of 1e-3 there: dS off by 4 %, dQ by 1.5 %). So
// both are held times a power of two made of the document's greatest |dO_i| |v_j|,
// which two small kernels find: it is added to the lse2 that scores are taken
// from, and taken off the sums, so it is exact and costs the large kernels nothing
// (the small ones read v once: 24 documents of 1024 tokens, 16 heads of 128, 0.69 ms
// where bf16 takes 0.65).
#include "attn_common.cuh"

namespace msim {
namespace {

constexpr int kTile = 128;
constexpr int kBoxRows = 64;

// DH: head size in shared memory; BC: columns of a score tile (rows of Q or
// keys that are walked over), 64 for each arithmetic warpgroup. Heads of 64 and
// fewer take tiles of 64 columns and two blocks an SM, whose phases interleave:
// against one block with tiles of 128 and S made a tile ahead that is 18 % faster
// at 150 tokens a document, 4 % at 256 and even at 1024 (12 heads), but 6 % slower on
// 160 ragged documents of 0 to 512 with a distance bias (0.388 against 0.412 ms).
// Heads of 128 fill TMEM with one block.
template <int DH, int BC, bool kDkv>
struct BwdShape {
  static constexpr int kGroups = BC / 64;
  static constexpr int kStages = 2;
  static constexpr int kPanels = DH / 64;
  static constexpr uint32_t kOwnPanel = kTile * 128, kOwnBytes = kPanels * kOwnPanel;
  static constexpr uint32_t kPanel = BC * 128, kBytes = kPanels * kPanel;
  static constexpr int kThreads = kGroups * 128 + 128;
  static constexpr int kBlocks = BC == 64 ? 2 : 1;
  static constexpr int kRegsLaunch = BC == 64 ? 128 : 168;
  // Registers of the arithmetic threads once they took over some of the
  // others'; dQ of capped scores also keeps the cap's derivatives.
  static constexpr int math_regs(bool cap) { return cap && !kDkv ? (BC == 64 ? 200 : 224) : (BC == 64 ? 168 : 208); }
  static constexpr int other_regs(bool cap) { return (kGroups + 1) * kRegsLaunch - kGroups * math_regs(cap); }
  static_assert(other_regs(true) >= 56 && other_regs(true) % 8 == 0 && other_regs(false) % 8 == 0, "register split");
  // TMEM columns: S, dP, then the sums
  static constexpr uint32_t kDp = BC, kSum0 = kDp + BC, kSum1 = kSum0 + DH, kNeed = kSum1 + DH;
  static constexpr uint32_t kTmemCols = kNeed <= 256 ? 256 : 512;
  static constexpr int kBars = 2 + 2 * kStages + 5 + 2 * kRing + 2;
  static constexpr uint32_t kSmem = 2 * kOwnBytes + 2 * kStages * kBytes + kGroups * 4 * kStageBytes<64> + 8 * kBars +
                                    kStages * BC * 8 + kRing * sizeof(Work) + 16 + 16;
};

// own_a, own_b: the 128 rows that the block keeps (K and V, or Q and dO);
// walk_a, walk_b: the stages of what it walks over (Q and dO, or K and V).
template <class S, int BC>
struct BwdSmem {
  uint32_t own_a, own_b, walk_a, walk_b, stage, bars;
  uint64_t* bar;
  float* stats;   // S::kStages x (BC times -lse2, BC times -delta) of the walked rows
  Work* info;
  uint32_t* tmem_slot;
  int* abort_flag;
  __device__ __forceinline__ explicit BwdSmem(uint8_t* raw) {
    uint8_t* base = raw;  // on a 1024-byte boundary, as the swizzled tiles need it
    own_a = smem_u32(base);
    own_b = own_a + S::kOwnBytes;
    walk_a = own_b + S::kOwnBytes;
    walk_b = walk_a + S::kStages * S::kBytes;
    uint8_t* end = base + 2 * S::kOwnBytes + 2 * S::kStages * S::kBytes;
    stage = walk_b + S::kStages * S::kBytes;
    end += S::kGroups * 4 * kStageBytes<64>;
    stats = reinterpret_cast<float*>(end);
    bar = reinterpret_cast<uint64_t*>(end + S::kStages * BC * 8);
    bars = smem_u32(bar);
    info = reinterpret_cast<Work*>(bar + S::kBars);
    tmem_slot = reinterpret_cast<uint32_t*>(info + kRing);
    abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  }
  __device__ __forceinline__ uint32_t own_full() const { return bars; }
  __device__ __forceinline__ uint32_t own_empty() const { return bars + 8; }
  __device__ __forceinline__ uint32_t walk_full(int s) const { return bars + 16 + 8 * s; }
  __device__ __forceinline__ uint32_t walk_empty(int s) const { return walk_full(S::kStages + s); }
  __device__ __forceinline__ uint32_t s_full() const { return walk_full(2 * S::kStages); }
  __device__ __forceinline__ uint32_t dp_full() const { return s_full() + 8; }
  __device__ __forceinline__ uint32_t p_full() const { return s_full() + 16; }
  __device__ __forceinline__ uint32_t ds_full() const { return s_full() + 24; }
  __device__ __forceinline__ uint32_t sum_full() const { return s_full() + 32; }
  __device__ __forceinline__ uint32_t info_full(int r) const { return s_full() + 40 + 8 * r; }
  __device__ __forceinline__ uint32_t info_empty(int r) const { return info_full(kRing + r); }
  __device__ __forceinline__ uint32_t done() const { return info_full(2 * kRing); }
  __device__ __forceinline__ uint32_t rest_full() const { return done() + 8; }
  __device__ __forceinline__ uint64_t* at(uint32_t b) const { return bar + (b - bars) / 8; }
};

// The tiles that an item walks over: `steps` of BC columns for each of `heads`
// heads, columns [begin, end) of the document.
struct Range {
  int begin, end, steps, heads;
};
template <bool kDkv, int BC>
__device__ __forceinline__ Range range_of(const AttnParams& p, const Work& w) {
  Range r;
  if constexpr (kDkv) {
    r.begin = w.row0 < w.keys ? (p.mask == MAXSIM_MASK_FULL || w.row0 < w.prefix ? 0 : w.row0) : w.len;
    r.end = w.len;
    r.heads = p.heads / p.kv_heads;
  } else {
    r.begin = 0;
    r.end = row_end(w, p.mask, min(w.len, w.row0 + kTile) - 1);
    r.heads = 1;
  }
  r.steps = (r.end - r.begin + BC - 1) / BC;
  return r;
}

struct BwdMaps {
  CUtensorMap own_a, own_b, walk_a, walk_b;
};

// ---------------------------------------------------------------- loads
template <class S, int BC, bool kDkv>
__device__ void bwd_loader(const AttnParams& p, const BwdSmem<S, BC>& sm, const BwdMaps& m) {
  if (debug_faults(p.status) & kDebugStallFwdLoader) return;  // test-only switch (maxsim_debug_set_faults)
  const int group = p.heads / p.kv_heads;
  uint32_t item = 0, step = 0;
  bool ok = true;
  const auto load = [&](uint32_t dst, uint32_t panel, const CUtensorMap* map, uint32_t bar, int head, int token, int boxes) {
    for (int b = 0; b < boxes; ++b)
      for (int pn = 0; pn < S::kPanels; ++pn)
        tma_load_3d_a(dst + pn * panel + b * (kBoxRows * 128), map, bar, pn * 64, head, token + b * kBoxRows);
  };
  for (uint32_t n = 0; ok; ++n) {
    const int r = n % kRing;
    if (!(ok = mbar_wait_inl_a(sm.info_full(r), (n / kRing) & 1, sm.abort_flag, p.status))) break;
    const Work w = sm.info[r];
    mbar_arrive_a(sm.info_empty(r));
    if (!w.live) break;
    const Range g = range_of<kDkv, BC>(p, w);
    if (g.steps <= 0) continue;
    if (!(ok = mbar_wait_inl_a(sm.own_empty(), (item & 1) ^ 1, sm.abort_flag, p.status))) break;
    const int own_boxes = (min(kTile, w.len - w.row0) + kBoxRows - 1) / kBoxRows;
    mbar_arrive_expect_tx_a(sm.own_full(), 2 * own_boxes * S::kPanels * (kBoxRows * 128));
    load(sm.own_a, S::kOwnPanel, &m.own_a, sm.own_full(), w.head, w.start + w.row0, own_boxes);
    load(sm.own_b, S::kOwnPanel, &m.own_b, sm.own_full(), w.head, w.start + w.row0, own_boxes);
    ++item;
    for (int h = 0; ok && h < g.heads; ++h) {
      const int head = kDkv ? w.head * group + h : w.head / group;
      for (int j = 0; j < g.steps; ++j) {
        const int s = step % S::kStages, from = g.begin + j * BC;
        if (!(ok = mbar_wait_inl_a(sm.walk_empty(s), ((step / S::kStages) & 1) ^ 1, sm.abort_flag, p.status))) break;
        const int boxes = (min(BC, g.end - from) + kBoxRows - 1) / kBoxRows;
        mbar_arrive_expect_tx_a(sm.walk_full(s), 2 * boxes * S::kPanels * (kBoxRows * 128));
        load(sm.walk_a + s * S::kBytes, S::kPanel, &m.walk_a, sm.walk_full(s), head, w.start + from, boxes);
        load(sm.walk_b + s * S::kBytes, S::kPanel, &m.walk_b, sm.walk_full(s), head, w.start + from, boxes);
        ++step;
      }
    }
  }
  if (!ok) {  // after an abort: wait (bounded) for the copies in flight
    if (item > 0) mbar_wait_drain(sm.at(sm.own_full()), (item - 1) & 1, p.status);
    for (uint32_t f = step > S::kStages ? step - S::kStages : 0; f < step; ++f)
      mbar_wait_drain(sm.at(sm.walk_full(f % S::kStages)), (f / S::kStages) & 1, p.status);
  }
}

// The walked rows' (lse2, delta), which every arithmetic thread needs: one
// warp brings them to shared memory beside the tiles. Its arrival is part of
// walk_full, so it also keeps an abort's drain from waiting for ever.
template <class S, int BC, bool kBf16>
__device__ void bwd_stats(const AttnParams& p, const BwdSmem<S, BC>& sm) {
  const int lane = threadIdx.x & 31, group = p.heads / p.kv_heads;
  const float2* src = reinterpret_cast<const float2*>(p.delta);
  uint32_t step = 0;
  for (uint32_t n = 0;; ++n) {
    const int r = n % kRing;
    if (!mbar_wait_warp(sm.info_full(r), (n / kRing) & 1, sm.abort_flag, p.status)) return;
    const Work w = sm.info[r];
    __syncwarp();
    if (lane == 0) mbar_arrive_a(sm.info_empty(r));
    if (!w.live) return;
    const Range g = range_of<true, BC>(p, w);
    const float shift = kBf16 ? 0.f : p.shifts[w.start].x;
    for (int h = 0; h < g.heads; ++h) {
      const float2* row = src + static_cast<int64_t>(w.head * group + h) * p.T + w.start;
      for (int j = 0; j < g.steps; ++j, ++step) {
        const int s = step % S::kStages, from = g.begin + j * BC;
        float2 v[BC / 32];
#pragma unroll
        for (int x = 0; x < BC / 32; ++x) {
          const int i = from + x * 32 + lane;
          v[x] = i < g.end ? row[i] : make_float2(-INFINITY, 0.f);
        }
        if (!mbar_wait_warp(sm.walk_empty(s), ((step / S::kStages) & 1) ^ 1, sm.abort_flag, p.status))
          return;
#pragma unroll
        for (int x = 0; x < BC / 32; ++x) {
          sm.stats[s * 2 * BC + x * 32 + lane] = kBf16 ? v[x].x : v[x].x + shift;
          sm.stats[(s * 2 + 1) * BC + x * 32 + lane] = v[x].y;
        }
        __syncwarp();
        if (lane == 0) mbar_arrive_a(sm.walk_full(s));
      }
    }
  }
}

// ------------------------------------------------------------- products
template <class S, int DH, int BC, bool kDkv, bool kBf16>
__device__ void bwd_products(const AttnParams& p, const BwdSmem<S, BC>& sm, uint32_t tmem) {
  const int lane = threadIdx.x & 31;
  const uint32_t idesc = idesc_f16(kBf16, kTile, 0);
  const uint32_t idesc_sum = idesc | static_cast<uint32_t>(DH >> 3) << 17 | kIdescBMnMajor;
  uint32_t item = 0, step = 0;
  const auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
    return mbar_wait_warp(bar, ph & 1, sm.abort_flag, p.status);
  };
  // 128 x cols scores of the block's rows and the walked ones of stage s
  const auto score = [&](uint32_t d_col, uint32_t own, uint32_t walked, int cols) {
    const uint32_t id = idesc | static_cast<uint32_t>(cols >> 3) << 17;
    const uint64_t a = sdesc_k_sw128(own), b = sdesc_k_sw128(walked);
#pragma unroll
    for (int kk = 0; kk < DH / 16; ++kk)
      umma_f16_el(tmem + d_col, a + (kk / 4) * (S::kOwnPanel >> 4) + (kk % 4) * 2,
                  b + (kk / 4) * (S::kPanel >> 4) + (kk % 4) * 2, id, kk != 0);
  };
  // sum += A (16-bit, over the score tile at a_col) * the walked rows of stage s
  const auto add = [&](uint32_t d_col, uint32_t a_col, uint32_t walked, int cols, bool first) {
    const uint64_t b = sdesc_mn_sw128(walked, S::kPanel);
    for (int kk = 0; kk < cols / 16; ++kk)
      umma_f16_ts_el(tmem + d_col, tmem + a_col + (kk / 4) * 64 + (kk % 4) * 8, b + kk * (2048 >> 4), idesc_sum,
                     !first || kk != 0);
  };
  bool ok = true;
  for (uint32_t n = 0; ok; ++n) {
    const int r = n % kRing;
    if (!wait(sm.info_full(r), n / kRing)) break;
    const Work w = uniform_work(sm.info[r]);
    __syncwarp();
    if (lane == 0) mbar_arrive_a(sm.info_empty(r));
    if (!w.live) break;
    const Range g = range_of<kDkv, BC>(p, w);
    if (g.steps <= 0) continue;
    const int total = g.steps * g.heads;
    int at = 0;  // step within the head of the tile that is made ready next
    // Waits for walked tile step + i, zeroes the rows behind its last one (up to
    // a multiple of 16): their weights are 0, and 0 * NaN would reach the sums.
    const auto ready = [&](int i, int& cols) -> bool {
      const int s = (step + i) % S::kStages, used = min(BC, g.end - g.begin - at * BC);
      if (++at == g.steps) at = 0;
      if (!wait(sm.walk_full(s), (step + i) / S::kStages)) return false;
      cols = (used + 15) & ~15;
      if (used != cols) {
        const uint32_t vec = (cols - used) * 8;
        for (uint32_t e = lane; e < vec * S::kPanels * 2; e += 32) {
          const uint32_t pn = (e / vec) % S::kPanels, base = e / vec < S::kPanels ? sm.walk_a : sm.walk_b;
          const uint32_t dst = base + s * S::kBytes + pn * S::kPanel + used * 128 + (e % vec) * 16;
          asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
        }
        fence_proxy_async_smem();
        __syncwarp();
      }
      return true;
    };
    int cols = 0, next = 0;  // columns of tiles i and i + 1
    const auto make_s = [&](int i, int& c) -> bool {
      if (!ready(i, c)) return false;
      tc_fence_after();
      score(0, sm.own_a, sm.walk_a + (step + i) % S::kStages * S::kBytes, c);
      umma_commit_el(sm.s_full());
      return true;
    };
    const auto make_dp = [&](int i, int c) {
      score(S::kDp, sm.own_b, sm.walk_b + (step + i) % S::kStages * S::kBytes, c);
      umma_commit_el(sm.dp_full());
    };
    ok = wait(sm.own_full(), item) && make_s(0, cols);
    if (!ok) break;
    make_dp(0, cols);
    for (int i = 0; i < total; ++i) {
      const uint32_t u = step + i, s = u % S::kStages;
      if (!(ok = wait(sm.p_full(), u))) break;
      tc_fence_after();
      add(S::kSum0, 0, (kDkv ? sm.walk_b : sm.walk_a) + s * S::kBytes, cols, i == 0);
      if (i + 1 < total && !(ok = make_s(i + 1, next))) break;
      if (!(ok = wait(sm.ds_full(), u))) break;
      tc_fence_after();
      add(S::kSum1, S::kDp, sm.walk_a + s * S::kBytes, cols, i == 0);
      umma_commit_el(sm.walk_empty(s));
      if (i + 1 < total) {
        make_dp(i + 1, next);
        if (i + 2 == total) umma_commit_el(sm.own_empty());
      }
      cols = next;
    }
    if (!ok) break;
    if (total == 1) umma_commit_el(sm.own_empty());
    umma_commit_el(sm.sum_full());
    step += total;
    ++item;
  }
  umma_commit_el(sm.done());
  mbar_wait_drain(sm.at(sm.done()), 0, p.status);
}

// ----------------------------------------------------------- arithmetic
// 64 columns of this warp's 32 rows of fp32 sums, times f (plus others, times
// f2), to memory in 16 bits.
template <bool kBf16, bool kOther>
__device__ __forceinline__ void store_sums(uint32_t col, uint32_t col2, uint32_t stage, uint16_t* dst, int64_t stride,
                                           int rows, int first, int d, float f, float f2, bool any) {
  uint32_t y[32] = {};
  if (any) {
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t o[32], o2[32];
      tmem_ld_32x32b_x32_issue(col + half * 32, o);
      if constexpr (kOther) tmem_ld_32x32b_x32_issue(col2 + half * 32, o2);
      tmem_wait_ld_regs(o);
      if constexpr (kOther) reg_order(o2);
#pragma unroll
      for (int x = 0; x < 32; x += 2) {
        float a, b;
        if constexpr (kBf16) {
          a = __uint_as_float(o[x]) * f;
          b = __uint_as_float(o[x + 1]) * f;
          if constexpr (kOther) {
            a = fmaf(__uint_as_float(o2[x]), f2, a);
            b = fmaf(__uint_as_float(o2[x + 1]), f2, b);
          }
        } else {
          Pair v = mul2(Pair(__uint_as_float(o[x]), __uint_as_float(o[x + 1])), Pair(f, f));
          if constexpr (kOther) v = fma2(Pair(__uint_as_float(o2[x]), __uint_as_float(o2[x + 1])), Pair(f2, f2), v);
          v.get(a, b);
        }
        y[half * 16 + x / 2] = pack2<kBf16>(a, b);
      }
    }
  }
  store_rows<64>(stage, y, dst, stride, rows, first, d);
}
__device__ __forceinline__ uint4* row_of(const HeadsView& v, int64_t token, int head) {
  return reinterpret_cast<uint4*>(static_cast<uint16_t*>(v.data) + token * v.token_stride + head * v.head_stride);
}

struct MathConst {
  float c, to_log2, cap2, in_cap;  // c brings held scores to log2 units
};

// This thread's 64 columns of a tile of scores: weights into e (times bend in
// the dK and dV kernel) and, in 16 bits, to TMEM. nl: minus the rows' lse2, of
// the walked rows in shared memory or of this thread's own row. In an edge tile
// columns outside [lo, hi) have weight 0 and those from `used` on are not
// looked at; one code for both, since its size counts.
template <bool kDkv, bool kBf16, Cap kCap, bool kBias>
__device__ __forceinline__ void make_weights(uint32_t s_col, const MathConst& k, const float* nl, float own_nl,
                                             float slope2, float far, bool live, bool edge, int used, int lo, int hi,
                                             float (&e)[64], float (&bend)[kCap && !kDkv ? 64 : 1]) {
  uint32_t u[2][32];
  tmem_ld_32x32b_x32_issue(s_col, u[0]);
  tmem_ld_32x32b_x32_issue(s_col + 32, u[1]);
  tmem_wait_ld_regs(u[0]);
  reg_order(u[1]);
  const Pair scale(k.c, k.c);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (q * 32 >= used) break;
    if constexpr (kCap != kNoCap) tanh_group<kCap == kWide>(u[q], k.in_cap, q * 32 + 32 <= used, live);
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
      float4 n;
      if constexpr (kDkv) n = *reinterpret_cast<const float4*>(nl + q * 32 + x);
      else n = make_float4(own_nl, own_nl, own_nl, own_nl);
      float z[4], d[4];
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        z[y] = __uint_as_float(u[q][x + y]);
        if constexpr (kCap != kNoCap) {
          d[y] = fmaf(-z[y], z[y], 1.f);  // z is the tangent here
          if constexpr (kBias) z[y] *= k.cap2;
        }
        if constexpr (kBias) {
          if constexpr (kCap == kNoCap) z[y] *= k.to_log2;
          z[y] = fmaf(-slope2, fabsf(far - static_cast<float>(q * 32 + x + y)), z[y]);
        }
      }
      fma2(Pair(z[0], z[1]), scale, Pair(n.x, n.y)).get(z[0], z[1]);
      fma2(Pair(z[2], z[3]), scale, Pair(n.z, n.w)).get(z[2], z[3]);
#pragma unroll
      for (int y = 0; y < 4; ++y) {
        z[y] = fast_exp2(z[y]);
        if constexpr (kCap != kNoCap) {
          if constexpr (kDkv) u[q][x + y] = __float_as_uint(z[y]), z[y] *= d[y];
          else bend[q * 32 + x + y] = d[y];
        }
        e[q * 32 + x + y] = z[y];
      }
    }
    if (edge) {
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (static_cast<unsigned>(q * 32 + x - lo) >= static_cast<unsigned>(hi - lo)) {
          e[q * 32 + x] = 0.f;
          if constexpr (kCap != kNoCap) {
            if constexpr (kDkv) u[q][x] = 0;
            else bend[q * 32 + x] = 0.f;
          }
        }
    }
    // to TMEM: the weights for dV, weights * bend for their product with K
    uint32_t pk[16];
#pragma unroll
    for (int x = 0; x < 32; x += 2) {
      const float *a = e + q * 32 + x, *g = bend + (kCap && !kDkv ? q * 32 + x : 0);
      if constexpr (kCap == kNoCap) pk[x / 2] = pack2<kBf16>(a[0], a[1]);
      else if constexpr (kDkv) pk[x / 2] = pack2<kBf16>(__uint_as_float(u[q][x]), __uint_as_float(u[q][x + 1]));
      else pk[x / 2] = pack2<kBf16>(a[0] * g[0], a[1] * g[1]);
    }
    tmem_st_32x32b_x16_issue(s_col + q * 16, pk);
  }
  tmem_wait_st();
}

// dS of the same columns to TMEM. nd: minus delta, as nl. `rest` gathers the
// sum over the row of e (dP - delta), which exact arithmetic makes 0.
template <bool kDkv, bool kBf16, Cap kCap>
__device__ __forceinline__ void make_ds(uint32_t dp_col, const float* nd, float own_nd, bool edge, int used,
                                        const float (&e)[64], const float (&bend)[kCap && !kDkv ? 64 : 1], Pair& rest) {
  uint32_t u[2][32];
  tmem_ld_32x32b_x32_issue(dp_col, u[0]);
  tmem_wait_ld_regs(u[0]);
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    if (q * 32 >= used) break;
    if (q == 0) tmem_ld_32x32b_x32_issue(dp_col + 32, u[1]);
    if (edge) {  // where nothing is seen dP may be anything
#pragma unroll
      for (int x = 0; x < 32; ++x)
        if (e[q * 32 + x] == 0.f) u[q][x] = 0;
    }
    uint32_t pk[16];
#pragma unroll
    for (int x = 0; x < 32; x += 4) {
      float4 n;
      if constexpr (kDkv) n = *reinterpret_cast<const float4*>(nd + q * 32 + x);
      else n = make_float4(own_nd, own_nd, own_nd, own_nd);
      const float* w = e + q * 32 + x;
      float d[4];
      Pair a = add2(Pair(__uint_as_float(u[q][x]), __uint_as_float(u[q][x + 1])), Pair(n.x, n.y));
      Pair b = add2(Pair(__uint_as_float(u[q][x + 2]), __uint_as_float(u[q][x + 3])), Pair(n.z, n.w));
      a = mul2(a, Pair(w[0], w[1]));
      b = mul2(b, Pair(w[2], w[3]));
      if constexpr (!kDkv) rest = add2(rest, add2(a, b));
      if constexpr (kCap && !kDkv) {
        const float* g = bend + q * 32 + x;
        a = mul2(a, Pair(g[0], g[1]));
        b = mul2(b, Pair(g[2], g[3]));
      }
      a.get(d[0], d[1]);
      b.get(d[2], d[3]);
      pk[x / 2] = pack2<kBf16>(d[0], d[1]);
      pk[x / 2 + 1] = pack2<kBf16>(d[2], d[3]);
    }
    tmem_st_32x32b_x16_issue(dp_col + q * 16, pk);
    if (q == 0) tmem_wait_ld_regs(u[1]);
  }
  tmem_wait_st();
}

template <class S, int DH, int BC, bool kDkv, bool kBf16, Cap kCap, bool kBias>
__device__ void bwd_math(const AttnParams& p, const BwdSmem<S, BC>& sm, uint32_t tmem) {
  const int wg = threadIdx.x >> 7, lane = threadIdx.x & 31, group = p.heads / p.kv_heads;
  const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;
  const uint32_t s_col = tmem + lanes + wg * 64, dp_col = s_col + S::kDp;
  const MathConst k = {kBias ? 1.f : kCap ? p.cap * kLog2e : p.scale * kLog2e, p.scale * kLog2e, p.cap * kLog2e,
                       kCap ? p.scale / p.cap : 0.f};
  uint32_t step = 0, item = 0, rows_done = 0;
  const auto wait = [&](uint32_t bar, uint32_t ph) -> bool {
    return mbar_wait_warp(bar, ph & 1, sm.abort_flag, p.status);
  };
  for (uint32_t n = 0;; ++n) {
    const int r = n % kRing;
    if (!wait(sm.info_full(r), n / kRing)) return;
    const Work w = sm.info[r];
    __syncwarp();
    if (lane == 0) mbar_arrive_a(sm.info_empty(r));
    if (!w.live) return;
    const Range g = range_of<kDkv, BC>(p, w);
    const int mine = w.row0 + static_cast<int>(threadIdx.x & 127);  // this thread's key, or row
    // columns [lo, hi) of the document that meet this thread's row, and the
    // columns from `clear` up to `clear_end` that meet every row of the block
    int lo = 0, hi = 0, clear, clear_end;
    float own_nl = -INFINITY, own_nd = 0.f;
    float2* own_stats = nullptr;
    if constexpr (kDkv) {
      lo = mine < w.keys ? (p.mask == MAXSIM_MASK_FULL || mine < w.prefix ? 0 : mine) : w.len;
      hi = w.len;
      const int last = w.row0 + kTile - 1;
      clear = last < w.keys ? (p.mask == MAXSIM_MASK_FULL || last < w.prefix ? 0 : last) : w.len;
      clear_end = w.len;
    } else {
      clear = 0;
      clear_end = w.row0 + kTile <= w.len ? row_end(w, p.mask, w.row0) : 0;
      if (mine < w.len) {
        hi = row_end(w, p.mask, mine);
        own_stats = reinterpret_cast<float2*>(p.delta) + static_cast<int64_t>(w.head) * p.T + w.start + mine;
        const float2 st = *own_stats;
        own_nl = kBf16 ? st.x : st.x + p.shifts[w.start + mine].x;
        own_nd = st.y;
      }
    }
    Pair rest(0.f, 0.f);
    for (int h = 0; h < g.heads; ++h) {
      const float slope2 = kBias && p.slopes ? p.slopes[kDkv ? w.head * group + h : w.head] * kLog2e : 0.f;
      for (int j = 0; j < g.steps; ++j, ++step) {
        const int from = g.begin + j * BC + wg * 64, used = min(64, g.end - from);  // this warpgroup's columns
        const bool edge = from < clear || g.begin + (j + 1) * BC > clear_end;
        const float* nl = sm.stats + (step % S::kStages) * 2 * BC + wg * 64;
        const float far = static_cast<float>(mine - from);
        float e[64], bend[kCap && !kDkv ? 64 : 1];
        if (!wait(sm.s_full(), step)) return;
        // the statistics came with the walked tile, whose products have been made from it
        if (kDkv && !wait(sm.walk_full(step % S::kStages), step / S::kStages)) return;
        tc_fence_after();
        if (used > 0)
          make_weights<kDkv, kBf16, kCap, kBias>(s_col, k, nl, own_nl, slope2, far, mine < w.len, edge, used, lo - from, hi - from, e, bend);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_a(sm.p_full());
        if (!wait(sm.dp_full(), step)) return;
        tc_fence_after();
        if (used > 0) make_ds<kDkv, kBf16, kCap>(dp_col, nl + BC, own_nd, edge, used, e, bend, rest);
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive_a(sm.ds_full());
          if constexpr (kDkv) mbar_arrive_a(sm.walk_empty(step % S::kStages));  // the statistics have been read
        }
      }
    }
    const bool any = g.steps > 0, live = mine < w.len;
    const float unshift = kBf16 || !any ? 1.f : p.shifts[w.start + w.row0].y;
    float off = 0.f;
    if constexpr (!kDkv) {
      float a, b;
      rest.get(a, b);
      off = a + b;
      if constexpr (S::kGroups == 2) {  // the other warpgroup has the other columns' part
        float* both = sm.stats + (rows_done & 1) * 256;  // read before anyone arrives for the row after next
        both[threadIdx.x] = off;
        __syncwarp();
        if (lane == 0) mbar_arrive_a(sm.rest_full());
        if (!wait(sm.rest_full(), rows_done)) return;
        ++rows_done;
        off = both[threadIdx.x & 127] + both[128 + (threadIdx.x & 127)];
      }
      off *= unshift;
      if (live && any && wg == 0) own_stats->y = own_nd - off;
    }
    if (any) {
      if (!wait(sm.sum_full(), item)) return;
      ++item;
      tc_fence_after();
    }
    const int row32 = w.row0 + static_cast<int>(threadIdx.x & 96), rows = w.len - row32;  // this warp's rows
    const int64_t token = w.start + static_cast<int64_t>(row32);
    const uint32_t stage = sm.stage + (threadIdx.x >> 5) * kStageBytes<64>;
    const auto base = [&](const HeadsView& v) {
      return static_cast<uint16_t*>(v.data) + token * v.token_stride + w.head * v.head_stride;
    };
    constexpr int kChunks = DH / 64;
    const uint32_t sum0 = tmem + lanes + S::kSum0, sum1 = tmem + lanes + S::kSum1;
    if constexpr (kDkv && kBf16) {
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {  // two warpgroups: one writes dV, one dK
        if (S::kGroups == 1 || wg == 0)
          store_sums<kBf16, false>(sum0 + q * 64, 0, stage, base(p.dv), p.dv.token_stride, rows, q * 64, p.d, 1.f, 0.f, any);
        if (S::kGroups == 1 || wg == 1)
          store_sums<kBf16, false>(sum1 + q * 64, 0, stage, base(p.dk), p.dk.token_stride, rows, q * 64, p.d, p.scale, 0.f, any);
      }
    } else if constexpr (kDkv) {
      // The same with a factor for dV too: one rolled code for both, with packed
      // products, since its size counts (2500 passages, 12 heads of 64: 1.54 ms, and
      // 1.62 written as above; bf16 at 400 documents of 150: 0.49 above, 0.51 here).
#pragma unroll 1
      for (int x = 0; x < 2 * kChunks / S::kGroups; ++x) {
        const bool is_dk = S::kGroups == 2 ? wg == 1 : x >= kChunks;
        const int q = x % kChunks;
        const HeadsView to = is_dk ? p.dk : p.dv;
        store_sums<kBf16, false>((is_dk ? sum1 : sum0) + q * 64, 0, stage, base(to), to.token_stride, rows, q * 64, p.d,
                                 is_dk ? p.scale * unshift : unshift, 0.f, any);
      }
    } else {
#pragma unroll
      for (int q = 0; q < kChunks; ++q)
        if (S::kGroups == 1 || q % 2 == wg)
          store_sums<kBf16, true>(sum1 + q * 64, sum0 + q * 64, stage, base(p.dq), p.dq.token_stride, rows, q * 64, p.d,
                                  p.scale * unshift, -off * p.scale * unshift, any);
    }
    tc_fence_before();  // the next item's first products overwrite the sums after its p_full / ds_full
  }
}

template <int DH, int BC, bool kDkv, bool kBf16, Cap kCap, bool kBias>
__global__ void __launch_bounds__(BwdShape<DH, BC, kDkv>::kThreads, BwdShape<DH, BC, kDkv>::kBlocks)
    attn_bwd_kernel(const __grid_constant__ BwdMaps m, const __grid_constant__ AttnParams p) {
  using S = BwdShape<DH, BC, kDkv>;
  extern __shared__ __align__(1024) uint8_t raw[];
  if (smem_u32(raw) & 1023) {  // cannot be, by the declaration; a tile copied there would fault
    if (threadIdx.x == 0) atomicOr(p.status, kDevErrTimeout);
    return;
  }
  const BwdSmem<S, BC> sm(raw);
  constexpr int kMathWarps = 4 * S::kGroups;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // known to be uniform, and the roles with it
  if (threadIdx.x == 0) {
    mbar_init(sm.at(sm.own_full()), 1);
    mbar_init(sm.at(sm.own_empty()), 1);
    for (int s = 0; s < S::kStages; ++s) {
      mbar_init(sm.at(sm.walk_full(s)), kDkv ? 2 : 1);                // the loader, and the statistics' warp
      mbar_init(sm.at(sm.walk_empty(s)), kDkv ? 1 + kMathWarps : 1);  // the products, and the statistics' readers
    }
    mbar_init(sm.at(sm.s_full()), 1);
    mbar_init(sm.at(sm.p_full()), kMathWarps);
    mbar_init(sm.at(sm.dp_full()), 1);
    mbar_init(sm.at(sm.ds_full()), kMathWarps);
    mbar_init(sm.at(sm.sum_full()), 1);
    for (int r = 0; r < kRing; ++r) {
      mbar_init(sm.at(sm.info_full(r)), 1);
      mbar_init(sm.at(sm.info_empty(r)), kMathWarps + (kDkv ? 3 : 2));
    }
    mbar_init(sm.at(sm.done()), 1);
    mbar_init(sm.at(sm.rest_full()), kMathWarps);
    *sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == kMathWarps + 1) {
    tmem_alloc(sm.tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *sm.tmem_slot, 0);
  if (warp >= kMathWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::other_regs(kCap)));
    if (warp == kMathWarps) {
      if ((threadIdx.x & 31) == 0) bwd_loader<S, BC, kDkv>(p, sm, m);
    } else if (warp == kMathWarps + 3) plan_work(p, sm, kTile, kDkv ? p.kv_heads : p.heads, !kDkv && p.mask != MAXSIM_MASK_FULL);
    else if (warp == kMathWarps + 1) bwd_products<S, DH, BC, kDkv, kBf16>(p, sm, tmem);
    else if (kDkv && warp == kMathWarps + 2) bwd_stats<S, BC, kBf16>(p, sm);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::math_regs(kCap)));
    bwd_math<S, DH, BC, kDkv, kBf16, kCap, kBias>(p, sm, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == kMathWarps + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

// A row's 16 bytes of this lane, as floats.
template <bool kBf16>
__device__ __forceinline__ void unpack8(const uint4& w, float (&f)[8]) {
  const uint32_t* x = &w.x;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    float2 y;
    if constexpr (kBf16) y = __bfloat1622float2(*reinterpret_cast<const __nv_bfloat162*>(x + k));
    else y = __half22float2(*reinterpret_cast<const __half2*>(x + k));
    f[2 * k] = y.x;
    f[2 * k + 1] = y.y;
  }
}

// Minus lse in log2 units, and minus <dO, out>, of every row and head,
// [heads][T]. A row is read by L lanes of 16 bytes each; a block takes kTokens
// tokens with all their heads, which lie together in memory. Bound by HBM
// (dO and out once). In fp16 it reads v beside them, for the greatest |dO|^2 and
// |v|^2 among a token's heads; ones that are not finite are left out, as their
// results are not finite in any range.
constexpr int kTokens = 8;
template <bool kBf16>
__global__ void __launch_bounds__(256) attn_stats_kernel(const AttnParams p, int log_l) {
  check_docs(p, blockIdx.x * int64_t(256) + threadIdx.x, gridDim.x * int64_t(256));
  const int64_t t0 = blockIdx.x * int64_t(kTokens);
  const unsigned tokens = static_cast<unsigned>(min(static_cast<int64_t>(kTokens), p.T - t0));
  const unsigned heads = p.heads, rows = tokens * heads;
  const int part = threadIdx.x & ((1 << log_l) - 1);
  __shared__ unsigned reach[2 * kTokens];
  if constexpr (!kBf16) {
    if (threadIdx.x < 2 * kTokens) reach[threadIdx.x] = 0;
    __syncthreads();
  }
#pragma unroll 2
  for (unsigned r0 = 0; r0 < rows; r0 += 256u >> log_l) {
    const unsigned r = r0 + (threadIdx.x >> log_l);
    const int64_t t = t0 + r / heads;
    const int h = static_cast<int>(r % heads);
    const bool keyed = !kBf16 && h < p.kv_heads;  // the row reads v of the head of its own number
    float s = 0.f, size = 0.f, size_v = 0.f;
    if (r < rows && part * 8 < p.d) {
      uint4 v = {};
      if (keyed) v = row_of(p.v, t, h)[part];
      float f[8], g[8];
      const uint4 a = row_of(p.dO, t, h)[part], b = row_of(p.out, t, h)[part];
      unpack8<kBf16>(a, f);
      unpack8<kBf16>(b, g);
#pragma unroll
      for (int k = 0; k < 8; k += 2) s = fmaf(f[k], g[k], fmaf(f[k + 1], g[k + 1], s));
      if constexpr (!kBf16) {
        unpack8<kBf16>(v, g);
        Pair x(0.f, 0.f), y(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const Pair a2(f[k], f[k + 1]), v2(g[k], g[k + 1]);
          x = fma2(a2, a2, x);
          y = fma2(v2, v2, y);
        }
        float lo, hi;
        x.get(lo, hi);
        size = lo + hi;
        y.get(lo, hi);
        size_v = lo + hi;
      }
    }
    for (int o = 1 << log_l >> 1; o; o >>= 1) {
      s += __shfl_xor_sync(0xffffffffu, s, o);
      if constexpr (!kBf16) {
        size += __shfl_xor_sync(0xffffffffu, size, o);
        size_v += __shfl_xor_sync(0xffffffffu, size_v, o);
      }
    }
    if (r < rows && part == 0) {
      const float lse = p.lse[static_cast<int64_t>(h) * p.T + t];
      reinterpret_cast<float2*>(p.delta)[static_cast<int64_t>(h) * p.T + t] =
          make_float2(lse == -INFINITY ? -INFINITY : -lse * kLog2e, -s);
      if (!kBf16 && size < INFINITY) atomicMax(&reach[r / heads], __float_as_uint(size));
      if (keyed && size_v < INFINITY) atomicMax(&reach[kTokens + r / heads], __float_as_uint(size_v));
    }
  }
  if constexpr (!kBf16) {
    __syncthreads();
    if (threadIdx.x < tokens)
      p.shifts[t0 + threadIdx.x] = make_float2(__uint_as_float(reach[threadIdx.x]), __uint_as_float(reach[kTokens + threadIdx.x]));
  }
}

// P and dS = P (dP - delta) are held in fp16 times 2^shift. |dP| <= |dO_i| |v_j| and
// |delta| <= |dO_i| |out_i|, with out_i among the visible v_j: twice the greatest
// product bounds dS, and times 2^shift that stays below 2^15. From 0, what they are
// without, to 14, which brings a weight of 1 to the upper end. Each token gets its
// document's (shift, 2^-shift), in place of its own |dO|^2 and |v|^2.
__global__ void __launch_bounds__(128) attn_shift_kernel(const AttnParams p) {
  for (int64_t b = blockIdx.x; b < p.B; b += gridDim.x) {
    bool bad;
    const Doc c = load_doc(p, b, bad);
    float2* of = p.shifts + c.start;
    unsigned a = 0, v = 0;  // (floats >= 0 compare as their bits)
#pragma unroll 4
    for (int i = threadIdx.x; i < c.len; i += 128) {
      const float2 x = of[i];
      a = max(a, __float_as_uint(x.x));
      if (i < c.keys) v = max(v, __float_as_uint(x.y));
    }
    a = __reduce_max_sync(0xffffffffu, a);
    v = __reduce_max_sync(0xffffffffu, v);
    __shared__ uint2 all[4];
    if ((threadIdx.x & 31) == 0) all[threadIdx.x >> 5] = make_uint2(a, v);
    __syncthreads();
    a = max(max(all[0].x, all[1].x), max(all[2].x, all[3].x));
    v = max(max(all[0].y, all[1].y), max(all[2].y, all[3].y));
    const float both = __uint_as_float(a) * __uint_as_float(v);         // of the squares: below 2^80
    const int x = static_cast<int>(__float_as_uint(both) >> 23) - 127;  // both < 2^(x+1)
    const int shift = max(0, min(14, 14 - ((x + 2) >> 1)));
    for (int i = threadIdx.x; i < c.len; i += 128)
      of[i] = make_float2(static_cast<float>(shift), __uint_as_float(static_cast<unsigned>(127 - shift) << 23));
    __syncthreads();
  }
}

template <int DH, int BC, bool kDkv, bool kBf16, Cap kCap, bool kBias>
cudaError_t bwd_launch(const BwdMaps& m, const AttnParams& p, int sm_count, cudaStream_t stream) {
  using S = BwdShape<DH, BC, kDkv>;
  auto kern = attn_bwd_kernel<DH, BC, kDkv, kBf16, kCap, kBias>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t items = (p.T / kTile + p.B) * (kDkv ? p.kv_heads : p.heads);
  const int64_t most = static_cast<int64_t>(sm_count) * S::kBlocks;
  kern<<<static_cast<int>(items < most ? items : most), S::kThreads, S::kSmem, stream>>>(m, p);
  return cudaGetLastError();
}

template <int DH, int BC, bool kDkv, bool kBf16>
cudaError_t bwd_variant(const BwdMaps& m, const AttnParams& p, int sm_count, cudaStream_t stream) {
  if (p.cap > kWideCap)  // (rare: one kernel, whose slopes may be missing)
    return bwd_launch<DH, BC, kDkv, kBf16, kWide, true>(m, p, sm_count, stream);
  if (p.cap > 0.f)
    return p.slopes ? bwd_launch<DH, BC, kDkv, kBf16, kNarrow, true>(m, p, sm_count, stream)
                    : bwd_launch<DH, BC, kDkv, kBf16, kNarrow, false>(m, p, sm_count, stream);
  return p.slopes ? bwd_launch<DH, BC, kDkv, kBf16, kNoCap, true>(m, p, sm_count, stream)
                  : bwd_launch<DH, BC, kDkv, kBf16, kNoCap, false>(m, p, sm_count, stream);
}

template <int DH, int BC>
cudaError_t bwd_both(const BwdMaps& dkv, const BwdMaps& dq, const AttnParams& p, int is_bf16, int sm_count,
                     cudaStream_t stream) {
  const cudaError_t e = is_bf16 ? bwd_variant<DH, BC, false, true>(dq, p, sm_count, stream)
                                : bwd_variant<DH, BC, false, false>(dq, p, sm_count, stream);
  if (e != cudaSuccess) return e;  // the other kernel takes the first one's deltas
  return is_bf16 ? bwd_variant<DH, BC, true, true>(dkv, p, sm_count, stream)
                 : bwd_variant<DH, BC, true, false>(dkv, p, sm_count, stream);
}

}  // namespace

maxsim_status launch_attn_bwd(const AttnParams& p, int is_bf16, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  alignas(64) BwdMaps dkv, dq;
  if (!attn_tmap(&dkv.own_a, p.k, p.T, p.kv_heads, p.d, is_bf16, kBoxRows) ||
      !attn_tmap(&dkv.own_b, p.v, p.T, p.kv_heads, p.d, is_bf16, kBoxRows) ||
      !attn_tmap(&dkv.walk_a, p.q, p.T, p.heads, p.d, is_bf16, kBoxRows) ||
      !attn_tmap(&dkv.walk_b, p.dO, p.T, p.heads, p.d, is_bf16, kBoxRows))
    return MAXSIM_ERR_CUDA;
  dq.own_a = dkv.walk_a;
  dq.own_b = dkv.walk_b;
  dq.walk_a = dkv.own_a;
  dq.walk_b = dkv.own_b;
  int log_l = 0;  // lanes of a row, a power of two
  while ((8 << log_l) < p.d) ++log_l;
  const unsigned blocks = static_cast<unsigned>((p.T + static_cast<int64_t>(kTokens) - 1) / kTokens);
  if (is_bf16) {
    attn_stats_kernel<true><<<blocks, 256, 0, stream>>>(p, log_l);
  } else {
    attn_stats_kernel<false><<<blocks, 256, 0, stream>>>(p, log_l);
    const int64_t most = 16 * static_cast<int64_t>(dev->sm_count);
    attn_shift_kernel<<<static_cast<int>(p.B < most ? p.B : most), 128, 0, stream>>>(p);
  }
  cudaError_t e = cudaGetLastError();
  if (e == cudaSuccess)
    e = p.d > 64 ? bwd_both<128, 128>(dkv, dq, p, is_bf16, dev->sm_count, stream)
                 : bwd_both<64, 64>(dkv, dq, p, is_bf16, dev->sm_count, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

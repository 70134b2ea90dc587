// attn_fwd.cu -- packed attention, forward, on tcgen05.
//
// A block owns NQ tiles of 128 rows of one document and head and walks over
// the keys that they see, 128 at a time:
//   S = Q K^T        128 x 128, both operands in shared memory, S in TMEM
//   P = 2^(S c - m)  by a warpgroup of 128 threads, one row each: no value
//                    crosses threads; P goes back to TMEM in 16 bits, over S
//   O += P V         P from TMEM, V as it lies in memory (N contiguous)
// One warp loads tiles by TMA, one issues the products; mbarriers pass tiles
// between them. The tensor cores run in order, so a product that reuses S or O
// needs no barrier behind the one that read it.
//
// The running maximum m of a row is only raised (and O and the sum rescaled)
// when it has grown by more than 2^8 since: weights then stay below 256, which
// 16 bits and the fp32 sums hold without loss, and the pass over O in TMEM is
// rare. Weights are rounded to the inputs' type for their product with V, as
// the tensor cores take nothing wider at this rate; their sum is made of the
// unrounded ones, so lse keeps fp32.
//
// Bound by the chain of one tile (softmax 1190 cycles, its two products 1033,
// the way between the warps 500), which two tiles at a time cover to seven
// tenths: 16411 causal tokens, 8 heads over 2 of 128: 0.36 ms (1.53 PFLOP/s, the
// tensor cores' burst 1.95); on documents shorter than a tile by the same chain
// over less work: 2500 passages of 78 tokens, 12 heads of 64: 0.31 ms (HBM 0.59).
//
// Keys past a document's last visible one are cut off the products (to a
// multiple of 16) and the up to 15 rows of V behind them are zeroed in shared
// memory: 0 * NaN would reach the sum.
#include <climits>

#include "attn_common.cuh"

namespace msim {
namespace {

constexpr int kTile = 128;
constexpr int kBoxRows = 64;
constexpr float kRaise = 8.f;  // log2 of how far a weight may exceed 1

template <int DH, int NQ>
struct FwdShape {
  static constexpr int kPanels = DH / 64;
  static constexpr uint32_t kPanelBytes = kTile * 128;
  static constexpr uint32_t kTileBytes = kPanels * kPanelBytes;
  static constexpr int kStages = DH == 64 || NQ == 2 ? 2 : 1;
  static constexpr int kStoreCols = NQ == 1 ? 32 : 64;  // of an output row at a time (two blocks an SM leave no more room)
  static constexpr int kQStages = DH == 64 ? 2 : 1;
  static constexpr int kThreads = NQ * 128 + 128;  // softmax warpgroups; loader, issuer, planner and an idle warp
  static constexpr int kBlocks = NQ == 1 ? 2 : 1;  // resident on an SM
  // Registers a thread: at launch (ptxas fills the launch bounds), and after
  // the softmax threads took over some of the others'.
  static constexpr int kRegsLaunch = NQ == 1 ? 128 : 168;
  static constexpr int kRegsSoftmax = NQ == 1 ? 176 : 208, kRegsOther = NQ == 1 ? 80 : 88;
  static_assert(NQ * kRegsSoftmax + kRegsOther <= (NQ + 1) * kRegsLaunch, "register split");
  static constexpr uint32_t kTmemCols = NQ == 1 ? 256 : 512;
  static constexpr uint32_t kO0 = NQ * kTile;  // TMEM columns: S of each tile, then O of each tile
  // barriers: k_full, k_empty, v_full, v_empty, s_full, p_full, o_full, info_full, info_empty, done, q_full, q_empty
  static constexpr int kBars = 4 * kStages + 3 * NQ + 2 * kRing + 1 + 2 * kQStages;
  static constexpr uint32_t kTiles = NQ * kQStages + 2 * kStages;
  static constexpr uint32_t kSmem = 1024 + kTiles * kTileBytes + NQ * 4 * kStageBytes<kStoreCols> + 8 * kBars + kRing * sizeof(Work) + 16;
};

template <int DH, int NQ>
struct FwdSmem {
  using S = FwdShape<DH, NQ>;
  uint32_t q, k, v, stage, bars;
  uint64_t* bar;
  Work* info;
  uint32_t* tmem_slot;
  int* abort_flag;
  __device__ __forceinline__ explicit FwdSmem(uint8_t* raw) {
    uint8_t* base = raw + ((1024 - (smem_u32(raw) & 1023)) & 1023);
    q = smem_u32(base);
    k = q + NQ * S::kQStages * S::kTileBytes;
    v = k + S::kStages * S::kTileBytes;
    stage = q + S::kTiles * S::kTileBytes;
    bar = reinterpret_cast<uint64_t*>(base + S::kTiles * S::kTileBytes + NQ * 4 * kStageBytes<S::kStoreCols>);
    bars = smem_u32(bar);
    info = reinterpret_cast<Work*>(bar + S::kBars);
    tmem_slot = reinterpret_cast<uint32_t*>(info + kRing);
    abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  }
  __device__ __forceinline__ uint32_t k_full(int s) const { return bars + 8 * s; }
  __device__ __forceinline__ uint32_t k_empty(int s) const { return k_full(S::kStages + s); }
  __device__ __forceinline__ uint32_t v_full(int s) const { return k_full(2 * S::kStages + s); }
  __device__ __forceinline__ uint32_t v_empty(int s) const { return k_full(3 * S::kStages + s); }
  __device__ __forceinline__ uint32_t s_full(int t) const { return k_full(4 * S::kStages + t); }
  __device__ __forceinline__ uint32_t p_full(int t) const { return s_full(NQ + t); }
  __device__ __forceinline__ uint32_t o_full(int t) const { return s_full(2 * NQ + t); }
  __device__ __forceinline__ uint32_t info_full(int r) const { return s_full(3 * NQ + r); }
  __device__ __forceinline__ uint32_t info_empty(int r) const { return s_full(3 * NQ + kRing + r); }
  __device__ __forceinline__ uint32_t done() const { return s_full(3 * NQ + 2 * kRing); }
  __device__ __forceinline__ uint32_t q_full(int s) const { return done() + 8 + 8 * s; }
  __device__ __forceinline__ uint32_t q_empty(int s) const { return q_full(S::kQStages + s); }
  __device__ __forceinline__ uint64_t* at(uint32_t b) const { return bar + (b - bars) / 8; }
};

// Keys that tile t of the item needs (0: it has no rows, or they see nothing).
__device__ __forceinline__ int tile_keys(const Work& w, int mask, int t) {
  const int first = w.row0 + t * kTile;
  return first < w.len ? row_end(w, mask, min(w.len, first + kTile) - 1) : 0;
}
__device__ __forceinline__ int tiles_of(int keys) { return (keys + kTile - 1) / kTile; }

// ---------------------------------------------------------------- loads
template <int DH, int NQ>
__device__ void fwd_loader(const AttnParams& p, const FwdSmem<DH, NQ>& sm, const CUtensorMap* mq, const CUtensorMap* mk,
                           const CUtensorMap* mv) {
  using S = FwdShape<DH, NQ>;
  if (debug_faults(p.status) & kDebugStallFwdLoader) return;  // test-only switch (maxsim_debug_set_faults)
  const int group = p.heads / p.kv_heads;
  uint32_t item = 0, kv = 0;  // items with keys; key tiles
  bool ok = true;
  const auto load = [&](uint32_t dst, const CUtensorMap* map, uint32_t bar, int head, int token, int rows) {
    const int boxes = (rows + kBoxRows - 1) / kBoxRows;
    for (int b = 0; b < boxes; ++b)
      for (int pn = 0; pn < S::kPanels; ++pn)
        tma_load_3d_a(dst + (b / 2) * S::kTileBytes + pn * S::kPanelBytes + (b % 2) * (kBoxRows * 128), map, bar, pn * 64,
                      head, token + b * kBoxRows);
  };
  const auto bytes = [](int rows) -> uint32_t { return (rows + kBoxRows - 1) / kBoxRows * S::kPanels * (kBoxRows * 128); };
  for (uint32_t n = 0; ok; ++n) {
    const int r = n % kRing;
    if (!(ok = mbar_wait_inl_a(sm.info_full(r), (n / kRing) & 1, sm.abort_flag, p.status))) break;
    const Work w = sm.info[r];
    mbar_arrive_a(sm.info_empty(r));
    if (!w.live) break;
    int keys = 0;
    for (int t = 0; t < NQ; ++t) keys = max(keys, tile_keys(w, p.mask, t));
    const int nk = tiles_of(keys);
    if (nk == 0) continue;
    const int sq = item % S::kQStages;
    if (!(ok = mbar_wait_inl_a(sm.q_empty(sq), ((item / S::kQStages) & 1) ^ 1, sm.abort_flag, p.status))) break;
    // tiles past the last row are not loaded: their products are not made either
    const int rows = min(NQ * kTile, w.len - w.row0);
    mbar_arrive_expect_tx_a(sm.q_full(sq), bytes(rows));
    load(sm.q + sq * NQ * S::kTileBytes, mq, sm.q_full(sq), w.head, w.start + w.row0, rows);
    ++item;
    for (int j = 0; j < nk; ++j, ++kv) {
      const int s = kv % S::kStages, left = min(kTile, keys - j * kTile);
      const uint32_t ph = ((kv / S::kStages) & 1) ^ 1;
      if (!(ok = mbar_wait_inl_a(sm.k_empty(s), ph, sm.abort_flag, p.status))) break;
      mbar_arrive_expect_tx_a(sm.k_full(s), bytes(left));
      load(sm.k + s * S::kTileBytes, mk, sm.k_full(s), w.head / group, w.start + j * kTile, left);
      if (!(ok = mbar_wait_inl_a(sm.v_empty(s), ph, sm.abort_flag, p.status))) {
        mbar_wait_drain(sm.at(sm.k_full(s)), ph ^ 1, p.status);  // K of this stage is in flight without its V
        break;
      }
      mbar_arrive_expect_tx_a(sm.v_full(s), bytes(left));
      load(sm.v + s * S::kTileBytes, mv, sm.v_full(s), w.head / group, w.start + j * kTile, left);
    }
  }
  if (!ok) {  // after an abort: wait (bounded) for the copies in flight
    for (uint32_t f = item > S::kQStages ? item - S::kQStages : 0; f < item; ++f)
      mbar_wait_drain(sm.at(sm.q_full(f % S::kQStages)), (f / S::kQStages) & 1, p.status);
    for (uint32_t f = kv > S::kStages ? kv - S::kStages : 0; f < kv; ++f) {
      mbar_wait_drain(sm.at(sm.k_full(f % S::kStages)), (f / S::kStages) & 1, p.status);
      mbar_wait_drain(sm.at(sm.v_full(f % S::kStages)), (f / S::kStages) & 1, p.status);
    }
  }
}

// ------------------------------------------------------------- products
template <int DH, int NQ, bool kBf16>
__device__ void fwd_products(const AttnParams& p, const FwdSmem<DH, NQ>& sm, uint32_t tmem) {
  using S = FwdShape<DH, NQ>;
  const int lane = threadIdx.x & 31;
  const uint32_t idesc = idesc_f16(kBf16, kTile, 0);
  uint32_t item = 0, kv = 0, seen_k = 0;
  uint32_t pn[NQ] = {};  // p_full phases passed
  const auto wait = [&](uint32_t bar, uint32_t ph) {
    return mbar_wait_warp(bar, ph & 1, sm.abort_flag, p.status);
  };
  bool ok = true;
  for (uint32_t n = 0; ok; ++n) {
    const int r = n % kRing;
    if (!wait(sm.info_full(r), n / kRing)) break;
    const Work w = uniform_work(sm.info[r]);
    __syncwarp();
    if (lane == 0) mbar_arrive_a(sm.info_empty(r));
    if (!w.live) break;
    int keys[NQ], most = 0;
#pragma unroll
    for (int t = 0; t < NQ; ++t) most = max(most, keys[t] = tile_keys(w, p.mask, t));
    const int nk = tiles_of(most);
    if (nk == 0) continue;
    const int sq = item % S::kQStages;
    // S_t of key tile j (keys kv + j of the stages)
    const auto score = [&](int t, int j) {
      const int cols = (min(kTile, keys[t] - j * kTile) + 15) & ~15;
      const uint32_t id = idesc | static_cast<uint32_t>(cols >> 3) << 17;
      const uint64_t a = sdesc_k_sw128(sm.q + (sq * NQ + t) * S::kTileBytes);
      const uint64_t b = sdesc_k_sw128(sm.k + (kv + j) % S::kStages * S::kTileBytes);
#pragma unroll
      for (int kk = 0; kk < DH / 16; ++kk) {
        const uint64_t step = (kk / 4) * (S::kPanelBytes >> 4) + (kk % 4) * 2;
        umma_f16_el(tmem + t * kTile, a + step, b + step, id, kk != 0);
      }
      umma_commit_el(sm.s_full(t));
    };
    const auto need_k = [&](int j) -> bool {  // waits for key tile j once
      if (seen_k > kv + j) return true;
      seen_k = kv + j + 1;
      return wait(sm.k_full((kv + j) % S::kStages), (kv + j) / S::kStages);
    };
    ok = wait(sm.q_full(sq), item / S::kQStages) && need_k(0);
    if (!ok) break;
    tc_fence_after();
#pragma unroll
    for (int t = 0; t < NQ; ++t)
      if (keys[t] > 0) score(t, 0);
    umma_commit_el(sm.k_empty(kv % S::kStages));
    if (nk == 1) umma_commit_el(sm.q_empty(sq));
    for (int j = 0; ok && j < nk; ++j) {
      const int s = (kv + j) % S::kStages;
      bool fresh = true;
#pragma unroll
      for (int t = 0; t < NQ; ++t) {
        const int left = keys[t] - j * kTile;
        if (left <= 0) continue;
        if (fresh) {
          fresh = false;
          if (!(ok = wait(sm.v_full(s), (kv + j) / S::kStages))) break;
          // rows of V behind the last key that any tile of this item sees
          const int used = min(kTile, most - j * kTile), whole = (used + 15) & ~15;
          if (used != whole) {
            const uint32_t vec = (whole - used) * 8;
            for (uint32_t e = lane; e < vec * S::kPanels; e += 32) {
              const uint32_t dst = sm.v + s * S::kTileBytes + (e / vec) * S::kPanelBytes + used * 128 + (e % vec) * 16;
              asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(dst), "r"(0) : "memory");
            }
            fence_proxy_async_smem();
            __syncwarp();
          }
        }
        if (!(ok = wait(sm.p_full(t), pn[t]))) break;
        ++pn[t];
        tc_fence_after();
        const int steps = (min(kTile, left) + 15) / 16;
        const uint64_t b = sdesc_mn_sw128(sm.v + s * S::kTileBytes, S::kPanelBytes);
        const uint32_t ido = idesc | static_cast<uint32_t>(DH >> 3) << 17 | kIdescBMnMajor;
        if (NQ == 2 && steps == 8) {  // whole tiles of long documents, without the loop's overhead (4 %)
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)
            umma_f16_ts_el(tmem + S::kO0 + t * DH, tmem + t * kTile + kk * 8, b + kk * (2048 >> 4), ido, (j | kk) != 0);
        } else {
          for (int kk = 0; kk < steps; ++kk)
            umma_f16_ts_el(tmem + S::kO0 + t * DH, tmem + t * kTile + kk * 8, b + kk * (2048 >> 4), ido, (j | kk) != 0);
        }
        if (left <= kTile) umma_commit_el(sm.o_full(t));
        if (left > kTile) {
          if (!(ok = need_k(j + 1))) break;
          tc_fence_after();
          score(t, j + 1);
        }
      }
      if (!ok) break;
      umma_commit_el(sm.v_empty(s));
      if (j + 1 < nk) {
        umma_commit_el(sm.k_empty((kv + j + 1) % S::kStages));
        if (j + 2 == nk) umma_commit_el(sm.q_empty(sq));
      }
    }
    kv += nk;
    ++item;
  }
  // every product issued here has completed before TMEM is freed
  umma_commit_el(sm.done());
  mbar_wait_drain(sm.at(sm.done()), 0, p.status);
}

// -------------------------------------------------------------- softmax
// What a softmax thread keeps of its row.
struct RowState {
  float m, sum;  // maximum in the units of the scores held, sum of the weights
  bool live;     // a row of the document: others hold what was left in shared memory, and have no say
};
struct ScoreConst {
  float c, to_log2, cap2, in_cap;  // c brings held scores to log2 units
};

// A group of 32 scores brought to the units that maxima are taken in; `far` is
// the row less the group's first key, `lim` how many of its keys are seen.
template <Cap kCap, bool kBias, bool kEdge>
__device__ __forceinline__ void finish_scores(uint32_t (&u)[32], const ScoreConst& k, float slope2, float far, int lim) {
#pragma unroll
  for (int x = 0; x < 32; ++x) {
    float z = __uint_as_float(u[x]);
    if constexpr (kCap == kNarrow) z = k.cap2 * fast_tanh(z * k.in_cap);
    if constexpr (kCap == kWide) z = k.cap2 * close_tanh(z * k.in_cap);
    if constexpr (kBias) {
      if constexpr (kCap == kNoCap) z *= k.to_log2;
      z = fmaf(-slope2, fabsf(far - static_cast<float>(x)), z);
    }
    if constexpr (kEdge) z = x < lim ? z : -INFINITY;
    u[x] = __float_as_uint(z);
  }
}
__device__ __forceinline__ float group_max(const uint32_t (&u)[32], float m) {
  float t[4] = {m, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int x = 0; x < 32; x += 2) t[x / 2 % 4] = max3(t[x / 2 % 4], __uint_as_float(u[x]), __uint_as_float(u[x + 1]));
  return fmaxf(max3(t[0], t[1], t[2]), t[3]);
}
// Weights of a group to TMEM; their sum is added to part.
template <bool kBf16>
__device__ __forceinline__ void group_weights(uint32_t p_col, const uint32_t (&u)[32], Pair scale, Pair shift, Pair (&part)[2]) {
  uint32_t pk[16];
#pragma unroll
  for (int x = 0; x < 32; x += 2) {
    float a, b;
    fma2(Pair(__uint_as_float(u[x]), __uint_as_float(u[x + 1])), scale, shift).get(a, b);
    a = fast_exp2(a);
    b = fast_exp2(b);
    part[x / 2 % 2] = add2(part[x / 2 % 2], Pair(a, b));
    pk[x / 2] = pack2<kBf16>(a, b);
  }
  tmem_st_32x32b_x16_issue(p_col, pk);
}

// The maximum of a row has become `now`: the first tile sets it, later ones
// raise it when it has grown a lot, and bring O and the sum to it.
template <int DH>
__device__ __forceinline__ void raise_max(uint32_t o_col, const ScoreConst& k, float now, bool first, RowState& st) {
  if (first) {
    st.m = now;
  } else if (__any_sync(0xffffffffu, st.live && (now - st.m) * k.c > kRaise)) {
    const float keep = now == -INFINITY ? 1.f : fast_exp2((st.m - now) * k.c);
    st.sum *= keep;
    st.m = now;
#pragma unroll 1
    for (int q = 0; q < DH / 16; ++q) {
      uint32_t o[16];
      tmem_ld_32x32b_x16(o_col + q * 16, o);
#pragma unroll
      for (int x = 0; x < 16; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * keep);
      tmem_st_32x32b_x16_issue(o_col + q * 16, o);
    }
  }
}

// One tile of scores, all seen by this thread's row, without a bias: weights to TMEM, m and sum brought
// up to date (and O with them). The scores are read twice, 32 at a time with the
// next group on its way, rather than kept: 128 registers of them spilled (0.70
// against 0.40 ms for 16411 causal tokens, 8 heads of 128). Bent scores are
// written back between.
template <int DH, bool kBf16, Cap kCap>
__device__ __forceinline__ void softmax_tile(uint32_t s_col, uint32_t o_col, const ScoreConst& k, bool first, RowState& st) {
  uint32_t u[2][32];
  float now = st.m;
  tmem_ld_32x32b_x32_issue(s_col, u[0]);
  tmem_wait_ld_regs(u[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q < 3) tmem_ld_32x32b_x32_issue(s_col + (q + 1) * 32, u[(q + 1) & 1]);
    finish_scores<kCap, false, false>(u[q & 1], k, 0.f, 0.f, 32);
    now = group_max(u[q & 1], now);
    if constexpr (kCap != kNoCap) tmem_st_32x32b_x32_issue(s_col + q * 32, u[q & 1]);
    if (q < 3) tmem_wait_ld_regs(u[(q + 1) & 1]);
  }
  if constexpr (kCap != kNoCap) tmem_wait_st();
  tmem_ld_32x32b_x32_issue(s_col, u[0]);
  raise_max<DH>(o_col, k, now, first, st);
  const float down = st.m == -INFINITY ? 0.f : -st.m * k.c;
  const Pair scale(k.c, k.c), shift(down, down);
  Pair part[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
  tmem_wait_ld_regs(u[0]);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    if (q < 3) tmem_ld_32x32b_x32_issue(s_col + (q + 1) * 32, u[(q + 1) & 1]);
    group_weights<kBf16>(s_col + q * 16, u[q & 1], scale, shift, part);
    if (q < 3) tmem_wait_ld_regs(u[(q + 1) & 1]);
  }
  float lo, hi;
  add2(part[0], part[1]).get(lo, hi);
  st.sum += lo + hi;
  tmem_wait_st();
}

// The same for any tile: of fewer than 128 columns, with some hidden from the row
// (those from `lim` on), with a distance bias: a loop over the groups of 32 that
// there are, which compares columns only where a row of the warp needs it. Short
// documents run here, and small code counts.
template <int DH, bool kBf16, Cap kCap, bool kBias>
__device__ __forceinline__ void softmax_edge(uint32_t s_col, uint32_t o_col, const ScoreConst& k, float slope2,
                                             float far, int cols, int lim, bool first, RowState& st) {
  uint32_t u[32];
  float now = st.m;
  const int groups = (cols + 31) / 32, whole = __reduce_min_sync(0xffffffffu, lim) / 32;  // groups that all rows see
#pragma unroll 1
  for (int q = 0; q < groups; ++q) {
    tmem_ld_32x32b_x32_issue(s_col + q * 32, u);
    tmem_wait_ld_regs(u);
    if (q < whole) finish_scores<kCap, kBias, false>(u, k, slope2, far - q * 32, 32);
    else finish_scores<kCap, kBias, true>(u, k, slope2, far - q * 32, lim - q * 32);
    now = group_max(u, now);
    if (kCap != kNoCap || kBias || q >= whole) tmem_st_32x32b_x32_issue(s_col + q * 32, u);
  }
  tmem_wait_st();
  raise_max<DH>(o_col, k, now, first, st);
  const float down = st.m == -INFINITY ? 0.f : -st.m * k.c;
  const Pair scale(k.c, k.c), shift(down, down);
  Pair part[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll 1
  for (int q = 0; q < groups; ++q) {
    tmem_ld_32x32b_x32_issue(s_col + q * 32, u);
    tmem_wait_ld_regs(u);
    group_weights<kBf16>(s_col + q * 16, u, scale, shift, part);
  }
  float lo, hi;
  add2(part[0], part[1]).get(lo, hi);
  st.sum += lo + hi;
  tmem_wait_st();
}

template <int DH, int NQ, bool kBf16, Cap kCap, bool kBias>
__device__ void fwd_softmax(const AttnParams& p, const FwdSmem<DH, NQ>& sm, uint32_t tmem) {
  using S = FwdShape<DH, NQ>;
  const int t = threadIdx.x >> 7, lane = threadIdx.x & 31;
  const uint32_t lanes = static_cast<uint32_t>((threadIdx.x >> 5) & 3) << 21;  // this warp's 32 TMEM lanes
  const uint32_t s_col = tmem + lanes + t * kTile, o_col = tmem + lanes + S::kO0 + t * DH;
  // scores are brought to log2 units by c, or are there already once bent or biased
  const ScoreConst k = {kCap || kBias ? 1.f : p.scale * kLog2e, p.scale * kLog2e, p.cap * kLog2e,
                        kCap == kWide ? p.scale / p.cap : kCap ? 2.f * kLog2e * p.scale / p.cap : 0.f};
  uint32_t sn = 0, on = 0;
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
    const int first = w.row0 + t * kTile, row = first + static_cast<int>(threadIdx.x & 127);
    if (first >= w.len) continue;
    const int keys = tile_keys(w, p.mask, t), nk = tiles_of(keys);
    const int end = row_end(w, p.mask, min(row, w.len - 1)), all_see = row_end(w, p.mask, first);
    const float slope2 = kBias && p.slopes ? p.slopes[w.head] * kLog2e : 0.f;
    RowState st = {-INFINITY, 0.f, row < w.len};
    for (int j = 0; j < nk; ++j, ++sn) {
      if (!wait(sm.s_full(t), sn)) return;
      tc_fence_after();
      const float far = static_cast<float>(row - j * kTile);
      if (!kBias && (j + 1) * kTile <= all_see)  // (a bias in unrolled code: 131 us where the loop takes 119)
        softmax_tile<DH, kBf16, kCap>(s_col, o_col, k, j == 0, st);
      else
        softmax_edge<DH, kBf16, kCap, kBias>(s_col, o_col, k, slope2, far, min(kTile, keys - j * kTile), end - j * kTile,
                                             j == 0, st);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_a(sm.p_full(t));
    }
    const bool some = st.sum > 0.f || st.sum != st.sum;  // a row that sees nothing is 0
    const float inv = some ? 1.f / st.sum : 0.f;
    if (nk > 0) {
      if (!wait(sm.o_full(t), on)) return;
      ++on;
      tc_fence_after();
    }
    const int64_t token = w.start + row;
    const int row32 = first + static_cast<int>(threadIdx.x & 96);  // this warp's first row
    uint16_t* dst = static_cast<uint16_t*>(p.out.data) + (w.start + static_cast<int64_t>(row32)) * p.out.token_stride +
                    w.head * p.out.head_stride;
    constexpr int kCols = S::kStoreCols;
#pragma unroll
    for (int q = 0; q < DH / kCols; ++q) {
      uint32_t o[2][32], y[kCols / 2] = {};
      if (nk > 0) {
        tmem_ld_32x32b_x32_issue(o_col + q * kCols, o[0]);
        if constexpr (kCols == 64) tmem_ld_32x32b_x32_issue(o_col + q * kCols + 32, o[1]);
        tmem_wait_ld_regs(o[0]);
        if constexpr (kCols == 64) reg_order(o[1]);
#pragma unroll
        for (int x = 0; x < kCols / 2; ++x)
          y[x] = pack2<kBf16>(__uint_as_float(o[x / 16][2 * x % 32]) * inv, __uint_as_float(o[x / 16][2 * x % 32 + 1]) * inv);
      }
      store_rows<kCols>(sm.stage + (threadIdx.x >> 5) * kStageBytes<kCols>, y, dst, p.out.token_stride, w.len - row32,
                        q * kCols, p.d);
    }
    if (p.lse && row < w.len)
      p.lse[static_cast<int64_t>(w.head) * p.T + token] = some ? (st.m * k.c + log2f(st.sum)) * kLn2 : -INFINITY;
  }
}

template <int DH, int NQ, bool kBf16, Cap kCap, bool kBias>
__global__ void __launch_bounds__(FwdShape<DH, NQ>::kThreads, FwdShape<DH, NQ>::kBlocks)
    attn_fwd_kernel(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                    const __grid_constant__ CUtensorMap mv, const __grid_constant__ AttnParams p) {
  using S = FwdShape<DH, NQ>;
  extern __shared__ uint8_t raw[];
  const FwdSmem<DH, NQ> sm(raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // known to be uniform, and the roles with it
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2 * S::kQStages; ++s) mbar_init(sm.at(sm.q_full(s)), 1);
    for (int s = 0; s < 4 * S::kStages; ++s) mbar_init(sm.at(sm.k_full(s)), 1);
    for (int t = 0; t < NQ; ++t) {
      mbar_init(sm.at(sm.s_full(t)), 1);
      mbar_init(sm.at(sm.p_full(t)), 4);      // a warpgroup's warps
      mbar_init(sm.at(sm.o_full(t)), 1);
    }
    for (int r = 0; r < kRing; ++r) {
      mbar_init(sm.at(sm.info_full(r)), 1);
      mbar_init(sm.at(sm.info_empty(r)), 4 * NQ + 2);  // softmax warps, the loader and the issuing warp
    }
    mbar_init(sm.at(sm.done()), 1);
    *sm.abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 4 * NQ + 1) {
    tmem_alloc(sm.tmem_slot, S::kTmemCols);
    tmem_relinquish();
  }
  check_docs(p, blockIdx.x * static_cast<int64_t>(S::kThreads) + threadIdx.x, gridDim.x * static_cast<int64_t>(S::kThreads));
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = __shfl_sync(0xffffffffu, *sm.tmem_slot, 0);
  if (warp >= 4 * NQ) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(S::kRegsOther));
    if (warp == 4 * NQ) {
      if ((threadIdx.x & 31) == 0) fwd_loader<DH, NQ>(p, sm, &mq, &mk, &mv);
    } else if (warp == 4 * NQ + 2) plan_work(p, sm, NQ * kTile, p.heads, p.mask != MAXSIM_MASK_FULL);
    else if (warp == 4 * NQ + 1) fwd_products<DH, NQ, kBf16>(p, sm, tmem);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(S::kRegsSoftmax));
    fwd_softmax<DH, NQ, kBf16, kCap, kBias>(p, sm, tmem);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4 * NQ + 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, S::kTmemCols);
  }
}

template <int DH, int NQ, bool kBf16, Cap kCap, bool kBias>
cudaError_t fwd_launch(const CUtensorMap* m, const AttnParams& p, int sm_count, cudaStream_t stream) {
  using S = FwdShape<DH, NQ>;
  auto kern = attn_fwd_kernel<DH, NQ, kBf16, kCap, kBias>;
  const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem);
  if (e != cudaSuccess) return e;
  const int64_t items = (p.T / (NQ * kTile) + p.B) * p.heads, most = static_cast<int64_t>(sm_count) * S::kBlocks;
  kern<<<static_cast<int>(items < most ? items : most), S::kThreads, S::kSmem, stream>>>(m[0], m[1], m[2], p);
  return cudaGetLastError();
}

template <int DH, int NQ, bool kBf16>
cudaError_t fwd_variant(const CUtensorMap* m, const AttnParams& p, int sm_count, cudaStream_t stream) {
  if (p.cap > kWideCap)  // (rare: one kernel, whose slopes may be missing)
    return fwd_launch<DH, NQ, kBf16, kWide, true>(m, p, sm_count, stream);
  if (p.cap > 0.f)
    return p.slopes ? fwd_launch<DH, NQ, kBf16, kNarrow, true>(m, p, sm_count, stream)
                    : fwd_launch<DH, NQ, kBf16, kNarrow, false>(m, p, sm_count, stream);
  return p.slopes ? fwd_launch<DH, NQ, kBf16, kNoCap, true>(m, p, sm_count, stream)
                  : fwd_launch<DH, NQ, kBf16, kNoCap, false>(m, p, sm_count, stream);
}

template <int DH, int NQ>
cudaError_t fwd_typed(const CUtensorMap* m, const AttnParams& p, int is_bf16, int sm_count, cudaStream_t stream) {
  return is_bf16 ? fwd_variant<DH, NQ, true>(m, p, sm_count, stream) : fwd_variant<DH, NQ, false>(m, p, sm_count, stream);
}

}  // namespace

bool attn_tmap(void* map, const HeadsView& v, int64_t T, int heads, int d, int is_bf16, int box_rows) {
  const uint64_t dims[3] = {static_cast<uint64_t>(d), static_cast<uint64_t>(heads), static_cast<uint64_t>(T)};
  const uint64_t strides[2] = {static_cast<uint64_t>(v.head_stride) * 2, static_cast<uint64_t>(v.token_stride) * 2};
  const uint32_t box[3] = {64, 1, static_cast<uint32_t>(box_rows)};
  return encode_tmap(map, is_bf16 ? 1 : 0, 3, v.data, dims, strides, box, 1);
}

maxsim_status launch_attn_fwd(const AttnParams& p, int is_bf16, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  alignas(64) CUtensorMap m[3];
  if (!attn_tmap(&m[0], p.q, p.T, p.heads, p.d, is_bf16, kBoxRows) ||
      !attn_tmap(&m[1], p.k, p.T, p.kv_heads, p.d, is_bf16, kBoxRows) ||
      !attn_tmap(&m[2], p.v, p.T, p.kv_heads, p.d, is_bf16, kBoxRows))
    return MAXSIM_ERR_CUDA;
  // Two tiles of rows a block halve the traffic of K and V, which heads of 128
  // need (24 documents of 1024 tokens, 16 heads: 159 against 197 us; 300 of 256,
  // 12 heads: 150 against 178), unless documents fit one tile. The number of pieces
  // is not looked at: where few leave SMs idle, tiles of their own gain little (one
  // document of 1024, 16 heads: 17.3 against 16.4 us; two: 18.1 against 20.5; one of
  // 4096, 4 heads: 49.3 against 47.5). Heads of 64 run
  // better as two blocks of one tile (300 documents of 256 tokens, 12 heads: 100
  // against 112 us; of 320: 181 against 231; 64 of 1024: 254 against 280; 200 of 512:
  // 223 against 216; 160 ragged ones with a distance bias: 119 against 131).
  const int n = dev->sm_count;
  const cudaError_t e = p.d <= 64              ? fwd_typed<64, 1>(m, p, is_bf16, n, stream)
                        : p.T / p.B >= 192 ? fwd_typed<128, 2>(m, p, is_bf16, n, stream)
                                           : fwd_typed<128, 1>(m, p, is_bf16, n, stream);
  return e == cudaSuccess ? MAXSIM_OK : MAXSIM_ERR_CUDA;
}

}  // namespace msim

// loss.cu -- softmax cross entropy over a vocabulary, whose logits are never kept,
// and its gradients.
//
//   z = scale x W^T,  lse = ln sum_v exp z_v,  loss = lse - z_target
//   dz = dloss scale (softmax - onehot),  dx = dz W,  dW = dz^T x
//
// Four matrix products, all by one kernel on tcgen05: two SMs form a pair that owns
// tiles of 256 x 256 (cta_group::2: each SM holds 128 rows of A and half of B's, so a
// tile costs each of them half the operand traffic of one that works alone), K in
// steps of 64 through six stages that TMA fills, two accumulators of 256 TMEM columns,
// so that eight warps empty one while the other is made.
//   kStats   z tile -> its rows' maxima and sums, 128 columns apart: [V / 128, T] pairs
//   kGrad    z tile again -> dz in 16 bits, a piece of the vocabulary at a time
//   kSums    the piece's dz -> dx (+= over pieces) and dW, in one launch: dx has few
//            and long tiles, dW many short ones that even out the pairs' work
// A piece's dz is bounded by 256 MB; logits live in TMEM and registers alone. Making
// them again costs a fourth product instead of T x V numbers kept between the calls.
// dz is held divided by the largest |dloss| (times 2^14 in fp16, whose range ends
// there): small gradients keep their bits, and where all rows weigh the same, which is
// usual, the -1 at the target is exact (scaled by powers of two alone it was off by up
// to 2^-9 in the same direction in every row). Its rounding to 16 bits is what the products' operands
// are: kept in two halves they would be four products instead of two. Beside the result's own rounding
// it shows where rows weigh differently (dx and dW off by 3.4e-4 in fp16, fp32 products 2.8e-4; bf16 1.9e-3
// and 1.7e-3). In fp16 dz has steps of 2^-38 of the largest dloss at the least: the dx of a row whose own
// is 2^-20 of it or less notices.
// Bound by the tensor cores (and by the power limit in long runs): 8192 rows, 65536
// columns of 2048 bf16: forward 1.04 ms (2.1 PFLOP/s; 1.15 in long runs), backward 3.4 (1.9; 3.83);
// tensor pipe active in 95 % (kStats), 92 % (kGrad), 96 % (kSums) of the cycles that SMs are. Few rows:
// 32, 30011 columns of 768 18 us on the GPU, of which 7 are W's bytes and 8 what two kernels take for
// nothing. Rows without a target go through all four products.
#include <cmath>
#include <type_traits>

#include "after.cuh"
#include "attn_common.cuh"
#include "loss.cuh"

namespace msim {
namespace {

constexpr int kEpiWarps = 8, kProducerWarp = 8, kMmaWarp = 9, kThreads = 384;
// Registers: launched with 168 a thread; the control warpgroup gives up 112 for the two that empty accumulators.
constexpr int kRegsCtl = 56, kRegsEpi = 224, kRegsLaunch = 168;
static_assert(2 * 128 * kRegsEpi + 128 * kRegsCtl <= kThreads * kRegsLaunch, "register split");
constexpr int kTile = 256, kHalf = 128, kStep = 64;
constexpr int kBox = 64;                       // 64 x 64 elements: a K-major operand comes as one copy of two
constexpr int kBoxBytes = kBox * 128;          // such boxes, one with M or N contiguous as two copies
constexpr int kStages = 6, kStageBytes = 4 * kBoxBytes;  // two boxes of A, two of B
constexpr int kAcc = 2;
constexpr int kStageOut = 32 * 128;            // a warp's way out: 32 rows of 128 bytes
constexpr int kBars = 2 * kStages + 2 * kAcc + 1;
constexpr int kSmallBytes = kBars * 8 + 16;
constexpr int kSmemBytes = 1024 + kStages * kStageBytes + kEpiWarps * kStageOut + kSmallBytes;
// The tensor core cuts each sum towards zero, so a logit of d = 2048 is off by some
// 1e-6 of itself in one direction. kStats and kGrad add no more than this many steps there and
// the parts in registers, with rounding: a quarter of that, and no more time (backward 8192 x
// 65536 x 2048 3831 us as one sum and 3831 in parts, 4096 x 16384 x 2048 492 and 506). Both have to:
// where exp(z - lse) is next to 1, what is left of it minus 1 is only as good as z is the forward's.
constexpr int kPartSteps = 8;
constexpr int kGroupM = 32;  // row tiles that share a pass over the vocabulary (4096 x 19456 x 2048: 32 165 us, 16 163, 8 166, 4 173)

constexpr uint32_t kIdescAMnMajor = 1u << 15;  // flag of the instruction descriptor: A has its M dimension contiguous

enum Mode { kStats, kGrad, kSums };

struct Maps {
  CUtensorMap a, b;        // z: x and W; dx: dz and W
  CUtensorMap a2, b2;      // dW: dz and x
  CUtensorMap out0, out1;  // kGrad: dz; kSums: dx (or its fp32 sums), dW
};

struct Params {
  LossShape s;
  int first, columns;       // the piece
  int tiles_m, tiles_n;     // of z
  int dx_m, dx_n, splits;   // kSums: dx tiles, and parts of their K
  int dw_m, dw_n, dw_splits;
  int dw_first, rounds;     // which kind is longer, and how many of the other are worth one
  int dx_wide, dw_wide;     // goes to fp32 sums
  int dx_adds;              // those of dx are added to
  const int64_t* targets;
  const float *lse, *dloss;
  float* top;               // the largest |dloss|
  int scan;                 // kGrad finds it (else it is there)
  float more;               // dz is held times this over the largest |dloss|
  float2* parts;
  float* hit;               // [T] the target's product
  float z2;                 // scale * log2(e)
  unsigned* status;
};

struct Smem {
  uint8_t *stages, *out;
  uint64_t* bars;
  uint32_t* tmem_slot;
  volatile int* abort_flag;
  uint32_t full, empty, accfull, accempty, done;
};
__device__ __forceinline__ Smem carve(uint8_t* raw) {
  Smem s;
  const uintptr_t base = (reinterpret_cast<uintptr_t>(raw) + 1023) & ~uintptr_t(1023);
  s.stages = reinterpret_cast<uint8_t*>(base);
  s.out = s.stages + kStages * kStageBytes;
  s.bars = reinterpret_cast<uint64_t*>(s.out + kEpiWarps * kStageOut);
  s.tmem_slot = reinterpret_cast<uint32_t*>(s.bars + kBars);
  s.abort_flag = reinterpret_cast<volatile int*>(s.tmem_slot + 1);
  s.full = smem_u32(s.bars);
  s.empty = s.full + 8 * kStages;
  s.accfull = s.empty + 8 * kStages;
  s.accempty = s.accfull + 8 * kAcc;
  s.done = s.accempty + 8 * kAcc;
  return s;
}

// One tile of a pair. A is K-major in z and dx, B in z alone; the others have their
// M or N dimension contiguous.
struct Tile {
  int m0, n0, n;    // n: the product's N, a multiple of 32
  int k0, steps;    // of 64
  int kind;         // 0 z, 1 dx, 2 dW
  int split;
};

__device__ __forceinline__ int width(int left) { return left >= kTile ? kTile : (left + 31) & ~31; }

template <int kMode>
__device__ __forceinline__ bool tile_of(const Params& p, int i, Tile& t) {
  const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
  t.split = 0;
  t.k0 = 0;
  if constexpr (kMode != kSums) {
    // 256 MB of parts or of dz are 2^16 tiles at the most, or as many as there are rows
    const uint32_t at = static_cast<uint32_t>(i) * pairs + pair, tiles_n = p.tiles_n;
    if (at >= static_cast<uint32_t>(p.tiles_m) * tiles_n) return false;
    const uint32_t per = kGroupM * tiles_n, group = at / per, in = at - group * per;
    const uint32_t rows = min(static_cast<uint32_t>(kGroupM), p.tiles_m - group * kGroupM), n = in / rows;
    t.kind = 0;
    t.m0 = static_cast<int>(group * kGroupM + in - n * rows) * kTile;
    t.n0 = static_cast<int>(n) * kTile;  // within the piece
    t.n = width(p.columns - t.n0);
    t.steps = (p.s.d + kStep - 1) / kStep;
    return true;
  } else {
    // The longer kind's tiles in turn, then the other's, of which pairs with one long
    // tile less have `rounds` more.
    const int n_dx = p.dx_m * p.dx_n * p.splits, n_dw = p.dw_m * p.dw_n * p.dw_splits;
    const int n_long = p.dw_first ? n_dw : n_dx, n_short = p.dw_first ? n_dx : n_dw;
    const int whole = n_long / pairs, rest = n_long - whole * pairs;
    const int mine = whole + (pair < rest);
    int64_t at;
    if (i < mine) {
      at = static_cast<int64_t>(i) * pairs + pair;
    } else {
      int k = i - mine;
      const int extra = rest ? p.rounds : 0, light = pairs - rest;
      if (pair >= rest && k < extra) {
        at = static_cast<int64_t>(k) * light + (pair - rest);
      } else {
        if (pair >= rest) k -= extra;
        at = static_cast<int64_t>(extra) * light + static_cast<int64_t>(k) * pairs + pair;
      }
      if (at >= n_short) return false;
    }
    t.kind = (i < mine) == (p.dw_first != 0) ? 2 : 1;
    const int tiles_n = t.kind == 1 ? p.dx_n : p.dw_n, per = (t.kind == 1 ? p.dx_m : p.dw_m) * tiles_n;
    const int splits = t.kind == 1 ? p.splits : p.dw_splits;
    const int steps = ((t.kind == 1 ? p.columns : p.s.T) + kStep - 1) / kStep;
    t.split = static_cast<int>(at / per);
    const int in = static_cast<int>(at - static_cast<int64_t>(t.split) * per), m = in / tiles_n;
    t.m0 = m * kTile;
    t.n0 = (in - m * tiles_n) * kTile;
    t.n = width(p.s.d - t.n0);
    t.k0 = static_cast<int>(static_cast<int64_t>(steps) * t.split / splits);
    t.steps = static_cast<int>(static_cast<int64_t>(steps) * (t.split + 1) / splits) - t.k0;
    return true;
  }
}

// ------------------------------------------------------------------ producer
constexpr uint64_t kSettleNs = 1000000;

// The producer and the issuer are whole warps that stay together, one elected lane
// of which does the work: their operands are then known to be uniform. As single
// threads beside 31 waiting ones they took 545 cycles a step, whatever the step held.

// A load into this CTA that completes on a barrier of either CTA of the pair.
__device__ __forceinline__ void tma_load_pair_el(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2"
      " [%0], [%1, {%3, %4}], [%2];\n\t}" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect_tx_el(uint32_t bar, uint32_t bytes) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar),
      "r"(bytes)
      : "memory");
}
__device__ __forceinline__ void umma_f16_pair_el(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc,
                                                 uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p, e;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate)
      : "memory");
}
__device__ __forceinline__ void umma_commit_pair_el(uint32_t bar, uint16_t mask) {
  asm volatile(
      "{\n\t.reg .pred e;\n\t"
      "elect.sync _|e, 0xffffffff;\n\t"
      "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t}" ::"r"(bar),
      "h"(mask)
      : "memory");
}

template <int kMode>
__device__ void produce(const Params& p, const Smem& sm, const Maps& maps, uint32_t rank) {
  if (debug_faults(p.status) & kDebugStallFwdLoader) return;
  const uint32_t stage0 = smem_u32(sm.stages), full_even = mapa_shared(sm.full, 0);
  uint32_t fills = 0;
  int s = 0;
  uint32_t ph = 0;
  Tile t;
  bool ok = true;
  for (int i = 0; ok && tile_of<kMode>(p, i, t); ++i) {
    const CUtensorMap *a = t.kind == 2 ? &maps.a2 : &maps.a, *b = t.kind == 2 ? &maps.b2 : &maps.b;
    const int am = t.m0 + static_cast<int>(rank) * kHalf, bn = t.n0 + static_cast<int>(rank) * (t.n / 2);
    const int boxes_b = t.kind == 0 || t.n / 2 > kBox ? 2 : 1;
    for (int k = 0; k < t.steps; ++k) {
      if (!mbar_wait_warp(sm.empty + 8 * s, ph ^ 1u, sm.abort_flag, p.status)) {
        ok = false;
        break;
      }
      const uint32_t bar = full_even + 8 * s, to = stage0 + static_cast<uint32_t>(s) * kStageBytes;
      const int kk = (t.k0 + k) * kStep;
      if (rank == 0) mbar_arrive_expect_tx_el(sm.full + 8 * s, 2 * (2 + boxes_b) * kBoxBytes);
      if (t.kind == 2) {
        tma_load_pair_el(to, a, bar, am, kk);
        tma_load_pair_el(to + kBoxBytes, a, bar, am + kBox, kk);
      } else {
        tma_load_pair_el(to, a, bar, kk, am);
      }
      if (t.kind == 0) {
        tma_load_pair_el(to + 2 * kBoxBytes, b, bar, kk, p.first + bn);
      } else {
        const int kb = (t.kind == 1 ? p.first : 0) + kk;
        tma_load_pair_el(to + 2 * kBoxBytes, b, bar, bn, kb);
        if (boxes_b == 2) tma_load_pair_el(to + 3 * kBoxBytes, b, bar, bn + kBox, kb);
      }
      ++fills;
      if (++s == kStages) s = 0, ph ^= 1u;
    }
  }
  if (ok || !fills) return;
  // Given up: copies in flight land before the block ends. The even CTA waits for
  // those that it announced; the odd one, whose copies signal there, for a
  // thousand times what a copy takes.
  if (rank == 0) {
    for (uint32_t f = fills > kStages ? fills - kStages : 0; f < fills; ++f)
      mbar_wait_drain(sm.bars + (f % kStages), (f / kStages) & 1u, p.status);
  }
  const uint64_t t0 = globaltimer_ns();
  while (globaltimer_ns() - t0 < kSettleNs) {
  }
}

// ------------------------------------------------- products (even CTA, one warp)
template <int kMode>
__device__ void multiply(const Params& p, const Smem& sm, uint32_t tmem_base) {
  const uint32_t stage0 = smem_u32(sm.stages);
  const uint64_t kmajor = sdesc_k_sw128(stage0), mnmajor = sdesc_mn_sw128(stage0, kBoxBytes);
  const uint16_t both = 3;
  int s = 0, a = 0;
  uint32_t ph = 0, aph = 0;
  Tile t;
  bool ok = true;
  for (int i = 0; ok && tile_of<kMode>(p, i, t); ++i) {
    if (t.steps == 0) continue;
    const bool a_mn = t.kind == 2, b_mn = t.kind != 0;
    const uint32_t idesc = idesc_f16(p.s.is_bf16, kTile, t.n) | (a_mn ? kIdescAMnMajor : 0u) | (b_mn ? kIdescBMnMajor : 0u);
    const uint64_t ad0 = a_mn ? mnmajor : kmajor, bd0 = (b_mn ? mnmajor : kmajor) + ((2 * kBoxBytes) >> 4);
    const uint64_t a_step = a_mn ? 2048 >> 4 : 2, b_step = b_mn ? 2048 >> 4 : 2;
    for (int k = 0; ok && k < t.steps;) {
      const int part = kMode == kSums ? t.steps : min(t.steps, k + kPartSteps);
      if (!mbar_wait_warp(sm.accempty + 8 * a, aph ^ 1u, sm.abort_flag, p.status)) {
        ok = false;
        break;
      }
      const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(a * kTile);
      uint32_t adds = 0;
      for (; k < part; ++k) {
        if (!mbar_wait_warp(sm.full + 8 * s, ph, sm.abort_flag, p.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        const uint64_t at = static_cast<uint64_t>((s * kStageBytes) >> 4);
#pragma unroll
        for (int x = 0; x < 4; ++x, adds = 1)
          umma_f16_pair_el(d_tmem, ad0 + at + x * a_step, bd0 + at + x * b_step, idesc, adds);
        umma_commit_pair_el(sm.empty + 8 * s, both);
        if (++s == kStages) s = 0, ph ^= 1u;
      }
      if (!ok) break;
      umma_commit_pair_el(sm.accfull + 8 * a, both);
      if (++a == kAcc) a = 0, aph ^= 1u;
    }
  }
  umma_commit_pair_el(sm.done, 1);  // TMEM is freed only after the last product
  mbar_wait_drain(sm.bars + kBars - 1, 0, p.status);
}

// ------------------------------------------------------------------ epilogue
// A warp's 32 rows of 128 bytes, 16-byte parts exchanged as TMA's 128-byte swizzle does.
__device__ __forceinline__ void put_row(uint32_t stage, int lane, const uint32_t (&w)[32]) {
#pragma unroll
  for (int c = 0; c < 8; ++c)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(stage + lane * 128 + ((c ^ (lane & 7)) * 16)),
                 "r"(w[4 * c]), "r"(w[4 * c + 1]), "r"(w[4 * c + 2]), "r"(w[4 * c + 3])
                 : "memory");
}
__device__ __forceinline__ void store_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void store_wait() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }
template <bool kAdd>
__device__ __forceinline__ void store_tile(const CUtensorMap* map, uint32_t from, int x, int y, int z) {
  if constexpr (kAdd)
    asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(from), "r"(x), "r"(y), "r"(z)
                 : "memory");
  else
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(from), "r"(x), "r"(y), "r"(z)
                 : "memory");
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}

// The warp's staged rows go out at column x of row y.
__device__ __forceinline__ void send(const CUtensorMap* map, uint32_t stage, int lane, int x, int y, int z, bool adds) {
  fence_proxy_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (adds) store_tile<true>(map, stage, x, y, z);
    else store_tile<false>(map, stage, x, y, z);
  }
}

// The sums of dz's products are multiplied by this at the end.
__device__ __forceinline__ float usable(float top) { return top > 0.f ? top : 1.f; }
// By both parts one after the other where their product leaves the normal numbers, which the
// results need not do.
struct Gain {
  float first, then;
  __device__ __forceinline__ float of(float sum) const { return sum * first * then; }
};
__device__ __forceinline__ Gain gain_of(const float* top, float scale, float more) {
  const float a = usable(*top) / more, both = a * scale;
  return both >= 0x1p-126f && both < INFINITY ? Gain{both, 1.f} : Gain{a, scale};
}
// The largest finite |dloss| of rows with a target, found by n threads (a row whose own is
// not spoils no other one's); bad targets are reported.
__device__ __forceinline__ float largest(const float* dloss, const int64_t* targets, int T, int64_t V, int thread, int n,
                                         unsigned* status) {
  float top = 0.f;
  for (int i = thread; i < T; i += n) {
    const int64_t t = targets[i];
    if (t >= V) atomicOr(status, kDevErrBadInput);
    const float size = fabsf(dloss[i]);
    if (t >= 0 && t < V && size < INFINITY) top = fmaxf(top, size);
  }
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  return top;
}

// Thread = row (TMEM lane); warps w and w + 4 share a lane quarter and take half of the columns each.
template <int kMode, bool kBf16>
__device__ void finish(const Params& p, const Smem& sm, const Maps& maps, uint32_t tmem_base, uint32_t rank) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, quarter = warp & 3, half = warp >> 2;
  const uint32_t lanes = static_cast<uint32_t>(quarter * 32) << 16, accempty_r = mapa_shared(sm.accempty, 0);
  const uint32_t stage = smem_u32(sm.out) + warp * kStageOut;
  int a = 0;
  uint32_t aph = 0;
  Tile t;
  float whole = 1.f;  // what dloss is divided by
  Gain gain = {};
  if constexpr (kMode == kGrad) {
    float top;
    if (p.scan) {  // each block finds it for itself, while its first tile is made
      top = largest(p.dloss, p.targets, p.s.T, p.s.V, threadIdx.x, 32 * kEpiWarps, p.status);
      float* s = reinterpret_cast<float*>(sm.out);
      if (lane == 0) s[warp * (kStageOut / 4)] = top;
      named_bar_sync(1, 32 * kEpiWarps);
      for (int w = 0; w < kEpiWarps; ++w) top = fmaxf(top, s[w * (kStageOut / 4)]);
      named_bar_sync(1, 32 * kEpiWarps);
      if (blockIdx.x == 0 && threadIdx.x == 0) *p.top = top;
    } else {
      top = *p.top;
    }
    whole = usable(top);
  }
  if constexpr (kMode == kSums) gain = gain_of(p.top, p.s.scale, p.more);  // for what is not summed on
  // what a tile's rows need is asked for while the tile before is worked on
  int64_t to_next = -1;
  float lse_next = 0.f, dloss_next = 0.f;
  const auto ask = [&](const Tile& u) {
    const int row = u.m0 + static_cast<int>(rank) * kHalf + quarter * 32 + lane;
    if (kMode == kSums || row >= p.s.T) return;
    to_next = p.targets[row];
    if constexpr (kMode == kGrad) lse_next = p.lse[row], dloss_next = p.dloss[row];
  };
  Tile next;
  bool another = tile_of<kMode>(p, 0, next);
  if (another) ask(next);
  for (int i = 0; another; ++i) {
    t = next;
    const int row0 = t.m0 + static_cast<int>(rank) * kHalf + quarter * 32, row = row0 + lane;
    const int col0 = half * kHalf;  // within the tile
    const int chunks = min(4, max(0, (t.n - col0 + 31) / 32));
    int target = -1;
    float lse2 = 0.f, coef = 0.f;
    if (kMode != kSums && row < p.s.T) {
      const int64_t g = to_next - p.first - t.n0 - col0;
      target = g >= 0 && g < kHalf ? static_cast<int>(g) : -1;
      lse2 = lse_next * kLog2e;
      coef = to_next >= 0 && to_next < p.s.V ? dloss_next / whole * p.more : 0.f;
    }
    another = tile_of<kMode>(p, i + 1, next);
    if (another) ask(next);
    if (t.steps == 0) continue;
    uint32_t v[4][32];
    bool ok = true;
    for (int k = 0; k < t.steps; k += kMode == kSums ? t.steps : kPartSteps) {
      __syncwarp();
      ok = mbar_wait_warp(sm.accfull + 8 * a, aph, sm.abort_flag, p.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t at = tmem_base + lanes + static_cast<uint32_t>(a * kTile + col0);
      if (k == 0) {
#pragma unroll
        for (int c = 0; c < 4; ++c)
          if (c < chunks) tmem_ld_32x32b_x32_issue(at + 32 * c, v[c]);
        tmem_wait_ld_regs(v[0]);
#pragma unroll
        for (int c = 1; c < 4; ++c) reg_order(v[c]);
      } else {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= chunks) continue;
          uint32_t u[32];
          tmem_ld_32x32b_x32_issue(at + 32 * c, u);
          tmem_wait_ld_regs(u);
#pragma unroll
          for (int x = 0; x < 32; ++x) v[c][x] = __float_as_uint(__uint_as_float(v[c][x]) + __uint_as_float(u[x]));
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        if (rank == 0) mbar_arrive_a(sm.accempty + 8 * a);
        else mbar_arrive_remote(accempty_r + 8 * a);
      }
      if (++a == kAcc) a = 0, aph ^= 1u;
    }
    if (!ok) break;
    // Most tiles are whole and hold no row's target: code of their own, without a question
    // for each 32 columns, across which the compiler would move nothing (8192 rows, 65536
    // columns of 64, where the epilogue is what bounds the forward: 219 -> 175 us).
    const int valid = kMode == kSums ? 0 : p.columns - t.n0 - col0;  // of this warp's columns
    const bool full = __all_sync(0xffffffffu, valid >= kHalf), hits = __any_sync(0xffffffffu, target >= 0);
    if constexpr (kMode == kStats) {
      const auto statistics = [&](auto is_full) {
        constexpr bool kFull = decltype(is_full)::value;
        float tops[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          tops[c] = -INFINITY;
          if (!kFull && c >= chunks) continue;
          if (!kFull)
#pragma unroll
            for (int x = 0; x < 32; ++x)
              if (c * 32 + x >= valid) v[c][x] = __float_as_uint(-INFINITY);
          float other = -INFINITY;
#pragma unroll
          for (int x = 0; x < 32; x += 4) {
            tops[c] = max3(tops[c], __uint_as_float(v[c][x]), __uint_as_float(v[c][x + 1]));
            other = max3(other, __uint_as_float(v[c][x + 2]), __uint_as_float(v[c][x + 3]));
          }
          tops[c] = fmaxf(tops[c], other);
        }
        const float m2 = fmaxf(max3(tops[0], tops[1], tops[2]), tops[3]) * p.z2;
        const Pair z2(p.z2, p.z2), less(-m2, -m2);
        Pair sums[2] = {Pair(0.f, 0.f), Pair(0.f, 0.f)};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (!kFull && c >= chunks) continue;
#pragma unroll
          for (int x = 0; x < 32; x += 2) {
            float e, f;
            fma2(Pair(__uint_as_float(v[c][x]), __uint_as_float(v[c][x + 1])), z2, less).get(e, f);
            sums[x / 2 & 1] = add2(sums[x / 2 & 1], Pair(fast_exp2(e), fast_exp2(f)));
          }
        }
        if (row < p.s.T && valid > 0) {
          float e, f;
          add2(sums[0], sums[1]).get(e, f);
          p.parts[static_cast<int64_t>((t.n0 + col0) / kHalf) * p.s.T + row] = make_float2(m2, e + f);
        }
      };
      if (hits) {
        float z = 0.f;
#pragma unroll
        for (int c = 0; c < 4; ++c)
#pragma unroll
          for (int x = 0; x < 32; ++x)
            if (target == c * 32 + x) z = __uint_as_float(v[c][x]);
        if (target >= 0) p.hit[row] = z;
      }
      if (full) statistics(std::true_type());
      else statistics(std::false_type());
    } else if constexpr (kMode == kGrad) {
      const Pair z2(p.z2, p.z2), less(-lse2, -lse2), factor(coef, coef);
      const auto gradients = [&](auto is_full) {
        constexpr bool kFull = decltype(is_full)::value;
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          if (!kFull && c >= chunks) continue;
          uint32_t w[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2) {
            float e[2];
            fma2(Pair(__uint_as_float(v[c + x / 32][x % 32]), __uint_as_float(v[c + x / 32][x % 32 + 1])), z2, less).get(e[0], e[1]);
            mul2(Pair(fast_exp2(e[0]), fast_exp2(e[1])), factor).get(e[0], e[1]);
            w[x / 2] = pack2<kBf16>(e[0], e[1]);
          }
          if (hits) {
#pragma unroll
            for (int x = 0; x < 64; ++x)
              if (target == c * 32 + x) {
                const float q = fast_exp2(fmaf(__uint_as_float(v[c + x / 32][x % 32]), p.z2, -lse2));
                const uint32_t one = pack2<kBf16>((q - 1.f) * coef, 0.f) & 0xFFFFu;
                w[x / 2] = x & 1 ? (w[x / 2] & 0xFFFFu) | one << 16 : (w[x / 2] & 0xFFFF0000u) | one;
              }
          }
          if (lane == 0) store_wait_read();
          __syncwarp();
          put_row(stage, lane, w);
          if (row0 < p.s.T && (kFull || t.n0 + col0 + c * 32 < p.columns))
            send(&maps.out0, stage, lane, t.n0 + col0 + c * 32, row0, 0, false);
        }
      };
      if (full) gradients(std::true_type());
      else gradients(std::false_type());
    } else {
      const bool dx = t.kind == 1;
      const int rows = dx ? p.s.T : p.columns;
      const int y = dx ? row0 : p.first + row0;
      if (dx ? p.dx_wide : p.dw_wide) {
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          if (c >= chunks) continue;
          if (lane == 0) store_wait_read();
          __syncwarp();
          put_row(stage, lane, v[c]);
          if (row0 < rows && t.n0 + col0 + c * 32 < p.s.d)
            send(dx ? &maps.out0 : &maps.out1, stage, lane, t.n0 + col0 + c * 32, row0, t.split, dx && p.dx_adds);
        }
      } else {
#pragma unroll
        for (int c = 0; c < 4; c += 2) {
          if (c >= chunks) continue;
          uint32_t w[32];
#pragma unroll
          for (int x = 0; x < 64; x += 2)
            w[x / 2] = pack2<kBf16>(gain.of(__uint_as_float(v[c + x / 32][x % 32])),
                                    gain.of(__uint_as_float(v[c + x / 32][x % 32 + 1])));
          if (lane == 0) store_wait_read();
          __syncwarp();
          put_row(stage, lane, w);
          if (row0 < rows && t.n0 + col0 + c * 32 < p.s.d)
            send(dx ? &maps.out0 : &maps.out1, stage, lane, t.n0 + col0 + c * 32, y, 0, false);
        }
      }
    }
  }
  if (kMode != kStats && lane == 0) store_wait();
}

template <int kMode, bool kBf16>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    loss_kernel(const __grid_constant__ Maps maps, const Params p) {
  extern __shared__ __align__(16) uint8_t raw[];
  const Smem sm = carve(raw);
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);  // known to be the same in all lanes
  const uint32_t rank = cluster_ctarank();
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(sm.bars + s, 1);            // full: the copies of both CTAs, on the even one
      mbar_init(sm.bars + kStages + s, 1);  // empty: the products' commit, to both CTAs
    }
    for (int i = 0; i < kAcc; ++i) {
      mbar_init(sm.bars + 2 * kStages + i, 1);                     // accfull
      mbar_init(sm.bars + 2 * kStages + kAcc + i, 2 * kEpiWarps);  // accempty: the warps of both CTAs, on the even one
    }
    mbar_init(sm.bars + kBars - 1, 1);
    *sm.abort_flag = 0;
    fence_mbar_init_cluster();
  }
  if (warp == kMmaWarp) tmem_alloc_pair(sm.tmem_slot, 512);
  if (warp == kProducerWarp && (threadIdx.x & 31) == 0) {
    tma_prefetch_desc(&maps.a);
    tma_prefetch_desc(&maps.b);
  }
  let_next_begin();
  tc_fence_before();
  cluster_sync_all();
  tc_fence_after();
  wait_for_previous();
  const uint32_t tmem_base = *sm.tmem_slot;
  if (warp >= kEpiWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsCtl));
    if (warp == kProducerWarp) produce<kMode>(p, sm, maps, rank);
    else if (warp == kMmaWarp && rank == 0) multiply<kMode>(p, sm, tmem_base);
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsEpi));
    finish<kMode, kBf16>(p, sm, maps, tmem_base, rank);
  }
  __syncwarp();
  tc_fence_before();
  cluster_sync_all();  // neither CTA leaves while the other may still signal it
  if (warp == kMmaWarp) {
    tc_fence_after();
    tmem_dealloc_pair(tmem_base, 512);
  }
}

// ------------------------------------------------------------- small kernels
// A row's parts become its lse and loss: 32 rows a block, 32 warps along the parts,
// each with eight loads in flight.
__global__ void __launch_bounds__(1024) join_kernel(const float2* parts, int n, int T, int64_t V, const int64_t* targets,
                                                    const float* hit, float z2, float* loss, float* lse,
                                                    unsigned* status) {
  __shared__ float2 s[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, row = blockIdx.x * 32 + lane;
  float top = -INFINITY, sum = 0.f;
  wait_for_previous();
  if (row < T)
    for (int i = warp; i < n; i += 256) {
      float2 q[8];
#pragma unroll
      for (int u = 0; u < 8; ++u)
        q[u] = i + 32 * u < n ? parts[static_cast<int64_t>(i + 32 * u) * T + row] : make_float2(-INFINITY, 0.f);
      float m = top;
#pragma unroll
      for (int u = 0; u < 8; ++u) m = fmaxf(m, q[u].x);
      const float base = m == -INFINITY ? 0.f : m;  // the first, or a part without a number
      sum *= exp2f(top - base);
#pragma unroll
      for (int u = 0; u < 8; ++u) sum += q[u].y * exp2f(q[u].x - base);
      top = m;
    }
  s[warp][lane] = make_float2(top, sum);
  __syncthreads();
  // a warp a row
  const float2 mine = s[lane][warp];
  top = mine.x;
#pragma unroll
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(~0u, top, o));
  sum = mine.y * exp2f(mine.x - (top == -INFINITY ? 0.f : top));
#pragma unroll
  for (int o = 16; o; o >>= 1) sum += __shfl_xor_sync(~0u, sum, o);
  const int mine_row = blockIdx.x * 32 + warp;
  if (lane || mine_row >= T) return;
  const float over = log2f(sum);  // the maximum's own logit included
  lse[mine_row] = (top + over) * kLn2;
  const int64_t t = targets[mine_row];
  if (t >= V) atomicOr(status, kDevErrBadInput);
  // from the maximum, not from lse: small losses are no difference of large rounded numbers
  loss[mine_row] = t >= 0 && t < V ? (over - fmaf(hit[mine_row], z2, -top)) * kLn2 : 0.f;
}

// The largest |dloss| of many rows: more than each block of kGrad should read. One block that
// reads them all, against each for itself: 512 rows, 2 columns of 64 14.4 and 12.7 us for the whole
// backward, 2048 16.8 and 16.9, 8192 20.7 and 24.9, 32768 29.0 and 47.5; 5000 columns of 512 29.0 and
// 28.4, 45.9 and 44.9, 91.2 and 100, 408 and 434. The one block takes 0.31 ms for 600001 rows.
constexpr int kScanRows = 2048;
__global__ void __launch_bounds__(1024) top_kernel(const float* dloss, const int64_t* targets, int T, int64_t V, float* out,
                                                   unsigned* status) {
  __shared__ float s[32];
  let_next_begin();
  float top = largest(dloss, targets, T, V, threadIdx.x, 1024, status);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = top;
  __syncthreads();
  if (threadIdx.x) return;
  for (int w = 1; w < 32; ++w) top = fmaxf(top, s[w]);
  *out = top;
}

// dx or dW: the parts' fp32 sums, times the gain.
template <typename T>
__global__ void __launch_bounds__(256) fold_kernel(const float* sums, int splits, int64_t n, int d, const float* top,
                                                   float scale, float more, T* out, int64_t stride) {
  const int64_t i = (blockIdx.x * int64_t(256) + threadIdx.x) * 8;
  wait_for_previous();
  if (i >= n) return;
  const Gain gain = gain_of(top, scale, more);
  float a[8] = {};
  for (int s = 0; s < splits; ++s) {
    const float4* q = reinterpret_cast<const float4*>(sums + s * n + i);
    const float4 u = q[0], v = q[1];
    a[0] += u.x, a[1] += u.y, a[2] += u.z, a[3] += u.w, a[4] += v.x, a[5] += v.y, a[6] += v.z, a[7] += v.w;
  }
  const int64_t row = i / d;
  alignas(16) T o[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) o[j] = static_cast<T>(gain.of(a[j]));
  *reinterpret_cast<uint4*>(out + row * stride + (i - row * d)) = *reinterpret_cast<uint4*>(o);
}

// x with rows that begin on 128-byte boundaries.
__global__ void __launch_bounds__(256) align_kernel(const uint16_t* x, int64_t stride, int64_t n, int d, uint16_t* out, int wide) {
  const int64_t i = (blockIdx.x * int64_t(256) + threadIdx.x) * 8;
  let_next_begin();
  if (i >= n) return;
  const int64_t row = i / d;
  *reinterpret_cast<uint4*>(out + row * wide + (i - row * d)) = *reinterpret_cast<const uint4*>(x + row * stride + (i - row * d));
}

// ---------------------------------------------------------------------- host
constexpr int64_t kPieceBytes = int64_t(256) << 20;

int up_to(int64_t v, int to) { return static_cast<int>((v + to - 1) / to); }
size_t padded(size_t bytes) { return (bytes + 255) & ~size_t(255); }

// Columns of a piece: at most 256 MB of dz, in whole tiles, one tile at least.
int piece_columns(const LossShape& s) {
  const int64_t most = kPieceBytes / (2 * static_cast<int64_t>(s.T)) / kTile * kTile;
  const int64_t all = static_cast<int64_t>(up_to(s.V, kTile)) * kTile;
  return static_cast<int>(most < kTile ? kTile : most < all ? most : all);
}

// Rows of 128-byte multiples are read in whole lines. Others straddle two, and where
// both operands of z do, the copies' requests bound the product (1531 rows, 50021 columns
// of 1000: 117 us, 79 without copies): x, the smaller one, is then copied into aligned
// rows first (101 us). That pays from 1e10 to 2e10 operations on (1000 rows, 4000 columns of
// 1000, 8e9: 29 us against 25; 300 rows, 20000 columns, 1.2e10: 29 against 31).
bool aligns(const LossShape& s) {
  return s.d % kStep != 0 && 2. * s.T * s.V * s.d >= 2e10;
}
int aligned_width(const LossShape& s) { return up_to(s.d, kStep) * kStep; }
size_t aligned_bytes(const LossShape& s, int64_t rows) {
  return aligns(s) ? padded(static_cast<size_t>(rows) * aligned_width(s) * 2) : 0;
}
// The view that z's product reads: `x` itself, or its copy at `to`.
bool aligned_rows(const LossShape& s, maxsim_rows* x, int64_t rows, void* to, cudaStream_t stream, bool* copied) {
  *copied = aligns(s) && (x->row_stride % kStep != 0 || reinterpret_cast<uintptr_t>(x->data) % 128 != 0);
  if (!*copied) return true;
  const int64_t n = rows * s.d;
  align_kernel<<<static_cast<int>((n / 8 + 255) / 256), 256, 0, stream>>>(
      static_cast<const uint16_t*>(x->data), x->row_stride, n, s.d, static_cast<uint16_t*>(to), aligned_width(s));
  *x = {to, aligned_width(s)};
  return cudaGetLastError() == cudaSuccess;
}

// How the tiles of dx are cut along the vocabulary, and those of dW along the rows: no
// part longer than a pair's share of the launch, with an epilogue counted as eight
// steps, nor shorter than 32 steps, which the launch that adds parts up costs (32 rows,
// 2000 columns of 256, both directions: cut at 16 steps 26.3 us captured and 55 called
// one by one, at 32 27.9 and 47; 2000 rows, 5000 columns of 512 the same).
void split_counts(const LossShape& s, int columns, int pairs, int* dx, int* dw) {
  const int64_t steps_v = up_to(columns, kStep), steps_t = up_to(s.T, kStep), n = up_to(s.d, kTile);
  int64_t share = (up_to(s.T, kTile) * n * (steps_v + 8) + up_to(columns, kTile) * n * (steps_t + 8)) / pairs;
  if (share < 32) share = 32;
  const auto count = [&](int64_t steps) { return static_cast<int>(steps <= share ? 1 : steps > 64 * share ? 64 : (steps + share - 1) / share); };
  *dx = count(steps_v);
  *dw = count(steps_t);
}

bool map_in(CUtensorMap* m, const LossShape& s, const void* data, int64_t stride, int64_t inner, int64_t rows, uint32_t box_rows) {
  const uint64_t dims[2] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(rows)};
  const uint64_t strides[1] = {static_cast<uint64_t>(stride) * 2};
  const uint32_t box[2] = {kBox, box_rows};
  return encode_tmap(m, s.is_bf16 ? 1 : 0, 2, const_cast<void*>(data), dims, strides, box, 1);
}
bool map_out(CUtensorMap* m, int type, int esize, void* data, int64_t stride, int64_t inner, int64_t rows, int64_t depth) {
  const uint64_t dims[3] = {static_cast<uint64_t>(inner), static_cast<uint64_t>(rows), static_cast<uint64_t>(depth)};
  const uint64_t strides[2] = {static_cast<uint64_t>(stride) * esize, depth > 1 ? static_cast<uint64_t>(stride) * rows * esize : static_cast<uint64_t>(stride) * esize};
  const uint32_t box[3] = {static_cast<uint32_t>(128 / esize), 32, 1};
  return encode_tmap(m, type, 3, data, dims, strides, box, 1);
}

template <int kMode>
cudaError_t launch(const Maps& maps, const Params& p, const DeviceInfo& dev, int64_t tiles, bool follows, cudaStream_t stream) {
  static Fits known[2];
  const auto go = [&](auto kernel, Fits& seen) {
    int fit = 1;
    const cudaError_t e = blocks_that_fit(seen, dev, kernel, kThreads, kSmemBytes, &fit);
    if (e != cudaSuccess) return e;
    const int64_t most = dev.sm_count / 2, pairs = tiles < most ? tiles : most;
    const int grid = static_cast<int>(2 * pairs);
    if (follows) return launch_after(kernel, grid, kThreads, kSmemBytes, stream, maps, p);
    kernel<<<grid, kThreads, kSmemBytes, stream>>>(maps, p);
    return cudaGetLastError();
  };
  return p.s.is_bf16 ? go(loss_kernel<kMode, true>, known[0]) : go(loss_kernel<kMode, false>, known[1]);
}

struct Space {  // of the backward's workspace
  size_t x, dz, sums, dw_sums, bytes;
  int columns, splits, dw_splits;
  bool wide;  // dx goes through fp32 sums
};
Space plan(const LossShape& s, int pairs) {
  Space w;
  w.columns = piece_columns(s);
  const int first = w.columns < s.V ? w.columns : static_cast<int>(s.V);
  split_counts(s, first, pairs, &w.splits, &w.dw_splits);
  w.wide = w.splits > 1 || w.columns < s.V;
  w.x = 256;  // after the largest |dloss|
  w.dz = w.x + aligned_bytes(s, s.T);
  w.sums = w.dz + padded(static_cast<size_t>(s.T) * w.columns * 2);
  w.dw_sums = w.sums + (w.wide ? padded(static_cast<size_t>(w.splits) * s.T * s.d * 4) : 0);
  w.bytes = w.dw_sums + (w.dw_splits > 1 ? padded(static_cast<size_t>(w.dw_splits) * first * s.d * 4) : 0);
  return w;
}

template <typename T>
cudaError_t fold(const float* sums, int splits, int64_t rows, const LossShape& s, const float* top, float more, void* out,
                 int64_t stride, cudaStream_t stream) {
  const int64_t n = rows * s.d;
  return launch_after(fold_kernel<T>, static_cast<int>((n / 8 + 255) / 256), 256, 0, stream, sums, splits, n, s.d, top,
                      s.scale, more, static_cast<T*>(out), stride);
}

}  // namespace

// The forward takes as many rows at a time as 256 MB hold the parts of.
static int stats_rows(const LossShape& s) {
  const int64_t most = kPieceBytes / (up_to(s.V, kHalf) * static_cast<int64_t>(sizeof(float2))) / kTile * kTile;
  const int64_t rows = most < kTile ? kTile : most;
  return rows < s.T ? static_cast<int>(rows) : s.T;
}

size_t loss_workspace_bytes(const LossShape& s) {
  const size_t rows = stats_rows(s);
  return aligned_bytes(s, rows) + padded(rows * 4) + up_to(s.V, kHalf) * rows * sizeof(float2);
}

maxsim_status launch_loss(const LossShape& s, const maxsim_rows& x, const maxsim_rows& w, const int64_t* targets,
                          float* loss, float* lse, void* workspace, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  alignas(64) Maps maps = {};
  if (!map_in(&maps.b, s, w.data, w.row_stride, s.d, s.V, kHalf)) return MAXSIM_ERR_CUDA;
  const int step = stats_rows(s);
  Params p = {};
  p.s = s;
  p.columns = static_cast<int>(s.V);
  p.tiles_n = up_to(s.V, kTile);
  p.hit = reinterpret_cast<float*>(static_cast<char*>(workspace) + aligned_bytes(s, step));
  p.parts = reinterpret_cast<float2*>(reinterpret_cast<char*>(p.hit) + padded(static_cast<size_t>(step) * 4));
  p.z2 = s.scale * kLog2e;
  p.status = dev->status;
  for (int64_t row = 0; row < s.T; row += step) {
    p.s.T = s.T - row < step ? static_cast<int>(s.T - row) : step;
    p.tiles_m = up_to(p.s.T, kTile);
    p.targets = targets + row;
    maxsim_rows from = {static_cast<char*>(x.data) + row * x.row_stride * 2, x.row_stride};
    bool copied;
    if (!aligned_rows(s, &from, p.s.T, workspace, stream, &copied) ||
        !map_in(&maps.a, s, from.data, from.row_stride, s.d, p.s.T, kHalf))
      return MAXSIM_ERR_CUDA;
    if (launch<kStats>(maps, p, *dev, static_cast<int64_t>(p.tiles_m) * p.tiles_n, copied || row > 0, stream) != cudaSuccess ||
        launch_after(join_kernel, up_to(p.s.T, 32), 1024, 0, stream, p.parts, up_to(s.V, kHalf), p.s.T, s.V, p.targets,
                     p.hit, p.z2, loss + row, lse + row, dev->status) != cudaSuccess)
      return MAXSIM_ERR_CUDA;
  }
  return MAXSIM_OK;
}

size_t loss_bwd_workspace_bytes(const LossShape& s) {
  const DeviceInfo* dev = device_info();
  return plan(s, dev ? dev->sm_count / 2 : 76).bytes;
}

maxsim_status launch_loss_bwd(const LossShape& s, const float* dloss, const maxsim_rows& x, const maxsim_rows& w,
                              const int64_t* targets, const float* lse, const maxsim_rows* dx, const maxsim_rows* dw,
                              void* workspace, cudaStream_t stream) {
  const DeviceInfo* dev = device_info();
  if (!dev) return MAXSIM_ERR_CUDA;
  const Space at = plan(s, dev->sm_count / 2);
  char* base = static_cast<char*>(workspace);
  float* top = reinterpret_cast<float*>(base);
  float* sums = reinterpret_cast<float*>(base + at.sums);
  const float more = s.is_bf16 ? 1.f : 16384.f;
  const bool scan = s.T <= kScanRows;
  if (!scan) {
    top_kernel<<<1, 1024, 0, stream>>>(dloss, targets, s.T, s.V, top, dev->status);
    if (cudaGetLastError() != cudaSuccess) return MAXSIM_ERR_CUDA;
  }
  maxsim_rows from = x;
  bool copied;
  if (!aligned_rows(s, &from, s.T, base + at.x, stream, &copied)) return MAXSIM_ERR_CUDA;
  for (int64_t first = 0; first < s.V; first += at.columns) {
    const int columns = s.V - first < at.columns ? static_cast<int>(s.V - first) : at.columns;
    alignas(64) Maps maps = {};
    if (!map_in(&maps.a, s, from.data, from.row_stride, s.d, s.T, kHalf) ||
        !map_in(&maps.b, s, w.data, w.row_stride, s.d, s.V, kHalf) ||
        !map_out(&maps.out0, s.is_bf16 ? 1 : 0, 2, base + at.dz, at.columns, columns, s.T, 1))
      return MAXSIM_ERR_CUDA;
    Params p = {};
    p.s = s;
    p.first = static_cast<int>(first);
    p.columns = columns;
    p.tiles_m = up_to(s.T, kTile);
    p.tiles_n = up_to(columns, kTile);
    p.targets = targets;
    p.lse = lse;
    p.dloss = dloss;
    p.top = top;
    p.scan = scan && first == 0;
    p.more = more;
    p.z2 = s.scale * kLog2e;
    p.status = dev->status;
    if (launch<kGrad>(maps, p, *dev, static_cast<int64_t>(p.tiles_m) * p.tiles_n, copied || first > 0 || !scan, stream) != cudaSuccess)
      return MAXSIM_ERR_CUDA;
    if (!map_in(&maps.a, s, base + at.dz, at.columns, columns, s.T, kHalf) ||
        !map_in(&maps.b, s, w.data, w.row_stride, s.d, s.V, kBox) ||
        !map_in(&maps.a2, s, base + at.dz, at.columns, columns, s.T, kBox) ||
        !map_in(&maps.b2, s, from.data, from.row_stride, s.d, s.T, kBox))
      return MAXSIM_ERR_CUDA;
    p.splits = at.splits;
    p.dw_splits = at.dw_splits;
    p.dw_wide = at.dw_splits > 1;
    if (dx) {
      p.dx_m = up_to(s.T, kTile);
      p.dx_n = up_to(s.d, kTile);
      p.dx_wide = at.wide;
      p.dx_adds = first > 0;
      if (!(at.wide ? map_out(&maps.out0, 3, 4, sums, s.d, s.d, s.T, at.splits)
                    : map_out(&maps.out0, s.is_bf16 ? 1 : 0, 2, dx->data, dx->row_stride, s.d, s.T, 1)))
        return MAXSIM_ERR_CUDA;
    }
    if (dw) {
      p.dw_m = up_to(columns, kTile);
      p.dw_n = up_to(s.d, kTile);
      if (!(p.dw_wide ? map_out(&maps.out1, 3, 4, base + at.dw_sums, s.d, s.d, columns, at.dw_splits)
                      : map_out(&maps.out1, s.is_bf16 ? 1 : 0, 2, dw->data, dw->row_stride, s.d, s.V, 1)))
        return MAXSIM_ERR_CUDA;
    }
    const int dx_cost = up_to(columns, kStep) / at.splits + 8, dw_cost = up_to(s.T, kStep) / at.dw_splits + 8;
    p.dw_first = dw_cost > dx_cost;
    const int longer = p.dw_first ? dw_cost : dx_cost, other = p.dw_first ? dx_cost : dw_cost;
    p.rounds = (longer + other / 2) / other;
    const int64_t tiles = static_cast<int64_t>(p.dx_m) * p.dx_n * p.splits +
                          static_cast<int64_t>(p.dw_m) * p.dw_n * p.dw_splits;
    if (tiles && launch<kSums>(maps, p, *dev, tiles, true, stream) != cudaSuccess) return MAXSIM_ERR_CUDA;
    if (dw && p.dw_wide) {
      const auto go = s.is_bf16 ? fold<__nv_bfloat16> : fold<__half>;
      if (go(reinterpret_cast<float*>(base + at.dw_sums), at.dw_splits, columns, s, top, more,
             static_cast<char*>(dw->data) + first * dw->row_stride * 2, dw->row_stride, stream) != cudaSuccess)
        return MAXSIM_ERR_CUDA;
    }
  }
  if (dx && at.wide) {
    const auto go = s.is_bf16 ? fold<__nv_bfloat16> : fold<__half>;
    if (go(sums, at.splits, s.T, s, top, more, dx->data, dx->row_stride, stream) != cudaSuccess) return MAXSIM_ERR_CUDA;
  }
  return MAXSIM_OK;
}

}  // namespace msim

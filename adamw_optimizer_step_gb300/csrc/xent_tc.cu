// Softmax cross entropy of a large-vocabulary classifier with its gradients
// (gbo_xent_forward, gbo_xent_backward, gbo_xent_grad), without n x v logits
// in fp32.
//
//   l = s H W^T;  lse_i = log sum_j exp l_ij;  loss_i = lse_i - l_iy + z lse_i^2
//   P_ij = w_i s ((1 + 2 z lse_i) exp(l_ij - lse_i) - [j = y_i])
//   dH = g P W,  dW = g P^T H
//
// Steps, all on one stream:
//   rows    the rows that count (label >= 0, weight != 0) get consecutive
//           places in their order, and H's rows are copied there: a batch
//           whose prompts are left out costs what its answers cost, and what
//           stands in a row that is left out (NaN, say) reaches nothing; the
//           label's logit is summed here, in fp32 in a warp
//   logits  tcgen05 GEMM over 256 x 256 tiles, whose epilogue leaves each
//           row's maximum and sum of exponentials over the tile (forward), or
//           P in bf16 (backward).  It puts the label's logit of the first
//           step in the place of its own: the tensor core cuts off the
//           partial sums that it adds up (K / 16 of them), which moved a
//           logit of 5 by 3e-5 at K = 2048, and a loss is lse minus exactly
//           that logit (relative error of the losses at 128256 x 2048: 1.7e-6
//           with the tile's logit, see the tests' bound)
//   lse     joins the tiles' maxima and sums per row in a fixed order
//   products dH += P W and dW = P^T H of one piece of the vocabulary in one
//           launch, from the piece's P
// The backward pass forms the logits again, piece by piece of the
// vocabulary, so its scratch is one piece of P.  Where the workspace has room
// for the whole vocabulary's P, gbo_xent_grad keeps the logits there between
// the passes instead, in 16 bits each (kKeepStep), which replaces one of the
// four products by a pass over that room (see kNarrow):
//   convert P in place of the kept logits
// P is rounded to bf16 once, from the fp32 lse (the tensor cores take 16-bit
// operands: the same rounding as a bf16 gradient of the logits), and sums
// over tokens and vocabulary are fp32.
//
// Bound: tensor cores (2 n v d operations a product) from a few hundred rows
// on, W's HBM traffic below.  Measured, of cuBLAS's 1944 TFLOP/s burst rate:
// losses of 4096 rows, 128256 x 2048: 1.04 ms alone, 1.22 ms in a loop under
// the power limit (2.07 and 1.76 PFLOP/s); losses and gradients of 8192 rows,
// 128000 x 2048: 7.75 and 8.2 ms (6 n v d operations: 1.65 and 1.56 PFLOP/s;
// forward 2.29 ms, convert 0.59 at 7.2 TB/s, products 4.70); 9.95 ms when the
// backward pass formed the logits again.  Converting the logits of one part
// of the rows beside the products of the next, in warps of their own, hid the
// conversion but slowed the products: 7.7 and 8.2 ms, not kept.  Prefetching
// operands to L2 slowed the products by a tenth.
//
// The GEMM kernel is warp-specialised and persistent like the Newton-Schulz
// one: CTA pairs (cta_group::2), 256 x 256 tiles, TMA ring of three 64 KB
// stages, two fp32 accumulators in TMEM, eight epilogue warps per CTA; every
// wait is bounded.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "device_common.cuh"
#include "internal.h"
#include "per_device.h"
#include "tc_common.cuh"

namespace gbo {

namespace {

constexpr int kTile = 256;                     // rows and columns of a pair's tile
constexpr int kBlockK = 64;                    // 64 bf16 = one 128-byte swizzle row
constexpr int kStageK = 2 * kBlockK;           // K of a stage
constexpr int kOpBytes = BM * kBlockK * 2;     // 16 KB: 128 rows of A, or of B, per CTA and K block
constexpr int kSubBytes = 2 * kOpBytes;
constexpr int kStageBytes = 2 * kSubBytes;
constexpr int kStages = 3;
// Epilogue warps: two per TMEM lane quarter, 128 columns of the tile each.
// With one, statistics, 16-bit logits and their store took 10,500 clocks a
// tile, more than the products of a tile below d = 1300 (8 d clocks).
constexpr int kEpiWarps = 8;
constexpr int kSpan = kTile / (kEpiWarps / 4);  // columns of a warp
constexpr int kBlockBytes = 2048;              // 32 x 32 16-bit values
constexpr int kWarpStage = 2 * kBlockBytes;    // two store slots a warp, or one of fp32
constexpr int kSmemUsed = kStages * kStageBytes + kEpiWarps * kWarpStage;
constexpr int kXentSmem = 1024 + kSmemUsed + 256;
constexpr int kXentThreads = 64 + 32 * kEpiWarps;
static_assert(kXentSmem <= 232448, "shared memory per CTA");
// Row tiles that sweep the vocabulary together: 8192 rows of H, which stay
// in L2 (33 MB at d = 2048) while W streams past once per sweep.
constexpr int kSweepTiles = 32;

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Logits kept between the passes: (l - label's logit) in bits, in steps of
// 2^-9, as 16-bit integers.  A step moves P by at most 2^-10 ln 2 = 2^-10.5 of
// it (2^-11.4 root mean square), against 2^-8 (2^-9.3) of P's rounding to
// bf16, whose error hides it: dH and dW of 8192 x 128000 x 2048 are off from 64
// bits by 9.379e-4 and 6.486e-4 (relative, in fp32) with kept logits and by
// 9.380e-4 and 6.485e-4 with logits formed again; written in bf16 by 1.906e-3
// and 1.731e-3 either way, where that rounding alone takes 1.66e-3 and
// 1.61e-3.  The range is 64 bits (44 nats) either way.  Entries below it are
// 2^-64 of the label's probability: taken as 0.  A row tile with an entry
// above it, or one that is not finite, is marked and its P formed again from H
// and W.
constexpr float kKeepStep = 512.f;  // steps a bit
constexpr float kKeepMost = 63.9f;  // bits

enum XentMode { kModeStats = 0, kModeP = 1, kModeProducts = 2 };

// Per-call scalars in the workspace.
struct XentHead {
  int32_t rows;      // rows that count
  float weight_sum;  // sum of their weights
  float g;           // factor of the gradients
  int32_t redo;      // some tile's kept logits are out of their range (see kKeepStep)
};

struct XentParams {
  CUtensorMap mapA, mapB;    // logits: H, W (K-major); products: P K-major, W MN-major (dH)
  CUtensorMap mapA2, mapB2;  // products: P MN-major, H MN-major (dW)
  CUtensorMap mapO;          // stores: kept logits, P or dW, 32 x 32 boxes
  const XentHead *head;
  const int32_t *idx, *lab;  // place -> row, label; up to a whole tile
  const float *wt, *lse2;    // weight (0: padding), lse in bits
  const float *ll2;          // the label's logit in bits
  float2 *part;              // forward: (maximum, sum) per vocabulary tile and place
  float *dh_acc;             // fp32 sums of dH, `splits` times places x d
  XentHead *head_out;        // forward with kept logits: where `redo` is set
  int32_t *redo;             // per row tile: its kept logits are out of range
  void *dh, *dw;
  int32_t *status;
  int64_t part_ld;           // places per vocabulary tile in part
  int64_t dh_stride, dw_stride, v0;
  int32_t v_piece, d;        // columns of this piece
  int32_t dh_f32, dw_f32, dh_vec, dw_vec, dw_add, first_piece, last_piece;
  int32_t dw_tma;            // products: dW leaves through mapO
  int32_t splits, split_kit; // dH: cuts of its K axis (the piece's columns), stages in each
  int32_t keep;              // forward: store the logits
  int32_t only_redo;         // P: only the tiles of `redo`
  int64_t acc_ld;            // elements of one split's dh_acc
  float scale2;              // logit scale in bits: s log2 e
  float scale, z;
};

__device__ __forceinline__ uint32_t idesc_of(bool a_mn, bool b_mn, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
         ((uint32_t)(n >> 3) << 17) | ((uint32_t)(kTile >> 4) << 24);
}

__device__ __forceinline__ void mma_pair(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc, uint32_t idesc,
                                         uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct XentItem {
  int tm, tn, kit, split;
  int steps;  // K in steps of 16: the last stage is multiplied as far as K goes
  int half;   // columns of B per CTA: 128, less in the last tile of d columns
  bool dw;
};

// What a launch has to do, from the number of rows that count.
struct XentPlan {
  int rows, m_tiles, n_tiles;       // logits: row tiles, vocabulary tiles
  int dh_items, dw_items, d_tiles;  // products
  int dh_kit, dw_kit;
  int ncl, cid;
  int extra, wide, mine;            // products: see Walk
};

// What an item of `kit` stages costs, in stages: its epilogue takes 5 of them
// where its products take less, and another goes to its start and end.
__host__ __device__ __forceinline__ int item_cost(int kit) { return (kit < 5 ? 5 : kit) + 1; }

template <int kMode>
__device__ __forceinline__ XentPlan make_plan(const XentParams &P, int cid, int ncl) {
  XentPlan q;
  q.rows = kMode == kModeP && P.only_redo && !P.head->redo ? 0 : P.head->rows;
  q.m_tiles = (q.rows + kTile - 1) / kTile;
  q.n_tiles = (P.v_piece + kTile - 1) / kTile;
  q.d_tiles = (P.d + kTile - 1) / kTile;
  q.dh_items = P.dh ? q.m_tiles * q.d_tiles * P.splits : 0;
  q.dw_items = P.dw ? q.n_tiles * q.d_tiles : 0;
  q.dh_kit = P.splits > 1 ? P.split_kit : (P.v_piece + kStageK - 1) / kStageK;
  q.dw_kit = (q.rows + kStageK - 1) / kStageK;
  q.ncl = ncl;
  q.cid = cid;
  q.wide = q.dh_items % ncl;
  q.mine = q.dh_items / ncl + (cid < q.wide ? 1 : 0);
  const int dw_cost = item_cost(q.dw_kit);
  q.extra = q.wide ? (item_cost(q.dh_kit) + dw_cost / 2) / dw_cost : 0;
  return q;
}

// The items of this pair, one after another.
//   logits: round-robin over the pairs; a sweep of kSweepTiles row tiles
//     takes the vocabulary tile by tile.
//   products: dH items (K = the piece's width, or a cut of it) first, round-robin;
//     `wide` pairs get one more than the others, who therefore take `extra`
//     dW items (K = rows) of the same total length first; the rest of dW is
//     dealt to all.  Items are independent, so the split changes no result.
// Tile coordinates advance by the step's quotient and remainder: a division
// per item and role took 1000 clocks, a sixth of a short item.
template <int kMode>
struct Walk {
  const XentPlan &q;
  const XentParams &P;
  int64_t t = 0;               // the next item of the phase
  int phase = 0, count = 0;
  int row = 0, col = 0;        // its coordinates; logits: row within the sweep
  int sweep = 0, rows = 1;     // logits: the sweep and its row tiles
  int step_row = 0, step_col = 0, step = 0;

  __device__ __forceinline__ Walk(const XentPlan &q_, const XentParams &P_) : q(q_), P(P_) {}

  __device__ __forceinline__ bool next(XentItem &it) {
    if constexpr (kMode != kModeProducts) {
      bool seek = phase == 0;
      if (seek) {
        phase = 1;
        t = q.cid;
      } else {
        t += q.ncl;
        row += step_row;
        col += step_col;
        if (row >= rows) row -= rows, ++col;
        seek = col >= q.n_tiles;
      }
      if (t >= (int64_t)q.m_tiles * q.n_tiles) return false;
      if (seek) {
        const int64_t size = (int64_t)kSweepTiles * q.n_tiles;
        sweep = (int)(t / size);
        const int r = (int)(t - sweep * size);
        rows = min(kSweepTiles, q.m_tiles - sweep * kSweepTiles);
        col = r / rows, row = r % rows;
        step_col = q.ncl / rows, step_row = q.ncl % rows;
      }
      it.tn = col;
      it.tm = sweep * kSweepTiles + row;
      it.kit = (P.d + kStageK - 1) / kStageK;
      it.steps = (P.d + 15) / 16;
      it.half = BM;
      it.dw = false;
      return true;
    } else {
      if (phase == 0) phase = 1;
      if (phase == 1) {
        if (count < q.mine) {
          const int i = q.cid + count * q.ncl, u = i / P.splits;
          ++count;
          it.split = i - u * P.splits;
          it.tm = u / q.d_tiles;
          it.tn = u - it.tm * q.d_tiles;
          const int k0 = it.split * q.dh_kit * kStageK;
          const int len = max(0, min(q.dh_kit * kStageK, P.v_piece - k0));
          it.kit = (len + kStageK - 1) / kStageK;
          it.steps = (len + 15) / 16;
          it.half = half_of(it.tn);
          it.dw = false;
          return true;
        }
        count = 0;
        if (q.cid >= q.wide && q.extra > 0) enter(2, q.cid - q.wide, q.ncl - q.wide);
        else enter(3, (int64_t)q.extra * (q.ncl - q.wide) + q.cid, q.ncl);
      }
      if (phase == 2 && count == q.extra) enter(3, (int64_t)q.extra * (q.ncl - q.wide) + q.cid, q.ncl);
      if (t >= q.dw_items) return false;
      it.tm = row;
      it.tn = col;
      it.kit = q.dw_kit;
      it.steps = (q.rows + 15) / 16;
      it.half = half_of(col);
      it.dw = true;
      ++count;
      t += step;
      row += step_row;
      col += step_col;
      if (col >= q.d_tiles) col -= q.d_tiles, ++row;
      return true;
    }
  }

 private:
  // the last tile of d columns multiplies no more than it holds (a multiple
  // of 32 columns, half of them per CTA)
  __device__ __forceinline__ int half_of(int tn) const { return min(BM, (P.d - tn * kTile + 31) / 32 * 16); }

  __device__ __forceinline__ void enter(int to, int64_t at, int by) {
    phase = to;
    t = at;
    step = by;
    row = (int)(at / q.d_tiles), col = (int)(at - (int64_t)row * q.d_tiles);
    step_row = by / q.d_tiles, step_col = by - step_row * q.d_tiles;
  }
};

struct Ring {
  int stage;
  uint32_t phase;
  __device__ __forceinline__ void next() {
    if (++stage == kStages) stage = 0, phase ^= 1;
  }
};

// Load one item's stages.  m0, n0: this CTA's first row of A and of B (their
// columns when MN-major); ka0, kb0: where K begins in A and B.  Only the leader arms
// the barrier, for both CTAs' bytes.
template <bool kAmn, bool kBmn>
__device__ __forceinline__ bool produce(const CUtensorMap *ma, const CUtensorMap *mb, int m0, int n0, int ka0, int kb0,
                                        int kit, int half, uint32_t smem, uint32_t full0, uint32_t empty0, uint32_t full_lead0,
                                        bool leader, Ring &ring, uint32_t *armed_parity, uint32_t &armed,
                                        volatile int32_t *abort_flag) {
  // MN-major B: boxes of 64 columns
  const int b_boxes = kBmn ? (half + 63) / 64 : 2;
  const uint32_t bytes = 2u * (kStageBytes - 2u * 8192u * (uint32_t)(2 - b_boxes));
  for (int kb = 0; kb < kit; ++kb) {
    if (!mbar_wait(empty0 + 8 * ring.stage, ring.phase ^ 1)) return false;
    if (*abort_flag) return true;
    if (leader) {
      mbar_expect_tx(full0 + 8 * ring.stage, bytes);
      armed |= 1u << ring.stage;
      armed_parity[ring.stage] = ring.phase;
    }
    const uint32_t fb = full_lead0 + 8 * ring.stage;
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const uint32_t sa = smem + ring.stage * kStageBytes + sub * kSubBytes, sb = sa + kOpBytes;
      const int k = kb * kStageK + sub * kBlockK;
      if constexpr (!kAmn) {
        tma_load_3d_pair(sa, ma, fb, ka0 + k, m0, 0);
      } else {
#pragma unroll
        for (int h = 0; h < 2; ++h) tma_load_3d_pair(sa + h * 8192, ma, fb, m0 + h * 64, ka0 + k, 0);
      }
      if constexpr (!kBmn) {
        tma_load_3d_pair(sb, mb, fb, kb0 + k, n0, 0);
      } else {
        for (int h = 0; h < b_boxes; ++h) tma_load_3d_pair(sb + h * 8192, mb, fb, n0 + h * 64, kb0 + k, 0);
      }
    }
    ring.next();
  }
  return true;
}

template <bool kAmn, bool kBmn>
__device__ __forceinline__ bool multiply(uint32_t smem, uint32_t full0, uint32_t empty0, uint32_t d_tmem,
                                         const XentItem &it, Ring &ring, bool &issued) {
  const uint32_t idesc = idesc_of(kAmn, kBmn, 2 * it.half);
  const uint64_t a0 = smem_desc(smem, kAmn ? 8192 : 16, 1024);
  const uint64_t b0 = smem_desc(smem + kOpBytes, kBmn ? 8192 : 16, 1024);
  constexpr uint32_t astep = (kAmn ? 2048 : 32) >> 4, bstep = (kBmn ? 2048 : 32) >> 4;
  for (int kb = 0; kb < it.kit; ++kb) {
    if (!mbar_wait(full0 + 8 * ring.stage, ring.phase)) return false;
    tc_fence_after();
    const int left = it.steps - kb * (kStageK / 16);
#pragma unroll
    for (int sub = 0; sub < 2; ++sub) {
      const uint32_t off = (uint32_t)(ring.stage * kStageBytes + sub * kSubBytes) >> 4;
#pragma unroll
      for (int k = 0; k < kBlockK / 16; ++k)
        if (sub * (kBlockK / 16) + k < left) mma_pair(d_tmem, a0 + off + k * astep, b0 + off + k * bstep, idesc, (kb | sub | k) != 0);
    }
    issued = true;
    mma_commit_pair_mc(empty0 + 8 * ring.stage, 0x3);
    ring.next();
  }
  return true;
}

// Running maximum and sum of one row over 32 more values (in bits).
__device__ __forceinline__ void softmax_add(const float (&t)[32], float &m, float &s) {
  float mx = t[0];
#pragma unroll
  for (int k = 1; k < 32; ++k) mx = fmaxf(mx, t[k]);
  const float mn = fmaxf(m, mx);
  const float at = mn == -INFINITY ? 0.f : mn;  // nothing but -inf so far: every term is 0
  float a = 0.f;
#pragma unroll
  for (int k = 0; k < 32; ++k) a += exp2_fast(t[k] - at);
  s = fmaf(s, exp2_fast(m - at), a);
  m = mn;
}

// 32 logits (in bits) as 16-bit steps from the row's label's logit.  A float
// of 1.5 2^23 plus an integer holds that integer in its low bits.
__device__ __forceinline__ void pack_steps(const float (&v)[32], float ll2, uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    uint32_t h[2];
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const float steps = fminf(fmaxf((v[2 * k + e] - ll2) * kKeepStep, -32768.f), 32767.f);
      h[e] = __float_as_uint(steps + 12582912.f);
    }
    w[k] = __byte_perm(h[0], h[1], 0x5410);
  }
}

__device__ __forceinline__ void pack_row(const float (&v)[32], uint32_t (&w)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k) w[k] = pack_bf16(v[2 * k], v[2 * k + 1]);
}

// Store a warp's 32 x 32 block of 16-bit values through the next of its two
// slots (64-byte rows in the 64-byte swizzle).
__device__ __forceinline__ void store_block(const CUtensorMap *map, uint32_t stage, int &slot, const uint32_t (&w)[16],
                                            int x0, int y0, int lane) {
  const uint32_t dst = stage + (uint32_t)(slot * kBlockBytes);
  slot ^= 1;
  if (lane == 0) bulk_wait_read<1>();  // the store that last used this slot has read it
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 4; ++q)
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(dst + sw64(lane, q)), "r"(w[4 * q]),
                 "r"(w[4 * q + 1]), "r"(w[4 * q + 2]), "r"(w[4 * q + 3])
                 : "memory");
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    tma_store_3d(map, dst, x0, y0, 0);
    bulk_commit();
  }
}

// Store, or add, a warp's 32 x 32 fp32 block, which takes both slots (128-byte
// rows in the 128-byte swizzle: 16-byte chunk q of row r at chunk q ^ (r & 7)).
__device__ __forceinline__ void store_block_f32(const CUtensorMap *map, uint32_t dst, const float (&v)[32], bool add,
                                                int x0, int y0, int lane) {
  if (lane == 0) bulk_wait_read<0>();
  __syncwarp();
#pragma unroll
  for (int q = 0; q < 8; ++q)
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(dst + lane * 128 + ((q ^ (lane & 7)) << 4)),
                 "f"(v[4 * q]), "f"(v[4 * q + 1]), "f"(v[4 * q + 2]), "f"(v[4 * q + 3])
                 : "memory");
  fence_async_smem();
  __syncwarp();
  if (lane == 0) {
    if (add)
      asm volatile("cp.reduce.async.bulk.tensor.3d.global.shared::cta.add.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                       reinterpret_cast<uint64_t>(map)),
                   "r"(dst), "r"(x0), "r"(y0), "r"(0)
                   : "memory");
    else
      tma_store_3d(map, dst, x0, y0, 0);
    bulk_commit();
  }
}

template <int kMode>
__global__ void __launch_bounds__(kXentThreads, 1) xent_kernel(const __grid_constant__ XentParams P) {
  pdl_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kSmemUsed);
  // bars: full[kStages], empty[kStages], accf[2], acce[2], drain, (TMEM address, abort flag)
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kStages + 5);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kStages);
  const uint32_t accf0 = smem_u32(bars + 2 * kStages), acce0 = smem_u32(bars + 2 * kStages + 2);
  const uint32_t drain = smem_u32(bars + 2 * kStages + 4);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = cluster_rank();
  const bool leader = crank == 0;
  // Barriers as in the Newton-Schulz pair kernel: full on the leader (both
  // CTAs' bytes), empty and accf in each CTA (multicast commits of the
  // leader's MMAs), acce on the leader (one arrival per epilogue warp of both).
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(accf0 + 8 * a, 1);
      mbar_init(acce0 + 8 * a, 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(kTmemCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  const uint32_t tmem_base = *tmem_slot;
  pdl_wait();
  const XentPlan q = make_plan<kMode>(P, blockIdx.x >> 1, gridDim.x >> 1);
  const uint32_t full_lead0 = map_to_rank(full0, 0), acce_lead0 = map_to_rank(acce0, 0);
  const uint32_t ring0 = smem_u32(smem);
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_status(P.status, GBO_STATUS_TIMEOUT);
  };

  if (warp == 0) {
    if (lane == 0) {
      Ring ring = {0, 0};
      uint32_t armed = 0, armed_parity[kStages] = {};
      XentItem it;
      Walk<kMode> walk(q, P);
      while (!*abort_flag && walk.next(it)) {
        if (kMode == kModeP && P.only_redo && !P.redo[it.tm]) continue;
        const int m0 = it.tm * kTile + (int)crank * BM, n0 = it.tn * kTile + (int)crank * it.half;
        bool ok;
        if constexpr (kMode != kModeProducts)
          ok = produce<false, false>(&P.mapA, &P.mapB, m0, (int)P.v0 + n0, 0, 0, it.kit, it.half, ring0, full0, empty0,
                                     full_lead0, leader, ring, armed_parity, armed, abort_flag);
        else if (!it.dw)
          ok = produce<false, true>(&P.mapA, &P.mapB, m0, n0, it.split * P.split_kit * kStageK,
                                    (int)P.v0 + it.split * P.split_kit * kStageK, it.kit, it.half, ring0, full0, empty0,
                                    full_lead0, leader, ring, armed_parity, armed, abort_flag);
        else
          ok = produce<true, true>(&P.mapA2, &P.mapB2, m0, n0, 0, 0, it.kit, it.half, ring0, full0, empty0, full_lead0,
                                   leader, ring, armed_parity, armed, abort_flag);
        if (!ok) { give_up(); break; }
      }
      if (*abort_flag && leader) {  // copies armed here land before shared memory goes away
        for (int s = 0; s < kStages; ++s)
          if (armed >> s & 1u) (void)mbar_wait(full0 + 8 * s, armed_parity[s]);
      }
    }
  } else if (warp == 1) {
    if (lane == 0 && leader) {
      Ring ring = {0, 0};
      int acc = 0;
      uint32_t acc_phase = 0;
      bool issued = false;
      XentItem it;
      Walk<kMode> walk(q, P);
      while (!*abort_flag && walk.next(it)) {
        if (kMode == kModeP && P.only_redo && !P.redo[it.tm]) continue;
        if (!mbar_wait_cluster(acce0 + 8 * acc, acc_phase ^ 1)) { give_up(); break; }
        tc_fence_after();
        const uint32_t d_tmem = tmem_base + (uint32_t)(acc * kTile);
        bool ok;
        if constexpr (kMode != kModeProducts)
          ok = multiply<false, false>(ring0, full0, empty0, d_tmem, it, ring, issued);
        else if (!it.dw)
          ok = multiply<false, true>(ring0, full0, empty0, d_tmem, it, ring, issued);
        else
          ok = multiply<true, true>(ring0, full0, empty0, d_tmem, it, ring, issued);
        if (!ok) { give_up(); break; }
        mma_commit_pair_mc(accf0 + 8 * acc, 0x3);
        if (++acc == 2) acc = 0, acc_phase ^= 1;
      }
      if (*abort_flag && issued) {
        mma_commit_pair(drain);
        (void)mbar_wait(drain, 0);
      }
    }
  } else {
    const int quarter = warp & 3, part = (warp - 2) >> 2;
    const uint32_t stage = smem_u32(smem + kStages * kStageBytes + (warp - 2) * kWarpStage);
    int slot = 0, acc = 0;
    uint32_t acc_phase = 0;
    XentItem it;
    Walk<kMode> walk(q, P);
    while (!*abort_flag && walk.next(it)) {
      if (kMode == kModeP && P.only_redo && !P.redo[it.tm]) continue;
      const int i0 = it.tm * kTile + (int)crank * BM + quarter * 32, i = i0 + lane;
      const int c0 = it.tn * kTile + part * kSpan;
      // per-row values of this tile, fetched while its products run
      int lab = -1;
      float wt = 0.f, lse2 = 0.f, ll2 = 0.f;
      if constexpr (kMode != kModeProducts) {
        if (i < q.rows) {
          lab = P.lab[i] - (int)P.v0, ll2 = P.ll2[i];
          if constexpr (kMode == kModeP) wt = P.wt[i], lse2 = P.lse2[i];
        }
      }
      if (!mbar_wait(accf0 + 8 * acc, acc_phase)) { give_up(); break; }
      tc_fence_after();
      const uint32_t trow = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kTile + part * kSpan);
      if constexpr (kMode == kModeStats) {
        if (i0 < q.rows || P.keep) {  // (rows behind the last one are stored too: their P is set to 0 later)
          float m = -INFINITY, s = 0.f;
#pragma unroll 1
          for (int ch = 0; ch < kSpan / 32; ++ch) {
            const int col0 = c0 + 32 * ch;
            if (col0 >= P.v_piece) break;
            float v[32];
            tmem_ld32(trow + ch * 32, v);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] *= P.scale2;
            if (lab >= col0 && lab < col0 + 32) {
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] = lab == col0 + j ? ll2 : v[j];
            }
            if (col0 + 32 > P.v_piece) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (col0 + j >= P.v_piece) v[j] = -INFINITY;
            }
            if (P.keep) {
              uint32_t w[16];
              pack_steps(v, ll2, w);
              store_block(&P.mapO, stage, slot, w, col0, i0, lane);
            }
            softmax_add(v, m, s);
          }
          if (P.keep && i < q.rows && !(m - ll2 <= kKeepMost && s < INFINITY)) {
            P.redo[it.tm] = 1;  // every writer writes the same
            P.head_out->redo = 1;
          }
          if (i < q.rows && c0 < P.v_piece) P.part[(int64_t)(it.tn * (kTile / kSpan) + part) * P.part_ld + i] = make_float2(m, s);
        }
      } else if constexpr (kMode == kModeP) {
        const float mult = wt * P.scale, peak = mult * fmaf(2.f * P.z, lse2 * kLn2, 1.f);
#pragma unroll 1
        for (int ch = 0; ch < kSpan / 32; ++ch) {
          const int col0 = c0 + 32 * ch;
          if (col0 >= P.v_piece) break;
          float v[32];
          tmem_ld32(trow + ch * 32, v);
          if (wt != 0.f) {
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = peak * exp2_fast(fmaf(v[j], P.scale2, -lse2));
            if (lab >= col0 && lab < col0 + 32) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (lab == col0 + j) v[j] = fmaf(peak, exp2_fast(ll2 - lse2), -mult);
            }
          } else {  // places behind the last row: their P multiplies zero rows of H, and must be finite
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          }
          uint32_t w[16];
          pack_row(v, w);
          store_block(&P.mapO, stage, slot, w, col0, i0, lane);
        }
      } else if (it.dw && P.dw_tma) {
        // through the staging slots; what is added to dW (fp32) is added by the store
        const float g = P.head->g;
#pragma unroll 1
        for (int ch = 0; ch < kSpan / 32; ++ch) {
          const int col0 = c0 + 32 * ch;
          if (col0 >= P.d || i0 >= P.v_piece) break;
          float v[32];
          tmem_ld32(trow + ch * 32, v);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = it.kit > 0 ? g * v[j] : 0.f;  // no rows: nothing was multiplied
          if (P.dw_f32) {
            store_block_f32(&P.mapO, stage, v, P.dw_add != 0, col0, (int)P.v0 + i0, lane);
          } else {
            uint32_t w[16];
            pack_row(v, w);
            store_block(&P.mapO, stage, slot, w, col0, (int)P.v0 + i0, lane);
          }
        }
      } else if (it.dw) {
        const float g = P.head->g;
        const int64_t row = P.v0 + i;
        const bool ok = i < P.v_piece;
#pragma unroll 1
        for (int ch = 0; ch < kSpan / 32; ++ch) {
          const int col0 = c0 + 32 * ch;
          if (col0 >= P.d || i0 >= P.v_piece) break;
          float v[32];
          tmem_ld32(trow + ch * 32, v);
          if (!ok) continue;
          const uint32_t mask = prefix_mask(P.d - col0);
          const bool vec = P.dw_vec && mask == 0xffffffffu;
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = it.kit > 0 ? g * v[j] : 0.f;  // no rows: nothing was multiplied
          const int64_t at = row * P.dw_stride + col0;
          if (P.dw_f32) {
            float *o = static_cast<float *>(P.dw) + at;
            if (P.dw_add) {
              float w[32];
              load_row32(o, w, vec, mask);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += w[j];
            }
            store_row32(o, v, vec, mask);
          } else {
            __nv_bfloat16 *o = static_cast<__nv_bfloat16 *>(P.dw) + at;
            if (P.dw_add) {
              float w[32];
              load_row32(o, w, vec, mask);
#pragma unroll
              for (int j = 0; j < 32; ++j) v[j] += w[j];
            }
            store_row32(o, v, vec, mask);
          }
        }
      } else {
        const float g = P.head->g;
        const bool ok = i < q.rows;
        const int64_t row = ok ? P.idx[i] : 0;
#pragma unroll 1
        for (int ch = 0; ch < kSpan / 32; ++ch) {
          const int col0 = c0 + 32 * ch;
          if (col0 >= P.d || i0 >= q.rows) break;
          float v[32];
          tmem_ld32(trow + ch * 32, v);
          if (!ok) continue;
          if (it.kit == 0) {  // a narrow last piece may end before the last cut: nothing was multiplied
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] = 0.f;
          }
          const uint32_t mask = prefix_mask(P.d - col0);
          const bool whole = mask == 0xffffffffu;
          // d is a multiple of 8: 32-byte aligned
          float *sum = P.dh_acc + it.split * P.acc_ld + (int64_t)i * P.d + col0;
          if (!P.first_piece) {
            float w[32];
            load_row32(sum, w, whole, mask);
#pragma unroll
            for (int j = 0; j < 32; ++j) v[j] += w[j];
          }
          if (!P.last_piece || P.splits > 1) {
            store_row32(sum, v, whole, mask);
            continue;
          }
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] *= g;
          const int64_t at = row * P.dh_stride + col0;
          const bool vec = P.dh_vec && whole;
          if (P.dh_f32) store_row32(static_cast<float *>(P.dh) + at, v, vec, mask);
          else store_row32(static_cast<__nv_bfloat16 *>(P.dh) + at, v, vec, mask);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(acce_lead0 + 8 * acc);
      if (++acc == 2) acc = 0, acc_phase ^= 1;
    }
    if (lane == 0) bulk_wait_all();
    __syncwarp();
  }

  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(kTmemCols) : "memory");
}

// ---------------------------------------------------------------------------
// few rows

// Statistics of at most 32 rows: W is read once and its HBM traffic is all
// there is, so the operands change places.  The vocabulary is M (tiles of 128
// rows of W), the rows are N = 16 or 32, a stage of the ring is 32 KB of W and
// 4 or 8 KB of H, and four of five are on their way while one is multiplied.
// A thread of the epilogue owns a row of W and keeps a running maximum and sum
// for every row of H; lanes join once, at the end.
// CTAs take whole tiles in turn, so that all SMs read one window of W; what
// the last rounds of them leave is cut equally, in one or two tiles a CTA with
// a box of their own height (a tile in boxes of 16 rows moves at a third of
// the rate, and one run of consecutive rows a CTA from the start costs 2%).
// One token over 128000 x 2048 (524 MB), the whole call: 102 us with the
// 256-wide tiles; here 97 us with runs that end in 16-row boxes, 87 us as it
// is (a plain reduction that reads W once takes 92 us).  Four or six stages,
// 64-row tiles and stages twice as wide measure the same or more: HBM is the
// bound.  Prefetching each next tile's rows to L2 made it 137 us.
constexpr int kScoreMost = 32;
constexpr int kScoreUnit = 16;                                   // rows of W that a run is made of
constexpr int kScoreStages = 5;
constexpr int kScoreWarps = 4;                                   // epilogue
constexpr int kScoreAhead = 4;                                   // rows whose sums run side by side

template <int kRows>
struct ScoreShape {
  static constexpr int kB = kRows * kBlockK * 2;                 // H's rows, one K block
  static constexpr int kStage = 2 * (kOpBytes + kB);
  static constexpr int kSmem = 1024 + kScoreStages * kStage + 256 + kRows * 8;
  static constexpr int kTmem = 2 * kRows;                        // two accumulators of 128 x kRows
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct ScoreParams {
  CUtensorMap mapW, mapRest, mapH;  // boxes of 128, `step` and kRows rows
  const XentHead *head;
  const int32_t *lab;
  const float *ll2;
  float2 *part;     // (maximum, sum) per CTA and epilogue warp, and row
  int32_t *status;
  int64_t part_ld;
  int32_t v, d;
  int32_t whole, step;  // whole tiles of a CTA, rows of its other tiles
  float scale2;
};

// The 32 lanes' rows of 16 consecutive fp32 TMEM columns.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, float (&v)[16]) {
  uint32_t r[16];
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k] = __uint_as_float(r[k]);
}

template <int kRows>
__global__ void __launch_bounds__(192, 1) xent_score_kernel(const __grid_constant__ ScoreParams P) {
  using Shape = ScoreShape<kRows>;
  constexpr int kScoreStage = Shape::kStage, kScoreB = Shape::kB;
  pdl_launch();
  extern __shared__ uint8_t smem_raw[];
  uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~(uintptr_t)1023);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + kScoreStages * kScoreStage);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + 2 * kScoreStages + 5);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  int32_t *lab_s = reinterpret_cast<int32_t *>(bars + 32);
  float *ll2_s = reinterpret_cast<float *>(lab_s + kRows);
  const uint32_t full0 = smem_u32(bars), empty0 = smem_u32(bars + kScoreStages);
  const uint32_t accf0 = smem_u32(bars + 2 * kScoreStages), acce0 = accf0 + 16, drain = accf0 + 32;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's rows of W: `whole` tiles, dealt out, then an equal run of what
  // is left, in tiles of `step` rows
  const int cid = blockIdx.x, ncta = gridDim.x, kit = (P.d + kStageK - 1) / kStageK;
  const int rest = P.whole * ncta * BM;
  const int units = (P.v - rest + kScoreUnit - 1) / kScoreUnit, base = units / ncta, rem = units % ncta;
  const int run0 = rest + kScoreUnit * (cid * base + min(cid, rem)), run = kScoreUnit * (base + (cid < rem ? 1 : 0));
  const int tiles = P.whole + (run + P.step - 1) / P.step;
  auto tile_row = [&](int t) { return t < P.whole ? (t * ncta + cid) * BM : run0 + (t - P.whole) * P.step; };
  if (threadIdx.x == 0) {
    for (int s = 0; s < kScoreStages; ++s) mbar_init(full0 + 8 * s, 1), mbar_init(empty0 + 8 * s, 1);
    for (int a = 0; a < 2; ++a) mbar_init(accf0 + 8 * a, 1), mbar_init(acce0 + 8 * a, kScoreWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == 1) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(Shape::kTmem)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();
  const int rows = P.head->rows;  // at most kRows
  if (threadIdx.x < kRows) {
    lab_s[threadIdx.x] = (int)threadIdx.x < rows ? P.lab[threadIdx.x] : -1;
    ll2_s[threadIdx.x] = (int)threadIdx.x < rows ? P.ll2[threadIdx.x] : 0.f;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem_base = *tmem_slot, ring0 = smem_u32(smem);
  auto give_up = [&]() {
    *abort_flag = 1;
    flag_status(P.status, GBO_STATUS_TIMEOUT);
  };
  int stage = 0;
  uint32_t phase = 0;
  auto next = [&]() {
    if (++stage == kScoreStages) stage = 0, phase ^= 1;
  };
  if (rows == 0) {
    // nothing counts
  } else if (warp == 0) {
    if (lane == 0) {
      uint32_t armed = 0, armed_parity = 0;
      bool ok = true;
      for (int t = 0; t < tiles && ok; ++t) {
        const bool full = t < P.whole;
        const int r0 = tile_row(t);
        const uint32_t bytes = 2u * (uint32_t)((full ? BM : P.step) * kBlockK * 2 + kScoreB);
        for (int kb = 0; kb < kit; ++kb) {
          if (!mbar_wait(empty0 + 8 * stage, phase ^ 1)) { give_up(); ok = false; break; }
          if (*abort_flag) { ok = false; break; }
          const uint32_t fb = full0 + 8 * stage;
          mbar_expect_tx(fb, bytes);
          armed |= 1u << stage;
          armed_parity = (armed_parity & ~(1u << stage)) | (phase << stage);
#pragma unroll
          for (int sub = 0; sub < 2; ++sub) {
            const uint32_t sa = ring0 + stage * kScoreStage + sub * kOpBytes;
            const uint32_t sb = ring0 + stage * kScoreStage + 2 * kOpBytes + sub * kScoreB;
            const int k = kb * kStageK + sub * kBlockK;
            tma_load_3d(sa, full ? &P.mapW : &P.mapRest, fb, k, r0, 0);
            tma_load_3d(sb, &P.mapH, fb, k, 0, 0);
          }
          next();
        }
      }
      if (*abort_flag)  // copies armed here land before shared memory goes away
        for (int s = 0; s < kScoreStages; ++s)
          if (armed >> s & 1u) (void)mbar_wait(full0 + 8 * s, armed_parity >> s & 1u);
    }
  } else if (warp == 1) {
    if (lane == 0) {
      const uint32_t idesc = (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)(kRows >> 3) << 17) |
                             ((uint32_t)(BM >> 4) << 24);
      const uint64_t a0 = smem_desc(ring0, 16, 1024), b0 = smem_desc(ring0 + 2 * kOpBytes, 16, 1024);
      bool issued = false, ok = true;
      for (int t = 0; t < tiles && ok && !*abort_flag; ++t) {
        const int acc = t & 1;
        if (!mbar_wait(acce0 + 8 * acc, ((t >> 1) & 1) ^ 1)) { give_up(); break; }
        tc_fence_after();
        for (int kb = 0; kb < kit; ++kb) {
          if (!mbar_wait(full0 + 8 * stage, phase)) { give_up(); ok = false; break; }
          tc_fence_after();
#pragma unroll
          for (int sub = 0; sub < 2; ++sub)
#pragma unroll
            for (int k = 0; k < kBlockK / 16; ++k) {
              const uint64_t ad = a0 + ((uint32_t)(stage * kScoreStage + sub * kOpBytes) >> 4) + 2 * k;
              const uint64_t bd = b0 + ((uint32_t)(stage * kScoreStage + sub * kScoreB) >> 4) + 2 * k;
              asm volatile(
                  "{\n\t.reg .pred p;\n\t"
                  "setp.ne.b32 p, %4, 0;\n\t"
                  "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(tmem_base + acc * kRows),
                  "l"(ad), "l"(bd), "r"(idesc), "r"((uint32_t)((kb | sub | k) != 0))
                  : "memory");
            }
          issued = true;
          mma_commit_one(empty0 + 8 * stage);
          next();
        }
        if (ok) mma_commit_one(accf0 + 8 * acc);
      }
      if (*abort_flag && issued) {
        mma_commit_one(drain);
        (void)mbar_wait(drain, 0);
      }
    }
  } else {
    const int quarter = warp & 3;
    float m[kRows], s[kRows];
#pragma unroll
    for (int j = 0; j < kRows; ++j) m[j] = -INFINITY, s[j] = 0.f;
    bool ok = true;
    for (int t = 0; t < tiles; ++t) {
      const int acc = t & 1, r0 = tile_row(t), r = r0 + quarter * 32 + lane;
      // (a tile of the run may end in rows that are the next CTA's, or in none)
      const int end = min(t < P.whole ? P.v : min(run0 + run, r0 + P.step), P.v);
      if (!mbar_wait(accf0 + 8 * acc, (t >> 1) & 1)) { give_up(); ok = false; break; }
      tc_fence_after();
      float v[kRows];
      const uint32_t at = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(acc * kRows);
      if constexpr (kRows == 16) tmem_ld16(at, v);
      else tmem_ld32(at, v);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(acce0 + 8 * acc);
#pragma unroll
      for (int j0 = 0; j0 < kRows; j0 += kScoreAhead) {
        if (j0 >= rows) break;
#pragma unroll
        for (int j = j0; j < j0 + kScoreAhead; ++j) {  // rows behind the last one: zeros that nobody reads
          const float l = r == lab_s[j] ? ll2_s[j] : v[j] * P.scale2;
          const float x = r < end ? l : -INFINITY;
          const float mn = fmaxf(m[j], x), at = mn == -INFINITY ? 0.f : mn;
          s[j] = fmaf(s[j], exp2_fast(m[j] - at), exp2_fast(x - at));
          m[j] = mn;
        }
      }
    }
    if (ok) {
#pragma unroll
      for (int j0 = 0; j0 < kRows; j0 += kScoreAhead) {
        if (j0 >= rows) break;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
#pragma unroll
          for (int j = j0; j < j0 + kScoreAhead; ++j) {
            const float m2 = __shfl_xor_sync(0xffffffffu, m[j], o), s2 = __shfl_xor_sync(0xffffffffu, s[j], o);
            const float mn = fmaxf(m[j], m2), at = mn == -INFINITY ? 0.f : mn;
            s[j] = s[j] * exp2_fast(m[j] - at) + s2 * exp2_fast(m2 - at);
            m[j] = mn;
          }
        }
#pragma unroll
        for (int j = j0; j < j0 + kScoreAhead; ++j)
          if (lane == 0 && j < rows)
            P.part[((int64_t)blockIdx.x * kScoreWarps + quarter) * P.part_ld + j] = make_float2(m[j], s[j]);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1)
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(Shape::kTmem) : "memory");
}

// ---------------------------------------------------------------------------
// rows

struct RowsParams {
  const __nv_bfloat16 *h, *w;
  const void *labels;
  const float *row_weight, *upstream;
  const float *lse_in;   // backward alone: the forward's lse per row
  XentHead *head;
  int32_t *idx, *lab;    // place -> row, label
  float *wt, *lse2, *ll2;
  __nv_bfloat16 *hc;     // H by places, rows hc_stride apart
  float *loss, *lse;     // of rows left out: 0
  void *dh;
  int32_t *status;
  int64_t n, v, d, h_stride, w_stride, dh_stride, hc_stride;
  int64_t per_block;     // rows a block takes, a multiple of 8
  float scale2;
  int32_t *redo;         // per row tile, cleared; NULL: no logits will be kept
  int32_t kept;          // logits and marks of an earlier forward stay
  int32_t labels64, mean, dh_f32, vec;
};

__device__ __forceinline__ bool row_counts(const RowsParams &R, int64_t i, int64_t &y, float &w) {
  y = R.labels64 ? reinterpret_cast<const int64_t *>(R.labels)[i] : reinterpret_cast<const int32_t *>(R.labels)[i];
  w = R.row_weight ? R.row_weight[i] : 1.f;
  return y >= 0 && y < R.v && w != 0.f;
}

// Eight consecutive bf16 values, 16-byte aligned or not.
__device__ __forceinline__ uint4 words8(const __nv_bfloat16 *p, bool vec) {
  if (vec) return *reinterpret_cast<const uint4 *>(p);
  const uint16_t *h = reinterpret_cast<const uint16_t *>(p);
  return make_uint4(h[0] | (uint32_t)h[1] << 16, h[2] | (uint32_t)h[3] << 16, h[4] | (uint32_t)h[5] << 16,
                    h[6] | (uint32_t)h[7] << 16);
}

// Every block counts the rows that count, all and those before its own (n
// labels from L2; cheaper than a launch of its own for the scan: 9 us at
// n = 4096), then takes its rows eight at a time, one warp each: the row's
// copy at its place, and its product with the label's row of W (8 products a
// lane and step, in fp32).  Rows left out get zero losses and gradients.  The
// rows n .. n + 255 stand for the places behind the last row up to a whole
// tile: they get zeros.  Sums are taken in the same order by every block.
// Latency bound: at 64 registers, four blocks an SM, 8192 rows of 2048 take
// 20 us (5 TB/s); without that bound, at 72 registers and three blocks, 22.
__global__ void __launch_bounds__(256, 4) xent_rows_kernel(const __grid_constant__ RowsParams R) {
  pdl_launch();
  __shared__ int32_t cnt[2][8];
  __shared__ float red[32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int64_t row0 = blockIdx.x * R.per_block;
  int all = 0, before = 0;
  float wsum = 0.f;
  bool bad = false;
#pragma unroll 8
  for (int64_t i = threadIdx.x; i < R.n; i += 256) {
    int64_t y;
    float w;
    if (row_counts(R, i, y, w)) {
      ++all;
      if (i < row0) ++before;
      wsum += w;
    }
    bad |= y >= R.v;
  }
  all = __reduce_add_sync(0xffffffffu, all);
  before = __reduce_add_sync(0xffffffffu, before);
  if (lane == 0) cnt[0][warp] = all, cnt[1][warp] = before;
  const float ws = block_sum(wsum, red);
  all = before = 0;
  for (int k = 0; k < 8; ++k) all += cnt[0][k], before += cnt[1][k];
  if (blockIdx.x == 0) {
    if (bad) flag_status(R.status, GBO_STATUS_BAD_LABEL);
    if (threadIdx.x == 0) {
      const float up = R.upstream ? *R.upstream : 1.f;
      R.head->rows = all;
      R.head->weight_sum = ws;
      R.head->g = R.mean ? (ws != 0.f ? up / ws : 0.f) : up;
      if (!R.kept) R.head->redo = 0;
    }
    if (R.redo)
      for (int64_t k = threadIdx.x; k < (R.n + kTile - 1) / kTile; k += 256) R.redo[k] = 0;
  }
  const int64_t end = ((int64_t)all + kTile - 1) / kTile * kTile;
  for (int64_t base = row0; base < min(row0 + R.per_block, R.n + kTile); base += 8) {
    int64_t y = -1;
    float w = 0.f;
    const bool in8 = lane < 8 && base + lane < R.n && row_counts(R, base + lane, y, w);
    const uint32_t mask = __ballot_sync(0xffffffffu, in8);
    y = __shfl_sync(0xffffffffu, y, warp);
    w = __shfl_sync(0xffffffffu, w, warp);
    const int64_t i = base + warp;
    const int64_t p = before + __popc(mask & ((1u << warp) - 1u));
    before += __popc(mask);
    if (mask >> warp & 1u) {
      const __nv_bfloat16 *src = R.h + i * R.h_stride, *lab = R.w + y * R.w_stride;
      __nv_bfloat16 *dst = R.hc + p * R.hc_stride;
      float dot = 0.f;
      // four loads of each row in flight (the copies' stores would order
      // loads that are issued one by one behind them)
      for (int64_t c0 = 8 * lane; c0 < R.d; c0 += 4 * 256) {
        uint4 a[4], b[4];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (c0 + 256 * u < R.d) {
            a[u] = words8(src + c0 + 256 * u, R.vec != 0);
            b[u] = *reinterpret_cast<const uint4 *>(lab + c0 + 256 * u);
          }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          if (c0 + 256 * u >= R.d) break;
          *reinterpret_cast<uint4 *>(dst + c0 + 256 * u) = a[u];
          const uint32_t a4[4] = {a[u].x, a[u].y, a[u].z, a[u].w}, b4[4] = {b[u].x, b[u].y, b[u].z, b[u].w};
          float s = 0.f;
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s = fmaf(__uint_as_float(a4[k] << 16), __uint_as_float(b4[k] << 16), s);
            s = fmaf(__uint_as_float(a4[k] & 0xffff0000u), __uint_as_float(b4[k] & 0xffff0000u), s);
          }
          dot += s;
        }
      }
      dot = warp_sum(dot);
      if (lane == 0) {
        R.idx[p] = (int32_t)i;
        R.lab[p] = (int32_t)y;
        R.wt[p] = w;
        R.ll2[p] = dot * R.scale2;
        if (R.lse_in) R.lse2[p] = R.lse_in[i] * kLog2e;
      }
    } else if (i < R.n) {
      if (lane == 0) {
        if (R.loss) R.loss[i] = 0.f;
        if (R.lse) R.lse[i] = 0.f;
      }
      if (R.dh)
        for (int64_t c = lane; c < R.d; c += 32) st_elem(R.dh, R.dh_f32 ? GBO_F32 : GBO_BF16, i * R.dh_stride + c, 0.f);
    } else if (all + (i - R.n) < end) {
      const int64_t t = all + (i - R.n);
      for (int64_t c = lane; c < R.d / 8; c += 32) reinterpret_cast<uint4 *>(R.hc + t * R.hc_stride)[c] = make_uint4(0, 0, 0, 0);
      if (lane == 0) R.idx[t] = 0, R.lab[t] = -1, R.wt[t] = 0.f, R.lse2[t] = 0.f, R.ll2[t] = 0.f;
    }
  }
}

struct LseParams {
  const XentHead *head;
  const float2 *part;
  const float *ll2, *wt;
  const int32_t *idx;
  float *lse2, *loss, *lse, *sums;
  int32_t *status;
  int64_t part_ld;
  int32_t tiles, rows_log2;
  float z;
};

constexpr int kLseThreads = 1024;

// Join the tiles' (maximum, sum) pairs of each row.  A block takes
// 2^rows_log2 rows, consecutive threads consecutive rows, and kLseThreads >>
// rows_log2 strands of tiles; strands join in a fixed tree.  Latency bound:
// 256 threads a block took 18 us for 8192 rows of 500 tiles.
__global__ void __launch_bounds__(kLseThreads) xent_lse_kernel(const __grid_constant__ LseParams L) {
  pdl_launch();
  __shared__ float2 red[kLseThreads];
  __shared__ float wl[kLseThreads];
  pdl_wait();
  const int nr = 1 << L.rows_log2, strands = kLseThreads >> L.rows_log2;
  const int r = threadIdx.x & (nr - 1), strand = threadIdx.x >> L.rows_log2;
  const int rows = L.head->rows;
  const int64_t i = (int64_t)blockIdx.x * nr + r;
  float m = -INFINITY, s = 0.f;
  auto join = [](float &m, float &s, float m2, float s2) {
    const float mn = fmaxf(m, m2), at = mn == -INFINITY ? 0.f : mn;
    s = s * exp2_fast(m - at) + s2 * exp2_fast(m2 - at);
    m = mn;
  };
  if (i < rows) {
    int t = strand;
    for (; t + 3 * strands < L.tiles; t += 4 * strands) {
      float2 p[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) p[u] = L.part[(int64_t)(t + u * strands) * L.part_ld + i];
#pragma unroll
      for (int u = 0; u < 4; ++u) join(m, s, p[u].x, p[u].y);
    }
    for (; t < L.tiles; t += strands) {
      const float2 p = L.part[(int64_t)t * L.part_ld + i];
      join(m, s, p.x, p.y);
    }
  }
  red[threadIdx.x] = make_float2(m, s);
  for (int h = strands >> 1; h > 0; h >>= 1) {
    __syncthreads();
    if (strand < h) {
      const float2 o = red[threadIdx.x + (h << L.rows_log2)];
      join(m, s, o.x, o.y);
      red[threadIdx.x] = make_float2(m, s);
    }
  }
  float weighted = 0.f;
  if (strand == 0 && i < rows) {
    const float lse2 = m + log2f(s), lse = lse2 * kLn2;
    const float loss = (lse2 - L.ll2[i]) * kLn2 + L.z * lse * lse;
    if (!isfinite(loss)) flag_status(L.status, GBO_STATUS_NONFINITE);
    L.lse2[i] = lse2;
    const int32_t row = L.idx[i];
    if (L.loss) L.loss[row] = loss;
    if (L.lse) L.lse[row] = lse;
    weighted = L.wt[i] * loss;
  }
  if (!L.sums) return;
  wl[threadIdx.x] = strand == 0 ? weighted : 0.f;
  __syncthreads();
  const float a = block_sum(wl[threadIdx.x], reinterpret_cast<float *>(red));
  if (threadIdx.x == 0) L.sums[blockIdx.x] = a;
}

struct TotalsParams {
  const float *sums;
  const XentHead *head;
  float *totals;
  int32_t n;
};

__global__ void __launch_bounds__(1024) xent_totals_kernel(const __grid_constant__ TotalsParams T) {
  pdl_launch();
  __shared__ float red[32];
  pdl_wait();
  float a = 0.f;
  for (int k = threadIdx.x; k < T.n; k += 1024) a += T.sums[k];
  a = block_sum(a, red);
  if (threadIdx.x == 0) T.totals[0] = a, T.totals[1] = T.head->weight_sum;
}

struct ConvertParams {
  const XentHead *head;
  const int32_t *redo, *lab;
  const float *wt, *lse2, *ll2;
  uint16_t *p;   // kept logits, replaced by P in bf16
  int64_t ld;
  int32_t v;
  float scale, z;
};

constexpr int kConvertThreads = 256, kConvertLoads = 4;
constexpr int kConvertCols = kConvertThreads * 8 * kConvertLoads;  // columns of a block

// P from the kept logits, in place: 2 bytes read and written per entry, HBM
// bound.  One row and kConvertCols columns a block; 1 / 2 / 4 / 8 loads of 16
// bytes in flight a thread: 835 / 639 / 586 / 587 us for 8192 x 128000 (7.2
// TB/s, the last logits of the forward pass from L2).
__global__ void __launch_bounds__(kConvertThreads) xent_convert_kernel(const __grid_constant__ ConvertParams C) {
  pdl_launch();
  const uint32_t across = (uint32_t)(C.v + kConvertCols - 1) / kConvertCols;
  const int64_t i = blockIdx.x / across;
  const int c0 = (int)(blockIdx.x % across) * kConvertCols + threadIdx.x * 8;
  pdl_wait();
  const int rows = C.head->rows, redo = C.redo[i / kTile];
  if (i >= ((int64_t)rows + kTile - 1) / kTile * kTile || redo) return;
  uint16_t *row = C.p + i * C.ld;
  uint4 raw[kConvertLoads];
#pragma unroll
  for (int u = 0; u < kConvertLoads; ++u)
    if (c0 + u * (8 * kConvertThreads) < C.v) raw[u] = *reinterpret_cast<const uint4 *>(row + c0 + u * (8 * kConvertThreads));
  float wt = 0.f, off = 0.f, peak = 0.f, mult = 0.f;
  int lab = -1;
  if (i < rows) {
    const float lse2 = C.lse2[i];
    wt = C.wt[i], lab = C.lab[i], off = C.ll2[i] - lse2;
    mult = wt * C.scale, peak = mult * fmaf(2.f * C.z, lse2 * kLn2, 1.f);
  }
#pragma unroll
  for (int u = 0; u < kConvertLoads; ++u) {
    const int c = c0 + u * (8 * kConvertThreads);
    if (c >= C.v) continue;
    const uint32_t w[4] = {raw[u].x, raw[u].y, raw[u].z, raw[u].w};
    float v[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int q = (int)(int16_t)(w[e / 2] >> (16 * (e & 1)));
      const float x = peak * exp2_fast(fmaf((float)q, 1.f / kKeepStep, off));
      v[e] = wt == 0.f || q == -32768 ? 0.f : x;
    }
    if (lab >= c && lab < c + 8) {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (lab == c + e) v[e] -= mult;
    }
    store8(reinterpret_cast<__nv_bfloat16 *>(row + c), v, 8, true);
  }
}

struct JoinParams {
  const XentHead *head;
  const int32_t *idx;
  const float *acc;
  void *dh;
  int64_t acc_ld, d, dh_stride;
  int32_t splits, dh_f32;
};

// dH from the cuts of its K axis, added in their order.  Four columns a thread.
__global__ void __launch_bounds__(256) xent_join_kernel(const __grid_constant__ JoinParams J) {
  pdl_launch();
  const int64_t i = blockIdx.x;
  pdl_wait();
  if (i >= J.head->rows) return;
  const float g = J.head->g;
  const int64_t row = J.idx[i] * J.dh_stride;
  for (int64_t c = 4 * threadIdx.x; c < J.d; c += 1024) {
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll 4
    for (int s = 0; s < J.splits; ++s) {
      const float4 b = *reinterpret_cast<const float4 *>(J.acc + s * J.acc_ld + i * J.d + c);
      a.x += b.x, a.y += b.y, a.z += b.z, a.w += b.w;
    }
    const float v[4] = {g * a.x, g * a.y, g * a.z, g * a.w};
#pragma unroll
    for (int e = 0; e < 4; ++e) st_elem(J.dh, J.dh_f32 ? GBO_F32 : GBO_BF16, row + c + e, v[e]);
  }
}

// ---------------------------------------------------------------------------
// host

int64_t up_to(int64_t x, int64_t m) { return (x + m - 1) / m * m; }

// Scratch of a call, in this order.
struct XentSpace {
  int64_t head, redo, idx, lab, wt, lse2, ll2, sums, hc, acc, part, p;  // byte offsets
  int64_t n_pad, bytes, hc_ld;
  int64_t piece;            // columns of a piece of the vocabulary
  int64_t ld;               // elements of a row of P: an odd number of 128-byte lines
  int32_t pieces;
  int32_t keep;             // logits are kept between the passes, in P's room
  int32_t splits, split_kit;
};

constexpr int64_t kPieceBytes = int64_t(2) << 30;  // P of one piece, unless the caller caps the workspace
constexpr int64_t kKeepBytes = int64_t(8) << 30;   // kept logits, likewise
// Logits are kept unless they are many and their rows narrow: then forming
// them again costs less than storing and converting them (us, kept / formed
// again, rows x columns: 4096 x 32000 at d = 64 312 / 263, d = 256 333 / 297,
// d = 512 414 / 395 alone and 419 / 412 in a loop, d = 1024 594 / 660; 256 x
// 32000 at d = 64 42.3 / 40.8, d = 256 48.5 / 48.2; 256 x 1000 at d = 64 24.8
// / 26.4, d = 256 28.1 / 31.0).
constexpr int64_t kNarrow = 512, kMany = int64_t(1) << 23;
constexpr int kPairs = 76;                         // CTA pairs of the device
constexpr int kMostSms = 256;

// grad: with the backward pass.  keep: the whole vocabulary's logits are kept
// from the forward pass (one piece); else piece: columns per piece (0: as many
// as kPieceBytes holds), and the tiles' statistics and P share their room (the
// statistics are done with before P is written).
XentSpace space_of(int64_t n, int64_t v, int64_t d, bool grad, bool forward, bool keep, int64_t piece) {
  XentSpace s = {};
  s.n_pad = up_to(std::max<int64_t>(n, 1), kTile);
  s.keep = keep;
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t r = at;
    at += up_to(bytes, 1024);
    return r;
  };
  s.head = take(sizeof(XentHead));
  s.redo = take(4 * s.n_pad / kTile);
  s.idx = take(4 * s.n_pad);
  s.lab = take(4 * s.n_pad);
  s.wt = take(4 * s.n_pad);
  s.lse2 = take(4 * s.n_pad);
  s.ll2 = take(4 * s.n_pad);
  s.sums = take(4 * s.n_pad);
  // rows of whole 128-byte lines: TMA reads a row that straddles two lines as two
  s.hc_ld = up_to(d, 64);
  s.hc = take(2 * s.n_pad * s.hc_ld);
  // statistics: per epilogue warp's columns, or (few rows) per CTA and epilogue warp
  int64_t slots = (v + kSpan - 1) / kSpan;
  if (n <= kScoreMost) slots = std::max<int64_t>(slots, kScoreWarps * kMostSms);
  const int64_t part = forward ? 8 * s.n_pad * slots : 0;
  if (!grad) {
    s.part = take(part);
    s.bytes = at;
    return s;
  }
  if (keep) piece = up_to(v, kTile);
  else if (piece <= 0) piece = kPieceBytes / (2 * s.n_pad);
  piece = std::max<int64_t>(kTile, piece / kTile * kTile);
  s.pieces = (int32_t)((v + piece - 1) / piece);
  s.piece = up_to((v + s.pieces - 1) / s.pieces, kTile);  // even pieces
  s.pieces = (int32_t)((v + s.piece - 1) / s.piece);
  // With few rows dH has few items, each with the whole piece as its K:
  // cut K until no item is longer than half a pair's share of the launch,
  // but no shorter than 8 stages.  777 x 32003 x 1032: products 184 us uncut
  // (20 items of 251 stages on 76 pairs).
  const int64_t m_tiles = s.n_pad / kTile, d_tiles = (d + kTile - 1) / kTile;
  const int64_t dh_kit = (s.piece + kStageK - 1) / kStageK;
  const int64_t share =
      std::max<int64_t>(1, (m_tiles * d_tiles * dh_kit + s.piece / kTile * d_tiles * item_cost((int)(s.n_pad / kStageK))) / kPairs);
  int64_t splits = std::min<int64_t>(std::min<int64_t>(16, std::max<int64_t>(1, dh_kit / 8)), (2 * dh_kit + share - 1) / share);
  s.split_kit = (int32_t)((dh_kit + splits - 1) / splits);
  s.splits = (int32_t)((dh_kit + s.split_kit - 1) / s.split_kit);
  s.acc = take(s.pieces > 1 || s.splits > 1 ? 4 * s.splits * s.n_pad * d : 0);
  // dW reads P by columns: rows a power of two apart would all lie in the same
  // few memory channels
  s.ld = s.piece + 64;
  if (keep) {
    s.part = take(part);
    s.p = take(2 * s.n_pad * s.ld);
  } else {
    s.part = s.p = take(std::max(part, 2 * s.n_pad * s.ld));
  }
  s.bytes = at;
  return s;
}

bool keeps(int64_t n, int64_t v, int64_t d) { return d >= kNarrow || up_to(n, kTile) * v < kMany; }

// What a call does without a cap.
XentSpace default_space(int64_t n, int64_t v, int64_t d) {
  const bool keep = keeps(n, v, d) && 2 * up_to(std::max<int64_t>(n, 1), kTile) * up_to(v, kTile) <= kKeepBytes;
  return space_of(n, v, d, true, true, keep, 0);
}

// The fastest schedule whose workspace fits `bytes`: kept logits (see
// kNarrow), else the widest pieces (false: not even one of kTile columns).
bool fit_space(int64_t n, int64_t v, int64_t d, bool forward, int64_t bytes, XentSpace *out) {
  if (forward && keeps(n, v, d)) {
    *out = space_of(n, v, d, true, true, true, 0);
    if (out->bytes <= bytes) return true;
  }
  *out = space_of(n, v, d, true, forward, false, 0);
  if (out->bytes <= bytes) return true;
  int64_t lo = 1, hi = up_to(v, kTile) / kTile;  // pieces of lo tiles fit, of hi do not
  if (space_of(n, v, d, true, forward, false, kTile).bytes > bytes) return false;
  while (hi - lo > 1) {
    const int64_t mid = (lo + hi) / 2;
    (space_of(n, v, d, true, forward, false, mid * kTile).bytes <= bytes ? lo : hi) = mid;
  }
  *out = space_of(n, v, d, true, forward, false, lo * kTile);
  return true;
}

int xent_fail(int code, const char *msg) { return report_error(code, msg); }

int check_args(const gbo_xent_args *a) {
  if (!a) return xent_fail(GBO_ERR_INVALID_ARG, "args is NULL");
  if (a->n < 0 || a->n > (int64_t(1) << 30)) return xent_fail(GBO_ERR_SHAPE, "n must be in 0..2^30");
  if (a->v < 1 || a->v > (int64_t(1) << 30)) return xent_fail(GBO_ERR_SHAPE, "v must be in 1..2^30");
  if (a->d < 8 || a->d % 8 || a->d > (1 << 20)) return xent_fail(GBO_ERR_SHAPE, "d must be a multiple of 8 in 8..2^20");
  if (a->h_stride < a->d || a->w_stride < a->d) return xent_fail(GBO_ERR_SHAPE, "a row stride is smaller than d");
  if (a->w_stride % 8) return xent_fail(GBO_ERR_SHAPE, "w_stride must be a multiple of 8 elements (16-byte rows)");
  if (!a->w || (reinterpret_cast<uintptr_t>(a->w) & 15))
    return xent_fail(GBO_ERR_INVALID_ARG, "w is NULL or not 16-byte aligned");
  if (a->n > 0 && (!a->h || (reinterpret_cast<uintptr_t>(a->h) & 1) || !a->labels))
    return xent_fail(GBO_ERR_INVALID_ARG, "h or labels NULL or misaligned");
  if (a->label_dtype != GBO_I32 && a->label_dtype != GBO_I64)
    return xent_fail(GBO_ERR_DTYPE, "labels must be GBO_I32 or GBO_I64");
  if (reinterpret_cast<uintptr_t>(a->labels) % (a->label_dtype == GBO_I64 ? 8 : 4))
    return xent_fail(GBO_ERR_INVALID_ARG, "labels misaligned");
  if ((reinterpret_cast<uintptr_t>(a->row_weight) & 3) || (reinterpret_cast<uintptr_t>(a->upstream) & 3))
    return xent_fail(GBO_ERR_INVALID_ARG, "row_weight or upstream misaligned");
  if (!std::isfinite(a->logit_scale) || !std::isfinite(a->z_loss))
    return xent_fail(GBO_ERR_INVALID_ARG, "non-finite logit_scale or z_loss");
  if (a->mean != 0 && a->mean != 1) return xent_fail(GBO_ERR_INVALID_ARG, "mean must be 0 or 1");
  if (a->keep != 0 && a->keep != 1) return xent_fail(GBO_ERR_INVALID_ARG, "keep must be 0 or 1");
  return GBO_OK;
}

int check_grads(const gbo_xent_args *a, const gbo_xent_grads *g) {
  if (!g || (!g->dh && !g->dw)) return xent_fail(GBO_ERR_INVALID_ARG, "no gradient is asked for");
  const int32_t types[2] = {g->dh_dtype, g->dw_dtype};
  const void *ptrs[2] = {g->dh, g->dw};
  const int64_t strides[2] = {g->dh_stride, g->dw_stride};
  for (int k = 0; k < 2; ++k) {
    if (!ptrs[k]) continue;
    if (types[k] != GBO_F32 && types[k] != GBO_BF16) return xent_fail(GBO_ERR_DTYPE, "gradients are GBO_F32 or GBO_BF16");
    if (reinterpret_cast<uintptr_t>(ptrs[k]) % (types[k] == GBO_F32 ? 4 : 2))
      return xent_fail(GBO_ERR_INVALID_ARG, "a gradient is misaligned");
    if (strides[k] < a->d) return xent_fail(GBO_ERR_SHAPE, "a gradient's row stride is smaller than d");
  }
  if (g->accumulate_dw != 0 && g->accumulate_dw != 1) return xent_fail(GBO_ERR_INVALID_ARG, "accumulate_dw must be 0 or 1");
  return GBO_OK;
}

// The launches of a call depend on one another alone, and its kernels are
// short when there are few rows: they carry the programmatic-dependent-launch
// attribute on direct launches too (one token over 128000 x 2048: 108.0 ->
// 101.8 us; 777 rows: 289.8 -> 277.1 us; thousands of rows: equal).
template <typename K>
cudaError_t chain(void (*kernel)(K), dim3 grid, dim3 block, cudaStream_t stream, const K &params) {
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), kernel, grid, block, 0, stream, 1, params);
}

// The kernel's shared memory limit was raised (or not), and the CTA pairs that
// are resident together.
struct PairState {
  cudaError_t err = cudaSuccess;
  int resident = 0;
};

template <int kMode>
cudaError_t launch_xent(const XentParams &P, int64_t items, int sm, int dev, cudaStream_t stream) {
  static PerDevice<PairState> states;
  const PairState *state = states.of(dev, [&](PairState &s) {
    s.err = cudaFuncSetAttribute(xent_kernel<kMode>, cudaFuncAttributeMaxDynamicSharedMemorySize, kXentSmem);
    if (s.err != cudaSuccess) return;
    cudaLaunchConfig_t cfg = {};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    cfg.blockDim = dim3(kXentThreads);
    cfg.dynamicSmemBytes = kXentSmem;
    cfg.gridDim = dim3(2 * std::max(1, sm / 2));
    if (cudaOccupancyMaxActiveClusters(&s.resident, xent_kernel<kMode>, &cfg) != cudaSuccess) s.resident = 0;
    (void)cudaGetLastError();
  });
  if (!state || state->err != cudaSuccess) return state ? state->err : cudaErrorInvalidDevice;
  const int resident = state->resident;
  const int64_t fit = std::max(1, resident > 0 ? std::min(resident, sm / 2) : sm / 2);
  const int clusters = (int)std::max<int64_t>(1, std::min(items, fit));
  const cudaError_t e = launch_kernel_as(pdl_allowed(), xent_kernel<kMode>, dim3(2 * clusters), dim3(kXentThreads),
                                         kXentSmem, stream, 2, P);
  count_launches(1);
  return e;
}

bool map_2d(CUtensorMap *m, const void *p, int64_t cols, int64_t rows, int64_t ld, uint32_t bc, uint32_t br,
            CUtensorMapSwizzle sw = CU_TENSOR_MAP_SWIZZLE_128B) {
  return encode_map(m, const_cast<void *>(p), cols, rows, 1, ld, bc, br, sw);
}

int cuda_err(cudaError_t e) {
  char msg[200];
  snprintf(msg, sizeof msg, "cross-entropy kernels: %s", cudaGetErrorString(e));
  return xent_fail(GBO_ERR_CUDA, msg);
}

// Few rows: which kernel takes their statistics (see xent_score_kernel; 0: the
// 256-wide tiles).  Up to 16 rows, and up to 32 where the table is large: the
// epilogue grows with the rows.  Us, 16 / 32 / wide, for 1 row of 128000 x 2048
// 87.0 / 88.0 / 103.3, of 32000 x 1024 15.8 / 16.5 / 19.8; 16 rows 88.7 / 89.5
// / 104.0 and 17.9 / 18.3 / 19.6, of 1000 x 64 10.6 / 10.7 / 10.0; 32 rows of
// 128000 x 2048 - / 91.6 / 101.7, 128000 x 320 - / 25.4 / 30.1, 50257 x 768 -
// / 22.2 / 21.1, 32000 x 1024 - / 21.0 / 19.5.
constexpr int64_t kScoreTable = 80000000;  // bytes
int score_rows(int64_t n, int64_t v, int64_t d) {
  return n <= 16 ? 16 : n <= kScoreMost && 2 * v * d >= kScoreTable ? 32 : 0;
}

// Statistics of at most kRows rows; *blocks: CTAs, each with a slot of
// statistics per epilogue warp.
template <int kRows>
int run_score(const gbo_xent_args *a, const XentParams &P, const RowsParams &R, int sm, int dev, cudaStream_t st,
              int *blocks) {
  ScoreParams Q;
  memset(&Q, 0, sizeof Q);
  Q.head = P.head, Q.lab = P.lab, Q.ll2 = P.ll2, Q.part = P.part, Q.part_ld = P.part_ld, Q.status = P.status;
  Q.v = (int32_t)a->v, Q.d = P.d, Q.scale2 = P.scale2;
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(xent_score_kernel<kRows>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             ScoreShape<kRows>::kSmem);
  });
  if (!err || *err != cudaSuccess) return cuda_err(err ? *err : cudaErrorInvalidDevice);
  // one CTA an SM, each with at least two 16-row units
  *blocks = (int)std::min<int64_t>(std::min(sm, kMostSms), std::max<int64_t>(1, a->v / (2 * kScoreUnit)));
  // rounds of whole tiles; the last round and what is left are one run a CTA
  const int64_t round = (int64_t)BM * *blocks;
  Q.whole = (int32_t)std::max<int64_t>(0, (a->v - 1) / round - 1);
  const int64_t units = (a->v - Q.whole * round + kScoreUnit - 1) / kScoreUnit, most = (units + *blocks - 1) / *blocks;
  const int64_t parts = (most * kScoreUnit + BM - 1) / BM;
  Q.step = (int32_t)((most + parts - 1) / parts * kScoreUnit);
  if (!map_2d(&Q.mapW, a->w, a->d, a->v, a->w_stride, kBlockK, BM) ||
      !map_2d(&Q.mapRest, a->w, a->d, a->v, a->w_stride, kBlockK, Q.step) ||
      !map_2d(&Q.mapH, R.hc, a->d, kTile, R.hc_stride, kBlockK, kRows))
    return xent_fail(GBO_ERR_CUDA, "tensor map of H or W");
  const cudaError_t e = launch_kernel_as(pdl_allowed(), xent_score_kernel<kRows>, dim3(*blocks), dim3(192),
                                         ScoreShape<kRows>::kSmem, st, 1, Q);
  count_launches(1);
  return e == cudaSuccess ? GBO_OK : cuda_err(e);
}

// forward: loss, lse, totals.  g: gradients too (lse_in: with the forward
// pass skipped, its lse).
int xent_run(const gbo_xent_args *a, bool forward, float *loss, float *lse, float *totals, const float *lse_in,
             const gbo_xent_grads *g, void *workspace, size_t ws_bytes, int32_t *status, gbo_stream_t stream) {
  int rc = check_args(a);
  if (rc != GBO_OK) return rc;
  if (g && (rc = check_grads(a, g)) != GBO_OK) return rc;
  if (!forward && a->n > 0 && !lse_in) return xent_fail(GBO_ERR_INVALID_ARG, "lse is NULL");
  if ((reinterpret_cast<uintptr_t>(loss) | reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(totals) |
       reinterpret_cast<uintptr_t>(lse_in) | reinterpret_cast<uintptr_t>(status)) & 3)
    return xent_fail(GBO_ERR_INVALID_ARG, "misaligned output, lse or status pointer");
  int dev, sm = 0;
  if ((rc = require_device(&dev, &sm)) != GBO_OK) return rc;
  XentSpace S;
  // the same schedule for both halves of a kept pair of calls
  const bool whole = (forward && g) || a->keep;
  if (g || a->keep) {
    if (!fit_space(a->n, a->v, a->d, whole, (int64_t)ws_bytes, &S))
      return xent_fail(GBO_ERR_WORKSPACE, "workspace too small for a piece of 256 columns");
  } else {
    S = space_of(a->n, a->v, a->d, false, true, false, 0);
  }
  if (!workspace || (int64_t)ws_bytes < S.bytes) return xent_fail(GBO_ERR_WORKSPACE, "workspace missing or too small");
  if (reinterpret_cast<uintptr_t>(workspace) & 255) return xent_fail(GBO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  char *ws = static_cast<char *>(workspace);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;

  RowsParams R = {};
  R.h = static_cast<const __nv_bfloat16 *>(a->h), R.w = static_cast<const __nv_bfloat16 *>(a->w);
  R.labels = a->labels, R.row_weight = a->row_weight, R.upstream = a->upstream, R.lse_in = forward ? nullptr : lse_in;
  R.head = reinterpret_cast<XentHead *>(ws + S.head);
  R.idx = reinterpret_cast<int32_t *>(ws + S.idx);
  R.lab = reinterpret_cast<int32_t *>(ws + S.lab);
  R.wt = reinterpret_cast<float *>(ws + S.wt);
  R.lse2 = reinterpret_cast<float *>(ws + S.lse2);
  R.ll2 = reinterpret_cast<float *>(ws + S.ll2);
  R.hc = reinterpret_cast<__nv_bfloat16 *>(ws + S.hc);
  R.loss = loss, R.lse = lse, R.dh = g ? g->dh : nullptr;
  int32_t *redo = reinterpret_cast<int32_t *>(ws + S.redo);
  R.redo = S.keep && forward ? redo : nullptr;
  R.kept = S.keep && !forward;
  R.status = status;
  R.n = a->n, R.v = a->v, R.d = a->d;
  R.h_stride = a->h_stride, R.w_stride = a->w_stride, R.dh_stride = g ? g->dh_stride : 0;
  R.hc_stride = S.hc_ld;
  R.scale2 = a->logit_scale * kLog2e;
  R.labels64 = a->label_dtype == GBO_I64, R.mean = a->mean;
  R.dh_f32 = g && g->dh_dtype == GBO_F32;
  R.vec = a->h_stride % 8 == 0 && (reinterpret_cast<uintptr_t>(a->h) & 15) == 0;
  // eight blocks an SM at most: each reads all labels
  const int64_t virt = a->n + kTile, most = (int64_t)8 * sm;
  R.per_block = up_to((virt + most - 1) / most, 8);
  if ((e = chain(xent_rows_kernel, dim3((unsigned)((virt + R.per_block - 1) / R.per_block)), dim3(256), st, R)) !=
      cudaSuccess)
    return cuda_err(e);

  XentParams P;
  memset(&P, 0, sizeof P);
  P.head = R.head, P.idx = R.idx, P.lab = R.lab, P.wt = R.wt, P.lse2 = R.lse2;
  P.ll2 = R.ll2;
  P.status = status;
  P.d = (int32_t)a->d;
  P.scale = a->logit_scale, P.scale2 = a->logit_scale * kLog2e, P.z = a->z_loss;
  const int64_t m_tiles = S.n_pad / kTile, d_tiles = (a->d + kTile - 1) / kTile;
  bool maps = true;
  if (a->n > 0) {
    maps = map_2d(&P.mapA, R.hc, a->d, S.n_pad, S.hc_ld, kBlockK, BM) &&
           map_2d(&P.mapB, a->w, a->d, a->v, a->w_stride, kBlockK, BM);
    if (!maps) return xent_fail(GBO_ERR_CUDA, "tensor map of H or W");
  }
  if (forward && a->n > 0) {
    P.part = reinterpret_cast<float2 *>(ws + S.part);
    P.keep = S.keep;
    if (S.keep) {
      P.redo = redo, P.head_out = R.head;
      if (!map_2d(&P.mapO, ws + S.p, a->v, S.n_pad, S.ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B))
        return xent_fail(GBO_ERR_CUDA, "tensor map of the logits");
    }
    P.part_ld = S.n_pad;
    P.v0 = 0, P.v_piece = (int32_t)a->v;
    const int64_t n_tiles = (a->v + kTile - 1) / kTile;
    int64_t slots = (a->v + kSpan - 1) / kSpan;
    if (const int few = S.keep ? 0 : score_rows(a->n, a->v, a->d)) {
      int blocks = 0;
      rc = few == 16 ? run_score<16>(a, P, R, sm, dev, st, &blocks) : run_score<32>(a, P, R, sm, dev, st, &blocks);
      if (rc != GBO_OK) return rc;
      slots = (int64_t)kScoreWarps * blocks;
    } else if ((e = launch_xent<kModeStats>(P, m_tiles * n_tiles, sm, dev, st)) != cudaSuccess) {
      return cuda_err(e);
    }
    LseParams L = {};
    L.head = R.head, L.part = P.part, L.ll2 = P.ll2, L.wt = R.wt, L.idx = R.idx;
    L.lse2 = R.lse2, L.loss = loss, L.lse = lse;
    L.sums = totals ? reinterpret_cast<float *>(ws + S.sums) : nullptr;
    L.status = status;
    L.part_ld = S.n_pad, L.tiles = (int32_t)slots, L.z = a->z_loss;
    // four rows a block (a sector of statistics), more where that is more than
    // two blocks an SM: with 32 rows a block from the start, 256 rows of
    // 128000 x 2048 took 113.5 us in all instead of 107.6
    while (L.rows_log2 < 5 && (1 << L.rows_log2) < a->n && (L.rows_log2 < 2 || a->n >> L.rows_log2 > 2 * sm)) ++L.rows_log2;
    const int blocks = (int)((a->n + (1 << L.rows_log2) - 1) >> L.rows_log2);
    if ((e = chain(xent_lse_kernel, dim3(blocks), dim3(kLseThreads), st, L)) != cudaSuccess) return cuda_err(e);
    if (totals && (e = chain(xent_totals_kernel, dim3(1), dim3(1024), st, TotalsParams{L.sums, R.head, totals, blocks})) !=
                      cudaSuccess)
      return cuda_err(e);
  } else if (forward && totals) {
    if ((e = chain(xent_totals_kernel, dim3(1), dim3(1024), st, TotalsParams{nullptr, R.head, totals, 0})) != cudaSuccess)
      return cuda_err(e);
  }
  if (g) {
    P.dh = a->n > 0 ? g->dh : nullptr, P.dw = g->dw;
    P.dh_stride = g->dh_stride, P.dw_stride = g->dw_stride;
    P.dh_f32 = g->dh_dtype == GBO_F32, P.dw_f32 = g->dw_dtype == GBO_F32;
    P.dh_vec = (reinterpret_cast<uintptr_t>(g->dh) & 15) == 0 && g->dh_stride % (P.dh_f32 ? 4 : 8) == 0;
    P.dw_vec = (reinterpret_cast<uintptr_t>(g->dw) & 15) == 0 && g->dw_stride % (P.dw_f32 ? 4 : 8) == 0;
    P.dw_add = g->accumulate_dw;
    P.dh_acc = reinterpret_cast<float *>(ws + S.acc);
    P.acc_ld = S.n_pad * a->d;
    P.splits = S.splits, P.split_kit = S.split_kit;
    void *pbuf = ws + S.p;
    if (S.keep && a->n > 0) {
      ConvertParams C = {};
      C.head = R.head, C.redo = redo, C.lab = R.lab, C.wt = R.wt, C.lse2 = R.lse2, C.ll2 = R.ll2;
      C.p = static_cast<uint16_t *>(pbuf), C.ld = S.ld, C.v = (int32_t)a->v;
      C.scale = a->logit_scale, C.z = a->z_loss;
      const int64_t blocks = (a->v + kConvertCols - 1) / kConvertCols * S.n_pad;
      if (blocks > INT32_MAX) return xent_fail(GBO_ERR_SHAPE, "more kept logits than one launch takes: cap the workspace");
      if ((e = chain(xent_convert_kernel, dim3((unsigned)blocks), dim3(kConvertThreads), st, C)) != cudaSuccess) return cuda_err(e);
      P.redo = redo, P.only_redo = 1;
    }
    for (int32_t c = 0; c < S.pieces; ++c) {
      P.v0 = c * S.piece;
      P.v_piece = (int32_t)std::min<int64_t>(S.piece, a->v - P.v0);
      P.first_piece = c == 0, P.last_piece = c + 1 == S.pieces;
      const int64_t n_tiles = (P.v_piece + kTile - 1) / kTile;
      XentParams Q = P;
      maps = map_2d(&P.mapO, pbuf, P.v_piece, S.n_pad, S.ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B) &&
             map_2d(&Q.mapA, pbuf, P.v_piece, S.n_pad, S.ld, kBlockK, BM) &&
             map_2d(&Q.mapB, a->w, a->d, a->v, a->w_stride, 64, kBlockK) &&
             map_2d(&Q.mapA2, pbuf, P.v_piece, S.n_pad, S.ld, 64, kBlockK) &&
             map_2d(&Q.mapB2, R.hc, a->d, S.n_pad, S.hc_ld, 64, kBlockK);
      // dW by TMA where its rows are 16-byte aligned (adding to bf16 stays with the
      // threads: the sum is rounded once)
      Q.dw_tma = P.dw && P.dw_vec && !(P.dw_add && !P.dw_f32);
      if (Q.dw_tma)  // (a table too far apart for a map stays with the threads)
        Q.dw_tma = P.dw_f32 ? encode_map(&Q.mapO, P.dw, a->d, a->v, 1, P.dw_stride, 32, 32, CU_TENSOR_MAP_SWIZZLE_128B,
                                         CU_TENSOR_MAP_DATA_TYPE_FLOAT32, 4)
                            : map_2d(&Q.mapO, P.dw, a->d, a->v, P.dw_stride, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B);
      if (!maps) return xent_fail(GBO_ERR_CUDA, "tensor map of P");
      if (a->n > 0 && (e = launch_xent<kModeP>(P, m_tiles * n_tiles, sm, dev, st)) != cudaSuccess) return cuda_err(e);
      const int64_t items = (P.dh ? m_tiles * d_tiles * S.splits : 0) + (P.dw ? n_tiles * d_tiles : 0);
      if (items > 0 && (e = launch_xent<kModeProducts>(Q, items, sm, dev, st)) != cudaSuccess) return cuda_err(e);
    }
    if (P.dh && S.splits > 1) {
      JoinParams J = {};
      J.head = R.head, J.idx = R.idx, J.acc = P.dh_acc, J.dh = P.dh;
      J.acc_ld = P.acc_ld, J.d = a->d, J.dh_stride = P.dh_stride;
      J.splits = S.splits, J.dh_f32 = P.dh_f32;
      if ((e = chain(xent_join_kernel, dim3((unsigned)a->n), dim3(256), st, J)) != cudaSuccess) return cuda_err(e);
    }
  }
  return report_ok();
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" size_t gbo_xent_workspace_bytes(int64_t n, int64_t v, int64_t d, int32_t grad, int64_t cap) {
  if (n < 0 || v < 1 || d < 8 || d % 8 || n > (int64_t(1) << 30) || v > (int64_t(1) << 30) || d > (1 << 20)) return 0;
  if (!grad) return (size_t)space_of(n, v, d, false, true, false, 0).bytes;
  XentSpace s;
  if (cap > 0) return fit_space(n, v, d, true, cap, &s) ? (size_t)s.bytes : 0;
  return (size_t)default_space(n, v, d).bytes;
}

extern "C" int gbo_xent_forward(const gbo_xent_args *args, float *loss, float *lse, float *totals, void *workspace,
                                size_t ws_bytes, int32_t *dev_status, gbo_stream_t stream) {
  return xent_run(args, true, loss, lse, totals, nullptr, nullptr, workspace, ws_bytes, dev_status, stream);
}

extern "C" int gbo_xent_backward(const gbo_xent_args *args, const float *lse, const gbo_xent_grads *grads,
                                 void *workspace, size_t ws_bytes, int32_t *dev_status, gbo_stream_t stream) {
  if (!grads) return xent_fail(GBO_ERR_INVALID_ARG, "grads is NULL");
  return xent_run(args, false, nullptr, nullptr, nullptr, lse, grads, workspace, ws_bytes, dev_status, stream);
}

extern "C" int gbo_xent_grad(const gbo_xent_args *args, float *loss, float *lse, float *totals,
                             const gbo_xent_grads *grads, void *workspace, size_t ws_bytes, int32_t *dev_status,
                             gbo_stream_t stream) {
  if (!grads) return xent_fail(GBO_ERR_INVALID_ARG, "grads is NULL");
  return xent_run(args, true, loss, lse, totals, nullptr, grads, workspace, ws_bytes, dev_status, stream);
}

// Pieces shared by the attention kernels: which keys a query sees, the mapping
// of a tile's rows to tokens and heads, TMEM and tcgen05 wrappers, bounded
// waits, tensor maps, and the checks of the arguments.
#pragma once

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "gbo.h"
#include "internal.h"
#include "pairs.cuh"
#include "per_device.h"
#include "tc_common.cuh"

namespace gbo {

constexpr int64_t kAttnMaxLength = int64_t(1) << 30;
constexpr int kAttnMaxPack = 5;          // heads of a block: 32 at most, so that a warp's rows are whole tokens
constexpr int kAttnTile = 128;           // rows and keys of a tile
constexpr int kAttnBlock = 128 * 128;    // bytes of 128 rows of 64 bf16 (one 128-byte line each)

// Which keys the queries of a sequence see.  Query t sees the keys of one
// interval, whose ends do not decrease with t; so does a key of its queries.
struct AttnMask {
  const int32_t *q_len, *k_len;  // per sequence, or NULL: sq, sk
  const int32_t *docs;           // first tokens of n_docs documents and the end of the last, or NULL
  int32_t n_docs, causal, window, sq, sk;
};

struct AttnSeq {
  int32_t q_lo, q_hi;  // queries that may see a key at all
  int32_t k_lo, k_hi;  // keys that may be seen at all: what stands in others reaches nothing
  int32_t shift;       // query t stands at position t + shift among the keys
};

struct Span {
  int32_t lo, hi;
  __device__ __forceinline__ bool empty() const { return hi <= lo; }
};

// (arguments of an entry point may hold anything a caller put on the device)
__device__ __forceinline__ int32_t clamp_to(int32_t v, int32_t most) { return min(max(v, 0), most); }

__device__ __forceinline__ AttnSeq attn_seq(const AttnMask &M, int b) {
  AttnSeq s;
  const int32_t lq = M.q_len ? clamp_to(M.q_len[b], M.sq) : M.sq, lk = M.k_len ? clamp_to(M.k_len[b], M.sk) : M.sk;
  s.shift = lk - lq;
  s.q_lo = 0, s.q_hi = lk > 0 ? lq : 0;
  s.k_lo = 0, s.k_hi = lq > 0 ? lk : 0;
  if (M.causal) s.q_lo = min(max(0, -s.shift), s.q_hi);
  if (M.docs) {
    s.q_lo = s.k_lo = clamp_to(M.docs[0], M.sk);
    s.q_hi = s.k_hi = max(s.k_lo, clamp_to(M.docs[M.n_docs], M.sk));
  }
  return s;
}

// 32 document starts (and the end of the last, where it is among them), one a
// lane: those from the document that holds some token on, or all of them.  A
// search in memory takes a dependent load a step, some 500 clocks each; one among
// lanes takes a shuffle a step.
struct DocWindow {
  int32_t base, v;
};

// All lanes of a warp, with the same t.
__device__ __forceinline__ DocWindow doc_window(const AttnMask &M, int t) {
  DocWindow w = {0, 0};
  if (!M.docs) return w;
  const int lane = threadIdx.x & 31;
  if (M.n_docs > 31)
    for (int len = M.n_docs; len > 1;) {
      const int step = (len + 31) / 32, at = w.base + lane * step;
      const int count = __popc(__ballot_sync(0xffffffffu, lane * step < len && M.docs[min(at, M.n_docs)] <= t));
      w.base = min(w.base + max(count - 1, 0) * step, M.n_docs - 1);
      len = step;
    }
  w.v = clamp_to(M.docs[min(w.base + lane, M.n_docs)], M.sk);
  return w;
}

// The document of token t: the last one that starts at or before it.  All lanes
// of a warp together, each with a token of its own.
__device__ __forceinline__ Span attn_doc(const AttnMask &M, const DocWindow &w, int t) {
  int at = 0;
  const int last = min(31, M.n_docs - 1 - w.base);
#pragma unroll
  for (int step = 16; step > 0; step >>= 1) {
    const int32_t start = __shfl_sync(0xffffffffu, w.v, (at + step) & 31);
    if (at + step <= last && start <= t) at += step;
  }
  Span d = {__shfl_sync(0xffffffffu, w.v, at), __shfl_sync(0xffffffffu, w.v, min(at + 1, 31))};
  if (at == 31) {  // more than 31 documents from the window's first on: those behind it
    int lo = w.base + 31, hi = M.n_docs - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (M.docs[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    d = {clamp_to(M.docs[lo], M.sk), clamp_to(M.docs[lo + 1], M.sk)};
  }
  return d;
}

// Keys that query t (q_lo <= t < q_hi) sees.  All lanes of a warp together.
__device__ __forceinline__ Span keys_of(const AttnMask &M, const AttnSeq &s, const DocWindow &w, int t) {
  Span r = {s.k_lo, s.k_hi};
  const int at = t + s.shift;
  if (M.causal) r.hi = min(r.hi, at + 1);
  if (M.window) r.lo = max(r.lo, at - M.window + 1);
  if (M.docs) {
    const Span d = attn_doc(M, w, t);
    r.lo = max(r.lo, d.lo), r.hi = min(r.hi, d.hi);
  }
  return r;
}

// Queries that see key j (k_lo <= j < k_hi).  All lanes of a warp together.
__device__ __forceinline__ Span queries_of(const AttnMask &M, const AttnSeq &s, const DocWindow &w, int j) {
  Span r = {s.q_lo, s.q_hi};
  const int at = j - s.shift;
  if (M.causal) r.lo = max(r.lo, at);
  if (M.window) r.hi = min(r.hi, at + M.window);
  if (M.docs) {
    const Span d = attn_doc(M, w, j);
    r.lo = max(r.lo, d.lo), r.hi = min(r.hi, d.hi);
  }
  return r;
}

// Division by a number known to the host, of numbers below 2^31 (a division takes
// some 100 clocks, and a CTA begins with several before its first load): with
// 2^shift >= d, n / d = (high(mul n) + n) >> shift.
struct FastDiv {
  uint32_t d, mul, shift;
  __device__ __forceinline__ int div(int n) const { return (int)((__umulhi(mul, (uint32_t)n) + (uint32_t)n) >> shift); }
  // n becomes n / d; returns what is left over
  __device__ __forceinline__ int split(int &n) const {
    const int q = div(n), r = n - q * (int)d;
    n = q;
    return r;
  }
};

inline FastDiv fast_div(int64_t d) {
  FastDiv f = {(uint32_t)d, 0, 0};
  while ((int64_t(1) << f.shift) < d) ++f.shift;
  f.mul = (uint32_t)((((uint64_t)1 << 32) * (((uint64_t)1 << f.shift) - (uint64_t)d)) / (uint64_t)d + 1);
  return f;
}

// Heads and tiles.  The `group` query heads of one key head are cut into
// blocks of 2^pack heads, and a tile's rows are those heads of consecutive
// tokens: row r is token t0 + (r >> pack), head h0 + (r & mask).  Heads of a
// block share the tile's keys and its causal border, so the shared keys are
// loaded once and the tiles along the border stay small.
struct AttnShape {
  int32_t batch, q_heads, k_heads, head_blocks, pack;  // head_blocks: per key head
  int32_t dk, dv, kb, vb;                              // elements of a head; blocks of 64 of them
  int32_t k_steps, v_cols;                             // dk in steps of 16, dv rounded up to 16
  float scale, scale2;                                 // scale, and scale log2(e)
  int32_t group;                                       // query heads of a key head
  FastDiv by_batch, by_k_heads, by_blocks, by_all;     // by_all: head blocks of all key heads
};

// What a row tile sees: tiles [j0, j1) of 128 keys, of which those within
// [full_lo, full_hi) need no mask.
struct TileKeys {
  int32_t j0, j1, full_lo, full_hi;
  __device__ __forceinline__ bool has(int j) const { return j >= j0 && j < j1; }
  __device__ __forceinline__ bool masked(int j) const { return j * kAttnTile < full_lo || (j + 1) * kAttnTile > full_hi; }
};

// All lanes of a warp, with the same tile.
__device__ __forceinline__ TileKeys tile_keys(const AttnMask &M, const AttnSeq &s, const DocWindow &w, int t0, int tokens) {
  TileKeys k = {0, 0, 0, 0};
  const int a = max(t0, s.q_lo), b = min(t0 + tokens, s.q_hi);
  if (a >= b) return k;
  const Span first = keys_of(M, s, w, a), last = keys_of(M, s, w, b - 1);
  if (last.hi <= first.lo) return k;
  k.j0 = first.lo / kAttnTile, k.j1 = (last.hi + kAttnTile - 1) / kAttnTile;
  // (rows that see nothing are written as zeros whatever they sum up)
  k.full_lo = last.lo, k.full_hi = first.hi;
  return k;
}

// ---------------------------------------------------------------------------
// PTX wrappers

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float y;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(y) : "f"(a), "f"(b), "f"(c));
  return y;
}

__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap *map, uint32_t bar, int x, int y, int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

__device__ __forceinline__ void tma_store_4d(const CUtensorMap *map, uint32_t src, int x, int y, int z, int w) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(src), "r"(x), "r"(y), "r"(z), "r"(w)
               : "memory");
}

// 32 columns of this warp's 32 lanes of TMEM; the values may be used after
// tmem_wait of the same registers, which orders every use behind the wait.
__device__ __forceinline__ void tmem_get(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,"
      "%16,%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]),
                 "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]),
                 "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]),
                 "+r"(r[30]), "+r"(r[31])
               :
               : "memory");
}

__device__ __forceinline__ void tmem_get16(uint32_t taddr, uint32_t *r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_wait16(uint32_t *r) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]),
                 "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15])
               :
               : "memory");
}

// kCols (16, 32 or 64) columns, waited for.
template <int kCols>
__device__ __forceinline__ void tmem_read(uint32_t taddr, uint32_t (&r)[kCols]) {
  if constexpr (kCols == 16) {
    tmem_get16(taddr, r);
    tmem_wait16(r);
  } else {
#pragma unroll
    for (int c = 0; c < kCols; c += 32) tmem_get(taddr + c, r + c);
#pragma unroll
    for (int c = 0; c < kCols; c += 32) tmem_wait(r + c);
  }
}

__device__ __forceinline__ void tmem_put(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,"
      "%17,%18,%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]),
      "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]),
      "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
      : "memory");
}

__device__ __forceinline__ void tmem_put16(uint32_t taddr, const uint32_t *r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]),
      "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
      : "memory");
}

__device__ __forceinline__ void tmem_put8(uint32_t taddr, const uint32_t *r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr), "r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
               : "memory");
}

// kCols values as bf16 pairs in kCols / 2 columns.
template <int kCols>
__device__ __forceinline__ void tmem_write(uint32_t taddr, const uint32_t (&r)[kCols / 2]) {
  if constexpr (kCols == 16) tmem_put8(taddr, r);
  else if constexpr (kCols == 32) tmem_put16(taddr, r);
  else tmem_put(taddr, r);
}

__device__ __forceinline__ void tmem_put_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ void tmem_free(uint32_t tmem, uint32_t columns) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(columns) : "memory");
}

// kind::f16: bf16 operands, fp32 sums, M = 128, N = n; A K-major.
__host__ __device__ constexpr uint32_t attn_idesc(bool b_mn_major, int n) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((b_mn_major ? 1u : 0u) << 16) | ((uint32_t)(n >> 3) << 17) |
         ((uint32_t)(128 >> 4) << 24);
}

// One lane of a converged warp, the same one each time.
__device__ __forceinline__ bool elect_one() {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "elect.sync _|p, 0xffffffff;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok));
  return ok != 0;
}

// The low word of a descriptor whose high word is this one: stride 1024 bytes,
// version 1, 128-byte swizzle.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ uint32_t desc_low(uint32_t addr, uint32_t lbo) { return ((addr & 0x3FFFFu) >> 4) | ((lbo >> 4) << 16); }

__device__ __forceinline__ void mma_ss(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}

// A from TMEM: 128 lanes, a 32-bit column holds two consecutive K.
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "mov.b64 y, {%2, %5};\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"(accumulate), "n"(kDescHigh)
      : "memory");
}

// The products are issued by one thread, and each step of 16 keeps the tensor
// cores busy for 64 clocks or less: the steps are unrolled and their descriptors
// are one base and constants.

// D (+)= A B^T over `steps` (1..4) steps of 16 of one block of 64 columns, both
// K-major.
__device__ __forceinline__ void product_block(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t idesc, bool accumulate) {
  const uint32_t al = desc_low(a, 16), bl = desc_low(b, 16);
  if (steps == 4) {
#pragma unroll
    for (int k = 0; k < 4; ++k) mma_ss(d, al + 2 * k, bl + 2 * k, idesc, accumulate || k > 0);
  } else {
    for (int k = 0; k < steps; ++k) mma_ss(d, al + 2 * k, bl + 2 * k, idesc, accumulate || k > 0);
  }
}

// D = A B^T over `steps` steps of 16, at most kBlocks blocks of 64 columns: A of
// 128 rows, B of n rows with b_block bytes a block.
template <int kBlocks>
__device__ __forceinline__ void product_ss(uint32_t d, uint32_t a, uint32_t b, int steps, uint32_t b_block, int n) {
  const uint32_t idesc = attn_idesc(false, n);
#pragma unroll
  for (int c = 0; c < kBlocks; ++c)
    if (4 * c < steps) product_block(d, a + c * kAttnBlock, b + c * b_block, min(4, steps - 4 * c), idesc, c > 0);
}

// D (+)= A B over kSteps steps of K = 16, A in TMEM, B with K along its rows
// (MN-major) in blocks of 64 columns of b_block bytes, n columns in all.  A was
// written by kParts warps, each to the start of its own part_stride columns.
// [kFrom, kTo) of each part's steps: a part may be multiplied piece by piece.
template <int kSteps, int kParts, int kFrom = 0, int kTo = kSteps / kParts>
__device__ __forceinline__ void product_ts(uint32_t d, uint32_t a, uint32_t part_stride, uint32_t b, uint32_t b_block, int n,
                                           bool accumulate) {
  constexpr int kEach = kSteps / kParts;
  const uint32_t idesc = attn_idesc(true, n);
  const uint32_t bl = desc_low(b, b_block);
#pragma unroll
  for (int part = 0; part < kParts; ++part)
#pragma unroll
    for (int k = kFrom; k < kTo; ++k)
      mma_ts(d, a + part * part_stride + k * 8, bl + (part * kEach + k) * (2048 >> 4), idesc,
             accumulate || part > 0 || k > kFrom);
}

// ---------------------------------------------------------------------------
// waits

// Bounded waits of one CTA: the first to run out of time raises the flag and
// the status, and every other wait of the CTA gives up when it sees the flag.
struct AttnGuard {
  volatile int32_t *abort_flag;
  int32_t *status;
  uint64_t limit = kWaitNs;

  __device__ __forceinline__ bool wait(uint32_t bar, uint32_t parity) const {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t spin = 1;; ++spin) {
      if (mbar_try(bar, parity)) return true;
      if ((spin & 63u) == 0) {
        if (*abort_flag) return false;
        if (global_ns() - t0 > limit) {
          *abort_flag = 1;
          flag_status(status, GBO_STATUS_TIMEOUT);
          return false;
        }
      }
    }
  }
  // The same by all lanes of a warp, which come back together with one answer.
  __device__ __forceinline__ bool wait_warp(uint32_t bar, uint32_t parity) const {
    if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
    const uint64_t t0 = global_ns();
    for (uint32_t spin = 1;; ++spin) {
      if (__all_sync(0xffffffffu, mbar_try(bar, parity))) return true;
      if ((spin & 63u) == 0) {
        const bool late = global_ns() - t0 > limit;
        if (__any_sync(0xffffffffu, late || *abort_flag)) {
          if (!*abort_flag) {
            *abort_flag = 1;
            flag_status(status, GBO_STATUS_TIMEOUT);
          }
          return false;
        }
      }
    }
  }
  __device__ __forceinline__ bool aborted() const { return *abort_flag != 0; }
};

// The copies that a CTA's loading warp has started, noted in shared memory when it is
// done.  Where a wait of any warp ran out, they land (or run out of time, too) behind the
// CTA's last barrier, before the CTA ends and with it its shared memory: not sooner,
// because until there another warp's wait may run out.
struct Started {
  volatile int32_t *at;  // a bit for each barrier that takes one copy; numbers of copies into two rings

  __device__ __forceinline__ void note(int32_t single, int32_t first, int32_t second) const {
    at[0] = single, at[1] = first, at[2] = second;
  }
  __device__ __forceinline__ void settle_single(const AttnGuard &guard, uint32_t bars) const {
    for (int s = 0; s < 2; ++s)
      if (at[0] >> s & 1) (void)mbar_wait_ns(bars + 8 * s, 0, guard.limit);
  }
  // ring: 1 or 2
  __device__ __forceinline__ void settle_ring(const AttnGuard &guard, int ring, uint32_t bars, int stages) const {
    const int n = at[ring];
    for (int k = max(0, n - stages); k < n; ++k) (void)mbar_wait_ns(bars + 8 * (k % stages), (k / stages) & 1, guard.limit);
  }
};
constexpr int kNotes = 32;  // bytes: where TMEM starts, the flag, these

// Wait until every product this warp's elected lane has issued is done: nothing
// reads shared memory or writes TMEM when the CTA goes on to give them up.
__device__ __forceinline__ void drain_products(uint32_t bar) {
  if (elect_one()) mma_commit_one(bar);
  __syncwarp();
  (void)mbar_wait(bar, 0);
  __syncwarp();
}

__device__ __forceinline__ void zero_rows(uint32_t tile, int blocks, int rows, uint32_t block_bytes, int lo, int hi, int lane);

// A ring of tiles that one warp fills by TMA and that tensor cores read.  A tile
// with rows that reach nothing (of which one may hold anything, and 0 x NaN is
// not 0) is loaded through a barrier of its own and those rows are zeroed before
// the tile counts as loaded.
struct TileRing {
  uint32_t full, empty, base, bytes;  // barriers, first tile, bytes from tile to tile
  int stages, stage = 0, loads = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ TileRing(uint32_t full_, uint32_t empty_, uint32_t base_, uint32_t bytes_, int stages_)
      : full(full_), empty(empty_), base(base_), bytes(bytes_), stages(stages_) {}

  // All lanes of the warp; false when a wait ran out.
  __device__ __forceinline__ bool load(const AttnGuard &guard, const CUtensorMap *map, int blocks, uint32_t block_bytes, int head,
                                       int token, int batch, bool dirty, uint32_t raw, uint32_t &raw_phase, int rows, int lo,
                                       int hi, int lane) {
    if (!guard.wait_warp(empty + 8 * stage, phase ^ 1)) return false;
    const uint32_t bar = dirty ? raw : full + 8 * stage, tile = base + stage * bytes;
    if (elect_one()) {
      mbar_expect_tx(bar, (uint32_t)blocks * block_bytes);
      for (int c = 0; c < blocks; ++c) tma_load_4d(tile + c * block_bytes, map, bar, 64 * c, head, token, batch);
    }
    __syncwarp();
    if (dirty) {
      if (!guard.wait_warp(raw, raw_phase)) {
        (void)mbar_wait_ns(raw, raw_phase, guard.limit);
        return false;
      }
      raw_phase ^= 1;
      zero_rows(tile, blocks, rows, block_bytes, lo, hi, lane);
      if (elect_one()) mbar_arrive(full + 8 * stage);
      __syncwarp();
    }
    ++loads;
    if (++stage == stages) stage = 0, phase ^= 1;
    return true;
  }
};

// A reader's place in such a ring.
struct RingAt {
  int stage = 0;
  uint32_t phase = 0;
  __device__ __forceinline__ void next(int stages) {
    if (++stage == stages) stage = 0, phase ^= 1;
  }
};

// Zero the rows outside [lo, hi) of a tile of `rows` rows in `blocks` blocks of 64
// columns, by the lanes of one warp, for tensor cores that read it next.
__device__ __forceinline__ void zero_rows(uint32_t tile, int blocks, int rows, uint32_t block_bytes, int lo, int hi, int lane) {
  for (int b = 0; b < blocks; ++b)
    for (int c = lane; c < rows * 8; c += 32) {
      const int r = c >> 3;
      if (r < lo || r >= hi)
        asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(tile + (uint32_t)b * block_bytes + (uint32_t)c * 16u),
                     "r"(0)
                     : "memory");
    }
  fence_async_smem();
  __syncwarp();
}

// 32 values of row r as bf16 into columns c0 .. c0 + 31 of a tile of 128 rows in
// blocks of 64 columns with the 128-byte swizzle of the tensor maps.
__device__ __forceinline__ void put_tile_row(uint32_t tile, int r, int c0, const float *v) {
  const uint32_t line = tile + (uint32_t)(c0 >> 6) * kAttnBlock + (uint32_t)r * 128u;
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const uint32_t chunk = (uint32_t)(((c0 & 63) >> 3) + q);
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(line + ((chunk ^ (uint32_t)(r & 7)) << 4)),
                 "r"(pack_bf16(v[8 * q], v[8 * q + 1])), "r"(pack_bf16(v[8 * q + 2], v[8 * q + 3])),
                 "r"(pack_bf16(v[8 * q + 4], v[8 * q + 5])), "r"(pack_bf16(v[8 * q + 6], v[8 * q + 7]))
                 : "memory");
  }
}

// A block of 128 rows of zeros at the start of shared memory, for a tile that sees
// nothing: its output is stored from there, and no pipeline starts for it.  All
// threads of the CTA; orders tcgen05.alloc before what follows, too.
__device__ __forceinline__ void zero_block(uint8_t *smem) {
  for (int i = threadIdx.x; i < kAttnBlock / 16; i += blockDim.x) reinterpret_cast<uint4 *>(smem)[i] = make_uint4(0, 0, 0, 0);
  fence_async_smem();
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
}

// ---------------------------------------------------------------------------
// host

namespace {

int attn_fail(int code, const char *msg) { return report_error(code, msg); }

int attn_cuda(cudaError_t e) {
  char msg[200];
  snprintf(msg, sizeof msg, "attention kernels: %s", cudaGetErrorString(e));
  return report_error(GBO_ERR_CUDA, msg);
}

// The current device.  On a thread that has made no runtime call yet (autograd's, say)
// the driver has no context to encode maps in: there the device's own is made current.
// One that is current stays, the device's own or not.
int attn_device(int *dev, int *sm) {
  const int rc = require_device(dev, sm);
  if (rc != GBO_OK) return rc;
  using GetCurrentFn = CUresult (*)(CUcontext *);
  static const GetCurrentFn current = [] {
    void *p = nullptr;
    cudaDriverEntryPointQueryResult q;
    const bool ok = cudaGetDriverEntryPointByVersion("cuCtxGetCurrent", &p, 4000, cudaEnableDefault, &q) == cudaSuccess &&
                    q == cudaDriverEntryPointSuccess;
    return ok ? reinterpret_cast<GetCurrentFn>(p) : nullptr;
  }();
  CUcontext ctx = nullptr;
  if (current && current(&ctx) == CUDA_SUCCESS && ctx) return GBO_OK;
  const cudaError_t e = cudaSetDevice(*dev);
  return e == cudaSuccess ? GBO_OK : attn_cuda(e);
}

// A map over (dim, heads, tokens, batch) of bf16 heads, box 64 x heads x tokens.
bool heads_map(CUtensorMap *map, const void *base, int64_t dim, int64_t heads, int64_t tokens, int64_t batch,
               const int64_t stride[3], uint32_t box_heads, uint32_t box_tokens) {
  EncodeTiledFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)dim, (cuuint64_t)heads, (cuuint64_t)tokens, (cuuint64_t)batch};
  // (an axis of length one may have any stride; a map wants multiples of 16 bytes)
  auto bytes = [](int64_t n, int64_t s) { return (cuuint64_t)(n > 1 ? s * 2 : 16); };
  const cuuint64_t strides[3] = {bytes(heads, stride[2]), bytes(tokens, stride[1]), bytes(batch, stride[0])};
  const cuuint32_t box[4] = {64, box_heads, box_tokens, 1};
  const cuuint32_t estr[4] = {1, 1, 1, 1};
  return fn(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

int check_heads(const void *p, const int64_t stride[3], int64_t batch, int64_t tokens, int64_t heads) {
  if (!p) return attn_fail(GBO_ERR_INVALID_ARG, "NULL tensor pointer");
  if (reinterpret_cast<uintptr_t>(p) & 15) return attn_fail(GBO_ERR_INVALID_ARG, "tensors must be 16-byte aligned");
  const int64_t n[3] = {batch, tokens, heads};
  for (int i = 0; i < 3; ++i)
    if (n[i] > 1 && (stride[i] <= 0 || stride[i] % 8 || stride[i] >= (int64_t(1) << 39)))
      return attn_fail(GBO_ERR_INVALID_ARG, "strides must be positive multiples of 8 elements, below 2^39");
  return GBO_OK;
}

// (no pointer is followed: sizes are asked for before memory is there)
int check_attn_sizes(const gbo_attn_args *a) {
  if (!a) return attn_fail(GBO_ERR_INVALID_ARG, "args is NULL");
  if (a->dtype != GBO_BF16) return attn_fail(GBO_ERR_DTYPE, "queries, keys and values must be GBO_BF16");
  if (a->batch < 0 || a->sq < 0 || a->sk < 0 || a->sq > kAttnMaxLength || a->sk > kAttnMaxLength || a->batch > kAttnMaxLength)
    return attn_fail(GBO_ERR_SHAPE, "batch, sq and sk must be in 0..2^30");
  if (a->k_heads < 1 || a->q_heads < a->k_heads || a->q_heads % a->k_heads)
    return attn_fail(GBO_ERR_SHAPE, "q_heads must be a positive multiple of k_heads");
  if (a->q_heads > 65536) return attn_fail(GBO_ERR_SHAPE, "at most 65536 heads");
  if (a->dk < 8 || a->dk % 8 || a->dk > GBO_ATTN_MAX_DK || a->dv < 8 || a->dv % 8 || a->dv > GBO_ATTN_MAX_DV)
    return attn_fail(GBO_ERR_SHAPE, "dk must be a multiple of 8 in 8..192, dv one in 8..128");
  if (!(a->scale > 0.f) || !std::isfinite(a->scale)) return attn_fail(GBO_ERR_INVALID_ARG, "scale must be > 0 and finite");
  if (a->causal != 0 && a->causal != 1) return attn_fail(GBO_ERR_INVALID_ARG, "causal must be 0 or 1");
  if (a->window < 0 || (a->window > 0 && !a->causal))
    return attn_fail(GBO_ERR_INVALID_ARG, "window must be >= 0, and needs causal = 1");
  if (a->documents) {
    if (a->n_documents < 1) return attn_fail(GBO_ERR_INVALID_ARG, "documents without a number of documents");
    if (a->batch > 1 || a->sq != a->sk || a->q_lengths || a->k_lengths)
      return attn_fail(GBO_ERR_INVALID_ARG, "documents need one row of as many queries as keys, without lengths");
  } else if (a->n_documents != 0) {
    return attn_fail(GBO_ERR_INVALID_ARG, "n_documents without documents");
  }
  return GBO_OK;
}

int check_attn(const gbo_attn_args *a) {
  int rc = check_attn_sizes(a);
  if (rc != GBO_OK) return rc;
  if ((reinterpret_cast<uintptr_t>(a->q_lengths) | reinterpret_cast<uintptr_t>(a->k_lengths) |
       reinterpret_cast<uintptr_t>(a->documents)) & 3)
    return attn_fail(GBO_ERR_INVALID_ARG, "misaligned lengths or documents");
  if (a->batch == 0 || a->sq == 0) return GBO_OK;
  rc = check_heads(a->q, a->q_stride, a->batch, a->sq, a->q_heads);
  if (rc == GBO_OK && a->sk > 0) rc = check_heads(a->k, a->k_stride, a->batch, a->sk, a->k_heads);
  if (rc == GBO_OK && a->sk > 0) rc = check_heads(a->v, a->v_stride, a->batch, a->sk, a->k_heads);
  return rc;
}

void fill_shape(const gbo_attn_args *a, AttnShape *S, AttnMask *M, int most_pack) {
  const int group = a->q_heads / a->k_heads;
  S->batch = (int32_t)a->batch, S->q_heads = a->q_heads, S->k_heads = a->k_heads;
  S->pack = 0;
  while (S->pack < most_pack && group % (2 << S->pack) == 0) ++S->pack;
  S->head_blocks = group >> S->pack;
  S->group = group;
  S->by_batch = fast_div(std::max<int64_t>(a->batch, 1)), S->by_k_heads = fast_div(a->k_heads);
  S->by_blocks = fast_div(S->head_blocks), S->by_all = fast_div((int64_t)a->k_heads * S->head_blocks);
  S->dk = a->dk, S->dv = a->dv;
  S->kb = (a->dk + 63) / 64, S->vb = (a->dv + 63) / 64;
  S->k_steps = (a->dk + 15) / 16, S->v_cols = (a->dv + 15) / 16 * 16;
  S->scale = a->scale, S->scale2 = a->scale * 1.4426950408889634f;
  M->q_len = a->q_lengths, M->k_len = a->k_lengths, M->docs = a->documents;
  M->n_docs = a->n_documents, M->causal = a->causal;
  M->sq = (int32_t)a->sq, M->sk = (int32_t)a->sk;
  // a window that spans every key hides none
  M->window = a->window >= a->sk ? 0 : (int32_t)a->window;
}

// Which instance of a kernel template a head size takes: blocks of 64 elements.
inline int attn_config(const gbo_attn_args *a) { return a->dk <= 64 && a->dv <= 64 ? 0 : a->dk <= 128 ? 1 : 2; }

}  // namespace

}  // namespace gbo

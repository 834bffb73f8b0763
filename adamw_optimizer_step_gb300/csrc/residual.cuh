// The residual update between two blocks with the norms on either side of it:
// what its forward pass and its gradients share.
//
// One row of d elements, rho(t) = 1 / sqrt(mean t^2 + eps):
//   forward   u = o rho(o) post_gain (or o);  x' = x + scale gate(a) m u;
//             h = x' rho(x') pre_gain         (m: dropout's factors)
//   backward  from x', o, a, dx' and dh:
//             n = x' rho(x'), w = pre_gain dh:  g = dx' + rho(x') (w - n mean(w n))
//             dx = g,  dpre_gain = sum dh n,  dscale = sum g gate m u,
//             da = g scale m u gate'(a),  du = g scale gate m,
//             v = o rho(o), w = post_gain du:  do = rho(o) (w - v mean(w v)),
//             dpost_gain = sum du v           (sums over rows)
// Floor: HBM; every tensor is read or written once.  What bounds the forward pass
// (without gate and dropout) is HBM, the gradients issue slots.
//
// Three forms, by size:
//   ring   rows of 505 to 8192 elements, a CTA each, through shared memory
//   group  shorter rows, 4 to 64 threads each, eight elements a thread
//   wide   longer ones, and those of which no ring holds two, a CTA each
// Each comes with 16-byte chunks of eight consecutive elements a thread and, for
// rows that 16 bytes do not divide or tensors that do not start there, with single
// elements strided over the threads (coalesced).  Measured, bf16, against one form
// for all (a group of threads that loads straight into registers, the row in
// registers between its sums), us of the gradients and of the forward pass:
//   32768 x 2048, gate and dropout    556 -> 231     (no gate or dropout) 84
//   65600 x 1023, the same           2748 -> 764     903 -> 395
//   8192 x 8192 (wide), the same     1652 -> 703     (ring) 163 -> 140
//   4096 x 16384 (wide), the same    1020 -> 612     244 -> 198
// The sums over rows stay with the thread that has the columns (registers; wide: shared
// memory), one partial row a group is left at the end, and a second kernel adds them in
// a fixed order.
#pragma once

#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "device_common.cuh"
#include "dropout.cuh"
#include "gbo.h"
#include "internal.h"
#include "pairs.cuh"
#include "per_device.h"
#include "tc_common.cuh"

namespace gbo {

namespace {

constexpr int kMaxGroup = 512;
constexpr int kGroupThreads = 128;  // of the group form
constexpr int kMaxStages = 6;

struct ResParams {
  const void *x, *block, *gate, *dxo, *dh;  // backward: x is the updated stream
  void *xo, *h;                             // forward; backward: dx, dblock
  void *dgate;
  const float *scale, *post_gain, *pre_gain;
  float *part;          // backward: partial rows of dpre_gain, dpost_gain, dscale
  int32_t *status;
  DropArgs drop;
  int64_t n, d;
  int64_t xs, bs, as, xos, hs, dxos, dhs, das;  // row strides
  float eps, inv_d;
  int32_t group, post, pre, gate_mode, sigmoid, scale_mode;
  int32_t want_pre, want_post, want_scale;
  int32_t stages, stage_bytes;  // of the ring
};

enum { kGateNone = 0, kGateElement = 1, kGateRow = 2 };
enum { kScaleNone = 0, kScaleOne = 1, kScaleVector = 2 };

// Sums of up to three values over the threads of a group; every thread gets
// them.  `red`: shared, 3 x 16 floats for each of two turns.
template <int kCount>
__device__ __forceinline__ void group_sum(float (&v)[kCount], int group, int in_group, float *red, int &turn, int barrier) {
#pragma unroll
  for (int o = 1; o < 32; o *= 2)
    if (o < group) {
#pragma unroll
      for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
    }
  if (group <= 32) return;
  float *r = red + turn * 48;
  turn ^= 1;  // the other turn's values may still be read
  const int warp = in_group >> 5, lane = in_group & 31, warps = group >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kCount; ++i) r[i * 16 + warp] = v[i];
  asm volatile("bar.sync %0, %1;" ::"r"(barrier), "r"(group) : "memory");
#pragma unroll
  for (int i = 0; i < kCount; ++i) v[i] = (lane & 15) < warps ? r[i * 16 + (lane & 15)] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o /= 2)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// A thread's eight elements in part `it` of a row: kVec, consecutive ones; else
// `group` apart.
template <bool kVec>
__device__ __forceinline__ int column(int it, int e, int in_group, int group) {
  return kVec ? (it * group + in_group) * 8 + e : (it * 8 + e) * group + in_group;
}

// (d = 0: a row that is not there, zeros)
template <typename T, bool kVec>
__device__ __forceinline__ void load_part(const T *row, int d, int it, int in_group, int group, float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<true>(it, 0, in_group, group);
    if (c >= d) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = 0.f;
    } else if constexpr (sizeof(T) == 2) {
      const uint4 u = *reinterpret_cast<const uint4 *>(row + c);
      const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
      for (int h = 0; h < 4; ++h) v[2 * h] = __uint_as_float(w[h] << 16), v[2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
    } else {
      const float4 a = *reinterpret_cast<const float4 *>(row + c), b = *reinterpret_cast<const float4 *>(row + c + 4);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(it, e, in_group, group);
      v[e] = c < d ? (float)row[c] : 0.f;
    }
  }
}

template <typename T, bool kVec>
__device__ __forceinline__ void store_part(T *row, int d, int it, int in_group, int group, const float (&v)[8]) {
  if constexpr (kVec) {
    const int c = column<true>(it, 0, in_group, group);
    if (c < d) store8<T>(row + c, v, 8, true);
  } else {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int c = column<false>(it, e, in_group, group);
      if (c < d) st_elem(row, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, c, v[e]);
    }
  }
}

// v *= a column table (gains, scales), where there is one.
template <bool kVec>
__device__ __forceinline__ void times_table(const float *t, int d, int it, int in_group, int group, float (&v)[8]) {
  if (!t) return;
  float w[8];
  load_part<float, kVec>(t, d, it, in_group, group, w);
#pragma unroll
  for (int e = 0; e < 8; ++e) v[e] *= w[e];
}

// v *= dropout's factors of row `row`, part `it`.  Eight consecutive elements share a
// counter.  Where a thread's elements are single ones, the counters of the lanes'
// elements are shared out: the lanes of a group in a warp (u of them, 8 or more)
// cover, for each e, u consecutive elements, u / 8 counters and one more where the
// row starts inside one.  The words cross through `slots`, the warp's own.
constexpr int kDropSlots = 64;  // counters' words of a warp: u + 8 for each of 32 / u groups

template <bool kVec>
__device__ __forceinline__ void row_drop(const ResParams &P, uint64_t key, int64_t row, int it, int in_group, int group,
                                         float (&v)[8], uint4 *slots) {
  if constexpr (kVec) {
    const uint64_t at = (uint64_t)(row * P.d + column<true>(it, 0, in_group, group));  // (a multiple of 8)
    const uint4 w = philox(key, at >> 3, P.drop.offset);
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] *= drop_factor(w, e, P.drop.limit, P.drop.keep);
  } else {
    const int u = min(group, 32), l = in_group & (u - 1);
    uint4 *const mine = slots + (threadIdx.x >> 5) * kDropSlots + (threadIdx.x & 31) / u * (u + 8);
    const uint64_t at = (uint64_t)(row * P.d + column<false>(it, 0, in_group - l, group));
#pragma unroll 1
    for (int q = l; q < u + 8; q += u)  // counter q / 8 of elements e = q % 8
      mine[q] = philox(key, ((at + (uint64_t)(q & 7) * group) >> 3) + (q >> 3), P.drop.offset);
    __syncwarp();
    const int x = (int)(at & 7) + l;
    const uint32_t *w = reinterpret_cast<const uint32_t *>(mine + (x >> 3) * 8) + ((x & 7) >> 1);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t draw = (x & 1) ? w[4 * e] >> 16 : w[4 * e] & 0xffffu;
      v[e] *= draw >= P.drop.limit ? P.drop.keep : 0.f;
    }
    __syncwarp();
  }
}

// 1 / (1 + exp(-a)) and its slope, or a and 1.  From e = exp(-a) and q = 1 / (1 + e)
// the gate is q, the slope e q q: nothing cancels.  e is held below 2^126, so that
// nothing overflows: a gate below 2^-126 becomes that.  (NaN stays: the minimum of
// a NaN is NaN.)
__device__ __forceinline__ float2 gate_of2(float2 a, int sigmoid, float2 &slope) {
  if (!sigmoid) {
    slope = f2_of(1.f);
    return a;
  }
  a = f2_mul(a, f2_of(-1.4426950408889634f));
  float2 e, q;
  asm("min.NaN.f32 %0, %1, 0f42FC0000;" : "=f"(a.x) : "f"(a.x));  // 126
  asm("min.NaN.f32 %0, %1, 0f42FC0000;" : "=f"(a.y) : "f"(a.y));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(a.x));
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(a.y));
  q = f2_add(e, f2_of(1.f));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.x) : "f"(q.x));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(q.y) : "f"(q.y));
  slope = f2_mul(f2_mul(e, q), q);
  return q;
}
__device__ __forceinline__ float gate_of(float a, int sigmoid, float *slope = nullptr) {
  float2 s;
  const float q = gate_of2(f2_of(a), sigmoid, s).x;
  if (slope) *slope = s.x;
  return q;
}

// u times post_gain, dropout, the elements' gate and scale (forward).
template <typename BT, bool kVec>
__device__ __forceinline__ void block_factors(const ResParams &P, uint64_t key, int64_t row, int d, int it, int in_group, int group,
                                              float (&u)[8], uint4 *slots) {
  times_table<kVec>(P.post_gain, d, it, in_group, group, u);
  if (P.drop.limit) row_drop<kVec>(P, key, row, it, in_group, group, u, slots);
  if (P.gate_mode == kGateElement) {
    float a[8];
    load_part<BT, kVec>(static_cast<const BT *>(P.gate) + row * P.as, d, it, in_group, group, a);
#pragma unroll
    for (int e = 0; e < 8; ++e) u[e] *= gate_of(a[e], P.sigmoid);
  }
  if (P.scale_mode == kScaleVector) times_table<kVec>(P.scale, d, it, in_group, group, u);
}

// ---------------------------------------------------------------------------
// rows through shared memory

// Rows come through a ring of stages in shared memory: the input tensors of a row
// one behind the other, by bulk copies that thread 0 issues up to `stages` rows
// ahead.  Loads are then in flight all the time at no cost in registers, while a
// row's sums over its threads and its arithmetic take their time.  A stage is filled
// again behind the first join of the next row, which every thread reaches after its
// last read of the stage.  (A warp of
// its own for the copies takes registers from the others: 18 warps an SM have 96
// each, 16 have 128.)  The column tables stand behind the ring: from global memory
// each use would wait for L2 behind the row's joins.  What bounds these kernels
// then is instructions: arithmetic is two lanes at a time, factors of a column are
// multiplied into one table at the start.
enum { kInX = 0, kInBlock = 1, kInGate = 2, kInDxo = 3, kInDh = 4, kInputs = 5 };

struct RowRing {
  uint32_t base, full0, stage_bytes;
  int stages;
  volatile int32_t *late;  // some thread's wait has run out
  int32_t *status;
  uint64_t limit = kWaitNs;
  int stage = 0, to_fill = 0;
  uint32_t phase = 0;
  bool gave_up = false;  // this thread took a row that had not arrived

  static __device__ __forceinline__ void copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
  }
  // All threads: the stage of the next row has arrived.  A wait that runs out is
  // flagged, and every later one passes at once: the outputs are invalid.
  __device__ __forceinline__ uint32_t take() {
    const uint32_t bar = full0 + 8 * stage;
    if (!mbar_try(bar, phase) && (*late || !mbar_wait_ns(bar, phase, limit))) {
      gave_up = true;
      if (!*late) {
        *late = 1;
        flag_status(status, GBO_STATUS_TIMEOUT);
      }
    }
    return base + (uint32_t)stage * stage_bytes;
  }
  __device__ __forceinline__ void next() {
    if (++stage == stages) stage = 0, phase ^= 1;
  }
  // Thread 0, at the end, where it gave up (else it has waited for every row that it
  // asked for): the copies under way, of `filled` that were started, land (or run out of
  // time, too) before shared memory goes away.
  __device__ __forceinline__ void settle(int64_t filled) const {
    for (int64_t k = max((int64_t)0, filled - stages); k < filled; ++k)
      (void)mbar_wait_ns(full0 + 8 * (uint32_t)(k % stages), (uint32_t)(k / stages) & 1, limit);
  }
};

// Thread 0: a row's tensors from `src` (NULL: none), `by` bytes on from row to row.
// kOdd: rows start anywhere; their place is 16 bytes longer, and what is copied are
// the 16-byte blocks that a row touches.  What a block holds beside the row lies
// between the tensor's first and last element, but for the first row's start and the
// last row's end: those elements are stored one by one.
template <bool kOdd>
struct RowFeed {
  const uint8_t *src[kInputs];
  int64_t by[kInputs];
  uint32_t bytes[kInputs];
  int64_t row, step, n;  // the next row, of n

  static __host__ __device__ __forceinline__ uint32_t place(uint32_t bytes) { return kOdd ? (bytes + 15) / 16 * 16 + 16 : bytes; }

  static __device__ __forceinline__ void by_hand(uint32_t dst, const uint8_t *p, uint32_t bytes) {
    for (uint32_t b = 0; b < bytes; b += 2)
      asm volatile("st.shared.u16 [%0], %1;" ::"r"(dst + b), "h"(*reinterpret_cast<const uint16_t *>(p + b)) : "memory");
  }
  // Nothing more where this thread gave up: the stage's barrier and place may still be a
  // copy's.  (Where others alone did, the rows that this one has taken have landed.)
  __device__ __forceinline__ void fill(RowRing &r) {
    if (row >= n || r.gave_up) return;
    const uint32_t bar = r.full0 + 8 * r.to_fill;
    uint32_t dst = r.base + (uint32_t)r.to_fill * r.stage_bytes;
    if constexpr (kOdd) {
      const bool first = row == 0, last = row == n - 1;
      const uint8_t *lo[kInputs], *hi[kInputs];
      uint32_t total = 0, at = dst;
#pragma unroll
      for (int i = 0; i < kInputs; ++i)
        if (src[i]) {
          const uint8_t *const p = src[i], *const end = p + bytes[i];
          const uint32_t head = -(uint32_t)reinterpret_cast<uintptr_t>(p) & 15, tail = (uint32_t)reinterpret_cast<uintptr_t>(end) & 15;
          const uint32_t before = (16 - head) & 15;  // bytes of p's block before it
          lo[i] = first ? p + head : p - before;
          hi[i] = last ? end - tail : end + ((16 - tail) & 15);
          if (first) by_hand(at + before, p, head);
          if (last) by_hand(at + before + (bytes[i] - tail), end - tail, tail);
          total += (uint32_t)(hi[i] - lo[i]);
          at += place(bytes[i]);
        }
      if (first | last) fence_async_smem();
      mbar_expect_tx(bar, total);
#pragma unroll
      for (int i = 0; i < kInputs; ++i)
        if (src[i]) {
          const uint32_t before = (uint32_t)reinterpret_cast<uintptr_t>(src[i]) & 15;
          RowRing::copy(dst + before + (int32_t)(lo[i] - src[i]), lo[i], (uint32_t)(hi[i] - lo[i]), bar);
          dst += place(bytes[i]);
        }
    } else {
      mbar_expect_tx(bar, r.stage_bytes);
#pragma unroll
      for (int i = 0; i < kInputs; ++i)
        if (src[i]) {
          RowRing::copy(dst, src[i], bytes[i], bar);
          dst += bytes[i];
        }
    }
#pragma unroll
    for (int i = 0; i < kInputs; ++i)
      if (src[i]) src[i] += by[i];
    row += step;
    if (++r.to_fill == r.stages) r.to_fill = 0;
  }
};

// Eight elements at a shared-memory address.
template <typename T>
__device__ __forceinline__ void lds8(uint32_t at, float2 *v) {
  uint32_t w[4];
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
  if constexpr (sizeof(T) == 2) {
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
  } else {
    v[0] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[1] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3])
                 : "r"(at + 16)
                 : "memory");
    v[2] = make_float2(__uint_as_float(w[0]), __uint_as_float(w[1]));
    v[3] = make_float2(__uint_as_float(w[2]), __uint_as_float(w[3]));
  }
}

template <typename T>
__device__ __forceinline__ void stg8(T *p, const float2 *v) {
  if constexpr (sizeof(T) == 2) {
    *reinterpret_cast<uint4 *>(p) = make_uint4(pack_bf16(v[0].x, v[0].y), pack_bf16(v[1].x, v[1].y), pack_bf16(v[2].x, v[2].y),
                                               pack_bf16(v[3].x, v[3].y));
  } else {
    float4 *f = reinterpret_cast<float4 *>(p);
    f[0] = make_float4(v[0].x, v[0].y, v[1].x, v[1].y), f[1] = make_float4(v[2].x, v[2].y, v[3].x, v[3].y);
  }
}

// Dropout's factors of eight elements, times v.
__device__ __forceinline__ void drop8(const DropArgs &D, uint64_t key, uint64_t element, float2 *v) {
  const uint4 w = philox(key, element >> 3, D.offset);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = f2_mul(v[k], make_float2(drop_factor(w, 2 * k, D.limit, D.keep), drop_factor(w, 2 * k + 1, D.limit, D.keep)));
}

// A thread's part `it` of a row in a ring's stage and in memory.
template <bool kOdd>
struct RowPart {
  int d, tid, threads;

  __device__ __forceinline__ int chunk(int it) const { return it * threads + tid; }
  __device__ __forceinline__ bool here(int it) const { return kOdd || chunk(it) * 8 < d; }
  __device__ __forceinline__ int column(int it, int e) const { return gbo::column<!kOdd>(it, e, tid, threads); }
  // `at`: the row's start
  template <typename T>
  __device__ __forceinline__ void get(uint32_t at, int it, float2 *v) const {
    if constexpr (!kOdd) {
      lds8<T>(at + chunk(it) * 8 * sizeof(T), v);
    } else {
      float w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column(it, e);
        w[e] = 0.f;
        if (c < d) {
          if constexpr (sizeof(T) == 2) {
            uint16_t x;
            asm volatile("ld.shared.u16 %0, [%1];" : "=h"(x) : "r"(at + c * 2) : "memory");
            w[e] = __uint_as_float((uint32_t)x << 16);
          } else {
            asm volatile("ld.shared.f32 %0, [%1];" : "=f"(w[e]) : "r"(at + c * 4) : "memory");
          }
        }
      }
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = make_float2(w[2 * k], w[2 * k + 1]);
    }
  }
  template <typename T>
  __device__ __forceinline__ void put(T *row, int it, const float2 *v) const {
    if constexpr (!kOdd) {
      stg8(row + chunk(it) * 8, v);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column(it, e);
        if (c < d) st_elem(row, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, c, (e & 1) ? v[e / 2].y : v[e / 2].x);
      }
    }
  }
  __device__ __forceinline__ void drop(const ResParams &P, uint64_t key, int64_t row, int it, float2 *v, uint4 *slots) const {
    if constexpr (!kOdd) {
      drop8(P.drop, key, (uint64_t)(row * P.d + chunk(it) * 8), v);
    } else {
      float w[8] = {v[0].x, v[0].y, v[1].x, v[1].y, v[2].x, v[2].y, v[3].x, v[3].y};
      row_drop<false>(P, key, row, it, tid, threads, w, slots);
#pragma unroll
      for (int k = 0; k < 4; ++k) v[k] = make_float2(w[2 * k], w[2 * k + 1]);
    }
  }
};

// Where a row of a tensor starts in its place of a stage.
template <bool kOdd, typename T>
__device__ __forceinline__ uint32_t row_start(uint32_t place, const T *p, int64_t row, int64_t stride) {
  return kOdd ? place + ((uint32_t)reinterpret_cast<uintptr_t>(p + row * stride) & 15) : place;
}

// A table's values of chunk c: first halves of all chunks, then second halves, so
// that a warp's 16-byte reads meet in no bank.  Each thread reads back what it
// wrote.
struct ColumnTable {
  uint32_t at, half;
  __device__ __forceinline__ void put(int c, const float *v) const {
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + 16 * c), "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3])
                 : "memory");
    asm volatile("st.shared.v4.f32 [%0], {%1, %2, %3, %4};" ::"r"(at + half + 16 * c), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7])
                 : "memory");
  }
  __device__ __forceinline__ void get(int c, float2 *v) const {
    float w[8];
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(w[0]), "=f"(w[1]), "=f"(w[2]), "=f"(w[3]) : "r"(at + 16 * c) : "memory");
    asm volatile("ld.shared.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(w[4]), "=f"(w[5]), "=f"(w[6]), "=f"(w[7])
                 : "r"(at + half + 16 * c)
                 : "memory");
#pragma unroll
    for (int k = 0; k < 4; ++k) v[k] = make_float2(w[2 * k], w[2 * k + 1]);
  }
};

__device__ __forceinline__ float table_at(const float *t, int64_t c) { return t ? t[c] : 1.f; }

// Sums of up to three values over a CTA of 2 to 16 warps.
template <int kCount>
__device__ __forceinline__ void cta_sum(float (&v)[kCount], float *red, int &turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
  float *r = red + turn;
  turn ^= 48;  // the other turn's values may still be read
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, warps = blockDim.x >> 5;
  if (lane == 0)
#pragma unroll
    for (int i = 0; i < kCount; ++i) r[i * 16 + warp] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kCount; ++i) v[i] = (lane & 15) < warps ? r[i * 16 + (lane & 15)] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o >>= 1)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
}

// Four sums over a warp in nine steps' work: each of the first two steps halves the
// values that a lane carries on.  Lanes 8 i to 8 i + 7 get sum i, in x.
__device__ __forceinline__ float4 warp_sum4(float4 v, int lane) {
  const bool hi = lane & 16, up = lane & 8;
  float a = hi ? v.z : v.x, b = hi ? v.w : v.y;
  a += __shfl_xor_sync(0xffffffffu, hi ? v.x : v.z, 16);
  b += __shfl_xor_sync(0xffffffffu, hi ? v.y : v.w, 16);
  float c = up ? b : a;
  c += __shfl_xor_sync(0xffffffffu, up ? a : b, 8);
#pragma unroll
  for (int o = 4; o > 0; o >>= 1) c += __shfl_xor_sync(0xffffffffu, c, o);
  return make_float4(c, 0.f, 0.f, 0.f);
}

// The warps' sums (2 to 16, zeros behind them) added up by every thread.
__device__ __forceinline__ float4 cta_join(const float4 *red, int warps) {
  float2 a = f2_of(0.f), b = f2_of(0.f);
  auto four = [&](int w) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float4 v = red[w + i];
      a = f2_add(a, make_float2(v.x, v.y)), b = f2_add(b, make_float2(v.z, v.w));
    }
  };
  four(0);
  if (warps > 4) four(4);
  if (warps > 8) four(8), four(12);
  return make_float4(a.x, a.y, b.x, b.y);
}

// ---------------------------------------------------------------------------
// host

int res_fail(int code, const char *msg) { return report_error(code, msg); }

int res_cuda(cudaError_t e) {
  char msg[200];
  snprintf(msg, sizeof msg, "residual kernels: %s", cudaGetErrorString(e));
  return report_error(GBO_ERR_CUDA, msg);
}

int size_of(int32_t dtype) { return dtype == GBO_BF16 ? 2 : 4; }

int check_rows(const void *p, int64_t stride, const gbo_residual_args *a, int64_t width, int32_t dtype) {
  if (!p) return res_fail(GBO_ERR_INVALID_ARG, "NULL tensor pointer");
  if (reinterpret_cast<uintptr_t>(p) % size_of(dtype)) return res_fail(GBO_ERR_INVALID_ARG, "misaligned tensor pointer");
  if (a->n > 1 && (stride < width || stride > (int64_t(1) << 40)))
    return res_fail(GBO_ERR_INVALID_ARG, "a row stride must be at least the row's length, and below 2^40");
  return GBO_OK;
}

int check_residual(const gbo_residual_args *a, DropArgs *drop) {
  if (!a) return res_fail(GBO_ERR_INVALID_ARG, "args is NULL");
  if (a->x_dtype != GBO_F32 && a->x_dtype != GBO_BF16) return res_fail(GBO_ERR_DTYPE, "x_dtype must be GBO_F32 or GBO_BF16");
  if (a->block_dtype != GBO_BF16 && !(a->block_dtype == GBO_F32 && a->x_dtype == GBO_F32))
    return res_fail(GBO_ERR_DTYPE, "block_dtype must be GBO_BF16, or GBO_F32 with x in GBO_F32");
  if (a->n < 0 || a->n > (int64_t(1) << 40)) return res_fail(GBO_ERR_SHAPE, "n must be in 0..2^40");
  if (a->d < 1 || a->d > GBO_RESIDUAL_MAX_D) return res_fail(GBO_ERR_SHAPE, "d must be in 1..16384");
  if (!(a->eps >= 0.f) || !std::isfinite(a->eps)) return res_fail(GBO_ERR_INVALID_ARG, "eps must be >= 0 and finite");
  if ((a->post_norm | a->pre_norm) & ~1) return res_fail(GBO_ERR_INVALID_ARG, "post_norm and pre_norm must be 0 or 1");
  if (a->gate_mode < GBO_GATE_NONE || a->gate_mode > GBO_GATE_ROW || (a->gate_sigmoid & ~1))
    return res_fail(GBO_ERR_INVALID_ARG, "unknown gate");
  if (a->scale_mode < GBO_SCALE_NONE || a->scale_mode > GBO_SCALE_VECTOR) return res_fail(GBO_ERR_INVALID_ARG, "unknown kind of scale");
  if (!drop_of(a->dropout, drop)) return res_fail(GBO_ERR_INVALID_ARG, "dropout must be in 0 <= p < 1 - 2^-17");
  drop->seed = a->seed, drop->offset = a->offset, drop->dev_seed = a->dev_seed;
  if (reinterpret_cast<uintptr_t>(a->dev_seed) & 7) return res_fail(GBO_ERR_INVALID_ARG, "misaligned dev_seed");
  if ((a->gate_mode != GBO_GATE_NONE) != (a->gate != nullptr) && a->n > 0)
    return res_fail(GBO_ERR_INVALID_ARG, "a gate and its kind go together");
  if ((a->scale_mode != GBO_SCALE_NONE) != (a->scale != nullptr)) return res_fail(GBO_ERR_INVALID_ARG, "a scale and its kind go together");
  if ((a->post_gain && !a->post_norm) || (a->pre_gain && !a->pre_norm)) return res_fail(GBO_ERR_INVALID_ARG, "a gain without its norm");
  if ((reinterpret_cast<uintptr_t>(a->scale) | reinterpret_cast<uintptr_t>(a->post_gain) |
       reinterpret_cast<uintptr_t>(a->pre_gain)) & 3)
    return res_fail(GBO_ERR_INVALID_ARG, "misaligned gain or scale");
  if (!a->has_block) {
    if (a->block || a->gate_mode || a->scale_mode || a->post_norm || drop->limit)
      return res_fail(GBO_ERR_INVALID_ARG, "a norm, gate, scale or dropout of a block's output without has_block");
    if (!a->pre_norm) return res_fail(GBO_ERR_INVALID_ARG, "neither a block's output nor a norm: nothing to do");
  }
  if (a->n == 0) return GBO_OK;
  int rc = GBO_OK;
  if (a->has_block) rc = check_rows(a->block, a->block_stride, a, a->d, a->block_dtype);
  if (rc == GBO_OK && a->gate_mode == GBO_GATE_ELEMENT) rc = check_rows(a->gate, a->gate_stride, a, a->d, a->block_dtype);
  if (rc == GBO_OK && a->gate_mode == GBO_GATE_ROW) rc = check_rows(a->gate, a->gate_stride, a, 1, a->block_dtype);
  return rc;
}

// Threads to a row, chunks to a thread, the ring.
enum { kFormGroup = 0, kFormRing = 1, kFormWide = 2 };
struct ResCut {
  int32_t form, group, iter, threads, blocks, stages, smem;
};

constexpr int kSmemMost = 220 * 1024;  // of an SM's shared memory, for rings and tables

// Ring: a row goes to as many threads as it has chunks of eight elements, up to 512;
// to half as many in the forward pass (what a row costs beside its elements is half
// as much then); 512 threads an SM.  Gradients of single elements, two chunks a thread,
// spill (8194 x 8190: 1303 us, the wide form 651): those rows take the wide form, shorter
// ones the ring (65600 x 1023: 764 us, wide 2544).
// `row_bytes`: of a row's inputs, in their places (0 where there are no rows: their
// pointers may be NULL).
ResCut cut_of(int64_t n, int64_t d, int sm, bool back, bool vec, int64_t row_bytes) {
  ResCut c;
  memset(&c, 0, sizeof c);
  row_bytes = std::max<int64_t>(row_bytes, 16);
  const int64_t chunks = (d + 7) / 8;
  auto blocks = [&](int per_sm, int64_t rows) {
    c.blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>((int64_t)sm * per_sm, (n + rows - 1) / rows));
  };
  if (chunks >= 64 && chunks <= 2 * kMaxGroup && (vec || !back || chunks <= kMaxGroup)) {
    c.group = 64;
    while (c.group < kMaxGroup && (int64_t)c.group * (back ? 1 : 2) < chunks) c.group *= 2;
    c.iter = (int32_t)((chunks + c.group - 1) / c.group);
    c.threads = c.group;
    const int64_t tables = 2 * 4 * (vec ? d : (int64_t)c.threads * c.iter * 8);
    for (int per_sm = std::max(1, 512 / c.threads); per_sm > 0; --per_sm) {
      const int64_t slots = vec ? 0 : kMaxGroup / 32 * kDropSlots * 16, room = kSmemMost / per_sm - tables - slots;
      if (room < 2 * row_bytes) continue;
      c.form = kFormRing;
      c.stages = (int32_t)std::min<int64_t>(kMaxStages, room / row_bytes);
      c.smem = (int32_t)(c.stages * row_bytes + tables);
      blocks(per_sm, 1);
      return c;
    }
  }
  if (chunks >= 64) {
    // x' in 32 bits; gradients: w, and two sums over rows
    c.form = kFormWide;
    c.group = c.threads = kMaxGroup;
    c.iter = (int32_t)((chunks + kMaxGroup - 1) / kMaxGroup);
    c.smem = c.iter * kMaxGroup * 8 * 4 * (back ? 3 : 1);
    blocks(back ? std::max(1, std::min(2, kSmemMost / (c.smem + 16384))) : 2, 1);
    return c;
  }
  c.group = vec ? 4 : 8;  // (single elements: dropout's counters are shared out by eight)
  while (c.group < chunks) c.group *= 2;
  c.iter = 1;
  c.threads = kGroupThreads;
  // gradients: as many blocks as leave the partial rows few; each goes over many rows
  blocks((back ? 512 : 1024) / c.threads, c.threads / c.group);
  return c;
}

// Partial rows of a backward call.
int64_t parts_of(const ResCut &c) { return (int64_t)c.blocks * (c.threads / std::max(c.group, 32)); }

// The most that any cut of these sizes leaves: a ring that has room for all of its
// CTAs, or none.
int64_t most_parts(int64_t n, int64_t d, int sm) {
  int64_t most = 0;
  for (bool vec : {false, true})
    for (int64_t row_bytes : {int64_t(1), int64_t(kSmemMost)})
      most = std::max(most, parts_of(cut_of(n, d, sm, true, vec, row_bytes)));
  return most;
}

using ResLaunch = cudaError_t (*)(ResParams &, const ResCut &, int, cudaStream_t);

template <auto kKernel>
cudaError_t launch_res(ResParams &P, const ResCut &c, int dev, cudaStream_t st) {
  P.group = c.group, P.stages = c.stages;
  if (c.smem) {
    static PerDevice<cudaError_t> limit;
    const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
      cudaFuncAttributes own;
      e = cudaFuncGetAttributes(&own, kKernel);
      const int most = std::min(kSmemMost, 232448 - (int)own.sharedSizeBytes);
      if (e == cudaSuccess) e = cudaFuncSetAttribute(kKernel, cudaFuncAttributeMaxDynamicSharedMemorySize, most);
    });
    if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  }
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), kKernel, dim3(c.blocks), dim3(c.threads), c.smem, st, 1, P);
}

bool vec_ok(const void *p, int64_t stride, int64_t n) {
  return !p || ((reinterpret_cast<uintptr_t>(p) & 15) == 0 && (n <= 1 || stride % 8 == 0));
}

void fill_res(const gbo_residual_args *a, const DropArgs &drop, ResParams *P) {
  memset(P, 0, sizeof *P);
  P->x = a->x, P->block = a->block, P->gate = a->gate;
  P->scale = a->scale, P->post_gain = a->post_gain, P->pre_gain = a->pre_gain;
  P->drop = drop;
  P->n = a->n, P->d = a->d, P->xs = a->x_stride, P->bs = a->block_stride, P->as = a->gate_stride;
  P->eps = a->eps, P->inv_d = 1.f / (float)a->d;
  P->post = a->post_norm, P->pre = a->pre_norm, P->gate_mode = a->gate_mode, P->sigmoid = a->gate_sigmoid && a->gate_mode;
  P->scale_mode = a->scale_mode;
}

// A row's inputs in their places of a ring's stage.
int64_t row_bytes(const ResParams &P, int32_t xt, int32_t bt, bool vec, bool back) {
  const int64_t sizes[kInputs] = {!back || P.pre ? size_of(xt) : 0, P.block ? size_of(bt) : 0,
                                  P.gate_mode == kGateElement ? size_of(bt) : 0, P.dxo ? size_of(xt) : 0, back && P.pre ? size_of(bt) : 0};
  int64_t sum = 0;
  for (int64_t size : sizes)
    if (size) sum += vec ? RowFeed<false>::place((uint32_t)(P.d * size)) : RowFeed<true>::place((uint32_t)(P.d * size));
  return sum;
}

bool inputs_vec(const gbo_residual_args *a) {
  return a->d % 8 == 0 && vec_ok(a->x, a->x_stride, a->n) && vec_ok(a->block, a->block_stride, a->n) &&
         (a->gate_mode != GBO_GATE_ELEMENT || vec_ok(a->gate, a->gate_stride, a->n)) && vec_ok(a->post_gain, 0, 0) &&
         vec_ok(a->pre_gain, 0, 0) && (a->scale_mode != GBO_SCALE_VECTOR || vec_ok(a->scale, 0, 0));
}

int32_t parts_wanted(const gbo_residual_grads *g) { return (g->dpre_gain != nullptr) + (g->dpost_gain != nullptr) + (g->dscale != nullptr); }

}  // namespace
}  // namespace gbo

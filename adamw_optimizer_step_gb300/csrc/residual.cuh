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
// Bound: HBM; every tensor is read or written once, a row stays in registers
// from its loads to its stores.
//
// A group of 4 to 512 threads takes a row, eight consecutive elements to a
// thread and chunk (16-byte loads); rows that 16 bytes do not divide take the
// elements strided over the threads instead (coalesced, one element each).  The
// sums of a row cross the group's warps through shared memory: two joins a row,
// each of all sums known by then.  The sums over rows stay in a thread's
// registers over all rows of its group (a thread keeps its columns), one partial
// row a group is left at the end, and a second kernel adds them in a fixed order.
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
#include "per_device.h"
#include "tc_common.cuh"

namespace gbo {

namespace {

constexpr int kMaxGroup = 512;
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
  for (int i = 0; i < kCount; ++i) {
    float t = 0.f;
    for (int w = 0; w < warps; ++w) t += r[i * 16 + w];
    v[i] = t;
  }
}

// A thread's elements of a row: kVec, kIter chunks of eight consecutive ones;
// else 8 kIter single ones, `group` apart.
template <bool kVec>
__device__ __forceinline__ int column(int it, int e, int in_group, int group) {
  return kVec ? (it * group + in_group) * 8 + e : (it * 8 + e) * group + in_group;
}

// (d = 0: a row that is not there, zeros)
template <typename T, int kIter, bool kVec>
__device__ __forceinline__ void row_load(const T *row, int d, int in_group, int group, float (&v)[kIter * 8]) {
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if constexpr (kVec) {
      const int c = column<true>(it, 0, in_group, group);
      if (c < d) {
        if constexpr (sizeof(T) == 2) {
          const uint4 u = *reinterpret_cast<const uint4 *>(row + c);
          const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
          for (int h = 0; h < 4; ++h) {
            v[it * 8 + 2 * h] = __uint_as_float(w[h] << 16);
            v[it * 8 + 2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
          }
        } else {
          const float4 a = *reinterpret_cast<const float4 *>(row + c), b = *reinterpret_cast<const float4 *>(row + c + 4);
          v[it * 8] = a.x, v[it * 8 + 1] = a.y, v[it * 8 + 2] = a.z, v[it * 8 + 3] = a.w;
          v[it * 8 + 4] = b.x, v[it * 8 + 5] = b.y, v[it * 8 + 6] = b.z, v[it * 8 + 7] = b.w;
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[it * 8 + e] = 0.f;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(it, e, in_group, group);
        v[it * 8 + e] = c < d ? (float)row[c] : 0.f;
      }
    }
  }
}

template <typename T, int kIter, bool kVec>
__device__ __forceinline__ void row_store(T *row, int d, int in_group, int group, const float (&v)[kIter * 8]) {
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if constexpr (kVec) {
      const int c = column<true>(it, 0, in_group, group);
      if (c < d) store8<T>(row + c, v + it * 8, 8, true);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(it, e, in_group, group);
        if (c < d) st_elem(row, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, c, v[it * 8 + e]);
      }
    }
  }
}

// A column table (a gain, the scale).  Kernels with a ring keep it in shared memory:
// a thread loads its own columns there once and reads them back (no other thread
// does).  From global memory each use would wait for L2, behind the row's joins.
template <int kIter, bool kVec, bool kRing>
struct Table {
  const float *at;  // NULL: none
  int d;

  __device__ __forceinline__ Table(const float *t, int d_, uint8_t *&smem, int in_group, int group) : at(t), d(d_) {
    if constexpr (kRing) {
      if (!t) return;
      float *keep = reinterpret_cast<float *>(smem);
      smem += (int64_t)d * 4;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int c = column<true>(it, 0, in_group, group);
        if (c < d) {
          float4 *to = reinterpret_cast<float4 *>(keep);
          const float4 *from = reinterpret_cast<const float4 *>(t + c);
          to[c / 8] = from[0], to[d / 8 + c / 8] = from[1];  // first halves, then second: no bank twice
        }
      }
      at = keep;
    }
  }
  __device__ __forceinline__ void load(int in_group, int group, float (&w)[kIter * 8]) const {
    if constexpr (kRing) {
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        const int c = column<true>(it, 0, in_group, group);
        if (c < d) {
          const float4 a = reinterpret_cast<const float4 *>(at)[c / 8], b = reinterpret_cast<const float4 *>(at)[d / 8 + c / 8];
          w[it * 8] = a.x, w[it * 8 + 1] = a.y, w[it * 8 + 2] = a.z, w[it * 8 + 3] = a.w;
          w[it * 8 + 4] = b.x, w[it * 8 + 5] = b.y, w[it * 8 + 6] = b.z, w[it * 8 + 7] = b.w;
        } else {
#pragma unroll
          for (int e = 0; e < 8; ++e) w[it * 8 + e] = 0.f;
        }
      }
    } else {
      row_load<float, kIter, kVec>(at, d, in_group, group, w);
    }
  }
  __device__ __forceinline__ void times(int in_group, int group, float (&v)[kIter * 8]) const {
    if (!at) return;
    float w[kIter * 8];
    load(in_group, group, w);
#pragma unroll
    for (int e = 0; e < kIter * 8; ++e) v[e] *= w[e];
  }
};

// u *= dropout's factors of row `row`.
template <int kIter, bool kVec>
__device__ __forceinline__ void row_drop(const ResParams &P, uint64_t key, int64_t row, int in_group, int group,
                                         float (&u)[kIter * 8]) {
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if constexpr (kVec) {
      const uint64_t at = (uint64_t)(row * P.d + column<true>(it, 0, in_group, group));  // (a multiple of 8)
      const uint4 w = philox(key, at >> 3, P.drop.offset);
#pragma unroll
      for (int e = 0; e < 8; ++e) u[it * 8 + e] *= drop_factor(w, e, P.drop.limit, P.drop.keep);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = column<false>(it, e, in_group, group);
        if (c < P.d) u[it * 8 + e] *= drop_one(P.drop, key, (uint64_t)(row * P.d + c));
      }
    }
  }
}

// 1 / (1 + exp(-a)) and its slope, or a and 1.  The slope is f f exp(-a) for
// positive a, where 1 - f would cancel, and f (1 - f) for others, where exp(-a)
// may be infinite.
__device__ __forceinline__ float gate_of(float a, int sigmoid, float *slope = nullptr) {
  if (!sigmoid) {
    if (slope) *slope = 1.f;
    return a;
  }
  const float e = __expf(-a), f = __fdividef(1.f, 1.f + e);
  if (slope) *slope = a > 0.f ? f * f * e : f * (1.f - f);
  return f;
}

// Rows on their way into shared memory, one a stage: the input tensors of a row
// one behind the other, by bulk copies that thread 0 issues `stages` rows ahead.
// Loads are then in flight all the time at no cost in registers, while a row's
// two sums over its threads and its arithmetic take their time.
template <bool kRing>
struct RowRing {
  const ResParams &P;
  uint8_t *base;
  uint32_t bar0;
  volatile int32_t *late;
  int stage = 0;
  uint32_t phase = 0;

  __device__ __forceinline__ RowRing(const ResParams &p, uint8_t *b, uint32_t bars, volatile int32_t *l)
      : P(p), base(b), bar0(bars), late(l) {}

  static __device__ __forceinline__ void copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
  }
  // Thread 0: start the copies of row `row` into stage s.
  template <typename XT, typename BT>
  __device__ __forceinline__ void fill(int s, int64_t row, bool back) {
    const uint32_t bar = bar0 + 8 * s, xb = (uint32_t)P.d * sizeof(XT), bb = (uint32_t)P.d * sizeof(BT);
    uint32_t dst = smem_u32(base) + (uint32_t)s * P.stage_bytes;
    mbar_expect_tx(bar, (uint32_t)P.stage_bytes);
    auto put = [&](const void *src, int64_t stride, uint32_t bytes) {
      copy(dst, static_cast<const uint8_t *>(src) + row * stride * (bytes / (uint32_t)P.d), bytes, bar);
      dst += bytes;
    };
    if (!back || P.pre) put(P.x, P.xs, xb);
    if (P.block) put(P.block, P.bs, bb);
    if (P.gate_mode == kGateElement) put(P.gate, P.as, bb);
    if (back && P.dxo) put(P.dxo, P.dxos, xb);
    if (back && P.pre) put(P.dh, P.dhs, bb);
  }
  // All threads: the stage of the next row has arrived (or, flagged, has not).
  __device__ __forceinline__ const uint8_t *wait() {
    if (!*late && !mbar_wait(bar0 + 8 * stage, phase)) {
      *late = 1;
      flag_status(P.status, GBO_STATUS_TIMEOUT);
    }
    return base + (int64_t)stage * P.stage_bytes;
  }
  __device__ __forceinline__ void next() {
    if (++stage == P.stages) stage = 0, phase ^= 1;
  }
};

// The places of a row's tensors: in global memory, or one behind the other in a
// stage of the ring.
template <typename XT, typename BT>
struct RowIn {
  const XT *x, *dxo;
  const BT *block, *gate, *dh;
};

template <typename XT, typename BT, bool kRing>
__device__ __forceinline__ RowIn<XT, BT> row_in(const ResParams &P, const uint8_t *stage, int64_t row, bool back) {
  RowIn<XT, BT> r;
  if constexpr (kRing) {
    auto take = [&](bool there, int64_t bytes) {
      const uint8_t *at = stage;
      if (there) stage += bytes;
      return at;
    };
    const int64_t xb = P.d * (int64_t)sizeof(XT), bb = P.d * (int64_t)sizeof(BT);
    r.x = reinterpret_cast<const XT *>(take(!back || P.pre, xb));
    r.block = reinterpret_cast<const BT *>(take(P.block != nullptr, bb));
    r.gate = reinterpret_cast<const BT *>(take(P.gate_mode == kGateElement, bb));
    r.dxo = reinterpret_cast<const XT *>(take(back && P.dxo, xb));
    r.dh = reinterpret_cast<const BT *>(take(back && P.pre, bb));
    if (P.gate_mode == kGateRow) r.gate = static_cast<const BT *>(P.gate) + row * P.as;
  } else {
    r.x = static_cast<const XT *>(P.x) + row * P.xs;
    r.block = static_cast<const BT *>(P.block) + row * P.bs;
    r.gate = static_cast<const BT *>(P.gate) + row * P.as;
    r.dxo = static_cast<const XT *>(P.dxo) + row * P.dxos;
    r.dh = static_cast<const BT *>(P.dh) + row * P.dhs;
  }
  return r;
}

// What both kernels begin with: groups of threads, their rows, the ring.
#define GBO_RESIDUAL_PROLOGUE(back)                                                                          \
  pdl_launch();                                                                                              \
  constexpr int N = kIter * 8;                                                                               \
  extern __shared__ __align__(128) uint8_t ring_smem[];                                                      \
  __shared__ float red[4][96];                                                                               \
  __shared__ uint64_t bars[kMaxStages];                                                                      \
  __shared__ int32_t late;                                                                                   \
  const int group = P.group, in_group = threadIdx.x & (group - 1), d = (int)P.d;                             \
  const int unit = max(group, 32), g = threadIdx.x / unit; /* a join of warps, or a warp of groups */        \
  const int groups = blockDim.x / group, sub = group < 32 ? (threadIdx.x & 31) / group : 0;                  \
  int turn = 0;                                                                                              \
  RowRing<kRing> ring(P, ring_smem, smem_u32(bars), &late);                                                  \
  if constexpr (kRing) {                                                                                     \
    if (threadIdx.x == 0) {                                                                                  \
      for (int s = 0; s < P.stages; ++s) mbar_init(smem_u32(bars + s), 1);                                   \
      late = 0;                                                                                              \
      asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");                                     \
    }                                                                                                        \
    __syncthreads();                                                                                         \
  }                                                                                                          \
  pdl_wait();                                                                                                \
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;                           \
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;                                               \
  uint8_t *table_smem = ring_smem + (kRing ? (int64_t)P.stages * P.stage_bytes : 0);                         \
  const Table<kIter, kVec, kRing> pre_gain(P.pre_gain, d, table_smem, in_group, group);                      \
  const Table<kIter, kVec, kRing> post_gain(P.post_gain, d, table_smem, in_group, group);                    \
  const Table<kIter, kVec, kRing> scale(P.scale_mode == kScaleVector ? P.scale : nullptr, d, table_smem, in_group, group); \
  const int64_t step = (int64_t)gridDim.x * groups;                                                          \
  const int64_t row0 = (int64_t)blockIdx.x * groups + (group < 32 ? g * (32 / group) : g);                   \
  if constexpr (kRing)                                                                                       \
    if (threadIdx.x == 0)                                                                                    \
      for (int s = 0; s < P.stages && row0 + s * step < P.n; ++s) ring.template fill<XT, BT>(s, row0 + s * step, back)

// ... and end a row with: the stage is read, its next row may come.
#define GBO_RESIDUAL_ROW_END(back)                                                                           \
  if constexpr (kRing) {                                                                                     \
    __syncthreads();                                                                                         \
    if (threadIdx.x == 0 && base + P.stages * step < P.n)                                                    \
      ring.template fill<XT, BT>(ring.stage, base + P.stages * step, back);                                  \
    ring.next();                                                                                             \
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
struct ResCut {
  int32_t group, iter, threads, blocks, stages;  // stages 0: no ring
};

constexpr int kSmemMost = 220 * 1024;  // of an SM's shared memory, for rings and tables

// A row goes to as many threads as it has chunks of eight elements, up to 512.
// Rows of 16-byte chunks and 128 threads or more come through a ring, whose CTAs
// (1024 threads an SM forward, 512 for the gradients) share the SM's shared memory.
// `row_bytes`: of a row's inputs; `table_bytes`: of the column tables.
ResCut cut_of(int64_t n, int64_t d, int sm, bool back, bool vec, int64_t row_bytes, int64_t table_bytes) {
  ResCut c;
  const int64_t chunks = (d + 7) / 8;
  c.group = 4;
  while (c.group < kMaxGroup && c.group < chunks) c.group *= 2;
  c.iter = 1;
  while ((int64_t)c.group * c.iter < chunks) c.iter *= 2;
  c.threads = std::max(c.group, 128);
  c.stages = 0;
  const int64_t groups = c.threads / c.group;
  const int per_sm = std::max(1, (back ? 512 : 1024) / c.threads);
  if (vec && c.group >= 128 && c.iter <= 2 && table_bytes + 2 * row_bytes <= kSmemMost)
    c.stages = (int32_t)std::min<int64_t>(kMaxStages, std::max<int64_t>(2, (kSmemMost / per_sm - table_bytes) / row_bytes));
  // gradients: as many blocks as leave the partial rows few; each goes over many rows
  const int64_t most = (int64_t)sm * per_sm;
  c.blocks = (int32_t)std::max<int64_t>(1, std::min(most, (n + groups - 1) / groups));
  return c;
}

// Partial rows of a backward call.
int64_t parts_of(const ResCut &c) { return (int64_t)c.blocks * (c.threads / std::max(c.group, 32)); }

using ResKernel = void (*)(ResParams);

int kernel_slot(const ResCut &c, int32_t xt, int32_t bt) {
  return (xt == GBO_BF16 ? 0 : bt == GBO_BF16 ? 1 : 2) * 2 + (c.iter > 1);
}

// kernel_of: the instance of the pass's kernel for two types, a cut and 16-byte chunks.
template <typename Pick>
cudaError_t dispatch_res(ResParams &P, const ResCut &c, bool vec, int32_t xt, int32_t bt, int64_t table_bytes, int dev, cudaStream_t st,
                         Pick kernel_of) {
  const ResKernel k = kernel_of(xt, bt, c, vec);
  P.group = c.group, P.stages = c.stages;
  const size_t smem = c.stages ? (size_t)c.stages * P.stage_bytes + table_bytes : 0;
  if (c.stages) {
    static PerDevice<cudaError_t> limit[6];
    const cudaError_t *err = limit[kernel_slot(c, xt, bt)].of(dev, [&](cudaError_t &e) {
      e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost);
    });
    if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  }
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), k, dim3(c.blocks), dim3(c.threads), smem, st, 1, P);
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

int64_t table_bytes(const gbo_residual_args *a) {
  return 4 * a->d * ((a->pre_gain != nullptr) + (a->post_gain != nullptr) + (a->scale_mode == GBO_SCALE_VECTOR));
}

bool inputs_vec(const gbo_residual_args *a) {
  return a->d % 8 == 0 && vec_ok(a->x, a->x_stride, a->n) && vec_ok(a->block, a->block_stride, a->n) &&
         (a->gate_mode != GBO_GATE_ELEMENT || vec_ok(a->gate, a->gate_stride, a->n)) && vec_ok(a->post_gain, 0, 0) &&
         vec_ok(a->pre_gain, 0, 0) && (a->scale_mode != GBO_SCALE_VECTOR || vec_ok(a->scale, 0, 0));
}

int32_t parts_wanted(const gbo_residual_grads *g) { return (g->dpre_gain != nullptr) + (g->dpost_gain != nullptr) + (g->dscale != nullptr); }

}  // namespace
}  // namespace gbo

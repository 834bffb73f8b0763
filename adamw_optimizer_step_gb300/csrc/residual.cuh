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
#include "pairs.cuh"
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
  for (int i = 0; i < kCount; ++i) v[i] = (lane & 15) < warps ? r[i * 16 + (lane & 15)] : 0.f;
#pragma unroll
  for (int o = 8; o > 0; o /= 2)
#pragma unroll
    for (int i = 0; i < kCount; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], o);
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

// v *= a column table (gains, scales), where there is one.
template <int kIter, bool kVec>
__device__ __forceinline__ void times_table(const float *t, int d, int in_group, int group, float (&v)[kIter * 8]) {
  if (!t) return;
  float w[kIter * 8];
  row_load<float, kIter, kVec>(t, d, in_group, group, w);
#pragma unroll
  for (int e = 0; e < kIter * 8; ++e) v[e] *= w[e];
}

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

// 1 / (1 + exp(-a)) and its slope, or a and 1.  From e = exp(-|a|) and q = 1 / (1 + e)
// the gate is q or e q, the slope e q q: nothing cancels, nothing overflows.
__device__ __forceinline__ float gate_of(float a, int sigmoid, float *slope = nullptr) {
  if (!sigmoid) {
    if (slope) *slope = 1.f;
    return a;
  }
  const float e = __expf(-fabsf(a)), q = __fdividef(1.f, 1.f + e), eq = e * q;
  if (slope) *slope = eq * q;
  return a >= 0.f ? q : a < 0.f ? eq : a;  // (NaN stays)
}

// ---------------------------------------------------------------------------
// rows through shared memory

// Rows of 16-byte chunks come through a ring of stages in shared memory: the
// input tensors of a row one behind the other, by bulk copies that thread 0
// issues up to `stages` rows ahead.  Loads are then in flight all the time at no
// cost in registers, while a row's two sums over its threads and its arithmetic
// take their time.  A stage is filled again behind the first join of the next
// row, which every thread reaches after its last read of the stage.  (A warp of
// its own for the copies takes registers from the others: 18 warps an SM have 96
// each, 16 have 128.)  The column tables stand behind the ring: from global memory
// each use would wait for L2 behind the row's joins.  What bounds these kernels
// then is instructions: arithmetic is two lanes at a time, factors of a column are
// multiplied into one table at the start.
enum { kInX = 0, kInBlock = 1, kInGate = 2, kInDxo = 3, kInDh = 4, kInputs = 5 };

struct RowRing {
  uint32_t base, full0, stage_bytes;
  int stages;
  volatile int32_t *late;
  int32_t *status;
  int stage = 0, to_fill = 0;
  uint32_t phase = 0;

  static __device__ __forceinline__ void copy(uint32_t dst, const void *src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst), "l"(src),
                 "r"(bytes), "r"(bar)
                 : "memory");
  }
  // All threads: the stage of the next row has arrived.  A wait that runs out is
  // flagged, and every later one passes at once: the outputs are invalid.
  __device__ __forceinline__ uint32_t take() const {
    const uint32_t bar = full0 + 8 * stage;
    if (!mbar_try(bar, phase) && !*late && !mbar_wait(bar, phase)) {
      *late = 1;
      flag_status(status, GBO_STATUS_TIMEOUT);
    }
    return base + (uint32_t)stage * stage_bytes;
  }
  __device__ __forceinline__ void next() {
    if (++stage == stages) stage = 0, phase ^= 1;
  }
};

// Thread 0: a row's tensors from `src` (NULL: none), `by` bytes on from row to row.
struct RowFeed {
  const uint8_t *src[kInputs];
  int64_t by[kInputs];
  uint32_t bytes[kInputs];
  int64_t left;  // rows

  __device__ __forceinline__ void fill(RowRing &r) {
    if (left <= 0) return;
    --left;
    const uint32_t bar = r.full0 + 8 * r.to_fill;
    uint32_t dst = r.base + (uint32_t)r.to_fill * r.stage_bytes;
    mbar_expect_tx(bar, r.stage_bytes);
#pragma unroll
    for (int i = 0; i < kInputs; ++i)
      if (src[i]) {
        RowRing::copy(dst, src[i], bytes[i], bar);
        src[i] += by[i];
        dst += bytes[i];
      }
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

// Dropout's factors of eight elements, times v.
__device__ __forceinline__ void drop8(const DropArgs &D, uint64_t key, uint64_t element, float2 *v) {
  const uint4 w = philox(key, element >> 3, D.offset);
#pragma unroll
  for (int k = 0; k < 4; ++k)
    v[k] = f2_mul(v[k], make_float2(drop_factor(w, 2 * k, D.limit, D.keep), drop_factor(w, 2 * k + 1, D.limit, D.keep)));
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

// A row goes to as many threads as it has chunks of eight elements, up to 512;
// where rows come through a ring, to half as many in the forward pass (what a row
// costs beside its elements is half as much then), one CTA of 64 threads or more
// a row, 512 threads an SM.  The cut of the gradients' partial rows is the same
// with a ring and without.  `row_bytes`: of a row's inputs.
ResCut cut_of(int64_t n, int64_t d, int sm, bool back, bool vec, int64_t row_bytes) {
  ResCut c;
  const int64_t chunks = (d + 7) / 8;
  c.stages = 0;
  if (vec && chunks >= 64 && chunks <= 2 * kMaxGroup) {
    c.group = 64;
    while (c.group < kMaxGroup && (int64_t)c.group * (back ? 1 : 2) < chunks) c.group *= 2;
    c.iter = (int32_t)((chunks + c.group - 1) / c.group);
    c.threads = c.group;
    for (int per_sm = std::max(1, 512 / c.threads); per_sm > 0; --per_sm) {
      const int64_t room = kSmemMost / per_sm - 2 * 4 * d;
      if (room < 2 * row_bytes) continue;
      c.stages = (int32_t)std::min<int64_t>(kMaxStages, room / row_bytes);
      c.blocks = (int32_t)std::max<int64_t>(1, std::min<int64_t>((int64_t)sm * per_sm, n));
      return c;
    }
  }
  c.group = 4;
  while (c.group < kMaxGroup && c.group < chunks) c.group *= 2;
  c.iter = 1;
  while ((int64_t)c.group * c.iter < chunks) c.iter *= 2;
  c.threads = std::max(c.group, 128);
  const int64_t groups = c.threads / c.group;
  // gradients: as many blocks as leave the partial rows few; each goes over many rows
  const int64_t most = (int64_t)sm * std::max(1, (back ? 512 : 1024) / c.threads);
  c.blocks = (int32_t)std::max<int64_t>(1, std::min(most, (n + groups - 1) / groups));
  return c;
}

// Partial rows of a backward call.
int64_t parts_of(const ResCut &c) { return (int64_t)c.blocks * (c.threads / std::max(c.group, 32)); }

// The most that any cut of these sizes leaves.
int64_t most_parts(int64_t n, int64_t d, int sm) {
  return std::max(parts_of(cut_of(n, d, sm, true, true, 1)), parts_of(cut_of(n, d, sm, true, false, 1)));
}

using ResKernel = void (*)(ResParams);

int kernel_slot(const ResCut &c, int32_t xt, int32_t bt) {
  return (xt == GBO_BF16 ? 0 : bt == GBO_BF16 ? 1 : 2) * 2 + (c.iter > 1);
}

// kernel_of: the instance of the pass's kernel for two types, a cut and 16-byte chunks.
template <typename Pick>
cudaError_t dispatch_res(ResParams &P, const ResCut &c, bool vec, int32_t xt, int32_t bt, int dev, cudaStream_t st, Pick kernel_of) {
  const ResKernel k = kernel_of(xt, bt, c, vec);
  P.group = c.group, P.stages = c.stages;
  const size_t smem = c.stages ? (size_t)c.stages * P.stage_bytes + 2 * 4 * P.d : 0;
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

bool inputs_vec(const gbo_residual_args *a) {
  return a->d % 8 == 0 && vec_ok(a->x, a->x_stride, a->n) && vec_ok(a->block, a->block_stride, a->n) &&
         (a->gate_mode != GBO_GATE_ELEMENT || vec_ok(a->gate, a->gate_stride, a->n)) && vec_ok(a->post_gain, 0, 0) &&
         vec_ok(a->pre_gain, 0, 0) && (a->scale_mode != GBO_SCALE_VECTOR || vec_ok(a->scale, 0, 0));
}

int32_t parts_wanted(const gbo_residual_grads *g) { return (g->dpre_gain != nullptr) + (g->dpost_gain != nullptr) + (g->dscale != nullptr); }

}  // namespace
}  // namespace gbo

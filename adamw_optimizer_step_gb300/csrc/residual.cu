// The residual update between two blocks with the norms on either side of it
// (gbo_residual_forward, gbo_residual_backward), and dropout (gbo_dropout).
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
// A group of 32 to 512 threads takes a row, eight consecutive elements to a
// thread and chunk (16-byte loads); rows that 16 bytes do not divide take the
// elements strided over the threads instead (coalesced, one element each).  The
// sums of a row cross the group's warps through shared memory: two joins a row,
// each of all sums known by then.  The sums over rows stay in a thread's
// registers over all rows of its group (a thread keeps its columns), one partial
// row a group is left at the end, and a second kernel adds them in a fixed order.
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

namespace gbo {

namespace {

constexpr int kMaxGroup = 512;

struct ResParams {
  const void *x, *block, *gate, *dxo, *dh;  // backward: x is the updated stream
  void *xo, *h;                             // forward; backward: dx, dblock, dgate
  void *dgate;
  const float *scale, *post_gain, *pre_gain;
  float *part;          // backward: partial rows of dpre_gain, dpost_gain, dscale
  DropArgs drop;
  int64_t n, d;
  int64_t xs, bs, as, xos, hs, dxos, dhs, das;  // row strides
  float eps, inv_d;
  int32_t group, post, pre, gate_mode, sigmoid, scale_mode;
  int32_t want_pre, want_post, want_scale;
};

enum { kGateNone = 0, kGateElement = 1, kGateRow = 2 };
enum { kScaleNone = 0, kScaleOne = 1, kScaleVector = 2 };

// Sums of up to three values over the threads of a group; every thread gets
// them.  `red`: shared, 3 x 16 floats for each of two turns a group.
template <int kCount>
__device__ __forceinline__ void group_sum(float (&v)[kCount], int group, int in_group, float *red, int &turn, int barrier) {
#pragma unroll
  for (int i = 0; i < kCount; ++i) v[i] = warp_sum(v[i]);
  if (group == 32) return;
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
__device__ __forceinline__ int64_t column(int it, int e, int in_group, int group) {
  return kVec ? ((int64_t)it * group + in_group) * 8 + e : (int64_t)(it * 8 + e) * group + in_group;
}

template <typename T, int kIter, bool kVec>
__device__ __forceinline__ void row_load(const T *row, int64_t d, int in_group, int group, float (&v)[kIter * 8]) {
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if constexpr (kVec) {
      const int64_t c = column<true>(it, 0, in_group, group);
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
        const int64_t c = column<false>(it, e, in_group, group);
        v[it * 8 + e] = c < d ? (float)row[c] : 0.f;
      }
    }
  }
}

template <typename T, int kIter, bool kVec>
__device__ __forceinline__ void row_store(T *row, int64_t d, int in_group, int group, const float (&v)[kIter * 8]) {
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if constexpr (kVec) {
      const int64_t c = column<true>(it, 0, in_group, group);
      if (c < d) store8<T>(row + c, v + it * 8, 8, true);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int64_t c = column<false>(it, e, in_group, group);
        if (c < d) st_elem(row, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, c, v[it * 8 + e]);
      }
    }
  }
}

// Column tables (gains, scales); `other` where there is none.
template <int kIter, bool kVec>
__device__ __forceinline__ void table_load(const float *t, float other, int64_t d, int in_group, int group,
                                           float (&v)[kIter * 8]) {
  if (t) {
    row_load<float, kIter, kVec>(t, d, in_group, group, v);
  } else {
#pragma unroll
    for (int e = 0; e < kIter * 8; ++e) v[e] = other;
  }
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
        const int64_t c = column<false>(it, e, in_group, group);
        if (c < P.d) u[it * 8 + e] *= drop_one(P.drop, key, (uint64_t)(row * P.d + c));
      }
    }
  }
}

__device__ __forceinline__ float gate_of(float a, int sigmoid) { return sigmoid ? 1.f / (1.f + __expf(-a)) : a; }

template <typename XT, typename BT, int kIter, bool kVec>
__global__ void __launch_bounds__(kMaxGroup) residual_forward_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  constexpr int N = kIter * 8;
  __shared__ float red[16][96];
  const int group = P.group, in_group = threadIdx.x & (group - 1), g = threadIdx.x / group, groups = blockDim.x / group;
  int turn = 0;
  pdl_wait();
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  for (int64_t row = (int64_t)blockIdx.x * groups + g; row < P.n; row += (int64_t)gridDim.x * groups) {
    float x[N];
    row_load<XT, kIter, kVec>(static_cast<const XT *>(P.x) + row * P.xs, P.d, in_group, group, x);
    if (P.block) {
      float u[N], t[N];
      row_load<BT, kIter, kVec>(static_cast<const BT *>(P.block) + row * P.bs, P.d, in_group, group, u);
      if (P.gate_mode == kGateElement)
        row_load<BT, kIter, kVec>(static_cast<const BT *>(P.gate) + row * P.as, P.d, in_group, group, t);
      if (P.post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int e = 0; e < N; ++e) sum[0] = fmaf(u[e], u[e], sum[0]);
        group_sum(sum, group, in_group, red[g], turn, 1 + g);
        const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
#pragma unroll
        for (int e = 0; e < N; ++e) u[e] *= r;
        if (P.post_gain) {
          float w[N];
          row_load<float, kIter, kVec>(P.post_gain, P.d, in_group, group, w);
#pragma unroll
          for (int e = 0; e < N; ++e) u[e] *= w[e];
        }
      }
      if (P.drop.limit) row_drop<kIter, kVec>(P, key, row, in_group, group, u);
      if (P.gate_mode == kGateElement) {
#pragma unroll
        for (int e = 0; e < N; ++e) u[e] *= gate_of(t[e], P.sigmoid);
      }
      if (P.scale_mode == kScaleVector) {
        float w[N];
        row_load<float, kIter, kVec>(P.scale, P.d, in_group, group, w);
#pragma unroll
        for (int e = 0; e < N; ++e) u[e] *= w[e];
      }
      const float f = s1 * (P.gate_mode == kGateRow ? gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid) : 1.f);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = fmaf(f, u[e], x[e]);
      row_store<XT, kIter, kVec>(static_cast<XT *>(P.xo) + row * P.xos, P.d, in_group, group, x);
    }
    if (P.pre) {
      float sum[1] = {0.f};
#pragma unroll
      for (int e = 0; e < N; ++e) sum[0] = fmaf(x[e], x[e], sum[0]);
      group_sum(sum, group, in_group, red[g], turn, 1 + g);
      const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= r;
      if (P.pre_gain) {
        float w[N];
        row_load<float, kIter, kVec>(P.pre_gain, P.d, in_group, group, w);
#pragma unroll
        for (int e = 0; e < N; ++e) x[e] *= w[e];
      }
      row_store<BT, kIter, kVec>(static_cast<BT *>(P.h) + row * P.hs, P.d, in_group, group, x);
    }
  }
}

template <int kIter, bool kVec>
__device__ __forceinline__ void part_store(float *row, int64_t d, int in_group, int group, const float (&v)[kIter * 8]) {
  row_store<float, kIter, kVec>(row, d, in_group, group, v);
}

template <typename XT, typename BT, int kIter, bool kVec>
__global__ void __launch_bounds__(kMaxGroup) residual_backward_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  constexpr int N = kIter * 8;
  __shared__ float red[16][96];
  const int group = P.group, in_group = threadIdx.x & (group - 1), g = threadIdx.x / group, groups = blockDim.x / group;
  int turn = 0;
  float a_pre[N], a_post[N], a_scale[N];  // sums over this group's rows
#pragma unroll
  for (int e = 0; e < N; ++e) a_pre[e] = a_post[e] = a_scale[e] = 0.f;
  pdl_wait();
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  for (int64_t row = (int64_t)blockIdx.x * groups + g; row < P.n; row += (int64_t)gridDim.x * groups) {
    float dx[N], o[N];
    if (P.dxo) {
      row_load<XT, kIter, kVec>(static_cast<const XT *>(P.dxo) + row * P.dxos, P.d, in_group, group, dx);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) dx[e] = 0.f;
    }
    if (P.block) row_load<BT, kIter, kVec>(static_cast<const BT *>(P.block) + row * P.bs, P.d, in_group, group, o);
    float ro = 1.f;
    {
      float x[N], w[N], sum[3] = {0.f, 0.f, 0.f};
      if (P.pre) {
        row_load<XT, kIter, kVec>(static_cast<const XT *>(P.x) + row * P.xs, P.d, in_group, group, x);
        row_load<BT, kIter, kVec>(static_cast<const BT *>(P.dh) + row * P.dhs, P.d, in_group, group, w);
        float gain[N];
        table_load<kIter, kVec>(P.pre_gain, 1.f, P.d, in_group, group, gain);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          sum[0] = fmaf(x[e], x[e], sum[0]);
          sum[1] = fmaf(w[e] * gain[e], x[e], sum[1]);
        }
      }
      if (P.post) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[2] = fmaf(o[e], o[e], sum[2]);
      }
      if (P.pre || P.post) group_sum(sum, group, in_group, red[g], turn, 1 + g);
      ro = P.post ? rsqrtf(fmaf(sum[2], P.inv_d, P.eps)) : 1.f;
      if (P.pre) {
        const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps)), c = sum[1] * P.inv_d * r * r;
        float gain[N];
        table_load<kIter, kVec>(P.pre_gain, 1.f, P.d, in_group, group, gain);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          a_pre[e] = fmaf(w[e], x[e] * r, a_pre[e]);
          dx[e] = fmaf(r, w[e] * gain[e] - x[e] * c, dx[e]);
        }
      }
    }
    if (P.xo) row_store<XT, kIter, kVec>(static_cast<XT *>(P.xo) + row * P.xos, P.d, in_group, group, dx);
    if (!P.block) continue;
    // v = o rho(o) in o; dx becomes g m, then du
#pragma unroll
    for (int e = 0; e < N; ++e) o[e] *= ro;
    if (P.drop.limit) row_drop<kIter, kVec>(P, key, row, in_group, group, dx);
    float a_row = 0.f;
    if (P.gate_mode == kGateRow) a_row = (float)static_cast<const BT *>(P.gate)[row * P.as];
    const float f_row = P.gate_mode == kGateRow ? gate_of(a_row, P.sigmoid) : 1.f;
    float sum[2] = {0.f, 0.f};
    {
      float gain[N], s[N], a[N];
      table_load<kIter, kVec>(P.post_gain, 1.f, P.d, in_group, group, gain);
      table_load<kIter, kVec>(P.scale_mode == kScaleVector ? P.scale : nullptr, s1, P.d, in_group, group, s);
      if (P.gate_mode == kGateElement)
        row_load<BT, kIter, kVec>(static_cast<const BT *>(P.gate) + row * P.as, P.d, in_group, group, a);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        const float u = o[e] * gain[e], gu = dx[e] * u;  // g m u
        const float f = P.gate_mode == kGateElement ? gate_of(a[e], P.sigmoid) : f_row;
        a_scale[e] = fmaf(gu, f, a_scale[e]);
        const float slope = P.sigmoid ? f * (1.f - f) : 1.f;
        a[e] = gu * s[e] * slope;
        sum[1] += a[e];
        dx[e] *= s[e] * f;
        a_post[e] = fmaf(dx[e], o[e], a_post[e]);
        dx[e] *= gain[e];
        sum[0] = fmaf(dx[e], o[e], sum[0]);
      }
      if (P.gate_mode == kGateElement && P.dgate)
        row_store<BT, kIter, kVec>(static_cast<BT *>(P.dgate) + row * P.das, P.d, in_group, group, a);
    }
    if (P.post || P.gate_mode == kGateRow) group_sum(sum, group, in_group, red[g], turn, 1 + g);
    if (P.gate_mode == kGateRow && P.dgate && in_group == 0)
      st_elem(P.dgate, sizeof(BT) == 2 ? GBO_BF16 : GBO_F32, row * P.das, sum[1]);
    if (P.h) {
      if (P.post) {
        const float c = sum[0] * P.inv_d;
#pragma unroll
        for (int e = 0; e < N; ++e) dx[e] = ro * (dx[e] - o[e] * c);
      }
      row_store<BT, kIter, kVec>(static_cast<BT *>(P.h) + row * P.hs, P.d, in_group, group, dx);
    }
  }
  float *part = P.part + ((int64_t)blockIdx.x * groups + g) * P.d;
  const int64_t rows = (int64_t)gridDim.x * groups * P.d;
  if (P.want_pre) part_store<kIter, kVec>(part, P.d, in_group, group, a_pre);
  if (P.want_pre) part += rows;
  if (P.want_post) part_store<kIter, kVec>(part, P.d, in_group, group, a_post);
  if (P.want_post) part += rows;
  if (P.want_scale) part_store<kIter, kVec>(part, P.d, in_group, group, a_scale);
}

// The partial rows added up, in a fixed order: 32 columns a block.  Of a scale
// that is one number the columns' sums are added by residual_one_kernel.
struct ResSum {
  const float *part[3];
  float *out[3];
  int64_t d;
  int32_t rows;
};

__global__ void __launch_bounds__(1024) residual_sum_kernel(const __grid_constant__ ResSum S) {
  pdl_launch();
  __shared__ float red[32][33];
  const int which = blockIdx.y;
  const int64_t col = (int64_t)blockIdx.x * 32 + threadIdx.x;
  pdl_wait();
  float a = 0.f;
  if (col < S.d) {
    const float *part = S.part[which] + col;
    for (int r0 = threadIdx.y; r0 < S.rows; r0 += 32 * 8) {  // eight rows in flight
      float v[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) v[u] = r0 + 32 * u < S.rows ? part[(int64_t)(r0 + 32 * u) * S.d] : 0.f;
#pragma unroll
      for (int u = 0; u < 8; ++u) a += v[u];
    }
  }
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  const float v = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int64_t out = (int64_t)blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < S.d) S.out[which][out] = v;
}

__global__ void __launch_bounds__(1024) residual_one_kernel(const float *__restrict__ columns, int64_t d, float *out) {
  pdl_launch();
  __shared__ float red[32];
  pdl_wait();
  float a = 0.f;
  for (int64_t c = threadIdx.x; c < d; c += 1024) a += columns[c];
  a = block_sum(a, red);
  if (threadIdx.x == 0) *out = a;
}

// ---------------------------------------------------------------------------
// dropout alone: eight elements of the tensor's order to a thread and turn

struct DropParams {
  const void *x;
  void *y;
  DropArgs drop;
  int64_t count, cols, xs, ys;  // elements; columns and row strides
  int32_t flat;                 // rows follow one another on 16-byte boundaries
};

template <typename T>
__global__ void __launch_bounds__(256) dropout_kernel(const __grid_constant__ DropParams P) {
  pdl_launch();
  pdl_wait();
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const int64_t chunks = (P.count + 7) / 8, step = (int64_t)gridDim.x * 256;
  const T *x = static_cast<const T *>(P.x);
  T *y = static_cast<T *>(P.y);
  for (int64_t c = (int64_t)blockIdx.x * 256 + threadIdx.x; c < chunks; c += step) {
    float v[8];
    const int64_t at = c * 8;
    if (P.flat && at + 8 <= P.count) {
      load8(x, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, at, 8, true, v);
      const uint4 w = P.drop.limit ? philox(key, (uint64_t)c, P.drop.offset) : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] *= drop_factor(w, e, P.drop.limit, P.drop.keep);
      store8<T>(y + at, v, 8, true);
    } else {
      const uint4 w = P.drop.limit ? philox(key, (uint64_t)c, P.drop.offset) : make_uint4(0, 0, 0, 0);
      int64_t row = at / P.cols, col = at - row * P.cols;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        if (at + e < P.count)
          st_elem(y, sizeof(T) == 2 ? GBO_BF16 : GBO_F32, row * P.ys + col,
                  (float)x[row * P.xs + col] * drop_factor(w, e, P.drop.limit, P.drop.keep));
        if (++col == P.cols) col = 0, ++row;
      }
    }
  }
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

// Threads to a row and chunks to a thread.
struct ResCut {
  int32_t group, iter, threads, blocks;
};

// A row goes to as few threads as leave each a chunk or two (a group of one
// warp needs no join through shared memory), and to 512 at most.
ResCut cut_of(int64_t n, int64_t d, int sm, bool back) {
  ResCut c;
  const int64_t chunks = (d + 7) / 8;
  c.group = 32;
  while (c.group < kMaxGroup && c.group < chunks) c.group *= 2;
  c.iter = 1;
  while ((int64_t)c.group * c.iter < chunks) c.iter *= 2;
  c.threads = std::max(c.group, 128);
  const int64_t groups = c.threads / c.group;
  // gradients: as many blocks as leave the partial rows few; each goes over many rows
  const int64_t most = (int64_t)sm * (back ? std::max(1, 1024 / c.threads) : std::max(1, 2048 / c.threads));
  c.blocks = (int32_t)std::max<int64_t>(1, std::min(most, (n + groups - 1) / groups));
  return c;
}

template <typename XT, typename BT, int kIter, bool kVec>
cudaError_t launch_res(const ResParams &P, const ResCut &c, bool back, cudaStream_t st) {
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), back ? residual_backward_kernel<XT, BT, kIter, kVec> : residual_forward_kernel<XT, BT, kIter, kVec>,
                          dim3(c.blocks), dim3(c.threads), 0, st, 1, P);
}

template <typename XT, typename BT>
cudaError_t dispatch_iter(const ResParams &P, const ResCut &c, bool vec, bool back, cudaStream_t st) {
  if (!vec) return c.iter == 1 ? launch_res<XT, BT, 1, false>(P, c, back, st) : launch_res<XT, BT, 4, false>(P, c, back, st);
  return c.iter == 1   ? launch_res<XT, BT, 1, true>(P, c, back, st)
         : c.iter == 2 ? launch_res<XT, BT, 2, true>(P, c, back, st)
                       : launch_res<XT, BT, 4, true>(P, c, back, st);
}

cudaError_t dispatch_res(const ResParams &P, const ResCut &c, bool vec, bool back, int32_t xt, int32_t bt, cudaStream_t st) {
  if (xt == GBO_BF16) return dispatch_iter<__nv_bfloat16, __nv_bfloat16>(P, c, vec, back, st);
  return bt == GBO_BF16 ? dispatch_iter<float, __nv_bfloat16>(P, c, vec, back, st) : dispatch_iter<float, float>(P, c, vec, back, st);
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

using namespace gbo;

extern "C" int gbo_residual_forward(const gbo_residual_args *a, void *x_out, int64_t x_out_stride, void *h, int64_t h_stride,
                                    gbo_stream_t stream) {
  DropArgs drop = {};
  int rc = check_residual(a, &drop);
  if (rc != GBO_OK) return rc;
  if (a->n > 0) {
    if ((rc = check_rows(a->x, a->x_stride, a, a->d, a->x_dtype)) != GBO_OK) return rc;
    if (a->has_block && (rc = check_rows(x_out, x_out_stride, a, a->d, a->x_dtype)) != GBO_OK) return rc;
    if (a->pre_norm && (rc = check_rows(h, h_stride, a, a->d, a->block_dtype)) != GBO_OK) return rc;
  }
  if (!a->has_block && x_out) return res_fail(GBO_ERR_INVALID_ARG, "x_out without has_block: the stream stays as it is");
  if (!a->pre_norm && h) return res_fail(GBO_ERR_INVALID_ARG, "h without pre_norm");
  int dev, sm = 0;
  if ((rc = require_device(&dev, &sm)) != GBO_OK) return rc;
  if (a->n == 0) return report_ok();
  ResParams P;
  fill_res(a, drop, &P);
  P.xo = x_out, P.xos = x_out_stride, P.h = h, P.hs = h_stride;
  const bool vec = inputs_vec(a) && vec_ok(x_out, x_out_stride, a->n) && vec_ok(h, h_stride, a->n);
  const ResCut c = cut_of(a->n, a->d, sm, false);
  P.group = c.group;
  const cudaError_t e = dispatch_res(P, c, vec, false, a->x_dtype, a->block_dtype, reinterpret_cast<cudaStream_t>(stream));
  return e == cudaSuccess ? report_ok() : res_cuda(e);
}

extern "C" size_t gbo_residual_workspace_bytes(int64_t n, int64_t d, int32_t sums) {
  int dev, sm = 0;
  if (n < 0 || d < 1 || d > GBO_RESIDUAL_MAX_D || sums < 0 || sums > 3 || require_device(&dev, &sm) != GBO_OK) return 0;
  const ResCut c = cut_of(n, d, sm, true);
  return sums ? (size_t)(c.blocks * (c.threads / c.group)) * d * sums * 4 + (size_t)d * 4 : 0;
}

extern "C" int gbo_residual_backward(const gbo_residual_args *a, const gbo_residual_grads *g, void *workspace, size_t ws_bytes,
                                     gbo_stream_t stream) {
  DropArgs drop = {};
  int rc = check_residual(a, &drop);
  if (rc != GBO_OK) return rc;
  if (!g) return res_fail(GBO_ERR_INVALID_ARG, "grads is NULL");
  if ((g->dpre_gain && !a->pre_gain) || (g->dpost_gain && !a->post_gain) || (g->dscale && a->scale_mode == GBO_SCALE_NONE) ||
      (g->dgate && a->gate_mode == GBO_GATE_NONE) || (g->dblock && !a->has_block))
    return res_fail(GBO_ERR_INVALID_ARG, "a gradient of something that is not there");
  if ((reinterpret_cast<uintptr_t>(g->dpre_gain) | reinterpret_cast<uintptr_t>(g->dpost_gain) |
       reinterpret_cast<uintptr_t>(g->dscale)) & 3)
    return res_fail(GBO_ERR_INVALID_ARG, "misaligned gradient of a gain or scale");
  if (g->dh && !a->pre_norm) return res_fail(GBO_ERR_INVALID_ARG, "dh without pre_norm");
  if (a->n > 0) {
    if (a->pre_norm && ((rc = check_rows(a->x, a->x_stride, a, a->d, a->x_dtype)) != GBO_OK ||
                        (rc = check_rows(g->dh, g->dh_stride, a, a->d, a->block_dtype)) != GBO_OK))
      return rc;
    if (!g->dx_out && !a->pre_norm) return res_fail(GBO_ERR_INVALID_ARG, "neither dx_out nor dh");
    if (g->dx_out && (rc = check_rows(g->dx_out, g->dx_out_stride, a, a->d, a->x_dtype)) != GBO_OK) return rc;
    if (g->dx && (rc = check_rows(g->dx, g->dx_stride, a, a->d, a->x_dtype)) != GBO_OK) return rc;
    if (g->dblock && (rc = check_rows(g->dblock, g->dblock_stride, a, a->d, a->block_dtype)) != GBO_OK) return rc;
    if (g->dgate && (rc = check_rows(g->dgate, g->dgate_stride, a, a->gate_mode == GBO_GATE_ROW ? 1 : a->d, a->block_dtype)) != GBO_OK)
      return rc;
  }
  int dev, sm = 0;
  if ((rc = require_device(&dev, &sm)) != GBO_OK) return rc;
  const int32_t sums = parts_wanted(g);
  if (sums) {
    if (!workspace || ws_bytes < gbo_residual_workspace_bytes(a->n, a->d, sums))
      return res_fail(GBO_ERR_WORKSPACE, "workspace missing or smaller than gbo_residual_workspace_bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return res_fail(GBO_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  }
  ResParams P;
  fill_res(a, drop, &P);
  P.dxo = g->dx_out, P.dxos = g->dx_out_stride, P.dh = g->dh, P.dhs = g->dh_stride;
  P.xo = g->dx, P.xos = g->dx_stride, P.h = g->dblock, P.hs = g->dblock_stride, P.dgate = g->dgate, P.das = g->dgate_stride;
  P.want_pre = g->dpre_gain != nullptr, P.want_post = g->dpost_gain != nullptr, P.want_scale = g->dscale != nullptr;
  P.part = static_cast<float *>(workspace);
  const bool vec = inputs_vec(a) && vec_ok(g->dx_out, g->dx_out_stride, a->n) && vec_ok(g->dh, g->dh_stride, a->n) &&
                   vec_ok(g->dx, g->dx_stride, a->n) && vec_ok(g->dblock, g->dblock_stride, a->n) &&
                   (a->gate_mode != GBO_GATE_ELEMENT || vec_ok(g->dgate, g->dgate_stride, a->n));
  const ResCut c = cut_of(a->n, a->d, sm, true);
  P.group = c.group;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->n > 0 || sums) e = dispatch_res(P, c, vec, true, a->x_dtype, a->block_dtype, st);
  if (e == cudaSuccess && sums) {
    ResSum S;
    memset(&S, 0, sizeof S);
    S.d = a->d, S.rows = c.blocks * (c.threads / c.group);
    const int64_t each = (int64_t)S.rows * a->d;
    float *columns = P.part + sums * each;  // of a scale that is one number
    float *const outs[3] = {g->dpre_gain, g->dpost_gain, g->dscale && a->scale_mode == GBO_SCALE_ONE ? columns : g->dscale};
    int k = 0;
    for (float *out : outs)
      if (out) S.part[k] = P.part + k * each, S.out[k] = out, ++k;
    count_launches(1);
    e = launch_kernel_as(pdl_allowed(), residual_sum_kernel, dim3((unsigned)((a->d + 31) / 32), k), dim3(32, 32), 0, st, 1, S);
    if (e == cudaSuccess && g->dscale && a->scale_mode == GBO_SCALE_ONE) {
      count_launches(1);
      e = launch_kernel_as(pdl_allowed(), residual_one_kernel, dim3(1), dim3(1024), 0, st, 1, columns, a->d, g->dscale);
    }
  }
  return e == cudaSuccess ? report_ok() : res_cuda(e);
}

extern "C" int gbo_dropout(const void *x, int64_t x_stride, void *y, int64_t y_stride, int64_t n, int64_t d, int32_t dtype, double p,
                           uint64_t seed, uint64_t offset, const int64_t *dev_seed, gbo_stream_t stream) {
  DropParams P;
  memset(&P, 0, sizeof P);
  if (dtype != GBO_F32 && dtype != GBO_BF16) return res_fail(GBO_ERR_DTYPE, "dtype must be GBO_F32 or GBO_BF16");
  if (n < 0 || d < 0 || (d > 0 && n > INT64_MAX / 16 / d)) return res_fail(GBO_ERR_SHAPE, "n or d negative or too large");
  if (!drop_of(p, &P.drop)) return res_fail(GBO_ERR_INVALID_ARG, "p must be in 0 <= p < 1 - 2^-17");
  if (reinterpret_cast<uintptr_t>(dev_seed) & 7) return res_fail(GBO_ERR_INVALID_ARG, "misaligned dev_seed");
  const int es = size_of(dtype);
  const int64_t count = n * d;
  if (count > 0) {
    if (!x || !y) return res_fail(GBO_ERR_INVALID_ARG, "NULL tensor pointer");
    if ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) % es) return res_fail(GBO_ERR_INVALID_ARG, "misaligned tensor pointer");
    if (n > 1 && (x_stride < d || y_stride < d)) return res_fail(GBO_ERR_INVALID_ARG, "a row stride must be at least d");
  }
  int dev, sm = 0;
  const int rc = require_device(&dev, &sm);
  if (rc != GBO_OK) return rc;
  if (count == 0) return report_ok();
  P.x = x, P.y = y, P.drop.seed = seed, P.drop.offset = offset, P.drop.dev_seed = dev_seed;
  P.count = count, P.cols = d, P.xs = n > 1 ? x_stride : d, P.ys = n > 1 ? y_stride : d;
  P.flat = P.xs == d && P.ys == d && ((reinterpret_cast<uintptr_t>(x) | reinterpret_cast<uintptr_t>(y)) & 15) == 0;
  const int64_t blocks = std::min<int64_t>(((count + 7) / 8 + 255) / 256, (int64_t)sm * 32);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  count_launches(1);
  const cudaError_t e = launch_kernel_as(pdl_allowed(), dtype == GBO_BF16 ? dropout_kernel<__nv_bfloat16> : dropout_kernel<float>,
                                         dim3((unsigned)blocks), dim3(256), 0, st, 1, P);
  return e == cudaSuccess ? report_ok() : res_cuda(e);
}

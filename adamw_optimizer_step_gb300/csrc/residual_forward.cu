// The residual update, forward (gbo_residual_forward), and dropout (gbo_dropout).
#include "residual.cuh"

namespace gbo {

namespace {

// Rows below 512 elements: a group of threads a row.
template <typename XT, typename BT, bool kVec>
__global__ void __launch_bounds__(kGroupThreads) residual_forward_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  __shared__ float red[kGroupThreads / 32][96];
  __shared__ uint4 slots[kVec ? 1 : kGroupThreads / 32 * kDropSlots];
  const int group = P.group, in_group = threadIdx.x & (group - 1), d = (int)P.d;
  const int unit = max(group, 32), g = threadIdx.x / unit;  // a join of warps, or a warp of groups
  const int groups = blockDim.x / group, sub = group < 32 ? (threadIdx.x & 31) / group : 0;
  int turn = 0;
  pdl_wait();
  const int64_t step = (int64_t)gridDim.x * groups;
  const int64_t row0 = (int64_t)blockIdx.x * groups + (group < 32 ? g * (32 / group) : g);
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  for (int64_t base = row0; base < P.n; base += step) {
    const int64_t row = base + sub;
    const int dr = row < P.n ? d : 0;  // (the last warp may hold fewer rows than groups)
    float x[8];
    load_part<XT, kVec>(static_cast<const XT *>(P.x) + row * P.xs, dr, 0, in_group, group, x);
    if (P.block) {
      float u[8];
      load_part<BT, kVec>(static_cast<const BT *>(P.block) + row * P.bs, dr, 0, in_group, group, u);
      float f = s1;
      if (P.post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(u[e], u[e], sum[0]);
        group_sum(sum, group, in_group, red[g], turn, 1 + g);
        f *= rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
      }
      block_factors<BT, kVec>(P, key, row, dr, 0, in_group, group, u, slots);
      if (P.gate_mode == kGateRow && dr) f *= gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid);
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = fmaf(f, u[e], x[e]);
      store_part<XT, kVec>(static_cast<XT *>(P.xo) + row * P.xos, dr, 0, in_group, group, x);
    }
    if (P.pre) {
      float sum[1] = {0.f};
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[0] = fmaf(x[e], x[e], sum[0]);
      group_sum(sum, group, in_group, red[g], turn, 1 + g);
      const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] *= r;
      times_table<kVec>(P.pre_gain, d, 0, in_group, group, x);
      store_part<BT, kVec>(static_cast<BT *>(P.h) + row * P.hs, dr, 0, in_group, group, x);
    }
  }
}

// Rows that no ring has room for: a CTA a row, x' in shared memory, the block's
// output read twice (the second time from L2).
template <typename XT, typename BT, bool kVec>
__global__ void __launch_bounds__(kMaxGroup, 2) residual_forward_wide_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float red[96];
  __shared__ uint4 slots[kVec ? 1 : kMaxGroup / 32 * kDropSlots];
  float *const kept = reinterpret_cast<float *>(ring_smem) + threadIdx.x;
  constexpr int threads = kMaxGroup;
  const int tid = threadIdx.x, d = (int)P.d, its = (d + 8 * threads - 1) / (8 * threads);
  int turn = 0;
  pdl_wait();
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  for (int64_t row = blockIdx.x; row < P.n; row += gridDim.x) {
    const XT *const x_row = static_cast<const XT *>(P.x) + row * P.xs;
    const BT *const o_row = static_cast<const BT *>(P.block) + row * P.bs;
    float f = s1, sum[1] = {0.f};
    if (P.post) {
      for (int it = 0; it < its; ++it) {
        float o[8];
        load_part<BT, kVec>(o_row, d, it, tid, threads, o);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(o[e], o[e], sum[0]);
      }
      cta_sum(sum, red, turn);
      f *= rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
    }
    if (P.gate_mode == kGateRow) f *= gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid);
    sum[0] = 0.f;
    for (int it = 0; it < its; ++it) {
      float x[8];
      load_part<XT, kVec>(x_row, d, it, tid, threads, x);
      if (P.block) {
        float u[8];
        load_part<BT, kVec>(o_row, d, it, tid, threads, u);
        block_factors<BT, kVec>(P, key, row, d, it, tid, threads, u, slots);
#pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = fmaf(f, u[e], x[e]);
        store_part<XT, kVec>(static_cast<XT *>(P.xo) + row * P.xos, d, it, tid, threads, x);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        sum[0] = fmaf(x[e], x[e], sum[0]);
        kept[(it * 8 + e) * threads] = x[e];
      }
    }
    if (!P.pre) continue;
    cta_sum(sum, red, turn);
    const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
    for (int it = 0; it < its; ++it) {
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = kept[(it * 8 + e) * threads] * r;
      times_table<kVec>(P.pre_gain, d, it, tid, threads, x);
      store_part<BT, kVec>(static_cast<BT *>(P.h) + row * P.hs, d, it, tid, threads, x);
    }
  }
}

// Rows through a ring, a CTA to a row.  post_gain and scale stand in one table:
// x' = x + (s1 rho(o) gate_row) table gate m o.  32768 x 2048 bf16 with both norms: 84 us,
// 6.4 TB/s (94% of a copy's rate); with an element gate and dropout 135 us, 5.0 TB/s.
template <typename XT, typename BT, int kIter, bool kOdd>
__global__ void __launch_bounds__(kMaxGroup) residual_forward_ring_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float red[96];
  __shared__ uint4 slots[kOdd ? kMaxGroup / 32 * kDropSlots : 1];
  __shared__ uint64_t bars[kMaxStages];
  __shared__ int32_t late;
  constexpr int N = kIter * 4;  // pairs of elements
  const int tid = threadIdx.x, threads = blockDim.x, d = (int)P.d, chunks = kOdd ? kIter * threads : d / 8;
  const RowPart<kOdd> part = {d, tid, threads};
  RowRing ring{smem_u32(ring_smem), smem_u32(bars), (uint32_t)P.stage_bytes, P.stages, &late, P.status};
  if (tid == 0) {
    for (int s = 0; s < P.stages; ++s) mbar_init(ring.full0 + 8 * s, 1);
    late = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  const int64_t row0 = blockIdx.x, step = gridDim.x;
  const uint32_t xb = (uint32_t)P.d * sizeof(XT), bb = (uint32_t)P.d * sizeof(BT);
  const uint32_t to_block = RowFeed<kOdd>::place(xb), to_gate = to_block + RowFeed<kOdd>::place(bb);  // (of a stage)
  RowFeed<kOdd> feed{};
  if (tid == 0) {
    auto set = [&](int i, const void *p, int64_t stride, uint32_t bytes, int size) {
      if (!p) return;
      feed.src[i] = static_cast<const uint8_t *>(p) + row0 * stride * size;
      feed.by[i] = step * stride * size, feed.bytes[i] = bytes;
    };
    set(kInX, P.x, P.xs, xb, sizeof(XT));
    set(kInBlock, P.block, P.bs, bb, sizeof(BT));
    if (P.gate_mode == kGateElement) set(kInGate, P.gate, P.as, bb, sizeof(BT));
    feed.row = row0, feed.step = step, feed.n = P.n;
    for (int s = 0; s < P.stages; ++s) feed.fill(ring);
  }
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  const ColumnTable mul = {ring.base + P.stages * ring.stage_bytes, (uint32_t)chunks * 16};
  const ColumnTable pre = {mul.at + 2 * mul.half, mul.half};
  const bool muls = P.post_gain || P.scale_mode == kScaleVector;
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if (part.here(it)) {
      float v[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = part.column(it, e);
        v[e] = w[e] = 0.f;
        if (c < d) {
          v[e] = table_at(P.post_gain, c) * table_at(P.scale_mode == kScaleVector ? P.scale : nullptr, c);
          w[e] = table_at(P.pre_gain, c);
        }
      }
      mul.put(part.chunk(it), v);
      pre.put(part.chunk(it), w);
    }
  }
  int turn = 0;
  for (int64_t row = row0; row < P.n; row += step) {
    const uint32_t at = ring.take();
    float2 x[N];
    const uint32_t x_at = row_start<kOdd>(at, static_cast<const XT *>(P.x), row, P.xs);
    bool joined = false;
    auto join = [&](float v) {
      float sum[1] = {v};
      cta_sum(sum, red, turn);
      if (!joined && tid == 0 && row != row0) feed.fill(ring);
      joined = true;
      return rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
    };
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      if (part.here(it)) {
        part.template get<XT>(x_at, it, x + 4 * it);
      } else {
#pragma unroll
        for (int k = 0; k < 4; ++k) x[4 * it + k] = f2_of(0.f);
      }
    }
    if (P.block) {
      float2 u[N];
      float2 ss = f2_of(0.f);
      const uint32_t o_at = row_start<kOdd>(at + to_block, static_cast<const BT *>(P.block), row, P.bs);
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        if (part.here(it)) {
          part.template get<BT>(o_at, it, u + 4 * it);
#pragma unroll
          for (int k = 0; k < 4; ++k) ss = f2_fma(u[4 * it + k], u[4 * it + k], ss);
        }
      }
      float f = s1;
      if (P.gate_mode == kGateRow) f *= gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid);
      if (P.post) f *= join(ss.x + ss.y);
      const float2 f2 = f2_of(f);
      XT *const out = static_cast<XT *>(P.xo) + row * P.xos;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        if (part.here(it)) {
          float2 *const v = u + 4 * it;
          if (muls) {
            float2 t[4];
            mul.get(part.chunk(it), t);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = f2_mul(v[k], t[k]);
          }
          if (P.drop.limit) part.drop(P, key, row, it, v, slots);
          if (P.gate_mode == kGateElement) {
            float2 a[4];
            part.template get<BT>(row_start<kOdd>(at + to_gate, static_cast<const BT *>(P.gate), row, P.as), it, a);
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              float2 slope;
              v[k] = f2_mul(v[k], gate_of2(a[k], P.sigmoid, slope));
            }
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) x[4 * it + k] = f2_fma(f2, v[k], x[4 * it + k]);
          part.put(out, it, x + 4 * it);
        }
      }
    }
    if (P.pre) {
      float2 ss = f2_of(0.f);
#pragma unroll
      for (int k = 0; k < N; ++k) ss = f2_fma(x[k], x[k], ss);
      const float2 r = f2_of(join(ss.x + ss.y));
      BT *const out = static_cast<BT *>(P.h) + row * P.hs;
#pragma unroll
      for (int it = 0; it < kIter; ++it) {
        if (part.here(it)) {
          float2 *const v = x + 4 * it;
#pragma unroll
          for (int k = 0; k < 4; ++k) v[k] = f2_mul(v[k], r);
          if (P.pre_gain) {
            float2 t[4];
            pre.get(part.chunk(it), t);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[k] = f2_mul(v[k], t[k]);
          }
          part.put(out, it, v);
        }
      }
    }
    if (!joined) {
      __syncthreads();
      if (tid == 0 && row != row0) feed.fill(ring);
    }
    ring.next();
  }
  if (tid == 0 && ring.gave_up) ring.settle((feed.row - row0) / step);
}

// ---------------------------------------------------------------------------
// dropout alone: eight elements of the tensor's order to a thread and turn, one counter.
// 32768 x 2048 bf16: 45.7 us, 5.9 TB/s (86% of a copy's rate); bound by the rounds'
// multiplications (integer pipe, 69% of the issue slots) and the writes behind them.

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

template <typename XT, typename BT, bool kVec>
ResLaunch pick(const ResCut &c) {
  if (c.form == kFormWide) return launch_res<residual_forward_wide_kernel<XT, BT, kVec>>;
  if (c.form == kFormGroup) return launch_res<residual_forward_kernel<XT, BT, kVec>>;
  return c.iter == 1 ? launch_res<residual_forward_ring_kernel<XT, BT, 1, !kVec>>
                     : launch_res<residual_forward_ring_kernel<XT, BT, 2, !kVec>>;
}

template <bool kVec>
ResLaunch launcher(int32_t xt, int32_t bt, const ResCut &c) {
  return xt == GBO_BF16 ? pick<__nv_bfloat16, __nv_bfloat16, kVec>(c)
                        : bt == GBO_BF16 ? pick<float, __nv_bfloat16, kVec>(c) : pick<float, float, kVec>(c);
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" int gbo_residual_forward(const gbo_residual_args *a, void *x_out, int64_t x_out_stride, void *h, int64_t h_stride,
                                    int32_t *dev_status, gbo_stream_t stream) {
  DropArgs drop = {};
  int rc = check_residual(a, &drop);
  if (rc != GBO_OK) return rc;
  if (reinterpret_cast<uintptr_t>(dev_status) & 3) return res_fail(GBO_ERR_INVALID_ARG, "misaligned status pointer");
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
  P.status = dev_status;
  P.stage_bytes = (int32_t)row_bytes(P, a->x_dtype, a->block_dtype, vec, false);
  const ResCut c = cut_of(a->n, a->d, sm, false, vec, P.stage_bytes);
  const ResLaunch launch = vec ? launcher<true>(a->x_dtype, a->block_dtype, c) : launcher<false>(a->x_dtype, a->block_dtype, c);
  const cudaError_t e = launch(P, c, dev, reinterpret_cast<cudaStream_t>(stream));
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

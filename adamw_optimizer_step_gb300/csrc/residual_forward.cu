// The residual update, forward (gbo_residual_forward), and dropout (gbo_dropout).
#include "residual.cuh"

namespace gbo {

namespace {

template <typename XT, typename BT, int kIter, bool kVec, bool kRing>
__global__ void __launch_bounds__(kMaxGroup) residual_forward_kernel(const __grid_constant__ ResParams P) {
  GBO_RESIDUAL_PROLOGUE(false);
  for (int64_t base = row0; base < P.n; base += step) {
    const int64_t row = base + sub;
    const int dr = row < P.n ? d : 0;  // (the last warp may hold fewer rows than groups)
    const uint8_t *stage = nullptr;
    if constexpr (kRing) stage = ring.wait();
    const RowIn<XT, BT> in = row_in<XT, BT, kRing>(P, stage, row, false);
    float x[N];
    row_load<XT, kIter, kVec>(in.x, dr, in_group, group, x);
    if (P.block) {
      float u[N];
      row_load<BT, kIter, kVec>(in.block, dr, in_group, group, u);
      float f = s1;
      if (P.post) {
        float sum[1] = {0.f};
#pragma unroll
        for (int e = 0; e < N; ++e) sum[0] = fmaf(u[e], u[e], sum[0]);
        group_sum(sum, group, in_group, red[g], turn, 1 + g);
        f *= rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
        post_gain.times(in_group, group, u);
      }
      if (P.drop.limit) row_drop<kIter, kVec>(P, key, row, in_group, group, u);
      if (P.gate_mode == kGateElement) {
        float a[N];
        row_load<BT, kIter, kVec>(in.gate, dr, in_group, group, a);
#pragma unroll
        for (int e = 0; e < N; ++e) u[e] *= gate_of(a[e], P.sigmoid);
      }
      scale.times(in_group, group, u);
      if (P.gate_mode == kGateRow && dr) f *= gate_of((float)*in.gate, P.sigmoid);
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] = fmaf(f, u[e], x[e]);
      row_store<XT, kIter, kVec>(static_cast<XT *>(P.xo) + row * P.xos, dr, in_group, group, x);
    }
    if (P.pre) {
      float sum[1] = {0.f};
#pragma unroll
      for (int e = 0; e < N; ++e) sum[0] = fmaf(x[e], x[e], sum[0]);
      group_sum(sum, group, in_group, red[g], turn, 1 + g);
      const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps));
#pragma unroll
      for (int e = 0; e < N; ++e) x[e] *= r;
      pre_gain.times(in_group, group, x);
      row_store<BT, kIter, kVec>(static_cast<BT *>(P.h) + row * P.hs, dr, in_group, group, x);
    }
    GBO_RESIDUAL_ROW_END(false)
  }
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

template <typename XT, typename BT>
ResKernel pick(const ResCut &c, bool vec) {
  if (c.stages) return c.iter == 1 ? residual_forward_kernel<XT, BT, 1, true, true> : residual_forward_kernel<XT, BT, 2, true, true>;
  if (vec) return c.iter == 1 ? residual_forward_kernel<XT, BT, 1, true, false> : residual_forward_kernel<XT, BT, 4, true, false>;
  return c.iter == 1   ? residual_forward_kernel<XT, BT, 1, false, false>
         : c.iter == 2 ? residual_forward_kernel<XT, BT, 2, false, false>
                       : residual_forward_kernel<XT, BT, 4, false, false>;
}

ResKernel kernel_of(int32_t xt, int32_t bt, const ResCut &c, bool vec) {
  return xt == GBO_BF16 ? pick<__nv_bfloat16, __nv_bfloat16>(c, vec)
                        : bt == GBO_BF16 ? pick<float, __nv_bfloat16>(c, vec) : pick<float, float>(c, vec);
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
  P.stage_bytes = (int32_t)(a->d * (size_of(a->x_dtype) + size_of(a->block_dtype) * (a->has_block + (a->gate_mode == GBO_GATE_ELEMENT))));
  const ResCut c = cut_of(a->n, a->d, sm, false, vec, P.stage_bytes, table_bytes(a));
  const cudaError_t e = dispatch_res(P, c, vec, a->x_dtype, a->block_dtype, table_bytes(a), dev, reinterpret_cast<cudaStream_t>(stream), kernel_of);
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

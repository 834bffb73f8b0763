// Gradients of the residual update (gbo_residual_backward).
#include "residual.cuh"

namespace gbo {

namespace {

// The groups of a warp added up: one partial row a warp.
template <int N>
__device__ __forceinline__ void warp_join(float (&v)[N], int group) {
#pragma unroll
  for (int o = 16; o > 0; o /= 2)
    if (o >= group) {
#pragma unroll
      for (int e = 0; e < N; ++e) v[e] += __shfl_xor_sync(0xffffffffu, v[e], o);
    }
}

template <typename XT, typename BT, int kIter, bool kVec, bool kRing>
__global__ void __launch_bounds__(kMaxGroup) residual_backward_kernel(const __grid_constant__ ResParams P) {
  GBO_RESIDUAL_PROLOGUE(true);
  float a_pre[N], a_post[N], a_scale[N];  // sums over this group's rows
#pragma unroll
  for (int e = 0; e < N; ++e) a_pre[e] = a_post[e] = a_scale[e] = 0.f;
  for (int64_t base = row0; base < P.n; base += step) {
    const int64_t row = base + sub;
    const int dr = row < P.n ? d : 0;
    const uint8_t *stage = nullptr;
    if constexpr (kRing) stage = ring.wait();
    const RowIn<XT, BT> in = row_in<XT, BT, kRing>(P, stage, row, true);
    float sum[3] = {0.f, 0.f, 0.f};
    if (P.pre) {
      float x[N], w[N];
      row_load<XT, kIter, kVec>(in.x, dr, in_group, group, x);
      row_load<BT, kIter, kVec>(in.dh, dr, in_group, group, w);
      pre_gain.times(in_group, group, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        sum[0] = fmaf(x[e], x[e], sum[0]);
        sum[1] = fmaf(w[e], x[e], sum[1]);
      }
    }
    float o[N];
    if (P.block) {
      row_load<BT, kIter, kVec>(in.block, dr, in_group, group, o);
      if (P.post) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[2] = fmaf(o[e], o[e], sum[2]);
      }
    }
    if (P.pre || P.post) group_sum(sum, group, in_group, red[g], turn, 1 + g);
    const float ro = P.post ? rsqrtf(fmaf(sum[2], P.inv_d, P.eps)) : 1.f;
    float dx[N];
    if (P.dxo) {
      row_load<XT, kIter, kVec>(in.dxo, dr, in_group, group, dx);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) dx[e] = 0.f;
    }
    if (P.pre) {
      float x[N], w[N];
      row_load<XT, kIter, kVec>(in.x, dr, in_group, group, x);
      row_load<BT, kIter, kVec>(in.dh, dr, in_group, group, w);
      const float r = rsqrtf(fmaf(sum[0], P.inv_d, P.eps)), c = sum[1] * P.inv_d * r * r;
#pragma unroll
      for (int e = 0; e < N; ++e) a_pre[e] = fmaf(w[e], x[e] * r, a_pre[e]);
      pre_gain.times(in_group, group, w);
#pragma unroll
      for (int e = 0; e < N; ++e) dx[e] = fmaf(r, w[e] - x[e] * c, dx[e]);
    }
    if (P.xo) row_store<XT, kIter, kVec>(static_cast<XT *>(P.xo) + row * P.xos, dr, in_group, group, dx);
    if (P.block) {
      // v = o rho(o) in o; dx becomes g m, then du, then post_gain du
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] *= ro;
      if (P.drop.limit) row_drop<kIter, kVec>(P, key, row, in_group, group, dx);
      float row_slope = 0.f;
      const float row_gate = P.gate_mode == kGateRow && dr ? gate_of((float)*in.gate, P.sigmoid, &row_slope) : 1.f;
      float u[N], da[N], join[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] = o[e];
      post_gain.times(in_group, group, u);
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] *= dx[e];  // g m u
      if (P.gate_mode == kGateElement) {
        row_load<BT, kIter, kVec>(in.gate, dr, in_group, group, da);
#pragma unroll
        for (int e = 0; e < N; ++e) {
          float slope;
          const float f = gate_of(da[e], P.sigmoid, &slope);
          a_scale[e] = fmaf(u[e], f, a_scale[e]);
          da[e] = u[e] * (s1 * slope);
          dx[e] *= s1 * f;
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e) {
          a_scale[e] = fmaf(u[e], row_gate, a_scale[e]);
          da[e] = u[e] * (s1 * row_slope);
          dx[e] *= s1 * row_gate;
        }
      }
      if (scale.at) {
        float w[N];
        scale.load(in_group, group, w);
#pragma unroll
        for (int e = 0; e < N; ++e) da[e] *= w[e], dx[e] *= w[e];
      }
      if (P.gate_mode == kGateElement && P.dgate)
        row_store<BT, kIter, kVec>(static_cast<BT *>(P.dgate) + row * P.das, dr, in_group, group, da);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        join[1] += da[e];
        a_post[e] = fmaf(dx[e], o[e], a_post[e]);
      }
      post_gain.times(in_group, group, dx);
#pragma unroll
      for (int e = 0; e < N; ++e) join[0] = fmaf(dx[e], o[e], join[0]);
      if (P.post || P.gate_mode == kGateRow) group_sum(join, group, in_group, red[g], turn, 1 + g);
      if (P.gate_mode == kGateRow && P.dgate && in_group == 0 && dr)
        st_elem(P.dgate, sizeof(BT) == 2 ? GBO_BF16 : GBO_F32, row * P.das, join[1]);
      if (P.h) {
        if (P.post) {
          const float c = join[0] * P.inv_d;
#pragma unroll
          for (int e = 0; e < N; ++e) dx[e] = ro * (dx[e] - o[e] * c);
        }
        row_store<BT, kIter, kVec>(static_cast<BT *>(P.h) + row * P.hs, dr, in_group, group, dx);
      }
    }
    GBO_RESIDUAL_ROW_END(true)
  }
  if (!(P.want_pre | P.want_post | P.want_scale)) return;
  warp_join(a_pre, group);
  warp_join(a_post, group);
  warp_join(a_scale, group);
  const int units = blockDim.x / unit;
  const int64_t rows = (int64_t)gridDim.x * units * P.d;
  float *part = P.part + ((int64_t)blockIdx.x * units + g) * P.d;
  const int dw = sub == 0 ? d : 0;
  if (P.want_pre) row_store<float, kIter, kVec>(part, dw, in_group, group, a_pre), part += rows;
  if (P.want_post) row_store<float, kIter, kVec>(part, dw, in_group, group, a_post), part += rows;
  if (P.want_scale) row_store<float, kIter, kVec>(part, dw, in_group, group, a_scale);
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

template <typename XT, typename BT>
ResKernel pick(const ResCut &c, bool vec) {
  if (c.stages) return c.iter == 1 ? residual_backward_kernel<XT, BT, 1, true, true> : residual_backward_kernel<XT, BT, 2, true, true>;
  if (vec) return c.iter == 1 ? residual_backward_kernel<XT, BT, 1, true, false> : residual_backward_kernel<XT, BT, 4, true, false>;
  return c.iter == 1   ? residual_backward_kernel<XT, BT, 1, false, false>
         : c.iter == 2 ? residual_backward_kernel<XT, BT, 2, false, false>
                       : residual_backward_kernel<XT, BT, 4, false, false>;
}

ResKernel kernel_of(int32_t xt, int32_t bt, const ResCut &c, bool vec) {
  return xt == GBO_BF16 ? pick<__nv_bfloat16, __nv_bfloat16>(c, vec)
                        : bt == GBO_BF16 ? pick<float, __nv_bfloat16>(c, vec) : pick<float, float>(c, vec);
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" size_t gbo_residual_workspace_bytes(int64_t n, int64_t d, int32_t sums) {
  int dev, sm = 0;
  if (n < 0 || d < 1 || d > GBO_RESIDUAL_MAX_D || sums < 0 || sums > 3 || require_device(&dev, &sm) != GBO_OK) return 0;
  const ResCut c = cut_of(n, d, sm, true, false, 0, 0);  // (the ring changes no block)
  return sums ? (size_t)parts_of(c) * d * sums * 4 + (size_t)d * 4 : 0;
}

extern "C" int gbo_residual_backward(const gbo_residual_args *a, const gbo_residual_grads *g, void *workspace, size_t ws_bytes,
                                     int32_t *dev_status, gbo_stream_t stream) {
  DropArgs drop = {};
  int rc = check_residual(a, &drop);
  if (rc != GBO_OK) return rc;
  if (!g) return res_fail(GBO_ERR_INVALID_ARG, "grads is NULL");
  if (reinterpret_cast<uintptr_t>(dev_status) & 3) return res_fail(GBO_ERR_INVALID_ARG, "misaligned status pointer");
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
  P.status = dev_status;
  P.stage_bytes = (int32_t)(a->d * (size_of(a->x_dtype) * (a->pre_norm + (g->dx_out != nullptr)) +
                                    size_of(a->block_dtype) * (a->has_block + (a->gate_mode == GBO_GATE_ELEMENT) + a->pre_norm)));
  const ResCut c = cut_of(a->n, a->d, sm, true, vec, P.stage_bytes, table_bytes(a));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  if (a->n > 0 || sums) e = dispatch_res(P, c, vec, a->x_dtype, a->block_dtype, table_bytes(a), dev, st, kernel_of);
  if (e == cudaSuccess && sums) {
    ResSum S;
    memset(&S, 0, sizeof S);
    S.d = a->d, S.rows = (int32_t)parts_of(c);
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


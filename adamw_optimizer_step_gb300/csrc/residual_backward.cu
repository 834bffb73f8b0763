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

// Rows below 512 elements: a group of threads a row.
template <typename XT, typename BT, bool kVec>
__global__ void __launch_bounds__(kGroupThreads, 4) residual_backward_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  constexpr int N = 8;
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
  float a_pre[N], a_post[N], a_scale[N];  // sums over this group's rows
#pragma unroll
  for (int e = 0; e < N; ++e) a_pre[e] = a_post[e] = a_scale[e] = 0.f;
  for (int64_t base = row0; base < P.n; base += step) {
    const int64_t row = base + sub;
    const int dr = row < P.n ? d : 0;
    struct {
      const XT *x, *dxo;
      const BT *block, *gate, *dh;
    } const in = {static_cast<const XT *>(P.x) + row * P.xs, static_cast<const XT *>(P.dxo) + row * P.dxos,
                  static_cast<const BT *>(P.block) + row * P.bs, static_cast<const BT *>(P.gate) + row * P.as,
                  static_cast<const BT *>(P.dh) + row * P.dhs};
    float sum[3] = {0.f, 0.f, 0.f};
    if (P.pre) {
      float x[N], w[N];
      load_part<XT, kVec>(in.x, dr, 0, in_group, group, x);
      load_part<BT, kVec>(in.dh, dr, 0, in_group, group, w);
      times_table<kVec>(P.pre_gain, d, 0, in_group, group, w);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        sum[0] = fmaf(x[e], x[e], sum[0]);
        sum[1] = fmaf(w[e], x[e], sum[1]);
      }
    }
    float o[N];
    if (P.block) {
      load_part<BT, kVec>(in.block, dr, 0, in_group, group, o);
      if (P.post) {
#pragma unroll
        for (int e = 0; e < N; ++e) sum[2] = fmaf(o[e], o[e], sum[2]);
      }
    }
    if (P.pre || P.post) group_sum(sum, group, in_group, red[g], turn, 1 + g);
    // (a row that is not there has sums of 0, and with eps = 0 a norm's factor of it would
    // be infinite: 0 times that, NaN, would stand in the sums over rows)
    const float ro = P.post ? dr ? rsqrtf(fmaf(sum[2], P.inv_d, P.eps)) : 0.f : 1.f;
    float dx[N];
    if (P.dxo) {
      load_part<XT, kVec>(in.dxo, dr, 0, in_group, group, dx);
    } else {
#pragma unroll
      for (int e = 0; e < N; ++e) dx[e] = 0.f;
    }
    if (P.pre) {
      float x[N], w[N];
      load_part<XT, kVec>(in.x, dr, 0, in_group, group, x);
      load_part<BT, kVec>(in.dh, dr, 0, in_group, group, w);
      const float r = dr ? rsqrtf(fmaf(sum[0], P.inv_d, P.eps)) : 0.f, c = sum[1] * P.inv_d * r * r;
#pragma unroll
      for (int e = 0; e < N; ++e) a_pre[e] = fmaf(w[e], x[e] * r, a_pre[e]);
      times_table<kVec>(P.pre_gain, d, 0, in_group, group, w);
#pragma unroll
      for (int e = 0; e < N; ++e) dx[e] = fmaf(r, w[e] - x[e] * c, dx[e]);
    }
    if (P.xo) store_part<XT, kVec>(static_cast<XT *>(P.xo) + row * P.xos, dr, 0, in_group, group, dx);
    if (P.block) {
      // v = o rho(o) in o; dx becomes g m, then du, then post_gain du
#pragma unroll
      for (int e = 0; e < N; ++e) o[e] *= ro;
      if (P.drop.limit) row_drop<kVec>(P, key, row, 0, in_group, group, dx, slots);
      float row_slope = 0.f;
      const float row_gate = P.gate_mode == kGateRow && dr ? gate_of((float)*in.gate, P.sigmoid, &row_slope) : 1.f;
      float u[N], da[N], join[2] = {0.f, 0.f};
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] = o[e];
      times_table<kVec>(P.post_gain, d, 0, in_group, group, u);
#pragma unroll
      for (int e = 0; e < N; ++e) u[e] *= dx[e];  // g m u
      if (P.gate_mode == kGateElement) {
        load_part<BT, kVec>(in.gate, dr, 0, in_group, group, da);
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
      if (P.scale_mode == kScaleVector) {
        float w[N];
        load_part<float, kVec>(P.scale, d, 0, in_group, group, w);
#pragma unroll
        for (int e = 0; e < N; ++e) da[e] *= w[e], dx[e] *= w[e];
      }
      if (P.gate_mode == kGateElement && P.dgate)
        store_part<BT, kVec>(static_cast<BT *>(P.dgate) + row * P.das, dr, 0, in_group, group, da);
#pragma unroll
      for (int e = 0; e < N; ++e) {
        join[1] += da[e];
        a_post[e] = fmaf(dx[e], o[e], a_post[e]);
      }
      times_table<kVec>(P.post_gain, d, 0, in_group, group, dx);
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
        store_part<BT, kVec>(static_cast<BT *>(P.h) + row * P.hs, dr, 0, in_group, group, dx);
      }
    }
  }
  if (!(P.want_pre | P.want_post | P.want_scale)) return;
  warp_join(a_pre, group);
  warp_join(a_post, group);
  warp_join(a_scale, group);
  const int units = blockDim.x / unit;
  const int64_t rows = (int64_t)gridDim.x * units * P.d;
  float *part = P.part + ((int64_t)blockIdx.x * units + g) * P.d;
  const int dw = sub == 0 ? d : 0;
  if (P.want_pre) store_part<float, kVec>(part, dw, 0, in_group, group, a_pre), part += rows;
  if (P.want_post) store_part<float, kVec>(part, dw, 0, in_group, group, a_post), part += rows;
  if (P.want_scale) store_part<float, kVec>(part, dw, 0, in_group, group, a_scale);
}

// Rows that no ring has room for: a CTA a row, its tensors read two or three times
// (from L2 after the first), w and the sums over rows in shared memory.  Names as
// in the ring's form below.
template <typename XT, typename BT, bool kVec>
__global__ void __launch_bounds__(kMaxGroup) residual_backward_wide_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float red[96];
  __shared__ uint4 slots[kVec ? 1 : kMaxGroup / 32 * kDropSlots];
  constexpr int threads = kMaxGroup;
  const int tid = threadIdx.x, d = (int)P.d, its = (d + 8 * threads - 1) / (8 * threads), n = its * 8 * threads;
  float *const w_kept = reinterpret_cast<float *>(ring_smem) + tid, *const a_pre = w_kept + n, *const a_all = a_pre + n;
  int turn = 0;
  for (int e = 0; e < its * 8; ++e) a_pre[e * threads] = a_all[e * threads] = 0.f;  // (a thread's own)
  pdl_wait();
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  const float *const scale = P.scale_mode == kScaleVector ? P.scale : nullptr;
  for (int64_t row = blockIdx.x; row < P.n; row += gridDim.x) {
    const XT *const x_row = static_cast<const XT *>(P.x) + row * P.xs, *const dx_row = static_cast<const XT *>(P.dxo) + row * P.dxos;
    const BT *const o_row = static_cast<const BT *>(P.block) + row * P.bs, *const dh_row = static_cast<const BT *>(P.dh) + row * P.dhs;
    float sum[3] = {0.f, 0.f, 0.f};
    for (int it = 0; it < its; ++it) {
      float a[8], b[8];
      if (P.pre) {
        load_part<XT, kVec>(x_row, d, it, tid, threads, a);
        load_part<BT, kVec>(dh_row, d, it, tid, threads, b);
        times_table<kVec>(P.pre_gain, d, it, tid, threads, b);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[0] = fmaf(a[e], a[e], sum[0]), sum[1] = fmaf(b[e], a[e], sum[1]);
      }
      if (P.post) {
        load_part<BT, kVec>(o_row, d, it, tid, threads, a);
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[2] = fmaf(a[e], a[e], sum[2]);
      }
    }
    if (P.pre || P.post) cta_sum(sum, red, turn);
    const float ro = P.post ? rsqrtf(fmaf(sum[2], P.inv_d, P.eps)) : 1.f;
    const float r = P.pre ? rsqrtf(fmaf(sum[0], P.inv_d, P.eps)) : 1.f, c = sum[1] * P.inv_d * r * r;
    float row_slope = 0.f, row_gate = 1.f;
    if (P.gate_mode == kGateRow) row_gate = gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid, &row_slope);
    float join[2] = {0.f, 0.f};
    for (int it = 0; it < its; ++it) {
      float dx[8], v[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) dx[e] = 0.f;
      if (P.dxo) load_part<XT, kVec>(dx_row, d, it, tid, threads, dx);
      if (P.pre) {
        load_part<XT, kVec>(x_row, d, it, tid, threads, v);
        load_part<BT, kVec>(dh_row, d, it, tid, threads, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) a_pre[(it * 8 + e) * threads] += w[e] * (v[e] * r);
        times_table<kVec>(P.pre_gain, d, it, tid, threads, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) dx[e] = fmaf(r, w[e] - v[e] * c, dx[e]);
      }
      if (P.xo) store_part<XT, kVec>(static_cast<XT *>(P.xo) + row * P.xos, d, it, tid, threads, dx);
      if (!P.block) continue;
      if (P.drop.limit) row_drop<kVec>(P, key, row, it, tid, threads, dx, slots);
      load_part<BT, kVec>(o_row, d, it, tid, threads, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = s1, v[e] *= ro;
      times_table<kVec>(P.post_gain, d, it, tid, threads, w);
      times_table<kVec>(scale, d, it, tid, threads, w);  // M
      float a[8];
      if (P.gate_mode == kGateElement) load_part<BT, kVec>(static_cast<const BT *>(P.gate) + row * P.as, d, it, tid, threads, a);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float f = row_gate, slope = row_slope;
        if (P.gate_mode == kGateElement) f = gate_of(a[e], P.sigmoid, &slope);
        const float t = dx[e] * v[e];
        a_all[(it * 8 + e) * threads] += t * f;
        a[e] = t * w[e] * slope;
        join[1] += a[e];
        join[0] = fmaf(t * f, w[e], join[0]);
        w[e] *= dx[e] * f;
      }
      if (P.gate_mode == kGateElement && P.dgate)
        store_part<BT, kVec>(static_cast<BT *>(P.dgate) + row * P.das, d, it, tid, threads, a);
      if (!P.h) continue;
      if (P.post) {
#pragma unroll
        for (int e = 0; e < 8; ++e) w_kept[(it * 8 + e) * threads] = w[e];
      } else {
        store_part<BT, kVec>(static_cast<BT *>(P.h) + row * P.hs, d, it, tid, threads, w);
      }
    }
    if (!(P.post || P.gate_mode == kGateRow)) continue;
    cta_sum(join, red, turn);
    if (P.gate_mode == kGateRow && P.dgate && tid == 0)
      st_elem(P.dgate, sizeof(BT) == 2 ? GBO_BF16 : GBO_F32, row * P.das, join[1]);
    if (!(P.h && P.post)) continue;
    for (int it = 0; it < its; ++it) {
      float v[8], w[8];
      load_part<BT, kVec>(o_row, d, it, tid, threads, v);
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = ro * (w_kept[(it * 8 + e) * threads] - v[e] * (ro * join[0] * P.inv_d));
      store_part<BT, kVec>(static_cast<BT *>(P.h) + row * P.hs, d, it, tid, threads, w);
    }
  }
  const int64_t rows = (int64_t)gridDim.x * P.d;
  for (int it = 0; it < its; ++it) {
    float *part = P.part + (int64_t)blockIdx.x * P.d;
    float v[8];
    if (P.want_pre) {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[e] = a_pre[(it * 8 + e) * threads];
      store_part<float, kVec>(part, d, it, tid, threads, v), part += rows;
    }
    for (int which = 0; which < 2; ++which)
      if (which == 0 ? P.want_post : P.want_scale) {
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = a_all[(it * 8 + e) * threads] * (which == 0 ? s1 : 1.f);
        times_table<kVec>(which == 0 ? scale : P.post_gain, d, it, tid, threads, v);
        store_part<float, kVec>(part, d, it, tid, threads, v), part += rows;
      }
  }
}

// Rows through a ring, a CTA to a row.  With t = g m v, v = o rho(o), the table
// M = scale post_gain (s1 where the scale is one number) and the gate f:
//   A = sum t f:  dscale = post_gain A, dpost_gain = scale A
//   da = t M f',  w = g m f M,  mean(w v) = mean(t f M),  do = rho(o) (w - v mean(w v))
// One join of the CTA a row: the sums that start row i and the one that ends row
// i - 1 cross the warps together, while the rows' other work fills the time between.
// kAll: both norms, and every gradient of a row is there, as in training.  Without
// the branches a row is few blocks of instructions whose loads and arithmetic
// overlap (32768 x 2048 with gate and dropout: 273 -> 231 us, 4.7 TB/s; the rest is
// issue slots, 600 instructions a warp and row at 60% of them).
template <typename XT, typename BT, int kIter, bool kOdd, bool kAll>
__global__ void __launch_bounds__(kMaxGroup) residual_backward_ring_kernel(const __grid_constant__ ResParams P) {
  pdl_launch();
  extern __shared__ __align__(128) uint8_t ring_smem[];
  __shared__ float4 red[2][16];
  __shared__ float red_gate[2][16];
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
  if (tid < 32) red[tid >> 4][tid & 15] = make_float4(0.f, 0.f, 0.f, 0.f);  // (warps that are not there)
  __syncthreads();
  pdl_wait();
  const int64_t row0 = blockIdx.x, step = gridDim.x;
  const uint32_t xb = (uint32_t)P.d * sizeof(XT), bb = (uint32_t)P.d * sizeof(BT);
  const bool gated = P.gate_mode == kGateElement;
  const bool pre_norm = kAll || P.pre, post_norm = kAll || P.post, has_block = kAll || P.block, has_dxo = kAll || P.dxo;
  const bool out_dx = kAll || P.xo, out_do = kAll || P.h;
  RowFeed<kOdd> feed{};
  if (tid == 0) {
    auto set = [&](int i, const void *p, int64_t stride, uint32_t bytes, int size) {
      if (!p) return;
      feed.src[i] = static_cast<const uint8_t *>(p) + row0 * stride * size;
      feed.by[i] = step * stride * size, feed.bytes[i] = bytes;
    };
    if (P.pre) set(kInX, P.x, P.xs, xb, sizeof(XT));
    set(kInBlock, P.block, P.bs, bb, sizeof(BT));
    if (gated) set(kInGate, P.gate, P.as, bb, sizeof(BT));
    set(kInDxo, P.dxo, P.dxos, xb, sizeof(XT));
    if (P.pre) set(kInDh, P.dh, P.dhs, bb, sizeof(BT));
    feed.row = row0, feed.step = step, feed.n = P.n;
    for (int s = 0; s < P.stages; ++s) feed.fill(ring);
  }
  // a stage's tensors
  const uint32_t xp = RowFeed<kOdd>::place(xb), bp = RowFeed<kOdd>::place(bb);
  const uint32_t to_block = pre_norm ? xp : 0, to_gate = to_block + (has_block ? bp : 0), to_dxo = to_gate + (gated ? bp : 0);
  const uint32_t to_dh = to_dxo + (has_dxo ? xp : 0);
  const uint64_t key = P.drop.dev_seed ? (uint64_t)*P.drop.dev_seed : P.drop.seed;
  const float s1 = P.scale_mode == kScaleOne ? *P.scale : 1.f;
  const float *const scale = P.scale_mode == kScaleVector ? P.scale : nullptr;
  const ColumnTable mul = {ring.base + P.stages * ring.stage_bytes, (uint32_t)chunks * 16};
  const ColumnTable pre = {mul.at + 2 * mul.half, mul.half};
  float2 a_pre[N], a_all[N];
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
#pragma unroll
    for (int k = 0; k < 4; ++k) a_pre[4 * it + k] = a_all[4 * it + k] = f2_of(0.f);
    if (part.here(it)) {
      float v[8], w[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const int c = part.column(it, e);
        v[e] = w[e] = 0.f;
        if (c < d) v[e] = s1 * table_at(P.post_gain, c) * table_at(scale, c), w[e] = table_at(P.pre_gain, c);
      }
      mul.put(part.chunk(it), v);
      pre.put(part.chunk(it), w);
    }
  }
  // this thread's part of a row's sums: x^2, pre_gain dh x, o^2
  auto x_at = [&](uint32_t at, int64_t row) { return row_start<kOdd>(at, static_cast<const XT *>(P.x), row, P.xs); };
  auto dh_at = [&](uint32_t at, int64_t row) { return row_start<kOdd>(at + to_dh, static_cast<const BT *>(P.dh), row, P.dhs); };
  auto o_at = [&](uint32_t at, int64_t row) { return row_start<kOdd>(at + to_block, static_cast<const BT *>(P.block), row, P.bs); };
  auto first_sums = [&](uint32_t at, int64_t row, float4 &s) {
    float2 s0 = f2_of(0.f), sx = f2_of(0.f), so = f2_of(0.f);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      if (part.here(it)) {
        if (pre_norm) {
          float2 t[4], x[4], dh[4];
          part.template get<XT>(x_at(at, row), it, x);
          part.template get<BT>(dh_at(at, row), it, dh);
          pre.get(part.chunk(it), t);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            s0 = f2_fma(x[k], x[k], s0);
            sx = f2_fma(f2_mul(dh[k], t[k]), x[k], sx);
          }
        }
        if (post_norm) {
          float2 o[4];
          part.template get<BT>(o_at(at, row), it, o);
#pragma unroll
          for (int k = 0; k < 4; ++k) so = f2_fma(o[k], o[k], so);
        }
      }
    }
    s.x = s0.x + s0.y, s.y = sx.x + sx.y, s.z = so.x + so.y;
  };
  const int warp = tid >> 5, lane = tid & 31;
  // of the last row: w and v, rho(o), the part of sum w v, of the row gate's gradient
  float2 g[N], o[N];
#pragma unroll
  for (int e = 0; e < N; ++e) g[e] = o[e] = f2_of(0.f);
  float ro = 1.f, j1 = 0.f;
  float4 sums = make_float4(0.f, 0.f, 0.f, 0.f);  // w: sum w v of the last row
  int turn = 0;
  uint32_t at = 0;
  if (row0 < P.n) first_sums(at = ring.take(), row0, sums);
  // this thread's row of each output, moved on from row to row (the block's gradient a row behind)
  XT *out_x = static_cast<XT *>(P.xo) + row0 * P.xos;
  BT *out_gate = static_cast<BT *>(P.dgate) + row0 * P.das, *out_o = static_cast<BT *>(P.h) + row0 * P.hs;
  const int64_t x_by = step * P.xos, gate_by = step * P.das, o_by = step * P.hs;
  for (int64_t row = row0; row < P.n + step; row += step) {  // (one turn more for the last row's block gradient)
    const int64_t last = row - step;
    sums = warp_sum4(sums, lane);
    if ((lane & 7) == 0) reinterpret_cast<float *>(&red[turn][warp])[lane >> 3] = sums.x;
    if (P.gate_mode == kGateRow) {
      const float v = warp_sum(j1);
      if (lane == 0) red_gate[turn][warp] = v;
    }
    __syncthreads();
    sums = cta_join(red[turn], threads >> 5);
    if (row != row0) {
      if (tid == 0) {
        feed.fill(ring);
        if (P.gate_mode == kGateRow && P.dgate) {
          float v = 0.f;
          for (int w = 0; w < threads >> 5; ++w) v += red_gate[turn][w];
          st_elem(P.dgate, sizeof(BT) == 2 ? GBO_BF16 : GBO_F32, last * P.das, v);
        }
      }
      if (out_do && post_norm) {
        const float2 m2 = f2_of(-sums.w * P.inv_d), ro2 = f2_of(ro);
#pragma unroll
        for (int it = 0; it < kIter; ++it) {
          if (part.here(it)) {
#pragma unroll
            for (int k = 0; k < 4; ++k) g[4 * it + k] = f2_mul(ro2, f2_fma(o[4 * it + k], m2, g[4 * it + k]));
            part.put(out_o, it, g + 4 * it);
          }
        }
        out_o += o_by;
      }
    }
    turn ^= 1;
    if (row >= P.n) break;
    // (the row is read again: held over the join, two chunks a thread would spill)
    const float r = rsqrtf(fmaf(sums.x, P.inv_d, P.eps));
    ro = post_norm ? rsqrtf(fmaf(sums.z, P.inv_d, P.eps)) : 1.f;
    const float2 r2 = f2_of(r), c2 = f2_of(-sums.y * P.inv_d * r * r), ro2 = f2_of(ro);
    float row_slope = 0.f;
    float row_gate = 1.f;
    if (P.gate_mode == kGateRow) row_gate = gate_of((float)static_cast<const BT *>(P.gate)[row * P.as], P.sigmoid, &row_slope);
    float2 j0 = f2_of(0.f), jg = f2_of(0.f);
#pragma unroll
    for (int it = 0; it < kIter; ++it) {
      if (part.here(it)) {
        float2 *const dx = g + 4 * it;
        if (has_dxo) {
          part.template get<XT>(row_start<kOdd>(at + to_dxo, static_cast<const XT *>(P.dxo), row, P.dxos), it, dx);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k) dx[k] = f2_of(0.f);
        }
        if (pre_norm) {
          float2 t[4], x[4], dh[4];
          part.template get<XT>(x_at(at, row), it, x);
          part.template get<BT>(dh_at(at, row), it, dh);
          pre.get(part.chunk(it), t);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            a_pre[4 * it + k] = f2_fma(dh[k], f2_mul(x[k], r2), a_pre[4 * it + k]);
            dx[k] = f2_fma(r2, f2_fma(x[k], c2, f2_mul(dh[k], t[k])), dx[k]);
          }
        }
        if (out_dx) part.put(out_x, it, dx);
        if (has_block) {
          float2 M[4], a[4];
          float2 *const v = o + 4 * it;
          part.template get<BT>(o_at(at, row), it, v);
          if (P.drop.limit) part.drop(P, key, row, it, dx, slots);
          mul.get(part.chunk(it), M);
          if (gated) part.template get<BT>(row_start<kOdd>(at + to_gate, static_cast<const BT *>(P.gate), row, P.as), it, a);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            v[k] = f2_mul(v[k], ro2);
            const float2 t = f2_mul(dx[k], v[k]);
            float2 f = f2_of(row_gate), slope = f2_of(row_slope);
            if (gated) f = gate_of2(a[k], P.sigmoid, slope);
            const float2 tm = f2_mul(t, M[k]);
            a_all[4 * it + k] = f2_fma(t, f, a_all[4 * it + k]);
            a[k] = f2_mul(tm, slope);
            jg = f2_add(jg, a[k]);
            j0 = f2_fma(tm, f, j0);
            dx[k] = f2_mul(dx[k], f2_mul(f, M[k]));
          }
          if (gated && P.dgate) part.put(out_gate, it, a);
          if (out_do && !post_norm) part.put(out_o, it, dx);
        }
      }
    }
    out_x += x_by, out_gate += gate_by;
    if (!post_norm) out_o += o_by;
    j1 = jg.x + jg.y;
    ring.next();
    sums = make_float4(0.f, 0.f, 0.f, j0.x + j0.y);
    if (row + step < P.n) first_sums(at = ring.take(), row + step, sums);
  }
  if (tid == 0 && ring.gave_up) ring.settle((feed.row - row0) / step);
  const int64_t rows = (int64_t)gridDim.x * P.d;
#pragma unroll
  for (int it = 0; it < kIter; ++it) {
    if (part.here(it)) {
      float *out = P.part + (int64_t)blockIdx.x * P.d;
      if (P.want_pre) part.put(out, it, a_pre + 4 * it), out += rows;
#pragma unroll
      for (int which = 0; which < 2; ++which)
        if (which == 0 ? P.want_post : P.want_scale) {
          float2 v[4];
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const float *const t = which == 0 ? scale : P.post_gain;
            const float one = which == 0 ? s1 : 1.f;
            const int c0 = min(part.column(it, 2 * k), d - 1), c1 = min(part.column(it, 2 * k + 1), d - 1);
            v[k] = f2_mul(a_all[4 * it + k], make_float2(one * table_at(t, c0), one * table_at(t, c1)));
          }
          part.put(out, it, v);
          out += rows;
        }
    }
  }
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

template <typename XT, typename BT, bool kVec>
ResLaunch pick(const ResCut &c, bool all) {
  if (c.form == kFormWide) return launch_res<residual_backward_wide_kernel<XT, BT, kVec>>;
  if (c.form == kFormGroup) return launch_res<residual_backward_kernel<XT, BT, kVec>>;
  if constexpr (!kVec) {
    return launch_res<residual_backward_ring_kernel<XT, BT, 1, true, false>>;
  } else {
    if (all)
      return c.iter == 1 ? launch_res<residual_backward_ring_kernel<XT, BT, 1, false, true>>
                         : launch_res<residual_backward_ring_kernel<XT, BT, 2, false, true>>;
    return c.iter == 1 ? launch_res<residual_backward_ring_kernel<XT, BT, 1, false, false>>
                       : launch_res<residual_backward_ring_kernel<XT, BT, 2, false, false>>;
  }
}

template <bool kVec>
ResLaunch launcher(int32_t xt, int32_t bt, const ResCut &c, bool all) {
  return xt == GBO_BF16 ? pick<__nv_bfloat16, __nv_bfloat16, kVec>(c, all)
                        : bt == GBO_BF16 ? pick<float, __nv_bfloat16, kVec>(c, all) : pick<float, float, kVec>(c, all);
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" size_t gbo_residual_workspace_bytes(int64_t n, int64_t d, int32_t sums) {
  int dev, sm = 0;
  if (n < 0 || d < 1 || d > GBO_RESIDUAL_MAX_D || sums < 0 || sums > 3 || require_device(&dev, &sm) != GBO_OK) return 0;
  return sums ? (size_t)most_parts(n, d, sm) * d * sums * 4 + (size_t)d * 4 : 0;
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
  P.stage_bytes = (int32_t)row_bytes(P, a->x_dtype, a->block_dtype, vec, true);
  const ResCut c = cut_of(a->n, a->d, sm, true, vec, P.stage_bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  const bool all = P.pre && P.post && P.block && P.dxo && P.xo && P.h;
  const ResLaunch launch = vec ? launcher<true>(a->x_dtype, a->block_dtype, c, all) : launcher<false>(a->x_dtype, a->block_dtype, c, all);
  if (a->n > 0 || sums) e = launch(P, c, dev, st);
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


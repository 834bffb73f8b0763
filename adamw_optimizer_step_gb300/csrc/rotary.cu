// Rotary positions and per-head norms of queries and keys, forward and
// backward (gbo_rope_forward, gbo_rope_backward).
//
// One head vector x of D elements, position t, frequencies f_j:
//   forward   u = x / r, r = sqrt(mean x^2 + eps);  y = R_t (gain u)
//   backward  e = R_t^T dy, w = gain e;  dx = (w - x mean(w x) / r^2) / r;
//             dgain_j = sum e_j u_j
// Bound: HBM.  Each element is read once and written once (backward: x and
// dy read, dx written); a head's norm stays in registers and warp shuffles.
//
// Work split.  A head is cut into units of two chunks: the two halves of a
// run of pairs (GBO_ROPE_HALF: 16 bytes at j and 16 at j + rot / 2), two
// consecutive chunks (GBO_ROPE_INTERLEAVED), or two chunks that are only
// copied.  A unit's pairs are thus in one thread, and no rotation crosses
// lanes.  A group of G lanes (a power of two) holds one head, one unit each
// (two for long fp32 heads); it walks over several heads of one token, so the
// cosines and sines of the token are computed once for them.  Shapes whose
// chunks are not 16-byte aligned take the same kernel with one-element
// chunks.
//
// Angles: t f_j in turns is a 64-bit fixed-point product modulo 2^64, exact
// for every 64-bit position; the top 32 bits go to sincospif.  No table of
// cosines is read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "device_common.cuh"
#include "gbo.h"
#include "internal.h"

namespace gbo {

namespace {

constexpr int kRopeThreads = 256;
constexpr int kRopeBackBlocks = 4;  // backward: resident blocks per SM that share out the tokens

struct RopeTensor {
  const void *x, *dy;
  void *y;
  const float *gain;
  float *part;             // backward: dgain partials, nblk rows of D, or NULL
  int64_t xs[3], ds[3], ys[3];
  int32_t heads, norm;
  int32_t per_item;        // heads a group walks over
  int32_t head_blocks;     // ceil(heads / per_item)
  int32_t block0, nblk;    // this tensor's blocks
  int64_t items;           // tokens * head_blocks
};

struct RopeParams {
  RopeTensor t[GBO_ROPE_MAX_TENSORS];
  uint64_t turns[GBO_ROPE_MAX_HEAD_DIM / 2];  // frequencies in turns per position, 64-bit fixed point
  const void *pos;
  int64_t pos_b, pos_s, start, seq;
  float magnitude, eps, inv_dim;
  int32_t n, dim, rot, offset, interleaved, pos64;
  int32_t units, group;
};

template <typename T, int CH>
struct Chunk;  // CH consecutive elements as fp32

template <>
struct Chunk<__nv_bfloat16, 8> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *v) {
    const uint4 raw = *reinterpret_cast<const uint4 *>(p);
    const uint32_t w[4] = {raw.x, raw.y, raw.z, raw.w};
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      v[2 * h] = __uint_as_float(w[h] << 16);
      v[2 * h + 1] = __uint_as_float(w[h] & 0xffff0000u);
    }
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) { store8(p, v, 8, true); }
};
template <>
struct Chunk<float, 4> {
  static __device__ __forceinline__ void load(const float *p, float *v) {
    const float4 f = *reinterpret_cast<const float4 *>(p);
    v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
  }
  static __device__ __forceinline__ void store(float *p, const float *v) {
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  }
};
template <>
struct Chunk<__nv_bfloat16, 1> {
  static __device__ __forceinline__ void load(const __nv_bfloat16 *p, float *v) { v[0] = __bfloat162float(*p); }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float *v) { *p = __float2bfloat16_rn(v[0]); }
};
template <>
struct Chunk<float, 1> {
  static __device__ __forceinline__ void load(const float *p, float *v) { v[0] = *p; }
  static __device__ __forceinline__ void store(float *p, const float *v) { *p = v[0]; }
};

// Element offsets of a unit's two chunks within the head (-1: no such chunk)
// and its first pair (-1: copied, not rotated).
struct Unit {
  int a, b, pair0;
};

template <int CH>
__device__ __forceinline__ Unit unit_of(const RopeParams &P, int u) {
  Unit r = {-1, -1, -1};
  const int rot_units = P.rot / (2 * CH);
  if (u >= P.units) return r;
  if (u < rot_units) {
    r.pair0 = u * CH;
    r.a = P.offset + (P.interleaved ? 2 * CH * u : CH * u);
    r.b = P.interleaved ? r.a + CH : r.a + P.rot / 2;
    return r;
  }
  // copied chunks in order: before the rotated part, then behind it
  const int rest = (P.dim - P.rot) / CH, before = P.offset / CH;
  const int c = 2 * (u - rot_units);
  r.a = c < before ? c * CH : P.rot + c * CH;
  if (c + 1 < rest) r.b = c + 1 < before ? (c + 1) * CH : P.rot + (c + 1) * CH;
  return r;
}

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rotate the unit's pairs in place; sign = -1 turns backwards.
template <int CH>
__device__ __forceinline__ void rotate(float *v, const float *c, const float *s, bool interleaved, float sign) {
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float a = v[2 * i], b = v[2 * i + 1], si = sign * s[i];
      v[2 * i] = a * c[i] - b * si;
      v[2 * i + 1] = a * si + b * c[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      const float a = v[i], b = v[CH + i], si = sign * s[i];
      v[i] = a * c[i] - b * si;
      v[CH + i] = a * si + b * c[i];
    }
  }
}

// UPL: units per lane.  kBack: gradients.
template <typename T, int CH, int UPL, bool kBack>
__global__ void __launch_bounds__(kRopeThreads) rope_kernel(const __grid_constant__ RopeParams P) {
  pdl_launch();
  constexpr int E = 2 * CH;  // elements of a unit
  __shared__ uint64_t turns[GBO_ROPE_MAX_HEAD_DIM / 2];
  __shared__ float gain_s[GBO_ROPE_MAX_HEAD_DIM];
  __shared__ float dg_s[kBack ? GBO_ROPE_MAX_HEAD_DIM : 1];
  int ti = 0;
  while (ti + 1 < P.n && (int)blockIdx.x >= P.t[ti + 1].block0) ++ti;
  const RopeTensor &X = P.t[ti];
  for (int i = threadIdx.x; i < P.rot / 2; i += kRopeThreads) turns[i] = P.turns[i];
  pdl_wait();
  if (X.norm)
    for (int i = threadIdx.x; i < P.dim; i += kRopeThreads) gain_s[i] = X.gain ? X.gain[i] : 1.f;
  __syncthreads();
  const int G = P.group, lane_g = threadIdx.x & (G - 1);
  const int groups = kRopeThreads / G, g = threadIdx.x / G;
  Unit unit[UPL];
#pragma unroll
  for (int k = 0; k < UPL; ++k) unit[k] = unit_of<CH>(P, lane_g + k * G);
  float dg[kBack ? UPL : 1][kBack ? E : 1];
  if constexpr (kBack) {
#pragma unroll
    for (int k = 0; k < UPL; ++k)
#pragma unroll
      for (int i = 0; i < E; ++i) dg[k][i] = 0.f;
  }
  const float sign = kBack ? -1.f : 1.f;
  const bool inter = P.interleaved != 0;
  // every group of a warp runs the same number of rounds (shuffles are warp-wide)
  const int64_t first = (int64_t)((int)blockIdx.x - X.block0) * groups;
  for (int64_t i0 = first; i0 < X.items; i0 += (int64_t)X.nblk * groups) {
    const bool live = i0 + g < X.items;
    const int64_t item = live ? i0 + g : X.items - 1;
    const int64_t tok = item / X.head_blocks;
    const int h0 = (int)(item - tok * X.head_blocks) * X.per_item;
    const int64_t b = tok / P.seq, s = tok - b * P.seq;
    int64_t t;
    if (!P.pos) t = P.start + s;
    else if (P.pos64) t = reinterpret_cast<const int64_t *>(P.pos)[b * P.pos_b + s * P.pos_s];
    else t = reinterpret_cast<const int32_t *>(P.pos)[b * P.pos_b + s * P.pos_s];
    float c[UPL][CH], sn[UPL][CH];
#pragma unroll
    for (int k = 0; k < UPL; ++k)
      if (unit[k].pair0 >= 0) {
#pragma unroll
        for (int i = 0; i < CH; ++i) {
          const int32_t top = (int32_t)((uint64_t)t * turns[unit[k].pair0 + i] >> 32);
          sincospif((float)top * 4.656612873077393e-10f, &sn[k][i], &c[k][i]);  // 2^-31: in half turns
          sn[k][i] *= P.magnitude;
          c[k][i] *= P.magnitude;
        }
      }
    const T *x = reinterpret_cast<const T *>(X.x) + b * X.xs[0] + s * X.xs[1];
    const T *dy = reinterpret_cast<const T *>(X.dy) + b * X.ds[0] + s * X.ds[1];
    T *y = reinterpret_cast<T *>(X.y) + b * X.ys[0] + s * X.ys[1];
    const bool need_x = !kBack || X.norm;
    for (int hh = 0; hh < X.per_item; ++hh) {
      const int h = min(h0 + hh, X.heads - 1);  // past the last head: compute it again, store nothing
      const bool store = live && h0 + hh < X.heads;
      float v[UPL][E], e[kBack ? UPL : 1][kBack ? E : 1];
#pragma unroll
      for (int k = 0; k < UPL; ++k) {
#pragma unroll
        for (int i = 0; i < E; ++i) v[k][i] = 0.f;
        if (need_x) {
          if (unit[k].a >= 0) Chunk<T, CH>::load(x + h * X.xs[2] + unit[k].a, v[k]);
          if (unit[k].b >= 0) Chunk<T, CH>::load(x + h * X.xs[2] + unit[k].b, v[k] + CH);
        }
        if constexpr (kBack) {
#pragma unroll
          for (int i = 0; i < E; ++i) e[k][i] = 0.f;
          if (unit[k].a >= 0) Chunk<T, CH>::load(dy + h * X.ds[2] + unit[k].a, e[k]);
          if (unit[k].b >= 0) Chunk<T, CH>::load(dy + h * X.ds[2] + unit[k].b, e[k] + CH);
          if (unit[k].pair0 >= 0) rotate<CH>(e[k], c[k], sn[k], inter, sign);
        }
      }
      float rho = 1.f;
      if (X.norm) {
        float ss = 0.f;
#pragma unroll
        for (int k = 0; k < UPL; ++k)
#pragma unroll
          for (int i = 0; i < E; ++i) ss = fmaf(v[k][i], v[k][i], ss);
        rho = rsqrtf(group_sum(ss, G) * P.inv_dim + P.eps);
      }
      if constexpr (!kBack) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          if (X.norm) {
#pragma unroll
            for (int i = 0; i < E; ++i) {
              const int at = i < CH ? unit[k].a + i : unit[k].b + i - CH;
              v[k][i] *= rho * gain_s[max(at, 0)];
            }
          }
          if (unit[k].pair0 >= 0) rotate<CH>(v[k], c[k], sn[k], inter, sign);
        }
      } else {
        if (X.norm) {
          float wx = 0.f;
#pragma unroll
          for (int k = 0; k < UPL; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) {
              const int at = i < CH ? unit[k].a + i : unit[k].b + i - CH;
              v[k][i] *= rho;  // u
              if (store) dg[k][i] = fmaf(e[k][i], v[k][i], dg[k][i]);
              e[k][i] *= gain_s[max(at, 0)];  // w
              wx = fmaf(e[k][i], v[k][i], wx);
            }
          wx = group_sum(wx, G) * P.inv_dim;
#pragma unroll
          for (int k = 0; k < UPL; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) v[k][i] = rho * (e[k][i] - v[k][i] * wx);
        } else {
#pragma unroll
          for (int k = 0; k < UPL; ++k)
#pragma unroll
            for (int i = 0; i < E; ++i) v[k][i] = e[k][i];
        }
      }
      if (store) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          if (unit[k].a >= 0) Chunk<T, CH>::store(y + h * X.ys[2] + unit[k].a, v[k]);
          if (unit[k].b >= 0) Chunk<T, CH>::store(y + h * X.ys[2] + unit[k].b, v[k] + CH);
        }
      }
    }
  }
  if constexpr (kBack) {
    if (!X.part) return;
    // the block's groups one after another, so that the order is fixed
    for (int i = threadIdx.x; i < P.dim; i += kRopeThreads) dg_s[i] = 0.f;
    for (int q = 0; q < groups; ++q) {
      __syncthreads();
      if (g == q) {
#pragma unroll
        for (int k = 0; k < UPL; ++k)
#pragma unroll
          for (int i = 0; i < E; ++i) {
            const int at = i < CH ? unit[k].a : unit[k].b;
            if (at >= 0) dg_s[at + (i < CH ? i : i - CH)] += dg[k][i];
          }
      }
    }
    __syncthreads();
    float *out = X.part + (int64_t)((int)blockIdx.x - X.block0) * P.dim;
    for (int i = threadIdx.x; i < P.dim; i += kRopeThreads) out[i] = dg_s[i];
  }
}

struct RopeSum {
  const float *part[GBO_ROPE_MAX_TENSORS];
  float *dgain[GBO_ROPE_MAX_TENSORS];
  int32_t rows[GBO_ROPE_MAX_TENSORS];
  int32_t dim;
};

// dgain[j] = sum of the blocks' partials: 32 columns a block, 32 strands of
// rows, joined in a fixed order.
__global__ void __launch_bounds__(1024) rope_dgain_kernel(const __grid_constant__ RopeSum S) {
  pdl_launch();
  __shared__ float red[32][33];
  const int col = blockIdx.x * 32 + threadIdx.x, ti = blockIdx.y;
  pdl_wait();
  if (!S.dgain[ti]) return;
  float a = 0.f;
  if (col < S.dim)
    for (int r = threadIdx.y; r < S.rows[ti]; r += 32) a += S.part[ti][(int64_t)r * S.dim + col];
  red[threadIdx.y][threadIdx.x] = a;
  __syncthreads();
  const float v = warp_sum(red[threadIdx.x][threadIdx.y]);
  const int out = blockIdx.x * 32 + threadIdx.y;
  if (threadIdx.x == 0 && out < S.dim) S.dgain[ti][out] = v;
}

int rope_fail(int code, const char *msg) { return report_error(code, msg); }

bool ptr_ok(const void *p, int32_t dtype) {
  return (reinterpret_cast<uintptr_t>(p) % (dtype == GBO_BF16 ? 2 : 4)) == 0;
}

int check_opts(const gbo_rope_opts *o) {
  if (!o) return rope_fail(GBO_ERR_INVALID_ARG, "opts is NULL");
  if (o->head_dim < 1 || o->head_dim > GBO_ROPE_MAX_HEAD_DIM)
    return rope_fail(GBO_ERR_SHAPE, "head_dim must be in 1..512");
  if (o->rot_dim < 0 || (o->rot_dim & 1)) return rope_fail(GBO_ERR_SHAPE, "rot_dim must be even and >= 0");
  if (o->offset < 0 || o->offset > o->head_dim || o->rot_dim > o->head_dim - o->offset)
    return rope_fail(GBO_ERR_SHAPE, "the rotated part does not lie within the head");
  if (o->layout != GBO_ROPE_HALF && o->layout != GBO_ROPE_INTERLEAVED)
    return rope_fail(GBO_ERR_INVALID_ARG, "layout must be GBO_ROPE_HALF or GBO_ROPE_INTERLEAVED");
  if (o->rot_dim > 0 && !o->freq) return rope_fail(GBO_ERR_INVALID_ARG, "freq is NULL");
  for (int j = 0; j < o->rot_dim / 2; ++j)
    if (!std::isfinite(o->freq[j])) return rope_fail(GBO_ERR_INVALID_ARG, "non-finite frequency");
  if (!std::isfinite(o->magnitude) || !(o->eps >= 0.f) || !std::isfinite(o->eps))
    return rope_fail(GBO_ERR_INVALID_ARG, "non-finite magnitude, or eps < 0 or not finite");
  return GBO_OK;
}

// Blocks that share a backward call's tokens over its tensors, in
// proportion to their heads (a function of the table and the device alone,
// so that dgain's order of summation does not change from call to call).
void back_blocks(const gbo_rope_tensor *t, int32_t n, int sm_count, int32_t *nblk) {
  int64_t heads = 0;
  for (int32_t i = 0; i < n; ++i) heads += t[i].heads;
  for (int32_t i = 0; i < n; ++i)
    nblk[i] = heads == 0 || t[i].heads == 0
                  ? 0
                  : (int32_t)std::max<int64_t>(1, (int64_t)kRopeBackBlocks * sm_count * t[i].heads / heads);
}

template <typename T, int CH, int UPL, bool kBack>
cudaError_t launch_rope(const RopeParams &P, int blocks, cudaStream_t stream) {
  return launch_kernel(rope_kernel<T, CH, UPL, kBack>, dim3(blocks), dim3(kRopeThreads), 0, stream, 1, P);
}

template <typename T, bool kBack>
cudaError_t dispatch_rope(const RopeParams &P, int chunk, int upl, int blocks, cudaStream_t stream) {
  constexpr int V = 16 / (int)sizeof(T);
  if (chunk == 1) {
    return upl <= 2 ? launch_rope<T, 1, 2, kBack>(P, blocks, stream) : launch_rope<T, 1, 8, kBack>(P, blocks, stream);
  }
  return upl == 1 ? launch_rope<T, V, 1, kBack>(P, blocks, stream) : launch_rope<T, V, 2, kBack>(P, blocks, stream);
}

int rope_run(const gbo_rope_tensor *tensors, int32_t n, const gbo_rope_opts *o, int64_t batch, int64_t seq,
             const gbo_rope_positions *pos, bool back, void *workspace, size_t ws_bytes, gbo_stream_t stream) {
  if (n < 0 || n > GBO_ROPE_MAX_TENSORS || (n > 0 && !tensors))
    return rope_fail(GBO_ERR_INVALID_ARG, "between 0 and 4 tensors per call");
  int rc = check_opts(o);
  if (rc != GBO_OK) return rc;
  if (batch < 0 || seq < 0 || (seq > 0 && batch > INT64_MAX / GBO_ROPE_MAX_HEAD_DIM / seq))
    return rope_fail(GBO_ERR_SHAPE, "batch or seq negative or too large");
  if (pos && pos->ptr) {
    if (pos->dtype != GBO_I32 && pos->dtype != GBO_I64)
      return rope_fail(GBO_ERR_DTYPE, "positions must be GBO_I32 or GBO_I64");
    if (reinterpret_cast<uintptr_t>(pos->ptr) % (pos->dtype == GBO_I64 ? 8 : 4))
      return rope_fail(GBO_ERR_INVALID_ARG, "positions misaligned");
  }
  bool any_dgain = false, chunks16 = true;
  int32_t dtype = n > 0 ? tensors[0].dtype : GBO_BF16;
  const bool none = n == 0 || batch == 0 || seq == 0;
  for (int32_t i = 0; i < n; ++i) {
    const gbo_rope_tensor &t = tensors[i];
    if (t.dtype != GBO_F32 && t.dtype != GBO_BF16) return rope_fail(GBO_ERR_DTYPE, "dtype must be GBO_F32 or GBO_BF16");
    if (t.dtype != dtype) return rope_fail(GBO_ERR_DTYPE, "the tensors of one call have one dtype");
    if (t.heads < 0) return rope_fail(GBO_ERR_SHAPE, "negative number of heads");
    if (t.norm != 0 && t.norm != 1) return rope_fail(GBO_ERR_INVALID_ARG, "norm must be 0 or 1");
    if (!t.norm && (t.gain || t.dgain)) return rope_fail(GBO_ERR_INVALID_ARG, "a gain without a norm");
    if (!back && (t.dgain || t.dy)) return rope_fail(GBO_ERR_INVALID_ARG, "dy and dgain belong to the backward pass");
    if (!ptr_ok(t.gain, GBO_F32) || !ptr_ok(t.dgain, GBO_F32))
      return rope_fail(GBO_ERR_INVALID_ARG, "misaligned gain");
    any_dgain |= t.dgain != nullptr;
    if (none || t.heads == 0) continue;
    const bool need_x = !back || t.norm;
    if (!t.y || (need_x && !t.x) || (back && !t.dy)) return rope_fail(GBO_ERR_INVALID_ARG, "NULL tensor pointer");
    if (!ptr_ok(t.x, dtype) || !ptr_ok(t.dy, dtype) || !ptr_ok(t.y, dtype))
      return rope_fail(GBO_ERR_INVALID_ARG, "misaligned tensor pointer");
    // 16-byte chunks need 16-byte aligned heads
    const int V = dtype == GBO_BF16 ? 8 : 4;
    const void *ptrs[3] = {need_x ? t.x : nullptr, back ? t.dy : nullptr, t.y};
    const int64_t *strides[3] = {t.x_stride, t.dy_stride, t.y_stride};
    for (int k = 0; k < 3; ++k) {
      if (!ptrs[k]) continue;
      if (reinterpret_cast<uintptr_t>(ptrs[k]) & 15) chunks16 = false;
      if ((batch > 1 && strides[k][0] % V) || (seq > 1 && strides[k][1] % V) || (t.heads > 1 && strides[k][2] % V))
        chunks16 = false;
    }
  }
  int dev, sm = 0;
  if ((rc = require_device(&dev, &sm)) != GBO_OK) return rc;
  if (any_dgain) {
    if (!workspace || ws_bytes < gbo_rope_workspace_bytes(tensors, n, o))
      return rope_fail(GBO_ERR_WORKSPACE, "workspace missing or smaller than gbo_rope_workspace_bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 15) return rope_fail(GBO_ERR_WORKSPACE, "workspace must be 16-byte aligned");
  }

  RopeParams P;
  memset(&P, 0, sizeof P);
  const int V = dtype == GBO_BF16 ? 8 : 4;
  // a unit is two chunks: pairs have to fill whole units
  const bool vec = chunks16 && o->head_dim % V == 0 && o->offset % V == 0 && o->rot_dim % (2 * V) == 0;
  const int CH = vec ? V : 1;
  P.units = o->rot_dim / (2 * CH) + ((o->head_dim - o->rot_dim) / CH + 1) / 2;
  P.group = 1;
  while (P.group < 32 && P.group < P.units) P.group *= 2;
  const int upl = (P.units + P.group - 1) / P.group;
  P.dim = o->head_dim, P.rot = o->rot_dim, P.offset = o->offset;
  P.interleaved = o->layout == GBO_ROPE_INTERLEAVED;
  P.magnitude = o->magnitude, P.eps = o->eps, P.inv_dim = 1.f / (float)o->head_dim;
  P.seq = std::max<int64_t>(seq, 1);
  if (pos) {
    P.pos = pos->ptr, P.pos_b = pos->stride_b, P.pos_s = pos->stride_s, P.start = pos->start;
    P.pos64 = pos->dtype == GBO_I64;
  }
  for (int j = 0; j < o->rot_dim / 2; ++j) {
    const double turn = o->freq[j] / 6.283185307179586476925286766559;
    const double frac = turn - std::floor(turn);  // [0, 1], 1 only by rounding
    P.turns[j] = frac >= 1.0 ? 0 : (uint64_t)std::ldexp(frac, 64);
  }
  P.n = 0;
  const int groups = kRopeThreads / P.group;
  const int64_t tokens = batch * seq;
  int32_t nblk[GBO_ROPE_MAX_TENSORS] = {};
  if (back) back_blocks(tensors, n, sm, nblk);
  int64_t all_heads = 0;
  for (int32_t i = 0; i < n; ++i) all_heads += tensors[i].heads;
  // heads a group walks over: up to 8 while the groups still fill the device
  // (four 256-thread blocks an SM), so that a token's cosines are shared
  int32_t per_item = 1;
  while (per_item < 8 && tokens * all_heads / (2 * per_item) >= (int64_t)sm * 4 * groups) per_item *= 2;
  float *part = static_cast<float *>(workspace);
  RopeSum S;
  memset(&S, 0, sizeof S);
  S.dim = o->head_dim;
  int64_t blocks = 0;
  for (int32_t i = 0; i < n; ++i) {
    const gbo_rope_tensor &t = tensors[i];
    const bool live = !none && t.heads > 0;
    if (back && t.dgain) {
      S.dgain[i] = t.dgain;
      S.part[i] = part;
    }
    if (live) {
      RopeTensor &X = P.t[P.n++];
      X.x = t.x, X.dy = t.dy, X.y = t.y, X.gain = t.gain;
      for (int k = 0; k < 3; ++k) X.xs[k] = t.x_stride[k], X.ds[k] = t.dy_stride[k], X.ys[k] = t.y_stride[k];
      X.heads = t.heads, X.norm = t.norm;
      X.head_blocks = (t.heads + per_item - 1) / per_item;
      X.per_item = (t.heads + X.head_blocks - 1) / X.head_blocks;
      X.items = tokens * X.head_blocks;
      const int64_t want = (X.items + groups - 1) / groups;
      const int64_t take = back ? std::min<int64_t>(want, nblk[i]) : std::min<int64_t>(want, 1 << 20);
      X.block0 = (int32_t)blocks;
      X.nblk = (int32_t)take;
      blocks += take;
      if (back && t.dgain) {
        X.part = part;
        S.rows[i] = X.nblk;
      }
    }
    if (back && t.dgain) part += (int64_t)nblk[i] * o->head_dim;
  }
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t err = cudaSuccess;
  if (blocks > 0) {
    if (dtype == GBO_BF16)
      err = back ? dispatch_rope<__nv_bfloat16, true>(P, CH, upl, (int)blocks, st)
                 : dispatch_rope<__nv_bfloat16, false>(P, CH, upl, (int)blocks, st);
    else
      err = back ? dispatch_rope<float, true>(P, CH, upl, (int)blocks, st)
                 : dispatch_rope<float, false>(P, CH, upl, (int)blocks, st);
    count_launches(1);
  }
  if (err == cudaSuccess && any_dgain) {
    err = launch_kernel(rope_dgain_kernel, dim3((o->head_dim + 31) / 32, n), dim3(32, 32), 0, st, 1, S);
    count_launches(1);
  }
  if (err != cudaSuccess) {
    char msg[200];
    snprintf(msg, sizeof msg, "rotary kernels: %s", cudaGetErrorString(err));
    return rope_fail(GBO_ERR_CUDA, msg);
  }
  return report_ok();
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" int gbo_rope_frequencies(int32_t rot_dim, double base, const gbo_rope_scaling *s, double *freq,
                                    double *magnitude) {
  if (rot_dim < 2 || (rot_dim & 1) || rot_dim > GBO_ROPE_MAX_HEAD_DIM)
    return rope_fail(GBO_ERR_SHAPE, "rot_dim must be even and in 2..512");
  if (!freq || !magnitude) return rope_fail(GBO_ERR_INVALID_ARG, "NULL output");
  if (!(base > 0.0) || !std::isfinite(base)) return rope_fail(GBO_ERR_INVALID_ARG, "base must be > 0 and finite");
  const int32_t kind = s ? s->kind : GBO_ROPE_SCALE_NONE;
  if (kind < GBO_ROPE_SCALE_NONE || kind > GBO_ROPE_SCALE_WAVELENGTH)
    return rope_fail(GBO_ERR_INVALID_ARG, "unknown kind of scaling");
  if (kind != GBO_ROPE_SCALE_NONE && !(s->factor > 0.0 && std::isfinite(s->factor)))
    return rope_fail(GBO_ERR_INVALID_ARG, "factor must be > 0 and finite");
  if (kind == GBO_ROPE_SCALE_NTK && rot_dim == 2)
    return rope_fail(GBO_ERR_SHAPE, "a changed base needs more than one pair");
  if (kind == GBO_ROPE_SCALE_YARN && !(base != 1.0))
    return rope_fail(GBO_ERR_INVALID_ARG, "base 1 gives one frequency: nothing to stretch by index");
  if ((kind == GBO_ROPE_SCALE_YARN || kind == GBO_ROPE_SCALE_WAVELENGTH) &&
      !(s->trained > 0.0 && std::isfinite(s->trained) && s->slow > 0.0 && s->fast > s->slow && std::isfinite(s->fast)))
    return rope_fail(GBO_ERR_INVALID_ARG, "trained > 0 and fast > slow > 0 are needed");
  const double two_pi = 6.283185307179586476925286766559;
  const int half = rot_dim / 2;
  double b = base;
  if (kind == GBO_ROPE_SCALE_NTK) b = base * std::pow(s->factor, rot_dim / (rot_dim - 2.0));
  *magnitude = kind == GBO_ROPE_SCALE_YARN ? 0.1 * std::log(s->factor) + 1.0 : 1.0;
  double low = 0.0, high = 0.0;
  if (kind == GBO_ROPE_SCALE_YARN) {
    auto index_at = [&](double turns) {
      return rot_dim * std::log(s->trained / (turns * two_pi)) / (2.0 * std::log(base));
    };
    low = std::max(std::floor(index_at(s->fast)), 0.0);
    high = std::min(std::ceil(index_at(s->slow)), rot_dim - 1.0);
  }
  for (int j = 0; j < half; ++j) {
    const double f = std::pow(b, -2.0 * j / rot_dim);
    if (kind == GBO_ROPE_SCALE_LINEAR) {
      freq[j] = f / s->factor;
    } else if (kind == GBO_ROPE_SCALE_YARN) {
      const double w = std::min(std::max((j - low) / std::max(high - low, 1e-3), 0.0), 1.0);
      freq[j] = f * (1.0 - w) + f / s->factor * w;
    } else if (kind == GBO_ROPE_SCALE_WAVELENGTH) {
      const double turns = s->trained * f / two_pi;
      const double keep = std::min(std::max((turns - s->slow) / (s->fast - s->slow), 0.0), 1.0);
      freq[j] = f * keep + f / s->factor * (1.0 - keep);
    } else {
      freq[j] = f;
    }
  }
  return report_ok();
}

extern "C" size_t gbo_rope_workspace_bytes(const gbo_rope_tensor *tensors, int32_t n, const gbo_rope_opts *opts) {
  if (!tensors || !opts || n < 1 || n > GBO_ROPE_MAX_TENSORS || opts->head_dim < 1) return 0;
  int dev, sm = 0;
  if (require_device(&dev, &sm) != GBO_OK) return 0;
  int32_t nblk[GBO_ROPE_MAX_TENSORS] = {};
  back_blocks(tensors, n, sm, nblk);
  size_t rows = 0;
  for (int32_t i = 0; i < n; ++i)
    if (tensors[i].dgain) rows += (size_t)nblk[i];
  return rows * (size_t)opts->head_dim * sizeof(float);
}

extern "C" int gbo_rope_forward(const gbo_rope_tensor *tensors, int32_t n, const gbo_rope_opts *opts, int64_t batch,
                                int64_t seq, const gbo_rope_positions *positions, gbo_stream_t stream) {
  return rope_run(tensors, n, opts, batch, seq, positions, false, nullptr, 0, stream);
}

extern "C" int gbo_rope_backward(const gbo_rope_tensor *tensors, int32_t n, const gbo_rope_opts *opts, int64_t batch,
                                 int64_t seq, const gbo_rope_positions *positions, void *workspace, size_t ws_bytes,
                                 gbo_stream_t stream) {
  return rope_run(tensors, n, opts, batch, seq, positions, true, workspace, ws_bytes, stream);
}

// Rotary positions and per-head norms of queries and keys, forward and
// backward (gbo_rope_forward, gbo_rope_backward).
//
// One head vector x of D elements, position t, frequencies f_j:
//   forward   u = x / r, r = sqrt(mean x^2 + eps);  y = R_t (gain u)
//   backward  e = R_t^T dy, w = gain e;  dx = (w - x mean(w x) / r^2) / r;
//             dgain_j = sum e_j u_j
// Bound: HBM.  Each element is read once and written once (backward: x and
// dy read, dx written); a head's norm stays in registers and warp shuffles.
// Measured on 32768 tokens x 20 heads of 128 in bf16: forward 54 us, 6.2 TB/s
// (91% of a copy); backward 90 us, 5.6 TB/s; 32768 x 32 heads of 192 with 64
// rotated and no norm: 117 us, 6.9 TB/s.  What carried the forward there from
// 88 us: the asynchronous ring (heads in flight without registers), two fp32
// lanes per instruction, hardware sines for bf16, 32-bit index division.  The
// bf16 forward with a norm holds to 64 registers for four blocks an SM, for
// which it spills 20 bytes: with 79, unspilled, three blocks take 57.1 us
// instead of 54.5.  The backward's 113 registers leave 16 warps an SM; at 80
// (24 warps) it spills and measured 127 us.  Carrying the ring on into the
// next item, sines kept negated in registers and sums without loops were
// slower or no faster; as many blocks as are resident, which loop, 67 us
// forward.
//
// Work split.  A head is cut into units of two 16-byte chunks: the two halves
// of a run of pairs (GBO_ROPE_HALF), two chunks of whole pairs
// (GBO_ROPE_INTERLEAVED), or two chunks that are only copied.  A unit's pairs
// are thus in one thread, and no rotation crosses lanes.  Heads, rotated parts
// or addresses that 16 bytes do not divide take chunks of 8 or 4 bytes, or of
// one element, in the same kernel.  A group of G lanes (a power of two) holds
// one head, one unit each (more for long heads in narrow chunks); it walks
// over several heads of one token, so the cosines and sines of the token are
// computed once for them.
//
// Angles: t f_j in turns is a 64-bit fixed-point product modulo 2^64, which
// rounds nothing for any 64-bit position; its top 32 bits are the angle
// (turn_of).  What is rounded is the factor, f_j / 2 pi (turns_of).  No table
// of cosines is read.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <cmath>
#include <cstdio>
#include <cstring>

#include "device_common.cuh"
#include "gbo.h"
#include "internal.h"
#include "per_device.h"

namespace gbo {

namespace {

// Threads of a block.  The gradients of a norm, whose 113 registers leave 16
// warps an SM either way, take their tokens in smaller blocks: 64 / 128 / 256
// threads 95 / 92 / 95 us (32768 tokens x 20 heads of 128 in bf16); forward
// 63 / 58 / 56.
constexpr int rope_threads(bool norm, bool back) { return norm && back ? 128 : 256; }
// Gradients of a norm: blocks per SM that share out the tokens (each leaves
// one row of partial gain gradients), four of them resident: 4 / 6 / 8 / 10 /
// 12 / 16 measured 91 / 102 / 88 / 94 / 88 / 89 us on the same tokens, 4 / 8 /
// 12 / 16 87 / 88 / 83 / 83 on 16384 in fp32.
constexpr int kRopeBackBlocks = 12;
// Heads a group walks over at most: 2 / 4 / 8 / 16 measured 111 / 67 / 57 / 58
// us forward on the same tokens.
constexpr int kMaxHeads = 8;

struct RopeTensor {
  const void *x, *dy;
  void *y;
  const float *gain;
  float *part;             // backward: dgain partials, nblk rows of D, or NULL
  int64_t xs[3], ds[3], ys[3];
  int32_t heads;
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

// Two fp32 values that are computed together (one instruction on sm_100 and up).
__device__ __forceinline__ uint64_t bits2(float2 a) { return *reinterpret_cast<uint64_t *>(&a); }
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  uint64_t d;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)), "l"(bits2(c)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  uint64_t d;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(d) : "l"(bits2(a)), "l"(bits2(b)));
  return *reinterpret_cast<float2 *>(&d);
}
__device__ __forceinline__ float2 twice(float a) { return make_float2(a, a); }

// A unit's two chunks of CH elements each, as CH pairs of fp32: the elements
// in order (first chunk, then second).  A chunk is 16, 8 or 4 bytes, or one
// element.
template <typename T, int CH>
struct Chunks {  // CH = 1
  static __device__ __forceinline__ void load(const T *a, const T *b, float2 *v) {
    v[0] = make_float2(a ? (float)*a : 0.f, b ? (float)*b : 0.f);
  }
  static __device__ __forceinline__ void store(T *p, const float2 *v, int which) { *p = (T)(which ? v[0].y : v[0].x); }
};

template <int kWords>
struct Words {
  uint32_t w[kWords];
};

template <int kWords>
__device__ __forceinline__ Words<kWords> lds_words(uint32_t from) {
  Words<kWords> r;
  if constexpr (kWords == 4)
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r.w[0]), "=r"(r.w[1]), "=r"(r.w[2]), "=r"(r.w[3]) : "r"(from) : "memory");
  else if constexpr (kWords == 2)
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(from) : "memory");
  else
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(r.w[0]) : "r"(from) : "memory");
  return r;
}

template <int kWords>
__device__ __forceinline__ void stg_words(void *p, const Words<kWords> &r) {
  if constexpr (kWords == 4) *reinterpret_cast<uint4 *>(p) = make_uint4(r.w[0], r.w[1], r.w[2], r.w[3]);
  else if constexpr (kWords == 2) *reinterpret_cast<uint2 *>(p) = make_uint2(r.w[0], r.w[1]);
  else *reinterpret_cast<uint32_t *>(p) = r.w[0];
}

template <int CH>
struct VecChunks16 {  // bf16: two elements a word
  static constexpr int kWords = CH / 2;
  static __device__ __forceinline__ void unpack(const Words<kWords> &raw, float2 *o) {
#pragma unroll
    for (int h = 0; h < kWords; ++h)
      o[h] = make_float2(__uint_as_float(raw.w[h] << 16), __uint_as_float(raw.w[h] & 0xffff0000u));
  }
  static __device__ __forceinline__ void store(__nv_bfloat16 *p, const float2 *v, int which) {
    Words<kWords> r;
#pragma unroll
    for (int h = 0; h < kWords; ++h) {
      const __nv_bfloat162 q = __float22bfloat162_rn(v[kWords * which + h]);
      r.w[h] = *reinterpret_cast<const uint32_t *>(&q);
    }
    stg_words<kWords>(p, r);
  }
};
template <int CH>
struct VecChunks32 {  // fp32
  static constexpr int kWords = CH;
  static __device__ __forceinline__ void unpack(const Words<kWords> &raw, float2 *o) {
#pragma unroll
    for (int h = 0; h < CH / 2; ++h) o[h] = make_float2(__uint_as_float(raw.w[2 * h]), __uint_as_float(raw.w[2 * h + 1]));
  }
  static __device__ __forceinline__ void store(float *p, const float2 *v, int which) {
    Words<kWords> r;
#pragma unroll
    for (int h = 0; h < CH / 2; ++h) {
      r.w[2 * h] = __float_as_uint(v[CH / 2 * which + h].x);
      r.w[2 * h + 1] = __float_as_uint(v[CH / 2 * which + h].y);
    }
    stg_words<kWords>(p, r);
  }
};
template <> struct Chunks<__nv_bfloat16, 8> : VecChunks16<8> {};
template <> struct Chunks<__nv_bfloat16, 4> : VecChunks16<4> {};
template <> struct Chunks<__nv_bfloat16, 2> : VecChunks16<2> {};
template <> struct Chunks<float, 4> : VecChunks32<4> {};
template <> struct Chunks<float, 2> : VecChunks32<2> {};

// One chunk to shared memory (16 bytes pass L1 by: neighbouring lanes fill
// whole sectors; narrower ones share lines with their neighbours' in L1).
template <int kBytes>
__device__ __forceinline__ void copy_async(uint32_t dst, const void *src) {
  if constexpr (kBytes == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(kBytes) : "memory");
}

// Cosine and sine of a 32-bit fraction of a turn (signed).  For bf16 outputs
// the hardware's approximation is enough: its error, 2^-21 for arguments
// within half a turn, is 2^-12 of the output's rounding.
template <typename T>
__device__ __forceinline__ void turn_of(int32_t top, float &c, float &s) {
  const float half_turns = (float)top * 4.656612873077393e-10f;  // 2^-31
  if constexpr (sizeof(T) == 2) {
    __sincosf(half_turns * 3.14159265358979f, &s, &c);
  } else {
    sincospif(half_turns, &s, &c);
  }
}

// A unit: element offsets of its two chunks within the head (-1: no such
// chunk), and the first pairs of its first and second CH / 2 pairs (-1:
// copied, not rotated).  The second chunks lie half the rotated part (half
// the copied chunks) behind the first, so that consecutive lanes read and
// write consecutive chunks; interleaved pairs are whole within a chunk.
struct Unit {
  int a, b, pair0, pair1;
};

template <int CH>
__device__ __forceinline__ Unit unit_of(const RopeParams &P, int u) {
  Unit r = {-1, -1, -1, -1};
  const int rot_units = P.rot / (2 * CH);
  if (u >= P.units) return r;
  if (u < rot_units) {
    if (CH == 1) {
      r.pair0 = u;
      r.a = P.offset + (P.interleaved ? 2 * u : u);
      r.b = P.interleaved ? r.a + 1 : r.a + P.rot / 2;
      return r;
    }
    r.a = P.offset + CH * u;
    r.b = r.a + P.rot / 2;
    r.pair0 = P.interleaved ? CH / 2 * u : CH * u;
    r.pair1 = P.interleaved ? P.rot / 4 + CH / 2 * u : CH * u + CH / 2;
    return r;
  }
  // copied chunks in order: before the rotated part, then behind it
  const int rest = (P.dim - P.rot) / CH, before = P.offset / CH, half = (rest + 1) / 2;
  auto at = [&](int c) { return c < before ? c * CH : P.rot + c * CH; };
  const int c = u - rot_units;
  r.a = at(c);
  if (c + half < rest) r.b = at(c + half);
  return r;
}

__device__ __forceinline__ float group_sum(float v, int group) {
  for (int o = group >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  return v;
}

// Rotate the unit's CH pairs in place (copied units have c = 1, s = 0).  c
// and s are in the order of the pairs, two and two.  With one-element
// chunks both layouts are one (a, b).
template <int CH>
__device__ __forceinline__ void rotate(float2 *v, const float2 *c, const float2 *s, bool interleaved) {
  if (CH == 1 || interleaved) {
#pragma unroll
    for (int i = 0; i < CH; ++i) {  // (a, b) c + (b, a) (-s, s)
      const float ci = i & 1 ? c[i / 2].y : c[i / 2].x, si = i & 1 ? s[i / 2].y : s[i / 2].x;
      v[i] = fma2(make_float2(v[i].y, v[i].x), make_float2(-si, si), mul2(v[i], twice(ci)));
    }
  } else {
#pragma unroll
    for (int i = 0; i < CH / 2; ++i) {
      const float2 a = v[i], b = v[CH / 2 + i];
      v[i] = fma2(make_float2(-b.x, -b.y), s[i], mul2(a, c[i]));
      v[CH / 2 + i] = fma2(b, c[i], mul2(a, s[i]));
    }
  }
}

constexpr int ring_depth(int ch) { return ch == 1 ? 0 : 4; }
// Bytes of a block's ring: per head in flight, x and / or dy, UPL units of two chunks a thread.
constexpr int ring_bytes(int chunk_bytes, int ch, int upl, bool norm, bool back) {
  return ring_depth(ch) * (norm && back ? 2 : 1) * upl * 2 * chunk_bytes * rope_threads(norm, back);
}

// UPL: units per lane.  kNorm: with the per-head norm.  kBack: gradients.
// kNorm wants the group to be a power of two (its sums are butterflies);
// without it a group is exactly the head's units.
//
// Heads on their way in are asynchronous copies, chunk by chunk, into a ring of
// shared memory in which every thread has slots of its own, so no thread
// waits for another and the loads in flight take no registers: kDepth heads a
// thread (forward 2 / 3 / 4: 60 / 58 / 57 us; backward 2 / 3 / 4: 97 / 95 / 94).
template <typename T, int CH, int UPL, bool kNorm, bool kBack>
__global__ void __launch_bounds__(rope_threads(kNorm, kBack), CH == 1 || UPL > 1 ? 1 : 4)
    rope_kernel(const __grid_constant__ RopeParams P) {
  pdl_launch();
  constexpr int kThreads = rope_threads(kNorm, kBack);
  constexpr bool kGrad = kNorm && kBack;
  constexpr bool kUseX = kNorm || !kBack;
  constexpr int kDepth = ring_depth(CH);
  constexpr int kIn = kGrad ? 2 : 1;           // tensors read
  constexpr int H2 = (CH + 1) / 2;             // CH cosines, two and two
  extern __shared__ __align__(16) uint8_t ring[];
  __shared__ uint64_t turns[GBO_ROPE_MAX_HEAD_DIM / 2];
  __shared__ __align__(16) float gain_s[kGrad ? GBO_ROPE_MAX_HEAD_DIM : 4];
  __shared__ float dg_s[kGrad ? GBO_ROPE_MAX_HEAD_DIM : 1];
  int ti = 0;
  while (ti + 1 < P.n && (int)blockIdx.x >= P.t[ti + 1].block0) ++ti;
  const RopeTensor &X = P.t[ti];
  for (int i = threadIdx.x; i < P.rot / 2; i += kThreads) turns[i] = P.turns[i];
  const int G = P.group, g = threadIdx.x / G, lane_g = threadIdx.x - g * G;
  const int groups = kThreads / G;
  Unit unit[UPL];
#pragma unroll
  for (int k = 0; k < UPL; ++k) {
    unit[k] = unit_of<CH>(P, lane_g + k * G);
    if (!kNorm && g >= groups) unit[k] = {-1, -1, -1, -1};  // the block's last threads, too few for a group
  }
  constexpr int kBytes = CH * (int)sizeof(T);  // of a chunk
  const uint32_t slot0 = (uint32_t)__cvta_generic_to_shared(ring) + threadIdx.x * kBytes;
  constexpr uint32_t kPiece = kThreads * kBytes;
  auto slot = [&](int d, int in, int k, int which) { return slot0 + (uint32_t)(((d * kIn + in) * UPL + k) * 2 + which) * kPiece; };
  if constexpr (kDepth > 0) {  // chunks that a unit lacks stay zero
    bool lacks = false;
#pragma unroll
    for (int k = 0; k < UPL; ++k) lacks |= unit[k].a < 0 || unit[k].b < 0;
    if (lacks)
      for (int p = 0; p < kDepth * kIn * UPL * 2; ++p)
#pragma unroll
        for (int w = 0; w < kBytes; w += 4)
          asm volatile("st.shared.b32 [%0], %1;" ::"r"(slot0 + p * kPiece + w), "r"(0) : "memory");
  }
  pdl_wait();
  // the lane's gains: in registers, or, in the backward pass, which needs
  // those for its sums, in shared memory
  auto gain_at = [&](int k, int i) {  // element i of the unit's 2 CH
    const int at = i < CH ? unit[k].a : unit[k].b;
    return at >= 0 && X.gain ? X.gain[at + (i < CH ? i : i - CH)] : 1.f;
  };
  float2 gain_r[kNorm && !kBack ? UPL : 1][CH], dg[kGrad ? UPL : 1][CH];
  if constexpr (kNorm && !kBack) {
#pragma unroll
    for (int k = 0; k < UPL; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i) gain_r[k][i] = make_float2(gain_at(k, 2 * i), gain_at(k, 2 * i + 1));
  }
  if constexpr (kGrad) {
    for (int i = threadIdx.x; i < P.dim; i += kThreads) gain_s[i] = X.gain ? X.gain[i] : 1.f;
#pragma unroll
    for (int k = 0; k < UPL; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i) dg[k][i] = make_float2(0.f, 0.f);
  }
  __syncthreads();
  const bool inter = P.interleaved != 0;
  // every group of a warp runs the same number of rounds (shuffles are warp-wide)
  const int64_t first = (int64_t)((int)blockIdx.x - X.block0) * groups;
  for (int64_t i0 = first; i0 < X.items; i0 += (int64_t)X.nblk * groups) {
    const bool live = g < groups && i0 + g < X.items;
    const int64_t item = live ? i0 + g : X.items - 1;
    int64_t tok, b;
    if (X.items <= 0x7fffffff) {  // 32-bit division: a third of the instructions
      tok = (uint32_t)item / (uint32_t)X.head_blocks;
      b = (uint32_t)tok / (uint32_t)min(P.seq, (int64_t)0x7fffffff);
    } else {
      tok = item / X.head_blocks;
      b = tok / P.seq;
    }
    const int h0 = (int)(item - tok * X.head_blocks) * X.per_item;
    const int64_t s = tok - b * P.seq;
    // heads of this item (0: the group has none); groups with fewer heads
    // than the others go through the rounds all the same, and store nothing
    const int nh = live ? min(X.per_item, X.heads - h0) : 0;
    const T *x = reinterpret_cast<const T *>(X.x) + b * X.xs[0] + s * X.xs[1] + h0 * X.xs[2];
    const T *dy = reinterpret_cast<const T *>(X.dy) + b * X.ds[0] + s * X.ds[1] + h0 * X.ds[2];
    T *y = reinterpret_cast<T *>(X.y) + b * X.ys[0] + s * X.ys[1] + h0 * X.ys[2];
    auto request = [&](int d, bool there) {  // the next head's copies, into slots d
      if (there) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          if constexpr (kUseX) {
            if (unit[k].a >= 0) copy_async<kBytes>(slot(d, 0, k, 0), x + unit[k].a);
            if (unit[k].b >= 0) copy_async<kBytes>(slot(d, 0, k, 1), x + unit[k].b);
          }
          if constexpr (kBack) {
            if (unit[k].a >= 0) copy_async<kBytes>(slot(d, kIn - 1, k, 0), dy + unit[k].a);
            if (unit[k].b >= 0) copy_async<kBytes>(slot(d, kIn - 1, k, 1), dy + unit[k].b);
          }
        }
        if constexpr (kUseX) x += X.xs[2];
        if constexpr (kBack) dy += X.ds[2];
      }
      asm volatile("cp.async.commit_group;" ::: "memory");
    };
    if constexpr (kDepth > 0) {
#pragma unroll
      for (int d = 0; d < kDepth; ++d) request(d, d < nh);
    }
    int64_t t;
    if (!P.pos) t = P.start + s;
    else if (P.pos64) t = reinterpret_cast<const int64_t *>(P.pos)[b * P.pos_b + s * P.pos_s];
    else t = reinterpret_cast<const int32_t *>(P.pos)[b * P.pos_b + s * P.pos_s];
    float2 c[UPL][H2], sn[UPL][H2];
#pragma unroll
    for (int k = 0; k < UPL; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        float ci = 1.f, si = 0.f;
        if (unit[k].pair0 >= 0) {
          turn_of<T>((int32_t)((uint64_t)t * turns[i < CH / 2 || CH == 1 ? unit[k].pair0 + i : unit[k].pair1 + i - CH / 2] >> 32), ci, si);
          ci *= P.magnitude;
          si *= kBack ? -P.magnitude : P.magnitude;
        }
        if (i & 1) c[k][i / 2].y = ci, sn[k][i / 2].y = si;
        else c[k][i / 2].x = ci, sn[k][i / 2].x = si;
      }
    int d = 0;
    for (int hh = 0; hh < X.per_item; ++hh) {
      const bool store = hh < nh;
      float2 v[kUseX ? UPL : 1][CH], e[kBack ? UPL : 1][CH];
      if constexpr (kDepth > 0) {
        asm volatile("cp.async.wait_group %0;" ::"n"(kDepth - 1) : "memory");
        auto take = [&](uint32_t from, float2 *o) { Chunks<T, CH>::unpack(lds_words<kBytes / 4>(from), o); };
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          if constexpr (kUseX) take(slot(d, 0, k, 0), v[k]), take(slot(d, 0, k, 1), v[k] + CH / 2);
          if constexpr (kBack) take(slot(d, kIn - 1, k, 0), e[k]), take(slot(d, kIn - 1, k, 1), e[k] + CH / 2);
        }
      } else {
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          const bool ha = unit[k].a >= 0 && store, hb = unit[k].b >= 0 && store;
          if constexpr (kUseX) Chunks<T, CH>::load(ha ? x + unit[k].a : nullptr, hb ? x + unit[k].b : nullptr, v[k]);
          if constexpr (kBack) Chunks<T, CH>::load(ha ? dy + unit[k].a : nullptr, hb ? dy + unit[k].b : nullptr, e[k]);
        }
        if constexpr (kUseX) x += X.xs[2];
        if constexpr (kBack) dy += X.ds[2];
      }
      if constexpr (kBack) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) rotate<CH>(e[k], c[k], sn[k], inter);
      }
      if constexpr (kNorm && !kBack) {
        float2 ss = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < UPL; ++k)
#pragma unroll
          for (int i = 0; i < CH; ++i) ss = fma2(v[k][i], v[k][i], ss);
        const float rho = rsqrtf(group_sum(ss.x + ss.y, G) * P.inv_dim + P.eps);
#pragma unroll
        for (int k = 0; k < UPL; ++k)
#pragma unroll
          for (int i = 0; i < CH; ++i) v[k][i] = mul2(v[k][i], mul2(gain_r[k][i], twice(rho)));
      }
      if constexpr (!kBack) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) rotate<CH>(v[k], c[k], sn[k], inter);
      }
      if constexpr (kGrad) {
        // both sums in one butterfly: sum x^2 and sum gain e x; then
        // dgain += rho e x and dx = rho (gain e - x rho^2 mean(gain e x))
        auto gains = [&](int k, float2 *o) {
          if constexpr (CH >= 4) {
#pragma unroll
            for (int i = 0; i < CH; i += 2) {  // two pairs, 16 bytes
              // a chunk that the unit lacks reads the first gains (16-byte aligned, and unused)
              const int at = 2 * i < CH ? max(0, unit[k].a) + 2 * i : max(0, unit[k].b) + 2 * i - CH;
              const float4 q = *reinterpret_cast<const float4 *>(gain_s + at);
              o[i] = make_float2(q.x, q.y), o[i + 1] = make_float2(q.z, q.w);
            }
          } else if constexpr (CH == 2) {
            o[0] = *reinterpret_cast<const float2 *>(gain_s + max(0, unit[k].a));
            o[1] = *reinterpret_cast<const float2 *>(gain_s + max(0, unit[k].b));
          } else {
            o[0] = make_float2(gain_s[max(0, unit[k].a)], gain_s[max(0, unit[k].b)]);
          }
        };
        float2 ss = make_float2(0.f, 0.f), wx2 = make_float2(0.f, 0.f);
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          float2 gain[CH];
          gains(k, gain);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            ss = fma2(v[k][i], v[k][i], ss);
            wx2 = fma2(mul2(gain[i], e[k][i]), v[k][i], wx2);
          }
        }
        float s1 = ss.x + ss.y, s2 = wx2.x + wx2.y;
        for (int o = G >> 1; o > 0; o >>= 1) {
          s1 += __shfl_xor_sync(0xffffffffu, s1, o);
          s2 += __shfl_xor_sync(0xffffffffu, s2, o);
        }
        const float rho = rsqrtf(s1 * P.inv_dim + P.eps), back = -rho * (rho * (s2 * P.inv_dim));
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          float2 gain[CH];
          gains(k, gain);
#pragma unroll
          for (int i = 0; i < CH; ++i) {
            if (store) dg[k][i] = fma2(mul2(twice(rho), e[k][i]), v[k][i], dg[k][i]);
            e[k][i] = mul2(twice(rho), fma2(v[k][i], twice(back), mul2(gain[i], e[k][i])));
          }
        }
      }
      // the slots have been read (the values above are computed from them):
      // the head kDepth further may come in
      if constexpr (kDepth > 0) {
        request(d, hh + kDepth < nh);
        if (++d == kDepth) d = 0;
      }
      if (store) {
#pragma unroll
        for (int k = 0; k < UPL; ++k) {
          const float2 *o = kBack ? e[kBack ? k : 0] : v[kUseX ? k : 0];
          if (unit[k].a >= 0) Chunks<T, CH>::store(y + unit[k].a, o, 0);
          if (unit[k].b >= 0) Chunks<T, CH>::store(y + unit[k].b, o, 1);
        }
        y += X.ys[2];
      }
    }
  }
  if constexpr (kDepth > 0) asm volatile("cp.async.wait_all;" ::: "memory");
  if constexpr (kGrad) {
    if (!X.part) return;
    // the groups of a warp by a butterfly, the warps one after another: a fixed order
    for (int i = threadIdx.x; i < P.dim; i += kThreads) dg_s[i] = 0.f;
#pragma unroll
    for (int k = 0; k < UPL; ++k)
#pragma unroll
      for (int i = 0; i < CH; ++i)
        for (int o = G; o < 32; o <<= 1) {
          dg[k][i].x += __shfl_xor_sync(0xffffffffu, dg[k][i].x, o);
          dg[k][i].y += __shfl_xor_sync(0xffffffffu, dg[k][i].y, o);
        }
    for (int q = 0; q < kThreads / 32; ++q) {
      __syncthreads();
      if ((int)(threadIdx.x >> 5) == q && (int)(threadIdx.x & 31) < G) {
#pragma unroll
        for (int k = 0; k < UPL; ++k)
#pragma unroll
          for (int i = 0; i < 2 * CH; ++i) {
            const int at = i < CH ? unit[k].a : unit[k].b;
            if (at >= 0) dg_s[at + (i < CH ? i : i - CH)] += i & 1 ? dg[k][i / 2].y : dg[k][i / 2].x;
          }
      }
    }
    __syncthreads();
    float *out = X.part + (int64_t)((int)blockIdx.x - X.block0) * P.dim;
    for (int i = threadIdx.x; i < P.dim; i += kThreads) out[i] = dg_s[i];
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
  if (col < S.dim) {
    const float *part = S.part[ti] + col;
    for (int r0 = threadIdx.y; r0 < S.rows[ti]; r0 += 32 * 16) {  // sixteen rows in flight
      float v[16];
#pragma unroll
      for (int u = 0; u < 16; ++u) v[u] = r0 + 32 * u < S.rows[ti] ? part[(int64_t)(r0 + 32 * u) * S.dim] : 0.f;
#pragma unroll
      for (int u = 0; u < 16; ++u) a += v[u];
    }
  }
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

// A frequency in turns per position, modulo one turn, in 64-bit fixed point.
// The quotient is off by at most 2^-52 of it (its rounding and that of 2 pi),
// its fraction is exact, and what falls below 2^-64 turns is cut off: an angle
// t f is off by at most |t| (2^-52 |f| + 2^-61) radians.  Formed from |f|: the
// fraction of a small negative quotient, 1 - |f| / 2 pi, would round to 2^-54
// turns whatever f (660 times that bound at f = -1e-4).  More bits of 2 pi
// would not help a frequency that a power of the base made: it has a double's
// rounding itself.
uint64_t turns_of(double f) {
  const double turn = std::fabs(f) / 6.283185307179586476925286766559;
  const uint64_t frac = (uint64_t)std::ldexp(turn - std::floor(turn), 64);
  return f < 0.0 ? 0 - frac : frac;
}

// Blocks that share a backward call's tokens over its tensors at most, in
// proportion to their heads: a function of the table's heads and the device
// alone, so that it bounds the scratch.  How many of them a launch takes, and
// with that dgain's order of summation, also goes by the number of tokens and
// by the chunks that the addresses allow: calls of one shape and alignment
// give the same bits.
void back_blocks(const gbo_rope_tensor *t, int32_t n, int sm_count, int32_t *nblk) {
  int64_t heads = 0;
  for (int32_t i = 0; i < n; ++i) heads += t[i].heads;
  for (int32_t i = 0; i < n; ++i)
    nblk[i] = heads == 0 || t[i].heads == 0
                  ? 0
                  : (int32_t)std::max<int64_t>(1, (int64_t)kRopeBackBlocks * sm_count * t[i].heads / heads);
}

template <typename T, int CH, int UPL, bool kNorm, bool kBack>
cudaError_t launch_rope_n(const RopeParams &P, int blocks, int dev, cudaStream_t stream) {
  constexpr int smem = ring_bytes(CH * (int)sizeof(T), CH, UPL, kNorm, kBack);
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(rope_kernel<T, CH, UPL, kNorm, kBack>, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  });
  if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  // A block's start (its units, gains and turns) overlaps the end of the kernel
  // before it on the stream, on direct launches too: queries and keys 56.3 ->
  // 54.3 us, their gradients 92.4 -> 90.1, heads of 192 119.9 -> 116.6 in a loop.
  return launch_kernel_as(pdl_allowed(), rope_kernel<T, CH, UPL, kNorm, kBack>, dim3(blocks),
                          dim3(rope_threads(kNorm, kBack)), smem, stream, 1, P);
}

template <typename T, int CH, int UPL, bool kBack>
cudaError_t launch_rope(const RopeParams &P, bool norm, int blocks, int dev, cudaStream_t stream) {
  return norm ? launch_rope_n<T, CH, UPL, true, kBack>(P, blocks, dev, stream)
              : launch_rope_n<T, CH, UPL, false, kBack>(P, blocks, dev, stream);
}

// units a lane: at most 256 pairs a head, over groups of 32 lanes
template <typename T, bool kBack>
cudaError_t dispatch_rope(const RopeParams &P, int chunk, int upl, bool norm, int blocks, int dev, cudaStream_t stream) {
  if (chunk == 1)
    return upl <= 2 ? launch_rope<T, 1, 2, kBack>(P, norm, blocks, dev, stream)
                    : launch_rope<T, 1, 8, kBack>(P, norm, blocks, dev, stream);
  if (chunk == 2)
    return upl == 1 ? launch_rope<T, 2, 1, kBack>(P, norm, blocks, dev, stream)
                    : launch_rope<T, 2, 4, kBack>(P, norm, blocks, dev, stream);
  if (chunk == 4)
    return upl == 1 ? launch_rope<T, 4, 1, kBack>(P, norm, blocks, dev, stream)
                    : launch_rope<T, 4, 2, kBack>(P, norm, blocks, dev, stream);
  if constexpr (sizeof(T) == 2) return launch_rope<T, 8, 1, kBack>(P, norm, blocks, dev, stream);
  return cudaErrorInvalidValue;  // fp32 chunks have at most four elements
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
  bool any_dgain = false, in_place = true;
  int32_t grain = 8;  // elements that every head's address is a multiple of, at most 16 bytes
  int32_t dtype = n > 0 ? tensors[0].dtype : GBO_BF16;
  const bool none = n == 0 || batch == 0 || seq == 0;
  for (int32_t i = 0; i < n; ++i) {
    const gbo_rope_tensor &t = tensors[i];
    if (t.dtype != GBO_F32 && t.dtype != GBO_BF16) return rope_fail(GBO_ERR_DTYPE, "dtype must be GBO_F32 or GBO_BF16");
    if (t.dtype != dtype) return rope_fail(GBO_ERR_DTYPE, "the tensors of one call have one dtype");
    if (t.heads < 0) return rope_fail(GBO_ERR_SHAPE, "negative number of heads");
    if (t.norm != 0 && t.norm != 1) return rope_fail(GBO_ERR_INVALID_ARG, "norm must be 0 or 1");
    if (t.norm != tensors[0].norm) return rope_fail(GBO_ERR_INVALID_ARG, "the tensors of one call have a norm, or none has");
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
    const int64_t *from = back ? t.dy_stride : t.x_stride;
    in_place = in_place && t.y == (back ? t.dy : t.x) && memcmp(from, t.y_stride, sizeof t.y_stride) == 0;
    const void *ptrs[3] = {need_x ? t.x : nullptr, back ? t.dy : nullptr, t.y};
    const int64_t *strides[3] = {t.x_stride, t.dy_stride, t.y_stride};
    const int es = dtype == GBO_BF16 ? 2 : 4;
    for (int k = 0; k < 3; ++k) {
      if (!ptrs[k]) continue;
      const int64_t at[4] = {(int64_t)(reinterpret_cast<uintptr_t>(ptrs[k]) / es), batch > 1 ? strides[k][0] : 0,
                             seq > 1 ? strides[k][1] : 0, t.heads > 1 ? strides[k][2] : 0};
      for (int64_t v : at)
        while (v % grain) grain /= 2;
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
  // the widest chunk (16 bytes at most) that divides every address, the head
  // and its rotated part; a unit is two chunks, so pairs have to fill whole units
  int CH = std::min(grain, dtype == GBO_BF16 ? 8 : 4);
  while (CH > 1 && (o->head_dim % CH || o->offset % CH || o->rot_dim % (2 * CH))) CH /= 2;
  const bool norm = n > 0 && tensors[0].norm;
  // without a norm and in place, the elements that are not rotated stay as they are
  P.units = o->rot_dim / (2 * CH) + (norm || !in_place ? ((o->head_dim - o->rot_dim) / CH + 1) / 2 : 0);
  if (P.units == 0) return report_ok();
  // with a norm, a power of two within a warp and several units a lane
  // beyond; without one, lanes of a block as they come
  P.group = 1;
  if (norm)
    while (P.group < 32 && P.group < P.units) P.group *= 2;
  else
    P.group = std::min(P.units, rope_threads(false, back));
  const int upl = (P.units + P.group - 1) / P.group;
  P.dim = o->head_dim, P.rot = o->rot_dim, P.offset = o->offset;
  P.interleaved = o->layout == GBO_ROPE_INTERLEAVED;
  P.magnitude = o->magnitude, P.eps = o->eps, P.inv_dim = 1.f / (float)o->head_dim;
  P.seq = std::max<int64_t>(seq, 1);
  if (pos) {
    P.pos = pos->ptr, P.pos_b = pos->stride_b, P.pos_s = pos->stride_s, P.start = pos->start;
    P.pos64 = pos->dtype == GBO_I64;
  }
  for (int j = 0; j < o->rot_dim / 2; ++j) P.turns[j] = turns_of(o->freq[j]);
  P.n = 0;
  const int groups = rope_threads(norm, back) / P.group;
  const int64_t tokens = batch * seq;
  int32_t nblk[GBO_ROPE_MAX_TENSORS] = {};
  if (back) back_blocks(tensors, n, sm, nblk);
  int64_t all_heads = 0;
  for (int32_t i = 0; i < n; ++i) all_heads += tensors[i].heads;
  // heads a group walks over: up to kMaxHeads while the groups still fill the
  // device (1024 threads an SM), so that a token's cosines are shared
  int32_t per_item = 1;
  while (per_item < kMaxHeads && tokens * all_heads / (2 * per_item) >= (int64_t)sm * (1024 / P.group)) per_item *= 2;
  int64_t rounds_all = 0;
  for (int32_t i = 0; i < n; ++i) rounds_all += (tokens * ((tensors[i].heads + per_item - 1) / per_item) + groups - 1) / groups;
  const bool few = rounds_all <= (int64_t)2 * kRopeBackBlocks * sm;
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
      X.heads = t.heads;
      X.head_blocks = (t.heads + per_item - 1) / per_item;
      X.per_item = (t.heads + X.head_blocks - 1) / X.head_blocks;
      X.items = tokens * X.head_blocks;
      const int64_t want = (X.items + groups - 1) / groups;
      // forward: a block goes on to further items until it has moved 32 KB (its
      // start, some 2 us, is not worth less), while four blocks an SM remain
      const int64_t round = (int64_t)groups * X.per_item * o->head_dim * (dtype == GBO_BF16 ? 2 : 4);
      const int64_t rounds = std::max<int64_t>(1, std::min<int64_t>((32768 + round - 1) / round, want / (4 * sm)));
      // gradients of a norm: a block's end (its sums of the gains) is dear, too:
      // where all blocks have two rounds at most, the resident ones (four an SM
      // with chunks of eight elements, eight with fewer) take them all (1974
      // tokens x 20 heads of 128: 18.6 -> 12.6 us)
      int64_t take = std::min<int64_t>((want + rounds - 1) / rounds, 1 << 20);
      if (back && norm)
        take = std::min<int64_t>(want, few ? std::max<int64_t>(1, nblk[i] * (CH == 8 ? 4 : 8) / kRopeBackBlocks) : nblk[i]);
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
      err = back ? dispatch_rope<__nv_bfloat16, true>(P, CH, upl, norm, (int)blocks, dev, st)
                 : dispatch_rope<__nv_bfloat16, false>(P, CH, upl, norm, (int)blocks, dev, st);
    else
      err = back ? dispatch_rope<float, true>(P, CH, upl, norm, (int)blocks, dev, st)
                 : dispatch_rope<float, false>(P, CH, upl, norm, (int)blocks, dev, st);
    count_launches(1);
  }
  if (err == cudaSuccess && any_dgain) {
    // (it depends on the kernel before it alone: its launch overlaps that one's end)
    err = launch_kernel_as(pdl_allowed(), rope_dgain_kernel, dim3((o->head_dim + 31) / 32, n), dim3(32, 32), 0, st, 1, S);
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
  // a context that is not stretched keeps its scores
  *magnitude = kind == GBO_ROPE_SCALE_YARN && s->factor > 1.0 ? 0.1 * std::log(s->factor) + 1.0 : 1.0;
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

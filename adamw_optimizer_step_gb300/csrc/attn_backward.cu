// Attention, gradients (gbo_attn_backward).  With P = softmax(scale Q K^T) over
// the keys seen and D_i = dy_i . y_i:
//   dV = P^T dY,  dS = scale P (dY V^T - D),  dQ = dS K,  dK = dS^T Q.
// P is formed again from the forward's lse: P = 2^(S c - lse log2(e)).
//
//   attn_delta_kernel     per row: -lse log2(e) and D
//   attn_few_kernel       the same of rows that see few keys, D from P and V
//   attn_backward_kernel  attn_dkv: a CTA holds 128 keys and walks over the rows that see them;
//                         attn_dq: a CTA holds 128 rows and walks over the keys that they see
//
// Two walks form S and dP twice (7 products instead of 5), and in return no
// sum crosses CTAs: no atomics, results that repeat bit for bit, no fp32 dQ in
// memory.  Every sum stays in TMEM for a CTA's whole walk, the query heads that
// share a key head among them.  P and dS are rounded to bf16 once, as operands of
// products (by 2^-8 of them at most); sums are fp32.  That makes dQ's and dK's error
// 2.4e-3 of them against 1.7e-3 of the outputs' rounding alone; dS as two bf16 numbers
// would take two products more.
//
// Measured, causal, 2 x 8192 tokens, 16 query and 4 key heads of 128: 1104 us at best, 1190
// over a second of calls (the power limit holds the clock at 1.78 GHz); the keys' walk alone
// 676 and 717 (1.63 and 1.53 PFLOP/s of the four products it forms), the queries' alone 493
// and 526 (1.67 and 1.57 of three), delta and few kernels with each: 86 and 91% of a library
// product's burst and sustained rates.  Heads of 192 and 128: 1863 us, 1.33 PFLOP/s of all
// seven at 1.95 GHz.
// Bound: tensor cores (active 72% at 4096 tokens, where the tail counts), then the
// elementwise warps between S and dS.  13 documents in 8192 tokens 141 us, 6 x 777
// tokens of 32 heads of 192 and 128 180 us: a CTA's start and end (9000 clocks).
// Resident CTAs with several tiles each, the next one looked up ahead: 488 us in place
// of 493 for the queries' walk, but 93 in place of 83 for the documents, whose tiles
// are uneven.  Not kept.
#include "attn_common.cuh"

namespace gbo {

namespace {

constexpr int kBwdWarps = 16;  // elementwise: four groups of four, each a quarter of a tile's columns
constexpr float kLog2ePlain = 1.4426950408889634f;

// ---------------------------------------------------------------------------
// -lse log2(e) and D of each row: 16 lanes to a row.  A row that sees nothing
// (lse = -inf) gets -inf and 0, whatever stands in it: its P and dS are 0.  Bound by
// HBM (dy and y once).
//
// D = dy . y takes over the rounding of y, an error that every dS of the row gets times
// its P: beside dS's own rounding it counts 1 / sqrt(n) over n keys of like weight.  Rows
// that see 64 keys or fewer form D = sum p (dy . v) instead: dQ's and dK's error is 2.4e-3
// of them, not 2.6e-3 (16 x 48 tokens, heads of 32) to 3.0e-3 (a handful of tokens), as it
// is with D from y for rows of more than 8 keys, and over values that lie close together,
// where D is a difference, it is smaller by orders.  Such rows are looked for among the
// first 64 tokens of each sequence or document (no later one of a causal sequence sees so
// few), or among all tokens where a narrow window or few keys may leave any row so few;
// where no row sees more, attn_delta_kernel does not run.
constexpr int kFewKeys = 64;
constexpr int kFewWarps = 4;    // of a CTA, 16 rows each
constexpr int kFewChunk = 80;   // keys in shared memory at a time: 64 and those of 16 tokens more
constexpr int kDeltaRows = 32;  // of a CTA, two to each 16 lanes: their loads are under way together

struct DeltaParams {
  const __nv_bfloat16 *dy, *y, *q, *k, *v;
  const float *lse;
  float2 *stats;
  AttnMask mask;
  int64_t ds[3], ys[3], qs[3], ks[3], vs[3], rows;
  float scale2;
  int32_t sq, heads, group, dk, dv;
  FastDiv by_heads, by_sq;  // of row numbers that fit 32 bits
  // rows of few keys: 2^pack heads that share a key head and 16 / 2^pack tokens to a warp,
  // `sets` of them to a key head of a sequence or document, chunks of four to a CTA
  FastDiv by_chunks, by_k_heads, by_blocks;
  int32_t pack, sets, every;  // every: all tokens are looked at
  int32_t all;                // no row sees more: those that see nothing are written, too
};

// Sum of the products of eight pairs of bf16.
__device__ __forceinline__ float dot8(const uint4 &u, const uint4 &v, float d) {
  const uint32_t a[4] = {u.x, u.y, u.z, u.w}, c[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    d = fmaf(__uint_as_float(a[e] << 16), __uint_as_float(c[e] << 16), d);
    d = fmaf(__uint_as_float(a[e] & 0xffff0000u), __uint_as_float(c[e] & 0xffff0000u), d);
  }
  return d;
}

// acc (16 rows x 8 columns) += A B^T over 32 elements of each row, of which a lane holds
// eight that follow one another, of A's rows lane / 4 and lane / 4 + 8 and of B's row
// lane / 4.  (In a sum of products any order of the elements will do, the same in both.)
__device__ __forceinline__ void mma_rows32(float (&acc)[4], const uint4 &a0, const uint4 &a1, const uint4 &b) {
  const uint32_t x[4] = {a0.x, a0.y, a0.z, a0.w}, y[4] = {a1.x, a1.y, a1.z, a1.w}, z[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
  for (int s = 0; s < 4; s += 2)
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(acc[0]), "+f"(acc[1]), "+f"(acc[2]), "+f"(acc[3])
        : "r"(x[s]), "r"(y[s]), "r"(x[s + 1]), "r"(y[s + 1]), "r"(z[s]), "r"(z[s + 1]));
}

// Keys and values of a chunk, a row 64 bytes longer than whole lines: two rows' 64 bytes
// that eight lanes read meet in no bank.
template <int kKb, int kVb>
struct Few {
  static constexpr int kKPitch = kKb * 128 + 64, kVPitch = kVb * 128 + 64;
  static constexpr int kVAt = kFewChunk * kKPitch, kSmem = kVAt + kFewChunk * kVPitch;
};

// Rows that see few keys.  A warp takes 16 rows of a key head, heads of a token side by
// side, held in registers; the CTA's warps go over the keys that any of their rows sees,
// a chunk in shared memory at a time.  Bound by the wait for rows and keys, at 16 warps an
// SM: some 5 us of a call where the first tokens alone are looked at; a window of 64 over
// 2 x 8192 tokens of 16 heads 60 us (issue slots 35%), 103 with fragments straight from
// global memory.
template <int kKb, int kVb>
__global__ void __launch_bounds__(32 * kFewWarps, 4) attn_few_kernel(const __grid_constant__ DeltaParams P) {
  pdl_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  using C = Few<kKb, kVb>;
  __shared__ int32_t range[2][kFewWarps];
  pdl_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, c0 = (lane & 3) * 8;
  int unit = (int)blockIdx.x;
  int set = P.by_chunks.split(unit) * kFewWarps + warp;
  const int kh = P.by_k_heads.split(unit);
  const bool mine = set < P.sets;
  const int h0 = kh * P.group + (P.by_blocks.split(set) << P.pack);
  int first = set * (16 >> P.pack), end = P.sq, b = unit;  // this warp's tokens
  if (!P.every) {
    int from;
    if (P.mask.docs) {
      b = 0, from = clamp_to(P.mask.docs[unit], P.mask.sq), end = clamp_to(P.mask.docs[unit + 1], P.mask.sq);
    } else {
      const AttnSeq seq = attn_seq(P.mask, b);
      from = seq.q_lo, end = seq.q_hi;
    }
    end = min(end, from + kFewKeys), first += from;
  }
  const AttnSeq seq = attn_seq(P.mask, b);
  const DocWindow docs = doc_window(P.mask, first);
  Span keys[2];
  int64_t row[2];
  float lse2[2];
  bool in[2];
  uint4 q[2][2 * kKb], dy[2][2 * kVb];
  int lo = INT32_MAX, hi = 0;  // (of no row: no chunk starts there)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = g + 8 * i, t = first + (r >> P.pack), h = h0 + (r & ((1 << P.pack) - 1));
    keys[i] = keys_of(P.mask, seq, docs, t);
    in[i] = mine && t < end && t >= seq.q_lo && t < seq.q_hi && !keys[i].empty() && keys[i].hi - keys[i].lo <= kFewKeys;
    if (!in[i]) keys[i] = {0, 0};
    if (in[i]) lo = min(lo, keys[i].lo), hi = max(hi, keys[i].hi);
    row[i] = ((int64_t)b * P.sq + t) * P.heads + h;
    lse2[i] = in[i] ? P.lse[row[i]] * kLog2ePlain : 0.f;
    const __nv_bfloat16 *const q_row = P.q + b * P.qs[0] + t * P.qs[1] + h * P.qs[2];
    const __nv_bfloat16 *const dy_row = P.dy + b * P.ds[0] + t * P.ds[1] + h * P.ds[2];
#pragma unroll
    for (int c = 0; c < 2 * kKb; ++c) {
      q[i][c] = make_uint4(0, 0, 0, 0);
      if (in[i] && c * 32 + c0 < P.dk) q[i][c] = *reinterpret_cast<const uint4 *>(q_row + c * 32 + c0);
    }
#pragma unroll
    for (int c = 0; c < 2 * kVb; ++c) {
      dy[i][c] = make_uint4(0, 0, 0, 0);
      if (in[i] && c * 32 + c0 < P.dv) dy[i][c] = *reinterpret_cast<const uint4 *>(dy_row + c * 32 + c0);
    }
  }
  lo = __reduce_min_sync(0xffffffffu, lo), hi = __reduce_max_sync(0xffffffffu, hi);
  if (lane == 0) range[0][warp] = lo, range[1][warp] = hi;
  __syncthreads();
  int from = INT32_MAX, to = 0;
#pragma unroll
  for (int w = 0; w < kFewWarps; ++w) from = min(from, range[0][w]), to = max(to, range[1][w]);
  const __nv_bfloat16 *const k = P.k + b * P.ks[0] + kh * P.ks[2], *const v = P.v + b * P.vs[0] + kh * P.vs[2];
  const uint32_t ktile = smem_u32(smem), vtile = ktile + C::kVAt;
  float sum[2] = {0.f, 0.f};
  for (int j0 = from; j0 < to; j0 += kFewChunk) {
    // rows of eight elements a thread; behind the last key and a row's last element zeros
    auto copy = [&](uint32_t tile, int pitch, int pieces, int dim, const __nv_bfloat16 *src, int64_t stride) {
      for (int i = threadIdx.x; i < kFewChunk * pieces; i += 32 * kFewWarps) {
        const int j = i / pieces, c = i - j * pieces;
        const bool here = j0 + j < to && c * 8 < dim;
        asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(tile + j * pitch + c * 16),
                     "l"(src + (here ? (j0 + j) * stride + c * 8 : 0)), "r"(here ? 16 : 0)
                     : "memory");
      }
    };
    copy(ktile, C::kKPitch, 8 * kKb, P.dk, k, P.ks[1]);
    copy(vtile, C::kVPitch, 8 * kVb, P.dv, v, P.vs[1]);
    asm volatile("cp.async.commit_group;\n\tcp.async.wait_group 0;" ::: "memory");
    __syncthreads();
    for (int m = 0; m < kFewChunk; m += 16) {
      if (j0 + m >= hi || j0 + m + 16 <= lo) continue;
      float s[2][4] = {}, dp[2][4] = {};
      auto eight = [&](uint32_t at) {
        uint4 x;
        asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w) : "r"(at) : "memory");
        return x;
      };
      const uint32_t kr = ktile + (m + g) * C::kKPitch + c0 * 2, vr = vtile + (m + g) * C::kVPitch + c0 * 2;
#pragma unroll
      for (int c = 0; c < 2 * std::max(kKb, kVb); ++c)
#pragma unroll
        for (int i = 0; i < 2; ++i) {  // (four chains of products, one beside the other)
          if (c < 2 * kKb) mma_rows32(s[i], q[0][c], q[1][c], eight(kr + 8 * i * C::kKPitch + c * 64));
          if (c < 2 * kVb) mma_rows32(dp[i], dy[0][c], dy[1][c], eight(vr + 8 * i * C::kVPitch + c * 64));
        }
      // (keys that a row does not see may hold anything)
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = j0 + m + 8 * i + (lane & 3) * 2 + (e & 1);
          if (key >= keys[e >> 1].lo && key < keys[e >> 1].hi)
            sum[e >> 1] = fmaf(ex2(fmaf(s[i][e], P.scale2, -lse2[e >> 1])), dp[i][e], sum[e >> 1]);
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 1);
    sum[i] += __shfl_xor_sync(0xffffffffu, sum[i], 2);
    if ((lane & 3) == 0 && in[i]) P.stats[row[i]] = lse2[i] == -INFINITY ? make_float2(-INFINITY, 0.f) : make_float2(-lse2[i], sum[i]);
    if ((lane & 3) == 0 && P.all && !in[i] && mine && first + ((g + 8 * i) >> P.pack) < end)
      P.stats[row[i]] = make_float2(-INFINITY, 0.f);
  }
}

__global__ void __launch_bounds__(256, 5) attn_delta_kernel(const __grid_constant__ DeltaParams P) {
  pdl_wait();
  const int64_t row0 = (int64_t)blockIdx.x * kDeltaRows + (threadIdx.x >> 4);
  const int lane = threadIdx.x & 15;
  constexpr int kEach = kDeltaRows / 16;
  int b[kEach], t[kEach];
  float lse[kEach];
  uint4 g[kEach], y[kEach];
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    const int64_t row = row0 + 16 * i;
    const bool in = row < P.rows;
    int h = 0;
    b[i] = t[i] = 0;
    if (P.rows <= INT32_MAX) {
      int at = in ? (int)row : 0;
      h = P.by_heads.split(at), t[i] = P.by_sq.split(at), b[i] = at;
    } else if (in) {
      const int64_t bt = row / P.heads;
      b[i] = (int)(bt / P.sq), h = (int)(row - bt * P.heads), t[i] = (int)(bt - (int64_t)b[i] * P.sq);
    }
    lse[i] = in ? P.lse[row] : -INFINITY;
    g[i] = y[i] = make_uint4(0, 0, 0, 0);
    if (in && lane * 8 < P.dv) {
      g[i] = *reinterpret_cast<const uint4 *>(P.dy + b[i] * P.ds[0] + t[i] * P.ds[1] + h * P.ds[2] + lane * 8);
      y[i] = *reinterpret_cast<const uint4 *>(P.y + b[i] * P.ys[0] + t[i] * P.ys[1] + h * P.ys[2] + lane * 8);
    }
  }
#pragma unroll
  for (int i = 0; i < kEach; ++i) {
    float d = dot8(g[i], y[i], 0.f);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) d += __shfl_xor_sync(0xffffffffu, d, o);
    if (row0 + 16 * i < P.rows && lane == 0)
      P.stats[row0 + 16 * i] = lse[i] == -INFINITY ? make_float2(-INFINITY, 0.f) : make_float2(-lse[i] * kLog2ePlain, d);
  }
  pdl_launch();
}

struct BwdParams {
  CUtensorMap q, k, v, dy;  // loads
  CUtensorMap o1, o2;       // stores: dK and dV, or dQ
  AttnMask mask;
  AttnShape shape;
  const float2 *stats;      // (batch, sq, heads)
  int32_t *status;
  int32_t tiles;            // of keys, or of tokens
  int32_t has1, has2;       // which outputs are wanted
};

// ---------------------------------------------------------------------------
// dK, dV

// Transposed: keys are the rows (lanes of TMEM), kQt query rows the columns.
//   S^T = K Q^T, P^T; dP^T = V dY^T, dS^T; dV += P^T dY, dK += dS^T Q
// P^T and dS^T go back into TMEM in bf16 over S^T and dP^T, as the A operand.
// Products run in the order
//   dV(i) S(i+1) dK(i) dP(i+1)
// so that the tensor cores form S(i+1) while dS(i) is computed, and dP(i+1) while
// P(i+1) is.
template <int kKb, int kVb, int kQt>
struct Dkv {
  static constexpr int kKTile = kKb * kAttnBlock, kVTile = kVb * kAttnBlock;
  static constexpr int kQBlock = kQt * 128, kQStage = kKb * kQBlock, kDStage = kVb * kQBlock;
  static constexpr int kQStages = 3, kDStages = kKb == 2 ? 2 : 3, kStats = 2;
  static constexpr int kRing = kKTile + kVTile, kStatAt = kRing + kQStages * kQStage + kDStages * kDStage;
  static constexpr int kUsed = kStatAt + kStats * kQt * 8;
  // kv, q full/empty, dy full/empty, stats full/empty, S, P, dP, dS, drained (two), raw, turns (two)
  static constexpr int kBars = 1 + 2 * kQStages + 2 * kDStages + 2 * kStats + 4 + 2 + 1 + 2;
  static constexpr int kSmem = kUsed + kBars * 8 + kNotes;
  static constexpr uint32_t kDp = kQt, kDv = 2 * kQt, kDk = 2 * kQt + kVb * 64;  // TMEM columns
  static_assert(kDk + kKb * 64 <= 512, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int kKb, int kVb, int kQt>
__device__ __forceinline__ void attn_dkv(const BwdParams &P, uint8_t *smem, int idx) {
  using C = Dkv<kKb, kVb, kQt>;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kUsed);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  const uint32_t kvfull = smem_u32(bars), qfull0 = kvfull + 8, qempty0 = qfull0 + 8 * C::kQStages;
  const uint32_t dfull0 = qempty0 + 8 * C::kQStages, dempty0 = dfull0 + 8 * C::kDStages;
  const uint32_t tfull0 = dempty0 + 8 * C::kDStages, tempty0 = tfull0 + 8 * C::kStats;
  const uint32_t sfull = tempty0 + 8 * C::kStats, pready = sfull + 8, dpfull = pready + 8, dsready = dpfull + 8;
  const uint32_t done0 = dsready + 8, raw = done0 + 16, turn0 = raw + 8;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 1 + 2 * C::kQStages + C::kDStages; ++s) mbar_init(kvfull + 8 * s, 1);
    for (int s = 0; s < C::kDStages; ++s) mbar_init(dempty0 + 8 * s, 2);  // dP and dV
    for (int s = 0; s < C::kStats; ++s) {
      mbar_init(tfull0 + 8 * s, 32);
      mbar_init(tempty0 + 8 * s, kBwdWarps);
    }
    mbar_init(sfull, 1);
    mbar_init(pready, kBwdWarps);
    mbar_init(dpfull, 1);
    mbar_init(dsready, kBwdWarps);
    for (int s = 0; s < 5; ++s) mbar_init(done0 + 8 * s, 1);  // (and raw and turns)
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kBwdWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();

  const AttnShape &A = P.shape;
  // early keys first: with a causal mask most queries see them
  const int kh = A.by_k_heads.split(idx), b = A.by_batch.split(idx), k0 = idx * kAttnTile;
  const AttnSeq seq = attn_seq(P.mask, b);
  const int shift = (kQt == 128 ? 7 : 6) - A.pack, tokens = 1 << shift;
  const DocWindow docs = doc_window(P.mask, k0);
  int tt0 = 0, n_tok = 0, full_lo = 0, full_hi = 0;  // token tiles that see these keys
  {
    const int a = max(k0, seq.k_lo), e = min(k0 + kAttnTile, seq.k_hi);
    if (e > a) {
      const Span first = queries_of(P.mask, seq, docs, a), last = queries_of(P.mask, seq, docs, e - 1);
      if (last.hi > first.lo) {
        tt0 = first.lo >> shift, n_tok = ((last.hi + tokens - 1) >> shift) - tt0;
        full_lo = last.lo, full_hi = first.hi;
      }
    }
  }
  const int steps = n_tok * A.head_blocks, group = A.group;
  if (steps == 0) {
    zero_block(smem);
    if (threadIdx.x == 0) {
      for (int r0 = 0; r0 < kAttnTile && k0 + r0 < P.mask.sk; r0 += 32) {
        if (P.has1)
          for (int c = 0; c < A.kb; ++c) tma_store_4d(&P.o1, smem_u32(smem), 64 * c, kh, k0 + r0, b);
        if (P.has2)
          for (int c = 0; c < A.vb; ++c) tma_store_4d(&P.o2, smem_u32(smem), 64 * c, kh, k0 + r0, b);
      }
      bulk_commit();
      bulk_wait_read<0>();
    }
    if (warp == kBwdWarps) tmem_free(*tmem_slot, 512);
    return;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t kt = smem_u32(smem), vt = kt + C::kKTile, qring = kt + C::kRing;
  const uint32_t dring = qring + C::kQStages * C::kQStage;
  float *const stats = reinterpret_cast<float *>(smem + C::kStatAt);
  const AttnGuard guard = {abort_flag, P.status};
  const Started started = {abort_flag + 1};

  if (warp == kBwdWarps + 2) {
    uint32_t raw_phase = 0;
    TileRing Q(qfull0, qempty0, qring, C::kQStage, C::kQStages), D(dfull0, dempty0, dring, C::kDStage, C::kDStages);
    if (steps > 0) {
      if (elect_one()) {
        mbar_expect_tx(kvfull, (uint32_t)(A.kb + A.vb) * kAttnBlock);
        for (int c = 0; c < A.kb; ++c) tma_load_4d(kt + c * kAttnBlock, &P.k, kvfull, 64 * c, kh, k0, b);
        for (int c = 0; c < A.vb; ++c) tma_load_4d(vt + c * kAttnBlock, &P.v, kvfull, 64 * c, kh, k0, b);
      }
      __syncwarp();
    }
    int tt = 0, hb = 0;
    for (int i = 0; i < steps; ++i) {
      const int h0 = kh * group + (hb << A.pack), t0 = (tt0 + tt) * tokens;
      const bool dirty = t0 < seq.q_lo || (t0 + tokens > seq.q_hi && seq.q_hi < P.mask.sq);
      const int lo = max(0, seq.q_lo - t0) << A.pack, hi = min(tokens, seq.q_hi - t0) << A.pack;
      if (!Q.load(guard, &P.q, A.kb, C::kQBlock, h0, t0, b, dirty, raw, raw_phase, kQt, lo, hi, lane)) break;
      if (!D.load(guard, &P.dy, A.vb, C::kQBlock, h0, t0, b, dirty, raw, raw_phase, kQt, lo, hi, lane)) break;
      if (++tt == n_tok) tt = 0, ++hb;
    }
    if (lane == 0) started.note(1, Q.loads, D.loads);
  } else if (warp == kBwdWarps + 3) {
    // the rows' statistics, a stage ahead of the elementwise warps
    int s = 0, tt = 0, hb = 0;
    uint32_t ph = 0;
    for (int i = 0; i < steps; ++i) {
      const int h0 = kh * group + (hb << A.pack), t0 = (tt0 + tt) * tokens;
      float2 x[kQt / 32];
#pragma unroll
      for (int u = 0; u < kQt / 32; ++u) {
        const int r = u * 32 + lane, t = t0 + (r >> A.pack);
        x[u] = make_float2(-INFINITY, 0.f);
        if (t >= seq.q_lo && t < seq.q_hi)
          x[u] = P.stats[((int64_t)b * P.mask.sq + t) * A.q_heads + h0 + (r & ((1 << A.pack) - 1))];
      }
      if (!guard.wait_warp(tempty0 + 8 * s, ph ^ 1)) break;
#pragma unroll
      for (int u = 0; u < kQt / 32; ++u) {
        stats[s * 2 * kQt + u * 32 + lane] = x[u].x;
        stats[s * 2 * kQt + kQt + u * 32 + lane] = x[u].y;
      }
      mbar_arrive(tfull0 + 8 * s);
      if (++s == C::kStats) s = 0, ph ^= 1;
      if (++tt == n_tok) tt = 0, ++hb;
    }
  } else if (warp == kBwdWarps) {
    // S(i + 1) behind dV(i), whose P stands over S(i).  The two issuing warps take
    // turns, so that S(i + 1) is not held up by dK(i) and dP(i + 1).
    RingAt Q, D;
    uint32_t turn = 1;
    bool ok = steps > 0 && guard.wait_warp(kvfull, 0);
    for (int i = 0; i <= steps && ok; ++i) {
      if (i < steps && !guard.wait_warp(qfull0 + 8 * Q.stage, Q.phase)) break;
      if (i > 0 && (!guard.wait_warp(dfull0 + 8 * D.stage, D.phase) || !guard.wait_warp(pready, (i - 1) & 1))) break;
      if (!guard.wait_warp(turn0, turn)) break;
      turn ^= 1;
      tc_fence_after();
      if (elect_one()) {
        if (i > 0) {
          product_ts<kQt / 16, 4>(tmem + C::kDv, tmem, kQt / 4, dring + D.stage * C::kDStage, C::kQBlock, A.v_cols, i > 1);
          mma_commit_one(dempty0 + 8 * D.stage);
        }
        if (i < steps) product_ss<kKb>(tmem, kt, qring + Q.stage * C::kQStage, A.k_steps, C::kQBlock, kQt);
        mbar_arrive(turn0 + 8);
        if (i < steps) mma_commit_one(sfull);
      }
      __syncwarp();
      if (i > 0) D.next(C::kDStages);
      if (i < steps) Q.next(C::kQStages);
    }
    drain_products(done0);
  } else if (warp == kBwdWarps + 1) {
    // dP(i + 1) behind dK(i), whose dS stands over dP(i); that is the last to read
    // the queries' tile
    RingAt Q, D;
    uint32_t turn = 0;
    bool ok = steps > 0 && guard.wait_warp(kvfull, 0);
    for (int i = 0; i <= steps && ok; ++i) {
      if (i < steps && !guard.wait_warp(dfull0 + 8 * D.stage, D.phase)) break;
      if (i > 0 && (!guard.wait_warp(qfull0 + 8 * Q.stage, Q.phase) || !guard.wait_warp(dsready, (i - 1) & 1))) break;
      if (!guard.wait_warp(turn0 + 8, turn)) break;
      turn ^= 1;
      tc_fence_after();
      if (elect_one()) {
        if (i > 0) {
          product_ts<kQt / 16, 4>(tmem + C::kDk, tmem + C::kDp, kQt / 4, qring + Q.stage * C::kQStage, C::kQBlock,
                                  A.k_steps * 16, i > 1);
          mma_commit_one(qempty0 + 8 * Q.stage);
        }
        if (i < steps) product_ss<kVb>(tmem + C::kDp, vt, dring + D.stage * C::kDStage, A.v_cols / 16, C::kQBlock, kQt);
        mbar_arrive(turn0);
        if (i < steps) {
          mma_commit_one(dpfull);
          mma_commit_one(dempty0 + 8 * D.stage);
        }
      }
      __syncwarp();
      if (i > 0) Q.next(C::kQStages);
      if (i < steps) D.next(C::kDStages);
    }
    drain_products(done0 + 8);
  } else {
    constexpr int kCols = kQt / 4;
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane, key = k0 + row;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t S = trow + grp * kCols, D = S + C::kDp;
    const bool live = key >= seq.k_lo && key < seq.k_hi;
    Span seen = queries_of(P.mask, seq, docs, key);
    if (!live) seen = {0, 0};
    const float2 c2 = make_float2(A.scale2, A.scale2);
    bool ok = true;
    int st = 0, tt = 0;
    uint32_t ph = 0;
    for (int i = 0; i < steps; ++i) {
      const int t0 = (tt0 + tt) * tokens;
      const bool masked = t0 < full_lo || t0 + tokens > full_hi;
      const int lo = (min(max(seen.lo - t0, 0), tokens) << A.pack) - grp * kCols;
      const int hi = (min(max(seen.hi - t0, 0), tokens) << A.pack) - grp * kCols;
      if (!(ok = guard.wait_warp(tfull0 + 8 * st, ph) && guard.wait_warp(sfull, i & 1))) break;
      tc_fence_after();
      const float4 *nl = reinterpret_cast<const float4 *>(stats + st * 2 * kQt + grp * kCols);
      const float4 *dl = reinterpret_cast<const float4 *>(stats + st * 2 * kQt + kQt + grp * kCols);
      uint32_t r[kCols], w[kCols / 2];
      tmem_read<kCols>(S, r);
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 l = nl[c / 4];
        const float2 x = f2_fma(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), c2, make_float2(l.x, l.y));
        const float2 y = f2_fma(make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])), c2, make_float2(l.z, l.w));
        float p[4] = {ex2(x.x), ex2(x.y), ex2(y.x), ex2(y.y)};
        if (masked) {
#pragma unroll
          for (int e = 0; e < 4; ++e)
            if (c + e < lo || c + e >= hi) p[e] = 0.f;
        }
#pragma unroll
        for (int e = 0; e < 4; ++e) r[c + e] = __float_as_uint(p[e]);
        w[c / 2] = pack_bf16(p[0], p[1]);
        w[c / 2 + 1] = pack_bf16(p[2], p[3]);
      }
      tmem_write<kCols>(S, w);
      tmem_put_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready);
      if (!(ok = guard.wait_warp(dpfull, i & 1))) break;
      tc_fence_after();
      uint32_t g[kCols];
      tmem_read<kCols>(D, g);
#pragma unroll
      for (int c = 0; c < kCols; c += 4) {
        const float4 d = dl[c / 4];
        float2 x = f2_add(make_float2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), make_float2(-d.x, -d.y));
        float2 y = f2_add(make_float2(__uint_as_float(g[c + 2]), __uint_as_float(g[c + 3])), make_float2(-d.z, -d.w));
        x = f2_mul(x, make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])));
        y = f2_mul(y, make_float2(__uint_as_float(r[c + 2]), __uint_as_float(r[c + 3])));
        if (masked) {
          float *e[4] = {&x.x, &x.y, &y.x, &y.y};
#pragma unroll
          for (int k = 0; k < 4; ++k)
            if (c + k < lo || c + k >= hi) *e[k] = 0.f;
        }
        w[c / 2] = pack_bf16(x.x, x.y);
        w[c / 2 + 1] = pack_bf16(y.x, y.y);
      }
      tmem_write<kCols>(D, w);
      tmem_put_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(dsready);
        mbar_arrive(tempty0 + 8 * st);
      }
      if (++st == C::kStats) st = 0, ph ^= 1;
      if (++tt == n_tok) tt = 0;
    }
    if (ok) ok = guard.wait_warp(done0, 0) && guard.wait_warp(done0 + 8, 0);
    tc_fence_after();
    if (ok) {
      // two groups write dV, the others dK, blocks of 64 columns in turn, through
      // the places of V and K
      const bool is_k = grp >= 2;
      const int blocks = is_k ? A.kb : A.vb, r0 = (warp & 3) * 32;
      const float f = is_k ? A.scale : 1.f;
      const uint32_t from = trow + (is_k ? C::kDk : C::kDv), out = is_k ? kt : vt;
      if (is_k ? P.has1 : P.has2) {
        for (int blk = grp & 1; blk < blocks; blk += 2) {
#pragma unroll 1
          for (int c = blk * 64; c < blk * 64 + 64; c += 32) {
            uint32_t r[32];
            float v[32];
            tmem_read<32>(from + c, r);
#pragma unroll
            for (int e = 0; e < 32; ++e) v[e] = live ? __uint_as_float(r[e]) * f : 0.f;
            put_tile_row(out, row, c, v);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0 && k0 + r0 < P.mask.sk) {
            tma_store_4d(is_k ? &P.o1 : &P.o2, out + blk * kAttnBlock + r0 * 128, 64 * blk, kh, k0 + r0, b);
            bulk_commit();
            bulk_wait_read<0>();  // (the writes themselves end with the kernel)
          }
          __syncwarp();
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBwdWarps) tmem_free(tmem, 512);
  if (warp == kBwdWarps + 2 && guard.aborted()) {
    started.settle_single(guard, kvfull);
    started.settle_ring(guard, 1, qfull0, C::kQStages);
    started.settle_ring(guard, 2, dfull0, C::kDStages);
  }
}

// ---------------------------------------------------------------------------
// dQ

// Rows are the lanes: S = Q K^T, dP = dY V^T, dS over S as the A operand,
// dQ += dS K.  With room for two S (heads of up to 128) the products run
//   S(j+1) dP(j+1) dQ(j)
// so dS(j) is computed beside two of them; else dP(j+1) dQ(j) S(j+1).
template <int kKb, int kVb>
struct Dq {
  static constexpr int kQTile = kKb * kAttnBlock, kDTile = kVb * kAttnBlock;
  static constexpr int kBufs = kKb == 3 ? 1 : 2;
  static constexpr int kKStages = kKb == 1 ? 4 : kKb == 2 ? 3 : 2, kVStages = kKb == 1 ? 4 : kKb == 2 ? 2 : 1;
  static constexpr int kKRing = kQTile + kDTile, kVRing = kKRing + kKStages * kQTile;
  static constexpr int kUsed = kVRing + kVStages * kDTile;
  // rows, K full/empty, V full/empty, S (two), dP, dP read, dS (two), drained (two), raw
  static constexpr int kBars = 1 + 2 * kKStages + 2 * kVStages + 6 + 2 + 1;
  static constexpr int kSmem = kUsed + kBars * 8 + kNotes;
  static constexpr uint32_t kDp = kBufs * 128, kDq = kDp + 128;  // TMEM columns
  static_assert(kDq + kKb * 64 <= 512, "TMEM columns");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

template <int kKb, int kVb>
__device__ __forceinline__ void attn_dq(const BwdParams &P, uint8_t *smem, int idx) {
  using C = Dq<kKb, kVb>;
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kUsed);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  const uint32_t rfull = smem_u32(bars), kfull0 = rfull + 8, kempty0 = kfull0 + 8 * C::kKStages;
  const uint32_t vfull0 = kempty0 + 8 * C::kKStages, vempty0 = vfull0 + 8 * C::kVStages;
  const uint32_t sfull0 = vempty0 + 8 * C::kVStages, dpfull = sfull0 + 16, dpread = dpfull + 8, dsready0 = dpread + 8;
  const uint32_t done0 = dsready0 + 16, raw = done0 + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 1 + 2 * C::kKStages + 2 * C::kVStages + 3; ++s) mbar_init(rfull + 8 * s, 1);
    mbar_init(dpread, kBwdWarps);
    // one for each place of S: the next step's S is formed before this step's dS is waited for, so the elementwise
    // warps may be a step ahead of the wait
    for (int s = 0; s < 2; ++s) mbar_init(dsready0 + 8 * s, kBwdWarps);
    for (int s = 0; s < 3; ++s) mbar_init(done0 + 8 * s, 1);  // (and raw)
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kBwdWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)), "r"(512)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();

  const AttnShape &A = P.shape;
  int kh = A.by_all.split(idx);
  const int b = A.by_batch.split(idx), tb = P.tiles - 1 - idx;  // later queries first
  const int hb = A.by_blocks.split(kh), h0 = kh * A.group + (hb << A.pack);
  const int tokens = kAttnTile >> A.pack, t0 = tb * tokens;
  const AttnSeq seq = attn_seq(P.mask, b);
  const DocWindow docs = doc_window(P.mask, t0);
  const TileKeys tk = tile_keys(P.mask, seq, docs, t0, tokens);
  const int steps = max(0, tk.j1 - tk.j0);
  if (steps == 0) {
    zero_block(smem);
    if (threadIdx.x == 0) {
      for (int r0 = 0; r0 < kAttnTile && t0 + (r0 >> A.pack) < P.mask.sq; r0 += 32)
        for (int c = 0; c < A.kb; ++c) tma_store_4d(&P.o1, smem_u32(smem), 64 * c, h0, t0 + (r0 >> A.pack), b);
      bulk_commit();
      bulk_wait_read<0>();
    }
    if (warp == kBwdWarps) tmem_free(*tmem_slot, 512);
    return;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t qt = smem_u32(smem), dt = qt + C::kQTile, kring = qt + C::kKRing, vring = qt + C::kVRing;
  const AttnGuard guard = {abort_flag, P.status};
  const Started started = {abort_flag + 1};

  if (warp == kBwdWarps + 2) {
    uint32_t raw_phase = 0;
    TileRing K(kfull0, kempty0, kring, C::kQTile, C::kKStages), V(vfull0, vempty0, vring, C::kDTile, C::kVStages);
    if (steps > 0) {
      if (elect_one()) {
        mbar_expect_tx(rfull, (uint32_t)(A.kb + A.vb) * kAttnBlock);
        for (int c = 0; c < A.kb; ++c) tma_load_4d(qt + c * kAttnBlock, &P.q, rfull, 64 * c, h0, t0, b);
        for (int c = 0; c < A.vb; ++c) tma_load_4d(dt + c * kAttnBlock, &P.dy, rfull, 64 * c, h0, t0, b);
      }
      __syncwarp();
    }
    for (int i = 0; i < steps; ++i) {
      const int k0 = (tk.j0 + i) * kAttnTile;
      const bool dirty = k0 < seq.k_lo || (k0 + kAttnTile > seq.k_hi && seq.k_hi < P.mask.sk);
      if (!K.load(guard, &P.k, A.kb, kAttnBlock, kh, k0, b, dirty, raw, raw_phase, kAttnTile, seq.k_lo - k0, seq.k_hi - k0, lane))
        break;
      if (!V.load(guard, &P.v, A.vb, kAttnBlock, kh, k0, b, false, raw, raw_phase, 0, 0, 0, lane)) break;
    }
    if (lane == 0) started.note(1, K.loads, V.loads);
  } else if (warp == kBwdWarps) {
    // S ahead of dQ where there are two places for S, else behind it
    RingAt K, behind;  // S's and dQ's tile of keys
    auto s_product = [&](int i) {
      if (!guard.wait_warp(kfull0 + 8 * K.stage, K.phase)) return false;
      tc_fence_after();
      if (elect_one()) {
        product_ss<kKb>(tmem + (i % C::kBufs) * 128, qt, kring + K.stage * C::kQTile, A.k_steps, kAttnBlock, kAttnTile);
        mma_commit_one(sfull0 + 8 * (i % C::kBufs));
      }
      __syncwarp();
      K.next(C::kKStages);
      return true;
    };
    bool ok = steps > 0 && guard.wait_warp(rfull, 0) && s_product(0);
    for (int i = 0; i < steps && ok; ++i) {
      if (C::kBufs == 2 && i + 1 < steps && !s_product(i + 1)) break;
      if (!guard.wait_warp(dsready0 + 8 * (i % C::kBufs), (i / C::kBufs) & 1)) break;
      tc_fence_after();
      if (elect_one()) {
        product_ts<8, 4>(tmem + C::kDq, tmem + (i % C::kBufs) * 128, 32, kring + behind.stage * C::kQTile, kAttnBlock,
                         A.k_steps * 16, i > 0);
        mma_commit_one(kempty0 + 8 * behind.stage);
      }
      __syncwarp();
      behind.next(C::kKStages);
      if (C::kBufs == 1 && i + 1 < steps) ok = s_product(i + 1);
    }
    drain_products(done0);
  } else if (warp == kBwdWarps + 1) {
    RingAt V;
    bool ok = steps > 0 && guard.wait_warp(rfull, 0);
    for (int i = 0; i < steps && ok; ++i) {
      if (!guard.wait_warp(vfull0 + 8 * V.stage, V.phase) || (i > 0 && !guard.wait_warp(dpread, (i - 1) & 1))) break;
      tc_fence_after();
      if (elect_one()) {
        product_ss<kVb>(tmem + C::kDp, dt, vring + V.stage * C::kDTile, A.v_cols / 16, kAttnBlock, kAttnTile);
        mma_commit_one(dpfull);
        mma_commit_one(vempty0 + 8 * V.stage);
      }
      __syncwarp();
      V.next(C::kVStages);
    }
    drain_products(done0 + 8);
  } else if (warp < kBwdWarps) {
    const int grp = warp >> 2, row = (warp & 3) * 32 + lane;
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const int token = t0 + (row >> A.pack), head = h0 + (row & ((1 << A.pack) - 1));
    const bool live = token >= seq.q_lo && token < seq.q_hi;
    Span keys = keys_of(P.mask, seq, docs, token);
    if (!live) keys = {0, 0};
    float2 stat = make_float2(-INFINITY, 0.f);
    if (live) {
      stat = P.stats[((int64_t)b * P.mask.sq + token) * A.q_heads + head];
    }
    const float2 c2 = make_float2(A.scale2, A.scale2), nl = make_float2(stat.x, stat.x), nd = make_float2(-stat.y, -stat.y);
    bool ok = true;
    for (int i = 0; i < steps; ++i) {
      const int buf = i % C::kBufs;
      const uint32_t S = trow + buf * 128 + grp * 32, D = trow + C::kDp + grp * 32;
      if (!(ok = guard.wait_warp(sfull0 + 8 * buf, (i / C::kBufs) & 1))) break;
      tc_fence_after();
      uint32_t r[32], g[32], w[16];
      tmem_read<32>(S, r);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        const float2 x = f2_fma(make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])), c2, nl);
        r[c] = __float_as_uint(ex2(x.x)), r[c + 1] = __float_as_uint(ex2(x.y));
      }
      if (!(ok = guard.wait_warp(dpfull, i & 1))) break;
      tc_fence_after();
      tmem_read<32>(D, g);
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dpread);
#pragma unroll
      for (int c = 0; c < 32; c += 2) {
        float2 x = f2_add(make_float2(__uint_as_float(g[c]), __uint_as_float(g[c + 1])), nd);
        x = f2_mul(x, make_float2(__uint_as_float(r[c]), __uint_as_float(r[c + 1])));
        g[c] = __float_as_uint(x.x), g[c + 1] = __float_as_uint(x.y);
      }
      if (tk.masked(tk.j0 + i)) {
        const int lo = keys.lo - (tk.j0 + i) * kAttnTile - grp * 32, hi = keys.hi - (tk.j0 + i) * kAttnTile - grp * 32;
#pragma unroll
        for (int c = 0; c < 32; ++c)
          if (c < lo || c >= hi) g[c] = 0u;
      }
#pragma unroll
      for (int c = 0; c < 16; ++c) w[c] = pack_bf16(__uint_as_float(g[2 * c]), __uint_as_float(g[2 * c + 1]));
      tmem_write<32>(S, w);
      tmem_put_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(dsready0 + 8 * buf);
    }
    if (ok) ok = guard.wait_warp(done0, 0);
    tc_fence_after();
    if (ok) {
      const int r0 = (warp & 3) * 32;
      for (int blk = grp; blk < A.kb; blk += 4) {  // through the queries' place
#pragma unroll 1
        for (int c = blk * 64; c < blk * 64 + 64; c += 32) {
          uint32_t r[32];
          float v[32];
          tmem_read<32>(trow + C::kDq + c, r);
#pragma unroll
          for (int e = 0; e < 32; ++e) v[e] = live ? __uint_as_float(r[e]) * A.scale : 0.f;
          put_tile_row(qt, row, c, v);
        }
        fence_async_smem();
        __syncwarp();
        if (lane == 0 && t0 + (r0 >> A.pack) < P.mask.sq) {
          tma_store_4d(&P.o1, qt + blk * kAttnBlock + r0 * 128, 64 * blk, h0, t0 + (r0 >> A.pack), b);
          bulk_commit();
          bulk_wait_read<0>();  // (the writes themselves end with the kernel)
        }
        __syncwarp();
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kBwdWarps) tmem_free(tmem, 512);
  if (warp == kBwdWarps + 2 && guard.aborted()) {
    started.settle_single(guard, rfull);
    started.settle_ring(guard, 1, kfull0, C::kKStages);
    started.settle_ring(guard, 2, vfull0, C::kVStages);
  }
}

// Both walks in one launch, the keys' tiles first: the queries' tiles start as the last
// of those end, and one tail is waited for instead of two (2 x 8192 causal 1147 -> 1111 us,
// 13 documents in 8192 tokens 175 -> 136).
struct BothParams {
  BwdParams keys, queries;
  int32_t key_tiles;  // CTAs of the keys' walk
};
constexpr int kBwdThreads = (kBwdWarps + 4) * 32;

template <int kKb, int kVb, int kQt>
__global__ void __launch_bounds__(kBwdThreads, 1) attn_backward_kernel(const __grid_constant__ BothParams P) {
  pdl_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  const int idx = blockIdx.x;
  if (idx < P.key_tiles) attn_dkv<kKb, kVb, kQt>(P.keys, smem, idx);
  else attn_dq<kKb, kVb>(P.queries, smem, idx - P.key_tiles);
}

// ---------------------------------------------------------------------------
// host

template <int kKb, int kVb>
cudaError_t launch_few(const DeltaParams &D, int64_t grid, int dev, cudaStream_t st) {
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(attn_few_kernel<kKb, kVb>, cudaFuncAttributeMaxDynamicSharedMemorySize, Few<kKb, kVb>::kSmem);
  });
  if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), attn_few_kernel<kKb, kVb>, dim3((unsigned)grid), dim3(32 * kFewWarps), Few<kKb, kVb>::kSmem,
                          st, 1, D);
}

template <int kKb, int kVb, int kQt>
cudaError_t launch_walks(const BothParams &P, int64_t grid, int dev, cudaStream_t st) {
  constexpr int kSmem = std::max(Dkv<kKb, kVb, kQt>::kSmem, Dq<kKb, kVb>::kSmem);
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(attn_backward_kernel<kKb, kVb, kQt>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
  });
  if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), attn_backward_kernel<kKb, kVb, kQt>, dim3((unsigned)grid), dim3(kBwdThreads), kSmem, st,
                          1, P);
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" size_t gbo_attn_backward_workspace_bytes(const gbo_attn_args *args) {
  if (check_attn_sizes(args) != GBO_OK) return 0;
  return (size_t)args->batch * args->sq * args->q_heads * sizeof(float2);
}

extern "C" int gbo_attn_backward(const gbo_attn_args *a, const gbo_attn_grads *g, void *workspace, size_t ws_bytes,
                                 int32_t *dev_status, gbo_stream_t stream) {
  int rc = check_attn(a);
  if (rc != GBO_OK) return rc;
  if (!g) return attn_fail(GBO_ERR_INVALID_ARG, "grads is NULL");
  if ((reinterpret_cast<uintptr_t>(g->lse) | reinterpret_cast<uintptr_t>(dev_status)) & 3)
    return attn_fail(GBO_ERR_INVALID_ARG, "misaligned lse or status pointer");
  const bool queries = a->batch > 0 && a->sq > 0, keys = a->batch > 0 && a->sk > 0;
  if (queries && keys) {
    if ((rc = check_heads(g->dy, g->dy_stride, a->batch, a->sq, a->q_heads)) != GBO_OK) return rc;
    if ((rc = check_heads(g->y, g->y_stride, a->batch, a->sq, a->q_heads)) != GBO_OK) return rc;
    if (!g->lse) return attn_fail(GBO_ERR_INVALID_ARG, "lse is NULL");
  }
  if (queries && g->dq && (rc = check_heads(g->dq, g->dq_stride, a->batch, a->sq, a->q_heads)) != GBO_OK) return rc;
  if (keys && g->dk && (rc = check_heads(g->dk, g->dk_stride, a->batch, a->sk, a->k_heads)) != GBO_OK) return rc;
  if (keys && g->dv && (rc = check_heads(g->dv, g->dv_stride, a->batch, a->sk, a->k_heads)) != GBO_OK) return rc;
  int dev, sm = 0;
  if ((rc = attn_device(&dev, &sm)) != GBO_OK) return rc;
  const int64_t rows = a->batch * a->sq * a->q_heads;
  if (queries && keys) {
    if (!workspace || ws_bytes < (size_t)rows * sizeof(float2))
      return attn_fail(GBO_ERR_WORKSPACE, "workspace missing or smaller than gbo_attn_backward_workspace_bytes");
    if (reinterpret_cast<uintptr_t>(workspace) & 255) return attn_fail(GBO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  }
  AttnShape S;
  AttnMask M;
  fill_shape(a, &S, &M, kAttnMaxPack);
  const int cfg = attn_config(a);
  const int qt = cfg == 2 ? 64 : kAttnTile;  // rows of a step of the keys' walk
  const uint32_t heads = 1u << S.pack;
  const int64_t q_tiles = (a->sq + (kAttnTile >> S.pack) - 1) / (kAttnTile >> S.pack), k_tiles = (a->sk + kAttnTile - 1) / kAttnTile;
  const int64_t dkv_grid = keys && (g->dk || g->dv) ? k_tiles * a->batch * a->k_heads : 0;
  const int64_t dq_grid = queries && g->dq ? q_tiles * a->batch * a->k_heads * S.head_blocks : 0;
  if (dkv_grid + dq_grid > INT32_MAX || rows > (int64_t)INT32_MAX * 16)
    return attn_fail(GBO_ERR_SHAPE, "more rows than one launch takes");
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = cudaSuccess;
  BothParams both;
  memset(&both, 0, sizeof both);
  BwdParams &P = both.keys, &Q = both.queries;
  P.mask = M, P.shape = S, P.stats = static_cast<const float2 *>(workspace), P.status = dev_status;
  Q.mask = M, Q.shape = S, Q.stats = P.stats, Q.status = dev_status;
  DeltaParams D;
  memset(&D, 0, sizeof D);
  int64_t few_grid = 0;
  bool maps = true;
  if (queries && keys) {
    D.dy = static_cast<const __nv_bfloat16 *>(g->dy), D.y = static_cast<const __nv_bfloat16 *>(g->y);
    D.lse = g->lse, D.stats = static_cast<float2 *>(workspace);
    const int64_t extent[3] = {a->batch, a->sq, a->q_heads};
    const int64_t k_extent[3] = {a->batch, a->sk, a->k_heads};
    for (int i = 0; i < 3; ++i) {
      D.ds[i] = extent[i] > 1 ? g->dy_stride[i] : 0, D.ys[i] = extent[i] > 1 ? g->y_stride[i] : 0;
      D.qs[i] = extent[i] > 1 ? a->q_stride[i] : 0;
      D.ks[i] = k_extent[i] > 1 ? a->k_stride[i] : 0, D.vs[i] = k_extent[i] > 1 ? a->v_stride[i] : 0;
    }
    D.q = static_cast<const __nv_bfloat16 *>(a->q), D.k = static_cast<const __nv_bfloat16 *>(a->k);
    D.v = static_cast<const __nv_bfloat16 *>(a->v);
    D.rows = rows, D.sq = (int32_t)a->sq, D.heads = a->q_heads, D.dk = a->dk, D.dv = a->dv;
    D.by_heads = fast_div(a->q_heads), D.by_sq = fast_div(a->sq);
    D.mask = M, D.scale2 = S.scale2, D.group = S.group;
    // (documents so short that looking at the first tokens of each is looking at more than all)
    D.all = a->sk <= kFewKeys || (a->window > 0 && a->window <= kFewKeys);
    D.every = D.all || (!a->causal && a->k_lengths) || (a->documents && (int64_t)a->n_documents * kFewKeys >= a->sq);
    D.pack = std::min(S.pack, 4);
    const int64_t units = D.every ? a->batch : a->documents ? a->n_documents : a->causal ? a->batch : 0;
    const int64_t tokens = 16 >> D.pack, blocks = S.group >> D.pack;
    const int64_t sets = ((D.every ? a->sq : kFewKeys) + tokens - 1) / tokens * blocks, chunks = (sets + kFewWarps - 1) / kFewWarps;
    // (where they are more than a launch takes: D = dy . y throughout)
    few_grid = sets <= INT32_MAX - kFewWarps && units * a->k_heads * chunks <= INT32_MAX ? units * a->k_heads * chunks : 0;
    D.all = D.all && few_grid;
    D.sets = (int32_t)sets, D.by_chunks = fast_div(chunks), D.by_k_heads = S.by_k_heads, D.by_blocks = fast_div(blocks);
    maps = heads_map(&P.k, a->k, a->dk, a->k_heads, a->sk, a->batch, a->k_stride, 1, kAttnTile) &&
           heads_map(&P.v, a->v, a->dv, a->k_heads, a->sk, a->batch, a->v_stride, 1, kAttnTile) &&
           heads_map(&P.q, a->q, a->dk, a->q_heads, a->sq, a->batch, a->q_stride, heads, qt >> S.pack) &&
           heads_map(&P.dy, g->dy, a->dv, a->q_heads, a->sq, a->batch, g->dy_stride, heads, qt >> S.pack);
    Q.k = P.k, Q.v = P.v, Q.q = P.q, Q.dy = P.dy;
    if (qt != kAttnTile)
      maps = maps && heads_map(&Q.q, a->q, a->dk, a->q_heads, a->sq, a->batch, a->q_stride, heads, kAttnTile >> S.pack) &&
             heads_map(&Q.dy, g->dy, a->dv, a->q_heads, a->sq, a->batch, g->dy_stride, heads, kAttnTile >> S.pack);
  }
  if (dkv_grid && g->dk) maps = maps && heads_map(&P.o1, g->dk, a->dk, a->k_heads, a->sk, a->batch, g->dk_stride, 1, 32);
  if (dkv_grid && g->dv) maps = maps && heads_map(&P.o2, g->dv, a->dv, a->k_heads, a->sk, a->batch, g->dv_stride, 1, 32);
  if (dq_grid) maps = maps && heads_map(&Q.o1, g->dq, a->dk, a->q_heads, a->sq, a->batch, g->dq_stride, heads, 32 >> S.pack);
  if (!maps) return attn_fail(GBO_ERR_CUDA, "tensor map of queries, keys, values or gradients");
  P.has1 = g->dk != nullptr, P.has2 = g->dv != nullptr;
  Q.tiles = (int32_t)q_tiles;
  if (queries && keys && (dkv_grid || dq_grid)) {
    if (!D.all) {
      count_launches(1);
      e = launch_kernel_as(pdl_allowed(), attn_delta_kernel, dim3((unsigned)((rows + kDeltaRows - 1) / kDeltaRows)), dim3(256), 0, st, 1, D);
    }
    if (e == cudaSuccess && few_grid)
      e = cfg == 0 ? launch_few<1, 1>(D, few_grid, dev, st)
                   : cfg == 1 ? launch_few<2, 2>(D, few_grid, dev, st) : launch_few<3, 2>(D, few_grid, dev, st);
  }
  both.key_tiles = (int32_t)dkv_grid;
  const int64_t grid = dkv_grid + dq_grid;
  if (e == cudaSuccess && grid)
    e = cfg == 0 ? launch_walks<1, 1, 128>(both, grid, dev, st)
                 : cfg == 1 ? launch_walks<2, 2, 128>(both, grid, dev, st) : launch_walks<3, 2, 64>(both, grid, dev, st);
  return e == cudaSuccess ? report_ok() : attn_cuda(e);
}

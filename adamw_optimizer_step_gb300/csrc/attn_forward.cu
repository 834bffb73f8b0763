// Attention, forward (gbo_attn_forward): y_i = sum_j softmax_j(scale q_i k_j) v_j
// over the keys j that query i sees, and lse_i = log sum_j exp(scale q_i k_j).
//
//   attn_forward_kernel  many rows: tcgen05 products of 128 x 128 tiles
//   attn_token_kernel    at most 16 rows a key head (answering): one pass over the cache
//   attn_join_kernel     joins the parts of rows whose keys were split over CTAs
//
// attn_forward_kernel.  A CTA holds two tiles of 128 rows (heads of consecutive
// tokens, see AttnShape) and streams their keys and values in tiles of 128.
// Per tile of rows and of keys: S = Q K^T (TMEM), P = 2^(S c - m) with c =
// scale log2(e) by the eight warps of the row tile, half a row to a thread, back
// into TMEM in bf16 over S, O += P V (TMEM).  While the softmax of one row tile
// runs, the tensor cores work for the other: PV0(j-1) S0(j) PV1(j-1) S1(j).  What
// bounds that turn is the time from S to P, so P V starts with the first half of each
// warp's P while the second is formed (2 x 8192 tokens: 380 -> 344 us), and that
// first half is formed from the maximum so far while the row's two warps exchange
// theirs (344 -> 339), again where the maximum moves.
// m is a running maximum that is moved, and O rescaled, only when a row's
// maximum grows by more than 2^8: until then P is at most 2^8 and its rounding
// is relative, so nothing is lost; sums are fp32.  P is rounded to bf16 once
// (2^-8 of it at most, as the operand of the product); the sum takes it unrounded.
// Measured, causal, 16 query and 4 key heads of 128: 2 x 8192 tokens 330 us at best, 356 over
// a second of calls (the power limit holds the clock at 1.88 GHz), 1.67 and 1.55 PFLOP/s of the
// products that count: 87% of a library product's burst, 91% of its sustained rate.  Heads of
// 192 and 128, V's ring of one stage: 540 us, 1.27 PFLOP/s at 2.0 GHz.  512 new tokens over a
// cache of 32768 (keys split, parts joined) 103 us, 1.33; four equal parts are 128 CTAs on
// 152 SMs.  Bound: the turn of the two row tiles, S to softmax to P V; the warps issue 39% of
// the time, mostly waiting for products.  Short sequences (documents, 777 tokens) are bound by
// a CTA's start and end, some 9000 clocks: 57 us at 1.5 to 2.0 TB/s.  A CTA that walks over
// several tiles instead (one launch of resident CTAs) lost at every length.
#include "attn_common.cuh"

namespace gbo {

namespace {

constexpr int kFwdSoftWarps = 16;  // for each row tile two groups of four, each half of the keys
constexpr int kFwdThreads = (kFwdSoftWarps + 3) * 32;
constexpr float kRescale = 8.f;  // in bits
constexpr float kLn2 = 0.6931471805599453f;

template <int kKb, int kVb>
struct Fwd {
  static constexpr int kQTile = kKb * kAttnBlock, kVTile = kVb * kAttnBlock;  // (a tile of keys is as large as one of queries)
  static constexpr int kKStages = kKb == 1 ? 5 : kKb == 2 ? 3 : 2, kVStages = kKb == 1 ? 5 : kKb == 2 ? 2 : 1;
  static constexpr int kKRing = 2 * kQTile, kVRing = kKRing + kKStages * kQTile;
  static constexpr int kUsed = kVRing + kVStages * kVTile;
  // queries (two), keys and values full/empty, raw, S, P, P's second half, O (two each), pairs of warps, drained (two),
  // turns (two)
  static constexpr int kBars = 2 + 2 * kKStages + 2 * kVStages + 1 + 8 + 8 + 2 + 2;
  static constexpr int kHalves = 2 * 2 * kAttnTile * 4;  // half of the keys, row tile, row: a float
  static constexpr int kSmem = kUsed + kHalves + kBars * 8 + kNotes;
  static constexpr uint32_t kO = 256;  // TMEM: S0, S1 of 128 columns, O0, O1 of kVb * 64
  static constexpr uint32_t kCols = 512;
  static_assert(kVb * kAttnBlock <= kQTile, "the output leaves through the queries' place");
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

struct FwdParams {
  CUtensorMap q, k, v, y;
  AttnMask mask;
  AttnShape shape;
  float *lse;       // or NULL
  float *part_o;    // splits > 1: splits x rows x dv, and their lse (in bits)
  float *part_lse;
  int32_t *status;
  int64_t rows;     // batch * sq * q_heads
  int32_t token_blocks, splits;
  FastDiv by_splits;
};

template <int kKb, int kVb>
__global__ void __launch_bounds__(kFwdThreads, 1) attn_forward_kernel(const __grid_constant__ FwdParams P) {
  using C = Fwd<kKb, kVb>;
  pdl_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  float *const halves = reinterpret_cast<float *>(smem + C::kUsed);
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kUsed + C::kHalves);
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(bars + C::kBars);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(tmem_slot + 1);
  const uint32_t qfull0 = smem_u32(bars), kfull0 = qfull0 + 16, kempty0 = kfull0 + 8 * C::kKStages;
  const uint32_t vfull0 = kempty0 + 8 * C::kKStages, vempty0 = vfull0 + 8 * C::kVStages, raw = vempty0 + 8 * C::kVStages;
  const uint32_t sfull0 = raw + 8, pready0 = sfull0 + 16, prest0 = pready0 + 16, odone0 = prest0 + 16, pair0 = odone0 + 16;
  const uint32_t drain0 = pair0 + 64, turn0 = drain0 + 16;
  const int warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) mbar_init(qfull0 + 8 * s, 1);
    for (int s = 0; s < C::kKStages; ++s) {
      mbar_init(kfull0 + 8 * s, 1);
      mbar_init(kempty0 + 8 * s, 2);  // both row tiles
    }
    for (int s = 0; s < C::kVStages; ++s) {
      mbar_init(vfull0 + 8 * s, 1);
      mbar_init(vempty0 + 8 * s, 2);
    }
    mbar_init(raw, 1);
    for (int t = 0; t < 2; ++t) {
      mbar_init(sfull0 + 8 * t, 1);
      mbar_init(pready0 + 8 * t, 8);
      mbar_init(prest0 + 8 * t, 8);
      mbar_init(odone0 + 8 * t, 1);
    }
    for (int t = 0; t < 8; ++t) mbar_init(pair0 + 8 * t, 2);
    for (int t = 0; t < 4; ++t) mbar_init(drain0 + 8 * t, 1);  // (and turns)
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  if (warp == kFwdSoftWarps) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                 "r"(C::kCols)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
  }
  pdl_wait();

  const AttnShape &A = P.shape;
  // later queries first: with a causal mask they have the most keys
  int idx = blockIdx.x;
  const int split = P.by_splits.split(idx);
  int kh = A.by_all.split(idx);
  const int b = A.by_batch.split(idx), tb = P.token_blocks - 1 - idx;
  const int hb = A.by_blocks.split(kh), h0 = kh * A.group + (hb << A.pack);
  const int tokens = kAttnTile >> A.pack, t0 = tb * 2 * tokens;
  const AttnSeq seq = attn_seq(P.mask, b);
  TileKeys tk[2];
  const DocWindow docs = doc_window(P.mask, t0);
  for (int t = 0; t < 2; ++t) tk[t] = tile_keys(P.mask, seq, docs, t0 + t * tokens, tokens);
  // the keys of both tiles together, and this CTA's share of them
  int J0 = 0, J1 = 0;
  if (tk[0].j1 > tk[0].j0) J0 = tk[0].j0, J1 = tk[0].j1;
  if (tk[1].j1 > tk[1].j0) {
    J0 = J1 > J0 ? min(J0, tk[1].j0) : tk[1].j0;
    J1 = max(J1, tk[1].j1);
  }
  if (P.splits > 1) {
    const int each = (J1 - J0 + P.splits - 1) / P.splits, from = J0 + split * each;
    J1 = min(J1, from + each);
    J0 = from;
    for (int t = 0; t < 2; ++t) {
      tk[t].j0 = max(tk[t].j0, J0);
      tk[t].j1 = max(tk[t].j0, min(tk[t].j1, J1));
    }
  }
  if (P.splits == 1 && J1 <= J0) {
    zero_block(smem);
    if (threadIdx.x == 0) {
      for (int r0 = 0; r0 < 2 * kAttnTile && t0 + (r0 >> A.pack) < P.mask.sq; r0 += 32)
        for (int c = 0; c < A.vb; ++c) tma_store_4d(&P.y, smem_u32(smem), 64 * c, h0, t0 + (r0 >> A.pack), b);
      bulk_commit();
      bulk_wait_read<0>();
    }
    for (int r = threadIdx.x; P.lse && r < 2 * kAttnTile; r += kFwdThreads) {
      const int token = t0 + (r >> A.pack), head = h0 + (r & ((1 << A.pack) - 1));
      if (token < P.mask.sq) P.lse[((int64_t)b * P.mask.sq + token) * A.q_heads + head] = -INFINITY;
    }
    if (warp == kFwdSoftWarps) tmem_free(*tmem_slot, C::kCols);
    return;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const uint32_t q0 = smem_u32(smem), kring = q0 + C::kKRing, vring = q0 + C::kVRing;
  const AttnGuard guard = {abort_flag, P.status};
  const Started started = {abort_flag + 1};

  if (warp == kFwdSoftWarps + 2) {
    uint32_t raw_phase = 0;
    TileRing K(kfull0, kempty0, kring, C::kQTile, C::kKStages), V(vfull0, vempty0, vring, C::kVTile, C::kVStages);
    int32_t queries = 0;
    for (int t = 0; t < 2; ++t)
      if (tk[t].j1 > tk[t].j0) {
        if (elect_one()) {
          mbar_expect_tx(qfull0 + 8 * t, (uint32_t)A.kb * kAttnBlock);
          for (int c = 0; c < A.kb; ++c)
            tma_load_4d(q0 + t * C::kQTile + c * kAttnBlock, &P.q, qfull0 + 8 * t, 64 * c, h0, t0 + t * tokens, b);
        }
        __syncwarp();
        queries |= 1 << t;
      }
    for (int j = J0; j < J1; ++j) {
      const int k0 = j * kAttnTile;
      if (!K.load(guard, &P.k, A.kb, kAttnBlock, kh, k0, b, false, raw, raw_phase, 0, 0, 0, lane)) break;
      const bool dirty = k0 < seq.k_lo || (k0 + kAttnTile > seq.k_hi && seq.k_hi < P.mask.sk);
      if (!V.load(guard, &P.v, A.vb, kAttnBlock, kh, k0, b, dirty, raw, raw_phase, kAttnTile, seq.k_lo - k0, seq.k_hi - k0, lane))
        break;
    }
    if (lane == 0) started.note(queries, K.loads, V.loads);
  } else if (warp >= kFwdSoftWarps) {
    // The tensor cores' work for row tile t: steps of PV(j - 1) and S(j); P stands
    // over S, and one thread's products run in order.  Each tile has a warp of its
    // own, whose waits lie beside the other's products, and the two take turns: with
    // products of both at once the tiles fall in step, and the tensor cores rest while
    // both wait for their softmax (474 us instead of 381 at 2 x 8192 tokens x 16 heads of 128, before P came in halves).
    const int t = warp - kFwdSoftWarps;
    const uint32_t S = tmem + t * 128, O = tmem + C::kO + t * kVb * 64, q = q0 + t * C::kQTile;
    bool started = false;
    uint32_t np = 0, turn = t ^ 1;
    RingAt K, V;
    for (int j = J0; j <= J1 && J1 > J0; ++j) {
      const bool pv = j > J0 && tk[t].has(j - 1), sc = j < J1 && tk[t].has(j);
      if (j > J0 && !guard.wait_warp(vfull0 + 8 * V.stage, V.phase)) break;
      if (j < J1 && !guard.wait_warp(kfull0 + 8 * K.stage, K.phase)) break;
      if (sc && !started && !guard.wait_warp(qfull0 + 8 * t, 0)) break;
      started |= sc;
      if (pv && !guard.wait_warp(pready0 + 8 * t, np & 1)) break;
      if (!guard.wait_warp(turn0 + 8 * t, turn)) break;
      turn ^= 1;
      tc_fence_after();
      if (pv) {
        const uint32_t v = vring + V.stage * C::kVTile;
        if (elect_one()) product_ts<8, 2, 0, 2>(O, S, 64, v, kAttnBlock, A.v_cols, np > 0);
        __syncwarp();
        if (!guard.wait_warp(prest0 + 8 * t, np & 1)) break;
        tc_fence_after();
      }
      if (elect_one()) {
        if (pv) {
          product_ts<8, 2, 2, 4>(O, S, 64, vring + V.stage * C::kVTile, kAttnBlock, A.v_cols, true);
          mma_commit_one(odone0 + 8 * t);
          mma_commit_one(vempty0 + 8 * V.stage);
        } else if (j > J0) {
          mbar_arrive(vempty0 + 8 * V.stage);
        }
        if (sc) product_ss<kKb>(S, q, kring + K.stage * C::kQTile, A.k_steps, kAttnBlock, kAttnTile);
        mbar_arrive(turn0 + 8 * (t ^ 1));
        if (sc) {
          mma_commit_one(sfull0 + 8 * t);
          mma_commit_one(kempty0 + 8 * K.stage);
        } else if (j < J1) {
          mbar_arrive(kempty0 + 8 * K.stage);
        }
      }
      __syncwarp();
      np += pv;
      if (j > J0) V.next(C::kVStages);
      if (j < J1) K.next(C::kKStages);
    }
    drain_products(drain0 + 8 * t);
  } else {
    // Rows of tile t, keys 64 half .. of each of its key tiles.  The two warps of
    // a row exchange their maxima, and their sums at the end.
    const int t = warp >> 3, half = warp >> 2 & 1, row = (warp & 3) * 32 + lane;
    const uint32_t pair = pair0 + 8 * (t * 4 + (warp & 3));
    const uint32_t trow = tmem + ((uint32_t)((warp & 3) * 32) << 16);
    const uint32_t S = trow + t * 128 + half * 64, O = trow + C::kO + t * kVb * 64;
    const int token = t0 + t * tokens + (row >> A.pack), head = h0 + (row & ((1 << A.pack) - 1));
    const bool live = token >= seq.q_lo && token < seq.q_hi;
    Span keys = keys_of(P.mask, seq, docs, token);
    if (!live) keys = {0, 0};
    float m = -INFINITY, l = 0.f;
    bool ok = true;
    int n = 0;
    float *const my_slot = halves + (half * 2 + t) * kAttnTile + row;
    const float *const their_slot = halves + ((half ^ 1) * 2 + t) * kAttnTile + row;
    // This row's value of the other warp, from share() to theirs().  A slot is written
    // again only after products that waited for both warps' P, and so for their reads.
    auto share = [&](float v) {
      *my_slot = v;
      __syncwarp();
      if (lane == 0) mbar_arrive(pair);
    };
    auto theirs = [&](int turn, float &other) {
      if (!guard.wait_warp(pair, turn & 1)) return false;
      other = *their_slot;
      return true;
    };
    for (int j = tk[t].j0; j < tk[t].j1; ++j, ++n) {
      if (!(ok = guard.wait_warp(sfull0 + 8 * t, n & 1))) break;
      tc_fence_after();
      const bool masked = tk[t].masked(j);
      const int lo = keys.lo - j * kAttnTile - half * 64, hi = keys.hi - j * kAttnTile - half * 64;
      const float2 c2 = make_float2(A.scale2, A.scale2);
      float2 sum[2];
      uint32_t p[16];
      // P of 32 scores, and their sums
      auto exponentials = [&](const uint32_t *r) {
        const float at = m == -INFINITY ? 0.f : -m;
        const float2 at2 = make_float2(at, at);
#pragma unroll
        for (int c = 0; c < 16; ++c) {
          float2 x = f2_fma(make_float2(__uint_as_float(r[2 * c]), __uint_as_float(r[2 * c + 1])), c2, at2);
          x.x = ex2(x.x), x.y = ex2(x.y);
          sum[c & 1] = f2_add(sum[c & 1], x);
          p[c] = pack_bf16(x.x, x.y);
        }
      };
      auto half_of_row = [&](int h) {
        uint32_t r[32];
        tmem_read<32>(S + 32 * h, r);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 32; ++c)
            if (32 * h + c < lo || 32 * h + c >= hi) r[c] = 0xff800000u;
        }
        exponentials(r);
      };
      sum[0] = sum[1] = make_float2(0.f, 0.f);
      float mine, other;
      {
        float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
        uint32_t r[64];
        tmem_read<64>(S, r);
        if (masked) {
#pragma unroll
          for (int c = 0; c < 64; ++c)
            if (c < lo || c >= hi) r[c] = 0xff800000u;  // -inf
        }
#pragma unroll
        for (int c = 0; c < 64; c += 8)
#pragma unroll
          for (int e = 0; e < 4; ++e) mx[e] = max3(mx[e], __uint_as_float(r[c + e]), __uint_as_float(r[c + e + 4]));
        mine = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3]));
        share(mine);
        // the first half beside the exchange, from the maximum so far: it mostly stays
        exponentials(r);
      }
      if (!(ok = theirs(n, other))) break;
      const float mn = fmaxf(m, fmaxf(mine, other) * A.scale2);
      if (__any_sync(0xffffffffu, mn > m + kRescale)) {
        const float a = ex2(m - (mn == -INFINITY ? 0.f : mn));  // (m = -inf: 0)
        l *= a;
        m = mn;
        if (n > 0) {
          if (!(ok = guard.wait_warp(odone0 + 8 * t, (n - 1) & 1))) break;
          tc_fence_after();
#pragma unroll 1
          for (int c = half * 32; c < A.vb * 64; c += 64) {
            uint32_t o[32];
            tmem_read<32>(O + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * a);
            tmem_put(O + c, o);
          }
        }
        sum[0] = sum[1] = make_float2(0.f, 0.f);
        half_of_row(0);
      }
      tmem_put16(S, p);
      tmem_put_wait();  // (the product starts with this half)
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(pready0 + 8 * t);
      half_of_row(1);
      tmem_put16(S + 16, p);
      const float2 both = f2_add(sum[0], sum[1]);
      l += both.x + both.y;
      tmem_put_wait();
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(prest0 + 8 * t);
    }
    if (ok && n > 0) {
      float other = 0.f;
      ok = guard.wait_warp(odone0 + 8 * t, (n - 1) & 1);
      share(l);
      ok = ok && theirs(n, other);
      l += other;
    }
    tc_fence_after();
    if (ok && t0 + t * tokens < P.mask.sq) {
      const bool in = token < P.mask.sq;
      const int64_t at = ((int64_t)b * P.mask.sq + token) * A.q_heads + head;
      // (a sum of 0 is a row that sees nothing; NaN stays)
      const float inv = live && l != 0.f ? 1.f / l : 0.f;
      if (P.splits == 1) {
        if (in && P.lse && half == 0) P.lse[at] = live ? m * kLn2 + logf(l) : -INFINITY;
        const uint32_t out = q0 + t * C::kQTile;  // the queries have been read
        for (int blk = half; blk < A.vb; blk += 2) {  // 64 columns
#pragma unroll 1
          for (int c = blk * 64; c < blk * 64 + 64; c += 32) {
            uint32_t o[32];
            float f[32];
            if (n > 0) tmem_read<32>(O + c, o);
#pragma unroll
            for (int e = 0; e < 32; ++e) f[e] = n > 0 && inv != 0.f ? __uint_as_float(o[e]) * inv : 0.f;
            put_tile_row(out, row, c, f);
          }
          fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            const int r0 = (warp & 3) * 32;  // this warp's rows
            tma_store_4d(&P.y, out + blk * kAttnBlock + r0 * 128, 64 * blk, h0, t0 + t * tokens + (r0 >> A.pack), b);
            bulk_commit();
            bulk_wait_read<0>();  // (the writes themselves end with the kernel)
          }
          __syncwarp();
        }
      } else {
        if (in && half == 0) P.part_lse[split * P.rows + at] = live && l != 0.f ? m + log2f(l) : -INFINITY;
        float *dst = P.part_o + (split * P.rows + at) * A.dv;
#pragma unroll 1
        for (int c = half * 32; c < A.dv; c += 64) {
          uint32_t o[32];
          if (n > 0) tmem_read<32>(O + c, o);
#pragma unroll
          for (int q = 0; q < 8; ++q)
            if (in && c + 4 * q < A.dv) {
              float4 f = make_float4(0.f, 0.f, 0.f, 0.f);
              if (n > 0 && inv != 0.f)
                f = make_float4(__uint_as_float(o[4 * q]) * inv, __uint_as_float(o[4 * q + 1]) * inv,
                                __uint_as_float(o[4 * q + 2]) * inv, __uint_as_float(o[4 * q + 3]) * inv);
              *reinterpret_cast<float4 *>(dst + c + 4 * q) = f;
            }
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == kFwdSoftWarps) tmem_free(tmem, C::kCols);
  if (warp == kFwdSoftWarps + 2 && guard.aborted()) {
    started.settle_single(guard, qfull0);
    started.settle_ring(guard, 1, kfull0, C::kKStages);
    started.settle_ring(guard, 2, vfull0, C::kVStages);
  }
}

// ---------------------------------------------------------------------------
// few rows: one pass over the keys and values of a key head

// Rows of a key head are its query heads' tokens, at most 16 (one M of
// mma.sync): a product costs a sixteenth of what its bytes cost, so the pass is
// bound by HBM.  Stages of 64 keys and values come by TMA; each of four warps
// takes 16 of the keys, with a running maximum, sum and output of its own, and
// the four are joined at the end.  Two CTAs an SM, so that one's start and end
// lie beside the other's stream.  Eight sequences' caches of 32768 to 65536 tokens, 4 key
// heads of 128: 133 us, 6.1 TB/s (89% of a copy's rate).
constexpr int kTokKeys = 64, kTokWarps = 4;
constexpr int kTokThreads = (kTokWarps + 1) * 32;
constexpr int kTokBlock = kTokKeys * 128;  // bytes of 64 rows of 64 elements

template <int kKb, int kVb>
struct Tok {
  static constexpr int kStage = (kKb + kVb) * kTokBlock;
  static constexpr int kStages = kKb == 1 ? 6 : kKb == 2 ? 3 : 2;
  static constexpr int kJoin = kTokWarps * 16 * (kVb * 64 + 4) * 4;  // outputs, maxima and sums of the warps
  static constexpr int kUsed = kStages * kStage > kJoin ? kStages * kStage : kJoin;
  static constexpr int kSmem = kUsed + (2 * kStages) * 8 + kNotes;
  static_assert(kSmem <= 113 * 1024, "two CTAs an SM");
};

struct TokParams {
  CUtensorMap k, v;
  AttnMask mask;
  AttnShape shape;
  const __nv_bfloat16 *q;
  __nv_bfloat16 *y;
  int64_t qs[3], ys[3];
  float *lse, *part_o, *part_lse;
  int32_t *status;
  int64_t rows;
  int32_t splits, group;
};

__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void ldsm4_trans(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void mma16816(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Address of 8 elements from column c (a multiple of 8) of row r of a stage's tile.
__device__ __forceinline__ uint32_t tok_at(uint32_t tile, int r, int c) {
  return tile + (uint32_t)(c >> 6) * kTokBlock + (uint32_t)r * 128u + ((uint32_t)(((c & 63) >> 3) ^ (r & 7)) << 4);
}

template <int kKb, int kVb>
__global__ void __launch_bounds__(kTokThreads, 2) attn_token_kernel(const __grid_constant__ TokParams P) {
  using C = Tok<kKb, kVb>;
  pdl_launch();
  extern __shared__ __align__(1024) uint8_t smem[];
  uint64_t *bars = reinterpret_cast<uint64_t *>(smem + C::kUsed);
  volatile int32_t *abort_flag = reinterpret_cast<volatile int32_t *>(bars + 2 * C::kStages);
  const uint32_t full0 = smem_u32(bars), empty0 = full0 + 8 * C::kStages, ring0 = smem_u32(smem);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < C::kStages; ++s) {
      mbar_init(full0 + 8 * s, 1);
      mbar_init(empty0 + 8 * s, kTokWarps);
    }
    *abort_flag = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  pdl_wait();
  const AttnShape &A = P.shape;
  int idx = blockIdx.x;
  const int split = idx % P.splits;
  idx /= P.splits;
  const int kh = idx % A.k_heads, b = idx / A.k_heads;
  const AttnSeq seq = attn_seq(P.mask, b);
  // stages that some row sees, and this CTA's share
  const int a0 = max(0, seq.q_lo), a1 = min(P.mask.sq, seq.q_hi);
  const DocWindow docs = doc_window(P.mask, a0);
  int J0 = 0, J1 = 0;
  if (a1 > a0) {
    const Span first = keys_of(P.mask, seq, docs, a0), last = keys_of(P.mask, seq, docs, a1 - 1);
    if (last.hi > first.lo) J0 = first.lo / kTokKeys, J1 = (last.hi + kTokKeys - 1) / kTokKeys;
  }
  const int each = (J1 - J0 + P.splits - 1) / P.splits;
  J0 += split * each;
  J1 = min(J1, J0 + each);
  const AttnGuard guard = {abort_flag, P.status};
  const Started started = {abort_flag + 1};
  const int blocks = A.kb + A.vb;
  const int rows = P.group * P.mask.sq;  // row r: token r / group, head r % group
  bool ok = true;
  float m[2] = {-INFINITY, -INFINITY}, l[2] = {0.f, 0.f};
  float o[kVb * 8][4];
#pragma unroll
  for (int n = 0; n < kVb * 8; ++n)
#pragma unroll
    for (int e = 0; e < 4; ++e) o[n][e] = 0.f;

  if (warp == kTokWarps) {
    if (lane == 0) {
      uint32_t phase = 0;
      int s = 0, j = J0;
      for (; j < J1; ++j) {
        if (!guard.wait(empty0 + 8 * s, phase ^ 1)) break;
        mbar_expect_tx(full0 + 8 * s, (uint32_t)(blocks * kTokBlock));
        const uint32_t st = ring0 + s * C::kStage;
        for (int c = 0; c < A.kb; ++c) tma_load_4d(st + c * kTokBlock, &P.k, full0 + 8 * s, 64 * c, kh, j * kTokKeys, b);
        for (int c = 0; c < A.vb; ++c)
          tma_load_4d(st + (kKb + c) * kTokBlock, &P.v, full0 + 8 * s, 64 * c, kh, j * kTokKeys, b);
        if (++s == C::kStages) s = 0, phase ^= 1;
      }
      started.note(0, j - J0, 0);
    }
  } else if (J1 > J0) {
    // the two rows of this lane, and the queries as the A operand
    const int r0 = lane >> 2, c0 = (lane & 3) * 2;
    uint32_t qa[kKb * 4][4];
    Span keys[2] = {{0, 0}, {0, 0}};
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int r = r0 + 8 * h, t = r / P.group, head = kh * P.group + r % P.group;
      const bool in = r < rows && t >= seq.q_lo && t < seq.q_hi;
      const Span seen = keys_of(P.mask, seq, docs, t);
      if (in) keys[h] = seen;
      const __nv_bfloat16 *src = P.q + (b * P.qs[0] + t * P.qs[1] + head * P.qs[2]);
#pragma unroll
      for (int k = 0; k < kKb * 4; ++k)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const int c = k * 16 + e * 8 + c0;
          qa[k][h + 2 * e] = in && c < A.dk ? *reinterpret_cast<const uint32_t *>(src + c) : 0u;
        }
    }
    int s = 0;
    uint32_t phase = 0;
    const int key0 = warp * 16;  // this warp's keys of a stage
    for (int j = J0; j < J1; ++j) {
      if (!(ok = guard.wait_warp(full0 + 8 * s, phase))) break;
      const uint32_t kt = ring0 + s * C::kStage, vt = kt + kKb * kTokBlock;
      const int at = j * kTokKeys + key0;
      if (at < seq.k_lo || (at + 16 > seq.k_hi && seq.k_hi < P.mask.sk)) {
        // values that no row sees may hold anything, and 0 x NaN is not 0
        for (int c = lane; c < 16 * 8 * A.vb; c += 32) {
          const int r = key0 + (c >> 3) % 16, blk = c / 128, key = j * kTokKeys + r;
          if (key < seq.k_lo || key >= seq.k_hi)
            asm volatile("st.shared.v4.b32 [%0], {%1, %1, %1, %1};" ::"r"(vt + blk * kTokBlock + r * 128 + (c & 7) * 16), "r"(0)
                         : "memory");
        }
        fence_async_smem();
        __syncwarp();
      }
      float sc[2][4] = {};
#pragma unroll
      for (int k = 0; k < kKb * 4; ++k)
        if (k < A.k_steps) {
          uint32_t f[4];
          ldsm4(tok_at(kt, key0 + (lane >> 4) * 8 + (lane & 7), k * 16 + ((lane >> 3) & 1) * 8), f);
          mma16816(sc[0], qa[k], f[0], f[1]);
          mma16816(sc[1], qa[k], f[2], f[3]);
        }
      uint32_t pa[4];
      float alpha[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float x[4], mx = -INFINITY;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int key = at + (e >> 1) * 8 + c0 + (e & 1);
          x[e] = key >= keys[h].lo && key < keys[h].hi ? sc[e >> 1][2 * h + (e & 1)] * A.scale2 : -INFINITY;
          mx = fmaxf(mx, x[e]);
        }
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
        mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
        const float mn = fmaxf(m[h], mx), base = mn == -INFINITY ? 0.f : mn;
        alpha[h] = m[h] == mn ? 1.f : ex2(m[h] - base);
        m[h] = mn;
        float sum = 0.f;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          x[e] = ex2(x[e] - base);
          sum += x[e];
        }
        l[h] = l[h] * alpha[h] + sum;
        pa[h] = pack_bf16(x[0], x[1]);
        pa[2 + h] = pack_bf16(x[2], x[3]);
      }
      if (__any_sync(0xffffffffu, alpha[0] != 1.f || alpha[1] != 1.f)) {
#pragma unroll
        for (int n = 0; n < kVb * 8; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) o[n][e] *= alpha[e >> 1];
      }
#pragma unroll
      for (int n = 0; n < kVb * 4; ++n)
        if (n * 16 < A.dv) {
          uint32_t f[4];
          ldsm4_trans(tok_at(vt, key0 + ((lane >> 3) & 1) * 8 + (lane & 7), n * 16 + (lane >> 4) * 8), f);
          mma16816(o[2 * n], pa, f[0], f[1]);
          mma16816(o[2 * n + 1], pa, f[2], f[3]);
        }
      __syncwarp();
      if (lane == 0) mbar_arrive(empty0 + 8 * s);
      if (++s == C::kStages) s = 0, phase ^= 1;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {  // a row's sum over its four lanes
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 1);
      l[h] += __shfl_xor_sync(0xffffffffu, l[h], 2);
    }
  }
  __syncthreads();  // every stage has been read
  if (guard.aborted()) {
    if (threadIdx.x == kTokWarps * 32) started.settle_ring(guard, 1, full0, C::kStages);
    return;
  }
  float *const jo = reinterpret_cast<float *>(smem), *const js = jo + kTokWarps * 16 * kVb * 64;
  if (warp < kTokWarps) {
#pragma unroll
    for (int n = 0; n < kVb * 8; ++n)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<float2 *>(jo + (warp * 16 + (lane >> 2) + 8 * h) * (kVb * 64) + n * 8 + (lane & 3) * 2) =
            make_float2(o[n][2 * h], o[n][2 * h + 1]);
    if ((lane & 3) == 0)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        js[(warp * 16 + (lane >> 2) + 8 * h) * 2] = m[h];
        js[(warp * 16 + (lane >> 2) + 8 * h) * 2 + 1] = l[h];
      }
  }
  __syncthreads();
  // pairs of output columns, over the CTA's threads
  const int pairs = A.dv / 2;
  for (int i = threadIdx.x; i < rows * pairs; i += kTokThreads) {
    const int r = i / pairs, c = (i - r * pairs) * 2, t = r / P.group, head = kh * P.group + r % P.group;
    float top = -INFINITY;
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) top = fmaxf(top, js[(w * 16 + r) * 2]);
    const float base = top == -INFINITY ? 0.f : top;
    float sum = 0.f;
    float2 v = make_float2(0.f, 0.f);
#pragma unroll
    for (int w = 0; w < kTokWarps; ++w) {
      const float e = ex2(js[(w * 16 + r) * 2] - base);
      sum = fmaf(js[(w * 16 + r) * 2 + 1], e, sum);
      const float2 x = *reinterpret_cast<const float2 *>(jo + (w * 16 + r) * (kVb * 64) + c);
      v.x = fmaf(x.x, e, v.x), v.y = fmaf(x.y, e, v.y);
    }
    const float inv = sum != 0.f ? 1.f / sum : 0.f;
    v.x *= inv, v.y *= inv;
    const int64_t row = ((int64_t)b * P.mask.sq + t) * A.q_heads + head;
    if (P.splits == 1) {
      *reinterpret_cast<uint32_t *>(P.y + (b * P.ys[0] + t * P.ys[1] + head * P.ys[2] + c)) = pack_bf16(v.x, v.y);
      if (c == 0 && P.lse) P.lse[row] = sum != 0.f ? base * kLn2 + logf(sum) : -INFINITY;
    } else {
      *reinterpret_cast<float2 *>(P.part_o + (split * P.rows + row) * A.dv + c) = v;
      if (c == 0) P.part_lse[split * P.rows + row] = sum != 0.f ? base + log2f(sum) : -INFINITY;
    }
  }
}

// ---------------------------------------------------------------------------
// parts of a row: y = sum_s 2^(lse_s - lse) y_s, fp32 parts, each read once.  A warp to a
// row; where there are more than eight parts (a few rows over a long cache), four warps,
// each every fourth group of four parts, which wait for memory a quarter as often in a
// row (one token over 8192 keys, 64 parts: 13.7 us in all -> 9.7; over 65536 33.1 ->
// 29.1; 64 tokens over 16384 32.3 -> 25.9).

struct JoinRows {
  const float *part_o, *part_lse;
  float *lse;
  __nv_bfloat16 *y;
  int64_t ys[3], rows;
  int32_t sq, heads, dv, splits;
};

constexpr int kMaxSplits = 64;

template <int kWarps>
__global__ void __launch_bounds__(128) attn_join_kernel(const __grid_constant__ JoinRows P) {
  pdl_launch();
  __shared__ float4 others[kWarps > 1 ? kWarps - 1 : 1][32];
  pdl_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, share = kWarps > 1 ? warp : 0;
  const int64_t row = kWarps > 1 ? (int64_t)blockIdx.x : (int64_t)blockIdx.x * 4 + warp;
  if (row >= P.rows) return;
  float w[kMaxSplits / 32], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int i = 0; i < kMaxSplits / 32; ++i) {
    const int s = lane + 32 * i;
    w[i] = s < P.splits ? P.part_lse[s * P.rows + row] : -INFINITY;
    top = fmaxf(top, w[i]);
  }
  top = warp_max(top);
  const float base = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int i = 0; i < kMaxSplits / 32; ++i) {
    w[i] = ex2(w[i] - base);
    sum += w[i];
  }
  sum = warp_sum(sum);
  const float inv = sum != 0.f ? 1.f / sum : 0.f;
  const bool in = lane * 4 < P.dv;
  float4 y = make_float4(0.f, 0.f, 0.f, 0.f);
  for (int s0 = 4 * share; s0 < P.splits; s0 += 4 * kWarps) {
    float4 x[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
      if (in && s0 + u < P.splits)
        x[u] = *reinterpret_cast<const float4 *>(P.part_o + ((s0 + u) * P.rows + row) * P.dv + lane * 4);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int s = s0 + u;
      const float e = __shfl_sync(0xffffffffu, s < 32 ? w[0] : w[1], s & 31) * inv;
      // (a part that saw nothing holds zeros)
      if (in && s < P.splits) y.x = fmaf(e, x[u].x, y.x), y.y = fmaf(e, x[u].y, y.y), y.z = fmaf(e, x[u].z, y.z), y.w = fmaf(e, x[u].w, y.w);
    }
  }
  if constexpr (kWarps > 1) {
    if (warp > 0) others[warp - 1][lane] = y;
    __syncthreads();
    if (warp > 0) return;
#pragma unroll
    for (int w = 0; w < kWarps - 1; ++w) {
      const float4 o = others[w][lane];
      y.x += o.x, y.y += o.y, y.z += o.z, y.w += o.w;
    }
  }
  const int64_t bt = row / P.heads;
  const int head = (int)(row - bt * P.heads);
  const int64_t b = bt / P.sq, t = bt - b * P.sq;
  if (in)
    *reinterpret_cast<uint2 *>(P.y + (b * P.ys[0] + t * P.ys[1] + head * P.ys[2] + lane * 4)) =
        make_uint2(pack_bf16(y.x, y.y), pack_bf16(y.z, y.w));
  if (lane == 0 && P.lse) P.lse[row] = sum != 0.f ? (base + log2f(sum)) * kLn2 : -INFINITY;
}

// ---------------------------------------------------------------------------
// host

constexpr int kTokRows = 16;

// How a call is cut: over the row tiles (or key heads), and each one's keys
// over `splits` CTAs.
struct FwdPlan {
  bool token;
  int32_t token_blocks, splits;
  int64_t items, rows;
  size_t o_bytes, bytes;
};

FwdPlan plan_forward(const gbo_attn_args *a, const AttnShape &S, int sm) {
  FwdPlan p;
  const int group = a->q_heads / a->k_heads;
  p.rows = a->batch * a->sq * a->q_heads;
  p.token = a->sq * group <= kTokRows;
  int64_t tiles;  // of keys
  if (p.token) {
    p.token_blocks = 1;
    p.items = a->batch * a->k_heads;
    tiles = (a->sk + kTokKeys - 1) / kTokKeys;
  } else {
    const int64_t per = 2 * (kAttnTile >> S.pack);
    p.token_blocks = (int32_t)((a->sq + per - 1) / per);
    p.items = (int64_t)p.token_blocks * a->batch * a->k_heads * S.head_blocks;
    tiles = (a->sk + kAttnTile - 1) / kAttnTile;
  }
  int64_t seen = a->window > 0 ? std::min<int64_t>(tiles, a->window / (p.token ? kTokKeys : kAttnTile) + 2) : tiles;
  if (a->documents) seen = std::min<int64_t>(seen, tiles / a->n_documents + 1);
  // The split that ends first, in microseconds: a step of a CTA takes 1.4 (128 keys
  // for two row tiles; 64 keys of a cache, two CTAs an SM; both of heads of 128 elements,
  // and taken for narrower and wider ones too), its start and end as
  // much as `fixed` steps, and the parts are written and read once, 4 bytes an
  // element, with a launch of 5.  Without the parts' bytes in the account, 8192 tokens
  // of 13 documents were split in two: 183 us instead of 68.
  const int64_t at_once = (int64_t)sm * (p.token ? 2 : 1), fixed = p.token ? 6 : 4;
  double best = 0.0;
  p.splits = 1;
  for (int s = 1; s <= kMaxSplits && (s == 1 || s * 2 <= seen); ++s) {
    const int64_t rounds = (p.items * s + at_once - 1) / at_once;
    const double join = s > 1 ? 5.0 + (double)p.rows * s * a->dv * 8.0 / 6e6 : 0.0;
    const double cost = (double)rounds * (double)((seen + s - 1) / s + fixed) * 1.4 + join;
    if (s == 1 || cost < best) best = cost, p.splits = s;
  }
  p.o_bytes = p.splits > 1 ? ((size_t)p.splits * p.rows * a->dv * 4 + 255) / 256 * 256 : 0;
  p.bytes = p.splits > 1 ? p.o_bytes + (size_t)p.splits * p.rows * 4 : 0;
  return p;
}

template <int kKb, int kVb>
cudaError_t launch_forward(const FwdParams &P, int64_t grid, int dev, cudaStream_t st) {
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(attn_forward_kernel<kKb, kVb>, cudaFuncAttributeMaxDynamicSharedMemorySize, Fwd<kKb, kVb>::kSmem);
  });
  if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), attn_forward_kernel<kKb, kVb>, dim3((unsigned)grid), dim3(kFwdThreads),
                          Fwd<kKb, kVb>::kSmem, st, 1, P);
}

template <int kKb, int kVb>
cudaError_t launch_token(const TokParams &P, int64_t grid, int dev, cudaStream_t st) {
  static PerDevice<cudaError_t> limit;
  const cudaError_t *err = limit.of(dev, [](cudaError_t &e) {
    e = cudaFuncSetAttribute(attn_token_kernel<kKb, kVb>, cudaFuncAttributeMaxDynamicSharedMemorySize, Tok<kKb, kVb>::kSmem);
  });
  if (!err || *err != cudaSuccess) return err ? *err : cudaErrorInvalidDevice;
  count_launches(1);
  return launch_kernel_as(pdl_allowed(), attn_token_kernel<kKb, kVb>, dim3((unsigned)grid), dim3(kTokThreads),
                          Tok<kKb, kVb>::kSmem, st, 1, P);
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" size_t gbo_attn_forward_workspace_bytes(const gbo_attn_args *args) {
  int dev, sm = 0;
  if (check_attn_sizes(args) != GBO_OK || require_device(&dev, &sm) != GBO_OK) return 0;
  AttnShape S;
  AttnMask M;
  fill_shape(args, &S, &M, kAttnMaxPack);
  return plan_forward(args, S, sm).bytes;
}

extern "C" int gbo_attn_forward(const gbo_attn_args *a, void *y, const int64_t *y_stride, float *lse, void *workspace,
                                size_t ws_bytes, int32_t *dev_status, gbo_stream_t stream) {
  int rc = check_attn(a);
  if (rc != GBO_OK) return rc;
  if ((reinterpret_cast<uintptr_t>(lse) | reinterpret_cast<uintptr_t>(dev_status)) & 3)
    return attn_fail(GBO_ERR_INVALID_ARG, "misaligned lse or status pointer");
  const bool none = a->batch == 0 || a->sq == 0;
  if (!none) {
    if (!y_stride) return attn_fail(GBO_ERR_INVALID_ARG, "y_stride is NULL");
    if ((rc = check_heads(y, y_stride, a->batch, a->sq, a->q_heads)) != GBO_OK) return rc;
  }
  int dev, sm = 0;
  if ((rc = attn_device(&dev, &sm)) != GBO_OK) return rc;
  if (none) return report_ok();
  AttnShape S;
  AttnMask M;
  fill_shape(a, &S, &M, kAttnMaxPack);
  const FwdPlan p = plan_forward(a, S, sm);
  if (p.items * p.splits > INT32_MAX || p.rows > (int64_t)INT32_MAX * 4) return attn_fail(GBO_ERR_SHAPE, "more rows than one launch takes");
  if (p.bytes && (!workspace || ws_bytes < p.bytes))
    return attn_fail(GBO_ERR_WORKSPACE, "workspace missing or smaller than gbo_attn_forward_workspace_bytes");
  if (p.bytes && (reinterpret_cast<uintptr_t>(workspace) & 255))
    return attn_fail(GBO_ERR_WORKSPACE, "workspace must be 256-byte aligned");
  float *part_o = static_cast<float *>(workspace);
  float *part_lse = reinterpret_cast<float *>(static_cast<char *>(workspace) + p.o_bytes);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e;
  bool maps = true;
  if (p.token) {
    TokParams T;
    memset(&T, 0, sizeof T);
    T.mask = M, T.shape = S;
    T.q = static_cast<const __nv_bfloat16 *>(a->q), T.y = static_cast<__nv_bfloat16 *>(y);
    const int64_t extent[3] = {a->batch, a->sq, a->q_heads};
    for (int i = 0; i < 3; ++i) T.qs[i] = extent[i] > 1 ? a->q_stride[i] : 0, T.ys[i] = extent[i] > 1 ? y_stride[i] : 0;
    T.lse = lse, T.part_o = part_o, T.part_lse = part_lse, T.status = dev_status;
    T.rows = p.rows, T.splits = p.splits, T.group = a->q_heads / a->k_heads;
    if (a->sk > 0)
      maps = heads_map(&T.k, a->k, a->dk, a->k_heads, a->sk, a->batch, a->k_stride, 1, kTokKeys) &&
             heads_map(&T.v, a->v, a->dv, a->k_heads, a->sk, a->batch, a->v_stride, 1, kTokKeys);
    if (!maps) return attn_fail(GBO_ERR_CUDA, "tensor map of keys or values");
    const int64_t grid = p.items * p.splits;
    const int cfg = attn_config(a);
    e = cfg == 0 ? launch_token<1, 1>(T, grid, dev, st) : cfg == 1 ? launch_token<2, 2>(T, grid, dev, st) : launch_token<3, 2>(T, grid, dev, st);
  } else {
    FwdParams F;
    memset(&F, 0, sizeof F);
    F.mask = M, F.shape = S;
    F.lse = lse, F.part_o = part_o, F.part_lse = part_lse, F.status = dev_status;
    F.rows = p.rows, F.token_blocks = p.token_blocks, F.splits = p.splits, F.by_splits = fast_div(p.splits);
    const uint32_t heads = 1u << S.pack;
    maps = heads_map(&F.q, a->q, a->dk, a->q_heads, a->sq, a->batch, a->q_stride, heads, kAttnTile >> S.pack) &&
           heads_map(&F.y, y, a->dv, a->q_heads, a->sq, a->batch, y_stride, heads, 32 >> S.pack);
    if (a->sk > 0)
      maps = maps && heads_map(&F.k, a->k, a->dk, a->k_heads, a->sk, a->batch, a->k_stride, 1, kAttnTile) &&
             heads_map(&F.v, a->v, a->dv, a->k_heads, a->sk, a->batch, a->v_stride, 1, kAttnTile);
    if (!maps) return attn_fail(GBO_ERR_CUDA, "tensor map of queries, keys, values or outputs");
    const int64_t grid = p.items * p.splits;
    const int cfg = attn_config(a);
    e = cfg == 0 ? launch_forward<1, 1>(F, grid, dev, st) : cfg == 1 ? launch_forward<2, 2>(F, grid, dev, st) : launch_forward<3, 2>(F, grid, dev, st);
  }
  if (e == cudaSuccess && p.splits > 1) {
    JoinRows J;
    memset(&J, 0, sizeof J);
    J.part_o = part_o, J.part_lse = part_lse, J.lse = lse, J.y = static_cast<__nv_bfloat16 *>(y);
    const int64_t extent[3] = {a->batch, a->sq, a->q_heads};
    for (int i = 0; i < 3; ++i) J.ys[i] = extent[i] > 1 ? y_stride[i] : 0;
    J.rows = p.rows, J.sq = (int32_t)a->sq, J.heads = a->q_heads, J.dv = a->dv, J.splits = p.splits;
    count_launches(1);
    const bool wide = p.splits > 8 && p.rows <= INT32_MAX;
    e = wide ? launch_kernel_as(pdl_allowed(), attn_join_kernel<4>, dim3((unsigned)p.rows), dim3(128), 0, st, 1, J)
             : launch_kernel_as(pdl_allowed(), attn_join_kernel<1>, dim3((unsigned)((p.rows + 3) / 4)), dim3(128), 0, st, 1, J);
  }
  return e == cudaSuccess ? report_ok() : attn_cuda(e);
}

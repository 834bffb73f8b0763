// Test hooks (gbo_testing.h): waits of the operators' kernels that run out, with a short
// limit, in kernels that are made of nothing but those waits.
#include "attn_common.cuh"
#include "residual.cuh"

namespace gbo {

namespace {

constexpr int kHookStages = 3, kHookThreads = 128, kHookRow = 1024;  // bytes of a row

// Rows through the residual kernels' ring.  The copy of row `lost` is asked for (its
// barrier expects the bytes) and never started, as one that does not land in time.
__global__ void __launch_bounds__(kHookThreads) ring_give_up_kernel(const uint8_t *rows, int n, int lost, int32_t *found,
                                                                    int32_t *status, uint64_t limit_ns) {
  __shared__ __align__(128) uint8_t place[kHookStages * kHookRow];
  __shared__ uint64_t bars[kHookStages];
  __shared__ int32_t late;
  const int tid = threadIdx.x;
  RowRing ring{smem_u32(place), smem_u32(bars), kHookRow, kHookStages, &late, status, limit_ns};
  if (tid == 0) {
    for (int s = 0; s < kHookStages; ++s) mbar_init(ring.full0 + 8 * s, 1);
    late = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  RowFeed<false> feed{};
  feed.src[kInX] = rows, feed.by[kInX] = kHookRow, feed.bytes[kInX] = kHookRow;
  feed.row = 0, feed.step = 1, feed.n = n;
  auto fill = [&] {
    if (feed.row != lost || ring.gave_up) return feed.fill(ring);
    mbar_expect_tx(ring.full0 + 8 * ring.to_fill, kHookRow);
    feed.src[kInX] += kHookRow;
    ++feed.row;
    if (++ring.to_fill == ring.stages) ring.to_fill = 0;
  };
  if (tid == 0)
    for (int s = 0; s < kHookStages; ++s) fill();
  for (int row = 0; row < n; ++row) {
    const uint32_t at = ring.take();
    __syncthreads();
    if (tid == 0) {
      if (row != 0) fill();
      int32_t first;
      asm volatile("ld.shared.s32 %0, [%1];" : "=r"(first) : "r"(at) : "memory");
      found[row] = ring.gave_up ? -1 : first;
    }
    ring.next();
  }
  if (tid != 0) return;
  const int filled = (int)feed.row;
  if (ring.gave_up) ring.settle(filled);
  int32_t landed = 0;
  for (int k = max(0, filled - kHookStages); k < filled; ++k)
    landed |= (int32_t)mbar_test(ring.full0 + 8 * (k % kHookStages), (k / kHookStages) & 1) << (k % kHookStages);
  found[n] = filled, found[n + 1] = landed;
}

// The attention kernels' waits.  Warp 0 loads tiles of 32 tokens into a ring of two
// stages that nobody empties, the second with rows to be zeroed, and waits for a place
// for the third; warp 1 waits by one thread, warp 2 by all of its lanes, for what never
// comes.  Warp `first` has the short limit, the others a hundred times as long.
constexpr int kHookTokens = 32, kHookTile = kHookTokens * 128;

__global__ void __launch_bounds__(96) attn_give_up_kernel(const __grid_constant__ CUtensorMap map, int first, int32_t *found,
                                                          int32_t *status, uint64_t limit_ns) {
  __shared__ __align__(1024) uint8_t place[2 * kHookTile];
  __shared__ uint64_t bars[6];  // full (two), empty (two), raw, never
  __shared__ int32_t flag[4];  // and what was started
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t full = smem_u32(bars), empty = full + 16, raw = full + 32, never = full + 40;
  if (threadIdx.x == 0) {
    for (int s = 0; s < 6; ++s) mbar_init(full + 8 * s, 1);
    flag[0] = 0;
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  }
  __syncthreads();
  const AttnGuard guard = {flag, status, warp == first ? limit_ns : 100 * limit_ns};
  const Started started = {flag + 1};
  const uint64_t t0 = global_ns();
  bool came = false;
  if (warp == 0) {
    TileRing ring(full, empty, smem_u32(place), kHookTile, 2);
    uint32_t raw_phase = 0;
    bool loaded[3] = {};
    for (int i = 0; i < 3; ++i) {
      loaded[i] = ring.load(guard, &map, 1, kHookTile, 0, i * kHookTokens, 0, i == 1, raw, raw_phase, kHookTokens, 8, 24, lane);
      if (!loaded[i]) break;
    }
    came = !loaded[0] || !loaded[1] || loaded[2];
    if (lane == 0) started.note(0, ring.loads, 0);
  } else if (warp == 1) {
    if (lane == 0) came = guard.wait(never, 0);
    __syncwarp();
  } else {
    came = guard.wait_warp(never, 0);
  }
  if (lane == 0) found[warp] = came, found[3 + warp] = (int32_t)((global_ns() - t0) / 1000);
  __syncthreads();
  if (threadIdx.x == 0 && guard.aborted()) {
    started.settle_ring(guard, 1, full, 2);
    found[6] = (int32_t)mbar_test(full, 0) | (int32_t)mbar_test(full + 8, 0) << 1;
    const int32_t *words = reinterpret_cast<const int32_t *>(place);  // rows of 32 words
    found[7] = words[0], found[8] = words[kHookTile / 4 + 8 * 32], found[9] = words[kHookTile / 4];
  }
}

}  // namespace
}  // namespace gbo

using namespace gbo;

extern "C" int gbo_testing_ring_give_up(const void *rows, int32_t n, int32_t lost, int32_t *found, int32_t *dev_status,
                                        uint32_t limit_us, gbo_stream_t stream) {
  if (!rows || (reinterpret_cast<uintptr_t>(rows) & 15) || !found || !dev_status ||
      ((reinterpret_cast<uintptr_t>(found) | reinterpret_cast<uintptr_t>(dev_status)) & 3))
    return report_error(GBO_ERR_INVALID_ARG, "NULL or misaligned pointer");
  if (n < 1 || n > 64 || lost < -1 || lost >= n) return report_error(GBO_ERR_INVALID_ARG, "n must be in 1..64, lost in -1..n-1");
  if (limit_us == 0 || limit_us > 1000000u) return report_error(GBO_ERR_INVALID_ARG, "limit_us must be in 1..10^6");
  int dev, sm = 0;
  const int rc = require_device(&dev, &sm);
  if (rc != GBO_OK) return rc;
  count_launches(1);
  ring_give_up_kernel<<<1, kHookThreads, 0, reinterpret_cast<cudaStream_t>(stream)>>>(
      static_cast<const uint8_t *>(rows), n, lost, found, dev_status, (uint64_t)limit_us * 1000u);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? report_ok() : res_cuda(e);
}

extern "C" int gbo_testing_attn_give_up(const void *tokens, int32_t first, int32_t *found, int32_t *dev_status,
                                        uint32_t limit_us, gbo_stream_t stream) {
  if (!tokens || (reinterpret_cast<uintptr_t>(tokens) & 15) || !found || !dev_status ||
      ((reinterpret_cast<uintptr_t>(found) | reinterpret_cast<uintptr_t>(dev_status)) & 3))
    return report_error(GBO_ERR_INVALID_ARG, "NULL or misaligned pointer");
  if (first < 0 || first > 2) return report_error(GBO_ERR_INVALID_ARG, "first must be in 0..2");
  if (limit_us == 0 || limit_us > 50000u) return report_error(GBO_ERR_INVALID_ARG, "limit_us must be in 1..50000");
  int dev, sm = 0;
  const int rc = attn_device(&dev, &sm);
  if (rc != GBO_OK) return rc;
  CUtensorMap map;
  const int64_t strides[3] = {64 * 2 * kHookTokens, 64, 64};
  if (!heads_map(&map, tokens, 64, 1, 2 * kHookTokens, 1, strides, 1, kHookTokens))
    return report_error(GBO_ERR_CUDA, "tensor map of the tokens");
  count_launches(1);
  attn_give_up_kernel<<<1, 96, 0, reinterpret_cast<cudaStream_t>(stream)>>>(map, first, found, dev_status,
                                                                            (uint64_t)limit_us * 1000u);
  const cudaError_t e = cudaGetLastError();
  return e == cudaSuccess ? report_ok() : attn_cuda(e);
}

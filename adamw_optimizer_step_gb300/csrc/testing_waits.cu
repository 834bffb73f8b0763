// Test hooks (gbo_testing.h): waits of the operators' kernels that run out, with a short
// limit, in kernels that are made of nothing but those waits.
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

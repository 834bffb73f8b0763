// Dropout's bits: Philox 4x32-10, the counter generator of Salmon, Moraes, Dror
// and Shaw, "Parallel random numbers: as easy as 1, 2, 3" (2011).  Eight
// consecutive elements share one counter: a 16-bit draw each, so a probability
// is a multiple of 2^-16, and an element costs an eighth of ten rounds.  With
// 32 bits an element the rounds alone, some 20 instructions an element, would
// take longer than HBM takes to move bf16 elements in and out.
#pragma once

#include <cmath>
#include <cstdint>

namespace gbo {

struct DropArgs {
  uint64_t seed, offset;
  const int64_t *dev_seed;  // or NULL: seed
  uint32_t limit;           // draws below it drop the element; 0: nothing is dropped
  float keep;               // what the kept elements are multiplied by
};

// The draws of elements 8 i .. 8 i + 7: draw e is half (e & 1), low first, of word e / 2.
__device__ __forceinline__ uint4 philox(uint64_t key, uint64_t i, uint64_t offset) {
  uint32_t a = (uint32_t)i, b = (uint32_t)(i >> 32), c = (uint32_t)offset, d = (uint32_t)(offset >> 32);
  uint32_t k0 = (uint32_t)key, k1 = (uint32_t)(key >> 32);
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t u = (uint64_t)0xD2511F53u * a, v = (uint64_t)0xCD9E8D57u * c;
    a = (uint32_t)(v >> 32) ^ b ^ k0;
    b = (uint32_t)v;
    c = (uint32_t)(u >> 32) ^ d ^ k1;
    d = (uint32_t)u;
    k0 += 0x9E3779B9u, k1 += 0xBB67AE85u;
  }
  return make_uint4(a, b, c, d);
}

// Factor of element e (0..7) of those draws: 0 or keep.
__device__ __forceinline__ float drop_factor(const uint4 &w, int e, uint32_t limit, float keep) {
  const uint32_t x = e < 2 ? w.x : e < 4 ? w.y : e < 6 ? w.z : w.w;
  return ((e & 1) ? x : x << 16) >= limit << 16 ? keep : 0.f;  // (compared in the upper half)
}

// limit and keep of a probability: nearest multiple of 2^-16, ties to even.
// False for one outside 0 <= p < 1 (or that would round to 1).
inline bool drop_of(double p, DropArgs *D) {
  if (!(p >= 0.0 && p < 1.0)) return false;
  const double limit = std::nearbyint(p * 65536.0);
  if (limit > 65535.0) return false;
  D->limit = (uint32_t)limit;
  D->keep = (float)(65536.0 / (65536.0 - limit));
  return true;
}

}  // namespace gbo

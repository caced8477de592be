// What the kernels of the attention over a paged cache share.
#pragma once
#include <cuda_runtime.h>

#include "attention.h"
#include "decay.cuh"
#include "ptx.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
// A base moves when a score exceeds the one that it was set by, the largest then, by more than kRoom powers of two.  Bases of f16 weights
// are set kBias below that score, so that weights down to 2^-20 of the largest stay in f16's normal range: a weight is
// 2^8 at most in bf16 and 2^14 in f16, whose numbers end below 2^16.
constexpr float kRoom = 8.f;
template <bool F16> constexpr float kBias = F16 ? 6.f : 0.f;
static_assert(kRoom + kBias<true> < 15.f, "weights stay finite in f16");

__device__ __forceinline__ float exp2_fast(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// 1 / x for sums of weights, to an ulp or so.
__device__ __forceinline__ float inverse(float x) {
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// `total` tiles in equal shares, the first ones a tile larger where that does not come out even.
struct Shares {
  uint32_t each, larger;
  __device__ __forceinline__ Shares(uint32_t total, uint32_t shares) : each(total / shares), larger(total - total / shares * shares) {}
  __device__ __forceinline__ uint32_t from(uint32_t share) const { return share * each + min(share, larger); }
};

// Keys of sequence n in its own pages, or -1 where its length is none.
__device__ __forceinline__ int length_of(const AttentionParams& p, int n) {
  const int64_t x = index_at(p.lengths, p.len_dtype, n);
  return x < 0 || x > (int64_t)p.max_pages * p.page_size ? -1 : (int)x;
}

}  // namespace gdn

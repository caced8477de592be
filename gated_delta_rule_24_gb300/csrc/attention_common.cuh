// What the kernels of the attention over a paged cache share.
#pragma once
#include <cuda_runtime.h>

#include "attention.h"
#include "decay.cuh"
#include "ptx.cuh"

namespace gdn {

constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;
constexpr float kRoom = 8.f;  // how far (powers of two) scores may exceed the base before it moves

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

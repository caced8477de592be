// Softmax attention of new tokens over a paged cache and a prefix that all sequences share, for sm_103a.
//
//   s_j = scale q . k_j,   out = sum_j exp(s_j) v_j / sum_j exp(s_j),   lse = log sum_j exp(s_j)
//
// One CTA for each (token, query head): its warps take every fourth key, with a running maximum and
// sum each, and join at the end.
#include <cuda_runtime.h>

#include "attention.h"
#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kWarps = 4;

template <bool F16>
__global__ void __launch_bounds__(32 * kWarps) gdn_attention_kernel(const __grid_constant__ AttentionParams p) {
  __shared__ float s_m[kWarps], s_l[kWarps];
  __shared__ float s_o[kWarps][kHeadDim];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int row = (int)(blockIdx.x / (unsigned)p.H_q), h = (int)(blockIdx.x % (unsigned)p.H_q);
  const int n = row / p.tokens, hk = h / (p.H_q / p.H_k);
  const int64_t length = index_at(p.lengths, p.len_dtype, n);
  const bool fits = length >= 0 && length <= (int64_t)p.max_pages * p.page_size;
  if (!fits && threadIdx.x == 0) atomicOr(p.dev_err, kDevErrLength);
  const int own = fits ? (int)length : 0;
  int bad = 0;  // pages of the sequence and of the prefix
  for (int i = threadIdx.x; i < (own + p.page_size - 1) / p.page_size; i += 32 * kWarps) {
    const int64_t page = index_at(p.table, p.table_dtype, n * p.table_st + i);
    bad |= page < 0 || page >= p.pages;
  }
  for (int i = threadIdx.x; i < (p.prefix + p.page_size - 1) / p.page_size; i += 32 * kWarps) {
    const int64_t page = index_at(p.prefix_pages, p.prefix_dtype, i);
    bad |= page < 0 || page >= p.pages;
  }
  if (__syncthreads_or(bad)) {
    if (threadIdx.x == 0) atomicOr(p.dev_err, kDevErrPage);
    return;
  }
  if (!fits) return;
  const uint2 qc = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.q) + row * p.q_st + h * p.q_sh + 4 * lane);
  const float2 q0 = unpack16<F16>(qc.x), q1 = unpack16<F16>(qc.y);
  const int seen = max(0, own - p.tokens + row % p.tokens + 1), keys = p.prefix + seen;
  float m = -INFINITY, l = 0.f, o[4] = {0.f, 0.f, 0.f, 0.f};
  for (int j = warp; j < keys; j += kWarps) {
    const bool shared = j < p.prefix;
    const int at = shared ? j : j - p.prefix, page_at = at / p.page_size, in = at % p.page_size;
    const int64_t page = shared ? index_at(p.prefix_pages, p.prefix_dtype, page_at) : index_at(p.table, p.table_dtype, n * p.table_st + page_at);
    const uint2 kc = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.k) + page * p.k_sp + in * p.k_st + hk * p.k_sh + 4 * lane);
    const uint2 vc = *reinterpret_cast<const uint2*>(reinterpret_cast<const uint16_t*>(p.v) + page * p.v_sp + in * p.v_st + hk * p.v_sh + 4 * lane);
    const float2 k0 = unpack16<F16>(kc.x), k1 = unpack16<F16>(kc.y), v0 = unpack16<F16>(vc.x), v1 = unpack16<F16>(vc.y);
    float s = q0.x * k0.x + q0.y * k0.y + q1.x * k1.x + q1.y * k1.y;
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) s += __shfl_xor_sync(0xffffffffu, s, d);
    s *= p.scale;
    const float top = fmaxf(m, s), base = top == -INFINITY ? 0.f : top;
    const float keep = expf(m - base), w = expf(s - base);
    m = top;
    l = l * keep + w;
    o[0] = o[0] * keep + w * v0.x;
    o[1] = o[1] * keep + w * v0.y;
    o[2] = o[2] * keep + w * v1.x;
    o[3] = o[3] * keep + w * v1.y;
  }
  if (lane == 0) { s_m[warp] = m; s_l[warp] = l; }
#pragma unroll
  for (int e = 0; e < 4; ++e) s_o[warp][4 * lane + e] = o[e];
  __syncthreads();
  float top = -INFINITY, total = 0.f, sum = 0.f;
  for (int w = 0; w < kWarps; ++w) top = fmaxf(top, s_m[w]);
  const float base = top == -INFINITY ? 0.f : top;
  for (int w = 0; w < kWarps; ++w) {
    const float c = expf(s_m[w] - base);
    total += c * s_l[w];
    sum += c * s_o[w][threadIdx.x];
  }
  reinterpret_cast<uint16_t*>(p.out)[row * p.o_st + h * p.o_sh + threadIdx.x] = (uint16_t)pack16x2<F16>(keys ? sum / total : 0.f, 0.f);
  if (p.lse && threadIdx.x == 0) p.lse[row * p.lse_st + h] = keys ? base + logf(total) : -INFINITY;
}

}  // namespace

cudaError_t launch_attention(const AttentionParams& p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.N * p.tokens * p.H_q;
  if (rows <= 0) return cudaSuccess;
  if (p.op_f16) gdn_attention_kernel<true><<<(unsigned)rows, 32 * kWarps, 0, stream>>>(p);
  else gdn_attention_kernel<false><<<(unsigned)rows, 32 * kWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn

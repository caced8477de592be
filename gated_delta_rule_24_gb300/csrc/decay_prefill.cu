// Linear attention with a decay over packed sequences, sm_103a: for each sequence and head,
// with the state S (V-major 128 x 128: row = value index, column = key index),
//
//   S_t = g_t S_{t-1} + v_t k_t^T,   o_t = scale S_t q_t.
//
// The token recurrence itself: a CTA of 256 threads holds one state in registers, two
// threads a row with 64 columns each, and takes the tokens one after another from tiles of
// 16 staged in shared memory.
#include <cuda_runtime.h>

#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kThreads = 256;
constexpr int kTile = 16;  // tokens staged at once

template <bool F16>
__global__ void __launch_bounds__(kThreads) gdn_decay_prefill_kernel(const __grid_constant__ DecayPrefillParams p) {
  __shared__ __align__(16) float sk[kTile][kHeadDim], sq[kTile][kHeadDim], sv[kTile][kHeadDim];
  __shared__ float sg[kTile];
  const int t = threadIdx.x, row = t >> 1, half = t & 1;
  const int n = blockIdx.x / p.H, h = blockIdx.x % p.H;
  const int64_t bos = index_at(p.cu, p.cu_dtype, n), eos = index_at(p.cu, p.cu_dtype, n + 1);
  const int64_t slot = p.state_idx ? index_at(p.state_idx, p.idx_dtype, n) : (int64_t)n;
  int err = 0;
  if (bos < 0 || eos < bos || eos > p.T) err |= kDevErrCu;
  if ((p.s_in && (slot < 0 || slot >= p.sin_slots)) || (p.s_out && (slot < 0 || slot >= p.sout_slots))) err |= kDevErrIdx;
  if (err) {
    if (t == 0) atomicOr(p.dev_err, err);
    return;
  }
  const int hq = h / (p.H / p.H_qk), hv = h / (p.H / p.H_v);
  float s[64];
#pragma unroll
  for (int e = 0; e < 64; ++e) {
    const int c = 4 * (2 * (e >> 2) + half) + (e & 3);  // 16-byte column groups alternate between the two threads
    s[e] = p.s_in ? real_of(p.s_in, p.sin_dtype, slot * p.sin_slot + (int64_t)h * p.sin_head + row * kHeadDim + c) : 0.f;
  }
  for (int64_t t0 = bos; t0 < eos; t0 += kTile) {
    const int len = (int)(eos - t0 < kTile ? eos - t0 : kTile);
    for (int e = t; e < len * (kHeadDim / 2); e += kThreads) {
      const int i = e / (kHeadDim / 2), c = 2 * (e % (kHeadDim / 2));
      const int64_t tok = t0 + i;
      auto pair = [&](const void* x, int64_t off) {
        return unpack16<F16>(*reinterpret_cast<const uint32_t*>(reinterpret_cast<const uint16_t*>(x) + off));
      };
      *reinterpret_cast<float2*>(&sk[i][c]) = pair(p.k, tok * p.k_st + (int64_t)hq * p.k_sh + c);
      *reinterpret_cast<float2*>(&sq[i][c]) = pair(p.q, tok * p.q_st + (int64_t)hq * p.q_sh + c);
      *reinterpret_cast<float2*>(&sv[i][c]) = pair(p.v, tok * p.v_st + (int64_t)hv * p.v_sh + c);
    }
    if (t < len) sg[t] = p.g ? gate_at(p.g, p.g_dtype, (t0 + t) * p.g_st + (int64_t)h * p.g_sh) : 1.f;
    __syncthreads();
    for (int i = 0; i < len; ++i) {
      const float g = sg[i], v = sv[i][row];
      float acc = 0.f;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        const float4 k = *reinterpret_cast<const float4*>(&sk[i][4 * (2 * j + half)]);
        const float4 q = *reinterpret_cast<const float4*>(&sq[i][4 * (2 * j + half)]);
        s[4 * j] = fmaf(g, s[4 * j], v * k.x);
        s[4 * j + 1] = fmaf(g, s[4 * j + 1], v * k.y);
        s[4 * j + 2] = fmaf(g, s[4 * j + 2], v * k.z);
        s[4 * j + 3] = fmaf(g, s[4 * j + 3], v * k.w);
        acc = fmaf(s[4 * j], q.x, acc);
        acc = fmaf(s[4 * j + 1], q.y, acc);
        acc = fmaf(s[4 * j + 2], q.z, acc);
        acc = fmaf(s[4 * j + 3], q.w, acc);
      }
      acc += __shfl_xor_sync(0xffffffffu, acc, 1);
      if (half == 0)
        reinterpret_cast<uint16_t*>(p.out)[(t0 + i) * p.o_st + (int64_t)h * p.o_sh + row] =
            (uint16_t)pack16x2<F16>(p.scale * acc, 0.f);
    }
    __syncthreads();
  }
  if (!p.s_out) return;
#pragma unroll
  for (int e = 0; e < 64; ++e) {
    const int c = 4 * (2 * (e >> 2) + half) + (e & 3);
    const int64_t i = slot * p.sout_slot + (int64_t)h * p.sout_head + row * kHeadDim + c;
    if (p.sout_dtype == kF32) reinterpret_cast<float*>(p.s_out)[i] = s[e];
    else if (p.sout_dtype == kF16) reinterpret_cast<__half*>(p.s_out)[i] = __float2half_rn(s[e]);
    else reinterpret_cast<__nv_bfloat16*>(p.s_out)[i] = __float2bfloat16_rn(s[e]);
  }
}

}  // namespace

cudaError_t launch_decay_prefill(const DecayPrefillParams& p, cudaStream_t stream) {
  const int64_t units = (int64_t)p.N * p.H;
  if (units <= 0) return cudaSuccess;
  if (p.op_f16) gdn_decay_prefill_kernel<true><<<(unsigned)units, kThreads, 0, stream>>>(p);
  else gdn_decay_prefill_kernel<false><<<(unsigned)units, kThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn

// RMS norm of every query and key head (128 values) and the rotation of its first R values
// by the token's position, in one pass for sm_103a:
//
//   y = x / sqrt(mean(x^2) + eps) * (w + offset),
//   (y_a, y_b) -> (y_a cos - y_b sin, y_a sin + y_b cos)   for the R / 2 pairs (a, b).
//
// Each value is read and written once and costs about seven flops: the pass is bound by
// HBM bandwidth.  Eight lanes hold a head, two vectors of 8 values each, chosen so that a
// lane owns both values of each of its pairs: neighbours (2i, 2i + 1) sit in one vector
// already, and for the halves (i, i + R / 2) lane l < R / 16 takes vectors l and l + R / 16.
// Either way a rotating lane needs the cosines and sines of pairs 8 l .. 8 l + 7.
#include <cuda_runtime.h>

#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 128;
constexpr int kRopeLanes = 8;  // lanes of one head

template <bool F16>
__global__ void __launch_bounds__(kRopeThreads) gdn_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  const int l = threadIdx.x % kRopeLanes;
  const int heads = p.t[0].heads + p.t[1].heads;
  const int64_t row = (int64_t)blockIdx.x * (kRopeThreads / kRopeLanes) + threadIdx.x / kRopeLanes;
  const int64_t tok = row / heads;
  const bool live = tok < p.T;
  const int hd = live ? (int)(row - tok * heads) : 0;
  const bool is_k = hd >= p.t[0].heads;
  const RopeTensor& t = p.t[is_k ? 1 : 0];
  const int h = is_k ? hd - p.t[0].heads : hd;
  const int rot = p.cos_sin ? p.rotary / 16 : 0;  // lanes that rotate
  const bool pairs = !p.interleaved && l < rot;
  const int v0 = pairs ? l : 2 * l, v1 = pairs ? l + rot : 2 * l + 1;
  int64_t place = 0;
  bool ok = live;
  if (ok && p.cos_sin) {
    place = p.positions ? index_at(p.positions, p.pos_dtype, tok) : tok;
    if (place < 0 || place >= p.places) {
      if (l == 0) atomicOr(p.dev_err, kDevErrPosition);
      ok = false;
    }
  }
  float a[8] = {}, b[8] = {};
  if (ok) {
    const uint16_t* x = reinterpret_cast<const uint16_t*>(t.x) + tok * t.x_st + (int64_t)h * t.x_sh;
    unpack16x8<F16>(*reinterpret_cast<const uint4*>(x + 8 * v0), a);
    unpack16x8<F16>(*reinterpret_cast<const uint4*>(x + 8 * v1), b);
  }
  float ss = 0.f;
#pragma unroll
  for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
  for (int d = kRopeLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
  if (!ok) return;
  const float r = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    a[e] *= r * (t.w ? real_of(t.w, t.w_dtype, 8 * v0 + e) + p.weight_offset : 1.f);
    b[e] *= r * (t.w ? real_of(t.w, t.w_dtype, 8 * v1 + e) + p.weight_offset : 1.f);
  }
  if (l < rot) {
    const float* cs = p.cos_sin + place * p.cs_stride + 8 * l;
    float c[8], s[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = cs[e]; s[e] = cs[p.rotary / 2 + e]; }
    if (p.interleaved) {
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float x0 = a[2 * e], x1 = a[2 * e + 1], y0 = b[2 * e], y1 = b[2 * e + 1];
        a[2 * e] = x0 * c[e] - x1 * s[e];
        a[2 * e + 1] = x0 * s[e] + x1 * c[e];
        b[2 * e] = y0 * c[4 + e] - y1 * s[4 + e];
        b[2 * e + 1] = y0 * s[4 + e] + y1 * c[4 + e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x0 = a[e], x1 = b[e];
        a[e] = x0 * c[e] - x1 * s[e];
        b[e] = x0 * s[e] + x1 * c[e];
      }
    }
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(t.y) + tok * t.y_st + (int64_t)h * t.y_sh;
  *reinterpret_cast<uint4*>(y + 8 * v0) = pack16x8<F16>(a);
  *reinterpret_cast<uint4*>(y + 8 * v1) = pack16x8<F16>(b);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t stream) {
  const int64_t rows = p.T * (p.t[0].heads + p.t[1].heads), per = kRopeThreads / kRopeLanes;
  if (rows <= 0) return cudaSuccess;
  const unsigned grid = (unsigned)((rows + per - 1) / per);
  if (p.in_f16) gdn_norm_rope_kernel<true><<<grid, kRopeThreads, 0, stream>>>(p);
  else gdn_norm_rope_kernel<false><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace gdn

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
// Norm and rotation are then y = r (x P + x' Q) with r the head's norm factor, x' the other
// value of the pair and P, Q made of the weights, cosines and sines once for a token (P the
// weight and Q zero where nothing turns).  A group of eight lanes walks some heads of one
// token with the loads of the next four under way.
#include <cuda_runtime.h>

#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 64;
constexpr int kRopeLanes = 8;                              // lanes of one head
constexpr int kRopeGroups = kRopeThreads / kRopeLanes;     // of a CTA

__device__ __forceinline__ void load8(const float* p, float (&x)[8]) {
  const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
  x[0] = a.x; x[1] = a.y; x[2] = a.z; x[3] = a.w; x[4] = b.x; x[5] = b.y; x[6] = b.z; x[7] = b.w;
}
// Eight weights plus the offset (1 without weights).
__device__ __forceinline__ void load_weight8(const RopeTensor& t, int at, float offset, float (&w)[8]) {
  if (!t.w) {
#pragma unroll
    for (int e = 0; e < 8; ++e) w[e] = 1.f;
    return;
  }
  if (t.w_dtype == kF32) {
    load8(reinterpret_cast<const float*>(t.w) + at, w);
  } else {
    const uint4 c = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(t.w) + at);
    if (t.w_dtype == kF16) unpack16x8<true>(c, w);
    else unpack16x8<false>(c, w);
  }
#pragma unroll
  for (int e = 0; e < 8; ++e) w[e] += offset;
}

// CTAs below q_ctas take q, the others k.  `per` heads a group; a token's groups side by side.
template <bool F16, bool kInterleaved, int kAhead>
__global__ void __launch_bounds__(kRopeThreads) gdn_norm_rope_kernel(const __grid_constant__ RopeParams p, unsigned q_ctas,
                                                                     int per) {
  const int l = threadIdx.x % kRopeLanes;
  const bool is_k = blockIdx.x >= q_ctas;
  const RopeTensor& t = p.t[is_k ? 1 : 0];
  const int parts = (t.heads + per - 1) / per;
  const int64_t first = (int64_t)(blockIdx.x - (is_k ? q_ctas : 0)) * kRopeGroups;
  int64_t tok = first / parts;
  int part = (int)(first - tok * parts) + threadIdx.x / kRopeLanes;
  tok += part / parts;
  part %= parts;
  const int rot = p.cos_sin ? p.rotary / 16 : 0;  // lanes that rotate
  const bool halves = !kInterleaved && l < rot;
  const int v0 = 8 * (halves ? l : 2 * l), v1 = 8 * (halves ? l + rot : 2 * l + 1);
  bool ok = tok < p.T;
  int64_t place = 0;
  if (ok && p.cos_sin) {
    place = p.positions ? index_at(p.positions, p.pos_dtype, tok) : tok;
    if (place < 0 || place >= p.places) {
      if (l == 0) atomicOr(p.dev_err, kDevErrPosition);
      ok = false;
    }
  }
  // `n` heads for every group of the warp, so that its lanes stay together; a group without a token or
  // with fewer heads left loads and stores nothing
  const int n = min(per, t.heads), own = ok ? min(per, t.heads - part * per) : 0;
  const int64_t sx = t.x_sh, sy = t.y_sh;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(t.x) + tok * t.x_st + (int64_t)part * per * sx;
  uint16_t* y = reinterpret_cast<uint16_t*>(t.y) + tok * t.y_st + (int64_t)part * per * sy;
  uint4 ra[kAhead], rb[kAhead];
  auto load = [&](int i, int h) {
    if (h < own) {
      ra[i] = __ldcs(reinterpret_cast<const uint4*>(x + h * sx + v0));
      rb[i] = __ldcs(reinterpret_cast<const uint4*>(x + h * sx + v1));
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    ra[i] = rb[i] = make_uint4(0, 0, 0, 0);
    load(i, i);
  }
  float2 pa[4], qa[4], pb[4], qb[4];  // P and Q of the two vectors
  {
    float wa[8], wb[8], c[8], s[8];
    load_weight8(t, v0, p.weight_offset, wa);
    load_weight8(t, v1, p.weight_offset, wb);
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
    if (ok && l < rot) {
      load8(p.cos_sin + place * p.cs_stride + 8 * l, c);
      load8(p.cos_sin + place * p.cs_stride + p.rotary / 2 + 8 * l, s);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (kInterleaved) {  // x' is the pair turned round
        pa[e] = make_float2(wa[2 * e] * c[e], wa[2 * e + 1] * c[e]);
        qa[e] = make_float2(-wa[2 * e + 1] * s[e], wa[2 * e] * s[e]);
        pb[e] = make_float2(wb[2 * e] * c[4 + e], wb[2 * e + 1] * c[4 + e]);
        qb[e] = make_float2(-wb[2 * e + 1] * s[4 + e], wb[2 * e] * s[4 + e]);
      } else {  // x' is the other vector's
        pa[e] = make_float2(wa[2 * e] * c[2 * e], wa[2 * e + 1] * c[2 * e + 1]);
        qa[e] = make_float2(-wb[2 * e] * s[2 * e], -wb[2 * e + 1] * s[2 * e + 1]);
        pb[e] = make_float2(wb[2 * e] * c[2 * e], wb[2 * e + 1] * c[2 * e + 1]);
        qb[e] = make_float2(wa[2 * e] * s[2 * e], wa[2 * e + 1] * s[2 * e + 1]);
      }
    }
  }
#pragma unroll 1
  for (int h0 = 0; h0 < n; h0 += kAhead) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) {
      const uint32_t ca[4] = {ra[i].x, ra[i].y, ra[i].z, ra[i].w}, cb[4] = {rb[i].x, rb[i].y, rb[i].z, rb[i].w};
      float2 a[4], b[4], sum = make_float2(0.f, 0.f);
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        a[e] = unpack16<F16>(ca[e]);
        b[e] = unpack16<F16>(cb[e]);
        sum = fma2(a[e], a[e], sum);
        sum = fma2(b[e], b[e], sum);
      }
      load(i, h0 + i + kAhead);
      float ss = sum.x + sum.y;
#pragma unroll
      for (int d = kRopeLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
      const float2 r = pair(rsqrtf(ss * (1.f / kHeadDim) + p.eps));
      uint32_t ya[4], yb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const float2 ta = kInterleaved ? make_float2(a[e].y, a[e].x) : b[e], tb = kInterleaved ? make_float2(b[e].y, b[e].x) : a[e];
        ya[e] = pack16x2<F16>(mul2(r, fma2(a[e], pa[e], mul2(ta, qa[e]))));
        yb[e] = pack16x2<F16>(mul2(r, fma2(b[e], pb[e], mul2(tb, qb[e]))));
      }
      if (h0 + i < own) {
        __stcs(reinterpret_cast<uint4*>(y + (h0 + i) * sy + v0), make_uint4(ya[0], ya[1], ya[2], ya[3]));
        __stcs(reinterpret_cast<uint4*>(y + (h0 + i) * sy + v1), make_uint4(yb[0], yb[1], yb[2], yb[3]));
      }
    }
  }
}

template <bool F16, int kAhead>
cudaError_t launch(const RopeParams& p, int per, cudaStream_t stream) {
  auto ctas = [&](int heads) { return (p.T * ((heads + per - 1) / per) + kRopeGroups - 1) / kRopeGroups; };
  const int64_t q = ctas(p.t[0].heads), k = ctas(p.t[1].heads);
  if (p.interleaved) gdn_norm_rope_kernel<F16, true, kAhead><<<(unsigned)(q + k), kRopeThreads, 0, stream>>>(p, (unsigned)q, per);
  else gdn_norm_rope_kernel<F16, false, kAhead><<<(unsigned)(q + k), kRopeThreads, 0, stream>>>(p, (unsigned)q, per);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t stream) {
  const int64_t rows = p.T * (p.t[0].heads + p.t[1].heads);
  if (rows <= 0) return cudaSuccess;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // Heads a group, up to 16, so that two rounds of groups are left on all SMs, and the loads of up to
  // four under way: 65536 tokens x 48 heads take 249 us with 16 heads a group, 290 with 4, 428 with 1
  // (6.6, 5.7 and 3.8 TB/s); 2000 tokens 14.6 us with 3 and two under way, 16.7 with 1, 27 with the
  // loop that has four.
  constexpr int kResident = 80, kRounds = 2;  // groups on an SM
  const int64_t most = rows / ((int64_t)sms * kResident * kRounds);
  const int per = (int)(most < 1 ? 1 : most > 16 ? 16 : most);
  if (per < 2) return p.in_f16 ? launch<true, 1>(p, 1, stream) : launch<false, 1>(p, 1, stream);
  if (per < 4) return p.in_f16 ? launch<true, 2>(p, per, stream) : launch<false, 2>(p, per, stream);
  return p.in_f16 ? launch<true, 4>(p, per, stream) : launch<false, 4>(p, per, stream);
}

}  // namespace gdn

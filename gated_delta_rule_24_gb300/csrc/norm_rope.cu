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
// Either way a rotating lane needs the cosines and sines of pairs 8 l .. 8 l + 7, the same
// for all heads of a token, and the weights of its 16 values, the same for all tokens: a
// group of lanes takes a run of heads of one token, with all their loads under way at once.
#include <cuda_runtime.h>

#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kRopeThreads = 128;
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

// kRun heads of one token and tensor for each group of eight lanes; a token's runs side by side.
template <bool F16, int kRun>
__global__ void __launch_bounds__(kRopeThreads) gdn_norm_rope_kernel(const __grid_constant__ RopeParams p) {
  const int l = threadIdx.x % kRopeLanes;
  const int q_runs = (p.t[0].heads + kRun - 1) / kRun, runs = q_runs + (p.t[1].heads + kRun - 1) / kRun;
  const int64_t first = (int64_t)blockIdx.x * kRopeGroups;  // of the CTA's (token, run) units
  int64_t tok = first / runs;
  int run = (int)(first - tok * runs) + threadIdx.x / kRopeLanes;
  if (run >= runs) {
    tok += run / runs;
    run %= runs;
  }
  const bool is_k = run >= q_runs;
  const RopeTensor& t = p.t[is_k ? 1 : 0];
  const int h0 = (is_k ? run - q_runs : run) * kRun;
  const int rot = p.cos_sin ? p.rotary / 16 : 0;  // lanes that rotate
  const bool halves = !p.interleaved && l < rot;
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
  uint4 ra[kRun], rb[kRun];
  const uint16_t* x = reinterpret_cast<const uint16_t*>(t.x) + tok * t.x_st + (int64_t)h0 * t.x_sh;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    ra[i] = rb[i] = make_uint4(0, 0, 0, 0);
    if (ok && h0 + i < t.heads) {
      ra[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * t.x_sh + v0));
      rb[i] = __ldcs(reinterpret_cast<const uint4*>(x + i * t.x_sh + v1));
    }
  }
  float wa[8], wb[8], c[8], s[8];
  load_weight8(t, v0, p.weight_offset, wa);
  load_weight8(t, v1, p.weight_offset, wb);
  const bool turn = ok && l < rot;
  if (turn) {
    load8(p.cos_sin + place * p.cs_stride + 8 * l, c);
    load8(p.cos_sin + place * p.cs_stride + p.rotary / 2 + 8 * l, s);
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(t.y) + tok * t.y_st + (int64_t)h0 * t.y_sh;
#pragma unroll
  for (int i = 0; i < kRun; ++i) {
    float a[8], b[8], ss = 0.f;
    unpack16x8<F16>(ra[i], a);
    unpack16x8<F16>(rb[i], b);
#pragma unroll
    for (int e = 0; e < 8; ++e) ss += a[e] * a[e] + b[e] * b[e];
#pragma unroll
    for (int d = kRopeLanes / 2; d > 0; d >>= 1) ss += __shfl_xor_sync(0xffffffffu, ss, d);
    const float r = rsqrtf(ss * (1.f / kHeadDim) + p.eps);
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      a[e] *= r * wa[e];
      b[e] *= r * wb[e];
    }
    if (turn) {
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
    if (ok && h0 + i < t.heads) {
      __stcs(reinterpret_cast<uint4*>(y + i * t.y_sh + v0), pack16x8<F16>(a));
      __stcs(reinterpret_cast<uint4*>(y + i * t.y_sh + v1), pack16x8<F16>(b));
    }
  }
}

template <int kRun>
cudaError_t launch(const RopeParams& p, cudaStream_t stream) {
  const int64_t units = p.T * ((p.t[0].heads + kRun - 1) / kRun + (p.t[1].heads + kRun - 1) / kRun);
  const unsigned grid = (unsigned)((units + kRopeGroups - 1) / kRopeGroups);
  if (p.in_f16) gdn_norm_rope_kernel<true, kRun><<<grid, kRopeThreads, 0, stream>>>(p);
  else gdn_norm_rope_kernel<false, kRun><<<grid, kRopeThreads, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t stream) {
  const int64_t rows = p.T * (p.t[0].heads + p.t[1].heads);
  if (rows <= 0) return cudaSuccess;
  // Runs of four heads where they still fill the SMs several times over; single heads where a
  // call is all latency.
  const int sms = device_sm_count();
  return rows >= (int64_t)sms * kRopeGroups * 4 * 8 ? launch<4>(p, stream) : launch<1>(p, stream);
}

}  // namespace gdn

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
//
// The general kernel takes positions on several axes as well (each pair has its axis, and a
// lane collects the cosines and sines of its eight pairs from the places of the axes they
// turn by) and appends: turned keys and untouched values go to a token's place in paged caches.
// Its norm can be left out; values that do not turn are then copied as they are, bit for bit.  Measured: 65536 tokens of 48 heads on three axes 243 us, 6.6 TB/s; 16384 tokens of as many heads appended
// 64.6 us, 6.2 TB/s; one token 2.7 us, a kernel's start.
#include <cuda_runtime.h>

#include <algorithm>

#include "decay.cuh"
#include "ptx.cuh"

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

// Cosines and sines of the eight pairs from 8 l on, each from the place of its axis.
__device__ __forceinline__ void load_axes8(const RopeParams& p, const int64_t (&place)[4], int l, float (&c)[8], float (&s)[8]) {
  const uint32_t mine = p.pair_axes[l >> 1] >> (16 * (l & 1));
#pragma unroll
  for (int a = 0; a < 4; ++a) {
    const uint32_t other = mine ^ (0x5555u * a), not_a = (other | other >> 1) & 0x5555u;
    if (a < p.axes && not_a != 0x5555u) {
      const float* row = p.cos_sin + place[a] * p.cs_stride + 8 * l;
      float ca[8], sa[8];
      load8(row, ca);
      load8(row + p.rotary / 2, sa);
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (!(not_a >> (2 * e) & 1u)) { c[e] = ca[e]; s[e] = sa[e]; }
    }
  }
}

// CTAs below q_ctas take q, those below qk_ctas k, the others v.  `per` heads a group; a token's groups side by side.
template <bool F16, bool kInterleaved, int kAhead, bool kGeneral>
__global__ void __launch_bounds__(kRopeThreads) gdn_norm_rope_kernel(const __grid_constant__ RopeParams p, unsigned q_ctas,
                                                                     unsigned qk_ctas, int per) {
  grid_wait();
  const int l = threadIdx.x % kRopeLanes;
  const bool is_k = blockIdx.x >= q_ctas, is_v = kGeneral && blockIdx.x >= qk_ctas;
  const RopeTensor& t = p.t[is_v ? 2 : is_k ? 1 : 0];
  // Eight groups a CTA: token and part of the thread's one.  (By 64-bit division it took a token with few heads 5 % longer.)
  const int parts = t.by_parts.by, cta = blockIdx.x - (is_v ? qk_ctas : is_k ? q_ctas : 0), whole = over(cta, t.by_parts);
  int part = (cta - whole * parts) * kRopeGroups + threadIdx.x / kRopeLanes;
  const int more = over(part, t.by_parts);
  const int64_t tok = (int64_t)whole * kRopeGroups + more;
  part -= more * parts;
  const int rot = p.cos_sin ? p.rotary / 16 : 0;  // lanes that rotate
  const bool halves = !kInterleaved && l < rot;
  const int v0 = 8 * (halves ? l : 2 * l), v1 = 8 * (halves ? l + rot : 2 * l + 1);
  bool ok = tok < p.T;
  const int own_in = kGeneral && ok ? min(per, t.heads - part * per) : 0;
  int64_t place = 0, places[4] = {0, 0, 0, 0}, slot = 0;
  if (kGeneral && ok && p.cos_sin) {  // every axis has to be on the table
    const int axes = p.axes ? p.axes : 1;
#pragma unroll
    for (int a = 0; a < 4; ++a)
      if (a < axes) places[a] = p.positions ? index_at(p.positions, p.pos_dtype, a * p.pos_axis + tok) : tok;
  }
  if (kGeneral && ok && is_k && p.slots) slot = index_at(p.slots, p.slot_dtype, tok);
  if (!kGeneral && ok && p.cos_sin) {
    place = p.positions ? index_at(p.positions, p.pos_dtype, tok) : tok;
    if (place < 0 || place >= p.places) {
      if (l == 0) atomicOr(p.dev_err, kDevErrPosition);
      ok = false;
    }
  }
  // `n` heads for every group of the warp, so that its lanes stay together; a group without a token or
  // with fewer heads left loads and stores nothing
  const int n = min(per, t.heads);
  int own = ok ? min(per, t.heads - part * per) : 0;
  const int64_t sx = t.x_sh, sy = t.y_sh;
  const uint16_t* x = reinterpret_cast<const uint16_t*>(t.x) + tok * t.x_st + (int64_t)part * per * sx;
  uint4 ra[kAhead], rb[kAhead];
  auto load = [&](int i, int h) {
    if (h < (kGeneral ? own_in : own)) {
      ra[i] = __ldcs(reinterpret_cast<const uint4*>(x + h * sx + v0));
      rb[i] = __ldcs(reinterpret_cast<const uint4*>(x + h * sx + v1));
    }
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) {
    ra[i] = rb[i] = make_uint4(0, 0, 0, 0);
    load(i, i);
  }
  int64_t row = tok * t.y_st;
  if (kGeneral) {  // places and the slot are looked at once the loads are on their way
    const int axes = p.cos_sin ? (p.axes ? p.axes : 1) : 0;
#pragma unroll
    for (int a = 0; a < 4; ++a) ok = ok && (a >= axes || (places[a] >= 0 && places[a] < p.places));
    if (!ok && tok < p.T && l == 0) atomicOr(p.dev_err, kDevErrPosition);
    if (!ok) own = 0;
    place = places[0];
    if (is_k && p.slots) {
      if (slot >= p.cache_slots && tok < p.T && l == 0) atomicOr(p.dev_err, kDevErrSlot);
      if (slot < 0 || slot >= p.cache_slots) own = 0;
      const int64_t page = p.page_shift >= 0 ? slot >> p.page_shift : slot / p.page_size;
      row = page * t.y_sp + (slot - page * p.page_size) * t.y_st;
    }
  }
  uint16_t* y = reinterpret_cast<uint16_t*>(t.y) + row + (int64_t)part * per * sy;
  float2 pa[4], qa[4], pb[4], qb[4];  // P and Q of the two vectors
  {
    float wa[8], wb[8], c[8], s[8];
    load_weight8(t, v0, p.weight_offset, wa);
    load_weight8(t, v1, p.weight_offset, wb);
#pragma unroll
    for (int e = 0; e < 8; ++e) { c[e] = 1.f; s[e] = 0.f; }
    if (kGeneral && ok && l < rot && p.axes && !is_v) {
      load_axes8(p, places, l, c, s);
    } else if (ok && l < rot && !is_v) {
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
      const float2 r = pair(kGeneral && !p.norm ? 1.f : rsqrtf(ss * (1.f / kHeadDim) + p.eps));
      uint32_t ya[4], yb[4];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        float2 ta = kInterleaved ? make_float2(a[e].y, a[e].x) : b[e], tb = kInterleaved ? make_float2(b[e].y, b[e].x) : a[e];
        if (kGeneral && l >= rot) ta = tb = pair(0.f);  // an infinity beside a value that does not turn stays out of it
        ya[e] = pack16x2<F16>(mul2(r, fma2(a[e], pa[e], mul2(ta, qa[e]))));
        yb[e] = pack16x2<F16>(mul2(r, fma2(b[e], pb[e], mul2(tb, qb[e]))));
      }
      if (kGeneral && (is_v || (!p.norm && l >= rot))) {
#pragma unroll
        for (int e = 0; e < 4; ++e) { ya[e] = ca[e]; yb[e] = cb[e]; }
      }
      if (h0 + i < own) {
        __stcs(reinterpret_cast<uint4*>(y + (h0 + i) * sy + v0), make_uint4(ya[0], ya[1], ya[2], ya[3]));
        __stcs(reinterpret_cast<uint4*>(y + (h0 + i) * sy + v1), make_uint4(yb[0], yb[1], yb[2], yb[3]));
      }
    }
  }
}

template <bool F16, int kAhead, bool kGeneral>
cudaError_t launch(RopeParams p, int per, cudaStream_t stream) {
  for (RopeTensor& t : p.t) t.by_parts = divisor((t.heads + per - 1) / per);
  auto ctas = [&](int heads) { return (p.T * ((heads + per - 1) / per) + kRopeGroups - 1) / kRopeGroups; };
  const int64_t q = ctas(p.t[0].heads), qk = q + ctas(p.t[1].heads);
  return launch_behind(p.interleaved ? gdn_norm_rope_kernel<F16, true, kAhead, kGeneral> : gdn_norm_rope_kernel<F16, false, kAhead, kGeneral>,
                       qk + ctas(p.t[2].heads), kRopeThreads, 0, stream, p, (unsigned)q, (unsigned)qk, per);
}
template <int kAhead>
cudaError_t launch(const RopeParams& p, int per, cudaStream_t stream) {
  if (p.general) return p.in_f16 ? launch<true, kAhead, true>(p, per, stream) : launch<false, kAhead, true>(p, per, stream);
  return p.in_f16 ? launch<true, kAhead, false>(p, per, stream) : launch<false, kAhead, false>(p, per, stream);
}

}  // namespace

cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t stream) {
  const int64_t rows = p.T * (p.t[0].heads + p.t[1].heads + p.t[2].heads);
  if (rows <= 0) return cudaSuccess;
  const int sms = device_sm_count();
  if (sms <= 0) return cudaErrorInvalidDevice;
  // Heads a group, a power of two up to 16 (heads come in such numbers, and a group with fewer waits for the others), so that one
  // round of groups is on the SMs; the loads of one, two or four heads under way.  2000 tokens x 32 heads take 6.8 us by eights, 8.2 by
  // fours, 10.2 by ones (plain; on three axes 8.3, 9.9 and 15.5); 8000 x 16 10.8 to 13.4 us by sixteens, 13.0 to 14.3 by eights;
  // 65536 x 48 249 us by sixteens, 290 by fours, 428 by ones; 1000 x 10 the same by ones and twos.
  constexpr int kResident = 80;  // groups on an SM
  const int64_t places = (int64_t)sms * kResident;
  int per = 1;
  while (per < 16 && per * places < rows) per *= 2;
  int ahead = per < 2 ? 1 : per < 16 ? 2 : 4;
  // The general kernel has few registers left beside four heads, and more groups on an SM are worth more than heads under way where a
  // group has less than that, in the mean: 178283 tokens x 4 + 1 heads 111 us with one, 118 with two, 141 with four; 100000 x 8 + 2 106, 100
  // and 107; 60000 x 12 + 4 94, 87 and 83.
  if (p.general) {
    int heads = 0, tensors = 0;
    for (const RopeTensor& t : p.t) {
      heads += t.heads < per ? t.heads : per;
      tensors += t.heads > 0;
    }
    ahead = std::min(ahead, heads < 4 * tensors ? 1 : heads < 8 * tensors ? 2 : 4);
  }
  if (ahead == 1) return launch<1>(p, per, stream);
  if (ahead == 2) return launch<2>(p, per, stream);
  return launch<4>(p, per, stream);
}

}  // namespace gdn

// One token of decay linear attention for sm_103a: for each batch row b and head h the
// state slot S (V-major 128 x 128: row = value index, column = key index) takes one token
// in place,
//
//   S' = g S + v k^T,   o = scale S' q.
//
// Row r of S' needs only row r of S, v_r, and all of k and q, so a state can be cut into
// blocks of rows that know nothing of each other.  S is read once and written once and
// nothing else counts (5 flops for 4 to 8 bytes): the step is bound by HBM bandwidth.  A
// warp takes 16 rows (8 of f32 states): 16 lanes (32) hold one row, 16 bytes of it each, so
// that every request of the warp is 512 contiguous bytes and each lane keeps its k and q
// columns in registers; all its loads are issued before the first is used.  Loads and stores
// are marked as streaming: a state is not seen again before the whole pool has passed.
// 1024 rows x 16 heads from a bf16 pool (1.09 GB) take 160 us, 6.8 TB/s (172 us with CTAs of
// four warps and plain loads and stores, 195 with eight); one row of 32 f32 states 4.5 us.
#include <cuda_runtime.h>

#include "decay.cuh"

namespace gdn {
namespace {

constexpr int kStepWarps = 2;  // of a CTA: it gives its place back the sooner
constexpr int kStepLoads = 8;  // 16-byte loads a lane has in flight

template <int SDT, bool F16>
__global__ void __launch_bounds__(32 * kStepWarps) gdn_decay_step_kernel(const __grid_constant__ DecayStepParams p) {
  using ST = StateType<SDT>;
  constexpr int kVec = ST::kVec, kLanes = kHeadDim / kVec;  // lanes of one row
  constexpr int kRowsPerLoad = 32 / kLanes;
  constexpr int kRows = kRowsPerLoad * kStepLoads;          // rows of a warp
  constexpr int kWarpsPerState = kHeadDim / kRows;
  const int lane = threadIdx.x & 31, col = (lane % kLanes) * kVec, sub = lane / kLanes;
  const int64_t w = (int64_t)blockIdx.x * kStepWarps + (threadIdx.x >> 5);
  const int64_t item = w / kWarpsPerState;
  if (item >= (int64_t)p.B * p.H) return;
  const int row0 = (int)(w % kWarpsPerState) * kRows + sub;
  const int b = (int)(item / p.H), h = (int)(item % p.H);
  const int64_t slot = p.state_idx ? index_at(p.state_idx, p.idx_dtype, b) : (int64_t)b;
  if (slot < 0 || slot >= p.st_slots) {
    if (lane == 0) atomicOr(p.dev_err, kDevErrIdx);
    return;
  }
  char* s = reinterpret_cast<char*>(p.state) +
            (slot * p.st_slot + (int64_t)h * p.st_head + (int64_t)row0 * kHeadDim + col) * ST::kBytes;
  uint4 raw[kStepLoads];
#pragma unroll
  for (int i = 0; i < kStepLoads; ++i)
    raw[i] = __ldcs(reinterpret_cast<const uint4*>(s + (int64_t)i * kRowsPerLoad * kHeadDim * ST::kBytes));
  const int hq = h / (p.H / p.H_qk), hv = h / (p.H / p.H_v);
  const char* kp = reinterpret_cast<const char*>(p.k) + (b * p.k_sb + (int64_t)hq * p.k_sh + col) * 2;
  const char* qp = reinterpret_cast<const char*>(p.q) + (b * p.q_sb + (int64_t)hq * p.q_sh + col) * 2;
  const uint16_t* vp = reinterpret_cast<const uint16_t*>(p.v) + b * p.v_sb + (int64_t)hv * p.v_sh + row0;
  float k[kVec], q[kVec], v[kStepLoads];
  if constexpr (kVec == 8) {
    unpack16x8<F16>(*reinterpret_cast<const uint4*>(kp), k);
    unpack16x8<F16>(*reinterpret_cast<const uint4*>(qp), q);
  } else {
    const uint2 kc = *reinterpret_cast<const uint2*>(kp), qc = *reinterpret_cast<const uint2*>(qp);
    const float2 k0 = unpack16<F16>(kc.x), k1 = unpack16<F16>(kc.y), q0 = unpack16<F16>(qc.x), q1 = unpack16<F16>(qc.y);
    k[0] = k0.x; k[1] = k0.y; k[2] = k1.x; k[3] = k1.y;
    q[0] = q0.x; q[1] = q0.y; q[2] = q1.x; q[3] = q1.y;
  }
#pragma unroll
  for (int i = 0; i < kStepLoads; ++i) v[i] = unpack16<F16>((uint32_t)vp[i * kRowsPerLoad]).x;
  const float g = p.g ? gate_at(p.g, p.g_dtype, b * p.g_sb + (int64_t)h * p.g_sh) : 1.f;
  uint16_t* o = reinterpret_cast<uint16_t*>(p.out) + b * p.o_sb + (int64_t)h * p.o_sh + row0;
#pragma unroll
  for (int i = 0; i < kStepLoads; ++i) {
    float x[kVec], acc = 0.f;
    ST::unpack(raw[i], x);
#pragma unroll
    for (int e = 0; e < kVec; ++e) {
      x[e] = fmaf(g, x[e], v[i] * k[e]);
      acc = fmaf(x[e], q[e], acc);
    }
    __stcs(reinterpret_cast<uint4*>(s + (int64_t)i * kRowsPerLoad * kHeadDim * ST::kBytes), ST::pack(x));
#pragma unroll
    for (int d = kLanes / 2; d > 0; d >>= 1) acc += __shfl_xor_sync(0xffffffffu, acc, d);
    if (lane % kLanes == 0) o[i * kRowsPerLoad] = (uint16_t)pack16x2<F16>(p.scale * acc, 0.f);
  }
}

template <int SDT, bool F16>
cudaError_t launch(const DecayStepParams& p, cudaStream_t stream) {
  constexpr int kWarpsPerState = kHeadDim / (32 / (kHeadDim / StateType<SDT>::kVec) * kStepLoads);
  const int64_t warps = (int64_t)p.B * p.H * kWarpsPerState;
  gdn_decay_step_kernel<SDT, F16>
      <<<(unsigned)((warps + kStepWarps - 1) / kStepWarps), 32 * kStepWarps, 0, stream>>>(p);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_decay_step(const DecayStepParams& p, cudaStream_t stream) {
  if ((int64_t)p.B * p.H <= 0) return cudaSuccess;
  switch (p.st_dtype) {
    case kF32: return p.in_f16 ? launch<0, true>(p, stream) : launch<0, false>(p, stream);
    case kBF16: return p.in_f16 ? launch<1, true>(p, stream) : launch<1, false>(p, stream);
    default: return p.in_f16 ? launch<2, true>(p, stream) : launch<2, false>(p, stream);
  }
}

}  // namespace gdn

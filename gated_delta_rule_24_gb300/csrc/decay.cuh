// Device helpers shared by the decay linear-attention kernels: loads of the dtypes that
// cross the C ABI and conversions of packed 16-bit pairs.
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <float.h>
#include <stdint.h>

#include "decay.h"
#include "prefill.h"

namespace gdn {

constexpr int32_t kDevErrCu = 0x1, kDevErrIdx = 0x2, kDevErrTimeout = 0x4, kDevErrPosition = 0x8, kDevErrSlot = 0x10,
                  kDevErrPage = 0x20, kDevErrLength = 0x40;

// n / d.by for 0 <= n < 2^31, in a fifth of the time that a division takes.
__device__ __forceinline__ int over(int n, const Divisor& d) { return (int)((__umulhi((uint32_t)n, d.mul) + (uint32_t)n) >> d.shift); }

__device__ __forceinline__ int64_t index_at(const void* p, int dtype, int64_t i) {
  return dtype == kI64 ? reinterpret_cast<const int64_t*>(p)[i] : (int64_t) reinterpret_cast<const int32_t*>(p)[i];
}
__device__ __forceinline__ float real_of(const void* p, int dtype, int64_t i) {
  if (dtype == kF32) return reinterpret_cast<const float*>(p)[i];
  if (dtype == kBF16) return __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(p)[i]);
  return __half2float(reinterpret_cast<const __half*>(p)[i]);
}
// A forget gate, clamped to [FLT_MIN, 1] as in the gated delta rule's kernels (a NaN gate
// becomes FLT_MIN there and here).
__device__ __forceinline__ float gate_at(const void* p, int dtype, int64_t i) {
  return fminf(fmaxf(real_of(p, dtype, i), FLT_MIN), 1.f);
}

// Two f32 operations in one instruction.
__device__ __forceinline__ float2 mul2(float2 a, float2 b) {
  float2 r;
  asm("{\n.reg .b64 x, y;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmul.rn.f32x2 x, x, y;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n.reg .b64 x, y, z;\nmov.b64 x, {%2, %3};\nmov.b64 y, {%4, %5};\nmov.b64 z, {%6, %7};\n"
      "fma.rn.f32x2 x, x, y, z;\nmov.b64 {%0, %1}, x;\n}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 pair(float x) { return make_float2(x, x); }
__device__ __forceinline__ float2 pair_at(const uint32_t* a) { return make_float2(__uint_as_float(a[0]), __uint_as_float(a[1])); }

template <bool F16>
__device__ __forceinline__ float2 unpack16(uint32_t w) {
  if (F16) return __half22float2(*reinterpret_cast<const __half2*>(&w));
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16x2(float lo, float hi) {
  if (F16) {
    __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<uint32_t*>(&h);
  }
  __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<uint32_t*>(&h);
}
template <bool F16>
__device__ __forceinline__ uint32_t pack16x2(float2 x) { return pack16x2<F16>(x.x, x.y); }
template <bool F16>
__device__ __forceinline__ void unpack16x8(const uint4& c, float (&x)[8]) {
  const uint32_t w[4] = {c.x, c.y, c.z, c.w};
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float2 f = unpack16<F16>(w[e]);
    x[2 * e] = f.x;
    x[2 * e + 1] = f.y;
  }
}
template <bool F16>
__device__ __forceinline__ uint4 pack16x8(const float (&x)[8]) {
  return make_uint4(pack16x2<F16>(x[0], x[1]), pack16x2<F16>(x[2], x[3]), pack16x2<F16>(x[4], x[5]),
                    pack16x2<F16>(x[6], x[7]));
}

// State element types of the kernels: 0 = f32, 1 = bf16, 2 = f16.  kVec elements fill 16 bytes.
template <int SDT>
struct StateType {
  static constexpr int kVec = SDT == 0 ? 4 : 8;
  static constexpr int kBytes = SDT == 0 ? 4 : 2;
  static __device__ __forceinline__ void unpack(const uint4& c, float (&x)[kVec]) {
    if constexpr (SDT == 0) {
      x[0] = __uint_as_float(c.x); x[1] = __uint_as_float(c.y);
      x[2] = __uint_as_float(c.z); x[3] = __uint_as_float(c.w);
    } else {
      unpack16x8<SDT == 2>(c, x);
    }
  }
  static __device__ __forceinline__ uint4 pack(const float (&x)[kVec]) {
    if constexpr (SDT == 0)
      return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    else
      return pack16x8<SDT == 2>(x);
  }
};

// Launches a kernel that waits by itself (grid_wait) for the one in front of it on the stream: its set-up is out of the way when that
// one ends, which saves some 2 us of a call among others.
template <typename... Params, typename... Args>
cudaError_t launch_behind(void (*kernel)(Params...), int64_t grid, int threads, int smem, cudaStream_t stream, const Args&... args) {
  cudaLaunchConfig_t c = {};
  c.gridDim = dim3((unsigned)grid);
  c.blockDim = dim3((unsigned)threads);
  c.dynamicSmemBytes = (size_t)smem;
  c.stream = stream;
  cudaLaunchAttribute a;
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  c.attrs = &a;
  c.numAttrs = 1;
  return cudaLaunchKernelEx(&c, kernel, args...);
}

}  // namespace gdn

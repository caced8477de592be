// Internal interface between the C-ABI host code (api.cpp) and the kernels of the decay
// linear-attention operators: the q/k norm with rotation (norm_rope.cu), the prefill
// (decay_prefill.cu) and the one-token step (decay_step.cu).  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdint.h>

namespace gdn {

// One head tensor of the norm-and-rotation kernel: [T, heads, 128], strides in elements.
struct RopeTensor {
  const void* x;
  int64_t x_st, x_sh;
  void* y;
  int64_t y_st, y_sh;
  const void* w;  // [128] or null
  int32_t heads, w_dtype;
};
struct RopeParams {
  RopeTensor t[2];        // q, then k (heads = 0: absent)
  const float* cos_sin;   // [places, rotary] f32 (cosines, then sines) or null
  int64_t cs_stride, places;
  const void* positions;  // [T] or null (token t takes place t)
  int32_t* dev_err;
  int64_t T;
  int32_t pos_dtype, rotary, interleaved, in_f16;
  float eps, weight_offset;
};
cudaError_t launch_norm_rope(const RopeParams& p, cudaStream_t stream);

// Linear attention with a decay over packed sequences: S <- g S + v k^T, o = scale S q.
struct DecayPrefillParams {
  CUtensorMap tm_q;  // [T, H_qk, 128], box (64 values, 1 head, kDecayChunk tokens), 128B swizzle
  CUtensorMap tm_k;
  CUtensorMap tm_v;  // [T, H_v, 128]
  CUtensorMap tm_o;  // output [T, H, 128] (stores)
  CUtensorMap tm_sin;   // state pools [slots, H, 128, 128], box (128 bytes of columns, 128 rows, 1, 1), 128B
  CUtensorMap tm_sout;  // swizzle; valid where sin_tma, sout_tma say so
  CUtensorMap tm_ws;    // the states of the workspace, as a pool of one head
  const void* g;     // [T, H] or null, strides in elements; a token stride of 0 is one decay for each head
  int64_t g_st, g_sh;
  const void* s_in;  // [slots, H, 128, 128] or null
  int64_t sin_slot, sin_head, sin_slots;
  void* s_out;
  int64_t sout_slot, sout_head, sout_slots;
  const void* state_idx;  // [N] or null
  const void* cu;         // [N + 1]
  void* out;              // [T, H, 128]
  int64_t o_st, o_sh;
  int32_t* dev_err;
  int64_t T;
  int32_t N, H, H_qk, H_v;
  int32_t g_dtype, sin_dtype, sout_dtype, idx_dtype, cu_dtype;
  float scale;
  int32_t op_f16;
  int32_t sin_tma, sout_tma;  // incoming states by TMA (f32 or of q's dtype), outgoing ones by TMA
  // Sequences cut into `splits` segments of whole chunks (1: not cut), segment x of a sequence of c
  // chunks holding chunks [c x / splits, c (x + 1) / splits).  With U = N H and unit nh = n H + h:
  float* ws;        // [U][splits - 1] states of 128 x 128: the state behind segment x, once joined
  float* ws_decay;  // [U][splits - 1] decays of whole segments
  int32_t splits;
  // Testing aids: the bound of every wait in ns (0: 0.2 s), and a first hand-off of every CTA, that of the gates, withheld.
  int32_t hold_gates;
  uint64_t wait_ns;
};
constexpr int kDecayChunk = 128;  // tokens of a chunk

// Segments a sequence for U units on `sms` SMs, `chunks` the mean chunks of a sequence.
int decay_splits(int64_t units, double chunks, int sms);
cudaError_t launch_decay_prefill(const DecayPrefillParams& p, cudaStream_t stream);

// The same recurrence for one token of each batch row, states updated in place.
struct DecayStepParams {
  const void* q;  // [B, H_qk, 128], strides in elements
  int64_t q_sb, q_sh;
  const void* k;
  int64_t k_sb, k_sh;
  const void* v;  // [B, H_v, 128]
  int64_t v_sb, v_sh;
  const void* g;  // [B, H] or null
  int64_t g_sb, g_sh;
  void* state;  // [slots, H, 128, 128]
  int64_t st_slot, st_head, st_slots;
  const void* state_idx;  // [B] or null
  void* out;              // [B, H, 128]
  int64_t o_sb, o_sh;
  int32_t* dev_err;
  int32_t B, H, H_qk, H_v;
  int32_t g_dtype, st_dtype, idx_dtype;
  float scale;
  int32_t in_f16;
};
cudaError_t launch_decay_step(const DecayStepParams& p, cudaStream_t stream);

}  // namespace gdn

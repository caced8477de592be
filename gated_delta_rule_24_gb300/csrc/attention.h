// Internal interface between the C-ABI host code (api.cpp) and the kernels of the attention over a
// paged cache (attention.cu).  Not part of the public ABI.
#pragma once
#include <cuda_runtime_api.h>
#include <stdint.h>

namespace gdn {

struct AttentionParams {
  const void* q;  // [N * tokens, H_q, 128], strides in elements
  int64_t q_st, q_sh;
  const void* k;  // [pages, page_size, H_k, 128]
  int64_t k_sp, k_st, k_sh;
  const void* v;
  int64_t v_sp, v_st, v_sh;
  const void* table;  // [N, max_pages]
  int64_t table_st;
  const void* lengths;  // [N]
  const void* prefix_pages;
  void* out;  // [N * tokens, H_q, 128]
  int64_t o_st, o_sh;
  float* lse;  // [N * tokens, H_q] or null
  int64_t lse_st;
  int32_t* dev_err;
  int64_t pages;
  int32_t N, tokens, H_q, H_k, page_size, max_pages, prefix;
  int32_t table_dtype, len_dtype, prefix_dtype;
  float scale;
  int32_t op_f16;
};
cudaError_t launch_attention(const AttentionParams& p, cudaStream_t stream);

}  // namespace gdn

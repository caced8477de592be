// Internal interface between the C-ABI host code (api.cpp) and the kernels of the attention over a
// paged cache (attention.cu).  Not part of the public ABI.
#pragma once
#include <cuda.h>
#include <cuda_runtime_api.h>
#include <stdint.h>

#include "decay.h"

namespace gdn {

constexpr int kOwnKeys = 64;                         // keys of a tile of attention_own.cuh
constexpr int kPrefixKeys = 128, kPrefixRows = 256;  // tiles of attention_prefix.cuh
constexpr uint64_t kAttentionWaitNs = 200000000;      // the bound of every wait, unless a test sets another
constexpr float kAttentionBad = -1.f;                // as a part's sum: it met a bad page, or gave up

struct AttentionParams {
  CUtensorMap tm_k;  // [pages, H_k, 2 halves, page_size, 64], box (64 values, box_rows places, 2 halves, 1 head, 1 page), 128B swizzle
  CUtensorMap tm_v;
  const void* q;  // [N * tokens, H_q, 128], strides in elements
  int64_t q_st, q_sh;
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
  int32_t N, tokens, H_q, H_k, group, page_size, max_pages, prefix;
  Divisor by_group, by_page;  // the two above
  int32_t box_rows;  // places of a box
  int32_t table_dtype, len_dtype, prefix_dtype;
  float scale;
  int32_t op_f16;
  // Workers, units and where their partial results go (attention.cu says what these are).
  int32_t workers;
  int32_t blocks, block_rows;          // row blocks of a (sequence, key head) and the rows of one
  int32_t block_groups, blocks_aside;  // groups of blocks, and the blocks of one (the last group may have fewer)
  Divisor by_groups, by_aside, by_rows, by_blocks, by_subs;  // block_groups, blocks_aside, block_rows, blocks, H_k * blocks
  int32_t prefix_blocks;       // 1 where the prefix is walked like the own pages, by one block of rows a key head, else 0
  float* part_o;               // [slots][block_rows][128]
  float* part_ml;              // [slots][block_rows][2]: base, sum
  int32_t* first_worker;       // [units], then
  int32_t* last_worker;        // [units]
  // The prefix by attention_prefix.cuh (prefix_blocks is then 0): units of a key head, workers at most, their parts, and the first and
  // the last worker of a unit.
  CUtensorMap tm_pk;  // [pages, page_size, H_k, 128], box (64 values, 1 head, prefix_box places, 1 page), 128B swizzle
  CUtensorMap tm_pv;
  int32_t prefix_box, prefix_units, prefix_workers;
  Divisor by_units;  // prefix_units
  int32_t *prefix_first, *prefix_last;  // [units]
  float* prefix_o;   // [slots][16][kPrefixRows][8]: columns by eights
  float* prefix_ml;  // [slots][kPrefixRows][2]
  // The bound of every wait in ns, and a testing aid: the first copy of every warp withheld.
  int32_t hold_copies;
  uint64_t wait_ns;
};

// Fills in what follows from the sizes (and the workspace, where it is given); returns the workspace's bytes.
size_t plan_attention(AttentionParams* p, int sms, void* workspace);
cudaError_t launch_attention(const AttentionParams& p, cudaStream_t stream);

}  // namespace gdn

// prep.h -- arguments of the kernel in prep.cu.
#pragma once
#include <cstdint>

#include <cuda_bf16.h>
#include <cuda_runtime.h>

namespace mla {

// q, kv, q_weight, kv_weight, rows, cache, new_lens and positions may be null.
struct PrepParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  int64_t q_stride, kv_stride;  // elements from a token to the next
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* kv_weight;
  const float* cos_sin;  // [max_position, 64]: cos 32, sin 32
  const int32_t* positions;
  const int32_t* new_lens;
  const int32_t* seq_lens;
  const int32_t* block_table;
  __nv_bfloat16* q_out;
  uint4* rows;
  uint4* cache;
  int32_t* status;
  float eps;
  int B, H, max_new, max_position, num_pages, max_pages;
  int max_len;  // that a sequence may have
};

}  // namespace mla

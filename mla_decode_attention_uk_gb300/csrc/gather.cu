// gather.cu -- reading a cache back: each sequence's newest tokens as bf16 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp4kv.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

namespace mla {

namespace {

constexpr int kGatherThreads = 288;  // four rows of 72 chunks

// One CTA per (sequence, page that holds any of the tokens): a thread has 16 bytes
// of every fourth row.
template <Kind kKind>
__global__ void __launch_bounds__(kGatherThreads)
gather_kernel(const uint8_t* __restrict__ cache, const float* __restrict__ kv_scale,
              const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
              int max_new, const int32_t* __restrict__ new_lens, int num_pages, int max_pages,
              uint4* __restrict__ rows, int32_t* __restrict__ status) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  NewTokens nt;
  if (!nt.load(seq_lens, new_lens, max_new, max_pages * kPage, b, threadIdx.x == 0, status))
    return;
  const int logical = nt.first / kPage + blockIdx.x;
  if (blockIdx.x >= nt.pages()) return;
  const int page = block_table[static_cast<size_t>(b) * max_pages + logical];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
    return;
  }
  float scale = 1.0f;
  if constexpr (kKind != Kind::kBf16) {
    scale = kv_scale[page];
    if (!scale_in_range(scale)) {
      if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
      scale = 1.0f;
    }
  }
  const int c = threadIdx.x % kChunks;
  const int r0 = max(nt.first - logical * kPage, 0), r1 = min(nt.len - logical * kPage, kPage);
  uint4* const dst = rows + (static_cast<ptrdiff_t>(b) * max_new + logical * kPage - nt.first) *
                                kChunks + c;
#pragma unroll 4
  for (int r = r0 + threadIdx.x / kChunks; r < r1; r += kGatherThreads / kChunks) {
    uint4 x;
    if constexpr (kKind == Kind::kBf16) {
      x = *reinterpret_cast<const uint4*>(
          cache + (static_cast<size_t>(page) * kPage + r) * (kDqk * 2) + c * 16);
    } else {
      float v[8];
      if constexpr (kKind == Kind::kFp8)
        values8x8(*reinterpret_cast<const uint2*>(cache + static_cast<size_t>(page) * kPageBytes8 +
                                                  r * kDqk + c * 8),
                  v);
      else
        row_values4(cache + static_cast<size_t>(page) * kPageBytes4 + r * kRow4, c, v);
      x = make_uint4(pack_bf16x2(v[0] * scale, v[1] * scale),
                     pack_bf16x2(v[2] * scale, v[3] * scale),
                     pack_bf16x2(v[4] * scale, v[5] * scale),
                     pack_bf16x2(v[6] * scale, v[7] * scale));
    }
    dst[static_cast<ptrdiff_t>(r) * kChunks] = x;
  }
}

}  // namespace

cudaError_t launch_gather(Kind kind, const void* cache, const float* kv_scale,
                          const int32_t* block_table, const int32_t* seq_lens, int max_new,
                          const int32_t* new_lens, int B, int num_pages, int max_pages,
                          void* rows, int32_t* status, cudaStream_t st) {
  const auto kern = kind == Kind::kFp4   ? gather_kernel<Kind::kFp4>
                    : kind == Kind::kFp8 ? gather_kernel<Kind::kFp8>
                                         : gather_kernel<Kind::kBf16>;
  return launch_pdl(kern, dim3(touched_pages(max_new, max_pages), B), dim3(kGatherThreads), 0, st,
                    static_cast<const uint8_t*>(cache), kv_scale, block_table, seq_lens, max_new,
                    new_lens, num_pages, max_pages, static_cast<uint4*>(rows), status);
}

}  // namespace mla

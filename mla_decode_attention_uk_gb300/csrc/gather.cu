// gather.cu -- reading a cache back: each sequence's newest tokens as bf16 rows.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <type_traits>

#include "common.cuh"
#include "fp4kv.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

namespace mla {

namespace {

constexpr int kGatherThreads = 288;  // four rows of 72 chunks

// Registers a thread: with 56 the 13 prompts below take 14.7 us from 4 bits instead of 13.0.
constexpr int gather_regs(Kind kind) { return kind == Kind::kBf16 ? 56 : 48; }

struct GatherParams {
  const uint8_t* cache;
  const float* kv_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  uint4* rows;
  int32_t* status;
  int B, max_new, num_pages, max_pages;
};

// A page's tokens: a thread has 16 bytes of every fourth row.
template <Kind kKind>
__device__ __forceinline__ void copy_page(const GatherParams& P, int b, int first, int len,
                                          int logical) {
  const auto [cache, kv_scale, block_table, seq_lens, new_lens, rows, status, B, max_new,
              num_pages, max_pages] = P;
  const int page = block_table[static_cast<size_t>(b) * max_pages + logical];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
    return;
  }
  // (Looked at behind the rows' loads: a trip to memory next to theirs, not before.)
  const float given = kKind != Kind::kBf16 ? kv_scale[page] : 1.0f;
  const bool in_range = scale_in_range(given);
  const float scale = in_range ? given : 1.0f;
  const int c = threadIdx.x % kChunks;
  const int r0 = max(first - logical * kPage, 0), r1 = min(len - logical * kPage, kPage);
  uint4* const dst = rows + (static_cast<ptrdiff_t>(b) * max_new + logical * kPage - first) *
                                kChunks + c;
  // Values are rounded once: products by a power of two, as every scale of the appends is,
  // are exact; others may need 28 bits.
  auto put = [&](int r, const float (&v)[8], const auto exact) {
    float x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = exact ? v[k] * scale : mul_odd(v[k], scale);
    dst[static_cast<ptrdiff_t>(r) * kChunks] =
        make_uint4(pack_bf16x2(x[0], x[1]), pack_bf16x2(x[2], x[3]), pack_bf16x2(x[4], x[5]),
                   pack_bf16x2(x[6], x[7]));
  };
  // kDeep rows' loads in flight.
  auto copy = [&](const auto deep, const auto exact) {
    constexpr int kStep = kGatherThreads / kChunks, kDeep = deep;
#pragma unroll 1
    for (int r = r0 + threadIdx.x / kChunks; r < r1; r += kStep * kDeep) {
      if constexpr (kKind == Kind::kBf16) {
        uint4 x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          x[k] = *reinterpret_cast<const uint4*>(
              cache + c * 16 +
              (static_cast<size_t>(page) * kPage + min(r + kStep * k, r1 - 1)) * (kDqk * 2));
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          if (r + kStep * k < r1) dst[static_cast<ptrdiff_t>(r + kStep * k) * kChunks] = x[k];
      } else if constexpr (kKind == Kind::kFp8) {
        uint2 x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          x[k] = *reinterpret_cast<const uint2*>(cache + static_cast<size_t>(page) * kPageBytes8 +
                                                 min(r + kStep * k, r1 - 1) * kDqk + c * 8);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          float v[8];
          values8x8(x[k], v);
          if (r + kStep * k < r1) put(r + kStep * k, v, exact);
        }
      } else {
        Raw4 x[kDeep];
#pragma unroll
        for (int k = 0; k < kDeep; ++k)
          x[k] = load_raw4(cache + static_cast<size_t>(page) * kPageBytes4 +
                               min(r + kStep * k, r1 - 1) * kRow4,
                           c);
#pragma unroll
        for (int k = 0; k < kDeep; ++k) {
          float v[8];
          values4(x[k], c, v);
          if (r + kStep * k < r1) put(r + kStep * k, v, exact);
        }
      }
    }
  };
  using std::integral_constant;
  copy(integral_constant<int, 8>{}, std::true_type{});
  // (Rare pages, a second time.  A branch in the loop above cost all pages 4 to 7 %, one in
  // front of it would wait for the scale.)
  if constexpr (kKind != Kind::kBf16)
    if ((__float_as_uint(scale) & 0x7fffffu) != 0)
      copy(integral_constant<int, 2>{}, std::false_type{});
  if (!in_range && threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
}

// One CTA per (sequence, page that it can touch).  13 prompts of 512 to 8190 tokens: 13.0
// us from 4 bits, 4.3 TB/s (three to start: lengths, table and scale one after the other;
// with a list of the pages 12.7, and 0.8 more for small calls; codes looked up instead of
// converted 13.8), 13.5 from 8 bits, 16.2 from bf16 (5.4 TB/s).
template <Kind kKind>
__global__ void __maxnreg__(gather_regs(kKind))
gather_kernel(const __grid_constant__ GatherParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  NewTokens nt;
  if (nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, b, threadIdx.x == 0,
              P.status) &&
      blockIdx.x < nt.pages())
    copy_page<kKind>(P, b, nt.first, nt.len, nt.first / kPage + static_cast<int>(blockIdx.x));
}

}  // namespace

cudaError_t launch_gather(Kind kind, const void* cache, const float* kv_scale,
                          const int32_t* block_table, const int32_t* seq_lens, int max_new,
                          const int32_t* new_lens, int B, int num_pages, int max_pages,
                          void* rows, int32_t* status, cudaStream_t st) {
  const GatherParams P{static_cast<const uint8_t*>(cache), kv_scale, block_table, seq_lens,
                       new_lens, static_cast<uint4*>(rows), status, B, max_new, num_pages,
                       max_pages};
  const auto kern = kind == Kind::kFp4   ? gather_kernel<Kind::kFp4>
                    : kind == Kind::kFp8 ? gather_kernel<Kind::kFp8>
                                         : gather_kernel<Kind::kBf16>;
  return launch_pdl(kern, dim3(touched_pages(max_new, max_pages), B), dim3(kGatherThreads), 0, st,
                    P);
}

}  // namespace mla

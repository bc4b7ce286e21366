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

constexpr int kGatherCtas = 4;  // on an SM, of a list

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
  float scale = 1.0f;
  if constexpr (kKind != Kind::kBf16) {
    scale = kv_scale[page];
    if (!scale_in_range(scale)) {
      if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
      scale = 1.0f;
    }
  }
  const int c = threadIdx.x % kChunks;
  const int r0 = max(first - logical * kPage, 0), r1 = min(len - logical * kPage, kPage);
  uint4* const dst = rows + (static_cast<ptrdiff_t>(b) * max_new + logical * kPage - first) *
                                kChunks + c;
  auto put = [&](int r, const float (&v)[8]) {
    dst[static_cast<ptrdiff_t>(r) * kChunks] =
        make_uint4(pack_bf16x2(v[0] * scale, v[1] * scale), pack_bf16x2(v[2] * scale, v[3] * scale),
                   pack_bf16x2(v[4] * scale, v[5] * scale),
                   pack_bf16x2(v[6] * scale, v[7] * scale));
  };
  // kDeep rows' loads in flight.
  constexpr int kStep = kGatherThreads / kChunks, kDeep = 8;
  for (int r = r0 + threadIdx.x / kChunks; r < r1; r += kStep * kDeep) {
    if constexpr (kKind == Kind::kBf16) {
      uint4 x[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        x[k] = *reinterpret_cast<const uint4*>(
            cache + (static_cast<size_t>(page) * kPage + min(r + kStep * k, r1 - 1)) * (kDqk * 2) +
            c * 16);
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
        if (r + kStep * k < r1) put(r + kStep * k, v);
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
        if (r + kStep * k < r1) put(r + kStep * k, v);
      }
    }
  }
}

// One CTA per (sequence, page that it can touch), or a list of the pages.
template <Kind kKind, bool kList>
__global__ void __launch_bounds__(kGatherThreads, kGatherCtas)
gather_kernel(const __grid_constant__ GatherParams P) {
  griddep_wait();
  griddep_launch_dependents();
  if constexpr (kList) {
    __shared__ UnitList list;
    const long long pages = list.make(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, P.B,
                                      P.status, [](const NewTokens& nt) { return nt.pages(); });
    for (long long f = blockIdx.x; f < pages; f += gridDim.x) {
      const int b = list.find(f), len = list.len[b];
      copy_page<kKind>(P, b, list.first[b], len,
                       (len - 1) / kPage - static_cast<int>(list.upto[b] - 1 - f));
    }
  } else {
    const int b = blockIdx.y;
    NewTokens nt;
    if (nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, b, threadIdx.x == 0,
                P.status) &&
        blockIdx.x < nt.pages())
      copy_page<kKind>(P, b, nt.first, nt.len, nt.first / kPage + static_cast<int>(blockIdx.x));
  }
}

template <Kind kKind>
cudaError_t launch(const GatherParams& P, int sm_count, cudaStream_t st) {
  const int touched = touched_pages(P.max_new, P.max_pages);
  if (use_list(P.max_new, P.B)) {
    const int64_t most = static_cast<int64_t>(touched) * P.B;
    const int ctas =
        most < sm_count * kGatherCtas ? static_cast<int>(most) : sm_count * kGatherCtas;
    return launch_pdl(gather_kernel<kKind, true>, dim3(ctas), dim3(kGatherThreads), 0, st, P);
  }
  return launch_pdl(gather_kernel<kKind, false>, dim3(touched, P.B), dim3(kGatherThreads), 0, st,
                    P);
}

}  // namespace

cudaError_t launch_gather(Kind kind, const void* cache, const float* kv_scale,
                          const int32_t* block_table, const int32_t* seq_lens, int max_new,
                          const int32_t* new_lens, int B, int num_pages, int max_pages,
                          void* rows, int32_t* status, int sm_count, cudaStream_t st) {
  const GatherParams P{static_cast<const uint8_t*>(cache), kv_scale, block_table, seq_lens,
                       new_lens, static_cast<uint4*>(rows), status, B, max_new, num_pages,
                       max_pages};
  return kind == Kind::kFp4   ? launch<Kind::kFp4>(P, sm_count, st)
         : kind == Kind::kFp8 ? launch<Kind::kFp8>(P, sm_count, st)
                              : launch<Kind::kBf16>(P, sm_count, st);
}

}  // namespace mla

// select.cu -- block-sparse decode: cheap scores of the cache's pages for each
// query token, and the selection of the pages that it attends to.
//
//   score(b, t, j) = max_h  query[b, t, h, :] . key_j      (576-wide, fp32 sums)
//   select(b, t)   = the first and last few pages, and the best-scored others
//
// The selection is a block table and lengths of its own, one line per query
// token: the decode step then runs on it as on any batch of sequences with one
// query token each.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"

namespace mla {

namespace {

// A sequence's length within [T, cap], as the planner clamps it.
__device__ __forceinline__ int clamp_len(int L, int T, int cap, bool report, int32_t* status) {
  if (L < T || L > cap) {
    if (report) record_status(status, MLA_STATUS_BOUNDS);
    return L < T ? T : cap;
  }
  return L;
}

// D += A B on the warp-level tensor pipe: 16 pages x 8 heads x 16 columns.
__device__ __forceinline__ void mma_16x8x16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0,
                                            uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, "
      "{%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

constexpr int kScoreThreads = 128;
constexpr int kScorePages = 64;               // 16 per warp
constexpr int kScoreRows = 16;                // query rows staged at a time
constexpr int kScoreStride = kDqk * 2 + 64;   // bytes; odd multiple of 64: no bank conflicts
constexpr int kSteps = kDqk / 32;             // 32 columns (16 bytes per thread) at a time

__global__ void __launch_bounds__(kScoreThreads)
score_kernel(const uint4* __restrict__ query, const uint4* __restrict__ keys,
             const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
             int T, int H, int num_pages, int max_pages, float* __restrict__ scores,
             int32_t* __restrict__ status) {
  __shared__ __align__(16) uint8_t q_sh[kScoreRows * kScoreStride];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int L = clamp_len(seq_lens[b], T, max_pages * kPage, threadIdx.x == 0 && blockIdx.x == 0,
                          status);
  const int page0 = blockIdx.x * kScorePages;
  const int held = (L + kPage - 1) / kPage;  // pages in use
  if (page0 >= held) {
    for (int i = threadIdx.x; i < T * kScorePages; i += kScoreThreads) {
      const int t = i / kScorePages, j = page0 + i % kScorePages;
      if (j < max_pages) scores[(static_cast<size_t>(b) * T + t) * max_pages + j] = -INFINITY;
    }
    return;
  }
  // This warp's 16 page keys stay in registers: thread (g, c) holds columns
  // 32 k + 8 c .. + 7 of pages g and g + 8 for every k.  (The order of the
  // columns inside a product does not matter as long as queries use the same.)
  const int g = lane >> 2, c = lane & 3;
  uint32_t a[kSteps][2][4];
  {
    int row[2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      const int j = page0 + 16 * warp + g + 8 * r;
      int p = j < held ? block_table[static_cast<size_t>(b) * max_pages + j] : 0;
      if (p < 0 || p >= num_pages) {
        record_status(status, MLA_STATUS_BOUNDS);
        p = 0;
      }
      row[r] = p;
    }
#pragma unroll
    for (int k = 0; k < kSteps; ++k) {
      const uint4 x = keys[static_cast<size_t>(row[0]) * (kDqk / 8) + 4 * k + c];
      const uint4 y = keys[static_cast<size_t>(row[1]) * (kDqk / 8) + 4 * k + c];
      a[k][0][0] = x.x; a[k][0][1] = y.x; a[k][0][2] = x.y; a[k][0][3] = y.y;
      a[k][1][0] = x.z; a[k][1][1] = y.z; a[k][1][2] = x.w; a[k][1][3] = y.w;
    }
  }
  for (int t = 0; t < T; ++t) {
    float top[2] = {-INFINITY, -INFINITY};
    for (int h0 = 0; h0 < H; h0 += kScoreRows) {
      __syncthreads();
      const uint4* src =
          query + (static_cast<size_t>(b) * T * H + static_cast<size_t>(t) * H + h0) * (kDqk / 8);
      for (int i = threadIdx.x; i < kScoreRows * (kDqk / 8); i += kScoreThreads)
        *reinterpret_cast<uint4*>(q_sh + (i / (kDqk / 8)) * kScoreStride + (i % (kDqk / 8)) * 16) =
            src[i];
      __syncthreads();
#pragma unroll
      for (int n = 0; n < kScoreRows / 8; ++n) {
        float d[4] = {};
        const uint8_t* q = q_sh + (8 * n + g) * kScoreStride + c * 16;
#pragma unroll
        for (int k = 0; k < kSteps; ++k) {
          const uint4 v = *reinterpret_cast<const uint4*>(q + 64 * k);
          mma_16x8x16(d, a[k][0], v.x, v.y);
          mma_16x8x16(d, a[k][1], v.z, v.w);
        }
        top[0] = fmaxf(top[0], fmaxf(d[0], d[1]));
        top[1] = fmaxf(top[1], fmaxf(d[2], d[3]));
      }
    }
    const int seen = (L - T + t + kPage) / kPage;  // pages that query t sees
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 1));
      top[r] = fmaxf(top[r], __shfl_xor_sync(0xffffffffu, top[r], 2));
      const int j = page0 + 16 * warp + g + 8 * r;
      if (c == 0 && j < max_pages)
        scores[(static_cast<size_t>(b) * T + t) * max_pages + j] = j < seen ? top[r] : -INFINITY;
    }
  }
}

constexpr int kSelThreads = 256;

// Keys in the order of the scores: larger is better, NaN below everything,
// the two zeros equal.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0u;
  const uint32_t u = __float_as_uint(x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Exclusive count of `flag` over the CTA's threads, and the total.
__device__ __forceinline__ int block_rank(bool flag, int* warp_cnt, int* total) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t m = __ballot_sync(0xffffffffu, flag);
  if (lane == 0) warp_cnt[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kSelThreads / 32; ++w) {
    const int n = warp_cnt[w];
    before += w < warp ? n : 0;
    all += n;
  }
  __syncthreads();
  *total = all;
  return before + __popc(m & ((1u << lane) - 1u));
}

// One CTA per query token.
__global__ void __launch_bounds__(kSelThreads)
select_kernel(const float* __restrict__ scores, const int32_t* __restrict__ block_table,
              const int32_t* __restrict__ seq_lens, int T, int max_pages, int top_k,
              int keep_first, int keep_last, int32_t* __restrict__ sel_table,
              int32_t* __restrict__ sel_pages, int32_t* __restrict__ sel_lens,
              int32_t* __restrict__ status) {
  __shared__ int hist[256];
  __shared__ int warp_cnt[kSelThreads / 32];
  __shared__ uint32_t prefix_sh;
  __shared__ int need_sh;
  griddep_wait();
  griddep_launch_dependents();
  const int row = blockIdx.x, b = row / T, t = row % T;
  const int L = clamp_len(seq_lens[b], T, max_pages * kPage, threadIdx.x == 0, status);
  const int keys = L - T + t + 1;              // keys that this query sees
  const int seen = (keys + kPage - 1) / kPage;
  const float* s = scores + static_cast<size_t>(row) * max_pages;
  const int32_t* table = block_table + static_cast<size_t>(b) * max_pages;
  int32_t* out_table = sel_table + static_cast<size_t>(row) * top_k;
  int32_t* out_pages = sel_pages ? sel_pages + static_cast<size_t>(row) * top_k : nullptr;
  const int count = min(seen, top_k);
  // The key of the last page that the scores select, and how many of the pages
  // with just that key are selected (those of the lowest numbers).
  uint32_t last_key = 0;
  int need = 0;
  if (seen > top_k) {
    need = top_k - keep_first - keep_last;
    uint32_t mask = 0;
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      for (int i = threadIdx.x; i < 256; i += kSelThreads) hist[i] = 0;
      __syncthreads();
      for (int j = keep_first + threadIdx.x; j < seen - keep_last; j += kSelThreads) {
        const uint32_t u = order_key(s[j]);
        if ((u & mask) == last_key) atomicAdd(&hist[(u >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        // The bin, from the top, in which the count of better keys passes
        // `need`: lane i owns bins 255 - 8 i downwards.
        const int lane = threadIdx.x;
        int own = 0;
        for (int k = 0; k < 8; ++k) own += hist[255 - 8 * lane - k];
        int upto = own;
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const int before = upto - own;
        if (before < need && need <= upto) {
          int left = need - before, bin = 255 - 8 * lane;
          while (left > hist[bin]) left -= hist[bin--];
          prefix_sh = last_key | (static_cast<uint32_t>(bin) << shift);
          need_sh = left;
        }
      }
      __syncthreads();
      last_key = prefix_sh;
      need = need_sh;
      mask |= 255u << shift;
      __syncthreads();
    }
    if (top_k == keep_first + keep_last) last_key = 0xffffffffu;  // none by score
  }
  int done = 0, ties = 0;  // selected so far; pages with last_key so far
  for (int j0 = 0; j0 < seen; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    bool take = j < seen, tie = false;
    if (seen > top_k && take && j >= keep_first && j < seen - keep_last) {
      const uint32_t u = order_key(s[j]);
      take = u > last_key;
      tie = u == last_key;
    }
    int n = 0;
    if (seen > top_k) {
      const int rank = ties + block_rank(tie, warp_cnt, &n);
      ties += n;
      take |= tie && rank < need;
    }
    const int at = done + block_rank(take, warp_cnt, &n);
    done += n;
    if (take && at < top_k) {
      out_table[at] = table[j];
      if (out_pages) out_pages[at] = j;
    }
  }
  for (int i = count + threadIdx.x; i < top_k; i += kSelThreads) {
    out_table[i] = -1;
    if (out_pages) out_pages[i] = -1;
  }
  if (threadIdx.x == 0) sel_lens[row] = keys - (seen - count) * kPage;
}

}  // namespace

cudaError_t launch_score(const void* query, const void* page_keys, const int32_t* block_table,
                         const int32_t* seq_lens, int B, int T, int H, int num_pages,
                         int max_pages, float* scores, int32_t* status, cudaStream_t st) {
  const dim3 grid((max_pages + kScorePages - 1) / kScorePages, B);
  return launch_pdl(score_kernel, grid, dim3(kScoreThreads), 0, st,
                    static_cast<const uint4*>(query), static_cast<const uint4*>(page_keys),
                    block_table, seq_lens, T, H, num_pages, max_pages, scores, status);
}

cudaError_t launch_select(const float* scores, const int32_t* block_table,
                          const int32_t* seq_lens, int B, int T, int max_pages, int top_k,
                          int keep_first, int keep_last, int32_t* sel_table, int32_t* sel_pages,
                          int32_t* sel_lens, int32_t* status, cudaStream_t st) {
  return launch_pdl(select_kernel, dim3(B * T), dim3(kSelThreads), 0, st, scores, block_table,
                    seq_lens, T, max_pages, top_k, keep_first, keep_last, sel_table, sel_pages,
                    sel_lens, status);
}

}  // namespace mla

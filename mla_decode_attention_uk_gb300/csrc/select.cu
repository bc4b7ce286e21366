// select.cu -- block-sparse decode: cheap scores of the cache's pages for each
// query token, and the selection of the pages that it attends to.
//
//   score(b, t, j) = max_h  query[b, t, h, :] . key_j      (576-wide, fp32 sums)
//   select(b, t)   = the first and last few pages, and the best-scored others
//
// The selection is a block table and lengths of its own, one line per query
// token: the decode step then runs on it as on any batch of sequences with one
// query token each.
#include <cuda.h>
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

// ---------------------------------------------------------------- scores
// One CTA scores kScorePages pages for up to 256 query rows, whole query tokens
// of H rows: D[page, row] = K Q^T on tcgen05, M = 128 pages, N = rows, over 576
// columns in nine stages of 64.  With the pages as TMEM lanes the maximum over
// the heads is one thread's own.  Page keys lie scattered through the pool, so
// threads gather them row by row (16-byte asynchronous copies, eight threads to
// a 128-byte piece of a row) into the swizzled layout that the tensor core
// reads; the queries come by TMA.  As many stages as shared memory holds are in
// flight: all nine up to 64 rows, four at 256.  Measured: 32 requests of up to 65k
// tokens, 2 queries x 128 heads 10.8 us, a wave of CTAs that each move 432 KB through
// four stages behind a chain of launch, length, table and first keys; plain
// arithmetic in place of tcgen05 took 49.  5 requests x 16 heads 5.1 us, the chain.
constexpr int kScoreThreads = 160;            // warps 0-3 gather and reduce, 4 drives
constexpr int kGatherThreads = 128;
constexpr int kScorePages = 128;
constexpr int kScoreABytes = kScorePages * 128;  // 128 pages x 64 columns: 16 KB
constexpr int kScoreRowsMax = 256;               // N of one MMA
constexpr int kScoreSmemMax = 224 * 1024;
constexpr int kStagesMin = 4;

__host__ __device__ constexpr int score_tokens(int T, int H) {
  return T < kScoreRowsMax / H ? T : kScoreRowsMax / H;
}
__host__ __device__ constexpr int score_stage_bytes(int rows) { return kScoreABytes + rows * 128; }
__host__ __device__ constexpr int score_stages(int rows) {
  const int n = kScoreSmemMax / score_stage_bytes(rows);
  return n < kBoxes ? n : kBoxes;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}
template <int kPending>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(kPending) : "memory");
}

__global__ void __launch_bounds__(kScoreThreads)
score_kernel(const __grid_constant__ CUtensorMap tm_q, const uint8_t* __restrict__ keys,
             const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
             int T, int H, int num_pages, int max_pages, float* __restrict__ scores,
             int32_t* __restrict__ status) {
  extern __shared__ uint8_t smem_raw[];
  __shared__ __align__(8) uint64_t full[kBoxes], free_[kBoxes], done;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh, timeout_sh;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int b = blockIdx.z, page0 = blockIdx.x * kScorePages;
  const int t0 = blockIdx.y * score_tokens(T, H), t1 = min(T, t0 + score_tokens(T, H));
  const int rows = (t1 - t0) * H;  // of this CTA; stages are sized for the most
  const int stages = score_stages(score_tokens(T, H) * H);
  const uint32_t base = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t stage_bytes = score_stage_bytes(score_tokens(T, H) * H);
  if (threadIdx.x == 0) {
    for (int i = 0; i < kBoxes; ++i) {
      mbar_init(smem_u32(&full[i]), kGatherThreads + 1);
      mbar_init(smem_u32(&free_[i]), 1);
    }
    mbar_init(smem_u32(&done), 1);
    abort_sh = timeout_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_q);
  }
  griddep_wait();
  griddep_launch_dependents();
  const int L = clamp_len(seq_lens[b], T, max_pages * kPage,
                          threadIdx.x == 0 && t0 == 0 && page0 == 0, status);
  // Query t sees (L - T + t + kPage) / kPage pages; the last one here the most.
  const int most = (L - T + t1 - 1 + kPage) / kPage;
  float* const out = scores + static_cast<size_t>(b) * T * max_pages;
  if (page0 >= most) {  // the whole CTA: nothing to compute
    const int j = page0 + threadIdx.x;
    if (threadIdx.x < kScorePages && j < max_pages)
      for (int t = t0; t < t1; ++t) out[static_cast<size_t>(t) * max_pages + j] = -INFINITY;
    return;
  }
  if (warp == 4) {
    tmem_alloc(smem_u32(&tmem_base_sh), kScoreRowsMax);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  bool ok = true;
  if (warp < 4) {
    // Thread (row group, chunk): 16-byte chunk `chunk` of rows rg, rg + 16, ...
    const int chunk = threadIdx.x & 7, rg = threadIdx.x >> 3;
    const uint8_t* src[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int j = page0 + rg + 16 * i;
      int p = j < most ? block_table[static_cast<size_t>(b) * max_pages + j] : 0;
      if (p < 0 || p >= num_pages) {
        record_status(status, MLA_STATUS_BOUNDS);
        p = 0;
      }
      src[i] = keys + static_cast<size_t>(p) * (kDqk * 2) + chunk * 16;
    }
    const uint32_t at = rg * 128 + ((chunk ^ (rg & 7)) << 4);  // (rows 16 apart share it)
    auto copy = [&](int k) {
      const uint32_t dst = base + (k % stages) * stage_bytes + at;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        cp_async16(dst + i * 16 * 128, src[i] + k * 128);
    };
#pragma unroll
    for (int k = 0; k < kBoxes; ++k) {
      if (k < stages) copy(k);
      cp_async_commit();
    }
    // Group k is complete once at most kBoxes - 1 - k younger ones are not.
    auto landed = [&](int k) {
      fence_proxy_async_smem();
      mbar_arrive(smem_u32(&full[k]));
    };
    cp_async_wait<8>(); landed(0);
    cp_async_wait<7>(); landed(1);
    cp_async_wait<6>(); landed(2);
    cp_async_wait<5>(); landed(3);  // (four stages at least)
    if (stages > 4) { cp_async_wait<4>(); landed(4); }
    if (stages > 5) { cp_async_wait<3>(); landed(5); }
    if (stages > 6) { cp_async_wait<2>(); landed(6); }
    if (stages > 7) { cp_async_wait<1>(); landed(7); }
    if (stages > 8) { cp_async_wait<0>(); landed(8); }
    // The others go out as their stage is free, and are waited for one behind
    // (with four stages the last five are a chain of loads else).
    for (int k = stages; k < kBoxes && ok; ++k) {
      ok = mbar_wait(smem_u32(&free_[k - stages]), 0, &abort_sh, &timeout_sh);
      if (!ok) break;
      copy(k);
      cp_async_commit();
      if (k > stages) {
        cp_async_wait<1>();
        landed(k - 1);
      }
    }
    cp_async_wait<0>();
    if (ok && stages < kBoxes) landed(kBoxes - 1);
    ok = ok && mbar_wait(smem_u32(&done), 0, &abort_sh, &timeout_sh);
    if (__all_sync(0xffffffffu, ok)) {
      tc_fence_after();
      const int j = page0 + threadIdx.x;
      for (int t = t0; t < t1; ++t) {
        float top = -INFINITY;
        for (int h = (t - t0) * H; h < (t - t0 + 1) * H; h += 16) {
          uint32_t v[16];
          tmem_ld_x16(tmem + (static_cast<uint32_t>(warp * 32) << 16) + h, v);
          tmem_wait_ld();
#pragma unroll
          for (int i = 0; i < 16; ++i) top = fmaxf(top, __uint_as_float(v[i]));
        }
        if (j < max_pages)
          out[static_cast<size_t>(t) * max_pages + j] =
              j < (L - T + t + kPage) / kPage ? top : -INFINITY;
      }
    }
  } else if (elect_one()) {
    // One thread brings the queries and issues the MMAs.
    const int row = (b * T + t0) * H;
    auto load = [&](int k) {
      const uint32_t dst = base + (k % stages) * stage_bytes + kScoreABytes;
      mbar_expect_tx(smem_u32(&full[k]), rows * 128);
      for (int r = 0; r < rows; r += H)
        tma_load_2d(dst + r * 128, &tm_q, k * kBoxCols, row + r, smem_u32(&full[k]));
    };
    int loaded = 0;
    for (; loaded < stages; ++loaded) load(loaded);
    const uint32_t idesc = idesc_bf16_f32(kScorePages, rows, false, false);
    for (int k = 0; k < kBoxes && ok; ++k) {
      ok = mbar_wait(smem_u32(&full[k]), 0, &abort_sh, &timeout_sh);
      if (!ok) break;
      tc_fence_after();
      const uint32_t a = base + (k % stages) * stage_bytes;
      const uint64_t da = sdesc_sw128(a, 16, 1024), dq = sdesc_sw128(a + kScoreABytes, 16, 1024);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) umma_bf16(tmem, da + 2 * kk, dq + 2 * kk, idesc, k | kk);
      umma_commit(smem_u32(&free_[k]));
      if (k + stages < kBoxes) {
        ok = mbar_wait(smem_u32(&free_[k]), 0, &abort_sh, &timeout_sh);
        if (ok) load(loaded++);
      }
    }
    umma_commit(smem_u32(&done));
    // Nothing is in flight when the CTA ends, after a timeout either.
    mbar_wait_drain(smem_u32(&done), 0, &timeout_sh);
    if (!ok)
      for (int k = 0; k < loaded; ++k) mbar_wait_drain(smem_u32(&full[k]), 0, &timeout_sh);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 4) {
    tc_fence_after();
    tmem_dealloc(tmem, kScoreRowsMax);
    if (lane == 0 && timeout_sh) record_status(status, MLA_STATUS_TIMEOUT);
  }
}

// ---------------------------------------------------------------- selection
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

// One CTA per query token: a radix selection of the key of the last page taken,
// eight bits at a time, then one ordered pass over the pages.  A line's keys are
// read once into shared memory where they fit (131k tokens).  A chain of at most
// four counts and a prefix sum per 256 pages: 80 queries of up to 512 pages, 33
// selected, 5.2 us; 8 of up to 256, 16 selected, 4.2.
constexpr int kSelKeys = 2048;

__global__ void __launch_bounds__(kSelThreads)
select_kernel(const float* __restrict__ scores, const int32_t* __restrict__ block_table,
              const int32_t* __restrict__ seq_lens, int T, int max_pages, int top_k,
              int keep_first, int keep_last, int32_t* __restrict__ sel_table,
              int32_t* __restrict__ sel_pages, int32_t* __restrict__ sel_lens,
              int32_t* __restrict__ status) {
  __shared__ int hist[4][256];
  __shared__ uint32_t keys_sh[kSelKeys];
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
  const bool held = seen <= kSelKeys;
  auto key = [&](int j) { return held ? keys_sh[j] : order_key(s[j]); };
  if (seen > top_k) {
    need = top_k - keep_first - keep_last;
    for (int i = threadIdx.x; i < 4 * 256; i += kSelThreads) (&hist[0][0])[i] = 0;
    if (held)
      for (int j = threadIdx.x; j < seen; j += kSelThreads) keys_sh[j] = order_key(s[j]);
    __syncthreads();
    uint32_t mask = 0;
    for (int shift = 24; shift >= 0 && need > 0; shift -= 8) {
      int* const h = hist[shift >> 3];
      for (int j = keep_first + threadIdx.x; j < seen - keep_last; j += kSelThreads) {
        const uint32_t u = key(j);
        if ((u & mask) == last_key) atomicAdd(&h[(u >> shift) & 255], 1);
      }
      __syncthreads();
      if (threadIdx.x < 32) {
        // The bin, from the top, in which the count of better keys passes
        // `need`: lane i owns bins 255 - 8 i downwards.
        const int lane = threadIdx.x;
        int own = 0;
#pragma unroll
        for (int k = 0; k < 8; ++k) own += h[255 - 8 * lane - k];
        int upto = own;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
          const int v = __shfl_up_sync(0xffffffffu, upto, o);
          if (lane >= o) upto += v;
        }
        const int before = upto - own;
        if (before < need && need <= upto) {
          int left = need - before, bin = 255 - 8 * lane;
          while (left > h[bin]) left -= h[bin--];
          prefix_sh = last_key | (static_cast<uint32_t>(bin) << shift);
          need_sh = left;
        }
      }
      __syncthreads();
      last_key = prefix_sh;
      need = need_sh;
      mask |= 255u << shift;
    }
    if (top_k == keep_first + keep_last) last_key = 0xffffffffu;  // none by score
  }
  int done = 0, ties = 0;  // selected so far; pages with last_key so far
  for (int j0 = 0; j0 < seen; j0 += kSelThreads) {
    const int j = j0 + threadIdx.x;
    bool take = j < seen, tie = false;
    if (seen > top_k && take && j >= keep_first && j < seen - keep_last) {
      const uint32_t u = key(j);
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

cudaError_t launch_score(const CUtensorMap& tm_q, const void* page_keys,
                         const int32_t* block_table, const int32_t* seq_lens, int B, int T, int H,
                         int num_pages, int max_pages, float* scores, int32_t* status,
                         cudaStream_t st) {
  const int tokens = score_tokens(T, H), rows = tokens * H;
  const int smem = 1024 + score_stages(rows) * score_stage_bytes(rows);
  static_assert(score_stages(kScoreRowsMax) >= kStagesMin, "the gather waits for four stages");
  // The attribute is the kernel's, not the launch's: always the same value, so
  // that calls of other shapes on other threads do not take it away.
  const cudaError_t e = cudaFuncSetAttribute(
      score_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kScoreSmemMax);
  if (e != cudaSuccess) return e;
  const dim3 grid((max_pages + kScorePages - 1) / kScorePages, (T + tokens - 1) / tokens, B);
  return launch_pdl(score_kernel, grid, dim3(kScoreThreads), smem, st, tm_q,
                    static_cast<const uint8_t*>(page_keys), block_table, seq_lens, T, H,
                    num_pages, max_pages, scores, status);
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

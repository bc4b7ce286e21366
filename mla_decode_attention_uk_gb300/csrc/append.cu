// append.cu -- new tokens into the 8-bit latent cache, and the pages' mean keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"

namespace mla {

namespace {

constexpr int kAppThreads = 512;
constexpr int kChunks = kDqk / 8;  // 16-byte chunks of a bf16 row: 72 (8-byte chunks of codes)

// The new tokens of one sequence: positions [first, len).  False (and an error
// on record, if `report`) if its lengths are out of range: the sequence is then
// left alone.
struct NewTokens {
  int first, len;
  __device__ bool load(const int32_t* seq_lens, const int32_t* new_lens, int max_new, int cap,
                       int b, bool report, int32_t* status) {
    len = seq_lens[b];
    const int n = new_lens ? new_lens[b] : max_new;
    first = len - n;
    if (len < 0 || len > cap || n < 0 || n > max_new || first < 0) {
      if (report) record_status(status, MLA_STATUS_BOUNDS);
      return false;
    }
    return n > 0;
  }
  __device__ int pages() const { return (len - 1) / kPage - first / kPage + 1; }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// Largest |x| of 8 packed bf16 values and `top`, NaN ignored.
__device__ __forceinline__ __nv_bfloat162 absmax8(__nv_bfloat162 top, const uint4& v) {
  top = __hmax2(__hmax2(top, __habs2(as_bf162(v.x))), __habs2(as_bf162(v.y)));
  return __hmax2(__hmax2(top, __habs2(as_bf162(v.z))), __habs2(as_bf162(v.w)));
}
// The same over finite values.
__device__ __forceinline__ float finite_absmax8(float top, const uint4& v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    const float a = fabsf(bf16_lo(w[k])), b = fabsf(bf16_hi(w[k]));
    top = fmaxf(top, fmaxf(a < INFINITY ? a : 0.0f, b < INFINITY ? b : 0.0f));
  }
  return top;
}
// 8 bf16 values times `inv` (a power of two: exact but for what vanishes) to codes.
__device__ __forceinline__ uint2 codes8(const uint4& v, __nv_bfloat162 inv) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  uint32_t c[4];
#pragma unroll
  for (int k = 0; k < 4; ++k)
    c[k] = __nv_cvt_float2_to_fp8x2(__bfloat1622float2(__hmul2(as_bf162(w[k]), inv)),
                                    __NV_SATFINITE, __NV_E4M3);
  return make_uint2(c[0] | (c[1] << 16), c[2] | (c[3] << 16));
}

// Maximum of `top` over the CTA, the same to all.
__device__ __forceinline__ float block_max(float top, float* warp_top) {
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kAppThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
  return top;
}

// The new rows of a page are contiguous: one bulk copy brings them into shared
// memory, from where they are read twice, for their maximum, hence the scale, and
// for the codes.
constexpr int kAppSmem = kPage * kDqk * 2;  // 73,728: three CTAs per SM

struct AppendParams {
  const uint4* rows;
  int max_new;
  const int32_t* new_lens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, num_pages, max_pages;
  uint8_t* kv8;
  float* kv_scale;
  int32_t* status;
};

struct AppendShared {
  float warp_top[kAppThreads / 32];
  alignas(8) uint64_t landed;
  int abort, timeout;
  int warp_sum[kAppThreads / 32];
  int b, first, len, page;  // the page in work: sequence, its new tokens, logical page
};

// Page `logical` of sequence b, whose new tokens are nt; `phase`: of sh.landed.
// False after a timeout.
__device__ bool append_page(const AppendParams& P, AppendShared& sh, uint4* rows_sh, int b,
                            const NewTokens& nt, int logical, uint32_t phase) {
  const int page = P.block_table[static_cast<size_t>(b) * P.max_pages + logical];
  const bool in_pool = page >= 0 && page < P.num_pages;
  if (!in_pool && threadIdx.x == 0) record_status(P.status, MLA_STATUS_BOUNDS);
  // Rows [r0, r1) of the page are new.
  const int r0 = max(nt.first - logical * kPage, 0);
  const int r1 = min(nt.len - logical * kPage, kPage);
  const int n = (r1 - r0) * kChunks;
  if (threadIdx.x == 0) {
    fence_proxy_async_smem();  // the last page's rows have been read
    mbar_expect_tx(smem_u32(&sh.landed), n * 16);
    bulk_load(smem_u32(rows_sh),
              P.rows + (static_cast<size_t>(b) * P.max_new + (logical * kPage + r0 - nt.first)) *
                           kChunks,
              n * 16, smem_u32(&sh.landed));
  }
  // Read before the barrier below: one thread replaces it at the end.
  float old = r0 > 0 && in_pool ? P.kv_scale[page] : 1.0f;
  if (!scale_in_range(old)) {
    if (threadIdx.x == 0) record_status(P.status, MLA_STATUS_BOUNDS);
    old = 1.0f;
  }
  // One warp polls, the others sleep at the barrier (sixteen polling warps take
  // the issue slots of the CTAs that have their rows).
  bool ok = true;
  if (threadIdx.x < 32) ok = mbar_wait(smem_u32(&sh.landed), phase, &sh.abort, &sh.timeout);
  if (!__syncthreads_and(ok)) {
    if (threadIdx.x == 0) {
      record_status(P.status, MLA_STATUS_TIMEOUT);
      mbar_wait_drain(smem_u32(&sh.landed), phase, &sh.timeout);
    }
    __syncthreads();
    return false;
  }
  __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
  for (int i = threadIdx.x; i < n; i += kAppThreads) most = absmax8(most, rows_sh[i]);
  float top = block_max(fmaxf(__low2float(most), __high2float(most)), sh.warp_top);
  if (top == INFINITY) {  // rare: once more, without the infinities
    __syncthreads();
    top = 0.0f;
    for (int i = threadIdx.x; i < n; i += kAppThreads) top = finite_absmax8(top, rows_sh[i]);
    top = block_max(top, sh.warp_top);
  }
  if (!in_pool) return true;
  float scale = exp2_int(page_scale_exp(top));
  if (r0 > 0) scale = fmaxf(scale, next_power_of_two(old));
  uint2* const dst = reinterpret_cast<uint2*>(P.kv8 + static_cast<size_t>(page) * kPageBytes8);
  const __nv_bfloat162 inv = __float2bfloat162_rn(1.0f / scale);
#pragma unroll 3
  for (int i = threadIdx.x; i < n; i += kAppThreads)
    dst[r0 * kChunks + i] = codes8(rows_sh[i], inv);
  if (threadIdx.x == 0) P.kv_scale[page] = scale;
  // Rows that stay: cleared in a page that starts here, re-coded if the scale
  // grew.
  if (r0 > 0 && scale == old) return true;
  const float ratio = old / scale;
  for (int i = threadIdx.x; i < kPage * kChunks; i += kAppThreads) {
    if (i >= r0 * kChunks && i < r1 * kChunks) continue;
    uint2 c = make_uint2(0u, 0u);
    if (r0 > 0) {
      c = dst[i];
      uint32_t w[2] = {c.x, c.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 p = e4m3x2_to_float2(w[k]), q = e4m3x2_to_float2(w[k] >> 16);
        w[k] = e4m3x4(p.x * ratio, p.y * ratio, q.x * ratio, q.y * ratio);
      }
      c = make_uint2(w[0], w[1]);
    }
    dst[i] = c;
  }
  return true;
}

__device__ __forceinline__ void append_begin(AppendShared& sh) {
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&sh.landed), 1);
    sh.abort = sh.timeout = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
}

// A few new tokens per sequence: one CTA per sequence and page that they can
// touch.
__global__ void __launch_bounds__(kAppThreads)
append_few_kernel(AppendParams P) {
  extern __shared__ __align__(128) uint4 rows_sh[];
  __shared__ AppendShared sh;
  append_begin(sh);
  NewTokens nt;
  if (!nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, blockIdx.y,
               threadIdx.x == 0, P.status))
    return;
  if (blockIdx.x < nt.pages())
    append_page(P, sh, rows_sh, blockIdx.y, nt, nt.first / kPage + blockIdx.x, 0);
}

// Prompts: a grid that fills the SMs shares the pages of all sequences out, page
// f to CTA f mod grid (with a CTA for every page that a sequence could have, the
// empty ones of ragged prompts took a third of the time).  The CTA counts the
// pages of 512 sequences at a time, one per thread, and finds its own among them.
__global__ void __launch_bounds__(kAppThreads, 3)
append_pages_kernel(AppendParams P) {
  extern __shared__ __align__(128) uint4 rows_sh[];
  __shared__ AppendShared sh;
  append_begin(sh);
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  long long f = blockIdx.x, base = 0;
  uint32_t phase = 0;
  for (int b0 = 0; b0 < P.B; b0 += kAppThreads) {
    const int b = b0 + threadIdx.x;
    NewTokens nt;
    int n = 0;
    if (b < P.B && nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, b,
                           blockIdx.x == 0, P.status))
      n = nt.pages();
    int upto = n;
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, upto, o);
      if (lane >= o) upto += v;
    }
    if (lane == 31) sh.warp_sum[warp] = upto;
    __syncthreads();
    // (At most 512 sequences of 2^24 pages: the sum may pass 32 bits.)
    long long before = base, all = base;
    for (int w = 0; w < kAppThreads / 32; ++w) {
      before += w < warp ? sh.warp_sum[w] : 0;
      all += sh.warp_sum[w];
    }
    before += upto - n;
    for (; f < all; f += gridDim.x, phase ^= 1) {
      if (f >= before && f < before + n) {
        sh.b = b;
        sh.first = nt.first;
        sh.len = nt.len;
        sh.page = nt.first / kPage + static_cast<int>(f - before);
      }
      __syncthreads();
      NewTokens mine;
      mine.first = sh.first;
      mine.len = sh.len;
      if (!append_page(P, sh, rows_sh, sh.b, mine, sh.page, phase)) return;
      __syncthreads();  // before the next page's rows and place
    }
    base = all;
    __syncthreads();
  }
}

constexpr int kKeyThreads = 288;

// One CTA per (sequence, page that holds new tokens): the mean of its filled
// rows.  Thread t sums columns 8 (t mod 72) .. + 7 over rows t / 72, + 4, ...
template <bool kFp8>
__global__ void __launch_bounds__(kKeyThreads)
page_keys_kernel(const uint8_t* __restrict__ cache, const float* __restrict__ kv_scale,
                 const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
                 int max_new, const int32_t* __restrict__ new_lens, int num_pages, int max_pages,
                 __nv_bfloat16* __restrict__ keys, int32_t* __restrict__ status) {
  __shared__ float part[4][kDqk];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  NewTokens nt;
  if (!nt.load(seq_lens, new_lens, max_new, max_pages * kPage, b, threadIdx.x == 0, status))
    return;
  const int logical = nt.first / kPage + blockIdx.x;
  if (logical * kPage >= nt.len) return;
  const int page = block_table[static_cast<size_t>(b) * max_pages + logical];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
    return;
  }
  const int filled = min(nt.len - logical * kPage, kPage);
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  float s[8] = {};
#pragma unroll 4
  for (int r = r0; r < filled; r += 4) {
    if constexpr (kFp8) {
      const uint2 v = *reinterpret_cast<const uint2*>(
          cache + static_cast<size_t>(page) * kPageBytes8 + r * kDqk + c * 8);
      const float2 x0 = e4m3x2_to_float2(v.x), x1 = e4m3x2_to_float2(v.x >> 16);
      const float2 x2 = e4m3x2_to_float2(v.y), x3 = e4m3x2_to_float2(v.y >> 16);
      s[0] += x0.x; s[1] += x0.y; s[2] += x1.x; s[3] += x1.y;
      s[4] += x2.x; s[5] += x2.y; s[6] += x3.x; s[7] += x3.y;
    } else {
      const uint4 v = *reinterpret_cast<const uint4*>(
          cache + (static_cast<size_t>(page) * kPage + r) * (kDqk * 2) + c * 16);
      s[0] += bf16_lo(v.x); s[1] += bf16_hi(v.x); s[2] += bf16_lo(v.y); s[3] += bf16_hi(v.y);
      s[4] += bf16_lo(v.z); s[5] += bf16_hi(v.z); s[6] += bf16_lo(v.w); s[7] += bf16_hi(v.w);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) part[r0][c * 8 + k] = s[k];
  __syncthreads();
  float scale = 1.0f;
  if constexpr (kFp8) {
    scale = kv_scale[page];
    if (!scale_in_range(scale)) {
      if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
      scale = 1.0f;
    }
  }
  const float mul = scale / static_cast<float>(filled);
  const int k = threadIdx.x * 2;
  const float x = ((part[0][k] + part[1][k]) + (part[2][k] + part[3][k])) * mul;
  const float y = ((part[0][k + 1] + part[1][k + 1]) + (part[2][k + 1] + part[3][k + 1])) * mul;
  *reinterpret_cast<uint32_t*>(keys + static_cast<size_t>(page) * kDqk + k) = pack_bf16x2(x, y);
}

}  // namespace

// Up to so many new tokens a sequence, a CTA for each of the two pages that they
// can touch; their rows fit the shared memory that needs no opt-in.
constexpr int kFewTokens = 32;

// Pages that max_new consecutive tokens can touch.
static int touched_pages(int max_new, int max_pages) {
  const int most = (max_new + kPage - 2) / kPage + 1;
  return most < max_pages ? most : max_pages;
}

cudaError_t launch_append(const void* rows, int max_new, const int32_t* new_lens,
                          const int32_t* block_table, const int32_t* seq_lens, int B,
                          int num_pages, int max_pages, uint8_t* kv8, float* kv_scale,
                          int32_t* status, int sm_count, cudaStream_t st) {
  const AppendParams P{static_cast<const uint4*>(rows), max_new, new_lens, block_table, seq_lens,
                       B, num_pages, max_pages, kv8, kv_scale, status};
  if (max_new <= kFewTokens)
    return launch_pdl(append_few_kernel, dim3(touched_pages(max_new, max_pages), B),
                      dim3(kAppThreads), max_new * kDqk * 2, st, P);
  const cudaError_t e = cudaFuncSetAttribute(
      append_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kAppSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(append_pages_kernel, dim3(3 * sm_count), dim3(kAppThreads), kAppSmem, st, P);
}

cudaError_t launch_page_keys(const void* cache, const float* kv_scale,
                             const int32_t* block_table, const int32_t* seq_lens, int max_new,
                             const int32_t* new_lens, int B, int num_pages, int max_pages,
                             __nv_bfloat16* keys, int32_t* status, cudaStream_t st) {
  auto kern = kv_scale ? page_keys_kernel<true> : page_keys_kernel<false>;
  return launch_pdl(kern, dim3(touched_pages(max_new, max_pages), B), dim3(kKeyThreads), 0, st,
                    static_cast<const uint8_t*>(cache), kv_scale, block_table, seq_lens, max_new,
                    new_lens, num_pages, max_pages, keys, status);
}

}  // namespace mla

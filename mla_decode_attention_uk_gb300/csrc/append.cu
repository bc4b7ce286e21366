// append.cu -- new tokens into the 8-bit latent cache, and the pages' mean keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"

namespace mla {

namespace {

constexpr int kAppThreads = 256;
constexpr int kChunks = kDqk / 8;  // 16-byte chunks of a bf16 row: 72 (8-byte chunks of codes)

// The new tokens of one sequence: positions [first, len).  False (and an error
// on record) if its lengths are out of range: the sequence is then left alone.
struct NewTokens {
  int first, len;
  __device__ bool load(const int32_t* seq_lens, const int32_t* new_lens, int max_new, int cap,
                       int b, int32_t* status) {
    len = seq_lens[b];
    const int n = new_lens ? new_lens[b] : max_new;
    first = len - n;
    if (len < 0 || len > cap || n < 0 || n > max_new || first < 0) {
      if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
      return false;
    }
    return true;
  }
};

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

// |x| of two packed bf16 values, their finite maximum folded into `top`.
__device__ __forceinline__ float finite_max2(float top, uint32_t w) {
  const uint32_t a = w & 0x7fffu, b = (w >> 16) & 0x7fffu;
  const uint32_t m = max(a < 0x7f80u ? a : 0u, b < 0x7f80u ? b : 0u);
  return fmaxf(top, __uint_as_float(m << 16));
}

// One CTA per (sequence, page that receives new tokens).  The new rows are read
// once, into registers (a full page: 18 16-byte loads per thread, all in
// flight), so that their maximum, hence the scale, is known before any code is
// formed.
constexpr int kPerThread = kPage * kChunks / kAppThreads;  // 18

__global__ void __launch_bounds__(kAppThreads, 2)
append_kernel(const uint4* __restrict__ rows, int max_new, const int32_t* __restrict__ new_lens,
              const int32_t* __restrict__ block_table, const int32_t* __restrict__ seq_lens,
              int num_pages, int max_pages, uint8_t* __restrict__ kv8,
              float* __restrict__ kv_scale, int32_t* __restrict__ status) {
  __shared__ float warp_top[kAppThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int b = blockIdx.y;
  NewTokens nt;
  if (!nt.load(seq_lens, new_lens, max_new, max_pages * kPage, b, status)) return;
  const int logical = nt.first / kPage + blockIdx.x;
  if (logical * kPage >= nt.len || nt.first == nt.len) return;
  const int page = block_table[static_cast<size_t>(b) * max_pages + logical];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
    return;
  }
  // Rows [r0, r1) of the page are new.
  const int r0 = max(nt.first - logical * kPage, 0);
  const int r1 = min(nt.len - logical * kPage, kPage);
  const int n = (r1 - r0) * kChunks;
  const uint4* src =
      rows + (static_cast<size_t>(b) * max_new + (logical * kPage + r0 - nt.first)) * kChunks;
  uint4 v[kPerThread];
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int i = threadIdx.x + k * kAppThreads;
    v[k] = i < n ? src[i] : make_uint4(0u, 0u, 0u, 0u);
  }
  // Read before the barrier below: one thread replaces it at the end.
  const float old = r0 > 0 ? kv_scale[page] : 0.0f;
  float top = 0.0f;
#pragma unroll
  for (int k = 0; k < kPerThread; ++k)
    top = finite_max2(finite_max2(finite_max2(finite_max2(top, v[k].x), v[k].y), v[k].z), v[k].w);
  for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
  if ((threadIdx.x & 31) == 0) warp_top[threadIdx.x >> 5] = top;
  __syncthreads();
  for (int w = 0; w < kAppThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
  float scale = exp2_int(page_scale_exp(top));
  if (r0 > 0) scale = fmaxf(scale, old);
  uint2* const dst = reinterpret_cast<uint2*>(kv8 + static_cast<size_t>(page) * kPageBytes8);
  const float inv = 1.0f / scale;  // exact: a power of two
#pragma unroll
  for (int k = 0; k < kPerThread; ++k) {
    const int i = threadIdx.x + k * kAppThreads;
    if (i < n)
      dst[r0 * kChunks + i] =
          make_uint2(e4m3x4(bf16_lo(v[k].x) * inv, bf16_hi(v[k].x) * inv, bf16_lo(v[k].y) * inv,
                            bf16_hi(v[k].y) * inv),
                     e4m3x4(bf16_lo(v[k].z) * inv, bf16_hi(v[k].z) * inv, bf16_lo(v[k].w) * inv,
                            bf16_hi(v[k].w) * inv));
  }
  if (threadIdx.x == 0) kv_scale[page] = scale;
  // Rows that stay: cleared in a page that starts here, re-coded if the scale
  // grew.
  if (r0 > 0 && scale == old) return;
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
  if (!nt.load(seq_lens, new_lens, max_new, max_pages * kPage, b, status)) return;
  const int logical = nt.first / kPage + blockIdx.x;
  if (logical * kPage >= nt.len || nt.first == nt.len) return;
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
  const float mul = (kFp8 ? kv_scale[page] : 1.0f) / static_cast<float>(filled);
  const int k = threadIdx.x * 2;
  const float x = ((part[0][k] + part[1][k]) + (part[2][k] + part[3][k])) * mul;
  const float y = ((part[0][k + 1] + part[1][k + 1]) + (part[2][k + 1] + part[3][k + 1])) * mul;
  *reinterpret_cast<uint32_t*>(keys + static_cast<size_t>(page) * kDqk + k) = pack_bf16x2(x, y);
}

}  // namespace

// Pages that max_new consecutive tokens can touch.
static int touched_pages(int max_new, int max_pages) {
  const int most = (max_new + kPage - 2) / kPage + 1;
  return most < max_pages ? most : max_pages;
}

cudaError_t launch_append(const void* rows, int max_new, const int32_t* new_lens,
                          const int32_t* block_table, const int32_t* seq_lens, int B,
                          int num_pages, int max_pages, uint8_t* kv8, float* kv_scale,
                          int32_t* status, cudaStream_t st) {
  return launch_pdl(append_kernel, dim3(touched_pages(max_new, max_pages), B), dim3(kAppThreads),
                    0, st, static_cast<const uint4*>(rows), max_new, new_lens, block_table,
                    seq_lens, num_pages, max_pages, kv8, kv_scale, status);
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

// append.cu -- new tokens into the 8-bit latent cache, and the pages' mean keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"

namespace mla {

namespace {

constexpr int kAppThreads = 384;  // that convert a page
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

// x * y rounded to odd: the nearest fp32 value with the last bit set where the
// product is between two, so that rounding it on to a code rounds the product
// itself (a product next to a tie of E4M3 would be rounded to the tie first).
__device__ __forceinline__ float mul_odd(float x, float y) {
  const float p = x * y, rest = fmaf(x, y, -p);
  const int u = __float_as_int(p);
  const bool even = rest != 0.0f && !(u & 1);
  return __int_as_float(even ? ((rest > 0.0f) == (p > 0.0f) ? u + 1 : u - 1) : u);
}

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

// A page to fill: its sequence, the new tokens there, and which of its pages.
struct Place {
  int b, first, len, logical;
  // Rows [r0, r1) of the page are new.
  __device__ int r0() const { return max(first - logical * kPage, 0); }
  __device__ int r1() const { return min(len - logical * kPage, kPage); }
};

// kAppThreads threads that fill a page together.
struct Group {
  uint32_t bar;     // their named barrier
  int tid;
  float* warp_top;  // [kAppThreads / 32]
  __device__ void sync() const { named_bar_sync(bar, kAppThreads); }
  // Maximum of `top` over them, the same to all.
  __device__ float max_of(float top) const {
    for (int o = 16; o; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((tid & 31) == 0) warp_top[tid >> 5] = top;
    sync();
    for (int w = 0; w < kAppThreads / 32; ++w) top = fmaxf(top, warp_top[w]);
    return top;
  }
};

// The new rows of a page are contiguous: one bulk copy (of one thread) brings them
// into shared memory, and threads take them from there.
constexpr int kRowsBytes = kPage * kDqk * 2;  // 73,728

__device__ __forceinline__ void load_rows(const AppendParams& P, const Place& at, uint4* rows_sh,
                                          uint64_t* landed) {
  const int r0 = at.r0(), bytes = (at.r1() - r0) * kDqk * 2;
  fence_proxy_async_smem();  // the rows that were there have been read
  mbar_expect_tx(smem_u32(landed), bytes);
  bulk_load(smem_u32(rows_sh),
            P.rows + (static_cast<size_t>(at.b) * P.max_new +
                      (at.logical * kPage + r0 - at.first)) * kChunks,
            bytes, smem_u32(landed));
}

// Whether the rows have landed, false after a timeout.  One warp polls, the others
// sleep at the barrier (twelve polling warps take the issue slots of those that
// have their rows).
__device__ __forceinline__ bool wait_rows(const Group& grp, uint64_t* landed, uint32_t phase,
                                          int* abort, int* timeout) {
  bool bad = false;
  if (grp.tid < 32) bad = !mbar_wait(smem_u32(landed), phase, abort, timeout);
  return !bar_any(grp.bar, kAppThreads, bad);
}

// The page and, where tokens stay, its scale.
struct Target {
  int page;
  float old;
  bool in_pool;
  __device__ Target(const AppendParams& P, const Place& at, bool report) {
    page = P.block_table[static_cast<size_t>(at.b) * P.max_pages + at.logical];
    in_pool = page >= 0 && page < P.num_pages;
    old = at.r0() > 0 && in_pool ? P.kv_scale[page] : 1.0f;
    const bool good = scale_in_range(old);
    if (report && !(in_pool && good)) record_status(P.status, MLA_STATUS_BOUNDS);
    if (!good) old = 1.0f;
  }
};

// Fills a page from its new rows, which a thread holds in registers between their
// maximum and the codes; `taken` is called once all have theirs.  kFew skips what
// a few rows do not fill, at a price for whole pages (14 -> 15.5 us).  (Every thread
// has its Target before the first barrier here; one thread replaces the scale
// behind it.)
template <bool kFew, typename Taken>
__device__ __forceinline__ void fill_page(const AppendParams& P, const Group& grp,
                                          const Place& at, const Target& to,
                                          const uint4* rows_sh, const Taken& taken) {
  constexpr int kHeld = kPage * kChunks / kAppThreads;
  static_assert(kHeld * kAppThreads == kPage * kChunks, "a page is whole passes");
  const int r0 = at.r0(), r1 = at.r1(), n = (r1 - r0) * kChunks;
  uint4 x[kHeld];
  __nv_bfloat162 most = __float2bfloat162_rn(0.0f);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = grp.tid + k * kAppThreads;
    if (kFew && k * kAppThreads >= n) break;
    x[k] = make_uint4(0u, 0u, 0u, 0u);
    if (i < n) x[k] = rows_sh[i];
    most = absmax8(most, x[k]);
  }
  float top = grp.max_of(fmaxf(__low2float(most), __high2float(most)));
  taken();
  if (top == INFINITY) {  // rare: once more, without the infinities
    grp.sync();
    top = 0.0f;
#pragma unroll
    for (int k = 0; k < kHeld; ++k)
      if (!kFew || k * kAppThreads < n) top = finite_absmax8(top, x[k]);
    top = grp.max_of(top);
  }
  if (!to.in_pool) return;
  float scale = exp2_int(page_scale_exp(top));
  if (r0 > 0) scale = fmaxf(scale, next_power_of_two(to.old));
  uint2* const dst = reinterpret_cast<uint2*>(P.kv8 + static_cast<size_t>(to.page) * kPageBytes8);
  const __nv_bfloat162 inv = __float2bfloat162_rn(1.0f / scale);
#pragma unroll
  for (int k = 0; k < kHeld; ++k) {
    const int i = grp.tid + k * kAppThreads;
    if (kFew && k * kAppThreads >= n) break;
    if (i < n) dst[r0 * kChunks + i] = codes8(x[k], inv);
  }
  if (grp.tid == 0) P.kv_scale[to.page] = scale;
  // Rows that stay: cleared in a page that starts here, re-coded if the scale
  // grew.
  if (r0 > 0 && scale == to.old) return;
  const float ratio = to.old / scale;
  for (int i = grp.tid; i < kPage * kChunks; i += kAppThreads) {
    if (i >= r0 * kChunks && i < r1 * kChunks) continue;
    uint2 c = make_uint2(0u, 0u);
    if (r0 > 0) {
      c = dst[i];
      uint32_t w[2] = {c.x, c.y};
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const float2 p = e4m3x2_to_float2(w[k]), q = e4m3x2_to_float2(w[k] >> 16);
        w[k] = e4m3x4(mul_odd(p.x, ratio), mul_odd(p.y, ratio), mul_odd(q.x, ratio),
                      mul_odd(q.y, ratio));
      }
      c = make_uint2(w[0], w[1]);
    }
    dst[i] = c;
  }
}

// A few new tokens per sequence: one CTA per sequence and page that they can
// touch.  One token for each of 128 sequences: 2.6 us in a graph, a launch and a
// chain of three reads (lengths, block table, scale) beside the row's.
__global__ void __launch_bounds__(kAppThreads)
append_few_kernel(AppendParams P) {
  extern __shared__ __align__(128) uint4 rows_sh[];
  __shared__ float warp_top[kAppThreads / 32];
  __shared__ alignas(8) uint64_t landed;
  __shared__ int abort_sh, timeout_sh;
  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&landed), 1);
    abort_sh = timeout_sh = 0;
    fence_mbar_init();
  }
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  NewTokens nt;
  if (!nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, blockIdx.y,
               threadIdx.x == 0, P.status) ||
      blockIdx.x >= nt.pages())
    return;
  const Place at{static_cast<int>(blockIdx.y), nt.first, nt.len,
                 nt.first / kPage + static_cast<int>(blockIdx.x)};
  if (threadIdx.x == 0) load_rows(P, at, rows_sh, &landed);
  const Group grp{1, static_cast<int>(threadIdx.x), warp_top};
  const Target to(P, at, threadIdx.x == 0);
  if (wait_rows(grp, &landed, 0, &abort_sh, &timeout_sh)) {
    fill_page<true>(P, grp, at, to, rows_sh, [] {});
  } else if (threadIdx.x == 0) {
    record_status(P.status, MLA_STATUS_TIMEOUT);
    mbar_wait_drain(smem_u32(&landed), 0, &timeout_sh);
  }
}

// Prompts: one CTA per SM, page f of all sequences to CTA f mod grid (with a CTA
// for every page that a sequence could have, the empty ones of ragged prompts took
// a third of the time).  The CTA's pages pass through a ring of three buffers, and
// two groups of threads take turns at filling them, so that loads and conversions
// overlap: 13 prompts of 512 to 8190 tokens 14.5 us, 4.5 TB/s; three CTAs of one
// buffer took 16.2, and two passes over shared memory in place of registers 16.
// What is left is mostly the start (lengths, sums, first loads: 2 us with nothing in
// flight) and the last pages' conversion.
constexpr int kRing = 3;
constexpr int kGroups = 2;
constexpr int kBars = kRing * kGroups;  // a barrier is always the same group's, whose
                                        // waits see each of its phases
constexpr int kPlanSeqs = 512;          // sequences looked at together
constexpr int kPagesThreads = kGroups * kAppThreads;

struct AppendShared {
  float warp_top[kGroups][kAppThreads / 32];
  alignas(8) uint64_t landed[kBars];
  Place place[kBars];
  int issued[kBars];
  int abort, timeout;
  int warp_sum[kPlanSeqs / 32];
  int first[kPlanSeqs], len[kPlanSeqs];
  long long upto[kPlanSeqs];  // pages up to and with the sequence's
};

__global__ void __launch_bounds__(kPagesThreads, 1)
append_pages_kernel(AppendParams P) {
  extern __shared__ __align__(128) uint4 ring_sh[];
  __shared__ AppendShared sh;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  if (tid == 0) {
    for (int i = 0; i < kBars; ++i) {
      mbar_init(smem_u32(&sh.landed[i]), 1);
      sh.issued[i] = 0;
    }
    sh.abort = sh.timeout = 0;
    fence_mbar_init();
  }
  griddep_wait();
  griddep_launch_dependents();
  const int gid = tid / kAppThreads;
  const Group grp{1u + gid, tid % kAppThreads, sh.warp_top[gid]};
  auto rows_of = [&](int k) { return ring_sh + (k % kRing) * (kRowsBytes / 16); };
  long long f = blockIdx.x, base = 0;  // this CTA's next page; pages before b0
  int k = 0;                           // this CTA's pages so far
  bool failed = false;
  for (int b0 = 0; b0 < P.B; b0 += kPlanSeqs) {
    // Pages per sequence, counted by a thread each.
    NewTokens nt{0, 0};
    int n = 0;
    if (tid < kPlanSeqs) {
      if (b0 + tid < P.B && nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage,
                                    b0 + tid, blockIdx.x == 0, P.status))
        n = nt.pages();
      int upto = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += v;
      }
      if (lane == 31) sh.warp_sum[warp] = upto;
      n = upto;
      sh.first[tid] = nt.first;
      sh.len[tid] = nt.len;
    }
    __syncthreads();
    if (tid < kPlanSeqs) {
      // (512 sequences of 2^25 pages: the sum may pass 32 bits.)
      long long upto = base + n;
      for (int w = 0; w < warp; ++w) upto += sh.warp_sum[w];
      sh.upto[tid] = upto;
    }
    __syncthreads();
    base = sh.upto[kPlanSeqs - 1];
    const int mine = f < base ? static_cast<int>((base - 1 - f) / gridDim.x) + 1 : 0;
    // One thread looks up the CTA's page i of these and starts its load.
    auto issue = [&](int i) {
      const long long page = f + static_cast<long long>(i) * gridDim.x;
      int lo = 0;  // the first sequence with upto > page
      for (int step = kPlanSeqs / 2; step; step >>= 1)
        if (sh.upto[lo + step - 1] <= page) lo += step;
      const int bar = (k + i) % kBars;
      const Place at{b0 + lo, sh.first[lo], sh.len[lo],
                     (sh.len[lo] - 1) / kPage - static_cast<int>(sh.upto[lo] - 1 - page)};
      sh.place[bar] = at;
      ++sh.issued[bar];
      load_rows(P, at, rows_of(k + i), &sh.landed[bar]);
    };
    if (tid == 0)
#pragma unroll 1
      for (int i = 0; i < min(kRing, mine); ++i) issue(i);
    for (int i = (k + gid) % kGroups; i < mine; i += kGroups) {
      const int bar = (k + i) % kBars;
      failed = !wait_rows(grp, &sh.landed[bar], ((k + i) / kBars) & 1, &sh.abort, &sh.timeout);
      if (failed) break;
      const Place at = sh.place[bar];  // (written before its load was issued)
      fill_page<false>(P, grp, at, Target(P, at, grp.tid == 0), rows_of(k + i), [&] {
        if (grp.tid == kAppThreads - 32 && i + kRing < mine) issue(i + kRing);
      });
    }
    k += mine;
    f += static_cast<long long>(mine) * gridDim.x;
    if (__syncthreads_or(failed)) {  // every copy lands before the CTA exits
      if (tid == 0) {
        record_status(P.status, MLA_STATUS_TIMEOUT);
        for (int q = 0; q < kBars; ++q)
          if (sh.issued[q] > 0)
            mbar_wait_drain(smem_u32(&sh.landed[q]), (sh.issued[q] - 1) & 1, &sh.timeout);
      }
      return;
    }
  }
}

constexpr int kKeyThreads = 288;

// One CTA per (sequence, page that holds new tokens): the mean of its filled
// rows.  Thread t sums columns 8 (t mod 72) .. + 7 over rows t / 72, + 4, ...
// Four rows in flight: 13 prompts of 512 to 8190 tokens 10.6 us from a bf16 cache, 4.1
// TB/s with the launch and the lengths' and the table's reads (eight rows in flight
// 11.2, sixteen 14.9: registers and the ragged pages' remainders); the last pages of
// 128 sequences 3.0 us, 8-bit.
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
// can touch; their rows fit the shared memory that needs no opt-in (42 rows).
// Against the ring of pages, us in a graph, new tokens 1 / 8 / 24 / 32 / 40: one
// sequence 2.1 / 2.3 / 2.6 / 2.8 / 2.9 and 3.6 / 3.6 / 3.8 / 3.8 / 4.0; 128 of them
// 2.6 / 3.0 / 3.6 / 3.8 / 4.1 and 4.1 / 4.2 / 5.2 / 5.2 / 5.2; 512 of them 4.3 / 6.0 /
// 9.9 / 11.6 / 12.9 and 6.9 / 7.7 / 10.4 / 11.5 / 13.0: where the large batches meet.
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
  const int smem = kRing * kRowsBytes;
  const cudaError_t e = cudaFuncSetAttribute(
      append_pages_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(append_pages_kernel, dim3(sm_count), dim3(kPagesThreads), smem, st, P);
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

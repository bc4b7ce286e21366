// append.cu -- new tokens into the 8-bit and the 4-bit latent cache, and the pages'
// mean keys.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp4kv.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

namespace mla {

namespace {

constexpr int kAppThreads = 384;  // that convert a page

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

// The block of 16 latent values that a thread's eight are half of: lanes l and l ^ 1
// hold its halves.  Its exponent field under the page's scale 2^se (se = 0: values in
// units of it), and the codes of this thread's eight.
struct Block4 {
  int e;
  uint32_t codes;
};
__device__ __forceinline__ Block4 block4(const float (&v)[8], int se) {
  float top = 0.0f;
  bool nan = false;
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    top = fmaxf(top, fabsf(v[k]));
    nan = nan || v[k] != v[k];
  }
  top = nan ? __uint_as_float(0x7fffffffu) : top;
  const float other = __shfl_xor_sync(0xffffffffu, top, 1);
  top = top == top && other == other ? fmaxf(top, other) : __uint_as_float(0x7fffffffu);
  Block4 b;
  b.e = block_exp4(top, se);
  b.codes = b.e == kExpNan4 ? 0u : e2m1x8(v, exp2_int(kExpBias4 - b.e - se));
  return b;
}
// Eight bf16 values times a power of two (exact but for what vanishes) to codes.
__device__ __forceinline__ uint32_t e2m1x8(const uint4& x, __nv_bfloat162 mul) {
  const uint32_t in[4] = {x.x, x.y, x.z, x.w};
  uint32_t w = 0;
#pragma unroll
  for (int k = 0; k < 4; ++k)
    w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(
             __bfloat1622float2(__hmul2(as_bf162(in[k]), mul)), __NV_E2M1, cudaRoundNearest))
         << (8 * k);
  return w;
}
// The largest size in a block, as its fp32 bits (NaN above all).
__device__ __forceinline__ uint32_t block_top(const uint4& a, const uint4& b) {
  __nv_bfloat162 m = max_abs(max_abs(max_abs(__habs2(as_bf162(a.x)), a.y), a.z), a.w);
  return larger_half(max_abs(max_abs(max_abs(max_abs(m, b.x), b.y), b.z), b.w));
}
// Four lanes' two exponents as a byte, for the first of them.
__device__ __forceinline__ uint8_t exps_byte(int e) {
  return static_cast<uint8_t>(e | (__shfl_xor_sync(0xffffffffu, e, 2) << 4));
}

struct AppendParams {
  const uint4* rows;
  int max_new;
  const int32_t* new_lens;
  const int32_t* block_table;
  const int32_t* seq_lens;
  int B, num_pages, max_pages;
  uint8_t* kv;  // 8 or 4 bits
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
  // The same of fp32 bits, NaN above all.
  __device__ uint32_t max_of_bits(uint32_t top) const {
    top = __reduce_max_sync(0xffffffffu, top);
    if ((tid & 31) == 0) warp_top[tid >> 5] = __uint_as_float(top);
    sync();
    for (int w = 0; w < kAppThreads / 32; ++w) top = max(top, __float_as_uint(warp_top[w]));
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

constexpr int kHeld = kPage * kChunks / kAppThreads;
static_assert(kHeld * kAppThreads == kPage * kChunks, "a page is whole passes");

// Fills a page from its new rows, which a thread holds in registers between their
// maximum and the codes; `taken` is called once all have theirs.  kFew skips what
// a few rows do not fill, at a price for whole pages (14 -> 15.5 us).  (Every thread
// has its Target before the first barrier here; one thread replaces the scale
// behind it.)
template <bool kFew, typename Taken>
__device__ __forceinline__ void fill_page8(const AppendParams& P, const Group& grp,
                                          const Place& at, const Target& to,
                                          const uint4* rows_sh, const Taken& taken) {
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
  uint2* const dst = reinterpret_cast<uint2*>(P.kv + static_cast<size_t>(to.page) * kPageBytes8);
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

// The same into the 4-bit cache: a thread has blocks of 16 values, two chunks of 16 bytes,
// first the rows' latent ones, then their RoPE columns (a warp's are of one kind).  Every
// other lane takes its second chunk first, so that eight lanes' loads meet all banks.
// The blocks' maxima stay in registers; the rows are read a second time for the codes
// (held, they were spilled).  13 prompts of 512 to 8190 tokens: 36 us with the rows held,
// 28 with eight values to a thread and a shuffle for the block's maximum, 19 with latent
// and RoPE blocks in one warp and the maxima found twice, 16 so; its ALU pipes are then busy
// for 40 % of it, and a page's barriers come next.
constexpr int kLatBlocks = kLora / kBlock4, kRopeBlocks = kRope / kBlock4;
constexpr int kBlocks = kLatBlocks + kRopeBlocks;  // of a row: 36
constexpr int kPasses = kPage * kBlocks / kAppThreads;
static_assert(kPasses * kAppThreads == kPage * kBlocks && kLatBlocks == 32, "whole passes");

template <bool kFew, typename Taken>
__device__ __forceinline__ void fill_page4(const AppendParams& P, const Group& grp,
                                           const Place& at, const Target& to,
                                           const uint4* rows_sh, const Taken& taken) {
  const int r0 = at.r0(), r1 = at.r1(), rows = r1 - r0, n = rows * kBlocks;
  const int swapped = (grp.tid ^ (grp.tid >> 2)) & 1;
  // Block i's first chunk.
  auto chunk_of = [&](int i) {
    const int u = i - rows * kLatBlocks;
    return u < 0 ? (i / kLatBlocks) * kChunks + 2 * (i % kLatBlocks)
                 : (u / kRopeBlocks) * kChunks + 2 * kLatBlocks + 2 * (u % kRopeBlocks);
  };
  uint32_t tops[kPasses], top = 0;
#pragma unroll
  for (int k = 0; k < kPasses; ++k) {
    const int i = grp.tid + k * kAppThreads;
    tops[k] = 0;
    if (kFew && k * kAppThreads >= n) break;
    if (i < n) {
      const uint4* const x = rows_sh + chunk_of(i);
      tops[k] = block_top(x[swapped], x[swapped ^ 1]);
    }
    top = max(top, tops[k]);
  }
  top = grp.max_of_bits(top);
  float largest = __uint_as_float(top);
  if (top >= 0x7f800000u) {  // rare: once more, without infinities and NaN
    grp.sync();
    largest = 0.0f;
    for (int i = grp.tid; i < rows * kChunks; i += kAppThreads)
      largest = finite_absmax8(largest, rows_sh[i]);
    largest = grp.max_of(largest);
  }
  float scale = exp2_int(page_scale_exp(largest));
  if (r0 > 0) scale = fmaxf(scale, next_power_of_two(to.old));
  const int se = static_cast<int>(__float_as_uint(scale) >> 23) - 127;
  uint8_t* const dst = P.kv + static_cast<size_t>(to.page) * kPageBytes4;
  if (to.in_pool) {
#pragma unroll
    for (int k = 0; k < kPasses; ++k) {
      if (kFew && k * kAppThreads >= n) break;
      const int i = grp.tid + k * kAppThreads, u = i - rows * kLatBlocks;
      const int e = block_exp4(__uint_as_float(tops[k]), se);
      const int next = __shfl_xor_sync(0xffffffffu, e, 1);
      if (i >= n) continue;
      const uint4* const x = rows_sh + chunk_of(i);
      const uint4 xa = x[swapped], xb = x[swapped ^ 1];
      if (u < 0) {
        uint8_t* const row = dst + (r0 + i / kLatBlocks) * kRow4;
        const int c = i % kLatBlocks;
        const __nv_bfloat162 mul = __float2bfloat162_rn(exp2_int(kExpBias4 - e - se));
        uint32_t wa = e2m1x8(xa, mul), wb = e2m1x8(xb, mul);
        if (e == kExpNan4) wa = wb = 0u;
        *reinterpret_cast<uint2*>(row + 8 * c) =
            swapped ? make_uint2(wb, wa) : make_uint2(wa, wb);
        if ((c & 1) == 0) row[kRowExps4 + (c >> 1)] = static_cast<uint8_t>(e | (next << 4));
      } else {
        const __nv_bfloat162 inv = __float2bfloat162_rn(1.0f / scale);
        const uint2 ca = codes8(xa, inv), cb = codes8(xb, inv);
        *reinterpret_cast<uint4*>(dst + (r0 + u / kRopeBlocks) * kRow4 + kRowRope4 +
                                  16 * (u % kRopeBlocks)) =
            swapped ? make_uint4(cb.x, cb.y, ca.x, ca.y) : make_uint4(ca.x, ca.y, cb.x, cb.y);
      }
    }
  }
  if (!kFew) {
    grp.sync();
    taken();
  }
  if (!to.in_pool) return;
  if (grp.tid == 0) P.kv_scale[to.page] = scale;
  if (r0 == 0) {  // a page that starts here: cleared behind the new rows
    uint4* const all = reinterpret_cast<uint4*>(dst);
    for (int i = r1 * (kRow4 / 16) + grp.tid; i < kPageBytes4 / 16; i += kAppThreads)
      all[i] = make_uint4(0u, 0u, 0u, 0u);
    return;
  }
  if (scale == to.old) return;
  // The scale grew: rows that stay are quantised again from their values.
  const float ratio = to.old / scale;
#pragma unroll 1
  for (int i = grp.tid; i < kPage * kChunks; i += kAppThreads) {
    const int r = i / kChunks, c = i % kChunks;
    const bool stays = r < r0 || r >= r1;
    uint8_t* const row = dst + r * kRow4;
    float v[8] = {};
    if (stays) values4(load_raw4(row, c), c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = mul_odd(v[k], ratio);
    const Block4 b = block4(v, 0);
    const uint8_t exps = exps_byte(b.e);  // (behind all four lanes' reads of the byte)
    if (!stays) continue;
    if (c < kLora / 8) {
      *reinterpret_cast<uint32_t*>(row + 4 * c) = b.codes;
      if ((c & 3) == 0) row[kRowExps4 + (c >> 2)] = exps;
    } else {
      *reinterpret_cast<uint2*>(row + kRowRope4 + 8 * (c - kLora / 8)) =
          make_uint2(e4m3x4(v[0], v[1], v[2], v[3]), e4m3x4(v[4], v[5], v[6], v[7]));
    }
  }
}

template <bool kFew, bool kFp4, typename Taken>
__device__ __forceinline__ void fill_page(const AppendParams& P, const Group& grp,
                                          const Place& at, const Target& to,
                                          const uint4* rows_sh, const Taken& taken) {
  if constexpr (kFp4)
    fill_page4<kFew>(P, grp, at, to, rows_sh, taken);
  else
    fill_page8<kFew>(P, grp, at, to, rows_sh, taken);
}

// A few new tokens per sequence: one CTA per sequence and page that they can
// touch.  One token for each of 128 sequences: 2.6 us in a graph, a launch and a
// chain of three reads (lengths, block table, scale) beside the row's.
template <bool kFp4>
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
    fill_page<true, kFp4>(P, grp, at, to, rows_sh, [] {});
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
// buffer took 16.2, and two passes over shared memory in place of registers 16.  (Into
// the 4-bit cache 16.)  What is left is mostly the start (lengths, sums, first loads: 2 us
// with nothing in flight) and the last pages' conversion.
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

template <bool kFp4>
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
      fill_page<false, kFp4>(P, grp, at, Target(P, at, grp.tid == 0), rows_of(k + i), [&] {
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

// Rows that a CTA sums side by side, 72 threads to each.  Eight of the 4-bit cache where
// there are few pages to an SM, as its codes' conversion is what takes long: the last pages
// of 128 sequences 3.5 us instead of 4.2, but 13 prompts by a list 9.7 instead of 8.6.
constexpr int key_groups(Kind kind, bool list) { return kind == Kind::kFp4 && !list ? 8 : 4; }
constexpr int key_threads(Kind kind, bool list) { return kChunks * key_groups(kind, list); }
constexpr int key_ctas(Kind kind, bool list) { return 16 / key_groups(kind, list); }  // an SM

struct KeyParams {
  const uint8_t* cache;
  const float* kv_scale;
  const int32_t* block_table;
  const int32_t* seq_lens;
  const int32_t* new_lens;
  __nv_bfloat16* keys;
  int32_t* status;
  int B, max_new, num_pages, max_pages;
};

// The mean of a page's filled rows.  Thread t sums columns 8 (t mod 72) .. + 7 over rows
// t / 72, + 4, ...  Caches that are not in L2, 13 prompts of 512 to 8190 tokens (63k): 13.9 us
// from bf16, 8.3 from 8 bits, 16.9 from 4 (its codes' conversion: two thirds of it on the
// ALUs); four rows in flight from the first two (bf16 with eight or sixteen: slower, for
// registers and the ragged pages' remainders).  The last pages of 128 sequences 2.8 us from
// 8 bits.
template <Kind kKind, int kSide>
__device__ __forceinline__ void page_mean(const KeyParams& P, int b, int len, int logical,
                                          float (&part)[kSide][kDqk]) {
  const auto [cache, kv_scale, block_table, seq_lens, new_lens, keys, status, B, max_new,
              num_pages, max_pages] = P;
  const int page = block_table[static_cast<size_t>(b) * max_pages + logical];
  if (page < 0 || page >= num_pages) {
    if (threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
    return;
  }
  // (Looked at behind the rows' loads: a trip to memory next to theirs, not before.  From
  // 8 bits it is loaded there, and all by way of the read-only path: 2.81 us on the last
  // pages of 128 sequences, 2.94 else.)
  float given = kKind == Kind::kFp4 ? kv_scale[page] : 1.0f;
  const int filled = min(len - logical * kPage, kPage);
  const int c = threadIdx.x % kChunks, r0 = threadIdx.x / kChunks;
  float s[8] = {};
  auto add = [&](const float (&x)[8]) {
#pragma unroll
    for (int k = 0; k < 8; ++k) s[k] += x[k];
  };
  if constexpr (kKind == Kind::kFp4) {
    const uint8_t* const base = cache + static_cast<size_t>(page) * kPageBytes4;
    constexpr int kDeep = 8, kStep = kSide;  // its rows' loads in flight
    for (int r = r0; r < filled; r += kStep * kDeep) {
      Raw4 raw[kDeep];
#pragma unroll
      for (int k = 0; k < kDeep; ++k)
        raw[k] = load_raw4(base + min(r + kStep * k, filled - 1) * kRow4, c);
#pragma unroll
      for (int k = 0; k < kDeep; ++k) {
        if (r + kStep * k >= filled) break;
        float x[8];
        values4(raw[k], c, x);
        add(x);
      }
    }
  } else {
#pragma unroll 4
    for (int r = r0; r < filled; r += 4) {
      float x[8];
      if constexpr (kKind == Kind::kFp8) {
        values8x8(__ldg(reinterpret_cast<const uint2*>(
                      cache + static_cast<size_t>(page) * kPageBytes8 + r * kDqk + c * 8)), x);
      } else {
        const uint4 v = __ldg(reinterpret_cast<const uint4*>(
            cache + (static_cast<size_t>(page) * kPage + r) * (kDqk * 2) + c * 16));
        x[0] = bf16_lo(v.x); x[1] = bf16_hi(v.x); x[2] = bf16_lo(v.y); x[3] = bf16_hi(v.y);
        x[4] = bf16_lo(v.z); x[5] = bf16_hi(v.z); x[6] = bf16_lo(v.w); x[7] = bf16_hi(v.w);
      }
      add(x);
    }
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) part[r0][c * 8 + k] = s[k];
  __syncthreads();
  if constexpr (kKind == Kind::kFp8) given = __ldg(kv_scale + page);
  const bool in_range = scale_in_range(given);
  const float mul = (in_range ? given : 1.0f) / static_cast<float>(filled);
  const int k = threadIdx.x * 2;
  if (k < kDqk) {
    float x = (part[0][k] + part[1][k]) + (part[2][k] + part[3][k]);
    float y = (part[0][k + 1] + part[1][k + 1]) + (part[2][k + 1] + part[3][k + 1]);
    if constexpr (kSide == 8) {
      x += (part[4][k] + part[5][k]) + (part[6][k] + part[7][k]);
      y += (part[4][k + 1] + part[5][k + 1]) + (part[6][k + 1] + part[7][k + 1]);
    }
    *reinterpret_cast<uint32_t*>(keys + static_cast<size_t>(page) * kDqk + k) =
        pack_bf16x2(x * mul, y * mul);
  }
  if (!in_range && threadIdx.x == 0) record_status(status, MLA_STATUS_BOUNDS);
}

// One CTA per (sequence, page that it can touch), or a list of the pages (launch_keys).
template <Kind kKind, bool kList>
__global__ void __launch_bounds__(key_threads(kKind, kList), key_ctas(kKind, kList))
page_keys_kernel(const __grid_constant__ KeyParams P) {
  __shared__ float part[key_groups(kKind, kList)][kDqk];
  griddep_wait();
  griddep_launch_dependents();
  if constexpr (kList) {
    __shared__ UnitList list;
    const long long pages = list.make(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, P.B,
                                      P.status, [](const NewTokens& nt) { return nt.pages(); });
    for (long long f = blockIdx.x; f < pages; f += gridDim.x) {
      const int b = list.find(f), len = list.len[b];
      const int logical = (len - 1) / kPage - static_cast<int>(list.upto[b] - 1 - f);
      page_mean<kKind, key_groups(kKind, kList)>(P, b, len, logical, part);
      __syncthreads();  // `part` has been read
    }
  } else {
    const int b = blockIdx.y;
    NewTokens nt;
    if (nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_pages * kPage, b, threadIdx.x == 0,
                P.status) &&
        blockIdx.x < nt.pages())
      page_mean<kKind, key_groups(kKind, kList)>(
          P, b, nt.len, nt.first / kPage + static_cast<int>(blockIdx.x), part);
  }
}

}  // namespace

// Up to so many new tokens a sequence, a CTA for each of the two pages that they
// can touch; their rows fit the shared memory that needs no opt-in (42 rows).
// Against the ring of pages, us in a graph, new tokens 1 / 8 / 24 / 32 / 40: one
// sequence 2.1 / 2.3 / 2.6 / 2.8 / 2.9 and 3.6 / 3.6 / 3.8 / 3.8 / 4.0; 128 of them
// 2.6 / 3.0 / 3.6 / 3.8 / 4.1 and 4.1 / 4.2 / 5.2 / 5.2 / 5.2; 512 of them 4.3 / 6.0 /
// 9.9 / 11.6 / 12.9 and 6.9 / 7.7 / 10.4 / 11.5 / 13.0: where the large batches meet.
constexpr int kFewTokens = 32;

cudaError_t launch_append(const void* rows, int max_new, const int32_t* new_lens,
                          const int32_t* block_table, const int32_t* seq_lens, int B,
                          int num_pages, int max_pages, uint8_t* kv, bool fp4, float* kv_scale,
                          int32_t* status, int sm_count, cudaStream_t st) {
  const AppendParams P{static_cast<const uint4*>(rows), max_new, new_lens, block_table, seq_lens,
                       B, num_pages, max_pages, kv, kv_scale, status};
  if (max_new <= kFewTokens)
    return launch_pdl(fp4 ? append_few_kernel<true> : append_few_kernel<false>,
                      dim3(touched_pages(max_new, max_pages), B), dim3(kAppThreads),
                      max_new * kDqk * 2, st, P);
  const int smem = kRing * kRowsBytes;
  const auto kern = fp4 ? append_pages_kernel<true> : append_pages_kernel<false>;
  const cudaError_t e = cudaFuncSetAttribute(
      kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  return launch_pdl(kern, dim3(sm_count), dim3(kPagesThreads), smem, st, P);
}

template <Kind kKind>
static cudaError_t launch_keys(const KeyParams& P, int sm_count, cudaStream_t st) {
  const int touched = touched_pages(P.max_new, P.max_pages);
  // Caches that are not in L2, us with a list and without: from 4 bits 100 prompts of 100 to
  // 2000 tokens 23.9 and 30.3, the 13 of 512 to 8190 16.9 and 17.4, 8 of 8000 (nothing to
  // skip) 16.9 and 16.2.  The others have more to load than to convert and want the padded
  // grid's CTAs: from 8 bits 17.3 and 13.9, 12.3 and 8.4, 12.4 and 8.6; from bf16 23.7 and
  // 23.5, 14.6 and 13.9, 15.3 and 14.7.
  if constexpr (kKind == Kind::kFp4)
    if (use_list(static_cast<int64_t>(touched) * P.B, 6 * sm_count, P.B, P.new_lens))
      return launch_pdl(page_keys_kernel<kKind, true>, dim3(sm_count * key_ctas(kKind, true)),
                        dim3(key_threads(kKind, true)), 0, st, P);
  return launch_pdl(page_keys_kernel<kKind, false>, dim3(touched, P.B),
                    dim3(key_threads(kKind, false)), 0, st, P);
}

cudaError_t launch_page_keys(Kind kind, const void* cache, const float* kv_scale,
                             const int32_t* block_table, const int32_t* seq_lens, int max_new,
                             const int32_t* new_lens, int B, int num_pages, int max_pages,
                             __nv_bfloat16* keys, int32_t* status, int sm_count,
                             cudaStream_t st) {
  const KeyParams P{static_cast<const uint8_t*>(cache), kv_scale, block_table, seq_lens, new_lens,
                    keys, status, B, max_new, num_pages, max_pages};
  return kind == Kind::kFp4   ? launch_keys<Kind::kFp4>(P, sm_count, st)
         : kind == Kind::kFp8 ? launch_keys<Kind::kFp8>(P, sm_count, st)
                              : launch_keys<Kind::kBf16>(P, sm_count, st);
}

}  // namespace mla

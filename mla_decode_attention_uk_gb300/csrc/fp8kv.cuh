// fp8kv.cuh -- what the kernels of the 8-bit latent cache share: its layout,
// its scales, and the PTX of 8-bit tensor-core operands.
//
// The cache holds a page of 64 tokens as 64 x 576 E4M3 codes ([c_kv 512 ||
// k_pe 64] per token, as the bf16 cache) and one fp32 scale per page: a value
// is code * scale.  E4M3 keeps four significant bits down to 2^-6, so a page
// whose largest value takes the top of the range (448) holds values to 2^-15
// of it at full precision, and one scale for the block of 64 tokens loses
// nothing against finer ones.  The scales that the library writes are powers
// of two: scaling and rescaling are then exact, and a code depends only on the
// value and the scale, not on how a quotient was rounded.
#pragma once
#include <cstdint>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "ptx.cuh"

namespace mla {

constexpr int kPageBytes8 = kPage * kDqk;  // one page of codes: 36,864 bytes
// Exponents of a page's scale.  bf16 latents of practical size lie far inside;
// the bound keeps every product of the attention step in fp32's range.
constexpr int kScaleExpMin = -32;
constexpr int kScaleExpMax = 32;

// The query's two E4M3 terms (attention step): q = scale * (hi + mid / 16).
constexpr float kQMidScale = 16.0f;
// One tile of query terms, 128 rows: rows 32 w + i and 32 w + 16 + i are the hi
// and mid terms of tile row 16 w + i, so that the two land in TMEM lanes of the
// same warp.
constexpr int kQTermRows = 2 * kTileRows;
constexpr int kQBox8 = kQTermRows * 128;  // 128 rows of 128 bytes: 16 KB
constexpr int kBoxes8 = 5;                // 128-byte-wide boxes of a cached row

// Exponent of the smallest power of two s with amax <= 448 s, within the
// bounds.  amax: finite, >= 0; exact (bit operations only).
__device__ __forceinline__ int scale_exp(float amax, int lo, int hi) {
  const uint32_t u = __float_as_uint(amax);
  const int k = static_cast<int>(u >> 23) - 127;  // amax = m 2^k, 1 <= m < 2 (normal numbers)
  const int e = k - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);  // 448 = 1.75 * 2^8
  return max(lo, min(hi, e));
}
__device__ __forceinline__ int page_scale_exp(float amax) {
  return scale_exp(amax, kScaleExpMin, kScaleExpMax);
}
__device__ __forceinline__ float exp2_int(int e) {
  return __uint_as_float(static_cast<uint32_t>(e + 127) << 23);
}

// A page's scale within the bounds (not so for NaN).
__device__ __forceinline__ bool scale_in_range(float s) {
  return s >= exp2_int(kScaleExpMin) && s <= exp2_int(kScaleExpMax);
}
// The smallest power of two that is not below s (s: normal, positive).
__device__ __forceinline__ float next_power_of_two(float s) {
  return __uint_as_float((__float_as_uint(s) + 0x7fffffu) & 0x7f800000u);
}

// Four values to four E4M3 codes, round to nearest even, finite values beyond
// 448 (infinities too) saturated; NaN keeps NaN's code.
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
  const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
  return lo | (hi << 16);
}
// Two E4M3 codes (low 16 bits) to fp32, exact.
__device__ __forceinline__ float2 e4m3x2_to_float2(uint32_t codes) {
  return __half22float2(static_cast<__half2>(__nv_cvt_fp8x2_to_halfraw2(
      static_cast<__nv_fp8x2_storage_t>(codes & 0xffffu), __NV_E4M3)));
}

__device__ __forceinline__ __nv_bfloat162 as_bf162(uint32_t w) {
  return *reinterpret_cast<const __nv_bfloat162*>(&w);
}
// Four bf16 values as two words of E4M3 codes: value = 2^e (hi + mid / 16) for |value|
// < 256 * 2^e, exactly down to |value| = 2^(e - 6) (cut to 2^(e - 13) below).
// down = 2^(-e - 120) brings E4M3's exponent field and steps (bias 7) onto
// bf16's (bias 127), subnormals too, so that a code is a bit field of the bf16
// number: hi is the value cut to four significant bits, mid 16 times the rest,
// which has at most four.  (Conversion instructions took twice as many.)
__device__ __forceinline__ uint32_t e4m3_field(uint32_t w) {  // of two, in bytes 0 and 2
  constexpr uint32_t kMagnitude = 0x007f007fu;
  return ((w >> 4) & kMagnitude) | ((w >> 8) & ~kMagnitude);
}
__device__ __forceinline__ void split_terms(uint2 x, __nv_bfloat162 down, uint32_t& hi,
                                            uint32_t& mid) {
  const __nv_bfloat162 down16 = __hmul2(down, __float2bfloat162_rn(kQMidScale));
  const uint32_t in[2] = {x.x, x.y};
  uint32_t h[2], m[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const __nv_bfloat162 v = __hmul2(as_bf162(in[i]), down);
    const uint32_t cut = *reinterpret_cast<const uint32_t*>(&v) & 0xfff0fff0u;
    const __nv_bfloat162 rest = __hfma2(as_bf162(cut), __float2bfloat162_rn(-kQMidScale),
                                        __hmul2(as_bf162(in[i]), down16));
    h[i] = e4m3_field(cut);
    m[i] = e4m3_field(*reinterpret_cast<const uint32_t*>(&rest));
  }
  hi = __byte_perm(h[0], h[1], 0x6420);
  mid = __byte_perm(m[0], m[1], 0x6420);
}

// A query row's exponent: amax <= 224 * 2^e, so that the row's largest value takes
// the top but one of E4M3's binades.  Rows of every size that bf16 has: e reaches
// 121 for the largest; below 2^-118 it stays at -126 (2^e remains a normal number)
// and the terms hold bf16's smallest values, multiples of 2^-133, exactly.
__device__ __forceinline__ int term_exp(float amax) { return scale_exp(amax, -127, 120) + 1; }

// split_terms' factor for a row's exponent, and what comes before it where 2^(-e -
// 120) is below bf16's normal numbers (rows beyond 224 * 2^6).
constexpr int kTermExpMax = 6;
__device__ __forceinline__ __nv_bfloat162 term_factor(int e) {
  return __float2bfloat162_rn(exp2_int(-min(e, kTermExpMax) - 120));
}
__device__ __forceinline__ uint2 lower_terms(uint2 x, int e) {
  const __nv_bfloat162 f = __float2bfloat162_rn(exp2_int(kTermExpMax - e));
  const __nv_bfloat162 a = __hmul2(as_bf162(x.x), f), b = __hmul2(as_bf162(x.y), f);
  return make_uint2(*reinterpret_cast<const uint32_t*>(&a), *reinterpret_cast<const uint32_t*>(&b));
}

// The largest size among a row's values, NaN above all, as its fp32 bits.
__device__ __forceinline__ __nv_bfloat162 max_abs(__nv_bfloat162 top, uint32_t w) {
  return __hmax2_nan(top, __habs2(as_bf162(w)));
}
__device__ __forceinline__ uint32_t larger_half(__nv_bfloat162 top) {
  return max(__float_as_uint(__low2float(top)), __float_as_uint(__high2float(top)));
}
// The factor of a row's terms; not a number for a row that is not finite.
__device__ __forceinline__ float row_scale(float amax, int e) {
  return amax < INFINITY ? exp2_int(e) : __uint_as_float(0x7fffffffu);
}

// A named barrier of n threads: whether any of them has `pred`.
__device__ __forceinline__ bool bar_any(uint32_t id, uint32_t n, bool pred) {
  uint32_t r;
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t"
      "setp.ne.u32 p, %1, 0;\n\t"
      "bar.red.or.pred q, %2, %3, p;\n\t"
      "selp.u32 %0, 1, 0, q;\n\t}\n"
      : "=r"(r)
      : "r"(pred ? 1u : 0u), "r"(id), "r"(n)
      : "memory");
  return r != 0;
}

// Records the first device-side error, where the caller asked for it.
__device__ __forceinline__ void record_status(int32_t* status, int code) {
  if (status) atomicCAS(status, 0, code);
}

// Instruction descriptor for kind::f8f6f4 with fp32 accumulation.  Formats: 0
// E4M3, 1 E5M2; a_mn / b_mn select MN-major (transposed) operands.
__host__ __device__ constexpr uint32_t idesc_f8_f32(int M, int N, uint32_t a_fmt, uint32_t b_fmt,
                                                    bool a_mn, bool b_mn) {
  return (1u << 4) | (a_fmt << 7) | (b_fmt << 10) | ((a_mn ? 1u : 0u) << 15) |
         ((b_mn ? 1u : 0u) << 16) | (static_cast<uint32_t>(N >> 3) << 17) |
         (static_cast<uint32_t>(M >> 4) << 24);
}
// D[tmem] (+)= A[smem] * B[smem]^T of 8-bit operands (K = 32), one thread.
__device__ __forceinline__ void umma_f8(uint32_t d_tmem, uint64_t adesc, uint64_t bdesc,
                                        uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "l"(adesc), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// The same with A in tensor memory: lane = row, four codes to a column.
__device__ __forceinline__ void umma_f8_ta(uint32_t d_tmem, uint32_t a_tmem, uint64_t bdesc,
                                           uint32_t idesc, uint32_t accumulate) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], [%1], %2, %3, p;\n\t}\n" ::"r"(d_tmem),
      "r"(a_tmem), "l"(bdesc), "r"(idesc), "r"(accumulate)
      : "memory");
}

// 16 lanes x 64 bits, 8 repetitions (16 columns): the lane and column mapping
// of tmem_ld_16x64b_x16.
__device__ __forceinline__ void tmem_st_16x64b_x8(uint32_t taddr, const uint32_t (&r)[8]) {
  asm volatile(
      "tcgen05.st.sync.aligned.16x64b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
      : "memory");
}
// 32 lanes x 32 bits, 16 consecutive columns (as tmem_ld_x16).
__device__ __forceinline__ void tmem_st_x16(uint32_t taddr, const uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16};" ::"r"(taddr),
      "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
      "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]),
      "r"(r[15])
      : "memory");
}

// Bulk copy of `bytes` from global to shared memory, completing on an
// mbarrier; both addresses and the size are multiples of 16 bytes.
__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes,
                                          uint32_t bar) {
  asm volatile(
      "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1], %2, [%3];" ::"r"(dst),
      "l"(src), "r"(bytes), "r"(bar)
      : "memory");
}

// 3-D tiled load of one box into shared memory (see tma_load_2d).
__device__ __forceinline__ void tma_load_3d(uint32_t dst, const CUtensorMap* m, int32_t c0,
                                            int32_t c1, int32_t c2, uint32_t bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%2, %3, %4}], [%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(m)), "r"(c0), "r"(c1), "r"(c2), "r"(bar)
      : "memory");
}

__device__ __forceinline__ uint2 ld_shared_v2(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ void st_shared_b32(uint32_t addr, uint32_t v) {
  asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
}
__device__ __forceinline__ void mbar_arrive_n(uint32_t bar, uint32_t n) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(bar), "r"(n) : "memory");
}

}  // namespace mla

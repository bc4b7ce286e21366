// fp4kv.cuh -- what the kernels of the 4-bit latent cache share: its layout and
// its conversions.
//
// A page holds 64 rows of 336 bytes:
//   256 bytes  512 latent values as E2M1 codes (a sign, 0 0.5 1 1.5 2 3 4 6), value
//              2 i in the low half of byte i
//    16 bytes  an exponent e of four bits for each 16 latent values (block 2 i in
//              the low half of byte i): their factor is 2^(e - 8); 15: all NaN
//    64 bytes  k_pe as E4M3 codes (the RoPE columns carry large values, and the
//              scores feel each error there; they are a ninth of the row)
// and has one fp32 scale, as a page of the 8-bit cache.  The exponents' range is
// that of E4M3: 6 * 2^6 = 384 is its last value but two, 0.5 * 2^-8 = 2^-9 its
// smallest.  So every value of the cache is an E4M3 code times the page's scale: a
// page expands exactly to one of the 8-bit cache, and the attention step (tensor
// cores, query terms, weights, the page's scale) is the same from there on.
// 16 values to a block: a latent row has a few large channels, which take the small
// values of their blocks with them.  Root mean square error of standard normal rows, and
// of rows in which every 97th channel is six times as large, relative: blocks of 16 0.110
// and 0.122, of 32 0.112 and 0.136, one scale a row 0.122 and 0.271; a row is 336 bytes,
// 328 and 321.
#pragma once
#include <cuda_fp4.h>

#include "fp8kv.cuh"

namespace mla {

constexpr int kBlock4 = 16;
constexpr int kRowExps4 = kLora / 2;                        // where the exponents start: 256
constexpr int kRowRope4 = kRowExps4 + kLora / kBlock4 / 2;  // the RoPE codes: 272
constexpr int kRow4 = kRowRope4 + kRope;                    // 336
constexpr int kPageBytes4 = kPage * kRow4;                  // 21,504
constexpr int kExpBias4 = 8;
constexpr int kExpNan4 = 15;
static_assert(kRow4 % 16 == 0 && kRowRope4 % 16 == 0, "16-byte parts");

// Exponent field of a block whose largest size is amax (fp32 bits that may be
// infinite; NaN gives kExpNan4), under the page's scale 2^se: the smallest e in
// 0..14 with amax <= 7 * 2^(e - 8 + se).  (Beyond 6 the nearest code is 6, off by
// at most half of the top step, as every other rounding.)
__device__ __forceinline__ int block_exp4(float amax, int se) {
  const int e = scale_exp(amax, se - 14, se) - se + 14;  // 448 = 7 * 2^6
  return amax == amax ? e : kExpNan4;
}

// Eight values times `mul` (a power of two: their block's 1 / 2^(e - 8 + se)) to
// E2M1 codes, round to nearest even, saturated; value i in bits 4 i .. 4 i + 3.
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float mul) {
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i)
    w |= static_cast<uint32_t>(__nv_cvt_float2_to_fp4x2(
             make_float2(v[2 * i] * mul, v[2 * i + 1] * mul), __NV_E2M1, cudaRoundNearest))
         << (8 * i);
  return w;
}

// Eight codes of a block with exponent field e as values in units of the page's
// scale: exact (fp16 holds 384 and 2^-9).
__device__ __forceinline__ void values4x8(uint32_t w, uint32_t e, float (&v)[8]) {
  const uint32_t f = e < kExpNan4 ? (e + 15 - kExpBias4) << 10 : 0x7fffu;
  const uint32_t f2 = f | (f << 16);
  const __half2 mul = *reinterpret_cast<const __half2*>(&f2);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const __half2 h = static_cast<__half2>(__nv_cvt_fp4x2_to_halfraw2(
        static_cast<__nv_fp4x2_storage_t>((w >> (8 * i)) & 0xffu), __NV_E2M1));
    const float2 x = __half22float2(__hmul2(h, mul));
    v[2 * i] = x.x;
    v[2 * i + 1] = x.y;
  }
}

// Eight E4M3 codes as values.
__device__ __forceinline__ void values8x8(uint2 c, float (&v)[8]) {
  const float2 x0 = e4m3x2_to_float2(c.x), x1 = e4m3x2_to_float2(c.x >> 16);
  const float2 x2 = e4m3x2_to_float2(c.y), x3 = e4m3x2_to_float2(c.y >> 16);
  v[0] = x0.x; v[1] = x0.y; v[2] = x1.x; v[3] = x1.y;
  v[4] = x2.x; v[5] = x2.y; v[6] = x3.x; v[7] = x3.y;
}

// Columns 8 c .. 8 c + 7 of a row of the 4-bit cache, as two words: the codes of latent
// columns and the word that holds their block's exponent, or eight RoPE codes.  (Two
// loads for either, so that lanes with either kind load together.)
struct Raw4 {
  uint32_t a, b;
};
__device__ __forceinline__ Raw4 load_raw4(const uint8_t* row, int c) {
  const bool latent = c < kLora / 8;
  const int at = latent ? 4 * c : kRowRope4 + 8 * (c - kLora / 8);
  return Raw4{*reinterpret_cast<const uint32_t*>(row + at),
              *reinterpret_cast<const uint32_t*>(row + (latent ? kRowExps4 + 4 * (c >> 4)
                                                               : at + 4))};
}
// Their values in units of the page's scale.
__device__ __forceinline__ void values4(const Raw4& x, int c, float (&v)[8]) {
  if (c < kLora / 8)
    values4x8(x.a, (x.b >> (4 * ((c >> 1) & 7))) & 15u, v);
  else
    values8x8(make_uint2(x.a, x.b), v);
}

}  // namespace mla

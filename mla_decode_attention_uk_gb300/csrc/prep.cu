// prep.cu -- norms and rotation of new tokens' queries and latents, in front of the
// cache: one pass over what the projections gave.
//
// For a token at position p, with cos and sin of its 32 angles:
//   query head    x = q or, with a norm, q / sqrt(mean(q^2) + eps) * w over its 192
//                 columns; the last 64 are rotated
//   latent row    c_kv / sqrt(mean(c_kv^2) + eps) * w over its 512 columns, k_pe
//                 (64) rotated; into rows of the same layout, or the bf16 cache's page
// A pair (a, b) becomes (a cos - b sin, b cos + a sin).  All in fp32, rounded once.
//
// Bound by memory.  A warp takes four heads of a token, eight lanes a head and 24
// columns a lane (three loads of 16 bytes, the third of them RoPE columns: every
// lane has work, and a head's norm is three shuffles), or a token's latent row.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "prep.h"
#include "ptx.cuh"
#include "tokens.cuh"

namespace mla {

namespace {

constexpr int kPrepThreads = 256;
constexpr int kHeadsPerWarp = 4;
constexpr int kHalf = kRope / 2;

__device__ __forceinline__ void unpack8(const uint4& x, float (&v)[8]) {
  v[0] = bf16_lo(x.x); v[1] = bf16_hi(x.x); v[2] = bf16_lo(x.y); v[3] = bf16_hi(x.y);
  v[4] = bf16_lo(x.z); v[5] = bf16_hi(x.z); v[6] = bf16_lo(x.w); v[7] = bf16_hi(x.w);
}
__device__ __forceinline__ uint4 pack8(const float (&v)[8]) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                    pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ float squares8(const float (&v)[8], float sum) {
#pragma unroll
  for (int k = 0; k < 8; ++k) sum = fmaf(v[k], v[k], sum);
  return sum;
}
__device__ __forceinline__ void scale8(float (&v)[8], float by, const uint4& w) {
  float f[8];
  unpack8(w, f);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = v[k] * by * f[k];
}

// RoPE columns 8 c .. 8 c + 7, rotated; the lanes of c = 0..7 are neighbours.
template <bool kInterleaved>
__device__ __forceinline__ void rotate8(float (&v)[8], const float* __restrict__ cos_sin, int c) {
  if constexpr (kInterleaved) {
    const float4 cs = *reinterpret_cast<const float4*>(cos_sin + 4 * c);
    const float4 sn = *reinterpret_cast<const float4*>(cos_sin + kHalf + 4 * c);
    const float co[4] = {cs.x, cs.y, cs.z, cs.w}, si[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float a = v[2 * k], b = v[2 * k + 1];
      v[2 * k] = a * co[k] - b * si[k];
      v[2 * k + 1] = b * co[k] + a * si[k];
    }
  } else {
    const float sign = c < 4 ? -1.0f : 1.0f;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 cs = *reinterpret_cast<const float4*>(cos_sin + 8 * (c & 3) + 4 * h);
      const float4 sn = *reinterpret_cast<const float4*>(cos_sin + kHalf + 8 * (c & 3) + 4 * h);
      const float co[4] = {cs.x, cs.y, cs.z, cs.w}, si[4] = {sn.x, sn.y, sn.z, sn.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float other = __shfl_xor_sync(0xffffffffu, v[4 * h + k], 4);
        v[4 * h + k] = v[4 * h + k] * co[k] + sign * (other * si[k]);
      }
    }
  }
}

template <bool kInterleaved>
__global__ void __launch_bounds__(kPrepThreads)
prep_kernel(const PrepParams P) {
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31;
  const int q_tasks = P.q ? P.H / kHeadsPerWarp : 0;
  const int per_token = q_tasks + (P.kv ? 1 : 0);
  const int tasks = P.B * P.max_new * per_token;
  const int warps = gridDim.x * (kPrepThreads / 32);
  for (int task = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5); task < tasks;
       task += warps) {
    const int token = task / per_token, part = task - token * per_token;
    const int b = token / P.max_new, i = token - b * P.max_new;
    NewTokens nt;
    const bool first = i == 0 && part == 0 && lane == 0;
    if (!nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_len, b, first, P.status) ||
        i >= nt.len - nt.first)
      continue;
    const int pos = P.positions ? P.positions[token] : nt.first + i;
    if (pos < 0 || pos >= P.max_position) {
      if (part == 0 && lane == 0) record_status(P.status, MLA_STATUS_BOUNDS);
      continue;
    }
    const float* const cos_sin = P.cos_sin + static_cast<size_t>(pos) * kRope;
    if (part < q_tasks) {
      const int c = lane & 7;
      const int head = part * kHeadsPerWarp + (lane >> 3);
      const uint4* const src =
          reinterpret_cast<const uint4*>(P.q + token * P.q_stride + head * kDq) + c;
      float v[3][8];
#pragma unroll
      for (int k = 0; k < 3; ++k) unpack8(src[8 * k], v[k]);
      if (P.q_weight) {
        float sum = squares8(v[2], squares8(v[1], squares8(v[0], 0.0f)));
#pragma unroll
        for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float by = rsqrtf(sum * (1.0f / kDq) + P.eps);
#pragma unroll
        for (int k = 0; k < 3; ++k)
          scale8(v[k], by, reinterpret_cast<const uint4*>(P.q_weight)[8 * k + c]);
      }
      rotate8<kInterleaved>(v[2], cos_sin, c);
      uint4* const dst =
          reinterpret_cast<uint4*>(P.q_out + (static_cast<int64_t>(token) * P.H + head) * kDq) + c;
#pragma unroll
      for (int k = 0; k < 3; ++k) dst[8 * k] = pack8(v[k]);
    } else {
      const uint4* const src = reinterpret_cast<const uint4*>(P.kv + token * P.kv_stride);
      const int c = lane & 7;
      float v[2][8], rope[8];
      unpack8(src[lane], v[0]);
      unpack8(src[32 + lane], v[1]);
      unpack8(src[64 + c], rope);
      if (P.kv_weight) {
        float sum = squares8(v[1], squares8(v[0], 0.0f));
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        const float by = rsqrtf(sum * (1.0f / kLora) + P.eps);
        scale8(v[0], by, reinterpret_cast<const uint4*>(P.kv_weight)[lane]);
        scale8(v[1], by, reinterpret_cast<const uint4*>(P.kv_weight)[32 + lane]);
      }
      rotate8<kInterleaved>(rope, cos_sin, c);
      const uint4 x0 = pack8(v[0]), x1 = pack8(v[1]), x2 = pack8(rope);
      auto store = [&](uint4* dst) {
        dst[lane] = x0;
        dst[32 + lane] = x1;
        if (lane < 8) dst[64 + lane] = x2;
      };
      if (P.rows) store(P.rows + static_cast<size_t>(token) * kChunks);
      if (P.cache) {
        const int at = nt.first + i;
        const int page = P.block_table[static_cast<size_t>(b) * P.max_pages + at / kPage];
        if (page >= 0 && page < P.num_pages)
          store(P.cache + (static_cast<size_t>(page) * kPage + at % kPage) * kChunks);
        else if (lane == 0)
          record_status(P.status, MLA_STATUS_BOUNDS);
      }
    }
  }
}

}  // namespace

cudaError_t launch_prep(const PrepParams& P, bool interleaved, int sm_count, cudaStream_t st) {
  const auto kern = interleaved ? prep_kernel<true> : prep_kernel<false>;
  const int64_t tasks = static_cast<int64_t>(P.B) * P.max_new *
                        ((P.q ? P.H / kHeadsPerWarp : 0) + (P.kv ? 1 : 0));
  const int64_t ctas = (tasks + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
  const int most = sm_count * 6;
  return launch_pdl(kern, dim3(ctas < most ? static_cast<int>(ctas) : most), dim3(kPrepThreads),
                    0, st, P);
}

}  // namespace mla

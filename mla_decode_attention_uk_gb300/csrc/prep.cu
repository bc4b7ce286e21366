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
// Measured: 7 prompts of 512 to 8190 tokens x 16 heads 58 us, 5.3 TB/s of what has to move
// (0.79 of a copy; without the next task's loads in flight 68; four CTAs an SM, which spill 36
// bytes a thread, 100 with pairs i and i + 32; three 57, five or six, which spill more, 92
// and more; cosines and sines loaded ahead as well 59, in two CTAs; two to five tasks ahead
// by asynchronous copies into shared memory 57 to 61: the rest is not for want of loads in
// flight); one token of 128 sequences x 128 heads 3.7 us, 3.4 TB/s; of two x 16 heads 2.2, a
// launch.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "../../include/mla_decode.h"
#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"
#include "tokens.cuh"

namespace mla {

namespace {

// The call's arguments, typed (q, kv, q_weight, kv_weight, positions, new_lens, rows and
// cache may be null).
struct PrepParams {
  const __nv_bfloat16* q;
  const __nv_bfloat16* kv;
  int64_t q_stride, kv_stride;
  const __nv_bfloat16* q_weight;
  const __nv_bfloat16* kv_weight;
  const float* cos_sin;
  const int32_t* positions;
  const int32_t* new_lens;
  const int32_t* seq_lens;
  const int32_t* block_table;
  __nv_bfloat16* q_out;
  uint4* rows;
  uint4* cache;
  int32_t* status;
  float eps;
  int B, H, max_new, max_position, num_pages, max_pages;
  int max_len;  // that a sequence may have
};

constexpr int kPrepThreads = 256;
constexpr int kPrepCtas = 4;  // on an SM
constexpr int kListFrom = 16384;  // tokens
constexpr int kHeadsPerWarp = 4;
constexpr int kHalf = kRope / 2;

// The absorb step reads q without a wait, as what stands in front of it has finished when
// it starts, unless that let it start early: so only a call without queries does.
__device__ __forceinline__ void wait_and_let_go(const PrepParams& P) {
  griddep_wait();
  if (!P.q) griddep_launch_dependents();
}

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

// A warp's task: four heads of a token, or its latent row.
struct Task {
  int b, first, i, part;  // token i of sequence b's new ones, which start at `first`
};

// What a lane has of it: 48 bytes of a head (RoPE columns last), or of the latent row
// (the last eight values, which lanes c, c + 8, ... share, RoPE columns).
__device__ __forceinline__ void load_task(const PrepParams& P, const Task& t, int q_tasks,
                                          uint4 (&x)[3]) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int64_t token = static_cast<int64_t>(t.b) * P.max_new + t.i;
  const bool q = t.part < q_tasks;
  const uint4* const src = reinterpret_cast<const uint4*>(
      q ? P.q + token * P.q_stride + (t.part * kHeadsPerWarp + (lane >> 3)) * kDq
        : P.kv + token * P.kv_stride);
  x[0] = src[q ? c : lane];
  x[1] = src[q ? c + 8 : lane + 32];
  x[2] = src[q ? c + 16 : 64 + c];
}

template <bool kInterleaved>
__device__ __forceinline__ void do_task(const PrepParams& P, const Task& t, int q_tasks,
                                        const uint4 (&x)[3]) {
  const int lane = threadIdx.x & 31, c = lane & 7;
  const int64_t token = static_cast<int64_t>(t.b) * P.max_new + t.i;
  const int pos = P.positions ? P.positions[token] : t.first + t.i;
  if (pos < 0 || pos >= P.max_position) {
    if (t.part == 0 && lane == 0) record_status(P.status, MLA_STATUS_BOUNDS);
    return;
  }
  const float* const cos_sin = P.cos_sin + static_cast<size_t>(pos) * kRope;
  const bool q = t.part < q_tasks;
  const __nv_bfloat16* const weight = q ? P.q_weight : P.kv_weight;
  float v[3][8];
#pragma unroll
  for (int k = 0; k < 3; ++k) unpack8(x[k], v[k]);
  if (weight) {
    // Over eight lanes and all their columns, or all lanes and the first two parts.
    float sum = squares8(v[1], squares8(v[0], 0.0f));
    if (q) sum = squares8(v[2], sum);
#pragma unroll
    for (int o = 1; o < 8; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    if (!q)
#pragma unroll
      for (int o = 8; o < 32; o <<= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float by = rsqrtf(sum * (q ? 1.0f / kDq : 1.0f / kLora) + P.eps);
    const uint4* const w = reinterpret_cast<const uint4*>(weight) + (q ? c : lane);
    scale8(v[0], by, w[0]);
    scale8(v[1], by, w[q ? 8 : 32]);
    if (q) scale8(v[2], by, w[16]);
  }
  rotate8<kInterleaved>(v[2], cos_sin, c);
  const uint4 y0 = pack8(v[0]), y1 = pack8(v[1]), y2 = pack8(v[2]);
  if (q) {
    uint4* const dst = reinterpret_cast<uint4*>(
        P.q_out + (token * P.H + t.part * kHeadsPerWarp + (lane >> 3)) * kDq);
    dst[c] = y0;
    dst[c + 8] = y1;
    dst[c + 16] = y2;
    return;
  }
  auto store = [&](uint4* dst) {
    dst[lane] = y0;
    dst[32 + lane] = y1;
    if (lane < 8) dst[64 + lane] = y2;
  };
  if (P.rows) store(P.rows + token * kChunks);
  if (P.cache) {
    const int at = t.first + t.i;
    const int page = P.block_table[static_cast<size_t>(t.b) * P.max_pages + at / kPage];
    if (page >= 0 && page < P.num_pages)
      store(P.cache + (static_cast<size_t>(page) * kPage + at % kPage) * kChunks);
    else if (lane == 0)
      record_status(P.status, MLA_STATUS_BOUNDS);
  }
}

// A list of the tokens: a warp takes tasks that follow each other, and has the next
// one's loads in flight.
template <bool kInterleaved>
__global__ void __launch_bounds__(kPrepThreads, kPrepCtas)
prep_list_kernel(const __grid_constant__ PrepParams P) {
  __shared__ UnitList list;
  wait_and_let_go(P);
  const int q_tasks = P.q ? P.H / kHeadsPerWarp : 0;
  const int per_token = q_tasks + (P.kv ? 1 : 0);
  const long long tasks =
      per_token * list.make(P.seq_lens, P.new_lens, P.max_new, P.max_len, P.B, P.status,
                            [](const NewTokens& nt) { return nt.len - nt.first; });
  const int warps = gridDim.x * (kPrepThreads / 32);
  const int w = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5);
  long long at = tasks * w / warps;
  const long long end = tasks * (w + 1) / warps;
  if (at >= end) return;
  Task t;
  {
    const long long token = at / per_token;
    t.part = static_cast<int>(at - token * per_token);
    t.b = list.find(token);
    t.first = list.first[t.b];
    t.i = static_cast<int>(token - (list.upto[t.b] - (list.len[t.b] - t.first)));
  }
  uint4 x[3];
  load_task(P, t, q_tasks, x);
#pragma unroll 1
  while (true) {
    const Task now = t;
    uint4 y[3] = {x[0], x[1], x[2]};
    const bool more = ++at < end;
    if (more) {
      if (++t.part == per_token) {
        t.part = 0;
        if (++t.i == list.len[t.b] - t.first) {
          t.b = list.find(list.upto[t.b]);  // (the next one with tokens)
          t.first = list.first[t.b];
          t.i = 0;
        }
      }
      load_task(P, t, q_tasks, x);
    }
    do_task<kInterleaved>(P, now, q_tasks, y);
    if (!more) break;
  }
}

// Every token that there may be, for single tokens and large batches of a few.
template <bool kInterleaved>
__global__ void __launch_bounds__(kPrepThreads, kPrepCtas)
prep_kernel(const __grid_constant__ PrepParams P) {
  wait_and_let_go(P);
  const int q_tasks = P.q ? P.H / kHeadsPerWarp : 0;
  const int per_token = q_tasks + (P.kv ? 1 : 0);
  const int tasks = P.B * P.max_new * per_token;
  const int warps = gridDim.x * (kPrepThreads / 32);
  for (int at = blockIdx.x * (kPrepThreads / 32) + (threadIdx.x >> 5); at < tasks; at += warps) {
    const int token = at / per_token;
    Task t;
    t.part = at - token * per_token;
    t.b = token / P.max_new;
    t.i = token - t.b * P.max_new;
    NewTokens nt;
    const bool report = t.i == 0 && t.part == 0 && (threadIdx.x & 31) == 0;
    if (!nt.load(P.seq_lens, P.new_lens, P.max_new, P.max_len, t.b, report, P.status) ||
        t.i >= nt.len - nt.first)
      continue;
    t.first = nt.first;
    uint4 x[3];
    load_task(P, t, q_tasks, x);
    do_task<kInterleaved>(P, t, q_tasks, x);
  }
}

}  // namespace

cudaError_t launch_prep(const mla_decode_norm_rope_args& a, const mla_decode_dims& d, int sm_count,
                        cudaStream_t st) {
  PrepParams P{};
  P.q = static_cast<const __nv_bfloat16*>(a.q);
  P.kv = static_cast<const __nv_bfloat16*>(a.kv);
  P.q_stride = a.q_stride;
  P.kv_stride = a.kv_stride;
  P.q_weight = static_cast<const __nv_bfloat16*>(a.q_weight);
  P.kv_weight = static_cast<const __nv_bfloat16*>(a.kv_weight);
  P.cos_sin = a.cos_sin;
  P.positions = a.positions;
  P.new_lens = a.new_lens;
  P.seq_lens = a.seq_lens;
  P.block_table = a.block_table;
  P.q_out = static_cast<__nv_bfloat16*>(a.q_out);
  P.rows = static_cast<uint4*>(a.rows);
  P.cache = static_cast<uint4*>(a.kv_cache);
  P.status = a.status;
  P.eps = a.eps;
  P.B = d.batch;
  P.H = d.num_heads;
  P.max_new = a.max_new;
  P.max_position = a.max_position;
  P.num_pages = d.num_pages;
  P.max_pages = d.max_pages_per_seq;
  P.max_len = d.max_pages_per_seq * kPage;
  const bool list = use_list(static_cast<int64_t>(P.B) * P.max_new, kListFrom, P.B, P.new_lens);
  const auto kern = list ? (a.interleaved ? prep_list_kernel<true> : prep_list_kernel<false>)
                         : (a.interleaved ? prep_kernel<true> : prep_kernel<false>);
  const int64_t tasks = static_cast<int64_t>(P.B) * P.max_new *
                        ((P.q ? P.H / kHeadsPerWarp : 0) + (P.kv ? 1 : 0));
  const int64_t ctas = (tasks + kPrepThreads / 32 - 1) / (kPrepThreads / 32);
  const int most = sm_count * kPrepCtas;
  return launch_pdl(kern, dim3(ctas < most ? static_cast<int>(ctas) : most), dim3(kPrepThreads),
                    0, st, P);
}

}  // namespace mla

// tokens.cuh -- what the kernels share that take each sequence's newest tokens (the
// appends, the page keys, reading back, norms and rotation).
#pragma once
#include "fp8kv.cuh"

namespace mla {

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

// The units (pages, tokens) of up to kListed sequences, one sequence's after the other's,
// as every CTA of a grid works them out for itself (at least kListed threads; `count`: a
// sequence's units).  Prompts of different lengths leave most of a padded grid empty; the
// list takes 1 us to make.  us with a list and without: norms and rotation (16 heads) of 13
// prompts of 512 to 8190 tokens 92 and 107, of 30 of 100 to 1000 32.0 and 35.8, of 8 of 4096
// 80.7 and 76.3, of 65 tokens of each 4.3 and 3.0; page keys: see launch_keys.
constexpr int kListed = 256;
struct UnitList {
  long long warp_sum[kListed / 32];
  long long upto[kListed];  // units up to and with the sequence's
  int first[kListed], len[kListed];

  template <typename Count>
  __device__ long long make(const int32_t* seq_lens, const int32_t* new_lens, int max_new,
                            int cap, int B, int32_t* status, const Count& count) {
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    long long n = 0;
    if (tid < kListed) {
      NewTokens nt{0, 0};
      if (tid < B &&
          nt.load(seq_lens, new_lens, max_new, cap, tid, blockIdx.x == 0, status))
        n = count(nt);
      first[tid] = nt.first;
      len[tid] = nt.len;
      for (int o = 1; o < 32; o <<= 1) {
        const long long v = __shfl_up_sync(0xffffffffu, n, o);
        if (lane >= o) n += v;
      }
      if (lane == 31) warp_sum[warp] = n;
    }
    __syncthreads();
    if (tid < kListed) {
      for (int w = 0; w < warp; ++w) n += warp_sum[w];
      upto[tid] = n;
    }
    __syncthreads();
    return upto[kListed - 1];
  }
  // The sequence of a unit below the total.
  __device__ int find(long long unit) const {
    int b = 0;
    for (int step = kListed / 2; step; step >>= 1)
      if (upto[b + step - 1] <= unit) b += step;
    return b;
  }
};
// Worth it where lengths may differ and the padded grid is large.
inline bool use_list(int64_t padded, int64_t from, int B, const int32_t* new_lens) {
  return new_lens && B > 1 && B <= kListed && padded >= from;
}

// Pages that max_new consecutive tokens can touch.
inline int touched_pages(int max_new, int max_pages) {
  const int most = (max_new + kPage - 2) / kPage + 1;
  return most < max_pages ? most : max_pages;
}

}  // namespace mla

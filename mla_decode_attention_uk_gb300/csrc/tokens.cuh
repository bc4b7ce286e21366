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

// Pages that max_new consecutive tokens can touch.
inline int touched_pages(int max_new, int max_pages) {
  const int most = (max_new + kPage - 2) / kPage + 1;
  return most < max_pages ? most : max_pages;
}

}  // namespace mla

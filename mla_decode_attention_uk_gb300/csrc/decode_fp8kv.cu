// decode_fp8kv.cu -- the attention step over the 8-bit latent cache.
//
// The cache holds E4M3 codes and one scale s per page (fp8kv.cuh).  With the
// absorbed query q and codes c_j of a page:
//   x_j   = scale log2(e) s (q . c_j)        p_j = 2^(x_j - m)
//   o_lat = sum_j (p_j s) c_j[0:512] / sum_j p_j,   lse = (m + log2 sum p_j) ln 2
// Split-KV ranges, the plan, the merge of partial results and the lse's
// first-order correction are those of the bf16 cache's step (decode.cu).
//
// GB300 mapping: both products run on the 8-bit tensor-core path (kind::f8f6f4,
// K = 32 per instruction), so the codes go from memory to the tensor core as
// they are, half the bytes of a bf16 page at every level.  What the other
// operand loses in 8 bits is given back by a second term:
//   * Q = scale_row (hi + mid / 16), both E4M3: hi is the value cut to four
//     significant bits, mid the rest times 16.  A bf16 value has eight and the
//     two terms hold it exactly (down to 2^-13 of the row's largest value; smaller
//     ones to 2^-19 of that), so the product is that of the bf16 query.  The terms
//     are stacked as the M = 128 rows of one MMA: the full rate of the tensor
//     core for 64 query rows, where a 64-row MMA would run at half of it.  The
//     512 latent columns of the terms live in TMEM (128 columns), so that QK^T
//     reads only the page from shared memory (32 cycles an MMA instead of 48),
//     and the 64 KB that they would take there hold two more pages.
//   * P = hi + mid, both E5M2, the upper bytes of fp16: as both accumulate into
//     the same columns they cannot have scales of their own, and E5M2's range
//     (2^-16 to 2^15) keeps the small weights of a long context next to a large
//     one, which E4M3's would drop.  Two terms leave at most 2^-7 of a weight;
//     the row is divided by the sum of the weights as rounded, so a rounding
//     that all weights share cancels, and the lse takes the unrounded sum.
// Per page and 64 query rows: QK^T 18 MMAs of 128 x 64 x 32, PV 16 of 128 x N x 32
// (N: the tile's rows; O^T = C^T P^T, M = 128 latent columns).  A page comes in two
// copies into a ring of five 40 KB slots; a piece's query tile passes through
// two of them on its way to the terms.  The softmax runs on TMEM rows with a
// running maximum that is raised lazily, P^T goes into the page's RoPE box, O^T
// stays in TMEM.  The page's scale joins the exponent (p_j s = 2^(x_j + log2 s -
// m), m the running maximum of that sum), so that P never leaves E5M2's range
// however the scales of a sequence's pages differ.
//
// Warp roles: 0 TMA producer, 1 QK^T issuer, 2 and 3 PV issuers (latent halves;
// warp 2 also owns TMEM), 4-7 and 8-11 softmax and epilogue, 12-15 query terms.
// The two softmax groups take turns, page by page: a page's chain of waits,
// exponentials and stores is about 1,700 cycles long however many warps share
// it (measured with four and with eight), while the tensor core is done in
// 1,400, so two pages are in work at once.  They share the rows' running
// maxima: a group looks at a row's maximum once the other is through with it
// for the page before, and the sums, which each keeps for itself, follow it.
// (QK^T has one issuer: two that took turns would each see only some phases of a
// slot's barriers.)
//
// What bounds it: with 64 rows the tensor pipe, whose 34 MMAs take 1,376 cycles of
// the 1,500 that a page takes (PV 768, bound by shared-memory reads: 6 KB per
// MMA of 4 KB worth); with 16 heads memory, 6.1 TB/s while pages stream (both from
// time stamps on one SM).  Beside the pages a piece costs 5 to 6 us (its query
// terms and its epilogue are not hidden by each other's pages) and a launch 8 us:
// over the whole launch the tensor pipe is active 51 % of the time on the second
// case below and 42 % on the third, and DRAM at 51 % of its peak on the first.
// Measured (one GB300, with the query terms' tile, without absorb and merge): 64
// sequences of 4,096 tokens x 16 heads 36 us; 128 of 1,000-10,000 (500k tokens) x
// 128 heads 113 us; 61 ragged drafts of 4 queries x 128 heads (133k tokens) 101 us.
// Prefetching pages into L2 ahead of the ring only cost: 35 -> 39 us on the first,
// eight pages ahead.
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>

#include "common.cuh"
#include "fp8kv.cuh"
#include "ptx.cuh"

namespace mla {

int decode_q_box_rows(int T, int H);

namespace {

constexpr int kThreads = 512;                     // 16 warps
constexpr int kBox = kPage * 128;                 // 64 keys x 128 codes: 8 KB
constexpr int kSlot = kBoxes8 * kBox;             // 40 KB (the last box half empty)
constexpr int kSlots = 5;
constexpr int kSBufs = 2;                         // S buffers of 64 columns
constexpr int kRopeBox8 = kBoxes8 - 1;
constexpr int kSmemBytes = 1024 + kQBox8 + kSlots * kSlot;
constexpr uint32_t kTmemAll = 512;
constexpr uint32_t kTmemQ = 128;                  // the query's latent terms: 128 columns
constexpr uint32_t kTmemOut = 256;                // O^T blocks at 256 + 64 m
constexpr float kRaise = 8.0f;                    // log2 units
// The running maximum's weight is 2^kTopExp; it may grow by 2^kRaise before
// the maximum is raised, to 2^15 (E5M2 ends at 1.75 * 2^15).
constexpr float kTopExp = 7.0f;
// Weights from here on count as rounded in the row's normalising sum.  Smaller
// ones count as they are: near the end of E5M2's range their rounding is no
// longer small against them, and in a page of a small scale such weights may
// make up the sum while they add nothing to the output.
constexpr float kRoundedFrom = 1.0f / 512.0f;
constexpr float kLn2 = 0.6931471805599453f;

struct Params {
  const int32_t* block_table;
  const float* kv_scale;
  const int32_t* seq_len_eff;
  const PlanHeader* header;
  uint8_t* ws;
  const int32_t* seq_first;
  const int32_t* seq_nsplit;
  const int32_t* seq_slot;
  __nv_bfloat16* olat;
  float* lse;
  int32_t* status;
  int B, T, H, max_pages, num_pages;
  int tpg, sets, q_box_rows;
  float scale_log2;
};
// What depends on the plan's number of ranges, found out on the device.  (In
// shared memory, as every thread would hold it in registers else.)
struct PlanView {
  const int32_t* range_b;
  const int32_t* range_p;
  __nv_bfloat16* opart;
  float* lpart;
  int tasks;  // ranges * sets
};

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}

// Two fp32 values to two E5M2 codes in the high bytes of an fp16 pair: E5M2 is
// fp16's upper byte, so rounding is an addition and a mask (ties away from
// zero; |x| <= 2^15 and its rounding stay finite).
__device__ __forceinline__ __half2 e5m2_in_half2(__half2 x) {
  const uint32_t u = *reinterpret_cast<const uint32_t*>(&x);
  const uint32_t r = (u + 0x00800080u) & 0xff00ff00u;
  return *reinterpret_cast<const __half2*>(&r);
}
__device__ __forceinline__ uint32_t bits(__half2 x) { return *reinterpret_cast<uint32_t*>(&x); }

struct Piece {
  int task, b, pbeg, pend, len;
};

// The pieces (sequence, page range) of a CTA's tasks v = v0, v0 + groups, ...,
// in the order that all roles walk.  Task v is work range v / sets.
// (Few fields: every thread of the kernel has one.)
struct Pieces {
  int v, b, p, b1, p1;
  __device__ Pieces(const Params& P, const PlanView& V, int v0) : v(v0) { open(P, V); }
  __device__ void open(const Params& P, const PlanView& V) {
    if (v >= V.tasks) return;
    const int k = v / P.sets;
    b = V.range_b[k];
    p = V.range_p[k];
    b1 = V.range_b[k + 1];
    p1 = V.range_p[k + 1];
  }
  __device__ bool next(const Params& P, const PlanView& V, Piece& out) {
    while (v < V.tasks) {
      if (b < b1 || (b == b1 && p < p1)) {  // (never empty: a range starts inside a sequence)
        const int L = P.seq_len_eff[b];
        const int end = b == b1 ? p1 : (L + kPage - 1) / kPage;
        out = Piece{v, b, p, end, L};
        ++b;
        p = 0;
        return true;
      }
      v += gridDim.x / P.tpg;
      open(P, V);
    }
    return false;
  }
};

__global__ void __launch_bounds__(kThreads, 1)
decode_fp8kv_kernel(const __grid_constant__ CUtensorMap tm_lat,
                    const __grid_constant__ CUtensorMap tm_rope,
                    const __grid_constant__ CUtensorMap tm_q, Params P) {
  extern __shared__ uint8_t smem_raw[];
  // By slot: slot_full, a page has landed; slot_free, PV has read it and its P^T,
  // or the query terms are made of the tile that was there.
  // p_full[g mod kSlots]: P^T of page g is written (a page kSlots further on
  // is not in a slot before PV has read this one).
  // pv_done[g mod kSlots]: PV of page g is complete.  (slot_free does not tell a
  // softmax group: a query tile's release is one more of its phases, which may
  // come before the group has looked, and a parity then means another phase.  A
  // next phase here takes PV of page g + kSlots, which follows that of page g +
  // 1, the group's own.  The phase before is over: page g + 1 is in a slot, so PV
  // has read every page up to g + 1 - kSlots.)
  __shared__ __align__(8) uint64_t q_full, q_free, slot_full[kSlots], slot_free[kSlots],
      s_full[kSBufs], s_free[kSBufs], p_full[kSlots], pv_done[kSlots], q_raw, o_full, o_free,
      m_final[2][4], sums_full, epi_done, drain_bar[3];
  __shared__ PlanView view;
  __shared__ uint32_t tmem_base_sh;
  __shared__ int abort_sh;
  __shared__ float page_scale_sh[kSlots], q_scale_sh[kTileRows];
  __shared__ float alpha_sh[2][kTileRows], m_sh[kTileRows];
  __shared__ __align__(16) float inv_sh[8][kTileRows];
  __shared__ float l_sh[2][kTileRows], l_r_sh[2][kTileRows], m_l_sh[2][kTileRows];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // Tasks v = range * sets + set are dealt round robin to groups of tpg CTAs;
  // a group's CTA ti takes tile set * tpg + ti (as in decode.cu).
  const int tpg = P.tpg, sets = P.sets;
  const int ti = blockIdx.x % tpg, gi = blockIdx.x / tpg;
  const int TH = P.T * P.H;
  const uint32_t sQ = (smem_u32(smem_raw) + 1023u) & ~1023u;
  const uint32_t sSlot0 = sQ + kQBox8;

  if (threadIdx.x == 0) {
    mbar_init(smem_u32(&q_full), 12);
    mbar_init(smem_u32(&q_free), 1 + 8);  // QK^T, and the softmax warps (the rows' scales)
    for (int i = 0; i < kSlots; ++i) {
      mbar_init(smem_u32(&slot_full[i]), 1);
      mbar_init(smem_u32(&slot_free[i]), 2);
      mbar_init(smem_u32(&p_full[i]), 4);
      mbar_init(smem_u32(&pv_done[i]), 2);
    }
    mbar_init(smem_u32(&q_raw), 1);
    for (int i = 0; i < kSBufs; ++i) {
      mbar_init(smem_u32(&s_full[i]), 1);
      mbar_init(smem_u32(&s_free[i]), 4);
    }
    mbar_init(smem_u32(&o_full), 2);
    mbar_init(smem_u32(&o_free), 8);
    mbar_init(smem_u32(&sums_full), 8);
    mbar_init(smem_u32(&epi_done), 8);
    for (int i = 0; i < 8; ++i) mbar_init(smem_u32(&m_final[i >> 2][i & 3]), 1);
    for (int i = 0; i < 3; ++i) mbar_init(smem_u32(&drain_bar[i]), 1);
    abort_sh = 0;
    fence_mbar_init();
    tma_prefetch_desc(&tm_lat);
    tma_prefetch_desc(&tm_rope);
    tma_prefetch_desc(&tm_q);
  }
  griddep_wait();
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    const int R = P.header->num_ranges;
    const WsLayout L = make_layout(P.B, P.T, P.H, R);
    view.range_b = reinterpret_cast<const int32_t*>(P.ws + L.range_b);
    view.range_p = reinterpret_cast<const int32_t*>(P.ws + L.range_p);
    view.lpart = reinterpret_cast<float*>(P.ws + L.lpart);
    view.opart = reinterpret_cast<__nv_bfloat16*>(P.ws + L.opart);
    view.tasks = R * P.sets;
  }
  if (warp == 2) {
    tmem_alloc(smem_u32(&tmem_base_sh), kTmemAll);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = tmem_base_sh;
  Pieces walk(P, view, gi);
  Piece pc;

  if (warp == 0) {
    // ------------------------------------------------------------ producer
    // Lane 0 issues the copies.  The lanes look pages and scales up 32 at a
    // time, a block ahead, so that those dependent loads are off the path from
    // a free box to its copy (looked up page by page they bounded the kernel,
    // at 1,700 cycles a page, together with eight more copies and prefetches).
    int ring = 0, n = 0;  // slots filled, pieces
    bool ok = true;
    while (ok && walk.next(P, view, pc)) {
      const int nc = pc.pend - pc.pbeg;
      const int32_t* row = P.block_table + static_cast<size_t>(pc.b) * P.max_pages + pc.pbeg;
      int pg = 0, pg_next = 0;
      float sc = 1.0f, sc_next = 1.0f;
      auto look = [&](int i, int& page, float& scale) {
        if (i >= nc) return;
        page = __ldg(row + i);
        if (page < 0 || page >= P.num_pages) {
          record_status(P.status, MLA_STATUS_BOUNDS);
          page = 0;
        }
        scale = P.kv_scale[page];
        if (!scale_in_range(scale)) {
          record_status(P.status, MLA_STATUS_BOUNDS);
          scale = 1.0f;
        }
      };
      // The query tile comes first, through two slots.
      if (lane == 0) {
        const int row = pc.b * TH + ((pc.task % sets) * tpg + ti) * kTileRows;
        // (One tile at a time: the last one's terms are made, so its barrier's
        // phase is over and seen.)
        ok = n == 0 || mbar_wait(smem_u32(&q_full), (n - 1) & 1, &abort_sh, P.status);
        for (int r = ring; r < ring + 2 && ok; ++r)
          ok = r < kSlots || mbar_wait(smem_u32(&slot_free[r % kSlots]), (r / kSlots - 1) & 1,
                                       &abort_sh, P.status);
        if (ok) {
          // (Every fill of a slot is a phase of its barrier.)
          mbar_arrive(smem_u32(&slot_full[ring % kSlots]));
          mbar_arrive(smem_u32(&slot_full[(ring + 1) % kSlots]));
          mbar_expect_tx(smem_u32(&q_raw), kBoxes * P.q_box_rows * 128);
          for (int j = 0; j < kBoxes; ++j)
            tma_load_2d(sSlot0 + ((ring + j / kBoxes8) % kSlots) * kSlot + (j % kBoxes8) * kBox,
                        &tm_q, j * kBoxCols, row, smem_u32(&q_raw));
        }
      }
      ok = __shfl_sync(0xffffffffu, ok, 0);
      if (!ok) break;
      ring += 2;
      ++n;
      look(lane, pg_next, sc_next);
      for (int i = 0; i < nc; ++i, ++ring) {
        if ((i & 31) == 0) {
          pg = pg_next;
          sc = sc_next;
          look(i + 32 + lane, pg_next, sc_next);
        }
        const int page = __shfl_sync(0xffffffffu, pg, i & 31);
        const float scale = __shfl_sync(0xffffffffu, sc, i & 31);
        if (lane == 0) {
          const int s = ring % kSlots, u = ring / kSlots;
          ok = u == 0 || mbar_wait(smem_u32(&slot_free[s]), (u - 1) & 1, &abort_sh, P.status);
          if (ok) {
            // (The softmax is done with the slot's last page: PV followed it.)
            *static_cast<volatile float*>(&page_scale_sh[s]) = scale;
            const uint32_t fb = smem_u32(&slot_full[s]), dst = sSlot0 + s * kSlot;
            mbar_expect_tx(fb, kSlot);
            tma_load_3d(dst, &tm_lat, 0, page * kPage, 0, fb);
            tma_load_2d(dst + kRopeBox8 * kBox, &tm_rope, kLora, page * kPage, fb);
          }
        }
        ok = __shfl_sync(0xffffffffu, ok, 0);
        if (!ok) break;
      }
    }
    if (lane == 0) {
      // Every copy lands before the CTA exits, after an abort too.
      if (n > 0) mbar_wait_drain(smem_u32(&q_raw), (n - 1) & 1, P.status);
      for (int s = 0; s < kSlots; ++s) {
        const int k = (ring - s + kSlots - 1) / kSlots;  // fills of slot s
        if (k > 0) mbar_wait_drain(smem_u32(&slot_full[s]), (k - 1) & 1, P.status);
      }
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ MMA issuers
    if (elect_one()) {
      const uint64_t dq0 = sdesc_sw128(sQ, 16, 1024);
      const uint64_t dslot0 = sdesc_sw128(sSlot0, 16, 1024);
      const uint64_t dpv0 = sdesc_sw128(sSlot0, kBox, 1024);
      int g = 0, n = 0;
      bool ok = true;
      if (warp == 1) {
        constexpr uint32_t idesc = idesc_f8_f32(kQTermRows, kPage, 0, 0, false, false);
        while (ok && walk.next(P, view, pc)) {
          if (!mbar_wait(smem_u32(&q_full), n & 1, &abort_sh, P.status)) break;
          tc_fence_after();
          for (int i = pc.pbeg; i < pc.pend; ++i, ++g) {
            const int ring = g + 2 * (n + 1), s = ring % kSlots, sb = g % kSBufs;
            if (g >= kSBufs && !mbar_wait(smem_u32(&s_free[sb]), (g / kSBufs - 1) & 1, &abort_sh,
                                          P.status)) {
              ok = false;
              break;
            }
            if (!mbar_wait(smem_u32(&slot_full[s]), (ring / kSlots) & 1, &abort_sh, P.status)) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t bd = dslot0 + static_cast<uint64_t>((s * kSlot) >> 4);
#pragma unroll
            for (int kk = 0; kk < kLora / 32; ++kk)  // four steps to a box
              umma_f8_ta(tmem + 64 * sb, tmem + kTmemQ + 8 * kk,
                         bd + (((kk >> 2) * kBox) >> 4) + (kk & 3) * 2, idesc, kk != 0);
#pragma unroll
            for (int kk = 0; kk < kRope / 32; ++kk)
              umma_f8(tmem + 64 * sb, dq0 + kk * 2, bd + ((kRopeBox8 * kBox) >> 4) + kk * 2, idesc,
                      1);
            umma_commit(smem_u32(&s_full[sb]));
          }
          if (!ok) break;
          umma_commit(smem_u32(&q_free));
          ++n;
        }
      } else {
        const int half = warp - 2;
        while (ok && walk.next(P, view, pc)) {
          const int tile = (pc.task % sets) * tpg + ti;
          const int nrows = min(kTileRows, (TH - tile * kTileRows + 15) & ~15);
          const uint32_t idesc = idesc_f8_f32(128, nrows, 0, 1, true, false);
          for (int i = pc.pbeg; i < pc.pend; ++i, ++g) {
            const int s = (g + 2 * (n + 1)) % kSlots;
            const bool first = i == pc.pbeg;
            if (!mbar_wait(smem_u32(&p_full[g % kSlots]), (g / kSlots) & 1, &abort_sh, P.status) ||
                (first && n > 0 &&
                 !mbar_wait(smem_u32(&o_free), (n - 1) & 1, &abort_sh, P.status))) {
              ok = false;
              break;
            }
            tc_fence_after();
            const uint64_t ad0 = dpv0 + static_cast<uint64_t>((s * kSlot) >> 4);
            const uint64_t bd0 =
                dslot0 + static_cast<uint64_t>((s * kSlot + kRopeBox8 * kBox) >> 4);
#pragma unroll
            for (int m = 2 * half; m < 2 * half + 2; ++m) {
              // Steps 0, 1: the hi terms of keys 0-31 and 32-63; 2, 3: mid.
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                umma_f8(tmem + kTmemOut + 64 * m, ad0 + ((m * kBox + (kk & 1) * 4096) >> 4),
                        bd0 + kk * 2, idesc, !(first && kk == 0));
            }
            umma_commit(smem_u32(&pv_done[g % kSlots]));
            umma_commit(smem_u32(&slot_free[s]));
          }
          if (!ok) break;
          umma_commit(smem_u32(&o_full));
          ++n;
        }
      }
      const uint32_t db = smem_u32(&drain_bar[warp - 1]);
      umma_commit(db);
      mbar_wait_drain(db, 0, P.status);
    }
  } else {
    // ------------------------------------------------------------ query terms
    // Warps 12-15 turn the query tile into its terms, warp 12 + w tile rows 16 w
    // .. + 15, between the end of a piece's QK^T and that of its epilogue.  (A
    // kernel of its own took 3 to 14 us; the softmax warps' help, between their
    // last page and the epilogue, made the step slower: 138 -> 144 us on 128
    // sequences x 128 heads; making the terms in place before QK^T's end and
    // copying them after it too: 146.)  A CTA's first piece waits for its terms,
    // so all twelve warps make them.
    //
    // Lane layout of TMEM loads and stores of 16 lanes x 64 bits: this thread has
    // row rig of the quarter's 16, and the words (four codes) or keys of parity
    // par.
    const int wq = warp & 3;
    const uint32_t lane_off = static_cast<uint32_t>(wq * 32) << 16;
    const int rig = (lane >> 2) + 8 * (lane & 1);
    const int par = (lane >> 1) & 1;
    const int srow = 16 * wq + rig;
    const bool softmax = warp < 12;
    int g = 0, n = 0;
    bool fail = false;
    bool have = walk.next(P, view, pc);
    while (!fail && have) {
      if (n == 0 || !softmax) {
        // Where columns 64 block + 8 j + 4 half .. + 3 of a row are: four bf16
        // values, or in their place a word of hi codes and one of mid codes.
        auto word = [&](int row, int block, int j, int half) {
          const int ring = g + 2 * n + (block >= kBoxes8 ? 1 : 0);
          return sSlot0 + (ring % kSlots) * kSlot + (block % kBoxes8) * kBox + row * 128 +
                 ((j ^ (row & 7)) << 4) + 8 * half;
        };
        const int rows_here = min(kTileRows, TH - ((pc.task % sets) * tpg + ti) * kTileRows);
        bool ok = mbar_wait(smem_u32(&q_raw), n & 1, &abort_sh, P.status);
        int e = 0;
        float amax = 0.0f;
        if (n == 0) {
          // All warps share the rows out, whatever TMEM lanes they belong to (16
          // heads would leave three quarters of the SM idle else), and make the
          // terms in place.
          for (int row = warp - 4; row < rows_here; row += 12) {
            uint2 x[5];  // words lane, lane + 32, ... of the row's 144
            __nv_bfloat162 top = __float2bfloat162_rn(0.0f);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int w = lane + 32 * i;
              x[i] = make_uint2(0u, 0u);
              if (i < 4 || lane < 16) x[i] = ld_shared_v2(word(row, w >> 4, (w >> 1) & 7, w & 1));
              top = max_abs(max_abs(top, x[i].x), x[i].y);
            }
            const float amax =
                __uint_as_float(__reduce_max_sync(0xffffffffu, larger_half(top)));
            const int er = term_exp(amax);
            const __nv_bfloat162 down = term_factor(er);
            if (er > kTermExpMax)
#pragma unroll
              for (int i = 0; i < 5; ++i) x[i] = lower_terms(x[i], er);
            if (lane == 0) q_scale_sh[row] = row_scale(amax, er);
#pragma unroll
            for (int i = 0; i < 5; ++i) {
              const int w = lane + 32 * i;
              uint32_t hi, mid;
              split_terms(x[i], down, hi, mid);
              if (i < 4 || lane < 16) st_shared_v2(word(row, w >> 4, (w >> 1) & 7, w & 1), hi, mid);
            }
          }
          // (Here and below warps that share a named barrier leave together, or the
          // others would wait there for one that has given up.)
          __syncwarp();
          ok = !bar_any(3, 384, !ok);
        } else {
          __nv_bfloat162 top = __float2bfloat162_rn(0.0f);
#pragma unroll 1
          for (int block = 0; block < kBoxes; ++block)
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const uint2 x = ld_shared_v2(word(srow, block, j, par));
              top = max_abs(max_abs(top, x.x), x.y);
            }
          const uint32_t t = larger_half(top);
          amax = __uint_as_float(max(t, __shfl_xor_sync(0xffffffffu, t, 2)));
          e = term_exp(amax);
          // A loop of its own, as it is rare (rows past the last hold anything).
          const bool lower = srow < rows_here && e > kTermExpMax;
          if (__any_sync(0xffffffffu, lower))
#pragma unroll 1
            for (int w = 0; w < 8 * kBoxes; ++w) {
              const uint32_t at = word(srow, w >> 3, w & 7, par);
              if (lower) {
                const uint2 x = lower_terms(ld_shared_v2(at), e);
                st_shared_v2(at, x.x, x.y);
              }
            }
          ok = ok && mbar_wait(smem_u32(&q_free), (n - 1) & 1, &abort_sh, P.status);
        }
        const __nv_bfloat162 down = term_factor(e);
        if (!__all_sync(0xffffffffu, ok)) break;
        tc_fence_after();
        if (par == 0 && n > 0) q_scale_sh[srow] = row_scale(amax, e);
        const int b0 = n == 0 ? 3 * ((warp - 4) >> 2) : 0, b1 = n == 0 ? b0 + 3 : kBoxes;
#pragma unroll 1
        for (int block = b0; block < b1; ++block) {
          uint32_t hi[8], mid[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const uint2 x = ld_shared_v2(word(srow, block, j, par));
            hi[j] = x.x;
            mid[j] = x.y;
          }
          if (n > 0)
#pragma unroll
            for (int j = 0; j < 8; ++j)
              split_terms(make_uint2(hi[j], mid[j]), down, hi[j], mid[j]);
          if (block < kLatBoxes) {
            const uint32_t ta = tmem + lane_off + kTmemQ + 16 * block;
            tmem_st_16x64b_x8(ta, hi);
            tmem_st_16x64b_x8(ta + (16u << 16), mid);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) {  // word 2 j + par (row + 16: the same swizzle)
              const uint32_t a = sQ + (32 * wq + rig) * 128 +
                                 (((j >> 1) ^ (rig & 7)) << 4) + 8 * (j & 1) + 4 * par;
              st_shared_b32(a, hi[j]);
              st_shared_b32(a + 16 * 128, mid[j]);
            }
          }
        }
        tmem_wait_st();
        tc_fence_before();
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive_n(smem_u32(&q_full), n == 0 ? 1 : 3);
        if (!softmax) {
          // Everyone is done with the tile: its slots are free.
          if (warp == 12 && !mbar_wait(smem_u32(&q_full), n & 1, &abort_sh, P.status)) break;
          if (threadIdx.x == 12 * 32) {
            mbar_arrive_n(smem_u32(&slot_free[(g + 2 * n) % kSlots]), 2);
            mbar_arrive_n(smem_u32(&slot_free[(g + 2 * n + 1) % kSlots]), 2);
          }
          g += pc.pend - pc.pbeg;
          ++n;
          have = walk.next(P, view, pc);
          continue;
        }
      }
      // ---------------------------------------------------------- softmax + epilogue
      // Two groups of four warps take turns: group q has the pages g with g mod 2
      // = q, and S buffer q.  A warp has the rows of its TMEM lane quarter; this
      // thread row srow of the tile (its hi term in lane rig of the quarter, its
      // mid term in lane 16 + rig) and keys of parity par.
      const int q = (warp - 4) >> 2;
      const bool owner = par == 0;
      const int row0 = ((pc.task % sets) * tpg + ti) * kTileRows;  // of the sequence's T * H
      const int rows_here = min(kTileRows, TH - row0);
      // Where the rows' results go: row of o_lat, or ~row of the partial results.
      const int dest = P.seq_nsplit[pc.b] > 1
                           ? ~((P.seq_slot[pc.b] + pc.task / sets - P.seq_first[pc.b]) * TH + row0)
                           : pc.b * TH + row0;
      const int n_row = srow < rows_here ? pc.len - P.T + (row0 + srow) / P.H + 1 : 0;
      // The running maximum of a row is m_sh (one group raises it, the other
      // finds it raised); m_mine is the one that this thread's sums are in.
      float m_mine = -INFINITY;
      // The last piece's epilogue has read m_sh and the sums; the query is there.
      bool bad = (n > 0 && !mbar_wait(smem_u32(&epi_done), (n - 1) & 1, &abort_sh, P.status)) ||
                 !mbar_wait(smem_u32(&q_full), n & 1, &abort_sh, P.status);
      const float q_scale = q_scale_sh[srow] * P.scale_log2;
      // This thread's shares of the row's sums: exact, as rounded.  NaN from the
      // start where the query is not finite, whatever its codes give.
      float l = 0.0f * q_scale, l_r = l;
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&q_free));
      for (int i = pc.pbeg; i < pc.pend; ++i, ++g) {
        if ((g & 1) != q) continue;
        const int ring = g + 2 * (n + 1), s = ring % kSlots;
        // (The page has landed, QK^T has read it; its barrier orders the
        // producer's page_scale_sh.)
        bad = bad || !mbar_wait(smem_u32(&s_full[q]), (g >> 1) & 1, &abort_sh, P.status) ||
              !mbar_wait(smem_u32(&slot_full[s]), (ring / kSlots) & 1, &abort_sh, P.status);
        bad = __any_sync(0xffffffffu, bad);
        const float page_scale = *static_cast<volatile float*>(&page_scale_sh[s]);
        uint32_t v[32];  // v[j]: key kb + 2 j
        if (!bad) {
          tc_fence_after();
          tmem_ld_16x64b_x32(tmem + lane_off + 64 * q, v);
#pragma unroll
          for (int h = 0; h < 2; ++h) {  // (in halves for the registers)
            uint32_t v2[16];
            tmem_ld_16x64b_x16(tmem + lane_off + (16u << 16) + 64 * q + 32 * h, v2);
            tmem_wait_ld();
#pragma unroll
            for (int j = 0; j < 16; ++j)
              v[16 * h + j] = __float_as_uint(fmaf(__uint_as_float(v2[j]), 1.0f / kQMidScale,
                                                   __uint_as_float(v[16 * h + j])));
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&s_free[q]));
        const int kb = i * kPage + par;
        if (kb + 62 >= n_row) {
#pragma unroll
          for (int j = 0; j < 32; ++j)
            if (kb + 2 * j >= n_row) v[j] = __float_as_uint(-INFINITY);
        }
        float a3[11];
#pragma unroll
        for (int t = 0; t < 10; ++t)
          a3[t] = max3(__uint_as_float(v[3 * t]), __uint_as_float(v[3 * t + 1]),
                       __uint_as_float(v[3 * t + 2]));
        a3[10] = fmaxf(__uint_as_float(v[30]), __uint_as_float(v[31]));
        float vmax = fmaxf(max3(max3(a3[0], a3[1], a3[2]), max3(a3[3], a3[4], a3[5]),
                                max3(a3[6], a3[7], a3[8])),
                           fmaxf(a3[9], a3[10]));
        vmax = fmaxf(vmax, __shfl_xor_sync(0xffffffffu, vmax, 2));
        // Not zero, so that a hidden key's -inf times it stays -inf (a
        // product below 2^-100 is 0 to the exponent either way).
        const float mul = fmaxf(q_scale * page_scale, 7.9e-31f);
        const float shift = __log2f(page_scale);
        const float pmax = fmaf(vmax, mul, shift);
        // The page before, the other group's, is through with the maximum.
        if (g > 0)
          bad = !mbar_wait(smem_u32(&m_final[q ^ 1][wq]), ((g - 1) >> 1) & 1, &abort_sh,
                           P.status) || bad;
        const bool first = i == pc.pbeg;
        const float m_old = first ? -INFINITY : m_sh[srow];
        const bool raise = pmax > m_old + kRaise;
        const float m_used = raise ? pmax : m_old;
        __syncwarp();
        if (owner && (raise || first)) m_sh[srow] = m_used;
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&m_final[q][wq]));
        if (m_used != m_mine) {
          const float f = ex2_approx(m_mine - m_used);
          l *= f;
          l_r *= f;
          m_mine = m_used;
        }
        // One barrier of the group per page: a raised maximum (the group then
        // rescales O^T, rows are its columns), or a wait that gave up.
        if (bar_any(1 + q, 128, bad || (raise && !first))) {
          bool f = *static_cast<volatile int*>(&abort_sh) != 0;
          if (owner) alpha_sh[q][srow] = raise ? ex2_approx(m_old - pmax) : 1.0f;
          if (!f && !first &&
              !mbar_wait(smem_u32(&pv_done[(g - 1) % kSlots]), ((g - 1) / kSlots) & 1, &abort_sh,
                         P.status))
            f = true;
          if (bar_any(1 + q, 128, f)) { fail = true; break; }
          if (!first) {
            tc_fence_after();
#pragma unroll 1
            for (int m = 0; m < 4; ++m) {
#pragma unroll 1
              for (int h2 = 0; 16 * h2 < rows_here; ++h2) {
                uint32_t vv[16];
                const uint32_t ta = tmem + lane_off + kTmemOut + 64 * m + 16 * h2;
                tmem_ld_x16(ta, vv);
                tmem_wait_ld();
#pragma unroll
                for (int j = 0; j < 16; ++j)
                  vv[j] = __float_as_uint(__uint_as_float(vv[j]) * alpha_sh[q][16 * h2 + j]);
                tmem_st_x16(ta, vv);
              }
            }
            tmem_wait_st();
            tc_fence_before();
          }
        }
        // Codes are the upper bytes of fp16 pairs, four to a word.
        uint32_t hw[8], mw[8];
        if (m_used == -INFINITY) {
#pragma unroll
          for (int t = 0; t < 8; ++t) hw[t] = mw[t] = 0u;
          // No key yet, or NaN alone, which a maximum passes over.
          if (kb < n_row) l = l_r = __uint_as_float(0x7fffffffu);
        } else {
          const float add = shift + kTopExp - m_used;
          float se[4] = {};
          // What the rounding of this thread's 32 weights adds up to, in fp16: the
          // terms are exact and at most 2^-7 of a weight, so 16 sums rounded by
          // 2^-11 move the row's sum, which is fp32, by 2^-14 of it at most.
          __half2 err = __float2half2_rn(0.0f);
#pragma unroll
          for (int t = 0; t < 8; ++t) {
            uint32_t hb[2], mb[2];
#pragma unroll
            for (int j = 2 * t; j < 2 * t + 2; ++j) {
              const float p0 = ex2_approx(fmaf(__uint_as_float(v[2 * j]), mul, add));
              const float p1 = ex2_approx(fmaf(__uint_as_float(v[2 * j + 1]), mul, add));
              se[(2 * j) & 3] += p0;
              se[(2 * j + 1) & 3] += p1;
              const __half2 h = __floats2half2_rn(p0, p1);
              const __half2 hi = e5m2_in_half2(h);
              const __half2 mid = e5m2_in_half2(__hsub2(h, hi));
              err = __hfma2(__hsub2(__hadd2(hi, mid), h),
                            __hge2(h, __float2half2_rn(kRoundedFrom)), err);
              hb[j & 1] = bits(hi);
              mb[j & 1] = bits(mid);
            }
            hw[t] = __byte_perm(hb[0], hb[1], 0x7531);
            mw[t] = __byte_perm(mb[0], mb[1], 0x7531);
          }
          const float sum = (se[0] + se[1]) + (se[2] + se[3]);
          const float2 e = __half22float2(err);
          const float inv_scale = __frcp_rn(page_scale);
          l = fmaf(sum, inv_scale, l);
          l_r = fmaf(sum + (e.x + e.y), inv_scale, l_r);
        }
        // The even-key thread writes keys 0-31, the odd-key thread keys 32-63:
        // half of each thread's codes cross to its partner.
        uint32_t ph[8], pm[8];
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const uint32_t keep_h = par ? hw[4 + t] : hw[t], keep_m = par ? mw[4 + t] : mw[t];
          const uint32_t got_h = __shfl_xor_sync(0xffffffffu, par ? hw[t] : hw[4 + t], 2);
          const uint32_t got_m = __shfl_xor_sync(0xffffffffu, par ? mw[t] : mw[4 + t], 2);
          const uint32_t eh = par ? got_h : keep_h, oh = par ? keep_h : got_h;
          const uint32_t em = par ? got_m : keep_m, om = par ? keep_m : got_m;
          ph[2 * t] = __byte_perm(eh, oh, 0x5140);
          ph[2 * t + 1] = __byte_perm(eh, oh, 0x7362);
          pm[2 * t] = __byte_perm(em, om, 0x5140);
          pm[2 * t + 1] = __byte_perm(em, om, 0x7362);
        }
        // P^T row: 64 bytes of hi codes (chunks 0-3), 64 of mid codes (4-7),
        // into the page's RoPE box, which QK^T is done with.  Rows r and r + 8
        // of a quarter-warp's store share their swizzle, so the latter's
        // threads write mid before hi: eight distinct positions.
        const uint32_t rowaddr = sSlot0 + s * kSlot + kRopeBox8 * kBox + srow * 128;
        const bool late = (srow >> 3) & 1;
#pragma unroll
        for (int t = 0; t < 4; ++t) {
          const int h4 = 4 * (t & 1);
          const bool is_mid = (t >= 2) != late;
          const int chunk = (is_mid ? 4 : 0) + 2 * par + (t & 1);
          st_shared_v4(rowaddr + ((chunk ^ (srow & 7)) << 4), is_mid ? pm[h4] : ph[h4],
                       is_mid ? pm[h4 + 1] : ph[h4 + 1], is_mid ? pm[h4 + 2] : ph[h4 + 2],
                       is_mid ? pm[h4 + 3] : ph[h4 + 3]);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) mbar_arrive(smem_u32(&p_full[g % kSlots]));
      }
      if (fail) break;
      have = walk.next(P, view, pc);

      // ---------------- epilogue of this piece, a half of the columns each
      l += __shfl_xor_sync(0xffffffffu, l, 2);
      l_r += __shfl_xor_sync(0xffffffffu, l_r, 2);
      if (owner) {
        l_sh[q][srow] = l;
        l_r_sh[q][srow] = l_r;
        m_l_sh[q][srow] = m_mine;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&sums_full));
      bad = bad || !mbar_wait(smem_u32(&sums_full), n & 1, &abort_sh, P.status) ||
            !mbar_wait(smem_u32(&o_full), n & 1, &abort_sh, P.status);
      __syncwarp();
      if (bar_any(1 + q, 128, bad)) break;
      tc_fence_after();
      const size_t row_base = dest < 0 ? ~dest : dest;
      __nv_bfloat16* const out = (dest < 0 ? view.opart : P.olat) + row_base * kLora;
#pragma unroll 1
      for (int row = lane; row < rows_here; row += 32) {
        // The row's sums, in its last maximum.
        const float m = m_sh[row];
        const float w0 = m_l_sh[0][row] == -INFINITY ? 0.0f : ex2_approx(m_l_sh[0][row] - m);
        const float w1 = m_l_sh[1][row] == -INFINITY ? 0.0f : ex2_approx(m_l_sh[1][row] - m);
        const float total_r = fmaf(l_r_sh[0][row], w0, l_r_sh[1][row] * w1);
        inv_sh[warp - 4][row] = total_r == 0.0f ? 0.0f : 1.0f / total_r;  // (NaN stays NaN)
        if (q == 0 && wq == 0) {
          const float total = fmaf(l_sh[0][row], w0, l_sh[1][row] * w1);
          const float lse2 = total == 0.0f ? -INFINITY : m - kTopExp + __log2f(total);
          (dest < 0 ? view.lpart : P.lse)[row_base + row] = lse2 * kLn2;
        }
      }
      __syncwarp();
#pragma unroll 1
      for (int h = 0; 16 * h < rows_here; ++h) {
        uint32_t v[2][16];
        const uint32_t ta = tmem + lane_off + kTmemOut + 128 * q + 16 * h;
        tmem_ld_x16(ta, v[0]);
        tmem_ld_x16(ta + 64, v[1]);
        tmem_wait_ld();
        // Lane = latent column, v[.][j] = row j.  Of two rows the even lane
        // stores one and the odd lane the other, two columns each.
        uint32_t* const dst = reinterpret_cast<uint32_t*>(
            out + (16 * h + (lane & 1)) * kLora + 256 * q + 32 * wq + (lane & ~1));
#pragma unroll
        for (int j = 0; j < 16; j += 2) {
          const float2 il = *reinterpret_cast<const float2*>(&inv_sh[warp - 4][16 * h + j]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            const float x = __uint_as_float(v[m][j]) * il.x;
            const float y = __uint_as_float(v[m][j + 1]) * il.y;
            const float got = __shfl_xor_sync(0xffffffffu, lane & 1 ? x : y, 1);
            dst[j * (kLora / 2) + 64 * m] =
                lane & 1 ? pack_bf16x2(got, y) : pack_bf16x2(x, got);
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) {
        mbar_arrive(smem_u32(&o_free));
        mbar_arrive(smem_u32(&epi_done));
      }
      ++n;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == 2) {
    tc_fence_after();
    tmem_dealloc(tmem, kTmemAll);
  }
}

}  // namespace

cudaError_t launch_decode_fp8kv(const CUtensorMap& tm_lat, const CUtensorMap& tm_rope,
                                const CUtensorMap& tm_q, int sm_count,
                                const int32_t* block_table, const float* kv_scale,
                                const int32_t* seq_len_eff, const PlanHeader* header, void* ws,
                                const int32_t* seq_first, const int32_t* seq_nsplit,
                                const int32_t* seq_slot, __nv_bfloat16* olat, float* lse,
                                int32_t* status, int B, int T, int H, int max_pages,
                                int num_pages, float scale, cudaStream_t st) {
  Params P{};
  const DecodeShape shape = decode_shape(T, H, sm_count);
  const cudaError_t e = cudaFuncSetAttribute(
      decode_fp8kv_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
  if (e != cudaSuccess) return e;
  P.block_table = block_table;
  P.kv_scale = kv_scale;
  P.seq_len_eff = seq_len_eff;
  P.header = header;
  P.ws = static_cast<uint8_t*>(ws);
  P.seq_first = seq_first;
  P.seq_nsplit = seq_nsplit;
  P.seq_slot = seq_slot;
  P.q_box_rows = decode_q_box_rows(T, H);
  P.olat = olat;
  P.lse = lse;
  P.status = status;
  P.B = B;
  P.T = T;
  P.H = H;
  P.max_pages = max_pages;
  P.num_pages = num_pages;
  P.tpg = shape.tpg;
  P.sets = shape.sets;
  P.scale_log2 = scale * 1.4426950408889634f;
  return launch_pdl(decode_fp8kv_kernel, dim3(shape.groups * shape.tpg), dim3(kThreads),
                    kSmemBytes, st, tm_lat, tm_rope, tm_q, P);
}

}  // namespace mla

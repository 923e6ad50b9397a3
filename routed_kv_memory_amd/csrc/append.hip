// append.hip -- new tokens' K/V rows into the paged local cache, normed and rotated on the way.
//
// For every layer, new token t (i-th of sequence b's n_b) with local row r = kv_len[b] - n_b + i
// and position p = pos_off[b] + r:  k and q are scaled per head by w / sqrt(mean(x^2) + eps) where
// weights are given, then the pairs (e, e + 64) of each head are turned by p * theta^(-e/64);
// k and v go to row r % P of page page_table[b][r / P], q to its own output.
//
// Bound: HBM (each byte is read once and written once, ~6 flop an element): 3.85 GB, 8,704 tokens of 32 query heads in
// 18 layers, take 0.70-0.73 ms (5.3-5.5 TB/s), one token 6 us, where latency is all (a launch and three loads that
// wait for each other: q_off, the sequence's lengths, its page).  One wave takes one
// token in one layer: 8 lanes a head hold the 8-dim pieces 8 j .. 8 j + 7 and 64 + 8 j .. + 7, so
// both halves of every rotated pair sit in one lane, a row of 8 heads is one 2 KiB access of the
// wave, and the token's 64 angles are formed once for all its heads (8 in each lane).  Angles are
// formed and reduced to a fraction of a turn in fp64 (far positions lose their fraction in fp32):
// theta^(-e/64) for e = 8 j + i is a product of four powers the host passes, 10 fp64 products.
// Everything in between is fp32; one rounding to bf16.
#include "append_core.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

constexpr int kAppendWaves = 4;            // tokens per workgroup

template <bool NORM_K, bool NORM_Q>
__global__ void __launch_bounds__(64 * kAppendWaves)
append_kernel(int32_t B, int32_t n_q, int32_t Hq, const uint16_t* __restrict__ k_new,
              const uint16_t* __restrict__ v_new, const uint16_t* q, const int32_t* __restrict__ q_off,
              const int32_t* __restrict__ kv_len, const int32_t* __restrict__ pos_off,
              const int32_t* __restrict__ page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
              const uint16_t* __restrict__ w_k, const uint16_t* __restrict__ w_q, float eps, Turns pw,
              uint16_t* __restrict__ k_pages, uint16_t* __restrict__ v_pages, uint16_t* q_out) {
  const int lane = threadIdx.x & 63;
  const int32_t t = blockIdx.x * kAppendWaves + (threadIdx.x >> 6);
  const int64_t layer = blockIdx.y;
  if (t >= n_q) return;                     // whole waves; no barrier below
  const int32_t b = seq_of_token(q_off, B, t, lane);
  if (b >= B) return;                       // rows behind the last sequence are left as they are
  const int32_t q0 = q_off[b], q1 = q_off[b + 1];
  if (t < q0 || t >= q1) return;            // offsets that are not ascending
  const int64_t row = (int64_t)kv_len[b] - (q1 - t);
  const double pos = (double)(row + (pos_off ? pos_off[b] : 0));

  const int head = lane >> 3, j = lane & 7;
  const int64_t at = (layer * n_q + t) * kRow + head * kDim + 8 * j;
  u32x4 k_lo = *reinterpret_cast<const u32x4*>(k_new + at), k_hi = *reinterpret_cast<const u32x4*>(k_new + at + 64);
  const u32x4 v_lo = *reinterpret_cast<const u32x4*>(v_new + at),
              v_hi = *reinterpret_cast<const u32x4*>(v_new + at + 64);

  float cs[8], sn[8];
  angles(pos, j, pw, cs, sn);
  float w_lo[8], w_hi[8];
  if (NORM_K) {
    unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 8 * j), w_lo);
    unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 64 + 8 * j), w_hi);
  }
  norm_turn<NORM_K>(k_lo, k_hi, w_lo, w_hi, eps, true, cs, sn);
  if (row >= 0 && (row >> page_shift) < max_pages) {
    const int32_t page = page_table[(int64_t)b * max_pages + (row >> page_shift)];
    if (page >= 0 && page < n_pages) {
      const int64_t slot = ((layer * n_pages + page) << page_shift) + (row & ((1 << page_shift) - 1));
      uint16_t* kd = k_pages + slot * kRow + head * kDim + 8 * j;
      uint16_t* vd = v_pages + slot * kRow + head * kDim + 8 * j;
      *reinterpret_cast<u32x4*>(kd) = k_lo;
      *reinterpret_cast<u32x4*>(kd + 64) = k_hi;
      *reinterpret_cast<u32x4*>(vd) = v_lo;
      *reinterpret_cast<u32x4*>(vd + 64) = v_hi;
    }
  }
  if (q) {
    if (NORM_Q) {
      unpack8(*reinterpret_cast<const u32x4*>(w_q + layer * kDim + 8 * j), w_lo);
      unpack8(*reinterpret_cast<const u32x4*>(w_q + layer * kDim + 64 + 8 * j), w_hi);
    }
    const int64_t q_at = (layer * n_q + t) * Hq * kDim + head * kDim + 8 * j;
    for (int32_t h = 0; h < Hq; h += 8) {   // q_out may be q: a lane writes only what it has read
      u32x4 lo = *reinterpret_cast<const u32x4*>(q + q_at + h * kDim);
      u32x4 hi = *reinterpret_cast<const u32x4*>(q + q_at + h * kDim + 64);
      norm_turn<NORM_Q>(lo, hi, w_lo, w_hi, eps, true, cs, sn);
      *reinterpret_cast<u32x4*>(q_out + q_at + h * kDim) = lo;
      *reinterpret_cast<u32x4*>(q_out + q_at + h * kDim + 64) = hi;
    }
  }
}

}  // namespace

hipError_t launch_append(int32_t L, int32_t B, int32_t n_q, int32_t Hq, const uint16_t* k_new, const uint16_t* v_new,
                         const uint16_t* q, const int32_t* q_off, const int32_t* kv_len, const int32_t* pos_off,
                         const int32_t* page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
                         const uint16_t* w_k, const uint16_t* w_q, float eps, float theta, uint16_t* k_pages,
                         uint16_t* v_pages, uint16_t* q_out, hipStream_t s) {
  const Turns pw = turns_of(theta);
  const dim3 grid((unsigned)((n_q + kAppendWaves - 1) / kAppendWaves), (unsigned)L);
#define MSA_APPEND_LAUNCH(NK, NQ)                                                                                  \
  hipLaunchKernelGGL((append_kernel<NK, NQ>), grid, dim3(64 * kAppendWaves), 0, s, B, n_q, Hq, k_new, v_new, q,   \
                     q_off, kv_len, pos_off, page_table, max_pages, page_shift, n_pages, w_k, w_q, eps, pw,       \
                     k_pages, v_pages, q_out)
  if (w_k && w_q) MSA_APPEND_LAUNCH(true, true);
  else if (w_k) MSA_APPEND_LAUNCH(true, false);
  else if (w_q) MSA_APPEND_LAUNCH(false, true);
  else MSA_APPEND_LAUNCH(false, false);
#undef MSA_APPEND_LAUNCH
  return hipGetLastError();
}

}  // namespace msa

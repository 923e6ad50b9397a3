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
#include "msa_device.hpp"
#include "msa_kernels.hpp"

#include <cmath>

namespace msa {
namespace {

constexpr int kAppendWaves = 4;            // tokens per workgroup

// theta^(-1/64), its 8th, 16th and 32nd power
struct Turns {
  double r1, r8, r16, r32;
};

__device__ __forceinline__ void unpack8(u32x4 w, float* f) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}

__device__ __forceinline__ u32x4 pack8(const float* f) {
  u32x4 w;
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = pack2_bf16(f[2 * i], f[2 * i + 1]);
  return w;
}

// Sum over the 8 lanes of a head (an aligned half of a DPP row); every lane gets it.
__device__ __forceinline__ float lanes8_sum(float v) {
  int x = __float_as_int(v);
  v += __int_as_float(__builtin_amdgcn_update_dpp(x, x, 0xB1, 0xF, 0xF, false));    // quad_perm [1,0,3,2]
  x = __float_as_int(v);
  v += __int_as_float(__builtin_amdgcn_update_dpp(x, x, 0x4E, 0xF, 0xF, false));    // quad_perm [2,3,0,1]
  x = __float_as_int(v);
  return v + __int_as_float(__builtin_amdgcn_update_dpp(x, x, 0x141, 0xF, 0xF, false));   // row_half_mirror
}

// One head's row in 8 lanes: lo = dims 8 j .., hi = dims 64 + 8 j ..; normed (w != NULL) and turned.
template <bool NORM>
__device__ __forceinline__ void norm_turn(u32x4& lo, u32x4& hi, const float* w_lo, const float* w_hi, float eps,
                                          const float* cs, const float* sn) {
  float a[8], b[8];
  unpack8(lo, a);
  unpack8(hi, b);
  if (NORM) {
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss += a[i] * a[i] + b[i] * b[i];
    const float inv = 1.0f / sqrtf(lanes8_sum(ss) * (1.0f / kDim) + eps);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      a[i] *= inv * w_lo[i];
      b[i] *= inv * w_hi[i];
    }
  }
  float x[8], y[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = a[i] * cs[i] - b[i] * sn[i];
    y[i] = b[i] * cs[i] + a[i] * sn[i];
  }
  lo = pack8(x);
  hi = pack8(y);
}

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
  double f = (j & 1 ? pw.r8 : 1.0) * (j & 2 ? pw.r16 : 1.0) * (j & 4 ? pw.r32 : 1.0) * 0.15915494309189533577;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double turns = pos * f;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn[i], &cs[i]);
    f *= pw.r1;
  }
  float w_lo[8], w_hi[8];
  if (NORM_K) {
    unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 8 * j), w_lo);
    unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 64 + 8 * j), w_hi);
  }
  norm_turn<NORM_K>(k_lo, k_hi, w_lo, w_hi, eps, cs, sn);
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
      norm_turn<NORM_Q>(lo, hi, w_lo, w_hi, eps, cs, sn);
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
  const double l = std::log2((double)theta);
  const Turns pw = {std::exp2(-l / 64), std::exp2(-l / 8), std::exp2(-l / 4), std::exp2(-l / 2)};
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

// append4.hip -- new tokens' K/V rows into a paged local cache held in 4 bits, normed and rotated on the way.
//
// As append.hip (which says what a token's row and position are), but a row of K or V is stored in the format of
// cache4.hpp.  K is quantised from its value after norm and rotation, unrounded, V from its bf16 value.
// K's arithmetic is in fp64 to the code: a value next to a border of two codes comes out on the same side however
// it is computed, so a row's bytes depend on its token alone.
//
// One wave takes one token in one layer, 8 lanes a head; four of them hold a block of 32 dims.
#include "append_core.hpp"
#include "cache4.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

constexpr int kAppendWaves = 4;            // tokens per workgroup

template <typename T>
__device__ __forceinline__ T lanes4_max(T v) {
  v = fmax(v, __shfl_xor(v, 1, 64));
  return fmax(v, __shfl_xor(v, 2, 64));
}

// Exponent of a block whose largest magnitude is m (finite).
__device__ __forceinline__ int exponent4(double m) {
  const uint64_t u = (uint64_t)__double_as_longlong(m);
  const int e = (int)(u >> 52) - 1022 - ((u & 0xFFFFFFFFFFFFFull) <= 0xC000000000000ull ? 3 : 2);
  return e < -125 ? -125 : (e > 125 ? 125 : e);
}

// 8 of a block's values, the block in 4 lanes: their codes and the block's scale byte.
__device__ __forceinline__ uint32_t quantise8(const double* x, uint32_t* byte) {
  double m = 0.0;
  bool odd = false;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double a = fabs(x[i]);
    odd |= !(a < __builtin_huge_val());
    m = fmax(m, a);
  }
  m = lanes4_max(m);
  odd = lanes4_max(odd ? 1.f : 0.f) > 0.f;
  const int e = odd ? 0 : exponent4(m);
  const double unit = __longlong_as_double((long long)(1023 - e) << 52);
  uint32_t w = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double y = fabs(x[i]) * unit;
    const uint32_t c = (y > 0.25) + (y >= 0.75) + (y > 1.25) + (y >= 1.75) + (y > 2.5) + (y >= 3.5) + (y > 5.0);
    w |= (c | (uint32_t)(__double_as_longlong(x[i]) < 0 ? 8 : 0)) << (4 * i);
  }
  *byte = odd ? kNaN4 : (uint32_t)(e + 127);
  return odd ? 0u : w;
}

__device__ __forceinline__ double lanes8_sum(double v) {
  v += __shfl_xor(v, 1, 64);
  v += __shfl_xor(v, 2, 64);
  return v + __shfl_xor(v, 4, 64);
}

template <bool NORM_K, bool NORM_Q>
__global__ void __launch_bounds__(64 * kAppendWaves)
append4_kernel(int32_t B, int32_t n_q, int32_t Hq, const uint16_t* __restrict__ k_new,
               const uint16_t* __restrict__ v_new, const uint16_t* q, const int32_t* __restrict__ q_off,
               const int32_t* __restrict__ kv_len, const int32_t* __restrict__ pos_off,
               const int32_t* __restrict__ page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
               const uint16_t* __restrict__ w_k, const uint16_t* __restrict__ w_q, float eps, bool turn, Turns pw,
               uint8_t* __restrict__ k_pages, uint8_t* __restrict__ v_pages, uint16_t* q_out) {
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

  int64_t page = -1;                        // its first byte
  if (row >= 0 && (row >> page_shift) < max_pages) {
    const int32_t p = page_table[(int64_t)b * max_pages + (row >> page_shift)];
    if (p >= 0 && p < n_pages) page = ((layer * n_pages + p) << page_shift) * kRow4;
  }
  if (page >= 0) {
    const int64_t at = (layer * n_q + t) * kRow + head * kDim + 8 * j;
    float f[16], w[16];
    double x[16];
    unpack8(*reinterpret_cast<const u32x4*>(k_new + at), f);
    unpack8(*reinterpret_cast<const u32x4*>(k_new + at + 64), f + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = f[i];
    if (NORM_K) {
      unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 8 * j), w);
      unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 64 + 8 * j), w + 8);
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += x[i] * x[i];
      const double inv = 1.0 / sqrt(lanes8_sum(ss) * (1.0 / kDim) + (double)eps);
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] *= inv * (double)w[i];
    }
    if (turn) {
      double fr = (j & 1 ? pw.r8 : 1.0) * (j & 2 ? pw.r16 : 1.0) * (j & 4 ? pw.r32 : 1.0) * 0.15915494309189533577;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double turns = pos * fr;
        double sn, cs;
        sincospi(2.0 * (turns - rint(turns)), &sn, &cs);
        fr *= pw.r1;
        const double lo = x[i] * cs - x[i + 8] * sn, hi = x[i + 8] * cs + x[i] * sn;
        x[i] = lo;
        x[i + 8] = hi;
      }
    }
    const int r = (int)(row & ((1 << page_shift) - 1));
    auto store = [&](uint8_t* pages) {
      uint32_t s_lo, s_hi;
      const uint32_t lo = quantise8(x, &s_lo), hi = quantise8(x + 8, &s_hi);
      uint8_t* codes = pages + page + codes4_at(head, r, page_shift) + 4 * j;
      *reinterpret_cast<uint32_t*>(codes) = lo;
      *reinterpret_cast<uint32_t*>(codes + 32) = hi;
      uint8_t* scales = pages + page + scales4_at(head, r, page_shift) + (j >> 2);
      if ((j & 3) == 0) {
        scales[0] = (uint8_t)s_lo;
        scales[2] = (uint8_t)s_hi;
      }
    };
    store(k_pages);
    unpack8(*reinterpret_cast<const u32x4*>(v_new + at), f);
    unpack8(*reinterpret_cast<const u32x4*>(v_new + at + 64), f + 8);
#pragma unroll
    for (int i = 0; i < 16; ++i) x[i] = f[i];
    store(v_pages);
  }
  if (q) {
    float cs[8], sn[8];
    if (turn) {
      angles(pos, j, pw, cs, sn);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        cs[i] = 1.f;
        sn[i] = 0.f;
      }
    }
    float w_lo[8], w_hi[8];
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

hipError_t launch_append4(int32_t L, int32_t B, int32_t n_q, int32_t Hq, const uint16_t* k_new, const uint16_t* v_new,
                          const uint16_t* q, const int32_t* q_off, const int32_t* kv_len, const int32_t* pos_off,
                          const int32_t* page_table, int32_t max_pages, int32_t page_shift, int32_t n_pages,
                          const uint16_t* w_k, const uint16_t* w_q, float eps, float theta, uint8_t* k_pages,
                          uint8_t* v_pages, uint16_t* q_out, hipStream_t s) {
  const bool turn = theta > 0.f;
  const Turns pw = turns_of(turn ? theta : 1.f);
  const dim3 grid((unsigned)((n_q + kAppendWaves - 1) / kAppendWaves), (unsigned)L);
#define MSA_APPEND_LAUNCH(NK, NQ)                                                                                  \
  hipLaunchKernelGGL((append4_kernel<NK, NQ>), grid, dim3(64 * kAppendWaves), 0, s, B, n_q, Hq, k_new, v_new, q,  \
                     q_off, kv_len, pos_off, page_table, max_pages, page_shift, n_pages, w_k, w_q, eps, turn, pw, \
                     k_pages, v_pages, q_out)
  if (w_k && w_q) MSA_APPEND_LAUNCH(true, true);
  else if (w_k) MSA_APPEND_LAUNCH(true, false);
  else if (w_q) MSA_APPEND_LAUNCH(false, true);
  else MSA_APPEND_LAUNCH(false, false);
#undef MSA_APPEND_LAUNCH
  return hipGetLastError();
}

}  // namespace msa

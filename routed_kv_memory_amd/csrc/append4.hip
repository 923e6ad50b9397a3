// append4.hip -- new tokens' K/V rows into a paged local cache held in 4 bits, normed and rotated on the way.
//
// As append.hip (which says what a token's row and position are), but a row of K or V is stored in the format of
// cache4.hpp.  K is quantised from its value after norm and rotation, unrounded, V from its bf16 value.
// K's codes are those of fp64 arithmetic: a value next to a border of two codes comes out on the same side however
// it is computed, so a row's bytes depend on its token alone.
//
// One wave takes one token in one layer, 8 lanes a head; four of them hold a block of 32 dims.  K is computed in fp32
// first, with a bound of its error; where the value less and more that bound have different codes, or a block's
// exponent is open (one wave in a hundred or two), the wave computes its row again in fp64.
//
// Bound: HBM.  8,704 tokens of 32 query heads in 18 layers: 658 us, 5.1 TB/s (all of K in fp64: 773 us, bound by
// that); a batch's 128 tokens 16.5 us (21); one token 9 us, a launch and three loads that wait for each other.  Held
// to the registers of five waves a SIMD it spills and is slower.
#include "append_core.hpp"
#include "cache4.hpp"
#include "msa_kernels.hpp"

namespace msa {
namespace {

constexpr int kAppendWaves = 4;            // tokens per workgroup

// Largest of the four lanes of a block (an aligned quarter of a DPP row).
__device__ __forceinline__ uint32_t lanes4_max(uint32_t v) {
  v = max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0xB1, 0xF, 0xF, false));     // quad_perm [1,0,3,2]
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, 0x4E, 0xF, 0xF, false));  // quad_perm [2,3,0,1]
}
__device__ __forceinline__ double lanes4_max(double v) {
  v = fmax(v, __shfl_xor(v, 1, 64));
  return fmax(v, __shfl_xor(v, 2, 64));
}

// Exponent of a block whose largest magnitude is m (finite): mantissas up to 1.75 are within 7 * 2^e.
__device__ __forceinline__ int exponent4(double m) {
  const uint64_t u = (uint64_t)__double_as_longlong(m);
  const int e = (int)(u >> 52) - 1025 + ((u & 0xFFFFFFFFFFFFFull) > 0xC000000000000ull ? 1 : 0);
  return e < -125 ? -125 : (e > 125 ? 125 : e);
}
__device__ __forceinline__ int exponent4(uint32_t m) {       // of a float's bits
  const int e = (int)((m + 0x1FFFFFu) >> 23) - 129;
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
  odd = lanes4_max(odd ? 1u : 0u) != 0;
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

__device__ __forceinline__ uint32_t codes8(const float* x, float scale) {
  uint32_t w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[2], x[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[4], x[5], scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, x[6], x[7], scale, 3);
}

// The same in fp32, of values that are off by up to off[i] (null: none): *open where that leaves anything open.  The
// conversion rounds to the nearest, halfway to the even code, and stops at 6, as the format has it; blocks that hold no
// numbers, or near fp32's smallest, are left to fp64.
__device__ __forceinline__ uint32_t quantise8(const float* x, const float* off, uint32_t* byte, bool* open) {
  uint32_t m = 0, low = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(x[i]);
    m = max(m, __float_as_uint(off ? a + off[i] : a));
    if (off) low = max(low, __float_as_uint(fmaxf(a - off[i], 0.f)));
  }
  m = lanes4_max(m);
  const int e = exponent4(m);
  const float scale = __uint_as_float((uint32_t)(e + 127) << 23);
  *open |= m - 0x0D800000u >= 0x7F800000u - 0x0D800000u;     // below 2^-100, infinite or NaN
  *byte = (uint32_t)(e + 127);
  if (!off) return codes8(x, scale);
  *open |= exponent4(lanes4_max(low)) != e;
  float lo[8], hi[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    lo[i] = x[i] - off[i];
    hi[i] = x[i] + off[i];
  }
  const uint32_t w = codes8(lo, scale);
  *open |= w != codes8(hi, scale);
  return w;
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
  float cs[8], sn[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (turn) angles(pos, j, pw, cs, sn);
  if (page >= 0) {
    const int64_t at = (layer * n_q + t) * kRow + head * kDim + 8 * j;
    const int r = (int)(row & ((1 << page_shift) - 1));
    auto store = [&](uint8_t* pages, const uint32_t* w, const uint32_t* byte) {
      uint8_t* codes = pages + page + codes4_at(head, r, page_shift) + 4 * j;
      *reinterpret_cast<uint32_t*>(codes) = w[0];
      *reinterpret_cast<uint32_t*>(codes + 32) = w[1];
      uint8_t* scales = pages + page + scales4_at(head, r, page_shift) + (j >> 2);
      if ((j & 3) == 0) {
        scales[0] = (uint8_t)byte[0];
        scales[2] = (uint8_t)byte[1];
      }
    };
    const u32x4 k_lo = *reinterpret_cast<const u32x4*>(k_new + at), k_hi = *reinterpret_cast<const u32x4*>(k_new + at + 64);
    const u32x4 v_lo = *reinterpret_cast<const u32x4*>(v_new + at), v_hi = *reinterpret_cast<const u32x4*>(v_new + at + 64);
    float f[16], w[16];
    uint32_t code[2], byte[2];
    bool open = false;
    unpack8(k_lo, f);
    unpack8(k_hi, f + 8);
    double inv = 1.0;
    if (NORM_K) {
      unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 8 * j), w);
      unpack8(*reinterpret_cast<const u32x4*>(w_k + layer * kDim + 64 + 8 * j), w + 8);
      double ss = 0.0;
#pragma unroll
      for (int i = 0; i < 16; ++i) ss += (double)f[i] * (double)f[i];
      inv = 1.0 / sqrt(lanes8_sum(ss) * (1.0 / kDim) + (double)eps);
    }
    {
      // With u = 2^-24, and by |a| + |b|: a value after the norm is off by 3 u (inv, inv w, the product), a cosine or sine
      // by 2.5 u (its angle's rounding, pi / 2 u, and sincospif: under 0.88 u for every float from -1 to 1, compared
      // one by one with fp64), a product by its rounding, u, and the sum by its own, u: 7.5 u in all.  x - off and x + off
      // are rounded once more, under 1.1 u.  12 u here; and where inv w is below the normal numbers, its 2^-150 times the key.
      open |= inv < 0x1p-126;
      float x[16], off[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float a = f[i], b = f[i + 8];
        if (NORM_K) {
          a *= (float)inv * w[i];
          b *= (float)inv * w[i + 8];
        }
        off[i] = (fabsf(a) + fabsf(b)) * (NORM_K || turn ? 12 * 0x1p-24f : 0.f);
        if (NORM_K) off[i] = fmaf(fabsf(f[i]) + fabsf(f[i + 8]), 0x1p-149f, off[i]);
        x[i] = turn ? a * cs[i] - b * sn[i] : a;
        x[i + 8] = turn ? b * cs[i] + a * sn[i] : b;
      }
      code[0] = quantise8(x, off, byte, &open);
      code[1] = quantise8(x + 8, off, byte + 1, &open);
    }
    if (__ballot(open)) {
      double x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = NORM_K ? (double)f[i] * (inv * (double)w[i]) : (double)f[i];
      if (turn) {
        double fr = (j & 1 ? pw.r8 : 1.0) * (j & 2 ? pw.r16 : 1.0) * (j & 4 ? pw.r32 : 1.0) * 0.15915494309189533577;
#pragma unroll 1
        for (int i = 0; i < 8; ++i) {
          const double turns = pos * fr;
          double s, c;
          sincospi(2.0 * (turns - rint(turns)), &s, &c);
          fr *= pw.r1;
#pragma unroll
          for (int n = 0; n < 8; ++n)               // registers have no index
            if (n == i) {
              const double lo = x[n] * c - x[n + 8] * s, hi = x[n + 8] * c + x[n] * s;
              x[n] = lo;
              x[n + 8] = hi;
            }
        }
      }
      code[0] = quantise8(x, byte);
      code[1] = quantise8(x + 8, byte + 1);
    }
    store(k_pages, code, byte);
    unpack8(v_lo, f);
    unpack8(v_hi, f + 8);
    open = false;
    code[0] = quantise8(f, nullptr, byte, &open);
    code[1] = quantise8(f + 8, nullptr, byte + 1, &open);
    if (__ballot(open)) {
      double x[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) x[i] = (double)f[i];
      code[0] = quantise8(x, byte);
      code[1] = quantise8(x + 8, byte + 1);
    }
    store(v_pages, code, byte);
  }
  if (q) {
    float w_lo[8], w_hi[8];
    if (NORM_Q) {
      unpack8(*reinterpret_cast<const u32x4*>(w_q + layer * kDim + 8 * j), w_lo);
      unpack8(*reinterpret_cast<const u32x4*>(w_q + layer * kDim + 64 + 8 * j), w_hi);
    }
    const int64_t q_at = (layer * n_q + t) * Hq * kDim + head * kDim + 8 * j;
    for (int32_t h = 0; h < Hq; h += 8) {   // q_out may be q: a lane writes only what it has read
      u32x4 lo = *reinterpret_cast<const u32x4*>(q + q_at + h * kDim);
      u32x4 hi = *reinterpret_cast<const u32x4*>(q + q_at + h * kDim + 64);
      norm_turn<NORM_Q>(lo, hi, w_lo, w_hi, eps, turn, cs, sn);
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

// append_core.hpp -- norm and rotation of new tokens' rows, shared by the appends to a cache in bf16 and in
// 4 bits.  8 lanes hold a head: lane j dims 8 j .. 8 j + 7 and 64 + 8 j .. + 7, so both halves of a rotated pair.
#pragma once

#include "msa_device.hpp"

#include <cmath>

namespace msa {
namespace {

// theta^(-1/64), its 8th, 16th and 32nd power
struct Turns {
  double r1, r8, r16, r32;
};

inline Turns turns_of(float theta) {
  const double l = std::log2((double)theta);
  return {std::exp2(-l / 64), std::exp2(-l / 8), std::exp2(-l / 4), std::exp2(-l / 2)};
}

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

// One head's row in 8 lanes: lo = dims 8 j .., hi = dims 64 + 8 j ..; normed (w != NULL) and turned (`turn`).  A turn
// by nothing is left out, not computed: 0 times an infinity is NaN, and the sum of -0 and 0 is 0.
template <bool NORM>
__device__ __forceinline__ void norm_turn(u32x4& lo, u32x4& hi, const float* w_lo, const float* w_hi, float eps, bool turn,
                                          const float* cs, const float* sn) {
  if (!NORM && !turn) return;
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
    x[i] = turn ? a[i] * cs[i] - b[i] * sn[i] : a[i];
    y[i] = turn ? b[i] * cs[i] + a[i] * sn[i] : b[i];
  }
  lo = pack8(x);
  hi = pack8(y);
}

// cos and sin of the angles of pairs 8 j .. 8 j + 7 at position `pos`.
__device__ __forceinline__ void angles(double pos, int j, Turns pw, float* cs, float* sn) {
  double f = (j & 1 ? pw.r8 : 1.0) * (j & 2 ? pw.r16 : 1.0) * (j & 4 ? pw.r32 : 1.0) * 0.15915494309189533577;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const double turns = pos * f;
    sincospif((float)(2.0 * (turns - rint(turns))), &sn[i], &cs[i]);
    f *= pw.r1;
  }
}

}  // namespace
}  // namespace msa

// cache4.hpp -- the rows of a local cache held in 4 bits.
//
// 128 dims of a head are four blocks of 32.  A block x is a power of two 2^e, in a byte e + 127, and 32 codes
// of a sign and an index into {0, 0.5, 1, 1.5, 2, 3, 4, 6}:
//   e     the smallest whole number with max|x| <= 7 * 2^e, kept in [-125, 125]
//   code  the nearest to |x| / 2^e (halfway: the even index; past 6: 6)
// so a code stands for an exact bf16 value; a block that holds an infinity or NaN has the byte 255 and reads
// as NaN.  7 and not 6 (nothing is cut off) or 8: the rms error of normal values is 0.1118 of their own, 0.1154 with
// 6, 0.1149 with 8.  These are the elements and scales that gfx950's conversions take.
//
// A page of P rows is [8 heads][P][64] bytes of codes, dim 2 i in the low half of byte i, then [8][P][4] bytes
// of scales: a head's rows follow each other, so a wave that streams one head reads whole lines.
#pragma once

#include "msa_device.hpp"

namespace msa {

constexpr int kCodes4 = kDim / 2;              // bytes of codes of a head's row
constexpr int kBlocks4 = kDim / 32;            // its scales
constexpr int kRow4 = kHeads * (kCodes4 + kBlocks4);   // bytes of a row: MSA_ROW4_BYTES
constexpr int kNaN4 = 255;

// Where row r of a page of P = 2^shift rows has a head's codes and scales, from the page's first byte.
__device__ __forceinline__ int codes4_at(int head, int r, int shift) { return ((head << shift) + r) * kCodes4; }
__device__ __forceinline__ int scales4_at(int head, int r, int shift) {
  return (kHeads * kCodes4 << shift) + ((head << shift) + r) * kBlocks4;
}

// A scale byte as the float that a conversion takes: it looks at the exponent alone, so 0 is 2^-127 and 255 NaN.
__device__ __forceinline__ float scale4(uint32_t byte) { return __uint_as_float(byte << 23); }

// 8 codes as packed bf16, each the value it stands for: exact, bf16's subnormal numbers (bytes 0 and 1) too; an infinity
// past its range (bytes 253 and 254).
__device__ __forceinline__ u32x4 values4(uint32_t codes, float scale) {
  u32x4 w;
  w[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0));
  w[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1));
  w[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2));
  w[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3));
  return w;
}

}  // namespace msa

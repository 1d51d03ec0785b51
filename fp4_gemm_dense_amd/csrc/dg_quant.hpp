// Device helpers of the quantising kernels (quant.hip, norm.hip): power-of-two
// block scales from a block's largest magnitude, and the E2M1 / e4m3 encoders.
#pragma once

#include "dg_device.hpp"

namespace dg {

typedef __bf16 qbf2 __attribute__((ext_vector_type(2)));

// UE8M0 byte (bias 127) of the smallest e >= -127 with QMAX * 2^e >= amax, amax
// given by its fp32 bit pattern (sign cleared; as an integer the pattern orders
// like the magnitude, with infinities and NaN above every number).  With
// amax = 1.f * 2^x the answer is x - 2 for QMAX = 6 = 1.5 * 2^2 (x - 8 for 448 =
// 1.75 * 2^8) unless f exceeds QMAX's own fraction, then one more: adding
// (2^23 - 1 - QMAX's fraction) carries into the exponent field exactly then.
// 127 (2^0) for amax = 0; 255 (NaN) for an infinity or NaN.
template <bool E4M3>
__device__ __forceinline__ uint32_t ue8m0_byte(uint32_t amax_bits) {
  constexpr uint32_t carry = E4M3 ? 0x1fffffu : 0x3fffffu;
  constexpr int down = E4M3 ? 8 : 2;
  const int e = (int)((amax_bits + carry) >> 23) - down;
  const uint32_t b = (uint32_t)(e < 0 ? 0 : e);
  if (amax_bits == 0) return 127u;
  return amax_bits >= 0x7f800000u ? 255u : b;
}

// 2^(byte - 127) as fp32 (byte 0: 2^-127, a subnormal; 255: NaN)
__device__ __forceinline__ float ue8m0_value(uint32_t byte) {
  return __uint_as_float(byte == 0 ? 0x00400000u : (byte == 255u ? 0x7fc00000u : byte << 23));
}

// Eight values -> eight E2M1 codes of x / scale (scale a power of two), value i in
// nibble i.  The conversion instruction rounds to nearest even and reads subnormal
// sources and scales exactly (checked over every bf16 pattern).
__device__ __forceinline__ uint32_t e2m1x8(const float (&v)[8], float scale) {
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
  return w;
}
__device__ __forceinline__ uint32_t e2m1x8(const v4i& v, float scale) {   // eight bf16
  // (named copies: a bit cast of a vector's element reads the vector's first one)
  const int a = v.x, b = v.y, c = v.z, d = v.w;
  uint32_t w = 0;
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(qbf2, a), scale, 0);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(qbf2, b), scale, 1);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(qbf2, c), scale, 2);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(w, __builtin_bit_cast(qbf2, d), scale, 3);
  return w;
}

// The bf16 values of eight E2M1 codes times scale (exact; beyond bf16: infinity)
__device__ __forceinline__ v4i e2m1x8_to_bf16(uint32_t w, float scale) {
  v4i r;
  r.x = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 0));
  r.y = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 1));
  r.z = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 2));
  r.w = __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, scale, 3));
  return r;
}

// Four values (|v| <= 448 up to a rounding, or NaN) -> four e4m3 codes, nearest even
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(a, b, 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(c, d, w, true);
}

// Two bf16 side by side: their magnitudes, and the larger ones of two pairs (as integers
// the patterns order like the magnitudes).
typedef unsigned short us2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ us2 us2abs(int w) { return __builtin_bit_cast(us2, w & 0x7fff7fff); }
__device__ __forceinline__ us2 us2max(us2 a, us2 b) { return __builtin_elementwise_max(a, b); }

// v of the lane at distance O = 1 or 2; for O = 4 and 8 of a lane of the neighbouring group
// of O lanes (the mirrored one: v has to be the same within a group of O).  On the vector
// ALUs; as shuffles through LDS 4096 x 7168 quantised both ways took 24.0 us for 22.8, one
// row 3.05 for 2.57.
template <int O>
__device__ __forceinline__ uint32_t lane_swap(uint32_t v) {
  static_assert(O == 1 || O == 2 || O == 4 || O == 8, "distance");
  constexpr int ctrl = O == 1 ? 0xb1 : O == 2 ? 0x4e : O == 4 ? 0x141 : 0x140;   // quad_perm, row_half_mirror, row_mirror
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, ctrl, 0xf, 0xf, true);
}

// Largest of v over the lane's aligned group of 4 / 16 lanes; every lane gets it.
__device__ __forceinline__ uint32_t umax(uint32_t a, uint32_t b) { return a > b ? a : b; }
template <int LANES>
__device__ __forceinline__ uint32_t group_max(uint32_t v) {
  static_assert(LANES == 4 || LANES == 16, "group");
  v = umax(v, lane_swap<1>(v));
  v = umax(v, lane_swap<2>(v));
  if constexpr (LANES == 16) {
    v = umax(v, lane_swap<4>(v));
    v = umax(v, lane_swap<8>(v));
  }
  return v;
}

// The scale word of a 128-wide block from its four bytes: byte i is held by lanes
// 4i .. 4i+3 of the lane's aligned group of 16; every lane gets the word.
__device__ __forceinline__ uint32_t scale_word(uint32_t byte) {
  uint32_t w = byte << (8 * ((threadIdx.x >> 2) & 3));
  w |= lane_swap<4>(w);
  w |= lane_swap<8>(w);
  return w;
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7fffffffu; }
__device__ __forceinline__ void unpack_bf16x8(const v4i& p, float (&v)[8]) {
  const uint32_t w[4] = {(uint32_t)p.x, (uint32_t)p.y, (uint32_t)p.z, (uint32_t)p.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
  }
}
__device__ __forceinline__ v4i pack_bf16x8(const float (&v)[8]) {
  return v4i{(int)pack_bf16x2_rne(v[0], v[1]), (int)pack_bf16x2_rne(v[2], v[3]), (int)pack_bf16x2_rne(v[4], v[5]),
             (int)pack_bf16x2_rne(v[6], v[7])};
}

}  // namespace dg

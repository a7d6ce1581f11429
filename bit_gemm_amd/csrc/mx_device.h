// Device helpers of the microscaled (MX) formats on gfx950.
//
// An MX row is cut into blocks of 32 consecutive elements that share one
// power-of-two scale 2^(byte - 127) (E8M0; byte 0xFF is NaN).  Elements are
// E2M1 (MXFP4, largest 6, its top binade starts at 4 = 2^2) or E4M3 (MXFP8,
// largest 448, top binade at 256 = 2^8).  With a = max |x_i| of a block,
//   byte = max(0, floor(log2 a) - emax + 127),  emax = 2 or 8,
//   code_i = round to nearest even of x_i / 2^(byte - 127), saturating,
// as in the published OCP Microscaling Formats specification.  Dividing by
// a power of two is exact, so each code is one rounding of its input.
#pragma once

#include "nvfp4_device.h"

namespace nvfp4 {

enum MxFormat { kMxFp4 = 0, kMxFp8 = 1 };  // NVFP4_MXFP4, NVFP4_MXFP8

template <int FMT>
constexpr int kMxEmax = FMT == kMxFp4 ? 2 : 8;

// Scale byte of a block whose largest |x| has the fp32 bit pattern `abits`
// (bit patterns of non-negative floats order like their values, with
// infinity and NaN on top, so an integer maximum keeps a NaN that fmaxf
// would drop).  A block with an infinity or NaN is NaN as a whole.  The
// exponent field of a subnormal reads as 0, one too high, and both clamp.
template <int FMT>
__device__ __forceinline__ uint32_t mx_scale_byte(uint32_t abits) {
  const int e = (int)(abits >> 23);
  return e == 255 ? 255u : (uint32_t)max(e - kMxEmax<FMT>, 0);
}

// 2^(127 - byte): the factor in front of the rounding (0 for a NaN block,
// whose codes are then those of +-0 or, for NaN inputs, unspecified).
__device__ __forceinline__ float mx_inv_scale(uint32_t byte) {
  return byte == 255u ? 0.0f : __uint_as_float((254u - byte) << 23);
}

// 2^(byte - 127); byte 0 is the subnormal 2^-127, byte 255 NaN.
__device__ __forceinline__ float mx_scale(uint32_t byte) {
  return __uint_as_float(byte == 0u ? 0x00400000u : byte == 255u ? 0x7FC00000u : byte << 23);
}

// Four scaled values -> four E4M3 codes (the conversion rounds to nearest
// even but turns what passes 448 into NaN, so the value is clamped first).
__device__ __forceinline__ uint32_t e4m3_pack4(float a, float b, float c, float d) {
  auto cl = [](float v) { return __builtin_amdgcn_fmed3f(v, -448.0f, 448.0f); };
  int r = __builtin_amdgcn_cvt_pk_fp8_f32(cl(a), cl(b), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(cl(c), cl(d), r, true);
}

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

// Two fp32 rounded to nearest even bf16 (NaN kept), packed.
__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  typedef __attribute__((ext_vector_type(2))) float f2;
  typedef __attribute__((ext_vector_type(2))) __bf16 b2;
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(f2{lo, hi}, b2));
}

// Maximum over a quad of lanes / over 8 consecutive lanes, by DPP.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_max(uint32_t v) {
  return max(v, (uint32_t)__builtin_amdgcn_update_dpp((int)v, (int)v, CTRL, 0xF, 0xF, true));
}
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
  v = dpp_max<0xB1>(v);   // quad_perm 1,0,3,2
  return dpp_max<0x4E>(v);  // quad_perm 2,3,0,1
}
__device__ __forceinline__ uint32_t oct_max(uint32_t v) { return dpp_max<0x141>(quad_max(v)); }  // row_half_mirror

}  // namespace nvfp4

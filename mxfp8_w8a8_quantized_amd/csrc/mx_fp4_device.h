// Device-side MXFP4 helpers for gfx950: E2M1 elements with one E8M0 scale per
// 32 elements along K.
//
// Shared exponent e = floor(log2 amax) - 2 clamped to [-127, 127] (2 is the
// exponent of E2M1's top binade), elements E2M1(x * 2^-e) rounded to nearest
// even after saturation to +-6; the sign of zero is kept. A group holding NaN
// or Inf gets scale 0xFF and every code 7 (E2M1 has no NaN: the scale alone
// marks the group). Codes: bit 3 sign, magnitudes 0, .5, 1, 1.5, 2, 3, 4, 6.
//
// Slab layout of an operand of `rows` rows, R = rows rounded up to 256 and
// S = ceil(K / 128): codes [S][R/16][4 groups][16 rows][16 bytes], element 2b
// of a group in the low half of byte b; scales [S][R][4]. A 16-row block of a
// slab is 1 KB whose bytes 16 l .. 16 l + 15 are what lane l of the
// 16x16x128 MFMA takes (row l % 16, K 32 (l / 16) .. + 31), so a wave loads a
// fragment as one contiguous run; and 16 consecutive rows of one group are 256
// consecutive bytes, which is also the LDS order that a 16-lane phase of
// ds_read_b128 reads without bank conflicts, with no swizzle.
#pragma once

#include "mx_device.h"

namespace mx {

inline __host__ __device__ int64_t fp4_slabs(int64_t K) { return (K + 127) / 128; }

// E8M0 code of a group's scale from the biased exponent field E of its
// largest magnitude: e + 127 = E - 2, clamped to 0 (E <= 2); 255: NaN or Inf.
__device__ inline uint32_t fp4_scale_code(uint32_t E) { return E == 255u ? 0xFFu : (E > 2u ? E - 2u : 0u); }

// Largest bf16 magnitude (bits) of the values in the dwords x[0 .. N).
template <int N>
__device__ inline uint32_t bf16_amax_bits(const uint32_t (&x)[N]) {
  u16x2 m = __builtin_bit_cast(u16x2, x[0] & 0x7FFF7FFFu);
#pragma unroll
  for (int i = 1; i < N; ++i) m = __builtin_elementwise_max(m, __builtin_bit_cast(u16x2, x[i] & 0x7FFF7FFFu));
  return max((uint32_t)m[0], (uint32_t)m[1]);
}

// E2M1 codes of 8 bf16 values (4 dwords) under scale code `scode`. The gfx950
// scaled convert divides by the scale, rounds to nearest even and saturates
// at 6 (checked on the device over every finite bf16), so no clamp is needed.
__device__ inline uint32_t fp4_encode8_bf16(uint32_t x0, uint32_t x1, uint32_t x2, uint32_t x3, uint32_t scode) {
  const float sv = scale_value(scode);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x0), sv, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x1), sv, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x2), sv, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x3), sv, 3);
  return scode == 0xFFu ? 0x77777777u : r;
}

// 8 bf16 values per lane, the four lanes of a DPP quad holding one group of
// 32 (called together): the lane's 8 codes and the group's scale code.
__device__ inline uint32_t fp4_quantize8_bf16(const uint32_t (&x)[4], uint32_t& scode) {
  scode = fp4_scale_code(quad_max_u32(bf16_amax_bits(x)) >> 7);
  return fp4_encode8_bf16(x[0], x[1], x[2], x[3], scode);
}

// The same from 8 f32 values.
__device__ inline uint32_t fp4_quantize8_f32(const float (&x)[8], uint32_t& scode) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 8; ++i) m = max(m, __float_as_uint(x[i]) & 0x7FFFFFFFu);
  scode = fp4_scale_code(quad_max_u32(m) >> 23);
  const float sv = scale_value(scode);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[0], x[1], sv, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[2], x[3], sv, 1);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[4], x[5], sv, 2);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(r, x[6], x[7], sv, 3);
  return scode == 0xFFu ? 0x77777777u : r;
}

// Value of one E2M1 code (low 4 bits of c) before its scale.
__device__ inline float fp4_value(uint32_t c) {
  const uint32_t m = c & 7u;
  // Twice the magnitude: 0, 1, 2, 3, 4, 6, 8, 12, one 4-bit field each.
  const uint32_t twice = (0xC8643210u >> (4 * m)) & 15u;
  const float a = 0.5f * (float)twice;
  return (c & 8u) ? -a : a;
}

// Workgroups are dealt to the 8 XCDs in turn: logical index of workgroup
// `pid` of `n` so that each XCD gets a contiguous range.
__device__ inline uint32_t xcd_order(uint32_t pid, uint32_t n) {
  const uint32_t q = n >> 3, r = n & 7, xcd = pid & 7;
  return xcd * q + (xcd < r ? xcd : r) + (pid >> 3);
}

}  // namespace mx

// What the few-token kernels (mx_fp4_small.hip, mx_experts_few.hip) share: bf16 tokens
// quantized into the lanes' operands of v_mfma_scale_f32_16x16x128_f8f6f4, and scales
// brought to the lanes that want them.
#pragma once

#include "mx_fp4_device.h"

namespace mx {
namespace {

// E4M3 codes of 8 bf16 values under scale code `scode` (as quantize8_bf16).
__device__ __forceinline__ i32x2 e4m3_encode8_bf16(i32x4 x, uint32_t scode) {
  const float sv = scale_value(scode);
  const uint32_t lim = ((scode + 8u) << 7) | 0x60u;  // bf16 bits of 448 * 2^e
  const u16x2 lim_u = {(unsigned short)(lim | 0x8000u), (unsigned short)(lim | 0x8000u)};
  const i16x2 lim_i = {(short)lim, (short)lim};
  bf16x2 c[4];
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const u16x2 a = __builtin_elementwise_min(__builtin_bit_cast(u16x2, (uint32_t)x[d]), lim_u);
    c[d] = __builtin_bit_cast(bf16x2, __builtin_elementwise_min(__builtin_bit_cast(i16x2, a), lim_i));
  }
  s16x2 r0 = {0, 0}, r1 = {0, 0};
  r0 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r0, c[0], sv, false);
  r0 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r0, c[1], sv, true);
  r1 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r1, c[2], sv, false);
  r1 = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r1, c[3], sv, true);
  if (scode == 0xFFu) return i32x2{0x7F7F7F7F, 0x7F7F7F7F};
  return i32x2{__builtin_bit_cast(int, r0), __builtin_bit_cast(int, r1)};
}

// Largest bf16 magnitude bits of 16 values (two 16-byte loads).
__device__ __forceinline__ uint32_t amax16(i32x4 a, i32x4 b) {
  const uint32_t w[8] = {(uint32_t)a[0], (uint32_t)a[1], (uint32_t)a[2], (uint32_t)a[3],
                         (uint32_t)b[0], (uint32_t)b[1], (uint32_t)b[2], (uint32_t)b[3]};
  return bf16_amax_bits(w);
}

// A lane's token operand of a 128-K slab from its 32 bf16 values (G = lane / 16): E2M1
// takes K 32 G .. + 31 in order, E4M3 two runs, K 16 G .. + 15 and 64 + 16 G .. + 15.
// scode: the scale code that the lane gives the MFMA, of K group G.
template <bool FP8>
__device__ __forceinline__ i32x8 quantize_operand(const i32x4 (&x)[4], int lane, int& scode) {
  i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0};
  if constexpr (!FP8) {
    const uint32_t m = max(amax16(x[0], x[1]), amax16(x[2], x[3]));
    scode = (int)fp4_scale_code(m >> 7);
#pragma unroll
    for (int u = 0; u < 4; ++u)
      b[u] = (int)fp4_encode8_bf16((uint32_t)x[u][0], (uint32_t)x[u][1], (uint32_t)x[u][2], (uint32_t)x[u][3],
                                   (uint32_t)scode);
  } else {
    // The lane holds halves of K groups G / 2 and 2 + G / 2; the other halves are 16
    // lanes away. It passes the MFMA the scale of group G: its own first for G = 0, its
    // own second for G = 3, and lanes of G = 1 and 2 swap.
    const int G = lane >> 4;
    uint32_t m0 = amax16(x[0], x[1]), m1 = amax16(x[2], x[3]);
    m0 = max(m0, (uint32_t)__shfl_xor((int)m0, 16, 64));
    m1 = max(m1, (uint32_t)__shfl_xor((int)m1, 16, 64));
    const uint32_t c0 = scale_code_from_exponent(m0 >> 7), c1 = scale_code_from_exponent(m1 >> 7);
    const int swapped = __shfl_xor((int)(G == 1 ? c1 : c0), 48, 64);
    scode = G == 0 ? (int)c0 : G == 3 ? (int)c1 : swapped;
    const i32x2 e0 = e4m3_encode8_bf16(x[0], c0), e1 = e4m3_encode8_bf16(x[1], c0);
    const i32x2 e2 = e4m3_encode8_bf16(x[2], c1), e3 = e4m3_encode8_bf16(x[3], c1);
    b = i32x8{e0[0], e0[1], e1[0], e1[1], e2[0], e2[1], e3[0], e3[1]};
  }
  return b;
}

// Lane 16 i + r holds the scales of row 16 i + r, group g in byte g; returns,
// in lane 16 g + r, the scale of group g of row 16 i + r in byte i: what the
// MFMA wants of that lane for fragment i, which op_sel picks. A 4 x 4
// transposition of bytes over the four lane rows: halves are exchanged 32 lanes
// apart, then bytes 16 lanes apart. Two swaps and two permutations replace four
// byte loads, which cost the load path as much as the codes' loads do.
__device__ __forceinline__ int transpose_scales(int x, int lane) {
  const auto h = __builtin_amdgcn_permlane32_swap((uint32_t)x, (uint32_t)x, false, false);
  const uint32_t y = __builtin_amdgcn_perm(h[1], h[0], lane < 32 ? 0x05040100u : 0x07060302u);
  const auto q = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return (int)__builtin_amdgcn_perm(q[1], q[0], (lane & 16) ? 0x07030501u : 0x06020400u);
}

}  // namespace
}  // namespace mx

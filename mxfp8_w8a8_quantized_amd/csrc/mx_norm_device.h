// What the norm kernels (mx_norm.hip, mx_block_norm.hip) share: a row's elements
// as they are held in registers, and the LDS staging of a tile of rows.
#pragma once

#include "mx_fp4_device.h"

namespace mx {
namespace {

enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

__device__ __forceinline__ float bf16_lo(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_hi(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// Eight consecutive values of h as they are held in registers: bf16 pairs, or
// f32 with an f32 residual.
template <int RES>
struct Held {
  uint32_t w[RES == RES_F32 ? 8 : 4];
  __device__ __forceinline__ float at(int i) const {
    if constexpr (RES == RES_F32) return __uint_as_float(w[i]);
    return (i & 1) ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
  }
};

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) v += __shfl_xor(v, off, 64);
  return v;
}

// Hides what h holds from the compiler, which would otherwise keep every
// element's float64 conversion from the sum of squares until its scaling.
template <int RES, int NCH>
__device__ __forceinline__ void hold(Held<RES> (&h)[NCH]) {
#pragma unroll
  for (int c = 0; c < NCH; ++c)
#pragma unroll
    for (auto& w : h[c].w) asm volatile("" : "+v"(w));
}

// LDS staging of a tile of 8 rows. MXFP8: per 64-K slab 8 rows x 64 bytes and
// 64 bytes of padding (the four slabs that a half-wave's 8-byte writes touch
// start 16 banks apart). MXFP4: per group 8 rows x 16 bytes and 16 bytes of
// padding (the 16 groups of a wave's dword writes cover the 64 banks once).
// The scales follow: 16 bytes per 64-K slab, 32 per 128-K slab.
constexpr int kTileRows = 8;
template <bool FP4>
struct Stage {
  static constexpr int kK = FP4 ? 128 : 64;  // K of a slab
  static constexpr int kCodes = FP4 ? 4 * 144 : 576;
  static constexpr int kScales = FP4 ? 32 : 16;
  __host__ __device__ static int slabs(int K) { return (K + kK - 1) / kK; }
  static int bytes(int K) { return slabs(K) * (kCodes + kScales); }
};

}  // namespace
}  // namespace mx

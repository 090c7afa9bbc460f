// What the experts' product kernels (mx_experts.hip, mx_experts_tile.hip) share.
#pragma once

#include <type_traits>

#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {

struct ProductParams {
  const uint8_t* x;   // codes of tokens (up) or of h (down)
  const uint8_t* xs;
  uint32_t pitch_q, pitch_s;
  uint32_t x_bytes, xs_bytes;  // up: of the whole operand
  const uint8_t* wq;
  const uint8_t* ws;
  int R;             // padded weight rows
  int k;
  int nsteps;
  int I, H;
  int tiles_n;
  const int32_t* rows;
  const ExpertTile* tiles;
  const int32_t* n_tiles;
  uint8_t* hq;  // up: h's codes and scales
  uint8_t* hs;
  uint32_t hpitch_q, hpitch_s;
  uint16_t* o;  // down: f16 [pairs][H]
  uint8_t* os;  // and the exponents of 32 columns
  uint32_t opitch_s;
};

// The products on tiles of 256 weight rows (mx_experts_tile.hip). up: h's codes,
// else o; gate: 0 SiLU, 1 GELU-tanh.
hipError_t launch_experts_tile(const ProductParams& p, bool up, bool fp8, int gate, int64_t max_tiles, hipStream_t stream);

// At most kFewTokens tokens with at most kFewPairs pairs (mx_experts_few.hip); h is
// indexed by pair.
constexpr int kFewTokens = 16, kFewPairs = 128;
struct FewParams {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  int T, k, E, H, I, RU, RD;  // RU, RD: padded rows of the weights
  const uint8_t *up_q, *up_s, *down_q, *down_s;
  uint8_t* hq;
  uint8_t* hs;
  uint32_t hpitch_q, hpitch_s;
  uint16_t* y;
  int tiles_n;
};
hipError_t launch_experts_few(const FewParams& p, bool fp8, int gate, hipStream_t stream);

namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef _Float16 f16x2 __attribute__((ext_vector_type(2)));
typedef _Float16 f16x8 __attribute__((ext_vector_type(8)));
typedef __attribute__((address_space(3))) void* lds_ptr;

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// 16 bytes a lane from `offset` into LDS, lane by lane from `to` on.
__device__ __forceinline__ void dma(__amdgpu_buffer_rsrc_t r, uint8_t* to, uint32_t offset) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_ptr)to, 16, offset, 0, 0, 0);
}

// E4M3 codes of two bf16 pairs under scale code `scode` (as quantize8_bf16).
__device__ __forceinline__ uint32_t e4m3_encode4_bf16(uint32_t x0, uint32_t x1, uint32_t scode) {
  const float sv = scale_value(scode);
  const uint32_t lim = ((scode + 8u) << 7) | 0x60u;  // bf16 bits of 448 * 2^e
  const u16x2 lim_u = {(unsigned short)(lim | 0x8000u), (unsigned short)(lim | 0x8000u)};
  const i16x2 lim_i = {(short)lim, (short)lim};
  const u16x2 a0 = __builtin_elementwise_min(__builtin_bit_cast(u16x2, x0), lim_u);
  const u16x2 a1 = __builtin_elementwise_min(__builtin_bit_cast(u16x2, x1), lim_u);
  const i16x2 c0 = __builtin_elementwise_min(__builtin_bit_cast(i16x2, a0), lim_i);
  const i16x2 c1 = __builtin_elementwise_min(__builtin_bit_cast(i16x2, a1), lim_i);
  s16x2 r = {0, 0};
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, c0), sv, false);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(r, __builtin_bit_cast(bf16x2, c1), sv, true);
  return scode == 0xFFu ? 0x7F7F7F7Fu : __builtin_bit_cast(uint32_t, r);
}
__device__ __forceinline__ uint32_t e2m1_encode4_bf16(uint32_t x0, uint32_t x1, uint32_t scode) {
  const float sv = scale_value(scode);
  uint32_t r = 0;
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x0), sv, 0);
  r = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(r, __builtin_bit_cast(bf16x2, x1), sv, 1);
  return scode == 0xFFu ? 0x7777u : r;
}

// act(g) of the gated product: SiLU g / (1 + exp(-g)) on the hardware's exp2 and
// reciprocal (about 1 ulp each; the product is rounded to bf16 next), or GELU.
template <int ACT>
__device__ __forceinline__ float activation(float g) {
  if constexpr (ACT == 1) return epilogue<1>(g);
  return g * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * -1.4426950408889634f));
}

__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
  const bf16x2 p = {(__bf16)a, (__bf16)b};
  return __builtin_bit_cast(uint32_t, p);
}

// o is kept as f16 with a power of two for each 32 columns of a row: 2^-11 of a value at
// most is lost (f32 would be 2^-24, and twice the bytes written here and read by the
// sum; bf16 2^-8, as much as y's own rounding). The largest finite one of the 32 is
// brought to [2^14, 2^15); values under 2^-28 of it lose bits. `e` is its biased f32
// exponent, in 15 .. 254. A lane holds 16 of a fragment's 32 columns of a pair, lane ^ 32
// the others.
__device__ __forceinline__ uint32_t o_exponent(const f32x16& a) {
  auto both = [](uint32_t b) {
    const auto sw = __builtin_amdgcn_permlane32_swap(b, b, false, false);
    return max((uint32_t)sw[0], (uint32_t)sw[1]) >> 23;
  };
  float m = 0.f;  // (fmaxf passes over NaN)
#pragma unroll
  for (int i = 0; i < 16; ++i) m = fmaxf(m, __builtin_fabsf(a[i]));
  uint32_t e = both(__float_as_uint(m));
  if (__builtin_expect(__builtin_amdgcn_ballot_w64(e == 255u) != 0, 0)) {  // an infinity: again without
    uint32_t f = 0;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t b = __float_as_uint(__builtin_fabsf(a[i]));
      f = max(f, b < 0x7F800000u ? b : 0u);
    }
    e = both(f);
  }
  return min(max(e, 15u), 254u);
}
// The lane's 16 columns 8 q + 4 hi .. + 3 (q = 0 .. 3), two dwords for each q.
__device__ __forceinline__ void o_pack(const f32x16& a, uint32_t e, uint32_t (&c)[8]) {
  const float f = __uint_as_float((268u - e) << 23);  // 2^(14 - (e - 127))
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const f16x2 x = {(_Float16)(a[2 * q] * f), (_Float16)(a[2 * q + 1] * f)};
    c[q] = __builtin_bit_cast(uint32_t, x);
  }
}

// Which tile a workgroup takes: groups of 4 tiles along the pairs x all weight tiles,
// of which each XCD takes a contiguous range, as in mx_fp4_gemm.hip. The number of
// tiles is known on the device only; workgroups past it take none.
__device__ __forceinline__ bool find_tile(const ProductParams& p, ExpertTile& tile, int& tn) {
  const int tiles_m = *p.n_tiles;
  const uint32_t total = (uint32_t)tiles_m * (uint32_t)p.tiles_n;
  if (blockIdx.x >= total) return false;
  constexpr int GM = 4;
  const int lid = (int)xcd_order(blockIdx.x, total);
  const int group = lid / (GM * p.tiles_n), gm = min(tiles_m - group * GM, GM);
  const int in_group = lid - group * GM * p.tiles_n;
  tile = p.tiles[group * GM + in_group % gm];
  tn = in_group / gm;
  return true;
}

}  // namespace
}  // namespace mx

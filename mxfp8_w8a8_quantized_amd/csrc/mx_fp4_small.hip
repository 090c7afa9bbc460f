// Few-token linear on MXFP4 weights: y = bf16(epi(sum_k xhat what + bias))
// for one to a few hundred tokens, with MXFP4 or MXFP8 activations, either
// quantized already (slab operands) or bf16 rows quantized in the kernel.
//
// Bound by the weights' bytes (N K / 2, read once from HBM) for a few tokens,
// and by the token operand's re-reads from the L2 (once per weight tile) for
// hundreds. A workgroup of 8 waves takes 16 WB weight rows and 16 TB tokens;
// its waves split K among themselves and add their partial sums in LDS in
// wave order, so there is one launch, no workspace and no dependence on
// timing, and N / (16 WB) workgroups are enough to fill the GPU.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, weights as the A operand (found on the
// device): lane l holds row l % 16; an E2M1 operand is 16 bytes, K 32 G .. + 31
// of the 128 with G = l / 16; an E4M3 operand is 32 bytes, K 16 G .. + 15 and
// 64 + 16 G .. + 15; the scale of lane l is that of K group G of row l % 16.
// Output: lane l holds D[4 (l / 16) + i][l % 16]. A 16-row block of an MXFP4
// slab is one 1 KB run in lane order, so operands go from memory straight to
// registers; nothing is shared between the waves but the final sums.
#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr int kWaves = 8;

// Token operand: MXFP4 or MXFP8 slab, or bf16 rows quantized to either.
enum { SRC_FP4 = 0, SRC_FP8 = 1, SRC_BF16_FP4 = 2, SRC_BF16_FP8 = 3 };

struct FewParams {
  const uint8_t* x;   // slab codes, or bf16 rows
  const uint8_t* xs;  // slab scales
  const uint8_t* wq;
  const uint8_t* ws;
  const uint16_t* bias;
  uint16_t* y;
  int64_t ldx, RM, RN;
  int M, N, K;
  int tiles_m;
};

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

// The operands of one 128-K slab as loaded.
template <int SRC, int WB, int TB>
struct Step {
  static constexpr int NX = SRC == SRC_FP4 ? 1 : SRC == SRC_FP8 ? 2 : 4;  // 16-byte loads per token fragment
  i32x4 a[WB];
  i32x4 b[TB][NX];
  int sa[WB], sb[TB];
};

template <int SRC, int WB, int TB>
__device__ __forceinline__ void load_step(Step<SRC, WB, TB>& s, const FewParams& p, int64_t sl, int n0, int m0,
                                          int lane) {
  const int r = lane & 15, G = lane >> 4;
  const uint8_t* a = p.wq + (sl * (p.RN / 16) + n0 / 16) * 1024 + lane * 16;
  const uint8_t* sa = p.ws + (sl * p.RN + n0 + r) * 4 + G;
#pragma unroll
  for (int i = 0; i < WB; ++i) {
    s.a[i] = *(const i32x4*)(a + i * 1024);
    s.sa[i] = sa[i * 64];
  }
  const i32x4 zero = {0, 0, 0, 0};
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    if constexpr (SRC == SRC_FP4) {
      s.b[j][0] = *(const i32x4*)(p.x + (sl * (p.RM / 16) + m0 / 16 + j) * 1024 + lane * 16);
      s.sb[j] = p.xs[(sl * p.RM + m0 + 16 * j + r) * 4 + G];
    } else if constexpr (SRC == SRC_FP8) {
      // Two 64-K slabs; the second is past K where K % 128 = 64 (its codes
      // are taken as zeros: the weights' are, but a product with NaN bits
      // there would not be).
      const bool two = sl * 128 + 64 < p.K;
      const int64_t row = m0 + 16 * j + r;
      s.b[j][0] = *(const i32x4*)(p.x + (2 * sl * p.RM + row) * 64 + 16 * G);
      s.b[j][1] = two ? *(const i32x4*)(p.x + ((2 * sl + 1) * p.RM + row) * 64 + 16 * G) : zero;
      s.sb[j] = G < 2 || two ? p.xs[((2 * sl + (G >> 1)) * p.RM + row) * 2 + (G & 1)] : 0;
    } else {
      // Rows past M repeat the last one; their outputs are not stored.
      const int64_t row = min(m0 + 16 * j + r, p.M - 1);
      const uint16_t* x = (const uint16_t*)p.x + row * p.ldx;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // E2M1: 32 consecutive elements; E4M3: two runs of 16.
        const int64_t k = sl * 128 + (SRC == SRC_BF16_FP4 ? 32 * G + 8 * u : 64 * (u >> 1) + 16 * G + 8 * (u & 1));
        s.b[j][u] = k < p.K ? *(const i32x4*)(x + k) : zero;
      }
    }
  }
}

template <int SRC, int WB, int TB>
__device__ __forceinline__ void mma_step(f32x4 (&acc)[WB][TB], const Step<SRC, WB, TB>& s, int lane) {
  constexpr int FB = SRC == SRC_FP4 || SRC == SRC_BF16_FP4 ? 4 : 0;  // token format: E2M1 or E4M3
#pragma unroll
  for (int j = 0; j < TB; ++j) {
    i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0};
    int sb;
    if constexpr (SRC == SRC_FP4) {
      b = i32x8{s.b[j][0][0], s.b[j][0][1], s.b[j][0][2], s.b[j][0][3], 0, 0, 0, 0};
      sb = s.sb[j];
    } else if constexpr (SRC == SRC_FP8) {
      b = i32x8{s.b[j][0][0], s.b[j][0][1], s.b[j][0][2], s.b[j][0][3],
                s.b[j][1][0], s.b[j][1][1], s.b[j][1][2], s.b[j][1][3]};
      sb = s.sb[j];
    } else if constexpr (SRC == SRC_BF16_FP4) {
      const uint32_t m = max(amax16(s.b[j][0], s.b[j][1]), amax16(s.b[j][2], s.b[j][3]));
      sb = (int)fp4_scale_code(m >> 7);
#pragma unroll
      for (int u = 0; u < 4; ++u)
        b[u] = (int)fp4_encode8_bf16((uint32_t)s.b[j][u][0], (uint32_t)s.b[j][u][1], (uint32_t)s.b[j][u][2],
                                     (uint32_t)s.b[j][u][3], (uint32_t)sb);
    } else {
      // The lane holds halves of K groups G / 2 and 2 + G / 2; the other
      // halves are 16 lanes away. It passes the MFMA the scale of group G:
      // its own first for G = 0, its own second for G = 3, and lanes of
      // G = 1 and 2 swap.
      const int G = lane >> 4;
      uint32_t m0 = amax16(s.b[j][0], s.b[j][1]), m1 = amax16(s.b[j][2], s.b[j][3]);
      m0 = max(m0, (uint32_t)__shfl_xor((int)m0, 16, 64));
      m1 = max(m1, (uint32_t)__shfl_xor((int)m1, 16, 64));
      const uint32_t c0 = scale_code_from_exponent(m0 >> 7), c1 = scale_code_from_exponent(m1 >> 7);
      const int swapped = __shfl_xor((int)(G == 1 ? c1 : c0), 48, 64);
      sb = G == 0 ? (int)c0 : G == 3 ? (int)c1 : swapped;
      const i32x2 e0 = e4m3_encode8_bf16(s.b[j][0], c0), e1 = e4m3_encode8_bf16(s.b[j][1], c0);
      const i32x2 e2 = e4m3_encode8_bf16(s.b[j][2], c1), e3 = e4m3_encode8_bf16(s.b[j][3], c1);
      b = i32x8{e0[0], e0[1], e1[0], e1[1], e2[0], e2[1], e3[0], e3[1]};
    }
#pragma unroll
    for (int i = 0; i < WB; ++i) {
      const i32x8 a = {s.a[i][0], s.a[i][1], s.a[i][2], s.a[i][3], 0, 0, 0, 0};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i][j], 4, FB, 0, s.sa[i], 0, sb);
    }
  }
}

// U: slabs whose loads are issued together.
template <int SRC, int WB, int TB, int U, int EPI>
__global__ __launch_bounds__(64 * kWaves) void fp4_few_kernel(FewParams p) {
  __shared__ f32x4 sums[kWaves][WB * TB][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Token tile fastest within an XCD's range of workgroups, so that those
  // that share a weight tile share an L2.
  const uint32_t lid = xcd_order(blockIdx.x, gridDim.x);
  const int tn = (int)(lid / (uint32_t)p.tiles_m), tm = (int)(lid - (uint32_t)tn * (uint32_t)p.tiles_m);
  const int n0 = tn * 16 * WB, m0 = tm * 16 * TB;
  const int S = (int)fp4_slabs(p.K);
  const int s0 = wave * S / kWaves, s1 = (wave + 1) * S / kWaves;
  f32x4 acc[WB][TB];
#pragma unroll
  for (int i = 0; i < WB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  for (int s = s0; s < s1; s += U) {
    // Slabs past the wave's range are loaded as its last one and not used,
    // so that the loads stay in one straight run.
    Step<SRC, WB, TB> st[U];
#pragma unroll
    for (int u = 0; u < U; ++u) load_step(st[u], p, min(s + u, s1 - 1), n0, m0, lane);
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (s + u < s1) mma_step(acc, st[u], lane);
  }
#pragma unroll
  for (int i = 0; i < WB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) sums[wave][i * TB + j][lane] = acc[i][j];
  __syncthreads();
  for (int f = wave; f < WB * TB; f += kWaves) {
    const int i = f / TB, j = f - i * TB;
    const int n = n0 + 16 * i + 4 * (lane >> 4), m = m0 + 16 * j + (lane & 15);
    f32x4 v = sums[0][f][lane];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) {
      const f32x4 o = sums[w][f][lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += o[r];
    }
    if (n >= p.N || m >= p.M) continue;
    if (p.bias != nullptr) {
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += (float)__builtin_bit_cast(_Float16, p.bias[n + r]);
    }
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] = epilogue<EPI>(v[r]);
    const bf16x2 q0 = {(__bf16)v[0], (__bf16)v[1]}, q1 = {(__bf16)v[2], (__bf16)v[3]};
    *(i32x2*)(p.y + (int64_t)m * p.N + n) = i32x2{__builtin_bit_cast(int, q0), __builtin_bit_cast(int, q1)};
  }
}

template <int SRC, int WB, int TB, int U>
hipError_t launch_few(FewParams& p, int epi, hipStream_t st) {
  p.tiles_m = (p.M + 16 * TB - 1) / (16 * TB);
  const unsigned blocks = (unsigned)(p.tiles_m * ((p.N + 16 * WB - 1) / (16 * WB)));
  if (epi == 1)
    hipLaunchKernelGGL((fp4_few_kernel<SRC, WB, TB, U, 1>), dim3(blocks), dim3(64 * kWaves), 0, st, p);
  else
    hipLaunchKernelGGL((fp4_few_kernel<SRC, WB, TB, U, 0>), dim3(blocks), dim3(64 * kWaves), 0, st, p);
  return hipGetLastError();
}

template <int SRC>
hipError_t dispatch_slab(FewParams& p, int epi, hipStream_t st) {
  if (p.M <= 16) return launch_few<SRC, 1, 1, 6>(p, epi, st);
  if (p.M <= 32) return launch_few<SRC, 1, 2, 4>(p, epi, st);
  if (p.M <= 64) return launch_few<SRC, 1, 4, 2>(p, epi, st);
  return launch_few<SRC, 1, 8, 2>(p, epi, st);
}

}  // namespace

hipError_t launch_fp4_linear_few(int fp8, const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K,
                                 const uint8_t* wq, const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                 hipStream_t stream) {
  FewParams p;
  p.x = xq;
  p.xs = xs;
  p.wq = wq;
  p.ws = ws;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldx = 0;
  p.RM = slab_rows(M);
  p.RN = slab_rows(N);
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  return fp8 ? dispatch_slab<SRC_FP8>(p, epi, stream) : dispatch_slab<SRC_FP4>(p, epi, stream);
}

hipError_t launch_fp4_linear_rows(int fp8, const void* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                                  const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                  hipStream_t stream) {
  FewParams p;
  p.x = (const uint8_t*)x;
  p.xs = nullptr;
  p.wq = wq;
  p.ws = ws;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.ldx = ldx;
  p.RM = 0;
  p.RN = slab_rows(N);
  p.M = (int)M;
  p.N = (int)N;
  p.K = (int)K;
  return fp8 ? launch_few<SRC_BF16_FP8, 1, 1, 4>(p, epi, stream) : launch_few<SRC_BF16_FP4, 1, 1, 4>(p, epi, stream);
}

}  // namespace mx

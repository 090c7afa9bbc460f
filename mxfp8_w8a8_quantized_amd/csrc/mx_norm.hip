// RMS norm with the residual's addition, into the slab of a quantized linear:
//
//   h = x + residual, rounded to the residual's type (h = x without one)
//   y = bf16( h * gain / sqrt(mean(h^2) + eps) )
//   q, s = the MX quantization of y: MXFP8 (mx_device.h) or MXFP4
//          (mx_fp4_device.h) codes and scales in their slab layouts
//
// h is written back as the new residual, y only where it is asked for. One
// pass over memory: a row stays in registers between its sum of squares and
// its codes. Bound by memory: 2 bytes of x, the residual twice and the codes
// per element.
//
// The squares are summed, and h * rstd * gain is multiplied out, in float64.
// The sum then neither overflows nor underflows for any bf16 or f32 row, and
// a code differs from the formula's only where float64 itself is in doubt. With
// a residual the float64 operations (three an element, and four conversions)
// stay hidden behind memory; without one they bound the kernel at about 1.4e12
// elements a second (75348 x 5120: 264 us, 4.4 TB/s).
//
// norm_tile_kernel, for many rows: a block takes 8 rows, a wave each; the
// codes pass through LDS in slab order, so that every slab's part of them
// leaves as one run (512 bytes; four of 128 for MXFP4) instead of one piece
// per row. norm_row_kernel, for few rows: one row per block, codes stored
// directly, the pad rows zeroed by blocks of their own.
#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

enum { RES_NONE = 0, RES_BF16 = 1, RES_F32 = 2 };

struct NormParams {
  const uint16_t* x;
  const void* res;
  const void* gain;  // null: 1
  void* res_out;     // null: not stored
  uint16_t* y;       // null: not stored
  uint8_t* q;
  uint8_t* s;
  int64_t ldx, ldr, ldo, ldy;
  int64_t M, R;
  int K;
  int gain_f32;
  double eps;
};

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

// The wave's part of row `row`: chunks c = first, first + step, ... (NCH of
// them) of 512 elements, 8 per lane. Loads x and the residual, stores the new
// residual and returns the lane's sum of squares.
template <int RES, int NCH>
__device__ __forceinline__ double load_row(const NormParams& p, int64_t row, int first, int step, int lane,
                                           Held<RES> (&h)[NCH]) {
  i32x4 xv[NCH], ra[NCH], rb[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int k = (first + c * step) * 512 + 8 * lane;
    const bool in = k < p.K;
    xv[c] = in ? *(const i32x4*)(p.x + row * p.ldx + k) : i32x4{0, 0, 0, 0};
    if constexpr (RES == RES_BF16)
      ra[c] = in ? *(const i32x4*)((const uint16_t*)p.res + row * p.ldr + k) : i32x4{0, 0, 0, 0};
    if constexpr (RES == RES_F32) {
      const float* r = (const float*)p.res + row * p.ldr + k;
      ra[c] = in ? *(const i32x4*)r : i32x4{0, 0, 0, 0};
      rb[c] = in ? *(const i32x4*)(r + 4) : i32x4{0, 0, 0, 0};
    }
  }
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const uint32_t w = (uint32_t)xv[c][u];
      if constexpr (RES == RES_NONE) {
        h[c].w[u] = w;
      } else if constexpr (RES == RES_BF16) {
        const uint32_t r = (uint32_t)ra[c][u];
        h[c].w[u] = pack_bf16(bf16_lo(w) + bf16_lo(r), bf16_hi(w) + bf16_hi(r));
      } else {
        const uint32_t r0 = (uint32_t)(u < 2 ? ra[c][2 * u] : rb[c][2 * u - 4]);
        const uint32_t r1 = (uint32_t)(u < 2 ? ra[c][2 * u + 1] : rb[c][2 * u - 3]);
        h[c].w[2 * u] = __float_as_uint(bf16_lo(w) + __uint_as_float(r0));
        h[c].w[2 * u + 1] = __float_as_uint(bf16_hi(w) + __uint_as_float(r1));
      }
    }
    const int k = (first + c * step) * 512 + 8 * lane;
    if (RES != RES_NONE && p.res_out != nullptr && k < p.K) {
      if constexpr (RES == RES_F32) {
        float* o = (float*)p.res_out + row * p.ldo + k;
        *(i32x4*)o = i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
        *(i32x4*)(o + 4) = i32x4{(int)h[c].w[4], (int)h[c].w[5], (int)h[c].w[6], (int)h[c].w[7]};
      } else {
        *(i32x4*)((uint16_t*)p.res_out + row * p.ldo + k) =
            i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double d = (double)h[c].at(i);
      sum = __builtin_fma(d, d, sum);
    }
  }
  return sum;
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

// The bf16 norm of a lane's 8 elements at k, as packed pairs.
template <int RES>
__device__ __forceinline__ void scale8(const NormParams& p, const Held<RES>& h, int k, double rstd, uint32_t (&out)[4]) {
  float g[8];
  if (p.gain == nullptr || k >= p.K) {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = 1.f;
  } else if (p.gain_f32) {
    const f32x4 a = *(const f32x4*)((const float*)p.gain + k), b = *(const f32x4*)((const float*)p.gain + k + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = a[i];
      g[4 + i] = b[i];
    }
  } else {
    const i32x4 a = *(const i32x4*)((const uint16_t*)p.gain + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[2 * i] = bf16_lo((uint32_t)a[i]);
      g[2 * i + 1] = bf16_hi((uint32_t)a[i]);
    }
  }
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    v[i] = (float)((double)h.at(i) * rstd * (double)g[i]);
    // Two roundings, f64 to f32 to bf16, as written: left alone, the compiler
    // merges them into one that it spells out in ten operations an element.
    asm volatile("" : "+v"(v[i]));
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = pack_bf16(v[2 * i], v[2 * i + 1]);
}

__device__ __forceinline__ double rstd_of(const NormParams& p, double sum) {
  return 1.0 / __builtin_sqrt(sum / (double)p.K + p.eps);
}

__device__ __forceinline__ void store_y(const NormParams& p, int64_t row, int k, const uint32_t (&v)[4]) {
  if (p.y != nullptr && k < p.K)
    *(i32x4*)(p.y + row * p.ldy + k) = i32x4{(int)v[0], (int)v[1], (int)v[2], (int)v[3]};
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

template <int RES, bool FP4, int NCH>
__global__ __launch_bounds__(64 * kTileRows, 2) void norm_tile_kernel(NormParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using St = Stage<FP4>;
  const int t = threadIdx.x, lane = t & 63, rl = t >> 6;  // wave rl: row rl of the tile
  const int S = St::slabs(p.K);
  uint8_t* sc_lds = smem + S * St::kCodes;
  const int64_t r0 = (int64_t)xcd_order(blockIdx.x, gridDim.x) * kTileRows;
  const int64_t row = r0 + rl;
  const bool real = row < p.M;
  Held<RES> h[NCH];
  double sum = 0.0;
  if (real) sum = wave_sum(load_row<RES, NCH>(p, row, 0, 1, lane, h));
  const double rstd = rstd_of(p, sum);
  hold(h);
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4] = {0, 0, 0, 0};
    if (real) {
      scale8(p, h[ch], k, rstd, v);
      store_y(p, row, k, v);
    }
    if constexpr (FP4) {
      if (k >= p.K) v[0] = v[1] = v[2] = v[3] = 0;  // groups past K: zero codes and scales
      uint32_t sc;
      const uint32_t code = fp4_quantize8_bf16(v, sc);
      const int sg = ch * 16 + (lane >> 2);
      if (sg < 4 * S) {
        *(uint32_t*)(smem + sg * 144 + rl * 16 + (lane & 3) * 4) = code;
        if ((lane & 3) == 0) sc_lds[(sg >> 2) * 32 + rl * 4 + (sg & 3)] = (uint8_t)sc;
      }
    } else {
      uint32_t code[2], sc;
      quantize8_bf16(v, code, sc);
      const int sl = ch * 8 + (lane >> 3);
      if (sl < S) {
        *(i32x2*)(smem + sl * 576 + rl * 64 + (lane & 7) * 8) = i32x2{(int)code[0], (int)code[1]};
        if ((lane & 3) == 0) sc_lds[sl * 16 + rl * 2 + ((lane >> 2) & 1)] = (uint8_t)sc;
      }
    }
  }
  __syncthreads();
  // 32 threads per slab: 512 bytes of codes.
  const int piece = t & 31;
  for (int sl = t >> 5; sl < S; sl += 2 * kTileRows) {
    if constexpr (FP4) {
      const int g = piece >> 3, r = piece & 7;
      *(i32x4*)(p.q + ((int64_t)sl * (p.R / 16) + r0 / 16) * 1024 + g * 256 + ((r0 & 8) + r) * 16) =
          *(const i32x4*)(smem + (sl * 4 + g) * 144 + r * 16);
    } else {
      *(i32x4*)(p.q + ((int64_t)sl * p.R + r0) * 64 + piece * 16) = *(const i32x4*)(smem + sl * 576 + piece * 16);
    }
  }
  constexpr int P = St::kScales / 16;  // 16-byte scale pieces per slab
  for (int u = t; u < S * P; u += 64 * kTileRows)
    *(i32x4*)(p.s + ((int64_t)(u / P) * p.R + r0) * (St::kScales / kTileRows) + (u % P) * 16) =
        *(const i32x4*)(sc_lds + u * 16);
}

// Blocks 0 .. M-1: one row each, WPR waves. Blocks M ..: pad rows of one slab.
template <int RES, bool FP4, int WPR, int NCH>
__global__ __launch_bounds__(64 * WPR) void norm_row_kernel(NormParams p) {
  __shared__ double part[WPR];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int S = Stage<FP4>::slabs(p.K);
  if ((int64_t)blockIdx.x >= p.M) {
    const int64_t sl = (int64_t)blockIdx.x - p.M;
    const i32x4 zero = {0, 0, 0, 0};
    if constexpr (FP4) {
      for (int64_t u = p.M / 16 * 64 + t; u < p.R * 4; u += 64 * WPR)
        if (u / 64 * 16 + (u & 15) >= p.M) *(i32x4*)(p.q + sl * p.R * 64 + u * 16) = zero;
      for (int64_t r = p.M + t; r < p.R; r += 64 * WPR) *(uint32_t*)(p.s + (sl * p.R + r) * 4) = 0;
    } else {
      for (int64_t u = p.M * 4 + t; u < p.R * 4; u += 64 * WPR) *(i32x4*)(p.q + sl * p.R * 64 + u * 16) = zero;
      for (int64_t r = p.M + t; r < p.R; r += 64 * WPR) *(uint16_t*)(p.s + (sl * p.R + r) * 2) = 0;
    }
    return;
  }
  const int64_t row = blockIdx.x;
  Held<RES> h[NCH];
  double sum = wave_sum(load_row<RES, NCH>(p, row, wave, WPR, lane, h));
  if (lane == 0) part[wave] = sum;
  __syncthreads();
  sum = 0.0;
#pragma unroll
  for (int i = 0; i < WPR; ++i) sum += part[i];
  const double rstd = rstd_of(p, sum);
  hold(h);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = wave + c * WPR;
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4];
    scale8(p, h[c], k, rstd, v);
    store_y(p, row, k, v);
    if constexpr (FP4) {
      if (k >= p.K) v[0] = v[1] = v[2] = v[3] = 0;
      uint32_t sc;
      const uint32_t code = fp4_quantize8_bf16(v, sc);
      const int sg = ch * 16 + (lane >> 2);
      if (sg < 4 * S) {
        *(uint32_t*)(p.q + ((int64_t)(sg >> 2) * (p.R / 16) + row / 16) * 1024 + (sg & 3) * 256 + (row & 15) * 16 +
                     (lane & 3) * 4) = code;
        if ((lane & 3) == 0) p.s[((int64_t)(sg >> 2) * p.R + row) * 4 + (sg & 3)] = (uint8_t)sc;
      }
    } else {
      uint32_t code[2], sc;
      quantize8_bf16(v, code, sc);
      const int sl = ch * 8 + (lane >> 3);
      if (sl < S) {
        *(i32x2*)(p.q + ((int64_t)sl * p.R + row) * 64 + (lane & 7) * 8) = i32x2{(int)code[0], (int)code[1]};
        if ((lane & 3) == 0) p.s[((int64_t)sl * p.R + row) * 2 + ((lane >> 2) & 1)] = (uint8_t)sc;
      }
    }
  }
}

template <int RES, bool FP4, int NCH>
hipError_t launch_tile(const NormParams& p, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = norm_tile_kernel<RES, FP4, NCH>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Stage<FP4>::bytes(512 * NCH), configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.R / kTileRows)), dim3(64 * kTileRows), Stage<FP4>::bytes(p.K), st, p);
  return hipGetLastError();
}

template <int RES, bool FP4, int WPR, int NCH>
hipError_t launch_row(const NormParams& p, hipStream_t st) {
  const unsigned blocks = (unsigned)(p.M + (p.R > p.M ? Stage<FP4>::slabs(p.K) : 0));
  hipLaunchKernelGGL((norm_row_kernel<RES, FP4, WPR, NCH>), dim3(blocks), dim3(64 * WPR), 0, st, p);
  return hipGetLastError();
}

// Rows from which the tiled form is taken. Its blocks take eight rows each and
// their stores are whole lines, but a wave waits for its whole row; the row form
// spreads a row over 4 or 8 waves. us, tiled against row form, to MXFP8:
//                  no residual    bf16 residual          f32 residual
//   1024 x 2048    5.6, 4.9       6.8, 5.8               7.9, 6.5
//   2048 x 2048    5.9, 7.4       8.0, 9.3               11.0, 10.8
//   8192 x 2048    14.6, 22.6     22.4, 25.6             34.0, 31.3
//   75348 x 2048   110, 207       210, 233               322, 333
//   8192 x 4096    29.0, 28.0     46.1, 40.9             94.1, 78.4
//   32768 x 4096   99, 119        191, 197               317, 303
//   75348 x 4096   212, 266       426, 481               698, 737
//   32768 x 5120   122, 152       237, 263               385, 399
//   75348 x 5120   261, 344       521 (5.2 TB/s), 648    860, 969
//   32768 x 6144   181, 172       357, 307
//   75348 x 6144   392, 394       789, 774
//   75348 x 8192   451, 538       953, 1047
// To MXFP4 the tiled form does better by another 5 to 15%. One rule for all: at the
// border it costs up to 16% (bf16 residual, 6144, whose tiles hold registers for
// 8192) and 9% (f32 residual, 8192 x 2048) against the better form.
constexpr int64_t kTileMinRows = 32768;
constexpr int64_t kTileMinRowsShort = 2048;  // K <= 2048

template <int RES, bool FP4>
hipError_t dispatch(const NormParams& p, hipStream_t st) {
  const int ch = (p.K + 511) / 512;
  if (p.M >= (ch <= 4 ? kTileMinRowsShort : kTileMinRows)) {
    if (ch <= 4) return launch_tile<RES, FP4, 4>(p, st);
    if (ch <= 8) return launch_tile<RES, FP4, 8>(p, st);
    if (ch <= 10) return launch_tile<RES, FP4, 10>(p, st);
    if constexpr (RES != RES_F32)  // an f32 row of 16 chunks does not fit the registers
      if (ch <= 16) return launch_tile<RES, FP4, 16>(p, st);
  }
  if (ch <= 8) return launch_row<RES, FP4, 4, 2>(p, st);
  if (ch <= 12) return launch_row<RES, FP4, 4, 3>(p, st);
  if (ch <= 16) return launch_row<RES, FP4, 4, 4>(p, st);
  if (ch <= 24) return launch_row<RES, FP4, 8, 3>(p, st);
  if (ch <= 32) return launch_row<RES, FP4, 8, 4>(p, st);
  return launch_row<RES, FP4, 8, 16>(p, st);
}

}  // namespace

hipError_t launch_rmsnorm_slab(const RmsNormArgs& a, hipStream_t stream) {
  NormParams p;
  p.x = (const uint16_t*)a.x;
  p.res = a.residual;
  p.gain = a.weight;
  p.res_out = a.residual_out;
  p.y = (uint16_t*)a.y;
  p.q = a.q;
  p.s = a.s;
  p.ldx = a.ldx;
  p.ldr = a.ldr;
  p.ldo = a.ldo;
  p.ldy = a.ldy;
  p.M = a.M;
  p.R = slab_rows(a.M);
  p.K = (int)a.K;
  p.gain_f32 = a.weight_f32;
  p.eps = a.eps;
  if (a.residual == nullptr) return a.fp4 ? dispatch<RES_NONE, true>(p, stream) : dispatch<RES_NONE, false>(p, stream);
  if (a.residual_f32) return a.fp4 ? dispatch<RES_F32, true>(p, stream) : dispatch<RES_F32, false>(p, stream);
  return a.fp4 ? dispatch<RES_BF16, true>(p, stream) : dispatch<RES_BF16, false>(p, stream);
}

}  // namespace mx

// The norms around a block, fused with its gate and the scaled residual, into the
// slab of the next quantized linear:
//
//   n = x, or x * post_weight / sqrt(mean(x^2) + eps)
//   h = residual_scale * residual + gate * n, rounded to the residual's type
//   y = bf16( norm(h) * weight * (1 + scale) + shift ), the norm
//       h / sqrt(mean(h^2) + eps), or (h - mean h) / sqrt(var h + eps)
//   q, s = the MX quantization of y (MXFP8 or MXFP4), where a slab is wanted
//
// One pass over memory: a row stays in registers through up to three sums (of x^2,
// of h and h^2, and for an f32 residual of the squares around the mean), 7 bytes an
// element with a bf16 residual and MXFP8 codes. Few rows take a block each, many are
// tiled, a wave a row, with the codes passing through LDS.
//
// Sums and products are f64, each result rounded to f32 and then to its type: y is
// next rounded to few bits, where a sum off in its last f32 bit moves a code. What
// bounds it is the memory (5.2 TB/s would take 521 us for 75348 x 5120, bf16
// residual), with gate, post norm or modulation the 37 to 45 vector operations an
// element, a quarter of them conversions to f64. Measured there: RMS norm 555 us, layer
// norm without a gain 547, with gate and modulation 634, and a gain besides 681 (4.0
// TB/s), RMS norm behind a post norm 718; f32 products were no faster there, and move one
// code in 1e4. 4096 x 5120: 38 us; one row: 6 us. Rows of more than 16384 elements have 16
// chunks a wave and spill registers: 4096 x 20480 626 us (f32 residual 979), 114 (179) at
// the copy's rate, where 4096 x 16384 takes 127.
#include "mx_internal.h"
#include "mx_norm_device.h"

namespace mx {
namespace {

// A vector's row for one row of x. Where there is none, its neutral values are
// loaded instead, from the same eight for all k (mask 0), so that the code has no
// branches and one chunk's vectors are on their way while the chunk before is
// computed.
struct Vector {
  __amdgpu_buffer_rsrc_t r;
  int mask;
};
// 1, -0 (which changes no sum, not a zero's sign either) and 0; f32, then bf16.
__device__ const uint32_t kNeutral[3][2][8] = {
    {{0x3F800000, 0x3F800000, 0x3F800000, 0x3F800000, 0x3F800000, 0x3F800000, 0x3F800000, 0x3F800000},
     {0x3F803F80, 0x3F803F80, 0x3F803F80, 0x3F803F80}},
    {{0x80000000, 0x80000000, 0x80000000, 0x80000000, 0x80000000, 0x80000000, 0x80000000, 0x80000000},
     {0x80008000, 0x80008000, 0x80008000, 0x80008000}},
    {{0, 0, 0, 0, 0, 0, 0, 0}, {0, 0, 0, 0}}};
enum Neutral { ONE, NO_TERM, ZERO };
template <bool VF32>
__device__ __forceinline__ Vector vector_of(const BlockNormArgs& p, const void* v, int64_t row, int64_t ld, Neutral n) {
  constexpr int ES = VF32 ? 4 : 2;
  if (v == nullptr) return {make_rsrc(kNeutral[n][VF32 ? 0 : 1], 32u), 0};
  return {make_rsrc((const uint8_t*)v + row * ld * ES, (uint32_t)p.K * ES), -1};
}
struct Vectors {
  Vector post, gate, weight, scale, shift;
};
template <bool VF32>
__device__ __forceinline__ Vectors vectors_of(const BlockNormArgs& p, int64_t row) {
  const int64_t g = row / p.gate_period, m = row / p.mod_period;
  return {vector_of<VF32>(p, p.post_weight, 0, 0, ONE), vector_of<VF32>(p, p.gate, g, p.ldg, ONE),
          vector_of<VF32>(p, p.weight, 0, 0, ONE), vector_of<VF32>(p, p.scale, m, p.ldm, ZERO),
          vector_of<VF32>(p, p.shift, m, p.ldm, NO_TERM)};
}

// Eight consecutive values of a vector as loaded (past K zeros).
template <bool VF32>
struct Eight {
  i32x4 w[VF32 ? 2 : 1];
  __device__ __forceinline__ void load(const Vector& v, int k) {
    k &= v.mask;
    w[0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(v.r, k * (VF32 ? 4 : 2), 0, 0));
    if constexpr (VF32) w[1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(v.r, k * 4 + 16, 0, 0));
  }
  __device__ __forceinline__ double at(int i) const {
    if constexpr (VF32) return __uint_as_float((uint32_t)w[i >> 2][i & 3]);
    return (i & 1) ? bf16_hi((uint32_t)w[0][i >> 1]) : bf16_lo((uint32_t)w[0][i >> 1]);
  }
};

__device__ __forceinline__ double rstd_of(const BlockNormArgs& p, double sum) {
  return 1.0 / __builtin_sqrt(sum / (double)p.K + p.eps);
}

// Rounds f64 to f32; the asm keeps the rounding to bf16 that follows apart (merged,
// the compiler spells the two out in ten operations an element).
__device__ __forceinline__ float round_f32(double d) {
  float f = (float)d;
  asm volatile("" : "+v"(f));
  return f;
}

// A value that is the same in all lanes, in scalar registers.
__device__ __forceinline__ double uniform(double v) {
  const i32x2 w = __builtin_bit_cast(i32x2, v);
  return __builtin_bit_cast(double, i32x2{__builtin_amdgcn_readfirstlane(w[0]), __builtin_amdgcn_readfirstlane(w[1])});
}

// What goes before h and what follows the norm, where a kernel is built for it: a
// branch on an option costs the tiled form up to a tenth, the neutral values of what
// is not there as much again (75348 x 5120, RMS norm with a weight: 666 us with both,
// 546 without; layer norm with gate and modulation 663 and 639).
enum Pre { PRE_ANY = -1, PRE_NONE, PRE_GATE, PRE_POST };  // PRE_POST: with or without a gate
enum Mod { MOD_ANY = -1, MOD_NONE, MOD_SOME };

struct Statistics {
  double mean, rstd;  // the mean is 0 for the RMS norm
};

// The wave's part of row `row`: chunks first, first + step, ... (NCH of them) of
// 512 elements, 8 per lane. Computes and stores h, and returns the row's
// statistics. total(i, v): the row's sums of its waves' i-th sums v, in all lanes.
//
// The sums of h and h^2 are taken as h is made. For bf16 h the variance is their
// difference: a value other than the largest is at least 2^-8 of it away, so a
// variance that is not 0 is at least 2^-16 / K of the mean square. Where it is that
// small all values but a few are the same, the sums of their 16-bit squares are
// exact, and the mean's rounding, 2^-53 of the mean square, is 2^-21 of the variance
// at the largest K, 65536. Values that are all the same leave exactly 0. f32 h is
// summed again, around its mean.
template <int RES, bool VF32, int PRE, int NCH, typename Total>
__device__ __forceinline__ Statistics make_h(const BlockNormArgs& p, const Vectors& vec, int64_t row, int first, int step,
                                             int lane, Held<RES> (&h)[NCH], Total&& total) {
  i32x4 xv[NCH];
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int k = (first + c * step) * 512 + 8 * lane;
    const bool in = k < p.K;
    xv[c] = in ? *(const i32x4*)((const uint16_t*)p.x + row * p.ldx + k) : i32x4{0, 0, 0, 0};
    i32x4 ra = {0, 0, 0, 0}, rb = {0, 0, 0, 0};
    if constexpr (RES == RES_BF16) {
      if (in) ra = *(const i32x4*)((const uint16_t*)p.residual + row * p.ldr + k);
    } else {
      const float* r = (const float*)p.residual + row * p.ldr + k;
      if (in) {
        ra = *(const i32x4*)r;
        rb = *(const i32x4*)(r + 4);
      }
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      h[c].w[u] = (uint32_t)ra[u];
      if constexpr (RES == RES_F32) h[c].w[4 + u] = (uint32_t)rb[u];
    }
  }
  // Elements past K are zeros, but not the mean away from it.
  auto in = [&](int c) { return (first + c * step) * 512 + 8 * lane < p.K; };
  auto x_at = [&](int c, int i) -> double {
    return (i & 1) ? bf16_hi((uint32_t)xv[c][i >> 1]) : bf16_lo((uint32_t)xv[c][i >> 1]);
  };
  double post = 1.0;
  const bool with_post = PRE == PRE_ANY ? p.post : PRE == PRE_POST;
  if (with_post) {
    double sum[1] = {0.0};
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      double s = x_at(c, 0) * x_at(c, 0);
#pragma unroll
      for (int i = 1; i < 8; ++i) s = __builtin_fma(x_at(c, i), x_at(c, i), s);
      sum[0] += s;
      // The conversions are made again below rather than kept.
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        int w = xv[c][u];
        asm volatile("" : "+v"(w));
        xv[c][u] = w;
      }
    }
    total(0, sum);
    post = rstd_of(p, sum[0]);
  }
  const double alpha = p.residual_scale;
  double sums[2] = {0.0, 0.0};  // of h, of h^2
  Eight<VF32> pw, ga;
  if constexpr (PRE != PRE_NONE) ga.load(vec.gate, first * 512 + 8 * lane);
  if constexpr (PRE == PRE_ANY || PRE == PRE_POST) pw.load(vec.post, first * 512 + 8 * lane);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int k = (first + c * step) * 512 + 8 * lane;
    double g[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = PRE == PRE_NONE ? 1.0 : ga.at(i);
    if (with_post) {
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= post * pw.at(i);
    }
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i)
      d[i] = round_f32(__builtin_fma(alpha, (double)h[c].at(i), x_at(c, i) * g[i]));
    if (c + 1 < NCH) {
      if constexpr (PRE != PRE_NONE) ga.load(vec.gate, k + step * 512);
      if constexpr (PRE == PRE_ANY || PRE == PRE_POST) pw.load(vec.post, k + step * 512);
    }
    if constexpr (RES == RES_F32) {
#pragma unroll
      for (int i = 0; i < 8; ++i) h[c].w[i] = __float_as_uint(d[i]);
    } else {
#pragma unroll
      for (int u = 0; u < 4; ++u) h[c].w[u] = pack_bf16(d[2 * u], d[2 * u + 1]);
    }
    if (p.residual_out != nullptr && k < p.K) {
      if constexpr (RES == RES_F32) {
        float* o = (float*)p.residual_out + row * p.ldo + k;
        *(i32x4*)o = i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
        *(i32x4*)(o + 4) = i32x4{(int)h[c].w[4], (int)h[c].w[5], (int)h[c].w[6], (int)h[c].w[7]};
      } else {
        *(i32x4*)((uint16_t*)p.residual_out + row * p.ldo + k) =
            i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
      }
    }
    double s = h[c].at(0), s2 = s * s;
#pragma unroll
    for (int i = 1; i < 8; ++i) {
      const double v = h[c].at(i);
      s += v;
      s2 = __builtin_fma(v, v, s2);
    }
    sums[0] += s;
    sums[1] += s2;
  }
  hold(h);
  total(1, sums);
  Statistics st = {0.0, 0.0};
  if (p.layer) {
    st.mean = uniform(sums[0] / (double)p.K);
    if constexpr (RES == RES_F32) {
      double sum[1] = {0.0};
#pragma unroll
      for (int c = 0; c < NCH; ++c) {
        double s = 0.0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const double v = (double)h[c].at(i) - st.mean;
          s = __builtin_fma(v, v, s);
        }
        sum[0] += in(c) ? s : 0.0;
      }
      hold(h);
      total(3, sum);
      sums[1] = sum[0];
    } else {
      const double var = __builtin_fma(-sums[0], st.mean, sums[1]);
      sums[1] = var < 0.0 ? 0.0 : var;  // NaN stays
    }
  }
  st.rstd = uniform(rstd_of(p, sums[1]));
  return st;
}

// The vectors of a chunk's y.
template <bool VF32, int MOD>
struct After {
  Eight<VF32> weight, scale, shift;
  __device__ __forceinline__ void load(const Vectors& v, int k) {
    weight.load(v.weight, k);
    if constexpr (MOD != MOD_NONE) {
      scale.load(v.scale, k);
      shift.load(v.shift, k);
    }
  }
};

// The bf16 y of a lane's 8 elements at k, as packed pairs (zeros past K).
template <int RES, bool VF32, int MOD>
__device__ __forceinline__ void make_y(const BlockNormArgs& p, const After<VF32, MOD>& a, int64_t row,
                                       const Held<RES>& h, int k, const Statistics& st, uint32_t (&out)[4]) {
  double g[8];
  if (p.weight != nullptr) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      g[i] = st.rstd * a.weight.at(i);
      if constexpr (MOD != MOD_NONE) g[i] *= 1.0 + a.scale.at(i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) g[i] = MOD == MOD_NONE ? st.rstd : __builtin_fma(st.rstd, a.scale.at(i), st.rstd);
  }
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    d[i] = round_f32(__builtin_fma((double)h.at(i) - st.mean, g[i], MOD == MOD_NONE ? -0.0 : a.shift.at(i)));
  }
  const bool in = k < p.K;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = in ? pack_bf16(d[2 * i], d[2 * i + 1]) : 0u;
  if (p.y != nullptr && in)
    *(i32x4*)((uint16_t*)p.y + row * p.ldy + k) = i32x4{(int)out[0], (int)out[1], (int)out[2], (int)out[3]};
}

// Many rows: a block takes 8, a wave each; the codes pass through LDS. Two blocks a
// CU.
template <int RES, bool VF32, int PRE, int MOD, bool FP4, int NCH>
__global__ __launch_bounds__(64 * kTileRows, 4) void block_norm_tile_kernel(BlockNormArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using St = Stage<FP4>;
  // The wave's number in a scalar register: its row and the resources follow.
  const int t = threadIdx.x, lane = t & 63, rl = __builtin_amdgcn_readfirstlane(t >> 6);
  const int S = St::slabs((int)p.K);
  uint8_t* sc_lds = smem + S * St::kCodes;
  const int64_t r0 = (int64_t)xcd_order(blockIdx.x, gridDim.x) * kTileRows;
  const int64_t row = r0 + rl;
  const bool real = row < p.M;
  Held<RES> h[NCH];
  Statistics stats = {0.0, 0.0};
  const Vectors vec = vectors_of<VF32>(p, real ? row : p.M - 1);
  if (real) {
    stats = make_h<RES, VF32, PRE, NCH>(p, vec, row, 0, 1, lane, h, [](int, auto& v) {
      for (double& s : v) s = wave_sum(s);
    });
  }
  After<VF32, MOD> after;
  after.load(vec, 8 * lane);
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4] = {0, 0, 0, 0};
    if (real) make_y(p, after, row, h[ch], k, stats, v);
    if (ch + 1 < NCH) after.load(vec, k + 512);
    __builtin_amdgcn_sched_barrier(0);
    if (p.q == nullptr) continue;
    if constexpr (FP4) {
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
  if (p.q == nullptr) return;
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

// Few rows. Blocks 0 .. M-1: one row each, WPR waves. Blocks M ..: pad rows of one
// slab.
template <int RES, bool VF32, bool FP4, int WPR, int NCH>
__global__ __launch_bounds__(64 * WPR) void block_norm_row_kernel(BlockNormArgs p) {
  __shared__ double part[4][WPR];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int S = Stage<FP4>::slabs((int)p.K);
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
  const Vectors vec = vectors_of<VF32>(p, row);
  Held<RES> h[NCH];
  const Statistics stats = make_h<RES, VF32, PRE_ANY, NCH>(p, vec, row, wave, WPR, lane, h, [&](int i, auto& v) {
    for (double& s : v) {
      s = wave_sum(s);
      if (lane == 0) part[i + (&s - v)][wave] = s;
    }
    __syncthreads();
    for (double& s : v) {
      s = 0.0;
#pragma unroll
      for (int w = 0; w < WPR; ++w) s += part[i + (&s - v)][w];
    }
  });
  After<VF32, MOD_ANY> after;
  after.load(vec, wave * 512 + 8 * lane);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = wave + c * WPR;
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4];
    make_y(p, after, row, h[c], k, stats, v);
    if (c + 1 < NCH) after.load(vec, k + WPR * 512);
    if (p.q == nullptr) continue;
    if constexpr (FP4) {
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

template <int RES, bool VF32, int PRE, int MOD, bool FP4, int NCH>
hipError_t launch_tile(const BlockNormArgs& p, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = block_norm_tile_kernel<RES, VF32, PRE, MOD, FP4, NCH>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Stage<FP4>::bytes(512 * NCH), configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.R / kTileRows)), dim3(64 * kTileRows), Stage<FP4>::bytes((int)p.K), st, p);
  return hipGetLastError();
}

template <int RES, bool VF32, bool FP4, int NCH>
hipError_t launch_tile(const BlockNormArgs& p, hipStream_t st) {
  const bool mod = p.scale != nullptr || p.shift != nullptr;
  if (p.post) return mod ? launch_tile<RES, VF32, PRE_POST, MOD_SOME, FP4, NCH>(p, st)
                         : launch_tile<RES, VF32, PRE_POST, MOD_NONE, FP4, NCH>(p, st);
  if (p.gate != nullptr) return mod ? launch_tile<RES, VF32, PRE_GATE, MOD_SOME, FP4, NCH>(p, st)
                                    : launch_tile<RES, VF32, PRE_GATE, MOD_NONE, FP4, NCH>(p, st);
  return mod ? launch_tile<RES, VF32, PRE_NONE, MOD_SOME, FP4, NCH>(p, st)
             : launch_tile<RES, VF32, PRE_NONE, MOD_NONE, FP4, NCH>(p, st);
}

template <int RES, bool VF32, bool FP4, int WPR, int NCH>
hipError_t launch_row(const BlockNormArgs& p, hipStream_t st) {
  const unsigned blocks = (unsigned)(p.M + (p.q != nullptr && p.R > p.M ? Stage<FP4>::slabs((int)p.K) : 0));
  hipLaunchKernelGGL((block_norm_row_kernel<RES, VF32, FP4, WPR, NCH>), dim3(blocks), dim3(64 * WPR), 0, st, p);
  return hipGetLastError();
}

// The tiled form writes whole lines of codes and shares no sums; the row form has
// more rows on their way. Measured, tiled and row form, in us, the layer norm with
// gate and modulation: K = 2048, 1024 rows 10.0 and 9.3, 2048 rows 11.0 and 14.5,
// 32768 rows 126 and 166 (f32 residual 161 and 193); K = 4096, 16384 rows 140 and
// 118, 32768 rows 238 and 242, 65536 rows 445 and 470; K = 5120, 16384 rows 163 and
// 159, 65536 rows 590 and 635. Longer rows and f32 residuals beyond 2048 do not
// leave enough registers (K = 8192, 65536 rows 1130 and 915; f32, K = 4096, 32768
// rows 379 and 350).
constexpr int64_t kTileMinRows = 32768;
constexpr int64_t kTileMinRowsShort = 2048;  // K <= 2048

template <int RES, bool VF32, bool FP4>
hipError_t dispatch(const BlockNormArgs& p, hipStream_t st) {
  const int ch = (int)((p.K + 511) / 512);
  if (ch <= 4 && p.M >= kTileMinRowsShort) return launch_tile<RES, VF32, FP4, 4>(p, st);
  if constexpr (RES == RES_BF16) {
    if (ch <= 8 && p.M >= kTileMinRows) return launch_tile<RES, VF32, FP4, 8>(p, st);
    if (ch <= 10 && p.M >= kTileMinRows) return launch_tile<RES, VF32, FP4, 10>(p, st);
  }
  if (ch <= 8) return launch_row<RES, VF32, FP4, 4, 2>(p, st);
  if (ch <= 12) return launch_row<RES, VF32, FP4, 4, 3>(p, st);
  if (ch <= 16) return launch_row<RES, VF32, FP4, 4, 4>(p, st);
  if (ch <= 24) return launch_row<RES, VF32, FP4, 8, 3>(p, st);
  if (ch <= 32) return launch_row<RES, VF32, FP4, 8, 4>(p, st);
  return launch_row<RES, VF32, FP4, 8, 16>(p, st);
}

template <int RES, bool VF32>
hipError_t dispatch(const BlockNormArgs& p, hipStream_t st) {
  return p.fp4 ? dispatch<RES, VF32, true>(p, st) : dispatch<RES, VF32, false>(p, st);
}

}  // namespace

hipError_t launch_block_norm_slab(const BlockNormArgs& a, hipStream_t stream) {
  if (a.residual_f32) return a.vectors_f32 ? dispatch<RES_F32, true>(a, stream) : dispatch<RES_F32, false>(a, stream);
  return a.vectors_f32 ? dispatch<RES_BF16, true>(a, stream) : dispatch<RES_BF16, false>(a, stream);
}

}  // namespace mx

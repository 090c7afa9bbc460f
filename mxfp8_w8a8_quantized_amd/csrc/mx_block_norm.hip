// The norms around a block, fused with its gate and the scaled residual, into the
// slab of the next quantized linear:
//
//   n = x, or x * post_weight / sqrt(mean(x^2) + eps)
//   h = residual_scale * residual + gate * n, rounded to the residual's type
//   y = bf16( norm(h) * weight * (1 + scale) + shift ), the norm
//       h / sqrt(mean(h^2) + eps), or (h - mean h) / sqrt(var h + eps)
//   q, s = the MX quantization of y (MXFP8 or MXFP4), where a slab is wanted
//
// One pass over memory, as in mx_norm.hip: a row stays in registers through up to
// three sums (of x^2, of h, of the squares), 7 bytes an element with a bf16
// residual. Sums and products are f64, for the reason given there; the vectors
// (weights, gate, scale, shift) come from the caches, once for each row.
#include "mx_internal.h"
#include "mx_norm_device.h"

namespace mx {
namespace {

struct Vectors {  // the vectors' rows for one row of x; null where there is none
  const void *post, *gate, *weight, *scale, *shift;
};

// Eight consecutive values of a vector.
__device__ __forceinline__ void vector8(const void* v, int k, int f32, float (&out)[8]) {
  if (f32) {
    const f32x4 a = *(const f32x4*)((const float*)v + k), b = *(const f32x4*)((const float*)v + k + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[i] = a[i];
      out[4 + i] = b[i];
    }
  } else {
    const i32x4 a = *(const i32x4*)((const uint16_t*)v + k);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out[2 * i] = bf16_lo((uint32_t)a[i]);
      out[2 * i + 1] = bf16_hi((uint32_t)a[i]);
    }
  }
}

__device__ __forceinline__ const void* vector_row(const void* v, int64_t row, int64_t ld, int f32) {
  return v == nullptr ? nullptr : (const uint8_t*)v + row * ld * (f32 ? 4 : 2);
}
__device__ __forceinline__ Vectors vectors_of(const BlockNormArgs& p, int64_t row) {
  Vectors v;
  v.post = p.post_weight;
  v.weight = p.weight;
  v.gate = vector_row(p.gate, row / p.gate_period, p.ldg, p.vectors_f32);
  v.scale = vector_row(p.scale, row / p.mod_period, p.ldm, p.vectors_f32);
  v.shift = vector_row(p.shift, row / p.mod_period, p.ldm, p.vectors_f32);
  return v;
}

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

// The wave's part of row `row`: chunks first, first + step, ... (NCH of them) of
// 512 elements, 8 per lane. Computes and stores h, and returns the row's mean (0
// for the RMS norm) and 1 / sqrt(...). total(i, v): the row's i-th sum.
template <int RES, int NCH, typename Total>
__device__ __forceinline__ void make_h(const BlockNormArgs& p, const Vectors& vec, int64_t row, int first, int step,
                                       int lane, Held<RES> (&h)[NCH], double& mean, double& rstd, Total&& total) {
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
  double post = 1.0;
  if (p.post) {
    double sum = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const double a = (double)bf16_lo((uint32_t)xv[c][u]), b = (double)bf16_hi((uint32_t)xv[c][u]);
        sum = __builtin_fma(a, a, sum);
        sum = __builtin_fma(b, b, sum);
      }
    post = rstd_of(p, total(0, sum));
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        int w = xv[c][u];
        asm volatile("" : "+v"(w));  // no f64 conversions kept from above
        xv[c][u] = w;
      }
  }
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int k = (first + c * step) * 512 + 8 * lane;
    if (k < p.K) {
      double d[8];
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        d[2 * u] = (double)bf16_lo((uint32_t)xv[c][u]);
        d[2 * u + 1] = (double)bf16_hi((uint32_t)xv[c][u]);
      }
      if (p.post) {
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= post;
        if (vec.post != nullptr) {
          float g[8];
          vector8(vec.post, k, p.vectors_f32, g);
#pragma unroll
          for (int i = 0; i < 8; ++i) d[i] *= (double)g[i];
        }
      }
      if (vec.gate != nullptr) {
        float g[8];
        vector8(vec.gate, k, p.vectors_f32, g);
#pragma unroll
        for (int i = 0; i < 8; ++i) d[i] *= (double)g[i];
      }
      float f[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = round_f32(__builtin_fma(p.residual_scale, (double)h[c].at(i), d[i]));
      if constexpr (RES == RES_F32) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[c].w[i] = __float_as_uint(f[i]);
      } else {
#pragma unroll
        for (int u = 0; u < 4; ++u) h[c].w[u] = pack_bf16(f[2 * u], f[2 * u + 1]);
      }
      if (p.residual_out != nullptr) {
        if constexpr (RES == RES_F32) {
          float* o = (float*)p.residual_out + row * p.ldo + k;
          *(i32x4*)o = i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
          *(i32x4*)(o + 4) = i32x4{(int)h[c].w[4], (int)h[c].w[5], (int)h[c].w[6], (int)h[c].w[7]};
        } else {
          *(i32x4*)((uint16_t*)p.residual_out + row * p.ldo + k) =
              i32x4{(int)h[c].w[0], (int)h[c].w[1], (int)h[c].w[2], (int)h[c].w[3]};
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const double v = (double)h[c].at(i);
      sum = p.layer ? sum + v : __builtin_fma(v, v, sum);
    }
  }
  mean = 0.0;
  sum = total(1, sum);
  if (p.layer) {
    mean = sum / (double)p.K;
    hold(h);
    double sq = 0.0;
#pragma unroll
    for (int c = 0; c < NCH; ++c) {
      if ((first + c * step) * 512 + 8 * lane >= p.K) continue;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = (double)h[c].at(i) - mean;
        sq = __builtin_fma(v, v, sq);
      }
    }
    sum = total(2, sq);
  }
  rstd = rstd_of(p, sum);
  hold(h);
}

// The bf16 y of a lane's 8 elements at k, as packed pairs (zeros past K).
template <int RES>
__device__ __forceinline__ void make_y(const BlockNormArgs& p, const Vectors& vec, int64_t row, const Held<RES>& h, int k,
                                       double mean, double rstd, uint32_t (&out)[4]) {
  out[0] = out[1] = out[2] = out[3] = 0;
  if (k >= p.K) return;
  double d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) d[i] = ((double)h.at(i) - mean) * rstd;
  float g[8];
  if (vec.weight != nullptr) {
    vector8(vec.weight, k, p.vectors_f32, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= (double)g[i];
  }
  if (vec.scale != nullptr) {
    vector8(vec.scale, k, p.vectors_f32, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] *= 1.0 + (double)g[i];
  }
  if (vec.shift != nullptr) {
    vector8(vec.shift, k, p.vectors_f32, g);
#pragma unroll
    for (int i = 0; i < 8; ++i) d[i] += (double)g[i];
  }
  float f[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = round_f32(d[i]);
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
  if (p.y != nullptr)
    *(i32x4*)((uint16_t*)p.y + row * p.ldy + k) = i32x4{(int)out[0], (int)out[1], (int)out[2], (int)out[3]};
}

// Many rows: a block takes 8, a wave each; the codes pass through LDS.
template <int RES, bool FP4, int NCH>
__global__ __launch_bounds__(64 * kTileRows, 2) void block_norm_tile_kernel(BlockNormArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using St = Stage<FP4>;
  const int t = threadIdx.x, lane = t & 63, rl = t >> 6;
  const int S = St::slabs((int)p.K);
  uint8_t* sc_lds = smem + S * St::kCodes;
  const int64_t r0 = (int64_t)xcd_order(blockIdx.x, gridDim.x) * kTileRows;
  const int64_t row = r0 + rl;
  const bool real = row < p.M;
  Held<RES> h[NCH];
  double mean = 0.0, rstd = 0.0;
  Vectors vec = {nullptr, nullptr, nullptr, nullptr, nullptr};
  if (real) {
    vec = vectors_of(p, row);
    make_h<RES, NCH>(p, vec, row, 0, 1, lane, h, mean, rstd, [](int, double v) { return wave_sum(v); });
  }
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4] = {0, 0, 0, 0};
    if (real) make_y(p, vec, row, h[ch], k, mean, rstd, v);
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
template <int RES, bool FP4, int WPR, int NCH>
__global__ __launch_bounds__(64 * WPR) void block_norm_row_kernel(BlockNormArgs p) {
  __shared__ double part[3][WPR];
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
  const Vectors vec = vectors_of(p, row);
  Held<RES> h[NCH];
  double mean, rstd;
  make_h<RES, NCH>(p, vec, row, wave, WPR, lane, h, mean, rstd, [&](int i, double v) {
    v = wave_sum(v);
    if (lane == 0) part[i][wave] = v;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < WPR; ++w) sum += part[i][w];
    return sum;
  });
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = wave + c * WPR;
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4];
    make_y(p, vec, row, h[c], k, mean, rstd, v);
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

template <int RES, bool FP4, int NCH>
hipError_t launch_tile(const BlockNormArgs& p, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = block_norm_tile_kernel<RES, FP4, NCH>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Stage<FP4>::bytes(512 * NCH), configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.R / kTileRows)), dim3(64 * kTileRows), Stage<FP4>::bytes((int)p.K), st, p);
  return hipGetLastError();
}

template <int RES, bool FP4, int WPR, int NCH>
hipError_t launch_row(const BlockNormArgs& p, hipStream_t st) {
  const unsigned blocks = (unsigned)(p.M + (p.q != nullptr && p.R > p.M ? Stage<FP4>::slabs((int)p.K) : 0));
  hipLaunchKernelGGL((block_norm_row_kernel<RES, FP4, WPR, NCH>), dim3(blocks), dim3(64 * WPR), 0, st, p);
  return hipGetLastError();
}

// Rows from which the tiled form is taken, as in mx_norm.hip.
constexpr int64_t kTileMinRows = 32768;
constexpr int64_t kTileMinRowsShort = 2048;  // K <= 2048

template <int RES, bool FP4>
hipError_t dispatch(const BlockNormArgs& p, hipStream_t st) {
  const int ch = (int)((p.K + 511) / 512);
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

hipError_t launch_block_norm_slab(const BlockNormArgs& a, hipStream_t stream) {
  if (a.residual_f32) return a.fp4 ? dispatch<RES_F32, true>(a, stream) : dispatch<RES_F32, false>(a, stream);
  return a.fp4 ? dispatch<RES_BF16, true>(a, stream) : dispatch<RES_BF16, false>(a, stream);
}

}  // namespace mx

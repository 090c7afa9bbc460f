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
// residual.
//
// Products are f32: a conversion to f64 costs as much as four f32 operations, and
// an element has up to nine of them (75348 x 5120 with gate, modulation and layer
// norm: 1146 us in f64). Eight squares are added in f32, those sums in f64, so a
// row's sum is off by at most 8 * 2^-24; a row whose squares leave f32's range is
// summed again in f64 (SLOW below). The mean is subtracted in two parts. y is then
// off by less than 2^-20 of its terms before it is rounded to 8 bits.
#include "mx_internal.h"
#include "mx_norm_device.h"

namespace mx {
namespace {

// A vector's row for one row of x: an empty resource where there is none, whose
// loads give zeros without touching memory; `rest` is then added (1 for factors), so
// that the code has no branches and one chunk's vectors are on their way while the
// chunk before is computed (gate, scale and shift of 75348 x 5120: 698 to RESULT us).
struct Vector {
  __amdgpu_buffer_rsrc_t r;
  float rest;
};
template <bool VF32>
__device__ __forceinline__ Vector vector_of(const BlockNormArgs& p, const void* v, int64_t row, int64_t ld, float rest) {
  constexpr int ES = VF32 ? 4 : 2;
  return {make_rsrc(v == nullptr ? nullptr : (const uint8_t*)v + row * ld * ES, v == nullptr ? 0u : (uint32_t)p.K * ES),
          v == nullptr ? rest : 0.f};
}
struct Vectors {
  Vector post, gate, weight, scale, shift;
};
template <bool VF32>
__device__ __forceinline__ Vectors vectors_of(const BlockNormArgs& p, int64_t row) {
  const int64_t g = row / p.gate_period, m = row / p.mod_period;
  return {vector_of<VF32>(p, p.post_weight, 0, 0, 1.f), vector_of<VF32>(p, p.gate, g, p.ldg, 1.f),
          vector_of<VF32>(p, p.weight, 0, 0, 1.f), vector_of<VF32>(p, p.scale, m, p.ldm, 0.f),
          vector_of<VF32>(p, p.shift, m, p.ldm, 0.f)};
}

// Eight consecutive values of a vector as loaded (past K zeros).
template <bool VF32>
struct Eight {
  i32x4 w[VF32 ? 2 : 1];
  __device__ __forceinline__ void load(const Vector& v, int k) {
    w[0] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(v.r, k * (VF32 ? 4 : 2), 0, 0));
    if constexpr (VF32) w[1] = __builtin_bit_cast(i32x4, __builtin_amdgcn_raw_buffer_load_b128(v.r, k * 4 + 16, 0, 0));
  }
  __device__ __forceinline__ float at(int i) const {
    if constexpr (VF32) return __uint_as_float((uint32_t)w[i >> 2][i & 3]);
    return (i & 1) ? bf16_hi((uint32_t)w[0][i >> 1]) : bf16_lo((uint32_t)w[0][i >> 1]);
  }
};

// The squares' f32 sums cannot be relied on: too large, or so small that squares
// vanished and eps does not hide it.
__device__ __forceinline__ bool out_of_range(const BlockNormArgs& p, double sum) {
  return !(sum < 1e38) || (sum < 1e-30 && p.eps * (double)p.K < 1e-20);
}
__device__ __forceinline__ double rstd_of(const BlockNormArgs& p, double sum) {
  return 1.0 / __builtin_sqrt(sum / (double)p.K + p.eps);
}

// Sums over a lane's elements value(c, i), chunk c < NCH with in(c), i < 8; SLOW in
// f64.
template <bool SLOW, bool SQUARES, int NCH, typename In, typename Value>
__device__ __forceinline__ double sum_of(In&& in, Value&& value) {
  double sum = 0.0;
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    if constexpr (SLOW) {
      double s = 0.0;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const double v = value(c, i);
        s = SQUARES ? __builtin_fma(v, v, s) : s + v;
      }
      sum += in(c) ? s : 0.0;
    } else {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = value(c, i);
        s = SQUARES ? __builtin_fmaf(v, v, s) : s + v;
      }
      sum += (double)(in(c) ? s : 0.f);
    }
  }
  return sum;
}

struct Statistics {
  float mean, mean_low, rstd;  // mean + mean_low: the mean (0 for the RMS norm)
};

// The wave's part of row `row`: chunks first, first + step, ... (NCH of them) of
// 512 elements, 8 per lane. Computes and stores h, and returns the row's
// statistics. total(i, v): the row's sum of its waves' i-th sums.
template <int RES, bool VF32, int NCH, typename Total>
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
  auto hold_x = [&]() {  // as hold() below, of x
#pragma unroll
    for (int c = 0; c < NCH; ++c)
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        int w = xv[c][u];
        asm volatile("" : "+v"(w));
        xv[c][u] = w;
      }
  };
  // Words of a second, rare pass over the same elements: values of their own to the
  // compiler, which would keep the first pass's conversions for it.
  auto again = [](uint32_t w) {
    uint32_t zero = 0;
    asm volatile("" : "+v"(zero));
    return w ^ zero;
  };
  auto h_again = [&](int c, int i) -> double {
    if constexpr (RES == RES_F32) return (double)__uint_as_float(again(h[c].w[i]));
    const uint32_t w = again(h[c].w[i >> 1]);
    return (double)((i & 1) ? bf16_hi(w) : bf16_lo(w));
  };
  // Elements past K are zeros, but not the mean away from it.
  auto all = [](int) { return true; };
  auto in = [&](int c) { return (first + c * step) * 512 + 8 * lane < p.K; };
  auto x_at = [&](int c, int i) { return (i & 1) ? bf16_hi((uint32_t)xv[c][i >> 1]) : bf16_lo((uint32_t)xv[c][i >> 1]); };
  float post = 1.f;
  if (p.post) {
    double sum = total(0, sum_of<false, true, NCH>(all, x_at));
    if (out_of_range(p, sum))
      sum = total(1, sum_of<true, true, NCH>(all, [&](int c, int i) -> double {
                    const uint32_t w = again((uint32_t)xv[c][i >> 1]);
                    return (double)((i & 1) ? bf16_hi(w) : bf16_lo(w));
                  }));
    hold_x();
    post = (float)rstd_of(p, sum);
  }
  Eight<VF32> pw, ga;
  pw.load(vec.post, first * 512 + 8 * lane);
  ga.load(vec.gate, first * 512 + 8 * lane);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int k = (first + c * step) * 512 + 8 * lane;
    float d[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      d[i] = x_at(c, i) * post * (pw.at(i) + vec.post.rest);
      d[i] *= ga.at(i) + vec.gate.rest;
      d[i] = __builtin_fmaf(p.residual_scale, h[c].at(i), d[i]);
    }
    if (c + 1 < NCH) {
      pw.load(vec.post, k + step * 512);
      ga.load(vec.gate, k + step * 512);
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
  }
  Statistics st = {0.f, 0.f, 0.f};
  double m = 0.0;
  if (p.layer) {
    auto at = [&](int c, int i) { return h[c].at(i); };
    hold(h);
    m = total(2, sum_of<false, false, NCH>(all, at));
    if (!(__builtin_fabs(m) < 1e38)) m = total(3, sum_of<true, false, NCH>(all, h_again));
    m /= (double)p.K;
    st.mean = (float)m;
    st.mean_low = (float)(m - (double)st.mean);
  }
  hold(h);
  double sum = total(4, sum_of<false, true, NCH>(in, [&](int c, int i) { return h[c].at(i) - st.mean - st.mean_low; }));
  if (out_of_range(p, sum))
    sum = total(5, sum_of<true, true, NCH>(in, [&](int c, int i) { return h_again(c, i) - m; }));
  hold(h);
  st.rstd = (float)rstd_of(p, sum);
  return st;
}

// The vectors of a chunk's y.
template <bool VF32>
struct After {
  Eight<VF32> weight, scale, shift;
  __device__ __forceinline__ void load(const Vectors& v, int k) {
    weight.load(v.weight, k);
    scale.load(v.scale, k);
    shift.load(v.shift, k);
  }
};

// The bf16 y of a lane's 8 elements at k, as packed pairs (zeros past K).
template <int RES, bool VF32>
__device__ __forceinline__ void make_y(const BlockNormArgs& p, const Vectors& vec, const After<VF32>& a, int64_t row,
                                       const Held<RES>& h, int k, const Statistics& st, uint32_t (&out)[4]) {
  float d[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    d[i] = (h.at(i) - st.mean - st.mean_low) * st.rstd * (a.weight.at(i) + vec.weight.rest);
    d[i] = __builtin_fmaf(d[i], a.scale.at(i), d[i]) + a.shift.at(i);
  }
  const bool in = k < p.K;
#pragma unroll
  for (int i = 0; i < 4; ++i) out[i] = in ? pack_bf16(d[2 * i], d[2 * i + 1]) : 0u;
  if (p.y != nullptr && in)
    *(i32x4*)((uint16_t*)p.y + row * p.ldy + k) = i32x4{(int)out[0], (int)out[1], (int)out[2], (int)out[3]};
}

// Two blocks of 8 waves a CU where a row's registers allow it.
constexpr int waves_wanted(int res, int nch) { return nch <= (res == RES_F32 ? 8 : 10) ? 4 : 2; }

// Many rows: a block takes 8, a wave each; the codes pass through LDS.
template <int RES, bool VF32, bool FP4, int NCH>
__global__ __launch_bounds__(64 * kTileRows, waves_wanted(RES, NCH)) void block_norm_tile_kernel(BlockNormArgs p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using St = Stage<FP4>;
  const int t = threadIdx.x, lane = t & 63, rl = t >> 6;
  const int S = St::slabs((int)p.K);
  uint8_t* sc_lds = smem + S * St::kCodes;
  const int64_t r0 = (int64_t)xcd_order(blockIdx.x, gridDim.x) * kTileRows;
  const int64_t row = r0 + rl;
  const bool real = row < p.M;
  Held<RES> h[NCH];
  Statistics stats = {0.f, 0.f, 0.f};
  const Vectors vec = vectors_of<VF32>(p, real ? row : p.M - 1);
  if (real) {
    stats = make_h<RES, VF32, NCH>(p, vec, row, 0, 1, lane, h, [](int, double v) { return wave_sum(v); });
  }
  After<VF32> after;
  after.load(vec, 8 * lane);
#pragma unroll
  for (int ch = 0; ch < NCH; ++ch) {
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4] = {0, 0, 0, 0};
    if (real) make_y(p, vec, after, row, h[ch], k, stats, v);
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
  __shared__ double part[6][WPR];
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
  const Statistics stats = make_h<RES, VF32, NCH>(p, vec, row, wave, WPR, lane, h, [&](int i, double v) {
    v = wave_sum(v);
    if (lane == 0) part[i][wave] = v;
    __syncthreads();
    double sum = 0.0;
#pragma unroll
    for (int w = 0; w < WPR; ++w) sum += part[i][w];
    return sum;
  });
  After<VF32> after;
  after.load(vec, wave * 512 + 8 * lane);
#pragma unroll
  for (int c = 0; c < NCH; ++c) {
    const int ch = wave + c * WPR;
    const int k = ch * 512 + 8 * lane;
    uint32_t v[4];
    make_y(p, vec, after, row, h[c], k, stats, v);
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

template <int RES, bool VF32, bool FP4, int NCH>
hipError_t launch_tile(const BlockNormArgs& p, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = block_norm_tile_kernel<RES, VF32, FP4, NCH>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Stage<FP4>::bytes(512 * NCH), configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.R / kTileRows)), dim3(64 * kTileRows), Stage<FP4>::bytes((int)p.K), st, p);
  return hipGetLastError();
}

template <int RES, bool VF32, bool FP4, int WPR, int NCH>
hipError_t launch_row(const BlockNormArgs& p, hipStream_t st) {
  const unsigned blocks = (unsigned)(p.M + (p.q != nullptr && p.R > p.M ? Stage<FP4>::slabs((int)p.K) : 0));
  hipLaunchKernelGGL((block_norm_row_kernel<RES, VF32, FP4, WPR, NCH>), dim3(blocks), dim3(64 * WPR), 0, st, p);
  return hipGetLastError();
}

// Rows from which the tiled form is taken, as in mx_norm.hip.
constexpr int64_t kTileMinRows = 32768;
constexpr int64_t kTileMinRowsShort = 2048;  // K <= 2048

template <int RES, bool VF32, bool FP4>
hipError_t dispatch(const BlockNormArgs& p, hipStream_t st) {
  const int ch = (int)((p.K + 511) / 512);
  if (p.M >= (ch <= 4 ? kTileMinRowsShort : kTileMinRows)) {
    if (ch <= 4) return launch_tile<RES, VF32, FP4, 4>(p, st);
    if (ch <= 8) return launch_tile<RES, VF32, FP4, 8>(p, st);
    if (ch <= 10) return launch_tile<RES, VF32, FP4, 10>(p, st);
    if constexpr (RES != RES_F32)  // an f32 row of 16 chunks does not fit the registers
      if (ch <= 16) return launch_tile<RES, VF32, FP4, 16>(p, st);
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

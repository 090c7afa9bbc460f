// Few-token linear on MXFP4 weights: y = bf16(epi(sum_k xhat what + bias))
// for one to a few hundred tokens, with MXFP4 or MXFP8 activations, either
// quantized already (slab operands) or bf16 rows quantized in the kernel.
//
// Bound by the weights' bytes (N K / 2, read once from HBM) for a few tokens,
// and by the token operand's re-reads from the L2 (once per weight tile) for
// hundreds. A workgroup of 8 waves, or 16 on long rows, takes 16 WB weight rows
// and 16 TB tokens; its waves split K among themselves and add their partial sums
// in LDS in wave order, so there is one launch, no workspace and no dependence on
// timing, and N / (16 WB) workgroups are enough to fill the GPU.
//
// v_mfma_scale_f32_16x16x128_f8f6f4, weights as the A operand (found on the
// device): lane l holds row l % 16; an E2M1 operand is 16 bytes, K 32 G .. + 31
// of the 128 with G = l / 16; an E4M3 operand is 32 bytes, K 16 G .. + 15 and
// 64 + 16 G .. + 15; the scale of lane l is that of K group G of row l % 16.
// Output: lane l holds D[4 (l / 16) + i][l % 16]. A 16-row block of an MXFP4
// slab is one 1 KB run in lane order, so operands go from memory straight to
// registers; nothing is shared between the waves but the final sums.
//
// Measured (operands not in the L2): 5120 x 5120 weights, 16 tokens 5.0 us (2.8
// TB/s of weights; launch and the first round trip are about half of it), 15360
// x 5120 8.5 us (4.9 TB/s).
#include <type_traits>

#include "mx_fp4_few_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

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

// The operands of one 128-K slab as loaded. Scales come as one dword per row
// (its four groups) or, from an MXFP8 slab, two bytes per row and 64-K slab, for
// up to 64 rows in one load; see the transpositions below.
template <int SRC, int WB, int TB>
struct Step {
  static constexpr int NX = SRC == SRC_FP4 ? 1 : SRC == SRC_FP8 ? 2 : 4;  // 16-byte loads per token fragment
  static constexpr int NSA = (WB + 3) / 4;
  static constexpr int NSB = SRC == SRC_FP4 ? (TB + 3) / 4 : SRC == SRC_FP8 ? (TB + 1) / 2 : 1;
  i32x4 a[WB];
  i32x4 b[TB][NX];
  int sa[NSA], sb[NSB];
};

// The same for an MXFP8 slab pair: lane 32 h + 16 f + r holds the two scales of
// row 16 f + r in slab h; returns, in lane 16 g + r, the scale of group g = 2 h
// + byte of row 16 f + r in byte f.
__device__ __forceinline__ int transpose_scales_fp8(int x, int lane) {
  const auto q = __builtin_amdgcn_permlane16_swap((uint32_t)x, (uint32_t)x, false, false);
  return (int)__builtin_amdgcn_perm(q[1], q[0], (lane & 16) ? 0x0C0C0501u : 0x0C0C0400u);
}

// Loads slab `sl`. Past the wave's range (sl >= s1) nothing is read: the
// buffer resources are empty and every value becomes zero, so the loop's loads
// stay in one straight run.
template <int SRC, int WB, int TB>
__device__ __forceinline__ void load_step(Step<SRC, WB, TB>& s, const FewParams& p, int sl, int s1, int n0, int m0,
                                          int lane) {
  const int r = lane & 15, G = lane >> 4;
  const bool on = sl < s1;
  // Tiles need not divide the padded rows.
  const uint32_t wr = (uint32_t)min((int64_t)16 * WB, p.RN - n0);
  const uint32_t xr = SRC == SRC_FP4 || SRC == SRC_FP8 ? (uint32_t)min((int64_t)16 * TB, p.RM - m0) : 0u;
  const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.wq + ((int64_t)sl * (p.RN / 16) + n0 / 16) * 1024, on ? wr * 64 : 0u);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.ws + ((int64_t)sl * p.RN + n0) * 4, on ? wr * 4 : 0u);
#pragma unroll
  for (int i = 0; i < WB; ++i) s.a[i] = __builtin_amdgcn_raw_buffer_load_b128(ra, lane * 16 + i * 1024, 0, 0);
#pragma unroll
  for (int i = 0; i < Step<SRC, WB, TB>::NSA; ++i)
    s.sa[i] = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, lane * 4 + i * 256, 0, 0);
  if constexpr (SRC == SRC_FP4) {
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.x + ((int64_t)sl * (p.RM / 16) + m0 / 16) * 1024, on ? xr * 64 : 0u);
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(p.xs + ((int64_t)sl * p.RM + m0) * 4, on ? xr * 4 : 0u);
#pragma unroll
    for (int j = 0; j < TB; ++j) s.b[j][0] = __builtin_amdgcn_raw_buffer_load_b128(rb, lane * 16 + j * 1024, 0, 0);
#pragma unroll
    for (int j = 0; j < Step<SRC, WB, TB>::NSB; ++j)
      s.sb[j] = (int)__builtin_amdgcn_raw_buffer_load_b32(rt, lane * 4 + j * 256, 0, 0);
  } else if constexpr (SRC == SRC_FP8) {
    // Two 64-K slabs of 64-byte rows; the second is past K where K % 128 = 64.
    // Scales: lanes 0 .. 31 the first slab's, 32 .. 63 the second's, two bytes
    // for each of 32 rows.
    const bool two = on && sl * 128 + 64 < p.K;
    const uint8_t* x0 = p.x + (2 * (int64_t)sl * p.RM + m0) * 64;
    const uint8_t* t0 = p.xs + (2 * (int64_t)sl * p.RM + m0) * 2;
    const uint32_t next = (uint32_t)p.RM * 2;  // bytes to the next slab's scales
    const __amdgpu_buffer_rsrc_t rb0 = make_rsrc(x0, on ? xr * 64 : 0u);
    const __amdgpu_buffer_rsrc_t rb1 = make_rsrc(x0 + p.RM * 64, two ? xr * 64 : 0u);
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(t0, two ? next + xr * 2 : on ? xr * 2 : 0u);
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      s.b[j][0] = __builtin_amdgcn_raw_buffer_load_b128(rb0, r * 64 + 16 * G + j * 1024, 0, 0);
      s.b[j][1] = __builtin_amdgcn_raw_buffer_load_b128(rb1, r * 64 + 16 * G + j * 1024, 0, 0);
    }
#pragma unroll
    for (int j = 0; j < Step<SRC, WB, TB>::NSB; ++j)
      s.sb[j] = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rt, (lane & 31) * 2 + j * 64 + (lane >> 5) * next, 0, 0);
  } else {
    // Rows past M repeat the last one; their outputs are not stored.
    const int kend = on ? p.K : 0;
#pragma unroll
    for (int j = 0; j < TB; ++j) {
      const uint16_t* x = (const uint16_t*)p.x + min(m0 + 16 * j + r, p.M - 1) * p.ldx;
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        // E2M1: 32 consecutive elements; E4M3: two runs of 16.
        const int k = sl * 128 + (SRC == SRC_BF16_FP4 ? 32 * G + 8 * u : 64 * (u >> 1) + 16 * G + 8 * (u & 1));
        s.b[j][u] = k < kend ? *(const i32x4*)(x + k) : i32x4{0, 0, 0, 0};
      }
    }
  }
}

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

template <int SRC, int WB, int TB>
__device__ __forceinline__ void mma_step(f32x4 (&acc)[WB][TB], const Step<SRC, WB, TB>& s, int lane) {
  using St = Step<SRC, WB, TB>;
  constexpr int FB = SRC == SRC_FP4 || SRC == SRC_BF16_FP4 ? 4 : 0;  // token format: E2M1 or E4M3
  int sa[St::NSA], sbt[St::NSB];
#pragma unroll
  for (int i = 0; i < St::NSA; ++i) sa[i] = transpose_scales(s.sa[i], lane);
  if constexpr (SRC == SRC_FP4) {
#pragma unroll
    for (int j = 0; j < St::NSB; ++j) sbt[j] = transpose_scales(s.sb[j], lane);
  } else if constexpr (SRC == SRC_FP8) {
#pragma unroll
    for (int j = 0; j < St::NSB; ++j) sbt[j] = transpose_scales_fp8(s.sb[j], lane);
  }
  static_for<0, TB>([&](auto J) {
    constexpr int j = decltype(J)::value;
    constexpr int PER = SRC == SRC_FP4 ? 4 : 2;                   // token fragments per scale register
    constexpr int opb = SRC == SRC_FP4 || SRC == SRC_FP8 ? j % PER : 0;
    i32x8 b = {0, 0, 0, 0, 0, 0, 0, 0};
    int sb;
    if constexpr (SRC == SRC_FP4) {
      b = i32x8{s.b[j][0][0], s.b[j][0][1], s.b[j][0][2], s.b[j][0][3], 0, 0, 0, 0};
      sb = sbt[j / PER];
    } else if constexpr (SRC == SRC_FP8) {
      b = i32x8{s.b[j][0][0], s.b[j][0][1], s.b[j][0][2], s.b[j][0][3],
                s.b[j][1][0], s.b[j][1][1], s.b[j][1][2], s.b[j][1][3]};
      sb = sbt[j / PER];
    } else {
      b = quantize_operand<SRC == SRC_BF16_FP8>(s.b[j], lane, sb);
    }
    static_for<0, WB>([&](auto I) {
      constexpr int i = decltype(I)::value;
      const i32x8 a = {s.a[i][0], s.a[i][1], s.a[i][2], s.a[i][3], 0, 0, 0, 0};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i][j], 4, FB, i % 4, sa[i / 4], opb, sb);
    });
  });
}

// NW waves, each with one slab in flight. The partial sums go through LDS in
// rounds of at most kRound fragments, so that they take at most kRound KB per
// wave of it.
constexpr int kRound = 8;

template <int SRC, int WB, int TB, int NW, int EPI>
__global__ __launch_bounds__(64 * NW) void fp4_few_kernel(FewParams p) {
  constexpr int NF = WB * TB, C = NF < kRound ? NF : kRound;
  __shared__ f32x4 sums[NW][C][64];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  // Token tile fastest within an XCD's range of workgroups, so that those
  // that share a weight tile share an L2.
  const uint32_t lid = xcd_order(blockIdx.x, gridDim.x);
  const int tn = (int)(lid / (uint32_t)p.tiles_m), tm = (int)(lid - (uint32_t)tn * (uint32_t)p.tiles_m);
  const int n0 = tn * 16 * WB, m0 = tm * 16 * TB;
  const int S = (int)fp4_slabs(p.K);
  const int s0 = wave * S / NW, s1 = (wave + 1) * S / NW;
  f32x4 acc[WB][TB];
#pragma unroll
  for (int i = 0; i < WB; ++i)
#pragma unroll
    for (int j = 0; j < TB; ++j) acc[i][j] = f32x4{0.f, 0.f, 0.f, 0.f};
  Step<SRC, WB, TB> st;
  load_step(st, p, s0, s1, n0, m0, lane);
  for (int s = s0; s < s1; ++s) {
    mma_step(acc, st, lane);
    load_step(st, p, s + 1, s1, n0, m0, lane);
  }
#pragma unroll
  for (int f0 = 0; f0 < NF; f0 += C) {
    if (f0 > 0) __syncthreads();
#pragma unroll
    for (int f = f0; f < f0 + C && f < NF; ++f) sums[wave][f - f0][lane] = acc[f / TB][f % TB];
    __syncthreads();
    for (int c = wave; c < C && f0 + c < NF; c += NW) {
      const int i = (f0 + c) / TB, j = f0 + c - i * TB;
      const int n = n0 + 16 * i + 4 * (lane >> 4), m = m0 + 16 * j + (lane & 15);
      f32x4 v = sums[0][c][lane];
#pragma unroll
      for (int w = 1; w < NW; ++w) {
        const f32x4 o = sums[w][c][lane];
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
}

template <int SRC, int WB, int TB, int NW>
hipError_t launch_few(FewParams& p, int epi, hipStream_t st) {
  p.tiles_m = (p.M + 16 * TB - 1) / (16 * TB);
  const unsigned blocks = (unsigned)(p.tiles_m * ((p.N + 16 * WB - 1) / (16 * WB)));
  if (epi == 1)
    hipLaunchKernelGGL((fp4_few_kernel<SRC, WB, TB, NW, 1>), dim3(blocks), dim3(64 * NW), 0, st, p);
  else
    hipLaunchKernelGGL((fp4_few_kernel<SRC, WB, TB, NW, 0>), dim3(blocks), dim3(64 * NW), 0, st, p);
  return hipGetLastError();
}

// Fragments (16 x 16 outputs) per workgroup for one token fragment: enough that
// about 256 workgroups or fewer cover the output (one per CU), 1, 2 or 4. Weights
// from HBM, K = 5120 (us on 1, 2 and 4 fragments): one token on an MXFP4 slab, N =
// 4096 5.8, 6.0, 7.1; 5120 6.6, 6.1, 7.2; 8192 7.0, 6.4, 7.5; 13824 11.6, 9.8, 9.4;
// 16 bf16 rows to MXFP4, which every workgroup rounds for itself, N = 4096 8.7, 9.8,
// 12.0; 5120 16.3, 9.9, 12.1; 13824 30.5, 19.3, 13.0. So two workgroups a CU do not
// pay, though one round of them leaves CUs idle (160 workgroups at N = 5120).
int fragments(int64_t M, int64_t N) {
  const int64_t total = ((M + 15) / 16) * (N / 16);
  int f = 1;
  while (f < 4 && f * 256 < total) f *= 2;
  return f;
}

// Tile shapes. A sweep over WB = 1 .. 8, TB = 1 .. 4 (N = 3584 .. 13824, K = 2048 ..
// 13824, 33 to 200 tokens) has the time go with the loads that a wave issues per
// slab, codes and scales alike, as long as a CU has one workgroup; each further
// round of 256 workgroups adds about 0.6 of the first. With MXFP8 activations
// (us; loads): 128 x 13824 x 5120 on 80 x 32 15.2 (12), 96 x 32 16.8 (13), 128 x 32
// 18.4 (15), 64 x 64 19.9 (15), 48 x 32 on 428 workgroups 18.6 (9). MXFP4: 128 x 5120
// x 5120 on 64 x 48 6.9 (9), 64 x 64 7.7 (10), 80 x 32 7.8 (10); 200 x 5120 x 5120 on
// 80 x 64 9.1 (12), 128 x 64 10.7 (15).
struct Choice {
  double cost;  // loads a wave and slab, with the rounds
  hipError_t (*launch)(FewParams&, int, hipStream_t);
};
template <int SRC, int WB, int TB>
void consider(Choice& c, uint32_t nf, uint32_t mf) {
  constexpr int loads = WB + (WB + 3) / 4 + (SRC == SRC_FP8 ? 2 * TB + (TB + 1) / 2 : TB + (TB + 3) / 4);
  const uint64_t groups = (uint64_t)((nf + WB - 1) / WB) * ((mf + TB - 1) / TB);
  const double cost = loads * (0.4 + 0.6 * (double)((groups + 255) / 256));
  if (cost < c.cost) c = {cost, &launch_few<SRC, WB, TB, 8>};
}
template <int SRC>
Choice choose(int64_t M, int64_t N) {
  const uint32_t nf = (uint32_t)(N / 16), mf = (uint32_t)((M + 15) / 16);
  Choice c{1e300, nullptr};
  consider<SRC, 1, 1>(c, nf, mf);
  consider<SRC, 2, 1>(c, nf, mf);
  consider<SRC, 3, 1>(c, nf, mf);
  consider<SRC, 4, 1>(c, nf, mf);
  if constexpr (SRC == SRC_FP8) consider<SRC, 5, 1>(c, nf, mf);
  consider<SRC, 2, 2>(c, nf, mf);
  consider<SRC, 3, 2>(c, nf, mf);
  consider<SRC, 4, 2>(c, nf, mf);
  consider<SRC, 5, 2>(c, nf, mf);
  consider<SRC, 7, 2>(c, nf, mf);
  consider<SRC, 4, 3>(c, nf, mf);
  consider<SRC, 4, 4>(c, nf, mf);
  consider<SRC, 5, 4>(c, nf, mf);
  consider<SRC, 6, 4>(c, nf, mf);
  // (MXFP4 outputs of these costs are faster on tiles.)
  if constexpr (SRC == SRC_FP8) consider<SRC, 8, 4>(c, nf, mf);
  return c;
}

// Waves: eight; long rows on the smallest tiles take 16 (16 x 14336 x 2048: 6.2
// against 7.6 us). Not measured: more than one slab in flight a wave, and 16 waves
// on the larger tiles. Splitting K over workgroups too, with a second kernel adding
// the parts, was slower at nearly every shape (at best a fifth faster): not kept.
constexpr int64_t kLongK = 8192;

// Up to 16 tokens: one token fragment. Slab operands and bf16 rows take the same
// tiles and waves, so that both add their sums in the same order. 16 waves on long
// rows: rounding keeps a wave longer than its loads on bf16 rows (1 x 13824 x 5120:
// 10.6 against 11.7 us, to E4M3 13.4 against 15.2); with two fragments of weights
// an MXFP8 slab is faster on eight by up to 5% (16 x 8192 x 8192: 8.0 against 8.4).
template <int SRC>
hipError_t dispatch16(FewParams& p, int epi, hipStream_t st) {
  const int f = fragments(p.M, p.N);
  if (f == 1) return p.K >= kLongK ? launch_few<SRC, 1, 1, 16>(p, epi, st) : launch_few<SRC, 1, 1, 8>(p, epi, st);
  if (f == 2) return p.K >= kLongK ? launch_few<SRC, 2, 1, 16>(p, epi, st) : launch_few<SRC, 2, 1, 8>(p, epi, st);
  return launch_few<SRC, 4, 1, 8>(p, epi, st);
}

template <int SRC>
hipError_t dispatch(FewParams& p, int epi, hipStream_t st) {
  if (p.M <= 16) return dispatch16<SRC>(p, epi, st);
  const Choice c = choose<SRC>(p.M, p.N);
  if (c.launch == &launch_few<SRC, 1, 1, 8> && p.K >= kLongK) return launch_few<SRC, 1, 1, 16>(p, epi, st);
  return c.launch(p, epi, st);
}

}  // namespace

double fp4_few_cost(int fp8, int64_t M, int64_t N) {
  return fp8 ? choose<SRC_FP8>(M, N).cost : choose<SRC_FP4>(M, N).cost;
}

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
  return fp8 ? dispatch<SRC_FP8>(p, epi, stream) : dispatch<SRC_FP4>(p, epi, stream);
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
  return fp8 ? dispatch16<SRC_BF16_FP8>(p, epi, stream) : dispatch16<SRC_BF16_FP4>(p, epi, stream);
}

}  // namespace mx

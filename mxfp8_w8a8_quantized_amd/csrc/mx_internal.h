// Internal launchers shared by the C ABI layer (mx_api.cpp) and the kernels.
// Arguments are already validated when these are called.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <atomic>

namespace mx {

// Elementwise MX quantization of `rows` rows of K elements (pitch ld
// elements). kind: 0 = bf16 input, 1 = f32 input.
hipError_t launch_quantize(int kind, const void* x, int64_t rows, int64_t K, int64_t ld,
                           uint8_t* q, uint8_t* s, hipStream_t stream);

// Rows of a slab-layout operand: `rows` rounded up to the 256-row tile.
inline int64_t slab_rows(int64_t rows) { return (rows + 255) / 256 * 256; }

// The same quantization written in the slab layout (codes [K/64][R][64],
// scales [K/64][R][2], R = slab_rows(rows); pad rows are zero). K % 64 == 0.
hipError_t launch_quantize_slab(int kind, const void* x, int64_t rows, int64_t K, int64_t ld,
                                uint8_t* q, uint8_t* s, hipStream_t stream);

// Row-major codes [rows][K] and scales [rows][K/32] to the slab layout.
hipError_t launch_slab_pack(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K,
                            uint8_t* qo, uint8_t* so, hipStream_t stream);

// The block-scaled GEMM. When xs == nullptr, x is bf16 [M][K] and is
// quantized in the prologue; otherwise x holds E4M3 codes [M][K] and xs the
// E8M0 scales [M][K/32]. epi: 0 none, 1 GELU-tanh.
hipError_t launch_linear(const void* x, const uint8_t* xs, int64_t M, int64_t K,
                         const uint8_t* wq, const uint8_t* ws, int64_t N,
                         const void* bias, int epi, void* y, hipStream_t stream);

// The block-scaled GEMM on operands in the slab layout (mx.h): codes
// [K/64][R][64], scales [K/64][R][2], R = rows rounded up to 256; K % 64 == 0.
hipError_t launch_linear_slab(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K,
                              const uint8_t* wq, const uint8_t* ws, int64_t N,
                              const void* bias, int epi, void* y, hipStream_t stream);

// The same GEMM on 256 (weights) x 128 (tokens) tiles: twice the tiles of
// launch_linear_slab for the same shape, the same result bit for bit.
hipError_t launch_linear_slab_m128(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K,
                                   const uint8_t* wq, const uint8_t* ws, int64_t N,
                                   const void* bias, int epi, void* y, hipStream_t stream);

// The slab GEMM writing, instead of y, the MX quantization of bf16 y in the
// slab layout with rows M and K' = N: hq [N/64][RM][64], hs [N/64][RM][2],
// RM = slab_rows(M). N % 64 == 0 and RM * N < 2^31.
hipError_t launch_linear_slab_requant(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K,
                                      const uint8_t* wq, const uint8_t* ws, int64_t N, const void* bias,
                                      int epi, uint8_t* hq, uint8_t* hs, hipStream_t stream);

// Split-K slab GEMM: each tile's K/64 half-steps in `splits` ranges, one
// workgroup per (tile, range) writing fp32 partial sums into `part`
// (splits * tiles * 65536 floats), then a reduction kernel summing the
// ranges in order and applying bias, epilogue and bf16 into y [M][N].
// 1 <= splits <= K/64.
hipError_t launch_linear_slab_splitk(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq,
                                     const uint8_t* ws, int64_t N, const void* bias, int epi, void* y, int splits,
                                     float* part, hipStream_t stream);

// Few-token slab GEMM (128-token x 64-weight-row tiles, see mx_small.hip):
// splits == 1 writes y directly; splits > 1 writes f32 partials [splits][M][N]
// into `part` and reduces them in range order. small_tiles gives the tile
// count. 1 <= splits <= K/64, N % 16 == 0.
int64_t small_tiles(int64_t M, int64_t N);

// Measurement probe (mx_probe.hip): `blocks` workgroups of 4 waves, each
// lane loading 128 bytes of A and B codes (word index modulo bytes / 4), then
// 16 * iters scaled 32x32x64 MFMAs; one float per thread to sink.
hipError_t launch_mfma_probe(const uint8_t* a, const uint8_t* b, int64_t bytes, int iters, int blocks, float* sink,
                             hipStream_t stream);

// A one-wave kernel that occupies `stream` for about `microseconds` (the
// tuner queues its timed runs behind it, so that they run back to back).
hipError_t launch_delay(int microseconds, hipStream_t stream);
hipError_t launch_linear_slab_small(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq,
                                    const uint8_t* ws, int64_t N, const void* bias, int epi, void* y, int splits,
                                    float* part, hipStream_t stream);

// Balanced slab GEMM: the full rounds of ncu tiles data-parallel, the last,
// partial round split over K (at most 8 ranges, at least 2 slabs each) with
// fp32 partials in `part`. balanced_plan gives the number of data-parallel
// tiles, the split count (1: no split) and the partial bytes needed.
int64_t balanced_plan(int64_t M, int64_t K, int64_t N, int ncu, int64_t* full, int* splits);
hipError_t launch_linear_slab_balanced(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq,
                                       const uint8_t* ws, int64_t N, const void* bias, int epi, void* y, int ncu,
                                       float* part, hipStream_t stream);

// Per-output-channel FP8: rows of x (bf16, kind 0, or f32, kind 1; pitch ld)
// to E4M3 codes in the slab layout q [K/64][R][64] and one f32 scale per row
// s [R] (R = slab_rows(rows); pad rows zero). K % 64 == 0.
hipError_t launch_pc_quantize_slab(int kind, const void* x, int64_t rows, int64_t K, int64_t ld, uint8_t* q, float* s,
                                   hipStream_t stream);

// The slab GEMM on per-channel operands: codes as for launch_linear_slab,
// scales f32 per token row (xs [RM]) and per weight row (ws [RN]);
// y = bf16(epi(xs[m] ws[n] acc + bias[n])).
hipError_t launch_pc_linear_slab(const uint8_t* xq, const float* xs, int64_t M, int64_t K, const uint8_t* wq,
                                 const float* ws, int64_t N, const void* bias, int epi, void* y, hipStream_t stream);

// Raises a kernel's limit of dynamic LDS to `bytes`. The attribute belongs to
// one device's copy of the kernel, so it is set at its first launch on each:
// bit d of `done`, which the caller keeps per kernel, for device d (< 64).
inline hipError_t allow_dynamic_lds(const void* kernel, int bytes, std::atomic<uint64_t>& done) {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) return e;
  const uint64_t bit = uint64_t(1) << (dev & 63);
  if (done.load(std::memory_order_acquire) & bit) return hipSuccess;
  e = hipFuncSetAttribute(kernel, hipFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == hipSuccess) done.fetch_or(bit, std::memory_order_release);
  return e;
}

// MXFP4 (mx_fp4_device.h has the slab layout). Rows of bf16 (kind 0) or f32
// (kind 1) to a slab; a slab to row-major bf16 (kind 0) or f32 (kind 1) y;
// row-major packed codes to a slab; a slab to the MXFP8 slab of the same
// values (K % 64 == 0). Pitches in elements, K % 32 == 0.
hipError_t launch_fp4_quantize_slab(int kind, const void* x, int64_t rows, int64_t K, int64_t ld, uint8_t* q,
                                    uint8_t* s, hipStream_t stream);
hipError_t launch_fp4_dequantize_slab(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, int kind, void* y,
                                      int64_t ld, hipStream_t stream);
hipError_t launch_fp4_slab_pack(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, uint8_t* qo, uint8_t* so,
                                hipStream_t stream);
hipError_t launch_fp4_slab_unpack(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, uint8_t* qo,
                                  uint8_t* so, hipStream_t stream);

// Few-token MXFP4-weight linear (mx_fp4_small.hip) on a token slab (fp8: an
// MXFP8 slab, else an MXFP4 one), or on bf16 rows (at most 16) quantized in
// the kernel.
hipError_t launch_fp4_linear_few(int fp8, const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K,
                                 const uint8_t* wq, const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                 hipStream_t stream);
hipError_t launch_fp4_linear_rows(int fp8, const void* x, int64_t M, int64_t K, int64_t ldx, const uint8_t* wq,
                                  const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                  hipStream_t stream);

// Loads that a wave of the few-token kernel issues per slab on an output of more
// than 16 tokens, in units of a round of 256 workgroups: what its time goes with.
double fp4_few_cost(int fp8, int64_t M, int64_t N);

// The tile shape that launch_fp4_linear_tiles should be given for an output.
void fp4_linear_tile(int fp8, int64_t M, int64_t N, int* weight_tile, int* token_tile, int* halve);

// MXFP4-weight linear on tiles of 256, 128 or (MXFP8 tokens) 192 weight rows x
// 128 tokens, or (MXFP4 tokens) 256 x 256; N % 16 == 0, tiles below 2^24. halve:
// the tiles past the last whole round of 256 in two halves (256 weight rows only).
hipError_t launch_fp4_linear_tiles(int fp8, int weight_tile, int token_tile, int halve, const uint8_t* xq,
                                   const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq, const uint8_t* ws,
                                   int64_t N, const void* bias, int epi, void* y, hipStream_t stream);

// MXFP4 weights and tokens on tiles of 128 x 128 (mx_fp4_mid.hip); the same
// limits, and M <= kMidMaxRows (32-bit offsets between slabs of scales).
constexpr int64_t kMidMaxRows = int64_t(1) << 29;
hipError_t launch_fp4_linear_mid(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq,
                                 const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                 hipStream_t stream);

// Residual add, RMS norm and quantization into a slab (mx_norm.hip). K up to
// kNormMaxK (a row stays in one block's registers); residual, residual_out,
// weight and y may be null.
constexpr int64_t kNormMaxK = 65536;
constexpr int64_t kNormMaxRows = int64_t(1) << 22;  // blocks x threads stay below 2^32
struct RmsNormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  int residual_f32;
  const void* weight;
  int weight_f32;
  double eps;
  int64_t M, K;
  void* residual_out;
  int64_t ldo;
  void* y;
  int64_t ldy;
  int fp4;
  uint8_t* q;
  uint8_t* s;
};
hipError_t launch_rmsnorm_slab(const RmsNormArgs& a, hipStream_t stream);

// The norms around a block with its gate and scaled residual (mx_block_norm.hip).
// K up to kNormMaxK; residual_out, y, q (with s) and the vectors may be null. The
// vectors (f32 or bf16, all the same): post_weight and weight [K]; gate a row for
// every gate_period rows of x, scale and shift one for every mod_period.
struct BlockNormArgs {
  const void* x;
  int64_t ldx;
  const void* residual;
  int64_t ldr;
  double eps, residual_scale;
  const void *post_weight, *gate, *weight, *scale, *shift;
  int64_t gate_period, ldg, mod_period, ldm;
  int64_t M, R, K;  // R = slab_rows(M)
  void* residual_out;
  int64_t ldo;
  void* y;
  int64_t ldy;
  uint8_t* q;
  uint8_t* s;
  int residual_f32, vectors_f32, post, layer, fp4;
};
hipError_t launch_block_norm_slab(const BlockNormArgs& a, hipStream_t stream);

// The experts' products on MXFP4 weights (mx_experts.hip): x bf16 [T][ldx], k
// pairs (ids, weights) a token, up slabs of 2 I rows and K = H, down slabs of H
// rows and K = I for each of E experts; y bf16 [T][H]. gate: 0 SiLU, 1 GELU-tanh.
constexpr int kExpertTile = 128;  // pairs of a tile
constexpr int kMaxExperts = 1024;
struct ExpertTile {
  int32_t expert, first, count, pad;  // sorted rows first .. first + count - 1
};
struct ExpertsArgs {
  const void* x;
  int64_t ldx;
  const int32_t* ids;
  const float* weights;
  int64_t T, k, E, H, I;
  const uint8_t* up_q;
  const uint8_t* up_s;
  const uint8_t* down_q;
  const uint8_t* down_s;
  int gate, fp4;
  void* y;
  void* workspace;
};
struct ExpertsWorkspace {  // offsets of its parts
  int64_t xq, xs, hq, hs, o, os, rows, pos, tiles, n_tiles, counts, bytes;
  uint32_t xpitch_q, xpitch_s, hpitch_q, hpitch_s, opitch_s;
  int64_t max_tiles, chunks;
};
// The most tiles that T k pairs of E experts can take.
inline int64_t experts_max_tiles(int64_t T, int64_t k, int64_t E) {
  return T * k / kExpertTile + (E < T * k ? E : T * k);
}
ExpertsWorkspace experts_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int fp4);
hipError_t launch_fp4_experts(const ExpertsArgs& a, hipStream_t stream);

// Routing to experts (mx_route.hip). logits f32 or bf16 [T][ld]; bias may be null;
// scores: 0 softmax, 1 sigmoid; E <= kMaxExperts, groups divides E, groups and k
// <= 64; ids and weights [T][k].
struct RouteArgs {
  const void* logits;
  int64_t T, ld;
  const float* bias;
  int32_t* ids;
  float* weights;
  double factor;
  int f32, scores, E, groups, top_groups, k, renorm;
  // Set by the launch: rows, and the bias, are read four values at a time.
  int vector, vector_bias;
};
hipError_t launch_route(const RouteArgs& a, hipStream_t stream);

// Bytes of the library-owned scratch array of mx_linear_noalloc (per GPU).
constexpr int64_t kScratchBytes = int64_t(64) << 20;

// Device address of that array on the current device (looked up on the
// first call per device, then cached).
hipError_t scratch_buffer(void** ptr);

}  // namespace mx

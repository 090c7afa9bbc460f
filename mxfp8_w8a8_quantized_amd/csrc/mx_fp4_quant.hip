// MXFP4 quantizers (bf16 activations, f32 or bf16 weights to E2M1 codes and
// E8M0 scales in the slab layout of mx_fp4_device.h), the way back to bf16 or
// f32, row-major packed codes into slabs, and the exact conversion of an MXFP4
// slab to an MXFP8 one.
//
// All are bound by memory. A block takes a tile of 16 rows x 512 K (four
// slabs): row-major data moves as whole 1 KB (bf16) row segments, 8 elements
// per lane with a DPP quad holding one group of 32; the tile's codes pass
// through LDS, so that each slab's part of them is one contiguous run of 1 KB
// (its scales 64 bytes). The 16 groups of a row segment start 272 bytes
// apart in LDS (4 banks past a multiple of 64), so a wave's 64 dword accesses
// hit 64 banks.
#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr int kThreads = 256;
constexpr int kRows = 16, kSlabsPerTile = 4, kTileK = 128 * kSlabsPerTile;
constexpr int kGroupLds = 16 * kRows + 16;
constexpr int64_t kMaxBlocks = int64_t(1) << 22;  // blocks loop past this

struct Tiles {
  int64_t count, per_row_block;  // tiles, and tiles along K
};
inline Tiles tiles_of(int64_t R, int64_t K) {
  Tiles t;
  t.per_row_block = (fp4_slabs(K) + kSlabsPerTile - 1) / kSlabsPerTile;
  t.count = R / kRows * t.per_row_block;
  return t;
}
inline unsigned blocks_of(int64_t tiles) { return (unsigned)(tiles < kMaxBlocks ? tiles : kMaxBlocks); }

template <bool F32>
__global__ __launch_bounds__(kThreads) void fp4_quantize_kernel(const void* __restrict__ x, int64_t rows, int64_t K,
                                                                int64_t ld, int64_t R, int64_t tiles, int64_t nkt,
                                                                uint8_t* __restrict__ q, uint8_t* __restrict__ s) {
  __shared__ __attribute__((aligned(16))) uint8_t lq[4 * kSlabsPerTile * kGroupLds];  // [slab, group][row][16]
  __shared__ __attribute__((aligned(4))) uint8_t ls[kSlabsPerTile * kRows * 4];       // [slab][row][group]
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int sg = lane >> 2;  // slab and group of the lane's elements within the tile
  const int64_t S = fp4_slabs(K);
  for (int64_t tile = xcd_order(blockIdx.x, gridDim.x); tile < tiles; tile += gridDim.x) {
    const int64_t rb = tile / nkt, s0 = (tile - rb * nkt) * kSlabsPerTile;
    const int64_t k = s0 * 128 + 8 * lane;
    uint32_t raw[4][F32 ? 8 : 4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t row = rb * kRows + wave + 4 * j;
      const bool in = k < K && row < rows;
      if constexpr (F32) {
        const float* p = (const float*)x + row * ld + k;
        const i32x4 a = in ? *(const i32x4*)p : i32x4{0, 0, 0, 0};
        const i32x4 b = in ? *(const i32x4*)(p + 4) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          raw[j][u] = (uint32_t)a[u];
          raw[j][4 + u] = (uint32_t)b[u];
        }
      } else {
        const i32x4 a = in ? *(const i32x4*)((const uint16_t*)x + row * ld + k) : i32x4{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 4; ++u) raw[j][u] = (uint32_t)a[u];
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      uint32_t sc, code;
      if constexpr (F32) {
        float f[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) f[u] = __uint_as_float(raw[j][u]);
        code = fp4_quantize8_f32(f, sc);
      } else {
        code = fp4_quantize8_bf16(raw[j], sc);
      }
      const int row = wave + 4 * j;
      *(uint32_t*)(lq + sg * kGroupLds + row * 16 + (lane & 3) * 4) = code;
      if ((lane & 3) == 0) ls[(sg >> 2) * (kRows * 4) + row * 4 + (sg & 3)] = (uint8_t)sc;
    }
    __syncthreads();
    const int64_t sl = s0 + wave;  // wave w stores slab s0 + w of the tile
    if (sl < S) {
      *(i32x4*)(q + (sl * (R / 16) + rb) * 1024 + lane * 16) =
          *(const i32x4*)(lq + (t >> 4) * kGroupLds + (lane & 15) * 16);
      if (lane < 16) *(uint32_t*)(s + (sl * R + rb * kRows) * 4 + lane * 4) = *(const uint32_t*)(ls + wave * 64 + lane * 4);
    }
    __syncthreads();
  }
}

// A slab's values, row-major: exact in f32 and bf16 wherever they are finite
// there (at most two significant bits; from 2^128 on they become infinities).
template <bool F32>
__global__ __launch_bounds__(kThreads) void fp4_dequantize_kernel(const uint8_t* __restrict__ q,
                                                                  const uint8_t* __restrict__ s, int64_t rows,
                                                                  int64_t K, int64_t R, int64_t tiles, int64_t nkt,
                                                                  void* __restrict__ y, int64_t ld) {
  __shared__ __attribute__((aligned(16))) uint8_t lq[4 * kSlabsPerTile * kGroupLds];
  __shared__ __attribute__((aligned(4))) uint8_t ls[kSlabsPerTile * kRows * 4];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int sg = lane >> 2;
  const int64_t S = fp4_slabs(K);
  for (int64_t tile = xcd_order(blockIdx.x, gridDim.x); tile < tiles; tile += gridDim.x) {
    const int64_t rb = tile / nkt, s0 = (tile - rb * nkt) * kSlabsPerTile;
    const int64_t sl = s0 + wave;
    if (sl < S) {
      *(i32x4*)(lq + (t >> 4) * kGroupLds + (lane & 15) * 16) =
          *(const i32x4*)(q + (sl * (R / 16) + rb) * 1024 + lane * 16);
      if (lane < 16) *(uint32_t*)(ls + wave * 64 + lane * 4) = *(const uint32_t*)(s + (sl * R + rb * kRows) * 4 + lane * 4);
    }
    __syncthreads();
    const int64_t k = s0 * 128 + 8 * lane;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int row = wave + 4 * j;
      const int64_t rg = rb * kRows + row;
      if (k < K && rg < rows) {
        const uint32_t c = *(const uint32_t*)(lq + sg * kGroupLds + row * 16 + (lane & 3) * 4);
        const uint32_t sc = ls[(sg >> 2) * (kRows * 4) + row * 4 + (sg & 3)];
        const float sv = sc == 0xFFu ? __uint_as_float(0x7FC00000u) : scale_value(sc);
        float v[8];
#pragma unroll
        for (int u = 0; u < 8; ++u) v[u] = fp4_value(c >> (4 * u)) * sv;
        if constexpr (F32) {
          float* p = (float*)y + rg * ld + k;
          *(f32x4*)p = f32x4{v[0], v[1], v[2], v[3]};
          *(f32x4*)(p + 4) = f32x4{v[4], v[5], v[6], v[7]};
        } else {
          i32x4 o;
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const bf16x2 p = {(__bf16)v[2 * u], (__bf16)v[2 * u + 1]};
            o[u] = __builtin_bit_cast(int, p);
          }
          *(i32x4*)((uint16_t*)y + rg * ld + k) = o;
        }
      }
    }
    __syncthreads();
  }
}

// Row-major packed codes [rows][K/2] and scales [rows][K/32] to the slab
// layout: one group (16 bytes and its scale) per thread, in slab order.
__global__ __launch_bounds__(kThreads) void fp4_pack_kernel(const uint8_t* __restrict__ q,
                                                            const uint8_t* __restrict__ s, int64_t rows, int64_t K,
                                                            int64_t R, uint8_t* __restrict__ qo,
                                                            uint8_t* __restrict__ so) {
  const int64_t groups = K / 32, total = fp4_slabs(K) * R * 4;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total; u += (int64_t)gridDim.x * kThreads) {
    const int64_t blk = u >> 6, sl = blk / (R / 16), rb = blk - sl * (R / 16);
    const int64_t row = rb * 16 + (u & 15), g = sl * 4 + ((u >> 4) & 3);
    const bool in = row < rows && g < groups;
    *(i32x4*)(qo + u * 16) = in ? *(const i32x4*)(q + row * (K / 2) + g * 16) : i32x4{0, 0, 0, 0};
    so[(sl * R + row) * 4 + ((u >> 4) & 3)] = in ? s[row * groups + g] : 0;
  }
}

// Four E2M1 codes in the low halves of x's bytes to four E4M3 codes: the
// magnitudes are looked up in eight bytes (every E2M1 value is an E4M3 one),
// the sign moves from bit 3 to bit 7.
__device__ inline uint32_t e2m1_to_e4m3(uint32_t x) {
  return __builtin_amdgcn_perm(0x4C484440u, 0x3C383000u, x & 0x07070707u) | ((x & 0x08080808u) << 4);
}

// MXFP4 slab to the MXFP8 slab of the same values (same scales; a NaN group
// gets MXFP8's NaN codes): one group per thread, a wave taking one 16-row
// block of a slab, which becomes 16 rows of two consecutive 64-K slabs.
__global__ __launch_bounds__(kThreads) void fp4_unpack_kernel(const uint8_t* __restrict__ q,
                                                              const uint8_t* __restrict__ s, int64_t K, int64_t R,
                                                              uint8_t* __restrict__ qo, uint8_t* __restrict__ so) {
  const int64_t total = fp4_slabs(K) * R * 4;
  for (int64_t u = (int64_t)blockIdx.x * kThreads + threadIdx.x; u < total; u += (int64_t)gridDim.x * kThreads) {
    const int64_t blk = u >> 6, sl = blk / (R / 16), rb = blk - sl * (R / 16);
    const int64_t row = rb * 16 + (u & 15);
    const int g = (int)(u >> 4) & 3;
    const int64_t o = 2 * sl + (g >> 1);  // 64-K slab of the group
    if (o * 64 >= K) continue;
    const i32x4 v = *(const i32x4*)(q + u * 16);
    const uint8_t sc = s[(sl * R + row) * 4 + g];
    i32x8 w;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t even = e2m1_to_e4m3((uint32_t)v[i]), odd = e2m1_to_e4m3((uint32_t)v[i] >> 4);
      w[2 * i] = (int)__builtin_amdgcn_perm(odd, even, 0x05010400u);
      w[2 * i + 1] = (int)__builtin_amdgcn_perm(odd, even, 0x07030602u);
    }
    if (sc == 0xFFu) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i] = 0x7F7F7F7F;
    }
    i32x4* d = (i32x4*)(qo + (o * R + row) * 64 + (g & 1) * 32);
    d[0] = i32x4{w[0], w[1], w[2], w[3]};
    d[1] = i32x4{w[4], w[5], w[6], w[7]};
    so[(o * R + row) * 2 + (g & 1)] = sc;
  }
}

unsigned group_blocks(int64_t R, int64_t K) {
  const int64_t b = (fp4_slabs(K) * R * 4 + kThreads - 1) / kThreads;
  return (unsigned)(b < kMaxBlocks ? b : kMaxBlocks);
}

}  // namespace

hipError_t launch_fp4_quantize_slab(int kind, const void* x, int64_t rows, int64_t K, int64_t ld, uint8_t* q,
                                    uint8_t* s, hipStream_t stream) {
  const int64_t R = slab_rows(rows);
  const Tiles t = tiles_of(R, K);
  if (kind == 1)
    hipLaunchKernelGGL(fp4_quantize_kernel<true>, dim3(blocks_of(t.count)), dim3(kThreads), 0, stream, x, rows, K, ld,
                       R, t.count, t.per_row_block, q, s);
  else
    hipLaunchKernelGGL(fp4_quantize_kernel<false>, dim3(blocks_of(t.count)), dim3(kThreads), 0, stream, x, rows, K, ld,
                       R, t.count, t.per_row_block, q, s);
  return hipGetLastError();
}

hipError_t launch_fp4_dequantize_slab(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, int kind, void* y,
                                      int64_t ld, hipStream_t stream) {
  const int64_t R = slab_rows(rows);
  const Tiles t = tiles_of((rows + kRows - 1) / kRows * kRows, K);
  if (kind == 1)
    hipLaunchKernelGGL(fp4_dequantize_kernel<true>, dim3(blocks_of(t.count)), dim3(kThreads), 0, stream, q, s, rows, K,
                       R, t.count, t.per_row_block, y, ld);
  else
    hipLaunchKernelGGL(fp4_dequantize_kernel<false>, dim3(blocks_of(t.count)), dim3(kThreads), 0, stream, q, s, rows, K,
                       R, t.count, t.per_row_block, y, ld);
  return hipGetLastError();
}

hipError_t launch_fp4_slab_pack(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, uint8_t* qo, uint8_t* so,
                                hipStream_t stream) {
  const int64_t R = slab_rows(rows);
  hipLaunchKernelGGL(fp4_pack_kernel, dim3(group_blocks(R, K)), dim3(kThreads), 0, stream, q, s, rows, K, R, qo, so);
  return hipGetLastError();
}

hipError_t launch_fp4_slab_unpack(const uint8_t* q, const uint8_t* s, int64_t rows, int64_t K, uint8_t* qo,
                                  uint8_t* so, hipStream_t stream) {
  const int64_t R = slab_rows(rows);
  hipLaunchKernelGGL(fp4_unpack_kernel, dim3(group_blocks(R, K)), dim3(kThreads), 0, stream, q, s, K, R, qo, so);
  return hipGetLastError();
}

}  // namespace mx

// The experts' products on large tiles: 256 weight rows x 128 pairs a workgroup, four
// waves of 128 x 64 (mx_experts.hip says what the products are, and has the tiles of
// 128 rows that read few pairs' weights faster).
//
// What bounds the 128-row tiles when an expert has many pairs is the path of the loads:
// about 25 cycles of a CU for each 1 KB that a wave asks for, so 17 KB for the 512
// cycles of MFMA of a 128 x 128 step. Here a step takes 24 KB (32 with MXFP8 tokens) for
// twice the MFMAs, both operands through LDS, on the pipeline of mx_fp4_gemm.hip: a
// ring of four regions, a quarter of a refill issued by each wave, fragments of step j
// + 1 read between the MFMAs of step j, one barrier a step crossed while MFMAs issued
// ahead of it run.
//
// The pairs' rows are gathered: 64 (MXFP4) or 128 bytes of a row and step, in LDS with
// 16-byte chunk c of row r at c ^ swizzle(r). Scales come for four steps at a time: the
// weights' as one slot a step, the rows' 16 bytes a row. In the up product a wave's
// first 64 weight rows are Wg's and the other 64 Wu's for the same columns of h, so
// that fragments 0 and 2, 1 and 3 hold both factors of an element, and 32 columns of h
// lie in one fragment.
//
// Measured, 8192 tokens, E = 32, k = 4, H = 5120, I = 2048 with MXFP4 tokens: up 431 us
// (3.2 PFLOP/s), down 309 (2.2). The up product without its stores takes 402 us, with
// weights that stay in the L2 as well 365, without any loads 243. Five or six regions,
// eight waves of 64 x 64, other groupings of the tiles, stores left in flight take the
// same time. MFMAs are busy 40% (up) and 25% (down) of the time at 2.0 to 2.3 GHz, where
// mx_fp4_gemm.hip keeps them busy 68% at 1.6, so they wait. What differs from it: loads
// gathered in pieces of 64 or 128 bytes where the dense product reads 1 KB runs, and an
// epilogue that no MFMA overlaps. 4001 tokens, E = 64, k = 8, H = 4096 with MXFP8 tokens: up 485 (2.2),
// down 310 (1.7).
#include "mx_experts_device.h"

namespace mx {
namespace {

constexpr int NT = 256;
constexpr int MT = kExpertTile;  // pairs per tile
constexpr int BN = 256;          // weight rows
constexpr int IA = 4, JB = 2;    // fragments of 32 x 32 per wave
constexpr int RING = 4;
constexpr int64_t kWorkgroups = 256;  // a multiple of the 8 XCDs
constexpr int SW_SLOT = 4 * BN;  // weight scales of a step
constexpr int SX_SLOT = 16 * MT; // rows' scales of four steps

template <bool X8>
struct Shape {
  static constexpr int ROW = X8 ? 128 : 64;             // bytes of a row's step
  static constexpr int XB = MT * ROW / 4096;            // row DMAs per wave and step
  static constexpr int CL = IA + XB;                    // and with the weights'
  static constexpr int R_X = 64 * BN;                   // rows within a region
  static constexpr int REGION = R_X + MT * ROW;
  static constexpr int SW = RING * REGION;              // eight steps of weight scales
  static constexpr int SX = SW + 8 * SW_SLOT;           // eight steps of the rows'
  static constexpr int LDS = SX + 2 * SX_SLOT;
  static constexpr int NM = 2 * IA * JB;                // MFMAs per wave and step
  static constexpr int NBH = X8 ? 2 * JB : JB;          // 16-byte row reads per MFMA set
  static constexpr int H = IA + NBH;
  static constexpr int NC = 2 * H;
  static constexpr int NR = NC + IA + JB;               // and the scale pairs
  static constexpr int PRE = X8 ? 3 : 4;                // MFMAs ahead of the barrier
  static constexpr int SETUP = X8 ? 11 : 6;             // set-up instructions behind each
  static constexpr int RS = (NM - PRE) * 10 / 13;       // MFMAs after it that carry reads
  static constexpr int DS = X8 ? (NM - PRE) * 9 / 13 : (NM - PRE) * 18 / 26 + 1;  // and loads
  __device__ static int swizzle(int r) { return X8 ? (r >> 1) & 7 : (r >> 2) & 3; }
  static_assert(LDS <= 163840, "LDS");
};

template <bool X8>
struct Source {
  const uint8_t *x, *xs, *w, *ws;
  uint32_t x_bytes, xs_bytes;
  uint32_t xo[Shape<X8>::XB], xso, wo[IA], wso;  // the lane's offsets
  int R, nsteps;
};

// Loads of a step: past the last one from empty resources, so that every step has the
// same number of them.
template <class Sh>
struct LoadRes {
  __amdgpu_buffer_rsrc_t w, x;
  uint8_t* reg;
};
template <bool X8>
__device__ __forceinline__ LoadRes<Shape<X8>> load_res(const Source<X8>& S, uint8_t* smem, int j, int rg) {
  using Sh = Shape<X8>;
  const bool on = j < S.nsteps;
  return {make_rsrc(S.w + (int64_t)j * S.R * 64, on ? (uint32_t)S.R * 64u : 0u),
          make_rsrc(S.x + (int64_t)j * Sh::ROW, on ? S.x_bytes - (uint32_t)(j * Sh::ROW) : 0u), smem + rg * Sh::REGION};
}
// Code piece D of a step: one KB, weights and rows in turn while there are both.
template <int D, bool X8>
__device__ __forceinline__ void load_piece(const LoadRes<Shape<X8>>& L, const Source<X8>& S, int wave) {
  using Sh = Shape<X8>;
  constexpr int XB = Sh::XB, both = IA < XB ? IA : XB;
  constexpr bool W = D < 2 * both ? D % 2 == 0 : IA > XB;
  constexpr int u = D < 2 * both ? D / 2 : D - both;
  if constexpr (W)
    dma(L.w, L.reg + (wave * IA + u) * 1024, S.wo[u]);
  else
    dma(L.x, L.reg + Sh::R_X + (wave * XB + u) * 1024, S.xo[u]);
}
// Scales of steps s .. s + 3 (s a multiple of 4): a wave takes the weights' of one step
// and half of the rows (waves 2 and 3 the same halves as 0 and 1).
struct ScaleRes {
  __amdgpu_buffer_rsrc_t w, x;
  uint8_t *wto, *xto;
};
template <bool X8>
__device__ __forceinline__ ScaleRes scale_res(const Source<X8>& S, uint8_t* smem, int s, int wave) {
  using Sh = Shape<X8>;
  const int st = s + wave;
  return {make_rsrc(S.ws + (int64_t)st * S.R * 4, st < S.nsteps ? (uint32_t)S.R * 4u : 0u),
          make_rsrc(S.xs + (int64_t)s * 4, s < S.nsteps ? S.xs_bytes - (uint32_t)s * 4u : 0u),
          smem + Sh::SW + (st & 7) * SW_SLOT, smem + Sh::SX + ((s >> 2) & 1) * SX_SLOT + (wave & 1) * 1024};
}

template <bool X8>
struct Frags {
  i32x4 a[IA][2];              // [fragment][MFMA of the step]
  i32x4 b[JB][2][X8 ? 2 : 1];  // and, of an E4M3 operand, its two halves
  int sa[IA], sb[JB];          // byte s: the scale for MFMA s
};
struct FragAddr {
  const uint8_t *a, *sa, *sb;
  const uint8_t *b[2][2];  // [MFMA of the step][half]
};
template <bool X8>
__device__ __forceinline__ FragAddr frag_addr(const uint8_t* smem, int j, int rg, int wn, int wm, int lane) {
  using Sh = Shape<X8>;
  const int r32 = lane & 31, hi = lane >> 5, sw = Sh::swizzle(r32);
  const uint8_t* reg = smem + rg * Sh::REGION;
  const uint8_t* row = reg + Sh::R_X + (wm * 32 * JB + r32) * Sh::ROW;
  FragAddr A;
  A.a = reg + wn * (2048 * IA) + (r32 >> 4) * 1024 + (r32 & 15) * 16 + 512 * hi;
  A.sa = smem + Sh::SW + (j & 7) * SW_SLOT + (wn * 32 * IA + r32) * 4 + 2 * hi;
  A.sb = smem + Sh::SX + ((j >> 2) & 1) * SX_SLOT + (wm * 32 * JB + r32) * 16 + (j & 3) * 4 + 2 * hi;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    A.b[s][0] = row + (((X8 ? 2 * s + hi : 2 * hi + s) ^ sw) << 4);
    A.b[s][1] = X8 ? row + (((4 + 2 * s + hi) ^ sw) << 4) : A.b[s][0];
  }
  return A;
}
// Read piece r: the fragments' 16-byte parts in the order the MFMAs take them, then
// the scales.
template <int R, bool X8>
__device__ __forceinline__ void read_piece(Frags<X8>& F, const FragAddr& A) {
  using Sh = Shape<X8>;
  if constexpr (R < Sh::NC) {
    constexpr int s = R / Sh::H, r = R % Sh::H;
    constexpr int both = Sh::NBH < IA ? Sh::NBH : IA;
    constexpr bool isA = r < 2 * both ? r % 2 == 0 : IA > Sh::NBH;
    constexpr int f = r < 2 * both ? r / 2 : r - both;
    if constexpr (isA)
      F.a[f][s] = *(const i32x4*)(A.a + f * 2048 + s * 256);
    else if constexpr (X8)
      F.b[f / 2][s][f % 2] = *(const i32x4*)(A.b[s][f % 2] + (f / 2) * 32 * Sh::ROW);
    else
      F.b[f][s][0] = *(const i32x4*)(A.b[s][0] + f * 32 * Sh::ROW);
  } else if constexpr (R < Sh::NC + IA) {
    F.sa[R - Sh::NC] = *(const uint16_t*)(A.sa + 32 * 4 * (R - Sh::NC));
  } else {
    F.sb[R - Sh::NC - IA] = *(const uint16_t*)(A.sb + 32 * 16 * (R - Sh::NC - IA));
  }
}

template <int B, int E, bool X8>
__device__ __forceinline__ void mma(f32x16 (&acc)[IA][JB], const Frags<X8>& F) {
  static_for<B, E>([&](auto T) {
    constexpr int s = decltype(T)::value / (IA * JB), u = decltype(T)::value % (IA * JB), i = u / JB, j = u % JB;
    const i32x8 a = {F.a[i][s][0], F.a[i][s][1], F.a[i][s][2], F.a[i][s][3], 0, 0, 0, 0};
    const i32x4& b0 = F.b[j][s][0];
    if constexpr (X8) {
      const i32x4& b1 = F.b[j][s][1];
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 4, 0, s, F.sa[i], s, F.sb[j]);
    } else {
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], 0, 0, 0, 0};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 4, 4, s, F.sa[i], s, F.sb[j]);
    }
  });
}

// Reads [r0, r1) and loads [d0, d1) issued with the I-th MFMA after the barrier; SC:
// two of scales first.
template <class Sh, bool SC, int I>
struct Slot {
  static constexpr int N = Sh::CL + (SC ? 2 : 0);
  static constexpr int r0 = I < Sh::RS ? Sh::NR * I / Sh::RS : Sh::NR, r1 = I < Sh::RS ? Sh::NR * (I + 1) / Sh::RS : Sh::NR;
  static constexpr int d0 = I < Sh::DS ? N * I / Sh::DS : N, d1 = I < Sh::DS ? N * (I + 1) / Sh::DS : N;
};

// Step j, V = j % 4 (and its ring region).
template <int V, bool X8>
__device__ __forceinline__ void step(f32x16 (&acc)[IA][JB], Frags<X8>& cur, Frags<X8>& nxt, const Source<X8>& S,
                                     uint8_t* smem, int j, int wave, int wn, int wm, int lane) {
  using Sh = Shape<X8>;
  constexpr int NM = Sh::NM, PRE = Sh::PRE;
  constexpr bool SC = V == 0;
  __builtin_amdgcn_sched_barrier(0);
  const FragAddr A = frag_addr<X8>(smem, j + 1, (V + 1) % RING, wn, wm, lane);
  const LoadRes<Sh> L = load_res<X8>(S, smem, j + RING, V);
  ScaleRes C;
  if constexpr (SC) C = scale_res<X8>(S, smem, j + RING, wave);
  mma<0, PRE>(acc, cur);
  static_for<0, PRE>([&](auto) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
    __builtin_amdgcn_sched_group_barrier(0x006, Sh::SETUP, 0);  // set-up VALU / SALU
  });
  __builtin_amdgcn_sched_barrier(0);
  // Younger loads than step j + 1's: the codes of RING - 2 steps (those of scales, left
  // out, only make the wait stricter). The lgkmcnt(0) keeps a wave's refill from
  // overtaking another wave's last reads of the region.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((RING - 2) * Sh::CL) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  static_for<0, NM - PRE>([&](auto I) {
    using SL = Slot<Sh, SC, decltype(I)::value>;
    static_for<SL::r0, SL::r1>([&](auto R) { read_piece<decltype(R)::value>(nxt, A); });
    static_for<SL::d0, SL::d1>([&](auto D) {
      constexpr int d = decltype(D)::value - (SC ? 2 : 0);
      if constexpr (d == -2)
        dma(C.w, C.wto, S.wso);
      else if constexpr (d == -1)
        dma(C.x, C.xto, S.xso);
      else
        load_piece<d, X8>(L, S, wave);
    });
  });
  mma<PRE, NM>(acc, cur);
  static_for<0, NM - PRE>([&](auto I) {
    using SL = Slot<Sh, SC, decltype(I)::value>;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (SL::r1 > SL::r0) __builtin_amdgcn_sched_group_barrier(0x100, SL::r1 - SL::r0, 0);
    if constexpr (SL::d1 > SL::d0) __builtin_amdgcn_sched_group_barrier(0x020, SL::d1 - SL::d0, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
}

// A workgroup's tile: its pairs, and its first column of h (up) or of o.
struct Where {
  ExpertTile pairs;
  int n0;
  bool any;
};

// Buffer stores past a resource's end are dropped: rows past the tile's count are past
// it, columns past the operand's are sent there.
constexpr uint32_t kDrop = 0x80000000u;

// The upper 32 lanes of a change places with the lower 32 of b.
__device__ __forceinline__ void swap32(uint32_t& a, uint32_t& b) {
  const auto s = __builtin_amdgcn_permlane32_swap(a, b, false, false);
  a = s[0];
  b = s[1];
}

// Codes of the tile's 128 columns of h, straight from the registers: lane r32 + 32 hi
// of a fragment holds columns 8 q + 4 hi .. + 3 (q = 0 .. 3) of row r32; two swaps leave
// it columns 16 hi .. + 15.
template <bool X8, int ACT>
__device__ __forceinline__ void store_h(const f32x16 (&acc)[IA][JB], const ProductParams& p, const Where& t, int wn, int wm,
                                        int lane) {
  const int r32 = lane & 31, hi = lane >> 5;
  const __amdgpu_buffer_rsrc_t rq =
      make_rsrc(p.hq + (int64_t)t.pairs.first * p.hpitch_q, (uint32_t)t.pairs.count * p.hpitch_q);
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(p.hs + (int64_t)t.pairs.first * p.hpitch_s, (uint32_t)t.pairs.count * p.hpitch_s);
  const int n = t.n0 + 64 * wn;
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const uint32_t m = (uint32_t)(wm * 32 * JB + 32 * j + r32);
    uint32_t scales = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      uint32_t v[8];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        float h[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) h[r] = activation<ACT>(acc[i][j][4 * q + r]) * acc[i + 2][j][4 * q + r];
        v[2 * q] = pack_bf16(h[0], h[1]);
        v[2 * q + 1] = pack_bf16(h[2], h[3]);
      }
      uint32_t b = bf16_amax_bits(v), b2 = b;
      swap32(b, b2);
      const uint32_t E = max(b, b2) >> 7;
      const bool real = n + 32 * i < p.I;  // columns past I: zero codes and scales
      const uint32_t sc = X8 ? scale_code_from_exponent(E) : fp4_scale_code(E);
      scales |= (real ? sc : 0u) << (8 * i);
      uint32_t c[4];
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        c[q] = X8 ? e4m3_encode4_bf16(v[2 * q], v[2 * q + 1], sc) : e2m1_encode4_bf16(v[2 * q], v[2 * q + 1], sc);
        c[q] = real ? c[q] : 0u;
      }
      swap32(c[0], c[2]);
      swap32(c[1], c[3]);
      const uint32_t col = (uint32_t)(n + 32 * i + 16 * hi);
      if constexpr (X8)
        __builtin_amdgcn_raw_buffer_store_b128(i32x4{(int)c[0], (int)c[2], (int)c[1], (int)c[3]}, rq, m * p.hpitch_q + col, 0, 0);
      else
        __builtin_amdgcn_raw_buffer_store_b64(i32x2{(int)(c[0] | (c[2] << 16)), (int)(c[1] | (c[3] << 16))}, rq,
                                              m * p.hpitch_q + col / 2, 0, 0);
    }
    __builtin_amdgcn_raw_buffer_store_b16((uint16_t)scales, rs, hi == 0 ? m * p.hpitch_s + (uint32_t)n / 32 : kDrop, 0, 0);
  }
}

// o of the tile's 256 columns (mx_experts_device.h has its form), likewise: a lane's
// columns 8 q + 4 hi .. + 3 become 8 hi .. + 7 and 16 + 8 hi .. + 7.
__device__ __forceinline__ void store_o(const f32x16 (&acc)[IA][JB], const ProductParams& p, const Where& t, int wn, int wm,
                                        int lane) {
  const int r32 = lane & 31, hi = lane >> 5;
  const __amdgpu_buffer_rsrc_t ro = make_rsrc(p.o + (int64_t)t.pairs.first * p.H, (uint32_t)(t.pairs.count * p.H * 2));
  const __amdgpu_buffer_rsrc_t rs =
      make_rsrc(p.os + (int64_t)t.pairs.first * p.opitch_s, (uint32_t)t.pairs.count * p.opitch_s);
  const int n = t.n0 + 32 * IA * wn;
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const uint32_t m = (uint32_t)(wm * 32 * JB + 32 * j + r32);
    uint32_t exponents = 0;
#pragma unroll
    for (int i = 0; i < IA; ++i) {
      const uint32_t e = o_exponent(acc[i][j]);
      exponents |= e << (8 * i);
      uint32_t c[8];
      o_pack(acc[i][j], e, c);
      const uint32_t at = n + 32 * i < p.H ? (m * (uint32_t)p.H + (uint32_t)(n + 32 * i + 8 * hi)) * 2 : kDrop;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        swap32(c[4 * u], c[4 * u + 2]);
        swap32(c[4 * u + 1], c[4 * u + 3]);
        __builtin_amdgcn_raw_buffer_store_b128(
            i32x4{(int)c[4 * u], (int)c[4 * u + 1], (int)c[4 * u + 2], (int)c[4 * u + 3]}, ro, at + 32 * u, 0, 0);
      }
    }
    const uint32_t g = (uint32_t)n / 32;
    __builtin_amdgcn_raw_buffer_store_b32(exponents, rs, hi == 0 && g < p.opitch_s ? m * p.opitch_s + g : kDrop, 0, 0);
  }
}

// Workgroups stay for several tiles (256 of them, a CU each), so that a tile's first
// loads are on their way while the output of the one before is written
// (the MXFP4 case above: up 446 to 441 us, down 331 to 315).
template <bool UP, bool X8, int ACT>
__global__ __launch_bounds__(NT, 1) void tile_kernel(ProductParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using Sh = Shape<X8>;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;

  // Tiles in groups of 4 along the pairs x all weight tiles; each XCD has a contiguous
  // range of them, its workgroups take them in turn. Their number is known on the
  // device only.
  const int tiles_m = *p.n_tiles;
  const uint32_t total = (uint32_t)tiles_m * (uint32_t)p.tiles_n, xcd = blockIdx.x & 7;
  const uint32_t first = xcd * (total >> 3) + min(xcd, total & 7), end = first + (total >> 3) + (xcd < (total & 7) ? 1 : 0);
  uint32_t lid = first + (blockIdx.x >> 3);
  auto next_tile = [&]() -> Where {
    if (lid >= end) return {{0, 0, 0, 0}, 0, false};
    constexpr int GM = 4;
    const int group = (int)lid / (GM * p.tiles_n), gm = min(tiles_m - group * GM, GM);
    const int in_group = (int)lid - group * GM * p.tiles_n;
    lid += gridDim.x >> 3;
    return {p.tiles[group * GM + in_group % gm], in_group / gm * (UP ? BN / 2 : BN), true};
  };
  // Rows of the operand that the lane's DMAs take (rows past the tile's count repeat
  // its last one), and the scales'.
  constexpr int LPR = Sh::ROW / 16;  // lanes per row
  struct Rows {
    uint32_t x[Sh::XB], s;
  };
  auto rows_of = [&](const Where& t) -> Rows {
    auto source = [&](int r) -> uint32_t {
      const int c = min(r, t.pairs.count - 1);
      return UP ? (uint32_t)p.rows[t.pairs.first + c] : (uint32_t)c;
    };
    Rows R;
#pragma unroll
    for (int i = 0; i < Sh::XB; ++i) R.x[i] = source((wave * Sh::XB + i) * (64 / LPR) + lane / LPR);
    R.s = source(64 * (wave & 1) + lane);
    return R;
  };
  Source<X8> S;
  S.nsteps = p.nsteps;
  S.R = p.R;
  auto start = [&](const Where& t, const Rows& R) {  // the ring's first loads, as the loop would have issued them
    S.w = p.wq + (int64_t)t.pairs.expert * p.nsteps * p.R * 64;
    S.ws = p.ws + (int64_t)t.pairs.expert * p.nsteps * p.R * 4;
    // Weight row of the tile's row r (rows past the slab's read zeros).
    auto weight_row = [&](int r) {
      return UP ? t.n0 + (r >> 7) * 64 + (r & 63) + ((r >> 6) & 1) * p.I : t.n0 + r;
    };
#pragma unroll
    for (int u = 0; u < IA; ++u) S.wo[u] = (uint32_t)(weight_row((wave * IA + u) * 16) / 16 * 1024 + lane * 16);
    S.wso = (uint32_t)weight_row(4 * lane) * 4u;
    if constexpr (UP) {
      S.x = p.x;
      S.xs = p.xs;
      S.x_bytes = p.x_bytes;
      S.xs_bytes = p.xs_bytes;
    } else {
      S.x = p.x + (int64_t)t.pairs.first * p.pitch_q;
      S.xs = p.xs + (int64_t)t.pairs.first * p.pitch_s;
      S.x_bytes = (uint32_t)t.pairs.count * p.pitch_q;
      S.xs_bytes = (uint32_t)t.pairs.count * p.pitch_s;
    }
#pragma unroll
    for (int i = 0; i < Sh::XB; ++i) {
      const int r = (wave * Sh::XB + i) * (64 / LPR) + lane / LPR;
      S.xo[i] = (UP ? R.x[i] / (uint32_t)p.k : R.x[i]) * p.pitch_q + (uint32_t)(((lane % LPR) ^ Sh::swizzle(r)) * 16);
    }
    S.xso = (UP ? R.s / (uint32_t)p.k : R.s) * p.pitch_s;
    const ScaleRes C = scale_res<X8>(S, smem, 0, wave);
    dma(C.w, C.wto, S.wso);
    dma(C.x, C.xto, S.xso);
    static_for<0, RING>([&](auto J) {
      constexpr int j = decltype(J)::value;
      const LoadRes<Sh> L = load_res<X8>(S, smem, j, j);
      static_for<0, Sh::CL>([&](auto D) { load_piece<decltype(D)::value, X8>(L, S, wave); });
    });
  };

  Where tile = next_tile();
  if (!tile.any) return;
  start(tile, rows_of(tile));
  Where next = next_tile();
  Rows next_rows = rows_of(next.any ? next : tile);
  while (true) {
    f32x16 acc[IA][JB];
#pragma unroll
    for (int i = 0; i < IA; ++i)
#pragma unroll
      for (int j = 0; j < JB; ++j) {
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;
        asm volatile("" : "+a"(acc[i][j]));  // written here, inside the first loads' latency
      }
    __builtin_amdgcn_sched_barrier(0);
    // (The rows' loads and the stores of the tile before are younger than these loads, and
    // waited for as well.)
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((RING - 1) * Sh::CL) : "memory");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    Frags<X8> F[2];
    const FragAddr A0 = frag_addr<X8>(smem, 0, 0, wn, wm, lane);
    static_for<0, Sh::NR>([&](auto R) { read_piece<decltype(R)::value>(F[0], A0); });
    int j = 0;
    for (; j + RING <= S.nsteps; j += RING)
      static_for<0, RING>([&](auto V) {
        constexpr int v = decltype(V)::value;
        step<v>(acc, F[v % 2], F[(v + 1) % 2], S, smem, j + v, wave, wn, wm, lane);
      });
    static_for<0, RING - 1>([&](auto V) {
      constexpr int v = decltype(V)::value;
      if (j + v < S.nsteps) step<v>(acc, F[v % 2], F[(v + 1) % 2], S, smem, j + v, wave, wn, wm, lane);
    });
    __builtin_amdgcn_sched_barrier(0);
    // The last MFMAs' results are read 20 wait states after them at the earliest; the
    // compiler counts the scheduling directives above among its own.
#pragma unroll
    for (int i = 0; i < IA; ++i) asm volatile("s_nop 15\n\ts_nop 7" : "+a"(acc[i][0]), "+a"(acc[i][1]));
    // Every wave's last loads have landed and its last reads are done.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
    const Where done = tile;
    const bool more = next.any;
    if (more) {
      tile = next;
      const Rows rows = next_rows;
      next = next_tile();
      next_rows = rows_of(next.any ? next : tile);
      start(tile, rows);
    }
    if constexpr (UP)
      store_h<X8, ACT>(acc, p, done, wn, wm, lane);
    else
      store_o(acc, p, done, wn, wm, lane);
    if (!more) break;
  }
}

template <bool UP, bool X8, int ACT>
hipError_t launch(ProductParams p, int64_t max_tiles, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = tile_kernel<UP, X8, ACT>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Shape<X8>::LDS, configured);
  if (e != hipSuccess) return e;
  p.tiles_n = UP ? (p.I + 127) / 128 : (p.H + BN - 1) / BN;
  const int64_t tiles = (max_tiles * p.tiles_n + 7) / 8 * 8;
  hipLaunchKernelGGL(kern, dim3((unsigned)(tiles < kWorkgroups ? tiles : kWorkgroups)), dim3(NT), Shape<X8>::LDS, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_tile(const ProductParams& p, bool up, bool fp8, int gate, int64_t max_tiles, hipStream_t stream) {
  if (!up) return fp8 ? launch<false, true, 0>(p, max_tiles, stream) : launch<false, false, 0>(p, max_tiles, stream);
  if (fp8) return gate == 1 ? launch<true, true, 1>(p, max_tiles, stream) : launch<true, true, 0>(p, max_tiles, stream);
  return gate == 1 ? launch<true, false, 1>(p, max_tiles, stream) : launch<true, false, 0>(p, max_tiles, stream);
}

}  // namespace mx

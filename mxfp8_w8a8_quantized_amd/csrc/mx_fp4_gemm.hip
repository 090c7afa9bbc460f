// Linear on MXFP4 weights for many tokens, on slab operands (mx_fp4_device.h;
// the tokens MXFP4, or MXFP8 in their own slab layout); 128 x 128 tiles of MXFP4
// tokens have a kernel of their own (mx_fp4_mid.hip):
//
//   y[m][n] = bf16_rne( epi( sum_k xhat[m][k] * what[n][k] + f32(bias[n]) ) )
//
// 64 IA weight rows x 64 JB tokens per workgroup, four waves of 32 IA x 32 JB
// (one per SIMD) on v_mfma_scale_f32_32x32x64_f8f6f4 with the weights as the A
// operand. K advances in steps of one 128-K slab: 16 KB of codes per 256 rows,
// the bytes of an MXFP8 step of 64 K, for two MFMAs per fragment pair of half
// an FP8 MFMA's duration each. So the balance between matrix core, LDS and
// loads is the one of the MXFP8 slab GEMM at twice the arithmetic, and the
// same pipeline feeds it: a ring of RING LDS regions, each wave issuing a
// quarter of the refill of step j + RING during step j; the fragments of step
// j + 1 read from LDS into a second register set between the MFMAs of step j;
// one barrier per step, crossed while MFMAs issued ahead of it still run.
//
// Operand layout of the MFMA (found on the device): lane l holds 16 bytes, 32
// consecutive elements of row l % 32, and the scale of those elements. Which
// 32 is free as long as both operands agree: MFMA s (0, 1) of a step gives lane
// half h the group 2 h + s, so that a lane's two scales are neighbouring bytes
// and one 16-bit LDS read fetches both (op_sel takes byte s).
//
// A 16-row block of a slab is [group][row][16 bytes]: copied to LDS as it is,
// the 16 lanes of a ds_read_b128 phase (16 rows of one group) read 256
// consecutive bytes, without bank conflicts.
//
// MXFP8 tokens (X8; 128-token tiles): a step's token operand is two 64-K slabs
// of 128 rows, again 16 KB, and an MFMA takes as long as an FP8 one, so a step
// has the shape of the MXFP8 GEMM's on 256 x 256 tiles. E4M3 operands are 32
// bytes per lane: of the MFMA's 64 K, lane half h holds 16 h .. + 15 and 32 +
// 16 h .. + 15, and its scale is that of K 32 h .. + 31. With the weights' choice
// of groups, MFMA s takes bytes 32 s + 16 h .. + 15 of the row in both slabs,
// and the lane's scale is byte s of slab h. The 64-byte rows lie in LDS with
// chunk c of row r at c ^ ((r >> 2) & 3), which spreads a phase's 16 rows over
// the banks.
//
// The accumulators start at the bias. Sums are fp32 in a fixed order.
#include <type_traits>

#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int NT = 256;
constexpr int kDropOffset = 1 << 30;  // beyond every resource: the store is dropped
constexpr int kStoreAux = 2;          // non-temporal

struct GemmParams {
  const uint8_t* x;
  const uint8_t* xs;
  const uint8_t* wq;
  const uint8_t* ws;
  const uint16_t* bias;  // f16 bits, or null
  uint16_t* y;
  int64_t RM, RN;
  int M, N, nsteps;
  int x_slabs;  // 64-K slabs of MXFP8 tokens (the last step may have one)
  int tiles_m, tiles_n;
  int whole;  // tiles of their full size, the first in order; the others are halved
};

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// A tile's shape and its step's schedule. LDS: RING regions (weight codes, then
// token codes), the scale ring [weights, tokens][8 steps][1 KB], a 256-byte bias
// slot per wave. RING is even, since scales are fetched for two steps at a time,
// and RING + 2 scale slots are in use.
constexpr int SR_SLOT = 1024;
constexpr int SR_OP = 8 * SR_SLOT;

template <int IA, int JB, bool X8>
struct Shape {
  static_assert(X8 ? JB == 2 : IA == 4, "MXFP8 tokens come in tiles of 128, MXFP4 ones with 256 weight rows");
  static constexpr int BN = 64 * IA;                      // weight rows per tile
  static constexpr int MT = 64 * JB;                      // tokens per tile
  static constexpr int XB = X8 ? 2 * JB : JB;             // 1 KB token blocks per wave and step
  static constexpr int CL = IA + XB;                      // code DMAs per wave and step
  static constexpr int R_X = IA * 4096;                   // token codes within a region
  static constexpr int REGION = CL * 4096;
  static constexpr int RING = 4;
  static constexpr int SR = RING * REGION;
  static constexpr int BIAS = SR + 2 * SR_OP;
  static constexpr int STAGE = 32 * JB * 256;             // epilogue staging per wave
  static constexpr int LDS = BIAS + 4 * 256 > 4 * STAGE ? BIAS + 4 * 256 : 4 * STAGE;
  static constexpr int NM = 2 * IA * JB;                  // MFMAs per wave and step
  static constexpr int NBH = X8 ? 2 * JB : JB;            // 16-byte token reads per MFMA set
  static constexpr int H = IA + NBH;                      // and with the weights'
  static constexpr int NC = 2 * H;                        // 16-byte reads per wave and step
  static constexpr int NR = NC + IA + JB;                 // and the scale pairs
  // MFMAs issued ahead of the step's barrier, about 190 cycles of them, and
  // set-up instructions behind each.
  static constexpr int PRE = X8 ? 3 : JB == 4 ? 8 : 4;
  static constexpr int SETUP = X8 ? 11 : 6;
  static constexpr int RS = (NM - PRE) * 10 / 13;         // MFMAs after it that carry reads
  static constexpr int DS = X8 ? (NM - PRE) * 9 / 13 : (NM - PRE) * 18 / 26 + 1;  // and loads
  static constexpr int ND = CL + 1;                       // loads: the scale DMA, then the codes
  static_assert(LDS <= 163840 && RING % 2 == 0 && RING + 2 <= 8 && RS > 0 && DS > 0, "shape");
};

struct Src {
  const uint8_t* w;  // tile origin in slab 0
  const uint8_t* x;
  const uint8_t* ws;
  const uint8_t* xs;
  uint64_t w_slab, x_slab;  // bytes between code slabs
  int nsteps, x_slabs;
  int xoff;          // lane part of a token DMA's offset
  uint32_t w_bytes;  // codes of a slab that belong to the tile (a last tile may reach past the operand)
};

struct LoadRes {
  __amdgpu_buffer_rsrc_t w, x;
  uint8_t* reg;
};

// Steps past the last (and the slab past K of MXFP8 tokens) load zeros from an
// empty resource. MXFP8: waves 0, 1 move the step's first token slab, waves 2, 3
// its second. rg: the step's ring region.
template <class Sh, bool X8>
__device__ __forceinline__ LoadRes load_res(const Src& S, uint8_t* smem, int j, int rg, int wave) {
  LoadRes L;
  L.reg = smem + rg * Sh::REGION;
  L.w = make_rsrc(S.w + (uint64_t)j * S.w_slab, j < S.nsteps ? S.w_bytes : 0u);
  if constexpr (X8) {
    const int sl = 2 * j + (wave >> 1);
    L.x = make_rsrc(S.x + (uint64_t)sl * S.x_slab, sl < S.x_slabs ? 8192u : 0u);
  } else {
    L.x = make_rsrc(S.x + (uint64_t)j * S.x_slab, j < S.nsteps ? 64u * Sh::MT : 0u);
  }
  return L;
}

// Code piece D of a step: one 1 KB block (16 rows), weights and tokens in turn
// while there are both.
template <int D, int IA, class Sh, bool X8>
__device__ __forceinline__ void load_piece(const LoadRes& L, const Src& S, int wave, int lane) {
  constexpr int XB = Sh::XB, both = IA < XB ? IA : XB;
  constexpr bool W = D < 2 * both ? D % 2 == 0 : IA > XB;
  constexpr int u = D < 2 * both ? D / 2 : D - both;
  const int q = wave * (W ? IA : XB) + u;
  const int from = (W || !X8 ? q : q & 7) * 1024;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(W ? L.w : L.x, (lds_ptr)(L.reg + (W ? 0 : Sh::R_X) + q * 1024), 16,
                                           W ? lane * 16 : S.xoff, from, 0, 0);
}

// Scales of steps s and s + 1 (s even): weights by waves 0, 1, tokens by waves
// 2, 3, each a 1 KB slot (lanes past the tile's rows read zeros). MXFP8: 256
// bytes of each slab (lanes 16 .. 31 the second's; 32 .. 63 the same again).
struct ScaleLoad {
  __amdgpu_buffer_rsrc_t r;
  uint8_t* dst;
  uint32_t voff;
};

template <class Sh, bool X8>
__device__ __forceinline__ ScaleLoad scale_res(const Src& S, uint8_t* smem, int s, int wave, int lane) {
  const bool w = wave < 2;
  const int st = s + (wave & 1);
  ScaleLoad L;
  L.dst = smem + Sh::SR + (w ? 0 : SR_OP) + (st & 7) * SR_SLOT;
  L.voff = lane * 16;
  if (X8 && !w) {
    const uint32_t slab = (uint32_t)(S.x_slab >> 5);
    const uint32_t n = 2 * st + 1 < S.x_slabs ? slab + 256u : 2 * st < S.x_slabs ? 256u : 0u;
    L.r = make_rsrc(S.xs + (uint64_t)(2 * st) * slab, n);
    L.voff = (lane & 15) * 16 + ((lane >> 4) & 1) * slab;
  } else {
    const uint64_t slab = (w ? S.w_slab : S.x_slab) >> 4;
    L.r = make_rsrc((w ? S.ws : S.xs) + (uint64_t)st * slab, st < S.nsteps ? (w ? S.w_bytes >> 4 : 4u * Sh::MT) : 0u);
  }
  return L;
}

__device__ __forceinline__ void issue_scales(const ScaleLoad& L) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.r, (lds_ptr)L.dst, 16, L.voff, 0, 0, 0);
}

template <int IA, int JB, bool X8>
struct Frags {
  i32x4 a[IA][2];              // [fragment][MFMA of the step]
  i32x4 b[JB][2][X8 ? 2 : 1];  // and, of an E4M3 operand, its two halves
  int sa[IA], sb[JB];          // byte s: the scale for MFMA s
};

struct FragAddr {
  const uint8_t* a;
  const uint8_t* b;   // E4M3: of MFMA 0
  const uint8_t* b1;  // E4M3: of MFMA 1
  const uint8_t* sa;
  const uint8_t* sb;
};

// Fragments of step j, in ring region rg.
template <int IA, int JB, bool X8>
__device__ __forceinline__ FragAddr frag_addr(const uint8_t* smem, int j, int rg, int wn, int wm, int lane) {
  using Sh = Shape<IA, JB, X8>;
  const int r32 = lane & 31, hi = lane >> 5;
  const uint8_t* reg = smem + rg * Sh::REGION;
  const uint8_t* sc = smem + Sh::SR + (j & 7) * SR_SLOT;
  const int off = (r32 >> 4) * 1024 + (r32 & 15) * 16 + 512 * hi;
  FragAddr A;
  A.a = reg + wn * (2048 * IA) + off;
  A.sa = sc + (wn * 32 * IA + r32) * 4 + 2 * hi;
  if constexpr (X8) {
    const uint8_t* row = reg + Sh::R_X + (wm * 32 * JB + r32) * 64;
    const int sw = (r32 >> 2) & 3;
    A.b = row + ((hi ^ sw) << 4);
    A.b1 = row + (((2 + hi) ^ sw) << 4);
    A.sb = sc + SR_OP + hi * 256 + (wm * 32 * JB + r32) * 2;
  } else {
    A.b = reg + Sh::R_X + wm * (2048 * JB) + off;
    A.b1 = A.b;
    A.sb = sc + SR_OP + (wm * 32 * JB + r32) * 4 + 2 * hi;
  }
  return A;
}

// Read piece r: the fragments' 16-byte parts in the order the MFMAs take
// them (all of MFMA 0, then all of MFMA 1; within one, parts of A and B in
// turn while there are both), then the scales.
template <int R, int IA, int JB, bool X8>
__device__ __forceinline__ void read_piece(Frags<IA, JB, X8>& F, const FragAddr& A) {
  using Sh = Shape<IA, JB, X8>;
  constexpr int NC = Sh::NC, H = Sh::H, NBH = Sh::NBH;
  if constexpr (R < NC) {
    constexpr int s = R / H, r = R % H;
    constexpr int both = NBH < IA ? NBH : IA;
    constexpr bool isA = r < 2 * both ? r % 2 == 0 : IA > NBH;
    constexpr int f = r < 2 * both ? r / 2 : r - both;
    if constexpr (isA) {
      F.a[f][s] = *(const i32x4*)(A.a + f * 2048 + s * 256);
    } else if constexpr (X8) {
      // f: fragment f / 2, slab f % 2.
      F.b[f / 2][s][f % 2] = *(const i32x4*)((s ? A.b1 : A.b) + (f % 2) * 8192 + (f / 2) * 2048);
    } else {
      F.b[f][s][0] = *(const i32x4*)(A.b + f * 2048 + s * 256);
    }
  } else if constexpr (R < NC + IA) {
    F.sa[R - NC] = *(const uint16_t*)(A.sa + 32 * 4 * (R - NC));
  } else {
    F.sb[R - NC - IA] = *(const uint16_t*)(A.sb + 32 * (X8 ? 2 : 4) * (R - NC - IA));
  }
}

template <int B, int E, int IA, int JB, bool X8>
__device__ __forceinline__ void mma(f32x16 (&acc)[IA][JB], const Frags<IA, JB, X8>& F) {
  static_for<B, E>([&](auto T) {
    constexpr int s = decltype(T)::value / (IA * JB), u = decltype(T)::value % (IA * JB), i = u / JB, j = u % JB;
    const i32x8 a = {F.a[i][s][0], F.a[i][s][1], F.a[i][s][2], F.a[i][s][3], 0, 0, 0, 0};
    if constexpr (X8) {
      const i32x4 &b0 = F.b[j][s][0], &b1 = F.b[j][s][1];
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 4, 0, s, F.sa[i], s, F.sb[j]);
    } else {
      const i32x4& b0 = F.b[j][s][0];
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], 0, 0, 0, 0};
      acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[i][j], 4, 4, s, F.sa[i], s, F.sb[j]);
    }
  });
}

// Reads [r0, r1) and loads [d0, d1) issued with the i-th MFMA after the barrier.
template <class Sh, int I>
struct Slot {
  static constexpr int r0 = I < Sh::RS ? Sh::NR * I / Sh::RS : Sh::NR, r1 = I < Sh::RS ? Sh::NR * (I + 1) / Sh::RS : Sh::NR;
  static constexpr int d0 = I < Sh::DS ? Sh::ND * I / Sh::DS : Sh::ND, d1 = I < Sh::DS ? Sh::ND * (I + 1) / Sh::DS : Sh::ND;
};

// Step j, in ring region rg: the first MFMAs, which read registers only, cover
// the wait for this wave's loads of step j + 1, the barrier and the address
// set-up; the rest run with the LDS reads of step j + 1 and the loads of step j
// + RING (into region rg) between them. EVEN: j is even, and the scales of steps
// j + RING and j + RING + 1 are fetched too.
template <bool EVEN, int IA, int JB, bool X8>
__device__ __forceinline__ void step(f32x16 (&acc)[IA][JB], Frags<IA, JB, X8>& cur, Frags<IA, JB, X8>& nxt,
                                     const Src& S, uint8_t* smem, int j, int rg, int wave, int wn, int wm, int lane) {
  using Sh = Shape<IA, JB, X8>;
  constexpr int NM = Sh::NM, PRE = Sh::PRE;
  __builtin_amdgcn_sched_barrier(0);
  const FragAddr A = frag_addr<IA, JB, X8>(smem, j + 1, rg + 1 == Sh::RING ? 0 : rg + 1, wn, wm, lane);
  const LoadRes L = load_res<Sh, X8>(S, smem, j + Sh::RING, rg, wave);
  ScaleLoad SL;
  if constexpr (EVEN) SL = scale_res<Sh, X8>(S, smem, j + Sh::RING, wave, lane);
  mma<0, PRE>(acc, cur);
  static_for<0, PRE>([&](auto) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);          // one MFMA
    __builtin_amdgcn_sched_group_barrier(0x006, Sh::SETUP, 0);  // set-up VALU / SALU
  });
  __builtin_amdgcn_sched_barrier(0);
  // The lgkmcnt(0) keeps a wave's refill from overtaking another wave's last
  // reads of the region. Younger loads: those of the RING - 2 steps after j + 1,
  // each with its codes, every other one with a scale DMA.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((Sh::RING - 2) * Sh::CL + (Sh::RING - 2) / 2) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  static_for<0, NM - PRE>([&](auto I) {
    using SL_ = Slot<Sh, decltype(I)::value>;
    static_for<SL_::r0, SL_::r1>([&](auto R) { read_piece<decltype(R)::value>(nxt, A); });
    static_for<SL_::d0, SL_::d1>([&](auto D) {
      constexpr int d = decltype(D)::value;
      if constexpr (d == 0) {
        if constexpr (EVEN) issue_scales(SL);
      } else {
        load_piece<d - 1, IA, Sh, X8>(L, S, wave, lane);
      }
    });
  });
  mma<PRE, NM>(acc, cur);
  static_for<0, NM - PRE>([&](auto I) {
    using SL_ = Slot<Sh, decltype(I)::value>;
    constexpr int nr = SL_::r1 - SL_::r0;
    constexpr int nd = SL_::d1 - SL_::d0 - (!EVEN && SL_::d0 == 0 && SL_::d1 > 0 ? 1 : 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (nr > 0) __builtin_amdgcn_sched_group_barrier(0x100, nr, 0);
    if constexpr (nd > 0) __builtin_amdgcn_sched_group_barrier(0x020, nd, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
}

// Tile `lid` in the order of work -> (token tile, weight tile): groups of 4 token
// tiles x all weight tiles (token tile fastest), of which each XCD walks a
// contiguous range, so that the tiles in flight on an XCD share panels in its L2.
__device__ inline void tile_coords(int lid, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 4;
  const int group = lid / (GM * tiles_n);
  const int gm = min(tiles_m - group * GM, GM);
  const int in_group = lid - group * GM * tiles_n;
  tm = group * GM + in_group % gm;
  tn = in_group / gm;
}

// The wave's 32 IA (n) x 32 JB (m) outputs: bf16 through LDS ([m][n], rows of
// 256 bytes, 8-byte block nb of row m at nb ^ (m & 31): 32 lanes on 32 rows
// write 32 bank pairs), then whole row pieces of 64 IA bytes, 16 bytes a lane.
template <int EPI, int IA, int JB>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[IA][JB], const GemmParams& p, uint8_t* ep, int m0,
                                           int n0, int rows_m, int rows_n, int wn, int wm, int lane) {
  const int r32 = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int i = 0; i < IA; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int nb = 8 * i + 2 * q + hi;
#pragma unroll
      for (int j = 0; j < JB; ++j) {
        const int m = 32 * j + r32;
        float v[4];
#pragma unroll
        for (int r = 0; r < 4; ++r) v[r] = epilogue<EPI>(acc[i][j][4 * q + r]);
        const bf16x2 p0 = {(__bf16)v[0], (__bf16)v[1]};
        const bf16x2 p1 = {(__bf16)v[2], (__bf16)v[3]};
        *(i32x2*)(ep + m * 256 + ((nb ^ (m & 31)) << 3)) =
            i32x2{__builtin_bit_cast(int, p0), __builtin_bit_cast(int, p1)};
      }
    }
  // The staging rows pass data between lanes: no read may move above another
  // lane's write (LDS order within a wave is kept by the hardware).
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.y + (size_t)m0 * p.N, (uint32_t)(rows_m * p.N * 2));
  constexpr int LPR = IA == 2 ? 8 : 16;  // lanes per row
  const int c = lane % LPR;
  const int nl = wn * 32 * IA + 8 * c;
  const bool n_ok = c < 4 * IA && nl < rows_n;
#pragma unroll 8
  for (int it = 0; it < 32 * JB * LPR / 64; ++it) {
    const int m = 64 / LPR * it + lane / LPR;
    const int sw = m & 31;
    const i32x4 v = *(const i32x4*)(ep + m * 256 + ((((2 * c) ^ sw) & ~1) << 3));
    const i32x4 w = (sw & 1) ? i32x4{v[2], v[3], v[0], v[1]} : v;
    const int off = n_ok ? ((wm * 32 * JB + m) * p.N + n0 + nl) * 2 : kDropOffset;
    __builtin_amdgcn_raw_buffer_store_b128(w, ry, off, 0, kStoreAux);
  }
}

// The tile whose first token is m0 and first weight row n0.
template <int EPI, int IA, int JB, bool X8>
__device__ __forceinline__ void compute_tile(const GemmParams& p, uint8_t* smem, int m0, int n0) {
  using Sh = Shape<IA, JB, X8>;
  const int rows_m = min(p.M - m0, Sh::MT);
  const int rows_n = min(p.N - n0, Sh::BN);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wn = wave & 1, wm = wave >> 1;

  Src S;
  S.w_slab = (uint64_t)p.RN * 64;
  S.x_slab = (uint64_t)p.RM * 64;
  S.w = p.wq + (size_t)n0 * 64;
  S.x = p.x + (size_t)m0 * 64;
  S.ws = p.ws + (size_t)n0 * 4;
  S.xs = p.xs + (size_t)m0 * (X8 ? 2 : 4);
  S.nsteps = p.nsteps;
  S.x_slabs = p.x_slabs;
  // 192-row tiles need not end where the padded rows do.
  S.w_bytes = (uint32_t)min(p.RN - n0, (int64_t)Sh::BN) * 64u;
  // MXFP8: lane L takes row L / 4 of a block, chunk (L % 4) ^ (L / 16), into slot L % 4.
  S.xoff = X8 ? (lane >> 2) * 64 + (((lane & 3) ^ (lane >> 4)) << 4) : lane * 16;

  // Bias: the f16 values of the wave's weight rows into its slot, ahead of the
  // ring's first loads (columns past N read what the load leaves there; their
  // outputs are not stored). The DMA moves dwords, from 4-byte aligned addresses;
  // n0 is even, so the tensor's own address says whether they are. Halves are
  // loaded one by one otherwise, which waits for them here.
  uint8_t* slot = smem + Sh::BIAS + wave * 256;
  if (p.bias != nullptr) {
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.bias + n0, (uint32_t)rows_n * 2u);
    if (((uintptr_t)p.bias & 2) == 0) {
      __builtin_amdgcn_raw_ptr_buffer_load_lds(rb, (lds_ptr)slot, 4, lane * 4, wn * 64 * IA, 0, 0);
    } else {
      const uint32_t lo = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, lane * 4, wn * 64 * IA, 0);
      const uint32_t hi = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rb, lane * 4 + 2, wn * 64 * IA, 0);
      *(uint32_t*)(slot + lane * 4) = lo | (hi << 16);
    }
  } else {
    *(int*)(slot + lane * 4) = 0;
  }
  // The ring's first loads in the order the loop would have issued them (its
  // waits count on it): the scales of two steps before the codes of the first.
  static_for<0, Sh::RING>([&](auto J) {
    constexpr int j = decltype(J)::value;
    if constexpr (j % 2 == 0) issue_scales(scale_res<Sh, X8>(S, smem, j, wave, lane));
    const LoadRes L = load_res<Sh, X8>(S, smem, j, j, wave);
    static_for<0, Sh::CL>([&](auto D) { load_piece<decltype(D)::value, IA, Sh, X8>(L, S, wave, lane); });
  });
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(Sh::RING * Sh::CL + Sh::RING / 2) : "memory");  // the bias
  f32x16 acc[IA][JB];
#pragma unroll
  for (int i = 0; i < IA; ++i)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const i32x2 bq = *(const i32x2*)(slot + (32 * i + 8 * q + 4 * (lane >> 5)) * 2);
#pragma unroll
      for (int r = 0; r < 4; ++r) {
        const uint32_t w = (uint32_t)bq[r >> 1];
        const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)((r & 1) ? (w >> 16) : (w & 0xFFFFu)));
#pragma unroll
        for (int j = 0; j < JB; ++j) acc[i][j][4 * q + r] = b;
      }
    }
  // The accumulators are written here, inside the first loads' latency.
#pragma unroll
  for (int i = 0; i < IA; ++i)
#pragma unroll
    for (int j = 0; j < JB; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
  // Step 0: RING - 1 steps' codes and RING / 2 - 1 scale DMAs are younger.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((Sh::RING - 1) * Sh::CL + Sh::RING / 2 - 1) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  Frags<IA, JB, X8> F0, F1;
  const FragAddr A0 = frag_addr<IA, JB, X8>(smem, 0, 0, wn, wm, lane);
  static_for<0, Sh::NR>([&](auto R) { read_piece<decltype(R)::value>(F0, A0); });
  int j = 0, rg = 0;
  for (; j + 1 < p.nsteps; j += 2) {
    step<true>(acc, F0, F1, S, smem, j, rg, wave, wn, wm, lane);
    step<false>(acc, F1, F0, S, smem, j + 1, rg + 1, wave, wn, wm, lane);
    rg = rg + 2 == Sh::RING ? 0 : rg + 2;
  }
  if (j < p.nsteps) step<true>(acc, F0, F1, S, smem, j, rg, wave, wn, wm, lane);
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  store_tile<EPI>(acc, p, smem + wave * Sh::STAGE, m0, n0, rows_m, rows_n, wn, wm, lane);
}

template <int EPI, int IA, int JB, bool X8>
__global__ __launch_bounds__(NT, 1) void fp4_gemm_kernel(GemmParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using Sh = Shape<IA, JB, X8>;
  int tm, tn;
  tile_coords((int)xcd_order(blockIdx.x, gridDim.x), p.tiles_m, p.tiles_n, tm, tn);
  compute_tile<EPI, IA, JB, X8>(p, smem, tm * Sh::MT, tn * Sh::BN);
}

// Whole rounds of tiles, then the last round's, at most half a round of them, in
// two halves each: along the tokens where there are 256 (MXFP4), else along the
// weights. 4001 x 5120 x 5120 with MXFP8 tokens (2.5 rounds) 94.7 to 87.6 us, 2900 x
// 5120 x 7168 on MXFP4 tiles of 256 x 256 (1.3 rounds) 67.7 to 59.0.
template <int EPI, int IA, int JB, bool X8>
__global__ __launch_bounds__(NT, 1) void fp4_gemm_halved_kernel(GemmParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using Sh = Shape<IA, JB, X8>;
  constexpr int IH = JB == 4 ? IA : IA / 2, JH = JB == 4 ? JB / 2 : JB;
  int tm, tn;
  if ((int)blockIdx.x < p.whole) {
    tile_coords((int)xcd_order(blockIdx.x, (uint32_t)p.whole), p.tiles_m, p.tiles_n, tm, tn);
    compute_tile<EPI, IA, JB, X8>(p, smem, tm * Sh::MT, tn * Sh::BN);
  } else {
    const int r = (int)xcd_order(blockIdx.x - (uint32_t)p.whole, gridDim.x - (uint32_t)p.whole);
    tile_coords(p.whole + (r >> 1), p.tiles_m, p.tiles_n, tm, tn);
    const int m0 = tm * Sh::MT + (JB == 4 ? (r & 1) * (Sh::MT / 2) : 0);
    const int n0 = tn * Sh::BN + (JB == 4 ? 0 : (r & 1) * (Sh::BN / 2));
    if (m0 < p.M && n0 < p.N) compute_tile<EPI, IH, JH, X8>(p, smem, m0, n0);
  }
}

template <int EPI, int IA, int JB, bool X8>
hipError_t launch(GemmParams p, bool halve, hipStream_t st) {
  using Sh = Shape<IA, JB, X8>;
  p.tiles_m = (p.M + Sh::MT - 1) / Sh::MT;
  p.tiles_n = (p.N + Sh::BN - 1) / Sh::BN;
  const int tiles = p.tiles_m * p.tiles_n;
  if constexpr (IA == 4 && (JB == 4 || X8)) {
    if (halve) {
      static std::atomic<uint64_t> halved_configured{0};  // per instantiation
      auto kern = fp4_gemm_halved_kernel<EPI, IA, JB, X8>;
      const hipError_t e = allow_dynamic_lds((const void*)kern, Sh::LDS, halved_configured);
      if (e != hipSuccess) return e;
      p.whole = tiles & ~255;
      hipLaunchKernelGGL(kern, dim3((unsigned)(2 * tiles - p.whole)), dim3(NT), Sh::LDS, st, p);
      return hipGetLastError();
    }
  }
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = fp4_gemm_kernel<EPI, IA, JB, X8>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Sh::LDS, configured);
  if (e != hipSuccess) return e;
  p.whole = tiles;
  hipLaunchKernelGGL(kern, dim3((unsigned)tiles), dim3(NT), Sh::LDS, st, p);
  return hipGetLastError();
}

template <int IA, int JB, bool X8>
hipError_t launch(const GemmParams& p, bool halve, int epi, hipStream_t st) {
  return epi == 1 ? launch<1, IA, JB, X8>(p, halve, st) : launch<0, IA, JB, X8>(p, halve, st);
}

}  // namespace

// The tile shape for an output: the one whose rounds of workgroups (256, one a
// CU) take the least time, from the measured time of a round at K = 5120 (us;
// longer or shorter K scale all shapes about alike). A last round of at most 128
// tiles behind whole ones is run in halves; MXFP4 tiles of 128 x 128 (mx_fp4_mid.hip)
// run two a CU: up to 512 a round, and less time up to 256. Over 130 to 24000
// tokens, 1024 to 16384 outputs and K = 1056 to 12256 the choice was the fastest, or
// within 4% of it, in nearly every shape (at worst 18% slower, at K < 2048). E.g.
// MXFP4 (us, chosen first): 512 x 5120 128 x 128 12.4, 256 x 128 17.4, 256 x 256 26.3;
// 1024 x 5120 256 x 128 18.8, 128 x 128 20.6, 256 x 256 26.9; 4001 x 5120 256 x 256
// halved 58.0, 128 x 128 58.8, 256 x 128 63.6; 3000 x 15360 256 x 256 114, 256 x 128
// 125, 128 x 128 129. MXFP8 tokens: 1792 x 5120 256 x 128 halved 47.5, 192 x 128 47.3,
// 128 x 128 52.9; 9000 x 5120 256 x 128 182, 192 x 128 194, 128 x 128 213. 192-row tiles
// gain only with MXFP8 tokens: 1024 x 5120 24.5 against 26.8 on 256 x 128 (MXFP4: 18.2
// to 20.5 against 19.2), and so do halves of 256 x 128 (4001 x 5120 MXFP4: 58.3).
// At one workgroup a CU a tile of 256 x 256 spends 1136 cycles a step, 1120 of
// them in its MFMAs, one of 256 x 128 660 (560); from a few hundred workgroups the
// clock falls to what power allows (2.4 to 1.4 GHz), so the shapes' times differ by
// less than their cycles.
void fp4_linear_tile(int fp8, int64_t M, int64_t N, int* weight_tile, int* token_tile, int* halve) {
  struct Tile {
    int weights, tokens;
    double us;       // a round
    double us_pair;  // two workgroups a CU, where they fit
    double us_half;  // a round of halved tiles
  };
  static const Tile fp4_tiles[] = {{256, 256, 32.0, 0.0, 19.5}, {256, 128, 19.5, 0.0, 0.0}, {128, 128, 11.6, 21.3, 0.0}};
  static const Tile fp8_tiles[] = {{256, 128, 28.0, 0.0, 17.1}, {192, 128, 24.6, 0.0, 0.0}, {128, 128, 17.1, 0.0, 0.0}};
  const Tile* t = fp8 ? fp8_tiles : fp4_tiles;
  const int shapes = !fp8 && M > kMidMaxRows ? 2 : 3;
  double best = -1.0;
  for (int i = 0; i < shapes; ++i) {
    const int64_t tiles = (M + t[i].tokens - 1) / t[i].tokens * ((N + t[i].weights - 1) / t[i].weights);
    const int64_t rest = tiles % 256;
    const bool half = t[i].us_half > 0.0 && tiles > 256 && rest > 0 && rest <= 128;
    double us;
    if (t[i].us_pair > 0.0)
      us = (double)(tiles / 512) * t[i].us_pair +
           (tiles % 512 == 0 ? 0.0 : tiles % 512 <= 256 ? t[i].us : t[i].us_pair);
    else if (half)
      us = (double)(tiles / 256) * t[i].us + t[i].us_half;
    else
      us = (double)((tiles + 255) / 256) * t[i].us;
    if (best < 0.0 || us < best) {
      best = us;
      *weight_tile = t[i].weights;
      *token_tile = t[i].tokens;
      *halve = half;
    }
  }
}

hipError_t launch_fp4_linear_tiles(int fp8, int weight_tile, int token_tile, int halve, const uint8_t* xq, const uint8_t* xs,
                                   int64_t M, int64_t K, const uint8_t* wq, const uint8_t* ws, int64_t N,
                                   const void* bias, int epi, void* y, hipStream_t stream) {
  if (!fp8 && weight_tile == 128)
    return launch_fp4_linear_mid(xq, xs, M, K, wq, ws, N, bias, epi, y, stream);
  GemmParams p;
  p.x = xq;
  p.xs = xs;
  p.wq = wq;
  p.ws = ws;
  p.bias = (const uint16_t*)bias;
  p.y = (uint16_t*)y;
  p.RM = slab_rows(M);
  p.RN = slab_rows(N);
  p.M = (int)M;
  p.N = (int)N;
  p.nsteps = (int)fp4_slabs(K);
  p.x_slabs = (int)(K / 64);
  p.tiles_m = p.tiles_n = p.whole = 0;
  if (fp8) {
    if (weight_tile == 128) return launch<2, 2, true>(p, false, epi, stream);
    if (weight_tile == 192) return launch<3, 2, true>(p, false, epi, stream);
    return launch<4, 2, true>(p, halve, epi, stream);
  }
  return token_tile == 256 ? launch<4, 4, false>(p, halve, epi, stream) : launch<4, 2, false>(p, false, epi, stream);
}

}  // namespace mx

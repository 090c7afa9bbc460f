// Linear on MXFP4 weights and MXFP4 tokens, slab operands, on tiles of 128 x 128:
// outputs too small to give every CU a tile of mx_fp4_gemm.hip's, or whose larger
// tiles would leave a last round of them half empty.
//
// Such a tile's step of 128 K has 8 MFMAs a wave, 287 cycles of them (measured,
// nothing else in the loop), so what bounds it is the issue of everything else by
// the one wave of each SIMD, and loads cost most: about 25 cycles each, whatever
// their size. On four waves of 64 x 64 with both operands in LDS, as in
// mx_fp4_gemm.hip, a step takes 485 cycles; here 400:
//   - The four waves split the weight rows only, 32 each, and load their
//     fragments from memory straight into registers (a 16-row block of a slab is
//     in fragment order); the tokens, which all four share, go through LDS: 8 KB
//     in and 32 KB out a step. Four loads a wave and step, each of 1 KB.
//   - The scales of four steps come in one load, into a ring in LDS (with a load
//     for each operand and step, a step takes 454 cycles).
//   - 80 KB of LDS and 215 registers let two workgroups share a CU: 512 tiles run
//     in 21.3 us at K = 5120, 256 in 11.6 (25.6 and 12.6 before; a round of
//     workgroups is bound by power as well, at 1.5 GHz with two a CU).
//
// v_mfma_scale_f32_32x32x64_f8f6f4, weights as the A operand: lane l holds 32
// consecutive elements of row l % 32 and their scale; MFMA s (0, 1) of a step
// gives lane half h the group 2 h + s. Weight registers form a ring of D steps;
// at step j the slot that step j - 1 used is refilled for step j + D - 1. Tokens
// form a ring of D LDS regions, refilled for step j + D; the token fragments of
// step j + 1 are read into a second register set between the MFMAs of step j;
// one barrier a step. The accumulators start at the bias and the sums are fp32 in
// the order of the other tiles: the results are the same bits.
#include <type_traits>

#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef __attribute__((address_space(3))) void* lds_ptr;

constexpr int NT = 256;
constexpr int MT = 128;               // tokens, and weight rows, per tile
constexpr int JB = 4;                 // and their fragments, which every wave takes
constexpr int kDropOffset = 1 << 30;  // beyond every resource: the store is dropped
constexpr int kStoreAux = 2;          // non-temporal

struct MidParams {
  const uint8_t* x;
  const uint8_t* xs;
  const uint8_t* wq;
  const uint8_t* ws;
  const uint16_t* bias;  // f16 bits, or null
  uint16_t* y;
  int64_t RM, RN;
  int M, N, nsteps;
  int tiles_m, tiles_n;
};

template <int B, int E, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  if constexpr (B < E) {
    f(std::integral_constant<int, B>{});
    static_for<B + 1, E>(f);
  }
}

// LDS: D regions of token codes, then rings of scales, 16 steps of the tile's
// weight rows' and 16 of its tokens'.
constexpr int D = 8;
constexpr int REGION = 64 * MT;
constexpr int RING = 2 * D;  // steps of scales

constexpr int SC_SLOT = 4 * MT;              // scales of a step, of either operand
constexpr int WS = D * REGION, XS = WS + RING * SC_SLOT;
constexpr int LDS = XS + RING * SC_SLOT;
constexpr int NM = 2 * JB;      // MFMAs per wave and step
constexpr int NL = 4;           // loads per wave and step: two of token codes, two of weight codes
constexpr int NR = 1 + 3 * JB;  // LDS reads: scales, codes
constexpr int PRE = 2;          // MFMAs ahead of the barrier
constexpr int SPAN = NM - PRE - 1;  // MFMAs after it that carry reads and loads
constexpr int PITCH = 64;       // epilogue staging: bytes per token row of a wave
constexpr int STAGE = MT * PITCH;
static_assert(4 * STAGE <= LDS && 2 * LDS <= 163840, "two workgroups a CU");

// Loads per wave of the steps from .. to - 1, relative to a multiple of D
// (negative: earlier); every fourth step has one of scales.
constexpr int loads(int from, int to) {
  int n = 0;
  for (int j = from; j < to; ++j) n += NL + ((j & 3) == 0);
  return n;
}
static_assert(loads(-6, 2) <= 63, "vmcnt holds six bits");

struct Src {
  const uint8_t* w;  // the wave's rows in slab 0
  const uint8_t* x;  // the tile's tokens in slab 0
  const uint8_t* ws;  // the tile's rows
  const uint8_t* xs;
  uint64_t w_slab, x_slab;  // bytes between code slabs
  int nsteps;
};

struct Weights {  // one step
  i32x4 a[2];
};

// Loads of step j: past the last, zeros from an empty resource.
__device__ __forceinline__ __amdgpu_buffer_rsrc_t weight_res(const Src& S, int j) {
  return make_rsrc(S.w + (uint64_t)j * S.w_slab, j < S.nsteps ? 2048u : 0u);
}
template <int P>
__device__ __forceinline__ void load_weights(Weights& W, __amdgpu_buffer_rsrc_t r, int frag_off) {
  W.a[P] = __builtin_amdgcn_raw_buffer_load_b128(r, frag_off, P * 256, 0);
}

struct TokenRes {
  __amdgpu_buffer_rsrc_t r;
  uint8_t* reg;
};
__device__ __forceinline__ TokenRes token_res(const Src& S, uint8_t* smem, int j, int rg) {
  return {make_rsrc(S.x + (uint64_t)j * S.x_slab, j < S.nsteps ? (uint32_t)REGION : 0u), smem + rg * REGION};
}
template <int P>
__device__ __forceinline__ void load_tokens(const TokenRes& L, int wave, int lane) {
  const int b = (2 * wave + P) * 1024;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.r, (lds_ptr)(L.reg + b), 16, lane * 16, b, 0, 0);
}

// The scales of steps s .. s + 3, to ring slots sl .. sl + 3: each wave two steps
// (lanes 0 .. 31 the first), waves 0, 1 the weights', waves 2, 3 the tokens'.
struct ScaleLoad {
  __amdgpu_buffer_rsrc_t r;
  uint8_t* dst;
  uint32_t voff;
};
__device__ __forceinline__ ScaleLoad scale_load(const Src& S, uint8_t* smem, int s, int sl, int wave, int lane) {
  const bool w = wave < 2;
  const int u = 2 * (wave & 1), st = s + u;
  const uint32_t slab = (uint32_t)((w ? S.w_slab : S.x_slab) >> 4);
  ScaleLoad L;
  L.r = make_rsrc((w ? S.ws : S.xs) + (uint64_t)st * slab,
                  st + 1 < S.nsteps ? slab + SC_SLOT : st < S.nsteps ? (uint32_t)SC_SLOT : 0u);
  L.dst = smem + (w ? WS : XS) + (sl + u) * SC_SLOT;
  L.voff = (lane & 31) * 16 + (lane >> 5) * slab;
  return L;
}
__device__ __forceinline__ void issue_scales(const ScaleLoad& L) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(L.r, (lds_ptr)L.dst, 16, L.voff, 0, 0, 0);
}

// What a step's MFMAs take from LDS.
struct Frags {
  i32x4 b[JB][2];
  int sa, sb[JB];  // byte s: the scale for MFMA s
};
// codes: the lane's place in the step's region; ws, xs: in its slots of scales.
template <int R>
__device__ __forceinline__ void read_piece(Frags& F, const uint8_t* codes, const uint8_t* ws, const uint8_t* xs) {
  constexpr int C = R - 1 - JB;
  if constexpr (R == 0)
    F.sa = *(const uint16_t*)ws;
  else if constexpr (C < 0)
    F.sb[R - 1] = *(const uint16_t*)(xs + (R - 1) * 128);
  else
    F.b[C % JB][C / JB] = *(const i32x4*)(codes + C % JB * 2048 + C / JB * 256);
}

template <int B, int E>
__device__ __forceinline__ void mma(f32x16 (&acc)[JB], const Weights& W, const Frags& F) {
  static_for<B, E>([&](auto I) {
    constexpr int s = decltype(I)::value / JB, j = decltype(I)::value % JB;
    const i32x8 a = {W.a[s][0], W.a[s][1], W.a[s][2], W.a[s][3], 0, 0, 0, 0};
    const i32x8 b = {F.b[j][s][0], F.b[j][s][1], F.b[j][s][2], F.b[j][s][3], 0, 0, 0, 0};
    acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[j], 4, 4, s, F.sa, s, F.sb[j]);
  });
}

// Reads [r0, r1) and loads [d0, d1) issued with the I-th MFMA after the barrier;
// SC: scales among them.
template <bool SC, int I>
struct Slot {
  static constexpr int N = NL + (SC ? 1 : 0);
  static constexpr int r0 = I < SPAN ? NR * I / SPAN : NR, r1 = I < SPAN ? NR * (I + 1) / SPAN : NR;
  static constexpr int d0 = I < SPAN ? N * I / SPAN : N, d1 = I < SPAN ? N * (I + 1) / SPAN : N;
};

// Step j, U = j % D; sp: the scale slot of step j - U (0 or D). TAIL: the U-th of
// the last nsteps % D steps, which load nothing more.
template <int U, bool TAIL>
__device__ __forceinline__ void step(f32x16 (&acc)[JB], Weights (&W)[D], const Frags& cur, Frags& nxt, const Src& S,
                                     uint8_t* smem, int j, int sp, int wave, int lane, int frag_off, int scale_off) {
  constexpr bool SC = !TAIL && U % 4 == 0;
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("" : "+s"(wave));  // no LDS addresses of every slot kept in registers
  const int slot = U + 1 < D ? sp + U + 1 : D - sp;
  const uint8_t* codes = smem + (U + 1) % D * REGION + frag_off;
  const uint8_t* ws = smem + WS + slot * SC_SLOT + wave * 128 + scale_off;
  const uint8_t* xs = smem + XS + slot * SC_SLOT + scale_off;
  const __amdgpu_buffer_rsrc_t LW = weight_res(S, j + D - 1);
  const TokenRes LT = token_res(S, smem, j + D, U);
  ScaleLoad LS;
  if constexpr (SC) LS = scale_load(S, smem, j + D, D - sp + U, wave, lane);
  mma<0, PRE>(acc, W[U], cur);
  __builtin_amdgcn_sched_barrier(0);
  // Younger loads than step j + 1's: those of D - 2 steps. The lgkmcnt(0) keeps a
  // refill from overtaking another wave's last reads of the region.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(loads(U + 2 - D, TAIL ? 0 : U)) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  static_for<0, NM - PRE>([&](auto I) {
    using SL = Slot<SC, decltype(I)::value>;
    static_for<SL::r0, SL::r1>([&](auto R) { read_piece<decltype(R)::value>(nxt, codes, ws, xs); });
    static_for<SL::d0, SL::d1>([&](auto P) {
      constexpr int p = decltype(P)::value;
      if constexpr (TAIL)
        return;
      else if constexpr (p < 2)
        load_tokens<p>(LT, wave, lane);
      else if constexpr (p < NL)
        load_weights<p - 2>(W[(U + D - 1) % D], LW, frag_off);
      else
        issue_scales(LS);
    });
  });
  mma<PRE, NM>(acc, W[U], cur);
  static_for<0, NM - PRE>([&](auto I) {
    using SL = Slot<SC, decltype(I)::value>;
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (SL::r1 > SL::r0) __builtin_amdgcn_sched_group_barrier(0x100, SL::r1 - SL::r0, 0);
    if constexpr (!TAIL && SL::d1 > SL::d0) __builtin_amdgcn_sched_group_barrier(0x020, SL::d1 - SL::d0, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
}

// As in mx_fp4_gemm.hip: a range of tiles per XCD, in groups of 4 token tiles.
__device__ inline void tile_coords(uint32_t pid, int tiles_m, int tiles_n, int& tm, int& tn) {
  constexpr int GM = 4;
  const int lid = (int)xcd_order(pid, (uint32_t)(tiles_m * tiles_n));
  const int group = lid / (GM * tiles_n);
  const int gm = min(tiles_m - group * GM, GM);
  const int in_group = lid - group * GM * tiles_n;
  tm = group * GM + in_group % gm;
  tn = in_group / gm;
}

// The wave's 32 (n) x 128 (m) outputs: bf16 through LDS ([m][n], rows of 64
// bytes, 8-byte block nb of row m at nb ^ (m / 4 % 8): 32 lanes on 32 rows write
// 32 bank pairs), then row pieces of 64 bytes, 16 a lane.
template <int EPI>
__device__ __forceinline__ void store_tile(const f32x16 (&acc)[JB], const MidParams& p, uint8_t* ep, int m0, int n0,
                                           int rows_m, int cols, int lane) {
  const int r32 = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const int nb = 2 * q + hi;
      float v[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] = epilogue<EPI>(acc[j][4 * q + r]);
      const bf16x2 p0 = {(__bf16)v[0], (__bf16)v[1]}, p1 = {(__bf16)v[2], (__bf16)v[3]};
      *(i32x2*)(ep + (32 * j + r32) * PITCH + ((nb ^ (r32 >> 2)) << 3)) =
          i32x2{__builtin_bit_cast(int, p0), __builtin_bit_cast(int, p1)};
    }
  // No read may move above another lane's write (LDS order within a wave is kept
  // by the hardware).
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  const __amdgpu_buffer_rsrc_t ry = make_rsrc(p.y + (size_t)m0 * p.N, (uint32_t)(rows_m * p.N * 2));
  const int c = lane & 3;
  const bool n_ok = 8 * c < cols;
#pragma unroll 4
  for (int it = 0; it < MT / 16; ++it) {
    const int m = 16 * it + (lane >> 2);
    const int sw = (m & 31) >> 2;
    const i32x4 v = *(const i32x4*)(ep + m * PITCH + ((((2 * c) ^ sw) & ~1) << 3));
    const i32x4 w = (sw & 1) ? i32x4{v[2], v[3], v[0], v[1]} : v;
    __builtin_amdgcn_raw_buffer_store_b128(w, ry, n_ok ? (m * p.N + n0 + 8 * c) * 2 : kDropOffset, 0, kStoreAux);
  }
}

template <int EPI>
__global__ __launch_bounds__(NT, 2) void fp4_mid_kernel(MidParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  int tm, tn;
  tile_coords(blockIdx.x, p.tiles_m, p.tiles_n, tm, tn);
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int m0 = tm * MT, n0 = tn * MT + wave * 32;
  const int rows_m = min(p.M - m0, MT);
  const int r32 = lane & 31, hi = lane >> 5;

  Src S;
  S.w_slab = (uint64_t)p.RN * 64;
  S.x_slab = (uint64_t)p.RM * 64;
  S.w = p.wq + (size_t)n0 * 64;
  S.x = p.x + (size_t)m0 * 64;
  S.ws = p.ws + (size_t)tn * MT * 4;
  S.xs = p.xs + (size_t)m0 * 4;
  S.nsteps = p.nsteps;
  const int frag_off = (r32 >> 4) * 1024 + (r32 & 15) * 16 + 512 * hi;
  const int scale_off = r32 * 4 + hi * 2;

  // Bias of the lane's weight rows (columns past N: zero, not stored).
  i32x2 bias[4];
  const __amdgpu_buffer_rsrc_t rb =
      make_rsrc(p.bias != nullptr ? p.bias + n0 : nullptr, p.bias != nullptr && n0 < p.N ? (uint32_t)(p.N - n0) * 2u : 0u);
#pragma unroll
  for (int q = 0; q < 4; ++q)
    bias[q] = __builtin_bit_cast(i32x2, __builtin_amdgcn_raw_buffer_load_b64(rb, hi * 8, 16 * q, 0));
  __builtin_amdgcn_sched_barrier(0);
  // The rings' first loads, as the steps -D .. -1 would have issued them (the
  // loop's waits count on it): step v - D brings the tokens of step v, the
  // weights of step v - 1 and, every fourth, the scales of steps v .. v + 3.
  Weights W[D];
  static_for<0, D>([&](auto V) {
    constexpr int v = decltype(V)::value;
    const TokenRes LT = token_res(S, smem, v, v);
    static_for<0, 2>([&](auto P) { load_tokens<decltype(P)::value>(LT, wave, lane); });
    if constexpr (v % 4 == 0) issue_scales(scale_load(S, smem, v, v, wave, lane));
    if constexpr (v > 0) {
      const __amdgpu_buffer_rsrc_t LW = weight_res(S, v - 1);
      static_for<0, 2>([&](auto P) { load_weights<decltype(P)::value>(W[v - 1], LW, frag_off); });
    }
    __builtin_amdgcn_sched_barrier(0);
  });
  f32x16 acc[JB];
#pragma unroll
  for (int q = 0; q < 4; ++q)
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const uint32_t w = (uint32_t)bias[q][r >> 1];
      const float b = (float)__builtin_bit_cast(_Float16, (uint16_t)((r & 1) ? (w >> 16) : (w & 0xFFFFu)));
#pragma unroll
      for (int j = 0; j < JB; ++j) acc[j][4 * q + r] = b;
    }
  // The accumulators are written here, inside the first loads' latency.
#pragma unroll
  for (int j = 0; j < JB; ++j) asm volatile("" : "+a"(acc[j]));
  __builtin_amdgcn_sched_barrier(0);
  // Step 0's tokens and scales: the loads of D - 1 steps are younger.
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"(loads(1 - D, 0)) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  Frags F[2];
  static_for<0, NR>([&](auto R) {
    read_piece<decltype(R)::value>(F[0], smem + frag_off, smem + WS + wave * 128 + scale_off, smem + XS + scale_off);
  });
  int j = 0, sp = 0;
  for (; j + D <= p.nsteps; j += D, sp = D - sp)
    static_for<0, D>([&](auto V) {
      constexpr int v = decltype(V)::value;
      step<v, false>(acc, W, F[v % 2], F[(v + 1) % 2], S, smem, j + v, sp, wave, lane, frag_off, scale_off);
    });
  static_for<0, D - 1>([&](auto V) {
    constexpr int v = decltype(V)::value;
    if (j + v < p.nsteps)
      step<v, true>(acc, W, F[v % 2], F[(v + 1) % 2], S, smem, j + v, sp, wave, lane, frag_off, scale_off);
  });
  __builtin_amdgcn_sched_barrier(0);
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  store_tile<EPI>(acc, p, smem + wave * STAGE, m0, n0, rows_m, p.N - n0, lane);
}

template <int EPI>
hipError_t launch(MidParams p, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = fp4_mid_kernel<EPI>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, LDS, configured);
  if (e != hipSuccess) return e;
  p.tiles_m = (p.M + MT - 1) / MT;
  p.tiles_n = (p.N + MT - 1) / MT;
  hipLaunchKernelGGL(kern, dim3((unsigned)(p.tiles_m * p.tiles_n)), dim3(NT), LDS, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_fp4_linear_mid(const uint8_t* xq, const uint8_t* xs, int64_t M, int64_t K, const uint8_t* wq,
                                 const uint8_t* ws, int64_t N, const void* bias, int epi, void* y,
                                 hipStream_t stream) {
  MidParams p;
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
  p.tiles_m = p.tiles_n = 0;
  return epi == 1 ? launch<1>(p, stream) : launch<0>(p, stream);
}

}  // namespace mx

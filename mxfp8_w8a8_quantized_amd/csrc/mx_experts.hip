// The experts' products of a mixture-of-experts feed-forward block on MXFP4
// weights. For token t and each of its k pairs (expert e, weight w):
//
//   a = act(Wg[e] xhat) * (Wu[e] xhat),  o = Wd[e] hhat,  y = bf16(sum_j w_j o_j)
//
// xhat is the MX quantization of x's row, hhat that of bf16(a), both MXFP8 or
// MXFP4; sums are fp32 and the k terms are added in order j = 0, 1, ...
//
// Launches: (1) tokens to codes, and the plan: the pairs sorted by expert, in tiles
// of up to 128 pairs of one expert (with more than 4096 pairs a second launch ends
// the plan); (2) both halves of the up product, whose tiles gather their tokens'
// rows and write h as codes; (3) the down product, whose o is kept as f16 with an
// exponent a group; (4) the weighted sum of each token's rows. Pairs of an expert
// outside 0 .. E-1 are in no tile and add nothing. Two other forms of the products
// stand in files of their own: mx_experts_tile.hip's larger tiles for many pairs an
// expert, and mx_experts_few.hip for at most 16 tokens, in two launches.
//
// Codes of tokens and of h are row-major here, with K rounded up to 128 (zeros
// past K): a row's 128 K are 128 (MXFP8) or 64 (MXFP4) consecutive bytes, which
// a gather reads whole. Its scales are 4 bytes for each 128 K, the row padded to
// 32 bytes (8 steps, one gather of the product).
//
// Product kernels: 128 weight rows x 128 pairs a workgroup, four waves of 32
// weight rows x 128 pairs on v_mfma_scale_f32_32x32x64_f8f6f4 with the weights as
// the A operand, as in mx_fp4_mid.hip: the weights go from memory to registers
// (a 16-row block of their slab is in lane order), the pairs' rows through LDS.
// In the up product a wave's 32 rows are 16 of Wg and the 16 of Wu for the same
// columns of h, so that both factors of an element meet in one lane.
//
// Measured, 128 tokens, E = 64, k = 8, H = 4096, I = 1408, MXFP4 tokens: (1) 7.2 us,
// (2) 80, (3) 47, (4) 7: 588 MB of weights at 4.6 TB/s, which is what bounds few
// pairs an expert. With many, 8192 tokens, E = 32, k = 4, H = 5120: (1) 25 and 8 us,
// (4) 83 (341 MB in, 84 out).
#include "mx_experts_device.h"

namespace mx {
namespace {

constexpr int NT = 256;
constexpr int MT = kExpertTile;  // pairs per tile
constexpr int JB = 4;            // and their fragments of 32
constexpr int PLAN_THREADS = 1024;
constexpr int kPlanChunk = 4096;  // pairs

// ---------------------------------------------------------------------------
// (1) Plan and tokens' codes.

struct PrepareParams {
  const uint16_t* x;
  int64_t ldx;
  const int32_t* ids;
  int T, k, E, K;
  uint8_t* xq;
  uint8_t* xs;
  uint32_t pitch_q, pitch_s;
  int32_t* rows;  // sorted row -> pair
  int32_t* pos;   // pair -> sorted row, or -1
  ExpertTile* tiles;
  int32_t* n_tiles;
  int chunks;
  int32_t* counts;  // [chunks][kMaxExperts], with more than one chunk
};

// The plan. A chunk is kPlanChunk pairs, one workgroup's: a histogram of the experts
// in LDS gives each pair its place among the chunk's pairs of its expert. With one
// chunk (PLACE follows at once) the running sum over the experts makes it a row;
// with more, a second kernel first adds the histograms of the chunks before. The
// order of an expert's pairs is that in which the threads come; no output depends
// on it, since every row of a tile is computed alike.
struct Pairs {
  int32_t e[kPlanChunk / PLAN_THREADS], place[kPlanChunk / PLAN_THREADS];
};
__device__ __forceinline__ void count_chunk(const PrepareParams& p, int chunk, int32_t* count, Pairs& q) {
  const int t = threadIdx.x, P = p.T * p.k;
  count[t] = 0;
  __syncthreads();
#pragma unroll
  for (int u = 0; u < kPlanChunk / PLAN_THREADS; ++u) {
    const int i = chunk * kPlanChunk + u * PLAN_THREADS + t;
    int32_t e = i < P ? p.ids[i] : -1;
    if (e >= p.E) e = -1;
    q.e[u] = e;
    if (e >= 0) q.place[u] = atomicAdd(&count[e], 1);
  }
  __syncthreads();
}
// Thread e: expert e has n pairs, the chunk's begin at `before` among them. first[e]
// becomes the chunk's first row of the expert; `tiles`: write them down.
__device__ __forceinline__ void place_experts(const PrepareParams& p, int n, int before, bool tiles, int32_t* first) {
  __shared__ int32_t part[2][PLAN_THREADS / 64];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int nt = (n + MT - 1) / MT;
  int sn = n, st = nt;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int un = __shfl_up(sn, off, 64), ut = __shfl_up(st, off, 64);
    if (lane >= off) {
      sn += un;
      st += ut;
    }
  }
  if (lane == 63) {
    part[0][wave] = sn;
    part[1][wave] = st;
  }
  __syncthreads();
  for (int w = 0; w < wave; ++w) {
    sn += part[0][w];
    st += part[1][w];
  }
  first[t] = sn - n + before;
  if (tiles) {
    for (int i = 0; i < nt; ++i) p.tiles[st - nt + i] = {t, sn - n + i * MT, min(n - i * MT, MT), 0};
    if (t == PLAN_THREADS - 1) *p.n_tiles = st;
  }
  __syncthreads();
}
__device__ __forceinline__ void place_pairs(const PrepareParams& p, int chunk, const int32_t* first, const Pairs& q) {
  const int t = threadIdx.x, P = p.T * p.k;
#pragma unroll
  for (int u = 0; u < kPlanChunk / PLAN_THREADS; ++u) {
    const int i = chunk * kPlanChunk + u * PLAN_THREADS + t;
    if (i >= P) continue;
    const int r = q.e[u] >= 0 ? first[q.e[u]] + q.place[u] : -1;
    p.pos[i] = r;
    if (r >= 0) p.rows[r] = i;
  }
}
static_assert(kMaxExperts == PLAN_THREADS, "a thread an expert");

// The chunks' second pass.
__global__ __launch_bounds__(PLAN_THREADS) void place_kernel(PrepareParams p) {
  __shared__ int32_t first[kMaxExperts];
  const int t = threadIdx.x, chunk = blockIdx.x;
  int n = 0, before = 0;
  for (int c = 0; c < p.chunks; ++c) {
    const int v = p.counts[c * kMaxExperts + t];
    if (c < chunk) before += v;
    n += v;
  }
  Pairs q;
  const int P = p.T * p.k;
#pragma unroll
  for (int u = 0; u < kPlanChunk / PLAN_THREADS; ++u) {
    const int i = chunk * kPlanChunk + u * PLAN_THREADS + t;
    int32_t e = i < P ? p.ids[i] : -1;
    if (e >= p.E) e = -1;
    q.e[u] = e;
    q.place[u] = e >= 0 ? p.pos[i] : 0;
  }
  place_experts(p, n, before, chunk == 0, first);
  place_pairs(p, chunk, first, q);
}

// The first workgroups count a chunk of pairs each (the only one makes the plan);
// each wave of the others takes a token's row.
template <bool X8>
__global__ __launch_bounds__(PLAN_THREADS) void prepare_kernel(PrepareParams p) {
  if ((int)blockIdx.x < p.chunks) {
    __shared__ int32_t count[kMaxExperts];
    const int t = threadIdx.x, chunk = blockIdx.x;
    Pairs q;
    count_chunk(p, chunk, count, q);
    if (p.chunks == 1) {
      place_experts(p, count[t], 0, true, count);
      place_pairs(p, 0, count, q);
    } else {
      p.counts[chunk * kMaxExperts + t] = count[t];
#pragma unroll
      for (int u = 0; u < kPlanChunk / PLAN_THREADS; ++u)
        if (q.e[u] >= 0) p.pos[chunk * kPlanChunk + u * PLAN_THREADS + t] = q.place[u];
    }
    return;
  }
  const int lane = threadIdx.x & 63;
  const int64_t row = ((int64_t)blockIdx.x - p.chunks) * (PLAN_THREADS / 64) + (threadIdx.x >> 6);
  if (row >= p.T) return;
  const uint16_t* x = p.x + row * p.ldx;
  uint8_t* q = p.xq + row * p.pitch_q;
  uint8_t* s = p.xs + row * p.pitch_s;
  const int KP = (p.K + 127) & ~127;
  for (int k0 = 0; k0 < KP; k0 += 512) {
    const int k = k0 + 8 * lane;
    const i32x4 v = k < p.K ? *(const i32x4*)(x + k) : i32x4{0, 0, 0, 0};
    const uint32_t w[4] = {(uint32_t)v[0], (uint32_t)v[1], (uint32_t)v[2], (uint32_t)v[3]};
    uint32_t sc;
    if constexpr (X8) {
      uint32_t c[2];
      quantize8_bf16(w, c, sc);
      if (k < KP) *(i32x2*)(q + k) = i32x2{(int)c[0], (int)c[1]};
    } else {
      const uint32_t c = fp4_quantize8_bf16(w, sc);
      if (k < KP) *(uint32_t*)(q + k / 2) = c;
    }
    if (k < KP && (lane & 3) == 0) s[k / 32] = (uint8_t)sc;
  }
}

// ---------------------------------------------------------------------------
// (2), (3) Products.

template <bool X8>
struct Shape {
  static constexpr int D = X8 ? 4 : 8;          // steps in flight
  static constexpr int ROW = X8 ? 128 : 64;     // bytes of a row's step
  static constexpr int REGION = MT * ROW;
  static constexpr int NX = ROW * MT / 4096;    // row DMAs per wave and step
  static constexpr int L = NX + 3;              // loads per wave and step: rows, weights (2), their scales
  static constexpr int XS_SLOT = MT * 32;       // scales of 8 steps: [32 rows][4 steps][row][16]
  static constexpr int XS = D * REGION;
  static constexpr int LDS = XS + 2 * XS_SLOT;
  static constexpr int NB = X8 ? 2 : 1;         // 16-byte reads per fragment and MFMA
  // Chunk c (16 bytes) of row r is at c ^ swizzle(r): the 16 rows of a read's
  // phase then cover the banks once.
  __device__ static int swizzle(int r) { return X8 ? (r >> 1) & 7 : (r >> 2) & 3; }
};

template <bool X8>
struct Half {  // the pairs' fragments of one of a step's two MFMA sets
  i32x4 b[JB][Shape<X8>::NB];
};
struct Weights {  // of a step: fragments of MFMA sets 0 and 1, and their scales in bytes 0 and 1
  i32x4 a[2];
  int s;
};

template <bool X8>
struct Source {
  const uint8_t* x;  // the operand that the lane's row offsets count from
  const uint8_t* xs;
  uint32_t x_bytes, xs_bytes;
  uint32_t xo[Shape<X8>::NX], xso;  // the lane's offsets
  const uint8_t* w;  // the expert's slab 0
  const uint8_t* ws;
  uint32_t wo, wso;
  int R, nsteps;
};

// Loads of step j (past the last one zeros from an empty resource, so that every
// step has the same number of them).
template <int V, bool X8>
__device__ __forceinline__ void load_rows(const Source<X8>& S, uint8_t* smem, int j, int wave) {  // V = j % 8
  using Sh = Shape<X8>;
  const bool on = j < S.nsteps;
  if constexpr (V == 0) {
    const __amdgpu_buffer_rsrc_t r = make_rsrc(S.xs + (int64_t)j * 4, on ? S.xs_bytes - (uint32_t)j * 4u : 0u);
    dma(r, smem + Sh::XS + (j / 8 % 2) * Sh::XS_SLOT + wave * 1024, S.xso);
  }
  const __amdgpu_buffer_rsrc_t r =
      make_rsrc(S.x + (int64_t)j * Sh::ROW, on ? S.x_bytes - (uint32_t)(j * Sh::ROW) : 0u);
  uint8_t* reg = smem + (V % Sh::D) * Sh::REGION + wave * (Sh::NX * 1024);
#pragma unroll
  for (int i = 0; i < Sh::NX; ++i) dma(r, reg + i * 1024, S.xo[i]);
}
template <bool X8>
__device__ __forceinline__ void load_weights(Weights& W, const Source<X8>& S, int j) {
  const bool on = j < S.nsteps;
  const __amdgpu_buffer_rsrc_t r = make_rsrc(S.w + (int64_t)j * S.R * 64, on ? (uint32_t)S.R * 64u : 0u);
  const __amdgpu_buffer_rsrc_t rs = make_rsrc(S.ws + (int64_t)j * S.R * 4, on ? (uint32_t)S.R * 4u : 0u);
  W.a[0] = __builtin_amdgcn_raw_buffer_load_b128(r, S.wo, 0, 0);
  W.a[1] = __builtin_amdgcn_raw_buffer_load_b128(r, S.wo + 256u, 0, 0);
  W.s = (uint16_t)__builtin_amdgcn_raw_buffer_load_b16(rs, S.wso, 0, 0);
}

// Fragments of MFMA set `s` of step j. Lane half h of the set takes group 2 h + s
// of the step's four (mx_fp4_gemm.hip says why that is free); E4M3: 16 elements of
// group s, then 16 of group 2 + s.
template <bool X8, int s, int D>
__device__ __forceinline__ void read_half(Half<X8>& F, const uint8_t* smem, int lane) {  // D: the step's region
  using Sh = Shape<X8>;
  const int r32 = lane & 31, hi = lane >> 5, sw = Sh::swizzle(r32);
  const uint8_t* row = smem + D * Sh::REGION + r32 * Sh::ROW;
#pragma unroll
  for (int f = 0; f < JB; ++f) {
    if constexpr (X8) {
      F.b[f][0] = *(const i32x4*)(row + f * 32 * Sh::ROW + (((2 * s + hi) ^ sw) << 4));
      F.b[f][1] = *(const i32x4*)(row + f * 32 * Sh::ROW + (((4 + 2 * s + hi) ^ sw) << 4));
    } else {
      F.b[f][0] = *(const i32x4*)(row + f * 32 * Sh::ROW + (((2 * hi + s) ^ sw) << 4));
    }
  }
}
// The rows' scales of the four steps from j on, V = j % 8: the 16 bytes of each row of
// the four fragments in one conflict-free read (two bytes a row and step cost 15
// cycles of bank conflicts each).
template <bool X8, int V>
__device__ __forceinline__ void read_scales(i32x4 (&q)[JB], const uint8_t* smem, int j, int lane) {
  using Sh = Shape<X8>;
  const uint8_t* p = smem + Sh::XS + (j / 8 % 2) * Sh::XS_SLOT + V / 4 * 512 + (lane & 31) * 16;
#pragma unroll
  for (int f = 0; f < JB; ++f) q[f] = *(const i32x4*)(p + f * 1024);
}

template <bool X8, int s>
__device__ __forceinline__ void mma_half(f32x16 (&acc)[JB], const Weights& W, const Half<X8>& F, const int (&sb)[JB]) {
  const i32x8 a = {W.a[s][0], W.a[s][1], W.a[s][2], W.a[s][3], 0, 0, 0, 0};
  static_for<0, JB>([&](auto J) {
    constexpr int j = decltype(J)::value;
    const i32x4& b0 = F.b[j][0];
    if constexpr (X8) {
      const i32x4& b1 = F.b[j][1];
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], b1[0], b1[1], b1[2], b1[3]};
      acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[j], 4, 0, s, W.s, s, sb[j]);
    } else {
      const i32x8 b = {b0[0], b0[1], b0[2], b0[3], 0, 0, 0, 0};
      acc[j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(a, b, acc[j], 4, 4, s, W.s, s, sb[j]);
    }
  });
}

// Step j, V = j % 8: MFMA set 0 while set 1's fragments are read; one barrier, behind
// which step j + 1's rows are there and every wave is done with step j's; set 1 while
// step j + 1's first fragments are read and step j + D is sent for into the place of
// step j.
template <int V, bool X8>
__device__ __forceinline__ void step(f32x16 (&acc)[JB], Weights (&W)[Shape<X8>::D], Half<X8>& F0, Half<X8>& F1,
                                     i32x4 (&q)[JB], const Source<X8>& S, uint8_t* smem, int j, int wave, int lane) {
  using Sh = Shape<X8>;
  // Lane half h: the scales of groups 2 h and 2 h + 1 in bytes 0 and 1.
  int sb[JB];
#pragma unroll
  for (int f = 0; f < JB; ++f) sb[f] = (int)((uint32_t)q[f][V % 4] >> (lane >> 5 << 4));
  constexpr int D = Sh::D, v = V, d = V % D, refill = (V + D) % 8;
  read_half<X8, 1, d>(F1, smem, lane);
  mma_half<X8, 0>(acc, W[d], F0, sb);
  static_for<0, JB>([&](auto I) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if constexpr (decltype(I)::value < 2) __builtin_amdgcn_sched_group_barrier(0x100, 2 * Sh::NB, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
  // Younger loads than step j + 1's. The lgkmcnt(0) keeps the refill from
  // overtaking another wave's reads.
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"((D - 2) * Sh::L) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  read_half<X8, 0, (d + 1) % D>(F0, smem, lane);
  if constexpr (V % 4 == 3) read_scales<X8, (V + 1) % 8>(q, smem, j + 1, lane);
  load_rows<refill>(S, smem, j + D, wave);
  load_weights(W[(d + D - 1) % D], S, j + D - 1);
  mma_half<X8, 1>(acc, W[d], F1, sb);
  static_for<0, JB>([&](auto I) {
    constexpr int i = decltype(I)::value;
    constexpr int loads = Sh::L + (refill == 0 ? 1 : 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x100, Sh::NB + (V % 4 == 3 ? 1 : 0), 0);
    if constexpr (loads * (i + 1) / JB > loads * i / JB)
      __builtin_amdgcn_sched_group_barrier(0x020, loads * (i + 1) / JB - loads * i / JB, 0);
  });
  __builtin_amdgcn_sched_barrier(0);
}

// acc = the wave's 32 weight rows x 128 pairs.
template <bool X8>
__device__ __forceinline__ void product(f32x16 (&acc)[JB], const Source<X8>& S, uint8_t* smem, int wave, int lane) {
  using Sh = Shape<X8>;
  constexpr int D = Sh::D;
  Weights W[D];
  static_for<0, D>([&](auto V) {
    constexpr int v = decltype(V)::value;
    load_rows<v>(S, smem, v, wave);
    if constexpr (v > 0) load_weights(W[v - 1], S, v - 1);
    __builtin_amdgcn_sched_barrier(0);
  });
#pragma unroll
  for (int j = 0; j < JB; ++j)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[j][r] = 0.f;
  // (The loads of scales, one in 8 steps, are left out of the counts: a wait for
  // fewer loads in flight is on the safe side.)
  asm volatile("s_waitcnt vmcnt(%0)" ::"n"((D - 1) * Sh::L) : "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
  Half<X8> F0, F1;
  i32x4 q[JB];
  read_half<X8, 0, 0>(F0, smem, lane);
  read_scales<X8, 0>(q, smem, 0, lane);
  int j = 0;
  for (; j + 8 <= S.nsteps; j += 8)
    static_for<0, 8>([&](auto V) {
      step<decltype(V)::value>(acc, W, F0, F1, q, S, smem, j + decltype(V)::value, wave, lane);
    });
  static_for<0, 7>([&](auto V) {
    if (j + decltype(V)::value < S.nsteps)
      step<decltype(V)::value>(acc, W, F0, F1, q, S, smem, j + decltype(V)::value, wave, lane);
  });
  // The last MFMAs' results are read 20 wait states after them at the earliest; the
  // compiler counts the scheduling directives above among its own.
  asm volatile("s_nop 15\n\ts_nop 7" : "+v"(acc[0]), "+v"(acc[1]), "+v"(acc[2]), "+v"(acc[3]));
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_sched_barrier(0);
}

// Codes of the tile's 64 columns of h. Lane: pair 32 j + r32; registers 4 q + r
// of an accumulator are Wg's row (column of h) 16 wave + 8 q + 4 hi + r for q = 0,
// 1 and the same one's Wu for q = 2, 3. A group of 32 columns is in two waves: its
// largest magnitude is found through LDS.
template <bool X8, int ACT>
__device__ __forceinline__ void store_h(const f32x16 (&acc)[JB], const ProductParams& p, uint8_t* smem, int m0,
                                        int count, int n0, int wave, int lane) {
  constexpr int W = X8 ? 64 : 32;       // bytes of a row's codes
  constexpr int PITCH = W + 16;         // in LDS
  uint8_t* codes = smem;
  uint8_t* scales = smem + MT * PITCH;  // [pair][2]
  uint32_t* top = (uint32_t*)(scales + MT * 2);  // [wave][pair]
  const int r32 = lane & 31, hi = lane >> 5;
  uint32_t v[JB][4], m[JB];
#pragma unroll
  for (int j = 0; j < JB; ++j) {
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      float h[4];
#pragma unroll
      for (int r = 0; r < 4; ++r) h[r] = activation<ACT>(acc[j][4 * q + r]) * acc[j][8 + 4 * q + r];
      v[j][2 * q] = pack_bf16(h[0], h[1]);
      v[j][2 * q + 1] = pack_bf16(h[2], h[3]);
    }
    m[j] = bf16_amax_bits(v[j]);
    const auto sw = __builtin_amdgcn_permlane32_swap(m[j], m[j], false, false);
    m[j] = max((uint32_t)sw[0], (uint32_t)sw[1]);
    if (hi == 0) top[wave * MT + 32 * j + r32] = m[j];
  }
  __syncthreads();
  const bool real = n0 + 32 * (wave >> 1) < p.I;  // columns past I: zero codes and scales
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const uint32_t amax = max(m[j], top[(wave ^ 1) * MT + 32 * j + r32]);
    uint32_t sc = X8 ? scale_code_from_exponent(amax >> 7) : fp4_scale_code(amax >> 7);
    uint8_t* row = codes + (32 * j + r32) * PITCH;
#pragma unroll
    for (int q = 0; q < 2; ++q) {
      const int col = 16 * wave + 8 * q + 4 * hi;
      if constexpr (X8) {
        const uint32_t c = e4m3_encode4_bf16(v[j][2 * q], v[j][2 * q + 1], sc);
        *(uint32_t*)(row + col) = real ? c : 0u;
      } else {
        const uint32_t c = e2m1_encode4_bf16(v[j][2 * q], v[j][2 * q + 1], sc);
        *(uint16_t*)(row + col / 2) = (uint16_t)(real ? c : 0u);
      }
    }
    if ((wave & 1) == 0 && hi == 0) scales[(32 * j + r32) * 2 + (wave >> 1)] = (uint8_t)(real ? sc : 0u);
  }
  __syncthreads();
  constexpr int PIECES = W / 16;
  const int t = threadIdx.x;
  for (int u = t; u < count * PIECES; u += NT) {
    const int r = u / PIECES, c = u % PIECES;
    *(i32x4*)(p.hq + (int64_t)(m0 + r) * p.hpitch_q + n0 * W / 64 + 16 * c) = *(const i32x4*)(codes + r * PITCH + 16 * c);
  }
  if (t < count) *(uint16_t*)(p.hs + (int64_t)(m0 + t) * p.hpitch_s + n0 / 32) = *(const uint16_t*)(scales + 2 * t);
}

// o of the tile's 128 columns.
__device__ __forceinline__ void store_o(const f32x16 (&acc)[JB], const ProductParams& p, uint8_t* smem, int m0, int count,
                                        int n0, int wave, int lane) {
  constexpr int PITCH = 2 * MT + 16;
  uint8_t* scales = smem + MT * PITCH;  // [row][4]
  const int r32 = lane & 31, hi = lane >> 5;
#pragma unroll
  for (int j = 0; j < JB; ++j) {
    const uint32_t e = o_exponent(acc[j]);
    uint32_t c[8];
    o_pack(acc[j], e, c);
    uint8_t* row = smem + (32 * j + r32) * PITCH + 64 * wave + 8 * hi;
#pragma unroll
    for (int q = 0; q < 4; ++q) *(i32x2*)(row + 16 * q) = i32x2{(int)c[2 * q], (int)c[2 * q + 1]};
    if (hi == 0) scales[(32 * j + r32) * 4 + wave] = (uint8_t)e;
  }
  __syncthreads();
  const int t = threadIdx.x;
  for (int u = t; u < count * 16; u += NT) {
    const int r = u >> 4, c = u & 15;
    if (n0 + 8 * c < p.H)
      *(i32x4*)(p.o + (int64_t)(m0 + r) * p.H + n0 + 8 * c) = *(const i32x4*)(smem + r * PITCH + 16 * c);
  }
  if (t < count) *(uint32_t*)(p.os + (int64_t)(m0 + t) * p.opitch_s + n0 / 32) = *(const uint32_t*)(scales + 4 * t);
}

template <bool UP, bool X8, int ACT>
__global__ __launch_bounds__(NT, 2) void product_kernel(ProductParams p) {
  extern __shared__ __attribute__((aligned(16))) uint8_t smem[];
  using Sh = Shape<X8>;
  ExpertTile tile;
  int tn;
  if (!find_tile(p, tile, tn)) return;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int r32 = lane & 31, hi = lane >> 5;

  Source<X8> S;
  S.nsteps = p.nsteps;
  S.R = p.R;
  S.w = p.wq + (int64_t)tile.expert * p.nsteps * p.R * 64;
  S.ws = p.ws + (int64_t)tile.expert * p.nsteps * p.R * 4;
  // The lane's weight row; rows past the slab's read zeros.
  const int n0 = tn * (UP ? MT / 2 : MT);
  const int row = UP ? n0 + 16 * wave + (r32 & 15) + (r32 >> 4) * p.I : n0 + 32 * wave + r32;
  S.wo = (uint32_t)((row >> 4) * 1024 + (row & 15) * 16 + 512 * hi);
  S.wso = (uint32_t)(row * 4 + 2 * hi);
  // The pairs' rows: rows past the tile's count repeat its last one.
  if constexpr (UP) {
    S.x = p.x;
    S.xs = p.xs;
    S.x_bytes = p.x_bytes;
    S.xs_bytes = p.xs_bytes;
  } else {
    S.x = p.x + (int64_t)tile.first * p.pitch_q;
    S.xs = p.xs + (int64_t)tile.first * p.pitch_s;
    S.x_bytes = (uint32_t)tile.count * p.pitch_q;
    S.xs_bytes = (uint32_t)tile.count * p.pitch_s;
  }
  auto source_row = [&](int r) -> uint32_t {
    const int c = min(r, tile.count - 1);
    return UP ? (uint32_t)p.rows[tile.first + c] / (uint32_t)p.k : (uint32_t)c;
  };
  constexpr int LPR = Sh::ROW / 16;  // lanes per row
#pragma unroll
  for (int i = 0; i < Sh::NX; ++i) {
    const int r = (wave * Sh::NX + i) * (64 / LPR) + lane / LPR;
    S.xo[i] = source_row(r) * p.pitch_q + (uint32_t)(((lane % LPR) ^ Sh::swizzle(r)) * 16);
  }
  S.xso = source_row(32 * wave + (lane & 31)) * p.pitch_s + (uint32_t)(lane >> 5) * 16u;

  f32x16 acc[JB];
  product(acc, S, smem, wave, lane);
  if constexpr (UP)
    store_h<X8, ACT>(acc, p, smem, tile.first, tile.count, n0, wave, lane);
  else
    store_o(acc, p, smem, tile.first, tile.count, n0, wave, lane);
}

// ---------------------------------------------------------------------------
// (4) y[t] = bf16(sum_j w[t][j] o[pos[t][j]]), eight columns a thread.

__global__ __launch_bounds__(NT) void combine_kernel(const uint16_t* __restrict__ o, const uint8_t* __restrict__ os,
                                                     uint32_t opitch_s, const int32_t* __restrict__ pos,
                                                     const float* __restrict__ weights, int k, int H, int64_t pieces,
                                                     uint16_t* __restrict__ y) {
  const int64_t u = (int64_t)blockIdx.x * NT + threadIdx.x;
  if (u >= pieces) return;
  const int64_t t = u / (uint32_t)(H / 8);
  const int n = (int)(u - t * (H / 8)) * 8;
  float v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int j = 0; j < k; ++j) {
    const int r = pos[t * k + j];
    if (r < 0) continue;
    const uint32_t e = os[(int64_t)r * opitch_s + n / 32];
    const f16x8 a = *(const f16x8*)(o + (int64_t)r * H + n);
    const float w = weights[t * k + j], f = __uint_as_float((e - 14u) << 23);  // 2^(e - 127 - 14)
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = __builtin_fmaf(w, (float)a[i] * f, v[i]);
  }
  *(i32x4*)(y + t * H + n) = i32x4{(int)pack_bf16(v[0], v[1]), (int)pack_bf16(v[2], v[3]), (int)pack_bf16(v[4], v[5]),
                                   (int)pack_bf16(v[6], v[7])};
}

template <bool UP, bool X8, int ACT>
hipError_t launch_product(const ProductParams& p, int64_t max_tiles, hipStream_t st) {
  static std::atomic<uint64_t> configured{0};  // per instantiation
  auto kern = product_kernel<UP, X8, ACT>;
  const hipError_t e = allow_dynamic_lds((const void*)kern, Shape<X8>::LDS, configured);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(max_tiles * p.tiles_n)), dim3(NT), Shape<X8>::LDS, st, p);
  return hipGetLastError();
}

// Tiles of 256 weight rows where an expert has many pairs, by the average over all E.
// Measured, 128-row tiles and 256-row ones, in us: MXFP8 tokens, E = 32, H = 4096, I =
// 1408, k = 4: 64 pairs an expert 119 and 112, 128 145 and 127, 512 401 and 371; E = 8, H
// = 5120, I = 2048: 64 49 and 56, 128 64 and 62; E = 64, H = 2048, I = 768: 128 91 and 97.
// MXFP4, E = 32: 128 130 and 115. So the average alone is a coarse rule: it leaves out how
// the tiles fill the last round of workgroups, which loses 14% at the 64 pairs of E = 8
// and 7% at the 128 of E = 64, and experts without a token count in it.
bool large_tiles(const ExpertsArgs& a) { return a.T * a.k >= 64 * a.E; }

// A few tokens, whose products read each expert's weights once in two launches. Measured
// with tiles and in this form, in us: E = 64, H = 4096, I = 1408, k = 4, MXFP8 tokens: 1
// token 31.2 and 15.7, 16 tokens 106 and 91; nowhere up to 16 tokens slower. A column of
// the matrix instruction is a token (down) or a pair (up): 16.
bool few(const ExpertsArgs& a) { return a.T <= kFewTokens && a.T * a.k <= kFewPairs; }

template <bool X8>
hipError_t run(const ExpertsArgs& a, const ExpertsWorkspace& w, hipStream_t st) {
  uint8_t* base = (uint8_t*)a.workspace;
  const int64_t max_tiles = w.max_tiles;
  PrepareParams q;
  q.x = (const uint16_t*)a.x;
  q.ldx = a.ldx;
  q.ids = a.ids;
  q.T = (int)a.T;
  q.k = (int)a.k;
  q.E = (int)a.E;
  q.K = (int)a.H;
  q.xq = base + w.xq;
  q.xs = base + w.xs;
  q.pitch_q = w.xpitch_q;
  q.pitch_s = w.xpitch_s;
  q.rows = (int32_t*)(base + w.rows);
  q.pos = (int32_t*)(base + w.pos);
  q.tiles = (ExpertTile*)(base + w.tiles);
  q.n_tiles = (int32_t*)(base + w.n_tiles);
  q.chunks = (int)w.chunks;
  q.counts = (int32_t*)(base + w.counts);
  const unsigned blocks = (unsigned)(w.chunks + (a.T + PLAN_THREADS / 64 - 1) / (PLAN_THREADS / 64));
  hipLaunchKernelGGL(prepare_kernel<X8>, dim3(blocks), dim3(PLAN_THREADS), 0, st, q);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  if (w.chunks > 1) {
    hipLaunchKernelGGL(place_kernel, dim3((unsigned)w.chunks), dim3(PLAN_THREADS), 0, st, q);
    if ((e = hipGetLastError()) != hipSuccess) return e;
  }

  ProductParams p;
  p.x = q.xq;
  p.xs = q.xs;
  p.pitch_q = w.xpitch_q;
  p.pitch_s = w.xpitch_s;
  p.x_bytes = (uint32_t)(a.T * w.xpitch_q);
  p.xs_bytes = (uint32_t)(a.T * w.xpitch_s);
  p.wq = a.up_q;
  p.ws = a.up_s;
  p.R = (int)slab_rows(2 * a.I);
  p.k = (int)a.k;
  p.nsteps = (int)fp4_slabs(a.H);
  p.I = (int)a.I;
  p.H = (int)a.H;
  p.tiles_n = (int)(2 * fp4_slabs(a.I));
  p.rows = q.rows;
  p.tiles = q.tiles;
  p.n_tiles = q.n_tiles;
  p.hq = base + w.hq;
  p.hs = base + w.hs;
  p.hpitch_q = w.hpitch_q;
  p.hpitch_s = w.hpitch_s;
  p.o = (uint16_t*)(base + w.o);
  p.os = base + w.os;
  p.opitch_s = w.opitch_s;
  const bool large = large_tiles(a);
  e = large         ? launch_experts_tile(p, true, X8, a.gate, max_tiles, st)
      : a.gate == 1 ? launch_product<true, X8, 1>(p, max_tiles, st)
                    : launch_product<true, X8, 0>(p, max_tiles, st);
  if (e != hipSuccess) return e;

  p.x = p.hq;
  p.xs = p.hs;
  p.pitch_q = w.hpitch_q;
  p.pitch_s = w.hpitch_s;
  p.wq = a.down_q;
  p.ws = a.down_s;
  p.R = (int)slab_rows(a.H);
  p.nsteps = (int)fp4_slabs(a.I);
  p.tiles_n = (int)((a.H + MT - 1) / MT);
  e = large ? launch_experts_tile(p, false, X8, 0, max_tiles, st) : launch_product<false, X8, 0>(p, max_tiles, st);
  if (e != hipSuccess) return e;

  const int64_t pieces = a.T * (a.H / 8);
  hipLaunchKernelGGL(combine_kernel, dim3((unsigned)((pieces + NT - 1) / NT)), dim3(NT), 0, st, p.o, p.os, p.opitch_s, q.pos,
                     a.weights, (int)a.k, (int)a.H, pieces, (uint16_t*)a.y);
  return hipGetLastError();
}

}  // namespace

ExpertsWorkspace experts_workspace(int64_t T, int64_t k, int64_t E, int64_t H, int64_t I, int fp4) {
  ExpertsWorkspace w;
  const int64_t P = T * k, SH = fp4_slabs(H), SI = fp4_slabs(I);
  w.xpitch_q = (uint32_t)(SH * (fp4 ? 64 : 128));
  w.hpitch_q = (uint32_t)(SI * (fp4 ? 64 : 128));
  w.xpitch_s = (uint32_t)((SH + 7) / 8 * 32);
  w.hpitch_s = (uint32_t)((SI + 7) / 8 * 32);
  w.max_tiles = experts_max_tiles(T, k, E);
  int64_t at = 0;
  auto take = [&](int64_t bytes) {
    const int64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  w.xq = take(T * w.xpitch_q);
  w.xs = take(T * w.xpitch_s);
  w.hq = take(P * w.hpitch_q);
  w.hs = take(P * w.hpitch_s);
  w.opitch_s = (uint32_t)((H + 127) / 128 * 4);
  w.o = take(P * H * 2);
  w.os = take(P * w.opitch_s);
  w.rows = take(P * 4);
  w.pos = take(P * 4);
  w.tiles = take(w.max_tiles * (int64_t)sizeof(ExpertTile));
  w.n_tiles = take(4);
  w.chunks = (P + kPlanChunk - 1) / kPlanChunk;
  w.counts = take(w.chunks > 1 ? w.chunks * kMaxExperts * 4 : 0);
  w.bytes = at;
  return w;
}

hipError_t launch_fp4_experts(const ExpertsArgs& a, hipStream_t stream) {
  const ExpertsWorkspace w = experts_workspace(a.T, a.k, a.E, a.H, a.I, a.fp4);
  if (few(a)) {
    FewParams p;
    p.x = (const uint16_t*)a.x;
    p.ldx = a.ldx;
    p.ids = a.ids;
    p.weights = a.weights;
    p.T = (int)a.T;
    p.k = (int)a.k;
    p.E = (int)a.E;
    p.H = (int)a.H;
    p.I = (int)a.I;
    p.RU = (int)slab_rows(2 * a.I);
    p.RD = (int)slab_rows(a.H);
    p.up_q = a.up_q;
    p.up_s = a.up_s;
    p.down_q = a.down_q;
    p.down_s = a.down_s;
    p.hq = (uint8_t*)a.workspace + w.hq;
    p.hs = (uint8_t*)a.workspace + w.hs;
    p.hpitch_q = w.hpitch_q;
    p.hpitch_s = w.hpitch_s;
    p.y = (uint16_t*)a.y;
    p.tiles_n = 0;
    return launch_experts_few(p, !a.fp4, a.gate, stream);
  }
  return a.fp4 ? run<false>(a, w, stream) : run<true>(a, w, stream);
}

}  // namespace mx

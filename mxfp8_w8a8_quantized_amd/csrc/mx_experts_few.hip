// The experts' products (mx_experts.hip says what they are) for at most 16 tokens, where
// the weights of the experts in use are all there is to read: two launches, no plan.
//
// v_mfma_scale_f32_16x16x128_f8f6f4 with 16 weight rows as the A operand, from memory
// straight to registers, as in mx_fp4_small.hip; the columns are pairs of one expert in
// the up product, tokens in the down product. A wave takes a range of K and the partial
// sums meet in LDS in wave order.
//
// Up: a workgroup for each pair and 32 columns of h, which leaves unless its pair is
// the first of its expert; it takes all of the expert's pairs (their bf16 rows are
// quantized in the lanes) and writes h as codes. A second pair of a token with the same
// expert has the same o: only the first is computed.
//
// Down: a workgroup takes 16 output columns, for all experts in use one after the
// other, the (expert, 128-K) steps in ranges over 8 waves; a token's column of an
// expert's product is multiplied by its weight and added to the token's sum, so no o
// goes through memory and nothing is left to combine.
//
// Bound by the memory. Measured with MXFP8 tokens: 1 token, E = 64, k = 8, H = 5120, I =
// 2048: up 17.2 us (84 MB of codes, 4.9 TB/s), down 15.7 (42 MB, 2.7 TB/s: the waves'
// ranges are 16 steps long); 13 tokens, k = 4, H = 4096, I = 1408: 43 and 26.5.
#include "mx_experts_device.h"
#include "mx_fp4_few_device.h"

namespace mx {
namespace {

constexpr int kTokens = kFewTokens, kPairs = kFewPairs;

// ---------------------------------------------------------------------------
// Up.

constexpr int UW = 8;  // waves

template <bool X8, int ACT>
__global__ __launch_bounds__(64 * UW, 4) void few_up_kernel(FewParams p) {
  __shared__ f32x4 sums[UW][4][64];
  __shared__ int list[kTokens];
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int pair = (int)(blockIdx.x / (uint32_t)p.tiles_n), tn = (int)(blockIdx.x - (uint32_t)pair * (uint32_t)p.tiles_n);
  const int n0 = 32 * tn, P = p.T * p.k;

  // The expert's pairs, but those behind another one of the same token.
  const int e = p.ids[pair];
  if (e < 0 || e >= p.E) return;
  const int i0 = lane, i1 = 64 + lane;
  const uint64_t m0 = __ballot(i0 < P && p.ids[min(i0, P - 1)] == e), m1 = __ballot(i1 < P && p.ids[min(i1, P - 1)] == e);
  auto has = [&](int i) { return ((i < 64 ? m0 >> i : m1 >> (i - 64)) & 1) != 0; };
  auto counts = [&](int i) {
    if (i >= P || !has(i)) return false;
    for (int j = i / p.k * p.k; j < i; ++j)
      if (has(j)) return false;
    return true;
  };
  const uint64_t f0 = __ballot(counts(i0)), f1 = __ballot(counts(i1));
  const int first = f0 != 0 ? __builtin_ctzll(f0) : 64 + __builtin_ctzll(f1);
  if (pair != first) return;
  const int count = __builtin_popcountll(f0) + __builtin_popcountll(f1);  // at most one a token
  if (wave == 0) {
    const uint64_t below = (uint64_t(1) << lane) - 1;
    if ((f0 >> lane) & 1) list[__builtin_popcountll(f0 & below)] = i0;
    if ((f1 >> lane) & 1) list[__builtin_popcountll(f0) + __builtin_popcountll(f1 & below)] = i1;
  }
  __syncthreads();

  const int c = lane & 15, G = lane >> 4;
  const int column = list[min(c, count - 1)];  // columns past the last repeat it
  const bool real = n0 < p.I;                  // columns of h past I: zeros
  const int S = (int)fp4_slabs(p.H);
  const int s0 = real ? wave * S / UW : 0, s1 = real ? (wave + 1) * S / UW : 0;
  const uint8_t* wq = p.up_q + (int64_t)e * S * p.RU * 64;
  const uint8_t* ws = p.up_s + (int64_t)e * S * p.RU * 4;
  const uint16_t* x = p.x + (int64_t)(column / p.k) * p.ldx;
  // Blocks of 16 weight rows: two of Wg, two of Wu.
  auto block = [&](int i) { return (n0 + (i & 1) * 16 + (i >> 1) * p.I) / 16; };

  struct Step {
    i32x4 a[4], b[4];
    int sa;
  };
  auto load = [&](Step& st, int s) {
    const bool on = s < s1;
    const __amdgpu_buffer_rsrc_t r = make_rsrc(wq + (int64_t)s * p.RU * 64, on ? (uint32_t)p.RU * 64u : 0u);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(ws + (int64_t)s * p.RU * 4, on ? (uint32_t)p.RU * 4u : 0u);
#pragma unroll
    for (int i = 0; i < 4; ++i) st.a[i] = __builtin_amdgcn_raw_buffer_load_b128(r, lane * 16 + block(i) * 1024, 0, 0);
    st.sa = (int)__builtin_amdgcn_raw_buffer_load_b32(rs, (block(G) * 16 + c) * 4, 0, 0);
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int k = s * 128 + (X8 ? 64 * (u >> 1) + 16 * G + 8 * (u & 1) : 32 * G + 8 * u);
      st.b[u] = on && k < p.H ? *(const i32x4*)(x + k) : i32x4{0, 0, 0, 0};
    }
  };
  f32x4 acc[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) acc[i] = f32x4{0.f, 0.f, 0.f, 0.f};
  Step st;
  load(st, s0);
  for (int s = s0; s < s1; ++s) {
    const int sa = transpose_scales(st.sa, lane);
    int sb;
    const i32x8 b = quantize_operand<X8>(st.b, lane, sb);
    static_for<0, 4>([&](auto I) {
      constexpr int i = decltype(I)::value;
      const i32x8 a = {st.a[i][0], st.a[i][1], st.a[i][2], st.a[i][3], 0, 0, 0, 0};
      acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[i], 4, X8 ? 0 : 4, i, sa, 0, sb);
    });
    load(st, s + 1);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) sums[wave][i][lane] = acc[i];
  __syncthreads();
  if (wave < 4) {  // wave i: fragment i
    f32x4 v = sums[0][wave][lane];
#pragma unroll
    for (int w = 1; w < UW; ++w) {
      const f32x4 o = sums[w][wave][lane];
#pragma unroll
      for (int r = 0; r < 4; ++r) v[r] += o[r];
    }
    sums[0][wave][lane] = v;
  }
  __syncthreads();
  if (wave != 0) return;
  // Lane: columns 4 G .. + 3 of both halves of the group of 32, of pair c.
  uint32_t v[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const f32x4 g = sums[0][i][lane], u = sums[0][2 + i][lane];
    float h[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) h[r] = activation<ACT>(g[r]) * u[r];
    v[2 * i] = pack_bf16(h[0], h[1]);
    v[2 * i + 1] = pack_bf16(h[2], h[3]);
  }
  uint32_t m = bf16_amax_bits(v);
  m = max(m, (uint32_t)__shfl_xor((int)m, 16, 64));
  m = max(m, (uint32_t)__shfl_xor((int)m, 32, 64));
  const uint32_t sc = X8 ? scale_code_from_exponent(m >> 7) : fp4_scale_code(m >> 7);
  if (c >= count) return;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int col = n0 + 16 * i + 4 * G;
    if constexpr (X8) {
      const uint32_t code = e4m3_encode4_bf16(v[2 * i], v[2 * i + 1], sc);
      *(uint32_t*)(p.hq + (int64_t)column * p.hpitch_q + col) = real ? code : 0u;
    } else {
      const uint32_t code = e2m1_encode4_bf16(v[2 * i], v[2 * i + 1], sc);
      *(uint16_t*)(p.hq + (int64_t)column * p.hpitch_q + col / 2) = (uint16_t)(real ? code : 0u);
    }
  }
  if (G == 0) p.hs[(int64_t)column * p.hpitch_s + n0 / 32] = (uint8_t)(real ? sc : 0u);
}

// ---------------------------------------------------------------------------
// Down.

constexpr int DW = 8;     // waves
constexpr int DEPTH = 4;  // steps in flight a wave

template <bool X8>
__global__ __launch_bounds__(64 * DW, 4) void few_down_kernel(FewParams p) {
  __shared__ int32_t id[kPairs], lowest[kMaxExperts];
  __shared__ float weight[kPairs];
  __shared__ int32_t expert[kPairs];            // of a slot
  __shared__ int32_t pair_of[kPairs][kTokens];  // a token's first pair of the slot's expert, or -1
  __shared__ float weight_of[kPairs][kTokens];
  __shared__ int32_t slots[2];
  __shared__ f32x4 sums[DW][64];
  const int t = threadIdx.x, lane = t & 63;
  const int wave = __builtin_amdgcn_readfirstlane(t >> 6);
  const int n0 = 16 * (int)xcd_order(blockIdx.x, gridDim.x), P = p.T * p.k;

  // Slots: the experts in use in the order of their first pairs.
  int e = -1;
  if (t < P) {
    e = p.ids[t];
    weight[t] = p.weights[t];
    if (e >= p.E) e = -1;
    id[t] = e;
    if (e >= 0) lowest[e] = kPairs;
  }
  for (int i = t; i < kPairs * kTokens; i += 64 * DW) (&pair_of[0][0])[i] = -1;
  __syncthreads();
  if (e >= 0) atomicMin(&lowest[e], t);
  __syncthreads();
  const bool first = e >= 0 && lowest[e] == t;
  const uint64_t flags = __ballot(first);
  if (t < kPairs && lane == 0) slots[wave] = __builtin_popcountll(flags);
  __syncthreads();
  int slot = -1;
  if (first) {
    slot = __builtin_popcountll(flags & ((uint64_t(1) << lane) - 1)) + (wave == 1 ? slots[0] : 0);
    expert[slot] = e;
  }
  __syncthreads();
  if (first) lowest[e] = slot;  // from here on: the expert's slot
  __syncthreads();
  if (e >= 0) {
    const int tok = t / p.k;
    bool again = false;
    float w = 0.f;
    for (int j = tok * p.k; j < (tok + 1) * p.k; ++j)
      if (id[j] == e) {
        if (j < t) again = true;
        w += weight[j];
      }
    if (!again) {
      pair_of[lowest[e]][tok] = t;
      weight_of[lowest[e]][tok] = w;
    }
  }
  __syncthreads();

  const int S = (int)fp4_slabs(p.I), N = (slots[0] + slots[1]) * S;
  const int i0 = wave * N / DW, i1 = (wave + 1) * N / DW;
  const int c = lane & 15, G = lane >> 4;
  struct Step {
    i32x4 a, b[X8 ? 2 : 1];
    int sa, sb;
  };
  // The next step to load: slot lu, slab ls. Columns without a pair of the expert take
  // row 0; their products are not added.
  int li = i0, lu = N > 0 ? i0 / S : 0, ls = i0 - lu * S, ex = 0, row = 0;
  auto slot_of = [&]() {
    if (li < i1) {
      ex = __builtin_amdgcn_readfirstlane(expert[lu]);
      row = max(pair_of[lu][c], 0);
    }
  };
  auto load = [&](Step& st) {
    const bool on = li < i1;
    const int64_t slab = (int64_t)ex * S + ls;
    const __amdgpu_buffer_rsrc_t ra = make_rsrc(p.down_q + (slab * p.RD + n0) * 64, on ? 1024u : 0u);
    const __amdgpu_buffer_rsrc_t rs = make_rsrc(p.down_s + (slab * p.RD + n0) * 4, on ? 64u : 0u);
    const __amdgpu_buffer_rsrc_t rb = make_rsrc(p.hq, on ? (uint32_t)P * p.hpitch_q : 0u);
    const __amdgpu_buffer_rsrc_t rt = make_rsrc(p.hs, on ? (uint32_t)P * p.hpitch_s : 0u);
    st.a = __builtin_amdgcn_raw_buffer_load_b128(ra, lane * 16, 0, 0);
    st.sa = (int)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rs, c * 4 + G, 0, 0);
    const uint32_t at = (uint32_t)row * p.hpitch_q + (uint32_t)ls * (X8 ? 128u : 64u) + 16u * G;
    st.b[0] = __builtin_amdgcn_raw_buffer_load_b128(rb, at, 0, 0);
    if constexpr (X8) st.b[1] = __builtin_amdgcn_raw_buffer_load_b128(rb, at + 64u, 0, 0);
    st.sb = (int)(uint8_t)__builtin_amdgcn_raw_buffer_load_b8(rt, (uint32_t)row * p.hpitch_s + 4u * ls + G, 0, 0);
    ++li;
    if (++ls == S) {
      ls = 0;
      ++lu;
      slot_of();
    }
  };
  slot_of();
  f32x4 acc = {0.f, 0.f, 0.f, 0.f}, total = {0.f, 0.f, 0.f, 0.f};
  auto add = [&](int u) {  // the slot's product so far to the tokens' sums
    const bool has = pair_of[u][c] >= 0;
    const float w = weight_of[u][c];
#pragma unroll
    for (int r = 0; r < 4; ++r) total[r] = has ? __builtin_fmaf(w, acc[r], total[r]) : total[r];
    acc = f32x4{0.f, 0.f, 0.f, 0.f};
  };
  Step st[DEPTH];
  int u = lu, left = S - ls;  // the slot being computed, and its steps left
#pragma unroll
  for (int d = 0; d < DEPTH; ++d) load(st[d]);
  for (int i = i0; i < i1; i += DEPTH) {
#pragma unroll
    for (int d = 0; d < DEPTH; ++d) {
      if (i + d < i1) {
        if (left == 0) {
          add(u++);
          left = S;
        }
        --left;
        const Step& q = st[d];
        const i32x8 a = {q.a[0], q.a[1], q.a[2], q.a[3], 0, 0, 0, 0};
        i32x8 b = {q.b[0][0], q.b[0][1], q.b[0][2], q.b[0][3], 0, 0, 0, 0};
        if constexpr (X8) {
          b[4] = q.b[1][0];
          b[5] = q.b[1][1];
          b[6] = q.b[1][2];
          b[7] = q.b[1][3];
        }
        acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc, 4, X8 ? 0 : 4, 0, q.sa, 0, q.sb);
      }
      load(st[d]);
    }
  }
  if (i0 < i1) add(u);
  sums[wave][lane] = total;
  __syncthreads();
  if (wave != 0 || c >= p.T) return;
  f32x4 v = sums[0][lane];
#pragma unroll
  for (int w = 1; w < DW; ++w) {
    const f32x4 o = sums[w][lane];
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r] += o[r];
  }
  *(i32x2*)(p.y + (int64_t)c * p.H + n0 + 4 * G) = i32x2{(int)pack_bf16(v[0], v[1]), (int)pack_bf16(v[2], v[3])};
}

template <bool X8>
hipError_t run(FewParams p, int gate, hipStream_t st) {
  p.tiles_n = (int)(4 * fp4_slabs(p.I));
  const dim3 up((unsigned)(p.T * p.k * p.tiles_n));
  if (gate == 1)
    hipLaunchKernelGGL((few_up_kernel<X8, 1>), up, dim3(64 * UW), 0, st, p);
  else
    hipLaunchKernelGGL((few_up_kernel<X8, 0>), up, dim3(64 * UW), 0, st, p);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(few_down_kernel<X8>, dim3((unsigned)(p.H / 16)), dim3(64 * DW), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_experts_few(const FewParams& p, bool fp8, int gate, hipStream_t stream) {
  return fp8 ? run<true>(p, gate, stream) : run<false>(p, gate, stream);
}

}  // namespace mx

// Routing of tokens to experts: scores, choice of k experts within the best
// groups, weights.
//
//   l = logits, NaN as -inf, +inf as the largest f32
//   s = softmax(l) or 1 / (1 + exp(-l)), 0 where l = -inf
//   c = l, or with a bias f32(s + bias) with s in f64 (-inf where l is or c is NaN)
//   groups: the best by their highest c (with a bias by the f32 sum of their two
//           highest, one of -inf adding nothing) stay, the others' c becomes -inf
//   the k highest c, ties to the lower index; w = s (0 where c = -inf), divided by
//   their sum if asked, times a factor
//
// A choice next to a tie is decided by its last bits, so scores that decide are
// computed in f64 and rounded once; without a bias the order of the scores is that
// of the logits and no score of a loser is computed at all (but for the sum of an
// unnormalised softmax, in f32). Weights are computed in f64 for the k chosen.
//
// A team of L = 16 lanes (64 from 257 experts on) takes a token, expert i L + l
// in lane l, so a wave takes four tokens and its maxima need four DPP steps. A round
// of the choice is a maximum of order-preserving integer keys over the lanes' own
// best, a minimum of the indices that have it, and a new scan by the lane that won.
#include "mx_fp4_device.h"
#include "mx_internal.h"

namespace mx {
namespace {

constexpr int kWaves = 4;
constexpr uint32_t kNone = 0;                 // taken, or no such expert
constexpr uint32_t kMasked = 0x007FFFFFu;     // key of -inf
constexpr float kF32Max = 3.4028234663852886e38f;

// Keys in the order of the floats, above kNone; -0 is +0.
__device__ __forceinline__ uint32_t key_of(float c) {
  const uint32_t b = __float_as_uint(c + 0.0f);
  return b ^ ((b >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
__device__ __forceinline__ float value_of(uint32_t key) {
  return __uint_as_float(key ^ ((key >> 31) ? 0x80000000u : 0xFFFFFFFFu));
}

template <int CTRL>
__device__ __forceinline__ uint32_t dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
constexpr int kHalfMirror = 0x141, kMirror = 0x140;  // lanes 7 - l, and 15 - l, of a row of 16

template <int L>
__device__ __forceinline__ uint32_t team_max(uint32_t v) {
  v = max(v, dpp<kQuadXor1>(v));
  v = max(v, dpp<kQuadXor2>(v));
  v = max(v, dpp<kHalfMirror>(v));
  v = max(v, dpp<kMirror>(v));
  if constexpr (L == 64) {
    v = max(v, (uint32_t)__shfl_xor((int)v, 16, 64));
    v = max(v, (uint32_t)__shfl_xor((int)v, 32, 64));
  }
  return v;
}
template <int L>
__device__ __forceinline__ uint32_t team_min(uint32_t v) {
  return ~team_max<L>(~v);
}
template <int L, typename F>
__device__ __forceinline__ F team_sum(F v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ float logit(const RouteArgs& p, int64_t t, int e) {
  float l;
  if (p.f32)
    l = ((const float*)p.logits)[t * p.ld + e];
  else
    l = __uint_as_float((uint32_t)((const uint16_t*)p.logits)[t * p.ld + e] << 16);
  return l != l ? -__builtin_inff() : fminf(l, kF32Max);
}

template <int L, int NE>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs p) {
  constexpr int TEAMS = 64 / L, KS = 64 / L;  // tokens a wave; outputs (and groups) a lane
  __shared__ uint32_t table[kWaves][TEAMS][L * NE];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, team = lane / L, l = lane % L;
  const int64_t token = ((int64_t)blockIdx.x * kWaves + wave) * TEAMS + team;
  const int64_t t = token < p.T ? token : p.T - 1;  // the last waves repeat the last token
  const int E = p.E, k = p.k;

  float v[NE];
  uint32_t key[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) v[i] = i * L + l < E ? logit(p, t, i * L + l) : -__builtin_inff();

  // Softmax: the largest logit, and the sum where it is needed.
  const bool softmax = p.scores == 0;
  double top = 0.0, sum = 1.0;
  if (softmax) {
    uint32_t m = kNone;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = max(m, key_of(v[i]));
    const float f = value_of(team_max<L>(m));
    const bool any = f > -__builtin_inff();
    top = any ? (double)f : 0.0;
    if (p.bias != nullptr) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i) sum += exp((double)v[i] - top);
      sum = team_sum<L>(sum);
    } else if (!p.renorm) {
      float s = 0.f;
#pragma unroll
      for (int i = 0; i < NE; ++i) s += __builtin_amdgcn_exp2f((v[i] - (float)top) * 1.4426950408889634f);
      sum = (double)team_sum<L>(s);
    }
    if (!any) sum = 1.0;
  }
  auto score = [&](float x) {
    return softmax ? exp((double)x - top) / sum : 1.0 / (1.0 + exp(-(double)x));
  };
#pragma unroll
  for (int i = 0; i < NE; ++i) {
    const int e = i * L + l;
    float c = v[i];
    if (p.bias != nullptr && e < E && c > -__builtin_inff()) {
      c = (float)(score(c) + (double)p.bias[e]);
      if (c != c) c = -__builtin_inff();
    }
    key[i] = e < E ? key_of(c) : kNone;
  }

  if (p.groups > 1) {
    const int size = E / p.groups;
    uint32_t* tab = table[wave][team];
#pragma unroll
    for (int i = 0; i < NE; ++i) tab[i * L + l] = key[i];
    __syncthreads();
    uint32_t group[KS];
#pragma unroll
    for (int s = 0; s < KS; ++s) {
      group[s] = kNone;
      const int g = s * L + l;
      if (g < p.groups) {
        uint32_t b1 = kMasked, b2 = kMasked;
        int at = l % size;  // lanes start at different banks
        for (int i = 0; i < size; ++i) {
          const uint32_t x = tab[g * size + at];
          at = at + 1 == size ? 0 : at + 1;
          b2 = max(b2, min(b1, x));
          b1 = max(b1, x);
        }
        float c = value_of(b1);
        if (p.bias != nullptr && b2 > kMasked) c += value_of(b2);
        group[s] = c != c ? kMasked : key_of(c);
      }
    }
    uint64_t kept = 0;
    for (int r = 0; r < p.top_groups; ++r) {
      uint32_t b = kNone;
#pragma unroll
      for (int s = 0; s < KS; ++s) b = max(b, group[s]);
      b = team_max<L>(b);
      uint32_t at = 0xFFFFFFFFu;
#pragma unroll
      for (int s = KS - 1; s >= 0; --s)
        if (group[s] == b) at = (uint32_t)(s * L + l);
      at = team_min<L>(at);
      kept |= uint64_t(1) << at;
#pragma unroll
      for (int s = 0; s < KS; ++s)
        if (at == (uint32_t)(s * L + l)) group[s] = kNone;
    }
#pragma unroll
    for (int i = 0; i < NE; ++i) {
      const int e = i * L + l;
      if (e < E && !((kept >> (e / size)) & 1)) key[i] = kMasked;
    }
  }

  // The choice. Output j is kept by lane j % L.
  uint32_t best, at;
  auto scan = [&]() {
    best = kNone;
    at = 0xFFFFFFFFu;
#pragma unroll
    for (int i = 0; i < NE; ++i)
      if (key[i] > best) {
        best = key[i];
        at = (uint32_t)(i * L + l);
      }
  };
  scan();
  uint32_t chosen[KS], with[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) chosen[s] = with[s] = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t b = team_max<L>(best);
    const uint32_t e = team_min<L>(best == b ? at : 0xFFFFFFFFu);
#pragma unroll
    for (int s = 0; s < KS; ++s)
      if (s * L + l == j) {
        chosen[s] = e;
        with[s] = b;
      }
    if (at == e) {
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if ((uint32_t)(i * L + l) == e) key[i] = kNone;
      scan();
    }
  }

  double w[KS], total = 0.0;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const bool live = s * L + l < k && with[s] > kMasked;
    w[s] = live ? score(logit(p, t, (int)chosen[s])) : 0.0;
    total += w[s];
  }
  if (p.renorm) {
    total = team_sum<L>(total);
#pragma unroll
    for (int s = 0; s < KS; ++s) w[s] = total > 0.0 ? w[s] / total : 0.0;
  }
  if (token >= p.T) return;
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int j = s * L + l;
    if (j < k) {
      p.ids[t * k + j] = (int32_t)chosen[s];
      p.weights[t * k + j] = (float)(w[s] * p.factor);
    }
  }
}

template <int L, int NE>
hipError_t launch(const RouteArgs& p, hipStream_t st) {
  const int64_t per_block = (int64_t)kWaves * (64 / L);
  hipLaunchKernelGGL((route_kernel<L, NE>), dim3((unsigned)((p.T + per_block - 1) / per_block)), dim3(64 * kWaves), 0, st, p);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_route(const RouteArgs& p, hipStream_t stream) {
  if (p.E <= 64) return launch<16, 4>(p, stream);
  if (p.E <= 128) return launch<16, 8>(p, stream);
  if (p.E <= 256) return launch<16, 16>(p, stream);
  if (p.E <= 512) return launch<64, 8>(p, stream);
  return launch<64, 16>(p, stream);
}

}  // namespace mx

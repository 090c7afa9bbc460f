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
// computed in f64 (to 2^-42; see Exp2) and rounded once; without a bias the order
// of the scores is that of the logits and no score of a loser is computed at all (but
// for the sum of an unnormalised softmax). Weights are computed in f64 for the k chosen.
//
// A team of L = 16 lanes (64 from 257 experts on) takes a token, lane l experts l NE ..
// + NE - 1, so a wave takes four tokens and its maxima need four DPP steps. A lane sorts
// its keys (order-preserving integers) once; a round of the choice is a maximum over the
// lanes' first ones, which the lowest lane that has it takes out. Which expert of the lane
// it was is looked up at the end.
//
// A few tokens take a launch's time. Many are bound by vector operations, 1470 a wave:
// 32001 tokens x 256 experts, k = 8 of 4 out of 8 groups, sigmoid with a bias, 26 us; a
// renormalised softmax, k = 8, where logits decide, 16, an unnormalised one 19; the logits
// alone would take 7.
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
template <int L, typename F>
__device__ __forceinline__ F team_sum(F v) {
#pragma unroll
  for (int off = 1; off < L; off <<= 1) v += __shfl_xor(v, off, 64);
  return v;
}

__device__ __forceinline__ float sane(float l) { return l != l ? -__builtin_inff() : fminf(l, kF32Max); }
__device__ __forceinline__ float logit(const RouteArgs& p, int64_t t, int e) {
  if (p.f32) return sane(((const float*)p.logits)[t * p.ld + e]);
  return sane(__uint_as_float((uint32_t)((const uint16_t*)p.logits)[t * p.ld + e] << 16));
}

// 2^t for t <= 1000 to 2^-44: 2^round(t) times 1 + f q(f) of the rest f, |f| <= 1/2,
// where q interpolates (2^f - 1) / f in the nine Chebyshev nodes (2^0 is 1 exactly).
// Below f64's range the result is 0. The coefficients stay in scalar registers: left to
// itself the compiler moves each constant anew before each use.
struct Exp2 {
  double k[10] = {1.0,
                  0x1.62e42fefa39efp-1,
                  0x1.ebfbdff823cedp-3,
                  0x1.c6b08d7047e52p-5,
                  0x1.3b2ab7181b755p-7,
                  0x1.5d87fe86fe88ep-10,
                  0x1.4308ac85aa947p-13,
                  0x1.ffcb9515a8016p-17,
                  0x1.63d136366db24p-20,
                  0x1.b63880a30e9ffp-24};
  __device__ __forceinline__ Exp2() {
#pragma unroll
    for (int i = 0; i < 10; ++i) asm volatile("" : "+s"(k[i]));
  }
  __device__ __forceinline__ double operator()(double t) const {
    const double n = __builtin_rint(t), f = t - n;
    double r = k[9];
#pragma unroll
    for (int i = 8; i >= 0; --i) r = __builtin_fma(r, f, k[i]);
    return __builtin_amdgcn_ldexp(r, (int)n);
  }
};
constexpr double kLog2e = 1.44269504088896340736;

// 1 / d for d in [1, 2^1001): the hardware's estimate (off by 2^-24.3 at most, measured)
// and a Newton step.
__device__ __forceinline__ double fast_reciprocal(double d) {
  const double r = __builtin_amdgcn_rcp(d);
  return __builtin_fma(__builtin_fma(-d, r, 1.0), r, r);
}

// Falling order (Batcher's odd-even merges of runs of 1, 2, 4, ...).
template <int N>
__device__ __forceinline__ void sort_falling(uint32_t (&a)[N]) {
#pragma unroll
  for (int run = 1; run < N; run *= 2)
#pragma unroll
    for (int d = run; d >= 1; d /= 2)
#pragma unroll
      for (int i = d % run; i + d < N; i += 2 * d)
#pragma unroll
        for (int u = i; u < i + d; ++u)
          if (u + d < N && u / (2 * run) == (u + d) / (2 * run)) {
            const uint32_t x = a[u], y = a[u + d];
            a[u] = max(x, y);
            a[u + d] = min(x, y);
          }
}

template <int L, int NE>
__global__ __launch_bounds__(64 * kWaves) void route_kernel(RouteArgs p) {
  constexpr int TEAMS = 64 / L, KS = 64 / L;  // tokens a wave; outputs (and groups) a lane
  __shared__ __attribute__((aligned(16))) uint32_t table[kWaves][TEAMS][L * NE];  // keys
  __shared__ uint2 taken[kWaves][TEAMS][64];                                      // the choice: key; lane, rank
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, team = lane / L, l = lane % L;
  const int64_t token = ((int64_t)blockIdx.x * kWaves + wave) * TEAMS + team;
  const int64_t t = token < p.T ? token : p.T - 1;  // the last waves repeat the last token
  const int E = p.E, k = p.k, e0 = l * NE;

  float v[NE];
  uint32_t key[NE];
  if (p.vector) {  // rows of whole, aligned 16-byte pieces
#pragma unroll
    for (int i = 0; i < NE; i += 4) {
      float f[4] = {0.f, 0.f, 0.f, 0.f};
      if (e0 + i < E) {
        if (p.f32) {
          const f32x4 q = *(const f32x4*)((const float*)p.logits + t * p.ld + e0 + i);
#pragma unroll
          for (int u = 0; u < 4; ++u) f[u] = q[u];
        } else {
          const i32x2 q = *(const i32x2*)((const uint16_t*)p.logits + t * p.ld + e0 + i);
#pragma unroll
          for (int u = 0; u < 4; ++u)
            f[u] = __uint_as_float((u & 1) ? (uint32_t)q[u >> 1] & 0xFFFF0000u : (uint32_t)q[u >> 1] << 16);
        }
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) v[i + u] = e0 + i < E ? sane(f[u]) : -__builtin_inff();
    }
  } else {
#pragma unroll
    for (int i = 0; i < NE; ++i) v[i] = e0 + i < E ? logit(p, t, e0 + i) : -__builtin_inff();
  }

  // Softmax: the largest logit, and the sum where it is needed.
  const bool softmax = p.scores == 0;
  double top = 0.0, sum = 1.0;
  const Exp2 exp2_of;
  if (softmax) {
    uint32_t m = kNone;
#pragma unroll
    for (int i = 0; i < NE; ++i) m = max(m, key_of(v[i]));
    const float f = value_of(team_max<L>(m));
    const bool any = f > -__builtin_inff();
    top = any ? (double)f : 0.0;
    if (p.bias != nullptr || !p.renorm) {
      sum = 0.0;
#pragma unroll
      for (int i = 0; i < NE; ++i)
        sum += exp2_of(fmax(((double)v[i] - top) * kLog2e, -2000.0));
      sum = team_sum<L>(sum);
    }
    if (!any) sum = 1.0;
  }
  if (p.bias != nullptr) {
    float bias[NE];
    if (p.vector_bias) {
#pragma unroll
      for (int i = 0; i < NE; i += 4) {
        const f32x4 q = *(const f32x4*)(p.bias + (e0 + i < E ? e0 + i : 0));
#pragma unroll
        for (int u = 0; u < 4; ++u) bias[i + u] = q[u];
      }
    } else {
#pragma unroll
      for (int i = 0; i < NE; ++i) bias[i] = p.bias[e0 + i < E ? e0 + i : 0];
    }
    // (Masked logits give a score of 0 here and their own key.)
    auto take = [&](int i, double s) {
      const float c = (float)(s + (double)bias[i]);
      v[i] = v[i] > -__builtin_inff() && c == c ? c : -__builtin_inff();
    };
    if (softmax) {
      const double scale = 1.0 / sum;
#pragma unroll
      for (int i = 0; i < NE; ++i) take(i, exp2_of(fmax(((double)v[i] - top) * kLog2e, -2000.0)) * scale);
    } else {
      // Past +-690 the score is 1, or vanishes in f32.
#pragma unroll
      for (int i = 0; i < NE; ++i)
        take(i, fast_reciprocal(1.0 + exp2_of((double)__builtin_amdgcn_fmed3f(v[i], -690.f, 690.f) * -kLog2e)));
    }
  }
#pragma unroll
  for (int i = 0; i < NE; ++i) key[i] = e0 + i < E ? key_of(v[i]) : kNone;

  // A lane's keys in falling order: the choice takes them from the front. Where each
  // comes from is looked up at the end, in the table.
  uint32_t sorted[NE];
#pragma unroll
  for (int i = 0; i < NE; ++i) sorted[i] = key[i];
  if (p.groups > 1) {
    const int size = E / p.groups;
    auto score_of = [&](uint32_t b1, uint32_t b2) {
      float c = value_of(b1);
      if (p.bias != nullptr && b2 > kMasked) c += value_of(b2);
      return c != c ? kMasked : key_of(c);
    };
    // A round takes the best group that is left, the lowest of equal ones.
    if (size >= NE && size % NE == 0 && ((size / NE) & (size / NE - 1)) == 0) {
      // Groups of 1, 2, 4, ... whole lanes: the two highest by lane, then across them.
      const int lanes = size / NE;
      sort_falling(sorted);
      uint32_t b1 = max(kMasked, sorted[0]), b2 = max(kMasked, sorted[1]);
      for (int off = 1; off < lanes; off <<= 1) {
        const uint32_t o1 = (uint32_t)__shfl_xor((int)b1, off, 64), o2 = (uint32_t)__shfl_xor((int)b2, off, 64);
        b2 = max(min(b1, o1), max(b2, o2));
        b1 = max(b1, o1);
      }
      uint32_t group = e0 < E ? score_of(b1, b2) : kNone;  // of the lane's group
      const uint32_t mine = (uint32_t)(l / lanes);
      bool kept = false;
      for (int r = 0; r < p.top_groups; ++r) {
        const uint32_t b = team_max<L>(group);
        const uint64_t has = __ballot(group == b) >> (team * L);
        if ((uint32_t)__builtin_ctzll(has) / (uint32_t)lanes == mine) {
          kept = true;
          group = kNone;
        }
      }
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (e0 < E && !kept) key[i] = sorted[i] = kMasked;
    } else {
      uint32_t* tab = table[wave][team];
#pragma unroll
      for (int i = 0; i < NE; ++i) tab[e0 + i] = key[i];
      __syncthreads();
      uint32_t group[KS];  // of groups s L + l
#pragma unroll
      for (int s = 0; s < KS; ++s) {
        group[s] = kNone;
        const int g = s * L + l;
        if (g < p.groups) {
          uint32_t b1 = kMasked, b2 = kMasked;
#pragma unroll 4
          for (int i = 0; i < size; ++i) {
            const uint32_t x = tab[g * size + i];
            b2 = max(b2, min(b1, x));
            b1 = max(b1, x);
          }
          group[s] = score_of(b1, b2);
        }
      }
      uint64_t kept = 0;
      for (int r = 0; r < p.top_groups; ++r) {
        uint32_t b = kNone;
#pragma unroll
        for (int s = 0; s < KS; ++s) b = max(b, group[s]);
        b = team_max<L>(b);
        int at = -1;
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          const uint64_t has = (__ballot(group[s] == b) >> (team * L)) & (L == 64 ? ~uint64_t(0) : (uint64_t(1) << (L & 63)) - 1);
          if (at < 0 && has != 0) at = s * L + __builtin_ctzll(has);
        }
        kept |= uint64_t(1) << at;
#pragma unroll
        for (int s = 0; s < KS; ++s)
          if (at == s * L + l) group[s] = kNone;
      }
#pragma unroll
      for (int i = 0; i < NE; ++i)
        if (e0 + i < E && !((kept >> ((e0 + i) / size)) & 1)) key[i] = kMasked;
      __syncthreads();  // the table is written again below
#pragma unroll
      for (int i = 0; i < NE; ++i) sorted[i] = key[i];
      sort_falling(sorted);
    }
  } else {
    sort_falling(sorted);
  }

  // The choice: output j is the rank-th of its lane's experts with that key.
  uint2* out = taken[wave][team];
  uint32_t before = kNone, rank = 0;
  for (int j = 0; j < k; ++j) {
    const uint32_t b = team_max<L>(sorted[0]);
    const uint64_t has = __ballot(sorted[0] == b) >> (team * L);
    if (l == (int)__builtin_ctzll(has)) {
      rank = b == before ? rank + 1 : 0;
      before = b;
      out[j] = uint2{b, (uint32_t)l | rank << 8};
#pragma unroll
      for (int i = 0; i + 1 < NE; ++i) sorted[i] = sorted[i + 1];
      sorted[NE - 1] = kNone;
    }
  }
  uint32_t* tab = table[wave][team];
#pragma unroll
  for (int i = 0; i < NE; i += 4)
    *(i32x4*)(tab + e0 + i) = i32x4{(int)key[i], (int)key[i + 1], (int)key[i + 2], (int)key[i + 3]};
  __syncthreads();

  // Output s L + l in this lane.
  double w[KS], total = 0.0;
  uint32_t chosen[KS];
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    const int j = s * L + l;
    chosen[s] = 0x80000000u;
    w[s] = 0.0;
    if (j < k) {
      const uint2 o = out[j];
      const int first = (int)(o.y & 0xFF) * NE;
      uint32_t same = 0;  // the lane's experts with this key
#pragma unroll
      for (int i = NE - 4; i >= 0; i -= 4) {
        const i32x4 q = *(const i32x4*)(tab + first + i);
#pragma unroll
        for (int u = 3; u >= 0; --u) same = 2 * same + ((uint32_t)q[u] == o.x ? 1u : 0u);
      }
      for (uint32_t n = o.y >> 8; n > 0; --n) same &= same - 1;
      chosen[s] = (uint32_t)(first + __builtin_ctz(same)) | (o.x > kMasked ? 0u : 0x80000000u);
    }
    if (!(chosen[s] >> 31)) {
      const double x = (double)logit(p, t, (int)chosen[s]);
      w[s] = softmax ? exp(x - top) / sum : 1.0 / (1.0 + exp(-x));
    }
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
      p.ids[t * k + j] = (int32_t)(chosen[s] & 0x7FFFFFFFu);
      p.weights[t * k + j] = (float)(w[s] * p.factor);
    }
  }
}

// A launch has fewer than 2^32 threads: 2^26 tokens of 64 lanes each take two.
template <int L, int NE>
hipError_t launch(RouteArgs p, hipStream_t st) {
  constexpr int64_t per_block = (int64_t)kWaves * (64 / L), most = (int64_t(1) << 23) * per_block;
  for (int64_t left = p.T; left > 0; left -= p.T) {
    p.T = left < most ? left : most;
    hipLaunchKernelGGL((route_kernel<L, NE>), dim3((unsigned)((p.T + per_block - 1) / per_block)), dim3(64 * kWaves), 0, st, p);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
    p.logits = (const uint8_t*)p.logits + p.T * p.ld * (p.f32 ? 4 : 2);
    p.ids += p.T * p.k;
    p.weights += p.T * p.k;
  }
  return hipSuccess;
}

}  // namespace

hipError_t launch_route(const RouteArgs& a, hipStream_t stream) {
  RouteArgs p = a;
  const int es = p.f32 ? 4 : 2;
  p.vector_bias = p.E % 4 == 0 && (uintptr_t)p.bias % 16 == 0;
  p.vector = p.E % 4 == 0 && (p.ld * es) % (4 * es) == 0 && (uintptr_t)p.logits % (uintptr_t)(4 * es) == 0;
  if (p.E <= 64) return launch<16, 4>(p, stream);
  if (p.E <= 128) return launch<16, 8>(p, stream);
  if (p.E <= 256) return launch<16, 16>(p, stream);
  if (p.E <= 512) return launch<64, 8>(p, stream);
  return launch<64, 16>(p, stream);
}

}  // namespace mx

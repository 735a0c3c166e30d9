// Experts chosen by scores: sigmoid or softmax of the logits, a bias that takes
// part in the choice alone, groups of experts of which the best few stay, top-k,
// weights from the unbiased scores.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,  c_e = s_e + b_e
//   group value: the largest c of the group, or the sum of its two largest
//   the k largest c of the groups that stay; w = scale * s (/ sum of the k s)
//
// The choice is that of c in 64 bits: adding a bias to a score near 1 in float32
// drops the score's last bits and would decide some tokens by the rounding. 64-bit
// scores of every expert cost several times what the logits' bytes do, so the row
// kernel finds candidates in float32, with a bound on how far its values may be off,
// and decides among these in 64 bits. The few tokens where the bound does not rule the
// other experts or groups out (ties, mostly) are chosen in 64 bits altogether.
#include <type_traits>

#include "moe_kernels.h"
#include "moe_row.h"

namespace moe {
namespace sel {

constexpr int kThreads = 256;
constexpr int kWaves = kThreads / 64;

struct Args {
  float* logits;        // [T, E]; with parts, the first of them, and the sums are stored here
  const float* part;    // [nparts][T, E] more partial sums, or NULL
  int nparts;
  const float* lbias;   // [E] added to the logits' sums, or NULL
  const float* bias;    // [E] added to the scores for the choice, or NULL
  int T, E, k, score, n_group, topk_group, rule, renormalize;
  float scale;
  int32_t* idx;
  float* w;
};

// Logits first + i step of a row for i < n (at most N; the others come back NaN),
// summed over their parts (in order, then the bias) and stored where there are any.
template <int N>
__device__ __forceinline__ void logits_of(const Args& a, int64_t row, int first, int step, int n, float (&l)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) l[i] = i < n ? a.logits[row + first + i * step] : NAN;
  if (a.part == nullptr) return;
  const int64_t stride = int64_t(a.T) * a.E;
#pragma unroll 1
  for (int z = 0; z < a.nparts; ++z) {
    float p[N];
#pragma unroll
    for (int i = 0; i < N; ++i) p[i] = i < n ? a.part[z * stride + row + first + i * step] : 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i) l[i] += p[i];
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (i < n) {
      if (a.lbias != nullptr) l[i] += a.lbias[first + i * step];
      a.logits[row + first + i * step] = l[i];
    }
}

// ---------------------------------------------------------------------------
// Reductions without LDS: DPP steps inside rows of 16 lanes (swap neighbours, swap
// pairs, mirror the halves of 8, mirror the 16), on every lane of the row. A lane that is
// switched off hands out 0, so every lane of the wave takes them: never behind a && or a ?:
// whose condition differs between lanes.
// ---------------------------------------------------------------------------
template <int CTRL>
__device__ __forceinline__ uint32_t peer(uint32_t v) {
  return uint32_t(__builtin_amdgcn_update_dpp(0, int(v), CTRL, 0xF, 0xF, false));
}
template <int CTRL>
__device__ __forceinline__ float peer(float v) { return __uint_as_float(peer<CTRL>(__float_as_uint(v))); }
template <int CTRL>
__device__ __forceinline__ double peer(double v) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(peer<CTRL>(uint32_t(u))) | (uint64_t(peer<CTRL>(uint32_t(u >> 32))) << 32));
}
// over LANES (1, 2, 4, 8, 16) neighbouring lanes
template <int LANES, typename T, typename Op>
__device__ __forceinline__ T over(T v, Op op) {
  if constexpr (LANES > 1) v = op(v, peer<0xB1>(v));
  if constexpr (LANES > 2) v = op(v, peer<0x4E>(v));
  if constexpr (LANES > 4) v = op(v, peer<0x141>(v));
  if constexpr (LANES > 8) v = op(v, peer<0x140>(v));
  return v;
}
struct Max {
  __device__ __forceinline__ float operator()(float a, float b) const { return fmaxf(a, b); }
  __device__ __forceinline__ double operator()(double a, double b) const { return fmax(a, b); }
  __device__ __forceinline__ uint32_t operator()(uint32_t a, uint32_t b) const { return max(a, b); }
};
struct Min {
  __device__ __forceinline__ float operator()(float a, float b) const { return fminf(a, b); }
};
struct Add {
  template <typename T>
  __device__ __forceinline__ T operator()(T a, T b) const { return a + b; }
};
__device__ __forceinline__ double lane64(double v, int lane) {
  const uint64_t u = __builtin_bit_cast(uint64_t, v);
  return __builtin_bit_cast(double, uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u), lane))) |
                                        (uint64_t(uint32_t(__builtin_amdgcn_readlane(int(u >> 32), lane))) << 32));
}
template <typename Op>
__device__ __forceinline__ double wave64(double v, Op op) {
  v = over<16>(v, op);
  return op(op(lane64(v, 0), lane64(v, 16)), op(lane64(v, 32), lane64(v, 48)));
}

// ---------------------------------------------------------------------------
// Scores in 64 bits
// ---------------------------------------------------------------------------
// exp(l - m), 1 where the two are equal (both infinite), for a softmax's numerator and
// far sigmoids; else the sigmoid of l. (One copy of the exponential's code: most of the
// time of few tokens goes into fetching instructions.)
__device__ __forceinline__ double score64(bool below, float l, float m) {
  const double e = exp(below ? double(l) - double(m) : -double(l));
  return below ? (l == m ? 1.0 : e) : 1.0 / (1.0 + e);
}
__device__ __forceinline__ double ranked(double c) { return c == c ? c : -INFINITY; }

// ---------------------------------------------------------------------------
// One token by a whole wave, in 64 bits. Loops instead of registers: it is rarely
// run, and then its instructions come from memory.
// ---------------------------------------------------------------------------
template <int EPL>
struct Exact {
  double c[64 * EPL];  // choice values
  float l[64 * EPL];   // logits (in)
};
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// The choice values, the largest logit and a softmax's denominator; returns the groups
// that stay.
template <int EPL>
__device__ __forceinline__ uint64_t exact_groups(const Args& a, Exact<EPL>& s, float& m, double& den) {
  const int lane = lane_id();
  float lm = -INFINITY;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) lm = fmaxf(lm, s.l[e]);  // (drops NaN)
  m = wave_max_dpp(lm);
  double z = 0.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float l = s.l[e];
    const double v = l == l ? score64(a.score == 0, l, m) : 0.0;
    s.c[e] = v;
    z += v;
  }
  den = a.score == 0 ? wave64(z, Add()) : 1.0;
#pragma unroll 1
  for (int e = lane; e < a.E; e += 64) {
    const float l = s.l[e];
    double v = s.c[e];
    if (a.score == 0) v /= den;
    if (a.bias != nullptr) v += double(a.bias[e]);
    s.c[e] = l == l ? ranked(v) : -INFINITY;
  }
  wave_sync();
  if (a.topk_group == a.n_group) return ~0ull;
  const int per = a.E / a.n_group;
  double v = -INFINITY;
  if (lane < a.n_group) {
    double b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll 1
    for (int i0 = 0; i0 < per; i0 += 8) {
      double x[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) x[u] = i0 + u < per ? s.c[lane * per + i0 + u] : -INFINITY;
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        b2 = fmax(b2, fmin(b1, x[u]));
        b1 = fmax(b1, x[u]);
      }
    }
    v = ranked(a.rule == 0 || per == 1 ? b1 : b1 + b2);
  }
  int rank = 0;
#pragma unroll 1
  for (int g = 0; g < a.n_group; ++g) {
    const double o = lane64(v, g);
    rank += o > v || (o == v && g < lane);
  }
  return __ballot(lane < a.n_group && rank < a.topk_group);
}

template <int EPL>
__device__ __forceinline__ void choose_exact(const Args& a, Exact<EPL>& s, int t) {
  const int lane = lane_id();
  const int per = a.E / a.n_group;
  double den;
  float m;
  const uint64_t keep = exact_groups<EPL>(a, s, m, den);
  // a bit for each expert lane + 64 i that can still be taken
  uint32_t live = 0;
#pragma unroll 1
  for (int i = 0; lane + 64 * i < a.E; ++i) live |= uint32_t((keep >> ((lane + 64 * i) / per)) & 1) << i;
  int my_e = 0;
#pragma unroll 1
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    uint32_t be = 0x7FFFFFFFu;  // the lane's first expert with its largest value
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if ((live >> i) & 1u) {
        const double x = s.c[lane + 64 * i];
        if (be == 0x7FFFFFFFu || x > bv) {
          bv = x;
          be = uint32_t(lane + 64 * i);
        }
      }
    const double top = wave64(bv, Max());
    // the lowest of the lanes' (each a different expert)
    uint32_t e = bv == top ? be : 0x7FFFFFFFu;
    e = over<16>(e, [](uint32_t x, uint32_t y) { return min(x, y); });
    const uint32_t e0 = __builtin_amdgcn_readlane(e, 0), e1 = __builtin_amdgcn_readlane(e, 16),
                   e2 = __builtin_amdgcn_readlane(e, 32), e3 = __builtin_amdgcn_readlane(e, 48);
    e = min(min(e0, e1), min(e2, e3));
    if (be == e) live &= ~(1u << (e >> 6));
    if (lane == j) my_e = int(e);
  }
  const bool mine = lane < a.k;
  float ml = mine ? s.l[my_e] : -INFINITY;
  ml = ml == ml ? ml : -INFINITY;
  // (renormalised sigmoids far below 0 without their common factor: none underflows; all of
  // them at -infinity have none)
  const float top = wave_max_dpp(ml);
  const bool far = a.score != 0 && a.renormalize && top < -600.f && top > -INFINITY;
  const double v = mine ? score64(a.score == 0 || far, ml, far ? top : m) : 0.0;
  if (a.renormalize) den = wave64(v, Add());
  if (mine) {
    a.idx[int64_t(t) * a.k + lane] = my_e;
    a.w[int64_t(t) * a.k + lane] = m == -INFINITY ? NAN : float(v / den * double(a.scale));
  }
  wave_sync();
}

// Any sizes: a wave per token.
template <int EPL>
__global__ void __launch_bounds__(kThreads) wave_kernel(Args a) {
  __shared__ Exact<EPL> s[kWaves];
  const int wv = threadIdx.x >> 6;
  const int64_t token = int64_t(blockIdx.x) * kWaves + wv;
  if (token >= a.T) return;
  const int t = int(token);
  float l[EPL];
  logits_of<EPL>(a, int64_t(t) * a.E, lane_id(), 64, (a.E - lane_id() + 63) / 64, l);
#pragma unroll
  for (int i = 0; i < EPL; ++i) s[wv].l[lane_id() + 64 * i] = l[i];
  choose_exact<EPL>(a, s[wv], t);
}

// ---------------------------------------------------------------------------
// Four tokens per wave, 16 lanes each
// ---------------------------------------------------------------------------
// Float32 values find k + 2 candidates per token, one for each lane, and 64-bit
// values of these alone decide. A value's 32-bit key has the order of floats in its
// upper 24 (23 for more than 256 slots) bits and the slot below, so keys differ and a maximum of keys names its
// holder; the lanes' keys are sorted once and the candidates leave the heads of 16
// lists.
//
// Group g has L = 16 / (groups, up to a power of 2) lanes, each with q <= Q experts in
// a row: lane r of the row holds experts (r / L) per + (r % L) q + i in slots N r + i, N 16
// or 32.
struct Map {
  int log_l, q, per;
};

template <uint32_t MASK>
__device__ __forceinline__ uint32_t key_of(float f, int slot) {
  const uint32_t u = __float_as_uint(f);
  return ((u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u)) & ~MASK) | (MASK - uint32_t(slot));
}
// (-infinity, as any value whose bits a key cannot keep, comes back NaN)
template <uint32_t MASK>
__device__ __forceinline__ float value_of(uint32_t key) {
  key &= ~MASK;
  return __uint_as_float(key ^ (uint32_t(int32_t(~key) >> 31) | 0x80000000u));
}

// Descending order (odd-even merges).
template <int N>
__device__ __forceinline__ void sort_keys(uint32_t (&k)[N]) {
#pragma unroll
  for (int p = 1; p < N; p *= 2)
#pragma unroll
    for (int h = p; h >= 1; h /= 2)
#pragma unroll
      for (int j = h % p; j + h < N; j += 2 * h)
#pragma unroll
        for (int i = 0; i < h; ++i)
          if (i + j + h < N && (i + j) / (2 * p) == (i + j + h) / (2 * p)) {
            const uint32_t a = k[i + j], b = k[i + j + h];
            k[i + j] = max(a, b);
            k[i + j + h] = min(a, b);
          }
}

// Lanes of the row with a value above v (the own one's not counted).
template <int D = 1>
__device__ __forceinline__ int above(float v) {
  if constexpr (D == 16)
    return 0;
  else
    return int(peer<0x120 + D>(v) > v) + above<D + 1>(v);  // the lane D places round the row
}
// Lanes of the row that come before this one: a larger value, or the same and a lower
// expert.
template <int D = 1>
__device__ __forceinline__ int before(double v, uint32_t e) {
  if constexpr (D == 16) {
    return 0;
  } else {
    const double o = peer<0x120 + D>(v);
    const uint32_t oe = peer<0x120 + D>(e);
    return int(o > v || (o == v && oe < e)) + before<D + 1>(v, e);
  }
}

// exp(x), off by a step of float32 and by 1.22 x 2^-24 of |x|
__device__ __forceinline__ float exp_quick(float x) { return __builtin_amdgcn_exp2f(x * 1.44269504f); }
// exp(l - m), off by a step and a half: what its argument's roundings lose is put back.
__device__ __forceinline__ float exp_between(float l, float m) {
  const float d = l - m, b = d - l;
  const float lost = (l - (d - b)) - (m + b);  // l - m = d + lost
  const float x = d * 1.44269504f;
  const float rest = fmaf(d, 1.44269504f, -x) + fmaf(d, 1.92596299e-8f, lost * 1.44269504f);
  const float e = __builtin_amdgcn_exp2f(x);
  return e > 0.f ? fmaf(e, rest * 0.693147181f, e) : e;
}

// Q: slots of a lane; KM: most k. VEC: E = 16 Q in whole lanes, rows 16-byte aligned
// (8 for Q = 2).
template <int Q, int KM, bool VEC>
__global__ void __launch_bounds__(kThreads) row_kernel(Args a, Map map) {
  constexpr int EPL = Q < 4 ? 1 : Q / 4;
  constexpr int kPitch = Q + 1;  // (a lane's logits at odd distance: no bank twice)
  constexpr int N = Q > 16 ? 32 : 16;
  constexpr uint32_t MASK = 16 * N - 1;
  __shared__ Exact<EPL> s_exact[kWaves];
  __shared__ float s_l[kWaves][4][16 * kPitch];
  const int lane = lane_id(), r = lane & 15, row4 = lane >> 4, wv = threadIdx.x >> 6;
  const int64_t first_token = 4 * (int64_t(blockIdx.x) * kWaves + wv);
  if (first_token >= a.T) return;
  const int t0 = int(first_token);
  const bool here = first_token + row4 < a.T;
  const int t = here ? t0 + row4 : a.T - 1;  // (rows past the end repeat the last token and write nothing)
  const int64_t row = int64_t(t) * a.E;
  const int L = 1 << map.log_l;
  const int g = r >> map.log_l;  // the lane's group
  const int in_g = (r & (L - 1)) * map.q;
  const int first = g * map.per + in_g;
  const int n = VEC ? Q : g < a.n_group ? min(map.q, map.per - in_g) : 0;  // its experts (below 1: none)
  float l[Q], b[Q];
  auto load = [&](const float* from, float (&v)[Q]) {
    if constexpr (Q >= 4) {
#pragma unroll
      for (int i = 0; i < Q / 4; ++i) {
        const float4 f = reinterpret_cast<const float4*>(from)[i];
        v[4 * i] = f.x; v[4 * i + 1] = f.y; v[4 * i + 2] = f.z; v[4 * i + 3] = f.w;
      }
    } else {
      const float2 f = *reinterpret_cast<const float2*>(from);
      v[0] = f.x; v[1] = f.y;
    }
  };
  if constexpr (VEC) {
    float* p = a.logits + row + Q * r;
    load(p, l);
    if (a.part != nullptr) {
      const int64_t stride = int64_t(a.T) * a.E;
      for (int z0 = 0; z0 < a.nparts; z0 += 4) {
        float pv[4][Q];
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (z0 + u < a.nparts) load(a.part + (z0 + u) * stride + row + Q * r, pv[u]);
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (z0 + u < a.nparts)
#pragma unroll
            for (int i = 0; i < Q; ++i) l[i] += pv[u][i];
      }
      if (a.lbias != nullptr)
#pragma unroll
        for (int i = 0; i < Q; ++i) l[i] += a.lbias[Q * r + i];
      if (here)
#pragma unroll
        for (int i = 0; i < Q; ++i) p[i] = l[i];
    }
  } else {
    logits_of<Q>(a, row, first, 1, here || a.part == nullptr ? n : 0, l);
  }
  if (a.bias != nullptr) {
    const float* p = a.bias + first;
    if (VEC && (reinterpret_cast<uintptr_t>(a.bias) & 15u) == 0) {
      load(p, b);
    } else {  // the bias may sit at any float address
#pragma unroll
      for (int i = 0; i < Q; ++i) b[i] = i < n ? p[i] : 0.f;
    }
  }
  // logits of the wave's token `which` for exact_groups and choose_exact
  auto hand_over = [&](int which) {
#pragma unroll 1
    for (int e = lane; e < a.E; e += 64) {
      const int eg = e / map.per, in = e - eg * map.per, el = in / map.q;
      s_exact[wv].l[e] = s_l[wv][which][kPitch * ((eg << map.log_l) + el) + in - el * map.q];
    }
  };
  // (maxima drop NaN, which counts as -infinity)
  float lm = -INFINITY;
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    s_l[wv][row4][kPitch * r + i] = l[i];
    lm = fmaxf(lm, l[i]);
  }
  const float m = over<16>(lm, Max());
  // Values to choose by. Where the scores' order is the softmax logits' (no bias,
  // groups by their best), the logits themselves.
  const bool groups = a.topk_group < a.n_group;
  const bool by_logit = a.score == 0 && a.bias == nullptr && (!groups || a.rule == 0);
  double den = 1.0;
  float rden = 1.f;
  float c[Q];
  if (a.score == 0) {
    if (by_logit && a.renormalize) {
#pragma unroll
      for (int i = 0; i < Q; ++i) c[i] = l[i];
    } else {
      if (a.renormalize) {
        float z[Q];
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          c[i] = exp_quick(l[i] - m);
          z[i] = fmaxf(c[i], 0.f);
        }
#pragma unroll
        for (int h = Q / 2; h >= 1; h /= 2)
#pragma unroll
          for (int i = 0; i < h; ++i) z[i] += z[i + h];
        den = over<16>(z[0], Add());
      } else {
        // The weights are divided by it: a sum in 64 bits (16384 tokens, 256 experts: 8.1 -> 9.1
        // us; in 32 bits of exp_quick the weights were up to 15 x 2^-24 off, now 4).
        double z = 0.0;
#pragma unroll
        for (int i = 0; i < Q; ++i) {
          c[i] = exp_between(l[i], m);
          z += double(fmaxf(c[i], 0.f));
        }
        den = over<16>(z, Add());
      }
      rden = __builtin_amdgcn_rcpf(float(den));
#pragma unroll
      for (int i = 0; i < Q; ++i) c[i] = by_logit ? l[i] : c[i] * rden;
    }
  } else {
#pragma unroll
    for (int i = 0; i < Q; ++i) c[i] = __builtin_amdgcn_rcpf(1.f + exp_quick(-l[i]));
  }
  // How far a float32 score may be from the 64-bit one, as a part of the row's largest. A
  // sigmoid's: the exponential is a step (2^-23) off, and its argument's rounding and the
  // constant's are 1.22 x 2^-24 of |l|, all times 1 - s; the sum rounds by 2^-24, the
  // reciprocal by a step. Below 0 that is (5 + 1.22 |l|) x 2^-24 of the score, at the most
  // for the largest one; where that is above 0, 1 - s keeps all within 4 x 2^-24. A
  // softmax's: 22 x 2^-24 from the denominator (terms that are 10.6 x 2^-24 off on average at
  // the most, for 512 experts, added 9 deep; its reciprocal), which scales the whole row alike,
  // and 4 x 2^-24 of its own: the difference of two sums of two is at most 4 x 2^-20 off.
  const float s_max = a.score == 0 ? rden : __builtin_amdgcn_rcpf(1.f + exp_quick(-m));
  const float s_off =
      by_logit ? 0.f : s_max * (a.score == 0 ? 0x1p-20f : fmaf(fmaxf(-m, 0.f), 0x1.4p-24f, 0x1.4p-22f));
  // Logits up to this apart may have the same score in 64 bits, and then the lower id
  // comes first: their distances to the largest, below 600 where they count, round to
  // 2^-43 (and exponentials and quotients merge what is 2^-51 apart).
  constexpr float kSame = 0x1p-42f;
  // (scores without all their bits; infinite maxima, which the differences do not bear)
  bool unsure = !(s_max >= 0x1p-100f) || !(fabsf(m) < INFINITY);
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < Q; ++i) c[i] += b[i];
  }
  uint32_t key[Q];
#pragma unroll
  for (int i = 0; i < Q; ++i) {
    c[i] = VEC || i < n ? fmaxf(c[i], -INFINITY) : -INFINITY;
    key[i] = VEC || i < n ? key_of<MASK>(c[i], N * r + i) : 0u;
  }
  if (groups) {
    float b1 = -INFINITY, b2 = -INFINITY;
#pragma unroll
    for (int i = 0; i < Q; ++i) {
      b2 = fmaxf(b2, fminf(b1, c[i]));
      b1 = fmaxf(b1, c[i]);
    }
    auto join = [&](float o1, float o2) {
      b2 = fmaxf(fminf(b1, o1), fmaxf(b2, o2));
      b1 = fmaxf(b1, o1);
    };
    if (L > 1) join(peer<0xB1>(b1), peer<0xB1>(b2));
    if (L > 2) join(peer<0x4E>(b1), peer<0x4E>(b2));
    if (L > 4) join(peer<0x141>(b1), peer<0x141>(b2));
    const bool real = g < a.n_group;
    float v = a.rule == 0 || map.per == 1 ? b1 : b1 + b2;
    v = real && v == v ? v : -INFINITY;
    const int higher = above(v);
    bool kept = real && higher < (a.topk_group << map.log_l);
    const float lo = over<16>(kept ? v : INFINITY, Min()), hi = over<16>(real && !kept ? v : -INFINITY, Max());
    const int lanes = __popc(uint32_t(__ballot(kept) >> (16 * row4)) & 0xFFFFu);
    // Up to two scores on both sides, and on each side a rounding of 2^-24 of a value for
    // each bias and of up to two values for the sum: 2^-22 of the largest. Equal values keep
    // more groups, and values at -infinity differ by no number.
    // (lanes without a group hold -infinity and count for nothing)
    const float most = fmaxf(fabsf(b1), a.rule == 0 || map.per == 1 || !(b2 > -INFINITY) ? 0.f : fabsf(b2));
    const float size = over<16>(real ? most : 0.f, Max());
    const bool border = lanes != (a.topk_group << map.log_l) || !(lo - hi > (by_logit ? kSame : 4.f * s_off + size * 0x1p-21f));
    // such tokens' groups in 64 bits, by the whole wave
    wave_sync();
    for (uint64_t todo = __ballot(border && r == 0); todo != 0; todo &= todo - 1) {
      const int which = (__ffsll((unsigned long long)todo) - 1) >> 4;
      float me;
      double de;
      hand_over(which);
      const uint64_t keep = exact_groups<EPL>(a, s_exact[wv], me, de);
      if (row4 == which) kept = real && ((keep >> g) & 1);
    }
    if (!kept)
#pragma unroll
      for (int i = 0; i < Q; ++i) key[i] = 0;
  }
  sort_keys(key);
  // Two candidates more than asked for, as long as there are lanes: with one, a token or
  // two of 16384 (256 experts) have the next one within what a key drops, and a wave that
  // chooses altogether in 64 bits takes 3 to 6 us more.
  uint32_t mine = 0;
  const int cand = min(a.k + 2, 16);
#pragma unroll
  for (int j = 0; j < (KM < 16 ? KM + 2 : 16); ++j) {
    if (j < cand) {
      const uint32_t top = over<16>(key[0], Max());
      if (r == j) mine = top;
      uint32_t pop = key[0] == top ? ~0u : 0u;
      asm("" : "+v"(pop));  // (one mask, instead of a comparison for each of its uses)
#pragma unroll
      for (int i = 0; i + 1 < Q && i < KM + 2 - j; ++i) key[i] = (key[i + 1] & pop) | (key[i] & ~pop);
      if (Q < KM + 3 - j) key[Q - 1] &= ~pop;
    }
  }
  const uint32_t next = over<16>(key[0], Max());

  // The candidates' 64-bit values: the scores are without a softmax's denominator
  // where it changes no order.
  wave_sync();
  const bool is = mine != 0;  // (experts may be fewer)
  const int slot = int(MASK - (mine & MASK)), lr = is ? slot / N : 0, si = is ? slot % N : 0;
  const uint32_t e = is ? uint32_t((lr >> map.log_l) * map.per + (lr & (L - 1)) * map.q + si) : 0x7FFFFFFFu;
  const float ml = s_l[wv][row4][kPitch * lr + si];
  const bool none = !is || !(ml == ml);
  double s = 0.0, v = -INFINITY;
  if (!none) {
    s = score64(a.score == 0, ml, m);
    v = by_logit ? double(ml) : a.score == 0 ? s * double(rden) : s;
    if (a.bias != nullptr) v = ranked(v + double(a.bias[e]));
  }
  // The candidates come in the order of their keys, which is that of their values but
  // for neighbours within what a key drops.
  const double ahead = peer<0x121>(v);  // of the candidate before (lane 0: the last one's)
  // Beside a bias a softmax's float32 denominator may be what orders neighbours: those
  // tokens' denominators in 64 bits, by the whole wave.
  if (a.score == 0 && a.bias != nullptr) {
    const uint64_t close = __ballot(is && r > 0 && !(ahead - v > 2.0 * double(s_off)));
#pragma unroll 1
    for (int which = 0; which < 4; ++which) {
      if (((close >> (16 * which)) & 0xFFFFu) == 0) continue;
      const float mw = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(m), 16 * which));
      double z = 0.0;
#pragma unroll
      for (int i = 0; i < (16 * kPitch + 63) / 64; ++i) {
        const int at = lane + 64 * i;  // (the gaps between the lanes' logits aside)
        const float x = at < 16 * kPitch && at % kPitch < Q ? s_l[wv][which][at] : NAN;
        z += x == x ? score64(true, x, mw) : 0.0;
      }
      z = wave64(z, Add());
      if (row4 == which && !none) v = ranked(s / z + double(a.bias[e]));
    }
  }
  // (infinite values, whose difference is no number, among those that are never sure)
  if (by_logit) unsure = unsure || ((__ballot(is && r > 0 && ahead != v && !(fabs(ahead - v) > kSame)) >> (16 * row4)) & 0xFFFFu) != 0;
  int rank = r;
  const bool in_order = peer<0x121>(v) > v;
  if (__ballot(is && r > 0 && !in_order) != 0) rank = before(v, e);
  const bool chosen = is && rank < a.k;
  // No expert beside the candidates may come before the last chosen one: their values
  // lie at most the MASK steps that a key drops above the next key's.
  const double least = over<16>(chosen ? v : INFINITY, [](double x, double y) { return fmin(x, y); });
  const float limit = value_of<MASK>(next);
  unsure = unsure || (next != 0 && !(least > double(limit) + double(fabsf(limit) * (N == 16 ? 0x1p-14f : 0x1p-13f) + 2.f * s_off + kSame)));
  // softmax scores so far below the largest that they are equal, sigmoids whose sum
  // would lose bits, and NaN logits, which come behind those at -infinity
  const float low = over<16>(!chosen ? INFINITY : none ? -INFINITY : ml, Min());
  unsure = unsure || !((a.score == 0 ? low - m : low) > -600.f);
  const double sum = a.renormalize ? over<16>(chosen ? s : 0.0, Add()) : den;
  if (chosen && here && !unsure) {
    a.idx[int64_t(t) * a.k + rank] = int(e);
    a.w[int64_t(t) * a.k + rank] = float(s / sum * double(a.scale));
  }
  for (uint64_t todo = __ballot(unsure && here && r == 0); todo != 0; todo &= todo - 1) {
    const int which = (__ffsll((unsigned long long)todo) - 1) >> 4;
    hand_over(which);
    choose_exact<EPL>(a, s_exact[wv], t0 + which);
  }
}

}  // namespace sel

hipError_t launch_select(float* logits, const float* part, int nparts, const float* logit_bias, const float* bias, int T,
                         int E, int k, const Choice& c, int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  using namespace sel;
  // (groups that all stay are none)
  const bool groups = c.topk_group < c.n_group;
  const Args a{logits, part, nparts, logit_bias, bias, T, E, k, c.score, groups ? c.n_group : 1,
               groups ? c.topk_group : 1, c.group_rule, c.renormalize, c.scale, topk_idx, topk_w};
  // Four tokens per wave where 16 lanes of at most 32 experts hold a token's, a group
  // in lanes of its own (16384 tokens, 256 experts in 8 groups: a wave per token 50 us).
  int log_g = 0;
  while ((1 << log_g) < a.n_group) ++log_g;
  if (log_g <= 4 && k <= 16) {
    const int per = E / a.n_group, L = 16 >> log_g, q = (per + L - 1) / L;
    const Map map{4 - log_g, q, per};
    auto row = [&](auto q_t, auto vec_t) {
      constexpr int Q = decltype(q_t)::value;
      constexpr bool VEC = decltype(vec_t)::value;
      const dim3 grid(unsigned(ceil_div(T, 4 * kWaves)));
      auto* kern = k <= 8 ? row_kernel<Q, 8, VEC> : row_kernel<Q, 16, VEC>;
      hipLaunchKernelGGL(kern, grid, dim3(kThreads), 0, stream, a, map);
      return hipGetLastError();
    };
    typedef std::integral_constant<int, 2> Q2;
    typedef std::integral_constant<int, 4> Q4;
    typedef std::integral_constant<int, 8> Q8;
    typedef std::integral_constant<int, 16> Q16;
    typedef std::integral_constant<int, 32> Q32;
    const uintptr_t at = reinterpret_cast<uintptr_t>(logits) | reinterpret_cast<uintptr_t>(part);
    if (E == 16 * q && per == L * q && (at & (q == 2 ? 7u : 15u)) == 0) {
      if (q == 2) return row(Q2{}, std::true_type{});
      if (q == 4) return row(Q4{}, std::true_type{});
      if (q == 8) return row(Q8{}, std::true_type{});
      if (q == 16) return row(Q16{}, std::true_type{});
      if (q == 32) return row(Q32{}, std::true_type{});
    }
    if (q <= 4) return row(Q4{}, std::false_type{});
    if (q <= 8) return row(Q8{}, std::false_type{});
    if (q <= 16) return row(Q16{}, std::false_type{});
    if (q <= 32) return row(Q32{}, std::false_type{});
  }
  const dim3 grid(unsigned(ceil_div(T, kWaves)));
  auto wave = [&](auto epl) {
    hipLaunchKernelGGL(wave_kernel<decltype(epl)::value>, grid, dim3(kThreads), 0, stream, a);
    return hipGetLastError();
  };
  if (E <= 64) return wave(std::integral_constant<int, 1>{});
  if (E <= 128) return wave(std::integral_constant<int, 2>{});
  if (E <= 256) return wave(std::integral_constant<int, 4>{});
  if (E <= 512) return wave(std::integral_constant<int, 8>{});
  return wave(std::integral_constant<int, 16>{});
}

}  // namespace moe

// Experts chosen by scores: sigmoid or softmax of the logits, a bias that takes
// part in the choice alone, groups of experts of which the best few stay, top-k,
// weights from the unbiased scores.
//
//   s_e = sigmoid(l_e) or softmax(l)_e,  c_e = s_e + b_e
//   group value: the largest c of the group, or the sum of its two largest
//   the k largest c of the groups that stay; w = scale * s (/ sum of the k s)
//
// The choice is made on c in 64 bits. Adding a bias to a score near 1 in float32
// would drop the score's last bits and decide some tokens by the rounding.
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

// The logit of expert e, summed over its parts and stored where there are any
// (each by the lane that goes on with it).
__device__ __forceinline__ float logit(const Args& a, int64_t row, int e) {
  float l = a.logits[row + e];
  if (a.part != nullptr) {
    const int64_t stride = int64_t(a.T) * a.E;
    for (int z = 0; z < a.nparts; ++z) l += a.part[z * stride + row + e];
    if (a.lbias != nullptr) l += a.lbias[e];
    a.logits[row + e] = l;
  }
  return l;
}

__device__ __forceinline__ double wave_sum64(double v) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v += __shfl_xor(v, m, 64);
  return v;
}

// exp(l - m), 1 where the two are equal (both infinite)
__device__ __forceinline__ double exp_below(float l, float m) { return l == m ? 1.0 : exp(double(l) - double(m)); }

__device__ __forceinline__ double sigmoid64(float l) { return 1.0 / (1.0 + exp(-double(l))); }

__device__ __forceinline__ double ranked(double c) { return c == c ? c : -INFINITY; }

// One wave per token, expert lane + 64 i in slot i.
template <int EPL>
__global__ void __launch_bounds__(kThreads) select_kernel(Args a) {
  __shared__ double s_c[kWaves][64 * EPL];
  __shared__ float s_l[kWaves][64 * EPL];
  const int lane = lane_id(), wv = threadIdx.x >> 6;
  const int t = blockIdx.x * kWaves + wv;
  if (t >= a.T) return;
  const int64_t row = int64_t(t) * a.E;
  float l[EPL];
  float lm = -INFINITY;
  uint32_t nan = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    l[i] = e < a.E ? logit(a, row, e) : NAN;
    nan |= uint32_t(l[i] != l[i]) << i;
    l[i] = l[i] == l[i] ? l[i] : -INFINITY;
    if (e < a.E) s_l[wv][e] = l[i];
    lm = fmaxf(lm, l[i]);
  }
  const float m = wave_max(lm);
  double den = 1.0;
  if (a.score == 0) {
    double z = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (lane + 64 * i < a.E) z += exp_below(l[i], m);
    den = wave_sum64(z);
  }
  double c[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    c[i] = -INFINITY;
    if (e < a.E) {
      const double s = a.score == 0 ? exp_below(l[i], m) / den : sigmoid64(l[i]);
      c[i] = (nan >> i) & 1u ? -INFINITY : ranked(a.bias != nullptr ? s + double(a.bias[e]) : s);
      s_c[wv][e] = c[i];
    }
  }
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "workgroup");
  __builtin_amdgcn_wave_barrier();
  // groups that stay
  uint64_t keep = ~0ull;
  const int per = a.E / a.n_group;
  if (a.topk_group < a.n_group) {
    double v = -INFINITY;
    if (lane < a.n_group) {
      double b1 = -INFINITY, b2 = -INFINITY;
      for (int i = 0; i < per; ++i) {
        const double x = s_c[wv][lane * per + i];
        b2 = fmax(b2, fmin(b1, x));
        b1 = fmax(b1, x);
      }
      v = ranked(a.rule == 0 || per == 1 ? b1 : b1 + b2);
    }
    int rank = 0;
    for (int g = 0; g < a.n_group; ++g) {
      const double o = __shfl(v, g, 64);
      rank += o > v || (o == v && g < lane);
    }
    keep = __ballot(lane < a.n_group && rank < a.topk_group);
  }
  uint32_t live = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    if (e < a.E && ((keep >> (e / per)) & 1)) live |= 1u << i;
  }
  int my_e = 0;
  for (int j = 0; j < a.k; ++j) {
    double bv = -INFINITY;
    int be = 0x7FFFFFFF;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if ((live >> i) & 1u) {
        const int e = lane + 64 * i;
        if (be == 0x7FFFFFFF || c[i] > bv) {
          bv = c[i];
          be = e;
        }
      }
#pragma unroll
    for (int d = 32; d >= 1; d >>= 1) {
      const double ov = __shfl_xor(bv, d, 64);
      const int oe = __shfl_xor(be, d, 64);
      if (oe != 0x7FFFFFFF && (be == 0x7FFFFFFF || ov > bv || (ov == bv && oe < be))) {
        bv = ov;
        be = oe;
      }
    }
    if (lane == (be & 63)) live &= ~(1u << (be >> 6));
    if (lane == j) my_e = be;
  }
  // weights of the k chosen, from their logits. Renormalised sigmoids as
  // exp(min(l, 0) - shift) / (1 + exp(-|l|)): their common factor cannot
  // underflow.
  const bool mine = lane < a.k;
  const float ml = mine ? s_l[wv][my_e] : -INFINITY;
  double s;
  if (a.score == 0) {
    s = exp_below(ml, m);
  } else {
    const float top = a.renormalize ? fminf(wave_max(ml), 0.f) : 0.f;
    s = exp_below(fminf(ml, 0.f), top) / (1.0 + exp(-fabs(double(ml))));
  }
  if (a.renormalize) {
    double sum = 0.0;
    for (int j = 0; j < a.k; ++j) sum += __shfl(s, j, 64);
    den = sum;
  }
  if (mine) {
    a.idx[int64_t(t) * a.k + lane] = my_e;
    a.w[int64_t(t) * a.k + lane] = m == -INFINITY ? NAN : float(s / den * double(a.scale));
  }
}

}  // namespace sel

hipError_t launch_select(float* logits, const float* part, int nparts, const float* logit_bias, const float* bias, int T,
                         int E, int k, const Choice& c, int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  const sel::Args a{logits, part, nparts, logit_bias, bias, T, E, k, c.score, c.n_group, c.topk_group, c.group_rule,
                    c.renormalize, c.scale, topk_idx, topk_w};
  const dim3 grid(unsigned(ceil_div(T, sel::kWaves)));
  auto go = [&](auto epl) {
    hipLaunchKernelGGL(sel::select_kernel<decltype(epl)::value>, grid, dim3(sel::kThreads), 0, stream, a);
    return hipGetLastError();
  };
  if (E <= 64) return go(std::integral_constant<int, 1>{});
  if (E <= 128) return go(std::integral_constant<int, 2>{});
  if (E <= 256) return go(std::integral_constant<int, 4>{});
  if (E <= 512) return go(std::integral_constant<int, 8>{});
  return go(std::integral_constant<int, 16>{});
}

}  // namespace moe

// The whole share for a few tokens (at most 32) in two kernels.
//
//   y[t] = sum over local e in topk(t) of w[t, e] (silu(x[t] Wg_e) * (x[t] Wu_e)) Wd_e
//
// At a handful of tokens the used experts' weights are the whole cost (HBM),
// and the six launches of the general path cost more than reading them. Here
// few_logits_kernel scores the tokens and few_experts_kernel does the rest:
// every workgroup picks the tokens' experts for itself (a few thousand logits)
// and then takes items from one queue, first all gate/up items, then all down
// items:
//
//   gate/up item  (expert, k range, 64 outputs)   -> float32 partial sums; the
//                 last of an output panel's k ranges adds them in order and
//                 writes h = silu(g) * u
//   down item     (expert, k range, 128 outputs)  -> float32 partial sums; the
//                 last of an output panel's items adds them per token, slot by
//                 slot, and writes y
//
// An item's four waves share its k range and its 128 weight columns; a wave
// streams the weights into registers in the grouped GEMV's geometry
// (grouped_gemv.hip: 8 rows x 8 columns per lane and step, transposed in
// registers, v_mfma_f32_16x16x32_bf16 with the weights as the A operand) and
// the waves' sums meet in LDS. Two workgroups per CU, so that one streams
// while the other exchanges its sums. A down item asks for its weights before
// it waits for h.
//
// Waiting is safe however many workgroups run at a time and whatever else the
// GPU runs: items are handed out in order, a gate/up item waits for nothing,
// and a down item waits only for gate/up items, all of which were handed out
// before it to workgroups that are running.
//
// Sums are added in a fixed order by whichever workgroup is last, so y does
// not depend on the order of the items. h stays float32: it is multiplied as
// three bf16 parts that add up to it (exact products), so y is rounded once.
//
// What one workgroup writes for another (partial sums, h) goes through
// agent-scope atomic stores and loads, which pass the L2s of the eight XCDs;
// a counter is raised only after the stores before it have completed.
#include "gemm_dma.h"
#include "gemm_tile.h"
#include "moe_kernels.h"

#include <utility>

namespace moe {
namespace few {

using dma::panel::f32x4v;
using dma::panel::mfma16x16x32;
typedef __amdgpu_buffer_rsrc_t rsrc_t;

constexpr int kMaxE = 1024;
constexpr int kMaxSel = 1024;  // T k
constexpr int kThreads = 256, kWaves = 4;
constexpr int kSub = 512;       // k of a unit: 4 steps of 32 for each of the 4 waves
constexpr int kCols = 128;      // weight columns of an item
constexpr int kGateUp = 64;     // outputs of a gate/up item (gate and up columns)
constexpr int kStride = kCols + 4;
constexpr int kFewItems = 2048;  // items an operand is cut into where k allows (four per workgroup)
constexpr int kCoherent = 16;   // buffer cache policy sc1: agent scope
constexpr int kStream = 2;      // nt: each weight byte is read once
constexpr uint32_t kOutside = 0x80000000u;  // offset past every buffer: reads zero

struct Args {
  const uint16_t* x;
  const float* logits;
  const uint16_t* w_gate_up;
  const uint16_t* w_down;
  int T, H, I, E, k, e0, E_local, renormalize, y_f32;
  void* y;
  int* ticket;    // next item
  int* cnt_a;     // [expert][gate/up panel]: k ranges done
  int* cnt_h;     // [expert][512 of I]: panels of h written
  int* cnt_b;     // [down panel]: items done
  float* part_a;  // [row][k range][panel][128]
  float* part_b;  // [row][k range][H]
  float* h;       // [row][I]
};

// k ranges of an item: units of 512 per range, ranges. More experts, fewer
// ranges: their items alone keep the queue long.
struct Split {
  int units, ranges;
};
__host__ __device__ inline Split split(int K, int items) {
  const int u = (K + kSub - 1) / kSub;
  const int want = items >= kFewItems ? 1 : (kFewItems + items - 1) / items;
  const int units = want >= u ? 1 : (u + want - 1) / want;
  return {units, (u + units - 1) / units};
}

// ---------------------------------------------------------------------------
// Logits
// ---------------------------------------------------------------------------
// One workgroup per expert, float32 products and sums; TB >= T tokens at a
// time. Also clears the second kernel's counters.
template <int TB>
__global__ void __launch_bounds__(kThreads) few_logits_kernel(const uint16_t* x, const float* w, const float* bias,
                                                              int T, int H, int E, float* logits, int* counters,
                                                              int ncounters) {
  __shared__ float s[kWaves][TB];
  const int e = blockIdx.x;
  for (int i = e * kThreads + int(threadIdx.x); i < ncounters; i += int(gridDim.x) * kThreads) counters[i] = 0;
  float acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.f;
  for (int k = 4 * int(threadIdx.x); k < H; k += 4 * kThreads) {
    const float4 wv = *reinterpret_cast<const float4*>(w + int64_t(e) * H + k);
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      const uint2 xv = *reinterpret_cast<const uint2*>(x + int64_t(min(t, T - 1)) * H + k);
      acc[t] = fmaf(bf16_lo(xv.x), wv.x, acc[t]);
      acc[t] = fmaf(bf16_hi(xv.x), wv.y, acc[t]);
      acc[t] = fmaf(bf16_lo(xv.y), wv.z, acc[t]);
      acc[t] = fmaf(bf16_hi(xv.y), wv.w, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const float v = wave_sum(acc[t]);
    if (lane_id() == 0) s[threadIdx.x >> 6][t] = v;
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < T) logits[t * E + e] = s[0][t] + s[1][t] + s[2][t] + s[3][t] + (bias ? bias[e] : 0.f);
}

// ---------------------------------------------------------------------------
// Exchange between workgroups
// ---------------------------------------------------------------------------
__device__ __forceinline__ void put2(float* p, float a, float b) {
  const uint64_t v = uint64_t(__float_as_uint(a)) | (uint64_t(__float_as_uint(b)) << 32);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get2(const float* p) {
  const uint64_t v = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float(uint32_t(v)), __uint_as_float(uint32_t(v >> 32)));
}
// this wave's stores have reached the agent's point of coherence
__device__ __forceinline__ void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ int raise(int* c, int by) {
  return __hip_atomic_fetch_add(c, by, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---------------------------------------------------------------------------
// Selection, by every workgroup for itself
// ---------------------------------------------------------------------------
struct Tables {
  uint32_t mask[kMaxE];   // tokens that picked local expert e (T <= 32 bits)
  int row0[kMaxE];        // first row of local expert e
  int act[kMaxE];         // the local experts that have rows
  int16_t sel[kMaxSel];   // slot (t, j): local expert or -1
  float wt[kMaxSel];      // its weight
  uint8_t tok[kMaxSel];   // row: its token
};

// One wave per token: k rounds of the largest live logit, the lowest expert
// among equal ones; NQ registers per lane, expert l + 64 q.
template <int NQ>
__device__ __forceinline__ void pick(const Args& a, Tables& s, int t) {
  const int lane = lane_id();
  float v[NQ];
  uint32_t live = 0;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = lane + 64 * q;
    v[q] = -INFINITY;
    if (e < a.E) {
      const float f = a.logits[t * a.E + e];
      v[q] = f == f ? f : -INFINITY;
      live |= 1u << q;
    }
  }
  float top = 0.f, sum = 0.f, mine = 0.f;
  int my_e = -1;
  for (int j = 0; j < a.k; ++j) {
    float best = -INFINITY;
    int at = 1 << 30;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (((live >> q) & 1u) && (v[q] > best || at == 1 << 30)) {
        best = v[q];
        at = lane + 64 * q;
      }
    const float m = wave_max_dpp(best);
    uint64_t who = ballot(best == m && at != 1 << 30);
    int e = shfl(at, __builtin_ctzll(who));
    who &= who - 1;
    while (who) {
      e = min(e, shfl(at, __builtin_ctzll(who)));
      who &= who - 1;
    }
    if (e % 64 == lane) live &= ~(1u << (e / 64));
    if (j == 0) {
      top = m;
      if (!a.renormalize) {
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          if (lane + 64 * q < a.E) z += expf(v[q] - top);
        sum = wave_sum(z);
      }
    }
    const float p = expf(m - top);
    if (a.renormalize) sum += p;
    if (lane == j) {
      mine = p;
      my_e = e;
    }
  }
  if (lane < a.k) {
    const int e = my_e - a.e0;
    const bool local = e >= 0 && e < a.E_local;
    s.sel[t * a.k + lane] = int16_t(local ? e : -1);
    s.wt[t * a.k + lane] = mine / sum;
    if (local) atomicOr(&s.mask[e], 1u << t);
  }
}

// ---------------------------------------------------------------------------
// Items
// ---------------------------------------------------------------------------
__device__ __forceinline__ rsrc_t make_rsrc(const void* base, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(base), (short)0, int(bytes), 0x00020000);
}

// f(integral_constant<int, i>) for i = 0 .. N-1
template <typename F, int... I>
__device__ __forceinline__ void static_for_impl(F&& f, std::integer_sequence<int, I...>) {
  (f(std::integral_constant<int, I>{}), ...);
}
template <int N, typename F>
__device__ __forceinline__ void static_for(F&& f) {
  static_for_impl(f, std::make_integer_sequence<int, N>{});
}

// Sums over k range [unit0, unit0 + units) x 512 of an item's 128 columns for
// `rows` rows: acc[gi][c][v] of lane 16 g + m is column 8 (4 g + v) + c of row
// 16 gi + m (this wave's share of k). ready(): called once, after the first
// weights are asked for and before the first activations.
template <bool DOWN, int G, int D, typename Ready>
__device__ __forceinline__ void stream(const Args& a, const Tables& s, int e, int panel, int unit0, int units,
                                       int row0, int rows, f32x4v (&acc)[G][8], Ready ready) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), g = lane >> 4, m = lane & 15;
  const int K = DOWN ? a.I : a.H, ldw = DOWN ? a.H : 2 * a.I;
  uint32_t wvo;
  {
    int col;
    bool in;
    if (DOWN) {
      col = kCols * panel + 8 * m;
      in = col < a.H;
    } else {
      const int o = kGateUp * panel + 16 * (m >> 2) + 8 * (m & 1);
      in = o < a.I;
      col = (m & 2) ? a.I + o : o;
    }
    wvo = in ? uint32_t(8 * g * ldw + col) * 2u : kOutside;
  }
  const rsrc_t wr = make_rsrc((DOWN ? a.w_down : a.w_gate_up) + int64_t(e) * K * ldw, int64_t(K) * ldw * 2);
  // activations: x as it is (bf16), h as float32
  const rsrc_t xr = DOWN ? make_rsrc(a.h + int64_t(row0) * a.I, int64_t(rows) * a.I * 4)
                         : make_rsrc(a.x, int64_t(a.T) * a.H * 2);
  uint32_t xvo[G];
#pragma unroll
  for (int gi = 0; gi < G; ++gi) {
    const int r = 16 * gi + m;
    const uint32_t src = DOWN ? uint32_t(r) : uint32_t(s.tok[row0 + min(r, rows - 1)]);
    xvo[gi] = r < rows ? src * uint32_t(K) * (DOWN ? 4u : 2u) + uint32_t(g) * (DOWN ? 32u : 16u) : kOutside;
  }
  const int nsteps = 4 * units;
  const int kb = unit0 * kSub + 32 * w;  // step st covers k kb + 128 st .. + 31
  constexpr int XV = DOWN ? 2 : 1;
  u32x4 qw[D][8], qx[D][G][XV];
  // steps past the range, and rows past K, read zeros without touching memory
  auto in_k = [&](int st) { return st < nsteps && kb + 128 * st + 8 * g < K; };
  auto load_w = [&](auto d_t, int st) {
    constexpr int d = decltype(d_t)::value;
    const uint32_t vo = in_k(st) ? wvo : kOutside;
    const int so = st < nsteps && kb + 128 * st < K ? (kb + 128 * st) * ldw * 2 : 0;
#pragma unroll
    for (int r = 0; r < 8; ++r) qw[d][r] = __builtin_amdgcn_raw_buffer_load_b128(wr, vo, so + r * ldw * 2, kStream);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto load_x = [&](auto d_t, int st) {
    constexpr int d = decltype(d_t)::value;
    const int so = st < nsteps && kb + 128 * st < K ? (kb + 128 * st) * (DOWN ? 4 : 2) : 0;
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      const uint32_t vo = in_k(st) ? xvo[gi] : kOutside;
#pragma unroll
      for (int q = 0; q < XV; ++q)
        qx[d][gi][q] = __builtin_amdgcn_raw_buffer_load_b128(xr, vo + 16u * q, so, DOWN ? kCoherent : 0);
    }
    __builtin_amdgcn_sched_barrier(0);
  };
  auto consume = [&](auto d_t) {
    constexpr int d = decltype(d_t)::value;
    constexpr int P = DOWN ? 3 : 1;  // bf16 parts of an activation
    u32x4 xp[G][P];
#pragma unroll
    for (int gi = 0; gi < G; ++gi) {
      if constexpr (DOWN) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t hi[2], mid[2], lo[2];
#pragma unroll
          for (int b = 0; b < 2; ++b) {
            const int j = 2 * i + b;
            const float f = __uint_as_float(qx[d][gi][j >> 2][j & 3]);
            hi[b] = __float_as_uint(f) & 0xFFFF0000u;
            const float r1 = f - __uint_as_float(hi[b]);
            mid[b] = __float_as_uint(r1) & 0xFFFF0000u;
            lo[b] = __float_as_uint(r1 - __uint_as_float(mid[b]));
          }
          xp[gi][0][i] = __builtin_amdgcn_perm(hi[1], hi[0], 0x07060302u);
          xp[gi][1][i] = __builtin_amdgcn_perm(mid[1], mid[0], 0x07060302u);
          xp[gi][2][i] = __builtin_amdgcn_perm(lo[1], lo[0], 0x07060302u);
        }
      } else {
        xp[gi][0] = qx[d][gi][0];
      }
    }
#pragma unroll
    for (int c = 0; c < 8; ++c) {
      const uint32_t sel = (c & 1) ? 0x07060302u : 0x05040100u;
      u32x4 wv;
#pragma unroll
      for (int j = 0; j < 4; ++j) wv[j] = __builtin_amdgcn_perm(qw[d][2 * j + 1][c >> 1], qw[d][2 * j][c >> 1], sel);
#pragma unroll
      for (int p = P - 1; p >= 0; --p)
#pragma unroll
        for (int gi = 0; gi < G; ++gi) acc[gi][c] = mfma16x16x32(wv, xp[gi][p], acc[gi][c]);
    }
  };
#pragma unroll
  for (int gi = 0; gi < G; ++gi)
#pragma unroll
    for (int c = 0; c < 8; ++c) acc[gi][c] = f32x4v{0.f, 0.f, 0.f, 0.f};
  if constexpr (DOWN) {
    static_for<D>([&](auto d) { load_w(d, decltype(d)::value); });
    ready();
    static_for<D>([&](auto d) { load_x(d, decltype(d)::value); });
  } else {
    ready();
    static_for<D>([&](auto d) {
      load_x(d, decltype(d)::value);
      load_w(d, decltype(d)::value);
    });
  }
  for (int s0 = 0; s0 < nsteps; s0 += D)
    static_for<D>([&](auto d) {
      consume(d);
      load_x(d, s0 + decltype(d)::value + D);
      load_w(d, s0 + decltype(d)::value + D);
    });
}

// The item's sums of up to 16 rows over its four waves: thread i < 32 rows
// gets 4 consecutive positions, 4 (i % 32), of row i / 32, through put(row,
// position, value).
template <typename Put>
__device__ __forceinline__ void gather_sums(float* s_sum, const f32x4v (&acc)[8], int rows, Put put) {
  const int w = threadIdx.x >> 6, lane = lane_id(), g = lane >> 4, m = lane & 15;
  __syncthreads();  // s_sum is free
  if (m < rows) {
    float* p = s_sum + (w * 16 + m) * kStride + 32 * g;
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      *reinterpret_cast<float4*>(p + 8 * v) = make_float4(acc[0][v], acc[1][v], acc[2][v], acc[3][v]);
      *reinterpret_cast<float4*>(p + 8 * v + 4) = make_float4(acc[4][v], acc[5][v], acc[6][v], acc[7][v]);
    }
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 32 * rows; i += kThreads) {
    const int row = i >> 5, pos = 4 * (i & 31);
    float4 t = *reinterpret_cast<const float4*>(s_sum + row * kStride + pos);
#pragma unroll
    for (int q = 1; q < kWaves; ++q) {
      const float4 u = *reinterpret_cast<const float4*>(s_sum + (q * 16 + row) * kStride + pos);
      t.x += u.x;
      t.y += u.y;
      t.z += u.z;
      t.w += u.w;
    }
    put(row, pos, t);
  }
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + expf(-g)) * u; }

// TWO: an expert may have more than 16 rows (T > 16), which need two groups of
// accumulators.
template <bool TWO>
__global__ void __launch_bounds__(kThreads) __attribute__((amdgpu_waves_per_eu(2))) few_experts_kernel(Args a) {
  __shared__ Tables s;
  __shared__ __attribute__((aligned(16))) float s_sum[kWaves * 16 * kStride];
  __shared__ int s_tmp[kWaves];
  __shared__ int s_next, s_last;
  const int tid = threadIdx.x;
  int first = 0;
  if (tid == 0) first = raise(a.ticket, 1);
  for (int i = tid; i < a.E_local; i += kThreads) s.mask[i] = 0;
  __syncthreads();
  for (int t = tid >> 6; t < a.T; t += kWaves) {
    if (a.E <= 64)
      pick<1>(a, s, t);
    else if (a.E <= 256)
      pick<4>(a, s, t);
    else
      pick<16>(a, s, t);
  }
  __syncthreads();
  // rows, expert after expert, tokens in order
  constexpr int kPerT = kMaxE / kThreads;
  int n_rows, n_act;
  {
    int rows[kPerT], sum = 0, act = 0;
#pragma unroll
    for (int q = 0; q < kPerT; ++q) {
      const int e = tid * kPerT + q;
      rows[q] = e < a.E_local ? __popc(s.mask[e]) : 0;
      sum += rows[q];
      act += rows[q] > 0;
    }
    int r0 = block_exclusive_scan<kThreads>(sum, s_tmp, n_rows);
    int a0 = block_exclusive_scan<kThreads>(act, s_tmp, n_act);
#pragma unroll
    for (int q = 0; q < kPerT; ++q) {
      const int e = tid * kPerT + q;
      if (e < a.E_local) {
        s.row0[e] = r0;
        if (rows[q] > 0) s.act[a0] = e;
      }
      r0 += rows[q];
      a0 += rows[q] > 0;
    }
  }
  __syncthreads();
  auto row_of = [&](int e, int t) { return s.row0[e] + __popc(s.mask[e] & ((1u << t) - 1u)); };
  for (int i = tid; i < a.T * a.k; i += kThreads) {
    const int e = s.sel[i], t = i / a.k;
    if (e >= 0) s.tok[row_of(e, t)] = uint8_t(t);
  }
  if (tid == 0) s_next = first;
  __syncthreads();

  const int panels_a = (a.I + kGateUp - 1) / kGateUp, panels_b = (a.H + kCols - 1) / kCols;
  const int units_a = (a.H + kSub - 1) / kSub, units_b = (a.I + kSub - 1) / kSub;
  const Split sa = split(a.H, max(1, n_act) * panels_a), sb = split(a.I, max(1, n_act) * panels_b);
  const int items_a = n_act * sa.ranges * panels_a;
  // no local selection: the down items only write the zeros
  const int items = items_a + max(1, n_act) * (n_act ? sb.ranges : 1) * panels_b;

  // y of one down panel, from every row's partial sums
  auto combine = [&](int panel) {
    for (int i = tid; i < 32 * a.T; i += kThreads) {
      const int t = i >> 5, col = kCols * panel + 4 * (i & 31);
      if (col >= a.H) continue;
      float o[4] = {0.f, 0.f, 0.f, 0.f};
      for (int j = 0; j < a.k; ++j) {
        const int e = s.sel[t * a.k + j];
        if (e < 0) continue;
        const float* p = a.part_b + int64_t(row_of(e, t)) * sb.ranges * a.H + col;
        float v[4] = {0.f, 0.f, 0.f, 0.f};
        for (int r = 0; r < sb.ranges; ++r, p += a.H) {
          const float2 lo = get2(p), hi = get2(p + 2);
          v[0] += lo.x;
          v[1] += lo.y;
          v[2] += hi.x;
          v[3] += hi.y;
        }
        const float wt = s.wt[t * a.k + j];
#pragma unroll
        for (int q = 0; q < 4; ++q) o[q] = fmaf(wt, v[q], o[q]);
      }
      if (a.y_f32)
        *reinterpret_cast<float4*>(static_cast<float*>(a.y) + int64_t(t) * a.H + col) =
            make_float4(o[0], o[1], o[2], o[3]);
      else
        *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + int64_t(t) * a.H + col) =
            make_uint2(cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]));
    }
  };

  for (;;) {
    const int item = __builtin_amdgcn_readfirstlane(s_next);
    if (item >= items) break;
    int next = 0;
    if (item < items_a) {
      // expert, k range, panel (fastest: neighbours read neighbouring columns)
      const int panel = item % panels_a, er = item / panels_a;
      const int ai = er / sa.ranges, range = er - ai * sa.ranges;
      const int e = __builtin_amdgcn_readfirstlane(s.act[ai]);
      const int row0 = __builtin_amdgcn_readfirstlane(s.row0[e]);
      const int rows = __popc(__builtin_amdgcn_readfirstlane(int(s.mask[e])));
      const int units = min(sa.units, units_a - range * sa.units);
      auto ready = [&] {
        if (tid == 0) next = raise(a.ticket, 1);
      };
      auto put = [&](int gi) {
        return [&, gi](int r, int pos, const float4& t) {
          float* p = a.part_a + ((int64_t(row0 + 16 * gi + r) * sa.ranges + range) * panels_a + panel) * kCols + pos;
          put2(p, t.x, t.y);
          put2(p + 2, t.z, t.w);
        };
      };
      if (!TWO || rows <= 16) {
        f32x4v acc[1][8];
        stream<false, 1, 4>(a, s, e, panel, range * sa.units, units, row0, rows, acc, ready);
        gather_sums(s_sum, acc[0], rows, put(0));
      } else if constexpr (TWO) {
        f32x4v acc[2][8];
        stream<false, 2, 2>(a, s, e, panel, range * sa.units, units, row0, rows, acc, ready);
        gather_sums(s_sum, acc[0], 16, put(0));
        gather_sums(s_sum, acc[1], rows - 16, put(1));
      }
      stores_done();
      __syncthreads();
      if (tid == 0) {
        s_last = raise(a.cnt_a + ai * panels_a + panel, 1) == sa.ranges - 1;
        s_next = next;
      }
      __syncthreads();
      if (s_last) {
        // h of the panel's 64 outputs: 16 threads a row, 4 outputs each; the
        // gate of output o is at position 32 (o / 16) + o % 16, its up 16 on
        for (int i = tid; i < 16 * rows; i += kThreads) {
          const int r = i >> 4, o = 4 * (i & 15), oc = kGateUp * panel + o;
          if (oc >= a.I) continue;
          const float* p = a.part_a + (int64_t(row0 + r) * sa.ranges * panels_a + panel) * kCols + 32 * (o >> 4) + (o & 15);
          float gt[4] = {0.f, 0.f, 0.f, 0.f}, up[4] = {0.f, 0.f, 0.f, 0.f};
          for (int q = 0; q < sa.ranges; ++q, p += int64_t(panels_a) * kCols) {
            const float2 g0 = get2(p), g1 = get2(p + 2), u0 = get2(p + 16), u1 = get2(p + 18);
            gt[0] += g0.x;
            gt[1] += g0.y;
            gt[2] += g1.x;
            gt[3] += g1.y;
            up[0] += u0.x;
            up[1] += u0.y;
            up[2] += u1.x;
            up[3] += u1.y;
          }
          float* hp = a.h + int64_t(row0 + r) * a.I + oc;
          put2(hp, silu_mul(gt[0], up[0]), silu_mul(gt[1], up[1]));
          put2(hp + 2, silu_mul(gt[2], up[2]), silu_mul(gt[3], up[3]));
        }
        stores_done();
        __syncthreads();
        if (tid == 0) raise(a.cnt_h + ai * units_b + panel * kGateUp / kSub, 1);
      }
    } else if (n_act == 0) {
      combine(item - items_a);
      if (tid == 0) next = raise(a.ticket, 1);
      __syncthreads();
      if (tid == 0) s_next = next;
      __syncthreads();
    } else {
      const int bi = item - items_a;
      const int panel = bi % panels_b, er = bi / panels_b;
      const int ai = er / sb.ranges, range = er - ai * sb.ranges;
      const int e = __builtin_amdgcn_readfirstlane(s.act[ai]);
      const int row0 = __builtin_amdgcn_readfirstlane(s.row0[e]);
      const int rows = __popc(__builtin_amdgcn_readfirstlane(int(s.mask[e])));
      const int unit0 = range * sb.units, units = min(sb.units, units_b - unit0);
      // every panel of h in this k range is written
      auto ready = [&] {
        if (tid == 0) next = raise(a.ticket, 1);
        for (int u = tid; u < units; u += kThreads) {
          const int need = min(kSub / kGateUp, panels_a - (unit0 + u) * (kSub / kGateUp));
          while (__hip_atomic_load(a.cnt_h + ai * units_b + unit0 + u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < need)
            __builtin_amdgcn_s_sleep(1);
        }
        __syncthreads();
      };
      auto put = [&](int gi) {
        return [&, gi](int r, int pos, const float4& t) {
          const int col = kCols * panel + pos;
          if (col < a.H) {
            float* p = a.part_b + (int64_t(row0 + 16 * gi + r) * sb.ranges + range) * a.H + col;
            put2(p, t.x, t.y);
            put2(p + 2, t.z, t.w);
          }
        };
      };
      if (!TWO || rows <= 16) {
        f32x4v acc[1][8];
        stream<true, 1, 4>(a, s, e, panel, unit0, units, row0, rows, acc, ready);
        gather_sums(s_sum, acc[0], rows, put(0));
      } else if constexpr (TWO) {
        f32x4v acc[2][8];
        stream<true, 2, 2>(a, s, e, panel, unit0, units, row0, rows, acc, ready);
        gather_sums(s_sum, acc[0], 16, put(0));
        gather_sums(s_sum, acc[1], rows - 16, put(1));
      }
      stores_done();
      __syncthreads();
      if (tid == 0) {
        s_last = raise(a.cnt_b + panel, 1) == n_act * sb.ranges - 1;
        s_next = next;
      }
      __syncthreads();
      if (s_last) combine(panel);
    }
  }
}

struct Layout {
  size_t logits, counters, part_a, part_b, h, total;
  int n_counters, cnt_h, cnt_b;
};
// Rows times k ranges of an operand with `panels` panels per expert: with n
// experts in use there are at most min(cap, n T) rows, and ranges stay below
// kFewItems / (n panels) + 1.
inline int64_t row_ranges(int64_t cap, int T, int K, int panels) {
  const int64_t u = ceil_div(K, kSub);
  return std::min(cap * u, cap + int64_t(T) * ceil_div(kFewItems, panels));
}
inline Layout layout(int T, int H, int I, int E, int k, int E_local) {
  Layout L{};
  const int64_t cap = int64_t(T) * std::min(k, E_local), act = std::min<int64_t>(E_local, cap);
  const int pa = int(ceil_div(I, kGateUp)), pb = int(ceil_div(H, kCols));
  size_t o = 0;
  auto take = [&](int64_t n) {
    const size_t at = o;
    o = (o + size_t(n) * 4 + 255) / 256 * 256;
    return at;
  };
  L.cnt_h = int(1 + act * pa);
  L.cnt_b = int(L.cnt_h + act * ceil_div(I, kSub));
  L.n_counters = L.cnt_b + pb;
  L.logits = take(int64_t(T) * E);
  L.counters = take(L.n_counters);
  L.part_a = take(row_ranges(cap, T, H, pa) * pa * kCols);
  L.part_b = take(row_ranges(cap, T, I, pb) * H);
  L.h = take(cap * I);
  L.total = o;
  return L;
}

}  // namespace few

size_t few_workspace_bytes(int T, int H, int I, int E, int k, int E_local) {
  return few::layout(T, H, I, E, k, E_local).total;
}

hipError_t launch_few(const uint16_t* x, const float* w_router, const float* bias, const uint16_t* w_gate_up,
                      const uint16_t* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                      void* y, bool y_f32, char* ws, hipStream_t stream) {
  using namespace few;
  const Layout L = layout(T, H, I, E, k, E_local);
  float* logits = reinterpret_cast<float*>(ws + L.logits);
  int* ctr = reinterpret_cast<int*>(ws + L.counters);
  auto score = [&](auto tb) {
    hipLaunchKernelGGL(few_logits_kernel<decltype(tb)::value>, dim3(unsigned(E)), dim3(few::kThreads), 0, stream, x,
                       w_router, bias, T, H, E, logits, ctr, L.n_counters);
  };
  if (T == 1)
    score(std::integral_constant<int, 1>{});
  else if (T <= 4)
    score(std::integral_constant<int, 4>{});
  else if (T <= 8)
    score(std::integral_constant<int, 8>{});
  else if (T <= 16)
    score(std::integral_constant<int, 16>{});
  else
    score(std::integral_constant<int, 32>{});
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const Args a{x, logits, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, int(y_f32), y, ctr, ctr + 1,
               ctr + L.cnt_h, ctr + L.cnt_b, reinterpret_cast<float*>(ws + L.part_a),
               reinterpret_cast<float*>(ws + L.part_b), reinterpret_cast<float*>(ws + L.h)};
  hipLaunchKernelGGL(T > 16 ? few_experts_kernel<true> : few_experts_kernel<false>, dim3(unsigned(2 * device_cu_count())), dim3(few::kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe

// The whole share for a few tokens (at most 32) in two kernels.
//
//   y[t] = sum over local e in topk(t) of w[t, e] (silu(x[t] Wg_e) * (x[t] Wu_e)) Wd_e
//
// At a handful of tokens the used experts' weights are the whole cost (HBM),
// and the six launches of the general path cost more than reading them. Here
// few_logits_kernel scores the tokens and few_experts_kernel does the rest:
// every workgroup picks the tokens' experts for itself (a few thousand logits)
// and then takes items from queues, first all gate/up items, then all down
// items, then the weighted return:
//
//   gate/up item  (expert, k range, 128 gate or up columns) -> float32 partial
//                 sums; the last of a block of 128 outputs adds its k ranges
//                 and writes h = silu(g) * u
//   down item     (expert, k range, 128 outputs)  -> float32 partial sums
//   return item   (8 tokens, 128 outputs): adds the partial sums per token,
//                 slot by slot, weighted, and writes y
//
// An item's four waves share its k range and its 128 weight columns (256-byte
// pieces of every weight row); a wave streams the weights into registers in the
// grouped GEMV's geometry (grouped_gemv.hip: 8 rows x 8 columns per lane and
// step, transposed in registers, v_mfma_f32_16x16x32_bf16 with the weights as
// the A operand) and the waves' sums meet in LDS. Two workgroups per CU, so
// that one streams while the other exchanges its sums. A down item asks for
// its weights before it waits for h.
//
// Each kind's items lie in eight queues of consecutive items, one per XCD (every
// operation on a counter's line takes its turn: 512 workgroups on one counter
// were served in 7 us; every eighth item to an XCD left it a few 256-byte
// columns of every weight row, and so a few of its L2's channels). A workgroup
// takes its own queue's gate/up items, then its down items, then its return
// items. Waiting is safe however many workgroups run at a time and whatever
// else the GPU runs: a gate/up item waits for nothing; a workgroup that has
// waited for Args::polls polls (kFewPolls, some 2 ms) puts its item aside and
// takes what the other queues still hold of the kinds before it, gate/up items
// first, so all items that anybody waits for are with workgroups that are
// running.
//
// Bound: HBM from some eight tokens on (DeepSeek-R1-shaped EP=8 share, 16
// tokens, 1.13 GB of used experts: 198 us, the stream itself at 6 TB/s and
// more); below that the chain of exchanges (TP=8 share, one token, 95 MB: 38 us
// of which the weights take 14).
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
#include "moe_row.h"

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
constexpr int kStride = kCols + 4;
constexpr int kBatch = 8;       // exchanged values asked for at a time
constexpr int kTokens = 8;      // tokens of a return item
constexpr int kItems = 1024;    // items an operand is cut into where k allows (two per workgroup)
constexpr int kQueues = 8;      // of each kind of item, one per XCD (workgroup b runs on XCD b % 8)
constexpr int kPitch = 32;      // ints between counters: a 128-byte line each
constexpr int kCoherent = 16;   // buffer cache policy sc1: agent scope
constexpr int kStream = 2;      // nt: each weight byte is read once
constexpr uint32_t kOutside = 0x80000000u;  // offset past every buffer: reads zero

struct Args {
  const uint16_t* x;
  const float* logits;
  const uint16_t* w_gate_up;
  const uint16_t* w_down;
  int T, H, I, E, k, e0, E_local, renormalize, y_f32;
  int polls;  // before a waiting workgroup looks for items
  void* y;
  // counters, kPitch apart
  int* queue;     // [kind][queue]: items handed out
  int* cnt_a;     // [expert][128 of I]: gate and up items done
  int* cnt_h;     // [expert][512 of I]: blocks of h written
  int* cnt_b;     // [down panel]: items done
  float* part_a;  // [row][k range][gate panels, up panels][128]
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
  const int want = items >= kItems ? 1 : (kItems + items - 1) / items;
  const int units = want >= u ? 1 : (u + want - 1) / want;
  return {units, (u + units - 1) / units};
}

// ---------------------------------------------------------------------------
// Logits
// ---------------------------------------------------------------------------
// A workgroup scores TB tokens for one expert, float32 products and sums. (All
// of 32 tokens by one workgroup: 8.8 against 5.2 us for 32 experts of 2880; 16
// tokens, 256 experts of 7168: 8.2 against 7.5.) Also clears the second kernel's counters.
template <int TB>
__global__ void __launch_bounds__(kThreads) few_logits_kernel(const uint16_t* x, const float* w, const float* bias,
                                                              int T, int H, int E, float* logits, int* counters,
                                                              int ncounters) {
  __shared__ float s[kWaves][TB];
  const int e = blockIdx.x, t0 = TB * blockIdx.y;
  for (int i = (e + int(gridDim.x * blockIdx.y)) * kThreads + int(threadIdx.x); i < ncounters;
       i += int(gridDim.x * gridDim.y) * kThreads)
    counters[i] = 0;
  float acc[TB];
#pragma unroll
  for (int t = 0; t < TB; ++t) acc[t] = 0.f;
  for (int k = 4 * int(threadIdx.x); k < H; k += 4 * kThreads) {
    const float4 wv = *reinterpret_cast<const float4*>(w + int64_t(e) * H + k);
    uint2 xv[TB];
#pragma unroll
    for (int t = 0; t < TB; ++t) xv[t] = *reinterpret_cast<const uint2*>(x + int64_t(min(t0 + t, T - 1)) * H + k);
    __builtin_amdgcn_sched_barrier(0);  // all loads in flight before the first product
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      acc[t] = fmaf(bf16_lo(xv[t].x), wv.x, acc[t]);
      acc[t] = fmaf(bf16_hi(xv[t].x), wv.y, acc[t]);
      acc[t] = fmaf(bf16_lo(xv[t].y), wv.z, acc[t]);
      acc[t] = fmaf(bf16_hi(xv[t].y), wv.w, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < TB; ++t) {
    const float v = wave_sum_dpp(acc[t]);
    if (lane_id() == 0) s[threadIdx.x >> 6][t] = v;
  }
  __syncthreads();
  const int t = threadIdx.x;
  if (t < TB && t0 + t < T) logits[(t0 + t) * E + e] = s[0][t] + s[1][t] + s[2][t] + s[3][t] + (bias ? bias[e] : 0.f);
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
__device__ __forceinline__ int peek(const int* c) {
  return __hip_atomic_load(c, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
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
  int16_t sel[kMaxSel];   // slot (t, j): local expert, then its row, or -1
  float wt[kMaxSel];      // its weight
  uint8_t tok[kMaxSel];   // row: its token
};

// Largest / smallest value over rows of LANES lanes (16 or the whole wave), on
// every lane of the row: DPP steps inside 16 lanes, then scalar reads.
template <int LANES, typename Op>
__device__ __forceinline__ uint32_t row_reduce(uint32_t v, Op op) {
  auto step = [&](auto ctrl) {
    constexpr int c = decltype(ctrl)::value;
    v = op(v, uint32_t(__builtin_amdgcn_update_dpp(0, int(v), c, 0xF, 0xF, false)));
  };
  step(std::integral_constant<int, 0xB1>{});   // quad_perm [1,0,3,2]
  step(std::integral_constant<int, 0x4E>{});   // quad_perm [2,3,0,1]
  step(std::integral_constant<int, 0x141>{});  // row_half_mirror
  step(std::integral_constant<int, 0x140>{});  // row_mirror
  if constexpr (LANES == 64) {
    const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16),
                   c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
    v = op(op(a, b), op(c, d));
  }
  return v;
}

// A row of LANES lanes per token, expert li + LANES q in register q of lane
// li: k rounds of the largest logit left, the lowest expert among equal ones.
// Logits are compared as unsigned keys of the same order (-0 as +0, NaN as
// -infinity); a taken one becomes 0, below every key. t >= T: nothing is
// written.
template <int LANES, int NQ>
__device__ __forceinline__ void pick(const Args& a, Tables& s, int t) {
  const int li = lane_id() & (LANES - 1);
  uint32_t key[NQ];
  const float* row = a.logits + min(t, a.T - 1) * a.E;
#pragma unroll
  for (int q = 0; q < NQ; ++q) {
    const int e = li + LANES * q;
    const float f = row[min(e, a.E - 1)] + 0.f;
    const uint32_t u = __float_as_uint(f == f ? f : -INFINITY);
    key[q] = e < a.E ? (u >> 31 ? ~u : u | 0x80000000u) : 0u;
  }
  auto value = [](uint32_t k) { return __uint_as_float(k >> 31 ? k & 0x7FFFFFFFu : ~k); };
  auto larger = [](uint32_t x, uint32_t y) { return max(x, y); };
  auto smaller = [](uint32_t x, uint32_t y) { return min(x, y); };
  auto add = [](uint32_t x, uint32_t y) { return __float_as_uint(__uint_as_float(x) + __uint_as_float(y)); };
  constexpr int KS = LANES == 16 ? 2 : 1;  // selections a lane keeps (k <= 32)
  uint32_t got[KS] = {}, at[KS] = {};
  float top = 0.f, all = 0.f;
  for (int j = 0; j < a.k; ++j) {
    uint32_t best = 0, bq = 0;
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (key[q] > best) {
        best = key[q];
        bq = q;
      }
    const uint32_t m = row_reduce<LANES>(best, larger);
    const uint32_t mine = best == m ? uint32_t(li) + LANES * bq : 0xFFFFFFFFu;
    const uint32_t e = row_reduce<LANES>(mine, smaller);
    if (j == 0) {
      top = value(m);
      if (!a.renormalize) {
        float z = 0.f;
#pragma unroll
        for (int q = 0; q < NQ; ++q)
          if (key[q]) z += expf(value(key[q]) - top);
        all = __uint_as_float(row_reduce<LANES>(__float_as_uint(z), add));
      }
    }
#pragma unroll
    for (int q = 0; q < NQ; ++q)
      if (mine == e && bq == uint32_t(q)) key[q] = 0;
#pragma unroll
    for (int c = 0; c < KS; ++c)
      if (li + LANES * c == j) {
        got[c] = m;
        at[c] = e;
      }
  }
  float p[KS], sum = 0.f;
#pragma unroll
  for (int c = 0; c < KS; ++c) {
    p[c] = li + LANES * c < a.k ? expf(value(got[c]) - top) : 0.f;
    sum += p[c];
  }
  sum = __uint_as_float(row_reduce<LANES>(__float_as_uint(sum), add));
  if (!a.renormalize) sum = all;
#pragma unroll
  for (int c = 0; c < KS; ++c) {
    const int j = li + LANES * c;
    if (t < a.T && j < a.k) {
      const int e = int(at[c]) - a.e0;
      const bool local = e >= 0 && e < a.E_local;
      s.sel[t * a.k + j] = int16_t(local ? e : -1);
      s.wt[t * a.k + j] = p[c] / sum;
      if (local) atomicOr(&s.mask[e], 1u << t);
    }
  }
}

// The local slots of a return item's tokens.
struct Returns {
  int n[kTokens];
  int16_t row[kTokens][32];
  float wt[kTokens][32];
};

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

// Sums over k range [unit0, unit0 + units) x 512 of the `cols` (at most 128)
// columns from col0 for `rows` rows: acc[gi][c][v] of lane 16 g + m is column 8 (4 g + v) + c of row
// 16 gi + m (this wave's share of k). ready(): called once, after the first
// weights are asked for and before the first activations.
// Returns false, with nothing added, where ready() did.
template <bool DOWN, int G, int D, typename Ready>
__device__ __forceinline__ bool stream(const Args& a, const Tables& s, int e, int col0, int cols, int unit0,
                                       int units, int row0, int rows, f32x4v (&acc)[G][8], Ready ready) {
  const int w = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int lane = lane_id(), g = lane >> 4, m = lane & 15;
  const int K = DOWN ? a.I : a.H, ldw = DOWN ? a.H : 2 * a.I;
  const int col = 8 * m;
  const uint32_t wvo = col < cols ? uint32_t(8 * g * ldw + col0 + col) * 2u : kOutside;
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
            // (nothing is left of an infinity: inf - inf would make its products NaN)
            const float r1 = hi[b] == __float_as_uint(f) ? 0.f : f - __uint_as_float(hi[b]);
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
    if (!ready()) return false;
    static_for<D>([&](auto d) { load_x(d, decltype(d)::value); });
  } else {
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
  return true;
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
  __shared__ Returns s_ret;
  __shared__ int2 s_item, s_aside;
  __shared__ int s_last, s_ok;
  const int tid = threadIdx.x;
  int my_kind = 0, my_queue = blockIdx.x % kQueues, asked = 0;
  auto queue = [&](int kind, int q) { return a.queue + (kind * kQueues + q) * kPitch; };
  auto ask = [&] {
    if (tid == 0 && my_kind < 3) asked = raise(queue(my_kind, my_queue), 1);
  };
  ask();
  for (int i = tid; i < a.E_local; i += kThreads) s.mask[i] = 0;
  __syncthreads();
  if (a.E <= 256 && a.T > kWaves) {
    for (int t = tid >> 4; t < ((a.T + 15) & ~15); t += kThreads / 16) {
      if (a.E <= 32)
        pick<16, 2>(a, s, t);
      else if (a.E <= 64)
        pick<16, 4>(a, s, t);
      else
        pick<16, 16>(a, s, t);
    }
  } else {  // up to four tokens: a wave each
    for (int t = tid >> 6; t < a.T; t += kWaves) {
      if (a.E <= 256)
        pick<64, 4>(a, s, t);
      else
        pick<64, 16>(a, s, t);
    }
  }
  __syncthreads();
  // rows, expert after expert, tokens in order
  constexpr int kPerT = kMaxE / kThreads;
  int n_act;
  {
    // both prefixes in one scan: rows (at most T k = 1024) above, experts below
    int rows[kPerT], sum = 0, total;
#pragma unroll
    for (int q = 0; q < kPerT; ++q) {
      const int e = tid * kPerT + q;
      rows[q] = e < a.E_local ? __popc(s.mask[e]) : 0;
      sum += rows[q] * 65536 + (rows[q] > 0);
    }
    int pre = block_exclusive_scan<kThreads>(sum, s_tmp, total);
    n_act = total & 0xFFFF;
#pragma unroll
    for (int q = 0; q < kPerT; ++q) {
      const int e = tid * kPerT + q;
      if (e < a.E_local) {
        s.row0[e] = pre >> 16;
        if (rows[q] > 0) s.act[pre & 0xFFFF] = e;
      }
      pre += rows[q] * 65536 + (rows[q] > 0);
    }
  }
  __syncthreads();
  // from here on a slot holds its row instead of its expert
  for (int i = tid; i < a.T * a.k; i += kThreads) {
    const int e = s.sel[i], t = i / a.k;
    if (e >= 0) {
      const int r = s.row0[e] + __popc(s.mask[e] & ((1u << t) - 1u));
      s.tok[r] = uint8_t(t);
      s.sel[i] = int16_t(r);
    }
  }
  __syncthreads();

  const int blocks = (a.I + kCols - 1) / kCols;  // of 128 outputs of h; a gate and an up panel each
  const int panels_a = 2 * blocks, panels_b = (a.H + kCols - 1) / kCols;
  const int units_a = (a.H + kSub - 1) / kSub, units_b = (a.I + kSub - 1) / kSub;
  const Split sa = split(a.H, max(1, n_act) * panels_a), sb = split(a.I, max(1, n_act) * panels_b);
  const int items_a = n_act * sa.ranges * panels_a, items_b = n_act * sb.ranges * panels_b;
  const int items_c = (a.T + kTokens - 1) / kTokens * panels_b;

  auto items_of = [&](int kind) { return kind == 0 ? items_a : kind == 1 ? items_b : items_c; };
  auto left_of = [&](int kind, int q) {  // items of queue q at the start
    const int chunk = (items_of(kind) + kQueues - 1) / kQueues;
    return min(chunk, items_of(kind) - q * chunk);
  };
  auto item_at = [&](int kind, int q, int t) { return q * ((items_of(kind) + kQueues - 1) / kQueues) + t; };
  // The next item, by wave 0: ask() raises its queue's counter, without waiting
  // for the answer; answer() makes an item of it. kind 3: none left.
  auto answer = [&]() -> int2 {
    for (;;) {
      const int t = __builtin_amdgcn_readfirstlane(asked);
      if (t < left_of(my_kind, my_queue)) return make_int2(my_kind, item_at(my_kind, my_queue, t));
      if (++my_kind == 3) return make_int2(3, 0);
      ask();
    }
  };
  // Once the asked counter's value is there anyway: a queue found empty is left
  // for the next kind's, whose answer then comes while the sums are exchanged.
  auto settle = [&] {
    if (tid < 64 && my_kind < 2 && __builtin_amdgcn_readfirstlane(asked) >= left_of(my_kind, my_queue)) {
      ++my_kind;
      ask();
    }
  };
  // An item of a kind before `kind` from any queue (kind 3: none is left), by
  // wave 0; lane q < 8 looks at queue q.
  auto rescue = [&](int kind) -> int2 {
    const int lane = lane_id();
    for (int kd = 0; kd < kind; ++kd)
      for (;;) {
        bool left = false;
        if (lane < kQueues) left = peek(queue(kd, lane)) < left_of(kd, lane);
        const uint64_t any = ballot(left);
        if (any == 0) break;
        const int q = __builtin_ctzll(any);
        int t = 0;
        if (lane == 0) t = raise(queue(kd, q), 1);
        t = __builtin_amdgcn_readfirstlane(t);
        if (t < left_of(kd, q)) return make_int2(kd, item_at(kd, q, t));
      }
    return make_int2(3, 0);
  };
  // Polls until *c reaches n, at most a.polls times.
  auto poll = [&](const int* c, int n) {
    for (int i = 0; i < a.polls; ++i) {
      if (peek(c) >= n) return true;
      __builtin_amdgcn_s_sleep(1);
    }
    return false;
  };

  // y of one down panel for kTokens tokens, from their rows' partial sums:
  // slot by slot, k range by k range, kBatch loads at a time
  auto combine = [&](int panel, int t0) {
    const int lt = tid >> 5, t = t0 + lt, col = kCols * panel + 4 * (tid & 31);
    if (t >= a.T || col >= a.H) return;
    float o[4] = {0.f, 0.f, 0.f, 0.f}, v[4] = {0.f, 0.f, 0.f, 0.f};
    const int terms = s_ret.n[lt] * sb.ranges;
    int slot = 0, r = 0;  // of the next term to be added
    for (int i0 = 0; i0 < terms; i0 += kBatch) {
      float2 q[kBatch][2] = {};
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < terms) {
          const int sl = (i0 + i) / sb.ranges;
          const float* p = a.part_b + (int64_t(s_ret.row[lt][sl]) * sb.ranges + (i0 + i - sl * sb.ranges)) * a.H + col;
          q[i][0] = get2(p);
          q[i][1] = get2(p + 2);
        }
#pragma unroll
      for (int i = 0; i < kBatch; ++i)
        if (i0 + i < terms) {
          v[0] += q[i][0].x;
          v[1] += q[i][0].y;
          v[2] += q[i][1].x;
          v[3] += q[i][1].y;
          if (++r == sb.ranges) {
            const float wt = s_ret.wt[lt][slot];
#pragma unroll
            for (int c = 0; c < 4; ++c) {
              o[c] = fmaf(wt, v[c], o[c]);
              v[c] = 0.f;
            }
            ++slot;
            r = 0;
          }
        }
    }
    if (a.y_f32)
      *reinterpret_cast<float4*>(static_cast<float*>(a.y) + int64_t(t) * a.H + col) =
          make_float4(o[0], o[1], o[2], o[3]);
    else
      *reinterpret_cast<uint2*>(static_cast<uint16_t*>(a.y) + int64_t(t) * a.H + col) =
          make_uint2(cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]));
  };

  // s_item: the item at hand; s_aside: an item that waits while its workgroup
  // does a rescued one (kind 3: none)
  if (tid < 64) {
    const int2 f = answer();
    if (tid == 0) {
      s_item = f;
      s_aside = make_int2(3, 0);
    }
  }
  __syncthreads();
  for (;;) {
    const int kind = __builtin_amdgcn_readfirstlane(s_item.x), item = __builtin_amdgcn_readfirstlane(s_item.y);
    const bool rescued = __builtin_amdgcn_readfirstlane(s_aside.x) != 3;
    if (kind == 3) break;
    // The end of an item: the one put aside, or the next of the queue. Waves
    // other than the first see it after the caller's barrier.
    auto advance = [&] {
      if (tid >= 64) return;
      const int2 n = rescued ? s_aside : answer();
      if (tid == 0) {
        s_item = n;
        s_aside = make_int2(3, 0);
      }
    };
    // Nothing came: a rescued item first, this one again after it. (A rescued
    // down item was found with every gate/up item handed out: it just polls on.)
    auto put_aside = [&] {
      __syncthreads();
      if (tid < 64 && !rescued) {
        const int2 o = rescue(kind);
        if (tid == 0 && o.x != 3) {
          s_aside = make_int2(kind, item);
          s_item = o;
        }
      }
      __syncthreads();
    };
    // Asks for the item after this one: a gate/up item at its start, the
    // others when they need not wait any more (an item in the hands of a waiting
    // workgroup would wait with it).
    auto ask_next = [&] {
      if (!rescued) ask();
    };
    if (kind == 2) {
      const int panel = item % panels_b, t0 = item / panels_b * kTokens;
      // the tokens' local slots one after another, while the sums are waited for
      if (tid >= 64 && tid < 64 + kTokens) {
        const int lt = tid - 64, t = t0 + lt;
        int n = 0;
        if (t < a.T)
          for (int j = 0; j < a.k; ++j) {
            const int row = s.sel[t * a.k + j];
            if (row >= 0) {
              s_ret.row[lt][n] = int16_t(row);
              s_ret.wt[lt][n] = s.wt[t * a.k + j];
              ++n;
            }
          }
        s_ret.n[lt] = n;
      }
      if (tid == 0) s_ok = poll(a.cnt_b + panel * kPitch, n_act * sb.ranges);
      if (tid == 0 && s_ok) ask_next();
      __syncthreads();
      if (!s_ok) {
        put_aside();
        continue;
      }
      combine(panel, t0);
      advance();
      __syncthreads();
      continue;
    }
    // expert, k range, panel (fastest: neighbours read neighbouring columns)
    const bool down = kind == 1;
    const int np = down ? panels_b : panels_a, nr = down ? sb.ranges : sa.ranges;
    const int panel = item % np, er = item / np;
    const int ai = er / nr, range = er - ai * nr;
    const int e = __builtin_amdgcn_readfirstlane(s.act[ai]);
    const int row0 = __builtin_amdgcn_readfirstlane(s.row0[e]);
    const int rows = __popc(__builtin_amdgcn_readfirstlane(int(s.mask[e])));
    const int unit0 = range * (down ? sb.units : sa.units);
    const int units = min(down ? sb.units : sa.units, (down ? units_b : units_a) - unit0);
    if (!down) {
      const int block = panel < blocks ? panel : panel - blocks;
      const int col0 = kCols * block + (panel < blocks ? 0 : a.I), cols = min(kCols, a.I - kCols * block);
      auto ready = [] { return true; };
      ask_next();
      auto put = [&](int gi) {
        return [&, gi](int r, int pos, const float4& t) {
          float* p = a.part_a + ((int64_t(row0 + 16 * gi + r) * sa.ranges + range) * panels_a + panel) * kCols + pos;
          put2(p, t.x, t.y);
          put2(p + 2, t.z, t.w);
        };
      };
      if (!TWO || rows <= 16) {
        f32x4v acc[1][8];
        stream<false, 1, 4>(a, s, e, col0, cols, unit0, units, row0, rows, acc, ready);
        if (!rescued) settle();
        gather_sums(s_sum, acc[0], rows, put(0));
      } else if constexpr (TWO) {
        f32x4v acc[2][8];
        stream<false, 2, 2>(a, s, e, col0, cols, unit0, units, row0, rows, acc, ready);
        if (!rescued) settle();
        gather_sums(s_sum, acc[0], 16, put(0));
        gather_sums(s_sum, acc[1], rows - 16, put(1));
      }
      stores_done();
      __syncthreads();
      int before = 0;  // (its answer and the next item's arrive together)
      if (tid == 0) before = raise(a.cnt_a + (int64_t(ai) * blocks + block) * kPitch, 1);
      advance();
      if (tid == 0) s_last = before == 2 * sa.ranges - 1;
      __syncthreads();
      if (s_last) {
        // h of the block's 128 outputs, up to 8 rows at a time: 32 threads of 4
        // outputs per row, and with fewer rows the ranges dealt to the threads
        // left, whose sums meet in LDS
        const int rp = min(8, rows <= 1 ? 1 : 1 << (32 - __clz(rows - 1))), ng = 8 / rp;
        const int slot = tid >> 5, o = 4 * (tid & 31), oc = kCols * block + o;
        const int grp = slot / rp;
        for (int r0 = 0; r0 < rows; r0 += rp) {
          const int r = r0 + slot % rp;
          float gu[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
          if (r < rows && oc < a.I) {
            const float* p = a.part_a + (int64_t(row0 + r) * sa.ranges * panels_a + block) * kCols + o;
            constexpr int B = kBatch / 2;  // of four loads each
            for (int q0 = grp; q0 < sa.ranges; q0 += B * ng) {
              float2 v[B][4] = {};
#pragma unroll
              for (int q = 0; q < B; ++q)
                if (q0 + q * ng < sa.ranges) {
                  const float* pq = p + int64_t(q0 + q * ng) * panels_a * kCols;
                  v[q][0] = get2(pq);
                  v[q][1] = get2(pq + 2);
                  v[q][2] = get2(pq + int64_t(blocks) * kCols);
                  v[q][3] = get2(pq + int64_t(blocks) * kCols + 2);
                }
#pragma unroll
              for (int q = 0; q < B; ++q)
#pragma unroll
                for (int c = 0; c < 4; ++c) {
                  gu[2 * c] += v[q][c].x;
                  gu[2 * c + 1] += v[q][c].y;
                }
            }
          }
          if (ng > 1) {  // s_sum: [slot][8 values][32 threads]
            __syncthreads();
#pragma unroll
            for (int c = 0; c < 8; ++c) s_sum[(slot * 8 + c) * 32 + (tid & 31)] = gu[c];
            __syncthreads();
            if (grp == 0)
              for (int i = 1; i < ng; ++i)
#pragma unroll
                for (int c = 0; c < 8; ++c) gu[c] += s_sum[((slot + i * rp) * 8 + c) * 32 + (tid & 31)];
          }
          if (grp == 0 && r < rows && oc < a.I) {
            float* hp = a.h + int64_t(row0 + r) * a.I + oc;
            put2(hp, silu_mul(gu[0], gu[4]), silu_mul(gu[1], gu[5]));
            put2(hp + 2, silu_mul(gu[2], gu[6]), silu_mul(gu[3], gu[7]));
          }
        }
        stores_done();
        __syncthreads();
        if (tid == 0) raise(a.cnt_h + (int64_t(ai) * units_b + block * kCols / kSub) * kPitch, 1);
      }
    } else {
      const int col0 = kCols * panel, cols = min(kCols, a.H - col0);
      // every block of h in this k range is written
      auto ready = [&] {
        if (tid < 64) {
          bool ok = true;
          for (int u = tid; u < units && ok; u += 64)
            ok = poll(a.cnt_h + (int64_t(ai) * units_b + unit0 + u) * kPitch,
                      min(kSub / kCols, blocks - (unit0 + u) * (kSub / kCols)));
          const uint64_t no = ballot(!ok);
          if (tid == 0) s_ok = no == 0;
          if (no == 0) ask_next();
        }
        __syncthreads();
        return s_ok != 0;
      };
      auto put = [&](int gi) {
        return [&, gi](int r, int pos, const float4& t) {
          if (pos < cols) {
            float* p = a.part_b + (int64_t(row0 + 16 * gi + r) * sb.ranges + range) * a.H + col0 + pos;
            put2(p, t.x, t.y);
            put2(p + 2, t.z, t.w);
          }
        };
      };
      if (!TWO || rows <= 16) {
        f32x4v acc[1][8];
        if (!stream<true, 1, 4>(a, s, e, col0, cols, unit0, units, row0, rows, acc, ready)) {
          put_aside();
          continue;
        }
        if (!rescued) settle();
        gather_sums(s_sum, acc[0], rows, put(0));
      } else if constexpr (TWO) {
        f32x4v acc[2][8];
        if (!stream<true, 2, 2>(a, s, e, col0, cols, unit0, units, row0, rows, acc, ready)) {
          put_aside();
          continue;
        }
        if (!rescued) settle();
        gather_sums(s_sum, acc[0], 16, put(0));
        gather_sums(s_sum, acc[1], rows - 16, put(1));
      }
      stores_done();
      __syncthreads();
      if (tid == 0) raise(a.cnt_b + panel * kPitch, 1);
      advance();
      __syncthreads();
    }
  }
}

struct Layout {
  size_t logits, counters, part_a, part_b, h, total;
  int64_t n_counters, cnt_a, cnt_h, cnt_b;
};
// Rows times k ranges of an operand with `panels` panels per expert: with n
// experts in use there are at most min(cap, n T) rows, and ranges stay below
// kItems / (n panels) + 1.
inline int64_t row_ranges(int64_t cap, int T, int K, int panels) {
  const int64_t u = ceil_div(K, kSub);
  return std::min(cap * u, cap + int64_t(T) * ceil_div(kItems, panels));
}
inline Layout layout(int T, int H, int I, int E, int k, int E_local) {
  Layout L{};
  const int64_t cap = int64_t(T) * std::min(k, E_local), act = std::min<int64_t>(E_local, cap);
  const int blocks = int(ceil_div(I, kCols)), pa = 2 * blocks, pb = int(ceil_div(H, kCols));
  size_t o = 0;
  auto take = [&](int64_t n) {
    const size_t at = o;
    o = (o + size_t(n) * 4 + 255) / 256 * 256;
    return at;
  };
  L.cnt_a = 3 * kQueues * kPitch;
  L.cnt_h = L.cnt_a + act * blocks * kPitch;
  L.cnt_b = L.cnt_h + act * ceil_div(I, kSub) * kPitch;
  L.n_counters = L.cnt_b + int64_t(pb) * kPitch;
  L.logits = take(int64_t(T) * E);
  L.counters = take(L.n_counters);
  L.part_a = take(row_ranges(cap, T, H, pa) * pa * kCols);
  L.part_b = take(row_ranges(cap, T, I, pb) * H);
  L.h = take(cap * I);
  L.total = o;
  return L;
}

}  // namespace few

bool few_supported(int T, int H, int I, int k, int E_local) {
  // the counters are indexed with 31 bits (32 of them per 128 columns of each
  // expert in use); x and an expert's rows of h (float32, at most T of them) end
  // below the offset that stands for "outside"
  return int64_t(std::min<int64_t>(E_local, int64_t(T) * k)) * I < (int64_t(1) << 32) &&
         int64_t(T) * I < (int64_t(1) << 29) && int64_t(T) * H < (int64_t(1) << 30);
}

size_t few_workspace_bytes(int T, int H, int I, int E, int k, int E_local) {
  return few::layout(T, H, I, E, k, E_local).total;
}

hipError_t launch_few(const uint16_t* x, const float* w_router, const float* bias, const uint16_t* w_gate_up,
                      const uint16_t* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                      void* y, bool y_f32, int workgroups, int polls, char* ws, hipStream_t stream) {
  using namespace few;
  const Layout L = layout(T, H, I, E, k, E_local);
  float* logits = reinterpret_cast<float*>(ws + L.logits);
  int* ctr = reinterpret_cast<int*>(ws + L.counters);
  auto score = [&](auto tb) {
    hipLaunchKernelGGL(few_logits_kernel<decltype(tb)::value>, dim3(unsigned(E), unsigned(ceil_div(T, tb))),
                       dim3(few::kThreads), 0, stream, x, w_router, bias, T, H, E, logits, ctr, int(L.n_counters));
  };
  if (T == 1)
    score(std::integral_constant<int, 1>{});
  else if (T <= 4)
    score(std::integral_constant<int, 4>{});
  else
    score(std::integral_constant<int, 8>{});
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const Args a{x, logits, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, int(y_f32), polls, y, ctr,
               ctr + L.cnt_a, ctr + L.cnt_h, ctr + L.cnt_b, reinterpret_cast<float*>(ws + L.part_a),
               reinterpret_cast<float*>(ws + L.part_b), reinterpret_cast<float*>(ws + L.h)};
  // (at least one workgroup per queue: return items are not taken from another's)
  const int grid = std::max(kQueues, workgroups > 0 ? workgroups : 2 * device_cu_count());
  hipLaunchKernelGGL(T > 16 ? few_experts_kernel<true> : few_experts_kernel<false>, dim3(unsigned(grid)),
                     dim3(few::kThreads), 0, stream, a);
  return hipGetLastError();
}

}  // namespace moe

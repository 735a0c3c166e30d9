// Products of 8-bit integers with one scale per token (row of A) and one per
// weight channel (row of W), for the ragged expert segments or one matrix:
//
//   C[m, n] = sa[m] sw[n] sum_k A[m, k] W[n, k]
//
// The sum is exact: int8 x int8 products in int32 accumulators, |sum| <=
// 2^14 K < 2^31 for K < 2^17. It does not depend on tiling, k order or split,
// so every kernel here gives the same bits. The sum is converted to float32 and
// multiplied there by the product of the two scales; then comes the rounding to
// bf16.
//
// Both operands are k-contiguous (W is stored [N, K], a channel per row), so
// both feed v_mfma_i32_16x16x64_i8 without a transpose:
//   A fragment: lane l holds A[l % 16][16 (l / 16) .. +15]
//   B fragment: lane l holds B[16 (l / 16) .. +15][l % 16]
//   C: lane l holds column l % 16, rows 4 (l / 16) .. +3
// The weights are always the first operand, so a lane ends with 4 consecutive
// channels of one token and stores them as one vector.
//
// One kernel in a dozen tile shapes, from 16 x 32 (few rows: the weight stream is the
// whole cost) to 288 x 256. The operands come through LDS by direct-to-LDS loads
// of whole 128-byte lines. (Weight fragments loaded straight into registers, 16
// rows x 64 bytes an instruction, streamed a DeepSeek-R1-shaped rank's 1.41 GB at
// 8 rows per expert in 410 us; the tiles take 254.)
#include "gemm_dma.h"
#include "gemm_tile.h"
#include "moe_kernels.h"
#include "moe_row.h"

namespace moe {
namespace i8 {

using dma::dma16;
typedef dma::i32x4 i32x4;

constexpr int kMaxLocal = 1024;
constexpr int64_t kMaxGrid = 1 << 20;  // workgroups of a launch; the kernels stride over more work

__device__ __forceinline__ i32x4 mfma(const i32x4& w, const i32x4& a, const i32x4& c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(w, a, c, 0, 0, 0);
}

struct GemmArgs {
  const int8_t* A;            // rows of K bytes
  const float* sa;            // scale of each row of A
  const int32_t* gather_src;  // row n of a segment is row gather_src[n] / gather_k of A (NULL: row n)
  int gather_k, gather_rows;
  const int32_t* offsets;     // segments [offsets[e], offsets[e + 1]) (NULL: one, [0, capacity))
  int E_local;
  int64_t capacity;
  const int8_t* W;            // [E_local][wrows, K]
  const float* sw;            // [E_local, wrows]
  int wrows, K, N, up_off;    // N outputs; gate/up: channel n and up_off + n
  void* C;                    // [capacity, N]: bf16, or float32 h for gate/up
};

__device__ __forceinline__ void segment(const GemmArgs& p, int e, int& a, int& b) {
  if (p.offsets == nullptr) {
    a = 0;
    b = int(p.capacity);
    return;
  }
  const int64_t lo = min<int64_t>(max<int64_t>(p.offsets[e], 0), p.capacity);
  a = int(lo);
  b = int(max<int64_t>(lo, min<int64_t>(p.offsets[e + 1], p.capacity)));
}

__device__ __forceinline__ float silu_mul(float g, float u) { return g / (1.f + __expf(-g)) * u; }

// 4 consecutive outputs of one row
__device__ __forceinline__ void store4(const GemmArgs& p, int64_t row, int col, const i32x4& c, float sa,
                                       const float4& sw) {
  const float s[4] = {sw.x, sw.y, sw.z, sw.w};
  float o[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = float(c[v]) * (sa * s[v]);
  *reinterpret_cast<uint2*>(static_cast<uint16_t*>(p.C) + row * p.N + col) =
      make_uint2(cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]));
}
// 8 consecutive outputs of one row
__device__ __forceinline__ void store8(const GemmArgs& p, int64_t row, int col, const i32x4& c, const i32x4& d,
                                       float sa, const float4& s, const float4& t) {
  *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.C) + row * p.N + col) =
      u32x4{cvt_bf16x2(float(c[0]) * (sa * s.x), float(c[1]) * (sa * s.y)),
            cvt_bf16x2(float(c[2]) * (sa * s.z), float(c[3]) * (sa * s.w)),
            cvt_bf16x2(float(d[0]) * (sa * t.x), float(d[1]) * (sa * t.y)),
            cvt_bf16x2(float(d[2]) * (sa * t.z), float(d[3]) * (sa * t.w))};
}
__device__ __forceinline__ void store4_swiglu(const GemmArgs& p, int64_t row, int col, const i32x4& g, const i32x4& u,
                                              float sa, const float4& sg, const float4& su) {
  const float a[4] = {sg.x, sg.y, sg.z, sg.w}, b[4] = {su.x, su.y, su.z, su.w};
  float o[4];
#pragma unroll
  for (int v = 0; v < 4; ++v) o[v] = silu_mul(float(g[v]) * (sa * a[v]), float(u[v]) * (sa * b[v]));
  *reinterpret_cast<float4*>(static_cast<float*>(p.C) + row * p.N + col) = make_float4(o[0], o[1], o[2], o[3]);
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------
constexpr int kRowB = 128;  // bytes of k per stage: one whole line per operand row

__device__ __forceinline__ int chunk_pos(int r, int c) { return c ^ ((r >> 1) & 7); }

// ROWS operand rows x 128 bytes of k: load j (8 rows, 8 lanes each) is issued
// by wave j % W. Row r sits at 128 r, its 16-byte chunk c at c ^ ((r >> 1) & 7)
// (conflict-free for 16 lanes reading one chunk of 16 consecutive rows).
template <int ROWS, int W>
struct Loader {
  static constexpr int kLoads = ROWS / 8;
  static constexpr int kPer = (kLoads + W - 1) / W;
  static_assert(W % 2 == 0, "a lane's chunk does not depend on the load");
  i32x4 rsrc;
  uint32_t voff[kPer];
  // loads of this wave per stage
  __device__ __forceinline__ static int count(int w) { return (kLoads - w + W - 1) / W; }
  // the chunk this lane fetches in every load
  __device__ __forceinline__ static int chunk(int w) {
    const int lane = lane_id();
    return (lane & 7) ^ ((4 * (w & 1) + (lane >> 4)) & 7);
  }
  template <typename SrcRow>
  __device__ __forceinline__ void init(const int8_t* base, int64_t bytes, int ld, int w, SrcRow src_row) {
    rsrc = dma::buffer_rsrc(base, bytes);
    const int c = chunk(w);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      voff[i] = uint32_t(src_row(8 * (i * W + w) + (lane_id() >> 3))) * uint32_t(ld) + 16u * uint32_t(c);
  }
  // back: bytes a lane whose chunk lies past K steps back, to read inside its row
  __device__ __forceinline__ void issue(MOE_LDS char* dst, int w, uint32_t k0, uint32_t back = 0) const {
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kLoads % W == 0 || i * W + w < kLoads) dma16(rsrc, voff[i] - back, k0, dst + 1024 * (i * W + w));
  }
};

template <int N>
__device__ __forceinline__ void wait_vm() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  __builtin_amdgcn_s_waitcnt((N & 0xF) | (((N >> 4) & 3) << 14) | (0x7 << 4) | (0xF << 8));
}
template <int MAX>
__device__ __forceinline__ void wait_vm_dyn(int n) {
  if constexpr (MAX == 0) {
    wait_vm<0>();
  } else {
    if (n >= MAX)
      wait_vm<MAX>();
    else
      wait_vm_dyn<MAX - 1>(n);
  }
}

template <int NM, int NR>
__device__ __forceinline__ void alternate_mfma_reads() {
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);              // one MFMA
    if (i < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);  // one LDS read
  }
#pragma unroll
  for (int i = NM; i < NR; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
}

// KG groups of WR x WC waves; a tile is 16 FM WR rows x 16 FN WC channels, S
// stages in LDS per group. Group q takes k stages q, q + KG, ..; the groups'
// int32 sums meet in LDS (exact in any order). 16-row fragment f belongs to wave
// row f % WR; wave column wn holds channels 16 FN wn .. (gate/up: 8 FN of gate,
// then the matching up).
template <int WR_, int WC_, int FN_, int S_, int KG_>
struct Shape {
  static constexpr int WR = WR_, WC = WC_, FN = FN_, S = S_, KG = KG_;
  static constexpr int W = WR * WC, BN = 16 * FN * WC;
};

template <typename T, int FM>
constexpr int stage_bytes() { return (16 * FM * T::WR + T::BN) * kRowB; }

// Which channel of its wave column's C a weight fragment's row r holds: lane
// group g gets rows 4 g .. 4 g + 3 of each of the C / 16 fragments j, and these
// are its C / 4 consecutive channels, so that it stores whole vectors.
template <int C>
__device__ __forceinline__ int channel_of(int j, int r) { return C / 4 * (r >> 2) + 4 * j + (r & 3); }

template <typename T, int FM, bool SWIGLU, bool TAIL, typename SrcRow>
__device__ __forceinline__ void run_tile(MOE_LDS char* lds, const GemmArgs& p, const int8_t* a_base, int64_t a_bytes,
                                         SrcRow src_row, int rows, int r0, int e, int nj) {
  constexpr int WR = T::WR, FN = T::FN, S = T::S, W = T::W, BN = T::BN, KG = T::KG;
  constexpr int BM = 16 * FM * WR;
  constexpr int kA = BM * kRowB, kStage = stage_bytes<T, FM>();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave / W, w = wave % W, wm = w % WR, wn = w / WR;
  const int lane = lane_id();
  const int g = lane >> 4, l16 = lane & 15;
  const int nk_all = (p.K + kRowB - 1) / kRowB;
  const int nvalid = (p.K - (nk_all - 1) * kRowB) / 16;  // chunks of the last stage (TAIL: fewer than 8)
  const int nk = (nk_all + KG - 1) / KG;                 // iterations of every group
  const int mine = (nk_all - kg + KG - 1) / KG;          // stages of this one
  constexpr int kCols = SWIGLU ? BN / 2 : BN;            // outputs of a tile
  constexpr int kFrags = SWIGLU ? FN / 2 : FN;           // fragments of a wave's outputs
  const int c0 = nj * kCols;
  MOE_LDS char* const ring = lds + kg * S * kStage;

  typedef Loader<BM, W> LA;
  typedef Loader<BN, W> LB;
  LA la;
  LB lb;
  la.init(a_base, a_bytes, p.K, w, [&](int r) { return src_row(min(r, rows - 1)); });
  lb.init(p.W + int64_t(e) * p.wrows * p.K, int64_t(p.wrows) * p.K, p.K, w, [&](int s) {
    const int col = s / (16 * FN), j = s / 16 % FN, r = s % 16;  // wave column, fragment, row
    const int o = min(c0 + 16 * kFrags * col + channel_of<16 * kFrags>(j % kFrags, r), p.N - 1);
    return j < kFrags ? o : p.up_off + o;
  });
  const uint32_t back = TAIL && LA::chunk(w) >= nvalid ? 16u * uint32_t(LA::chunk(w)) : 0u;
  const int nl = LA::count(w) + LB::count(w);
  auto issue = [&](int st) {
    if (st < mine) {
      MOE_LDS char* d = ring + st % S * kStage;
      const int at = kg + KG * st;
      const uint32_t b = TAIL && at == nk_all - 1 ? back : 0u;
      la.issue(d, w, uint32_t(at) * kRowB, b);
      lb.issue(d + kA, w, uint32_t(at) * kRowB, b);
    }
  };
  // chunks of k that stage st of this group holds
  auto chunks = [&](int st) {
    if (KG > 1 && st >= mine) return 0;
    return TAIL && kg + KG * st == nk_all - 1 ? nvalid : 8;
  };
  // stage s landed for this wave; up to `last` were issued
  constexpr int kMaxAhead = (S - 1) * (LA::kPer + LB::kPer);
  auto wait_stage = [&](int s, int last) {
    __builtin_amdgcn_sched_barrier(0);
    const int n = max(0, min(last, mine - 1) - s) * nl;
    wait_vm_dyn<kMaxAhead>(n);
    __builtin_amdgcn_s_barrier();
    __builtin_amdgcn_sched_barrier(0);
  };
  // fragment addresses: row 16 (WR i + wm) + l16 of A, 16 (FN wn + j) + l16 of
  // B; k step q reads chunk 4 q + g (the swizzle does not depend on i or j)
  uint32_t fa[2], fb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int ra = 16 * wm + l16, rb = 16 * FN * wn + l16;
    fa[q] = uint32_t(ra * kRowB + 16 * chunk_pos(ra, 4 * q + g));
    fb[q] = uint32_t(kA + rb * kRowB + 16 * chunk_pos(rb, 4 * q + g));
  }
  auto read_a = [&](const MOE_LDS char* st, int q, int i) {
    return *reinterpret_cast<const MOE_LDS i32x4*>(st + fa[q] + 16 * WR * kRowB * i);
  };
  auto read_b = [&](const MOE_LDS char* st, int q, int j) {
    return *reinterpret_cast<const MOE_LDS i32x4*>(st + fb[q] + 16 * kRowB * j);
  };

  i32x4 acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = i32x4{0, 0, 0, 0};
  i32x4 a[FM], b[FN];

  for (int st = 0; st < S; ++st) issue(st);
  wait_stage(0, S - 1);
#pragma unroll
  for (int j = 0; j < FN; ++j) b[j] = read_b(ring, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) a[i] = read_a(ring, 0, i);

  constexpr int kH1 = (FM + 1) / 2;
  for (int kt = 0; kt < nk; ++kt) {
    const MOE_LDS char* cur = ring + kt % S * kStage;
    // k beyond K, or beyond the group's stages, counts as zeros (0 times any
    // byte is 0)
    const int have = TAIL || KG > 1 ? chunks(kt) : 8;
    if ((TAIL || KG > 1) && have < 8 && g >= have) {
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = i32x4{0, 0, 0, 0};
    }
    i32x4 bs[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bs[j] = read_b(cur, 1, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma(b[j], a[i], acc[i][j]);
      a[i] = read_a(cur, 1, i);
    }
    alternate_mfma_reads<FM * FN, FN + FM>();
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = bs[j];
    if ((TAIL || KG > 1) && have < 8 && 4 + g >= have) {
#pragma unroll
      for (int i = 0; i < FM; ++i) a[i] = i32x4{0, 0, 0, 0};
    }
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kH1; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma(b[j], a[i], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's reads of stage kt returned; after the barrier every wave's
    // have, and stage kt + 1 is in LDS: stage kt's buffer takes stage kt + S
    dma::wait_lgkm0();
    wait_stage(min(kt + 1, nk - 1), kt + S - 1);
    issue(kt + S);
    const MOE_LDS char* nxt = ring + (kt + 1) % S * kStage;
    i32x4 bn[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bn[j] = read_b(nxt, 0, j);
#pragma unroll
    for (int i = 0; i < kH1; ++i) a[i] = read_a(nxt, 0, i);
#pragma unroll
    for (int i = kH1; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma(b[j], a[i], acc[i][j]);
      a[i] = read_a(nxt, 0, i);
    }
    alternate_mfma_reads<(FM - kH1) * FN, FN + FM>();
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = bn[j];
    __builtin_amdgcn_sched_barrier(0);
  }
  dma::wait_lds_barrier();  // the next tile's loads may overwrite the stages

  if constexpr (KG > 1) {
    // the other groups' sums into the first: [group - 1][wave][fragment][lane]
    static_assert((KG - 1) * W * FM * FN * 1024 <= KG * S * kStage, "the sums fit the stages");
    MOE_LDS i32x4* const sums = (MOE_LDS i32x4*)lds;
    if (kg > 0) {
#pragma unroll
      for (int i = 0; i < FM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) sums[((((kg - 1) * W + w) * FM + i) * FN + j) * 64 + lane] = acc[i][j];
    }
    dma::wait_lds_barrier();
    if (kg == 0) {
#pragma unroll
      for (int q = 0; q < KG - 1; ++q)
#pragma unroll
        for (int i = 0; i < FM; ++i)
#pragma unroll
          for (int j = 0; j < FN; ++j) acc[i][j] += sums[(((q * W + w) * FM + i) * FN + j) * 64 + lane];
    }
    dma::wait_lds_barrier();
    if (kg > 0) return;
  }

  // lane group g holds 4 kFrags consecutive outputs of row l16 of a fragment,
  // 4 per fragment j
  const float* sw = p.sw + int64_t(e) * p.wrows;
  const int col = c0 + 16 * kFrags * wn + 4 * kFrags * g;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = 16 * (WR * i + wm) + l16;
    if (row >= rows) continue;
    const float sa = p.sa[p.gather_src ? p.gather_src[r0 + row] / p.gather_k : r0 + row];
    if constexpr (SWIGLU) {
#pragma unroll
      for (int j = 0; j < kFrags; ++j)
        if (col + 4 * j < p.N)
          store4_swiglu(p, r0 + row, col + 4 * j, acc[i][j], acc[i][j + kFrags], sa,
                        *reinterpret_cast<const float4*>(sw + col + 4 * j),
                        *reinterpret_cast<const float4*>(sw + p.up_off + col + 4 * j));
    } else {
#pragma unroll
      for (int j = 0; j + 1 < kFrags; j += 2)
        if (col + 4 * j < p.N)  // N is a multiple of 8, and so is col
          store8(p, r0 + row, col + 4 * j, acc[i][j], acc[i][j + 1], sa,
                 *reinterpret_cast<const float4*>(sw + col + 4 * j),
                 *reinterpret_cast<const float4*>(sw + col + 4 * j + 4));
      if constexpr (kFrags == 1)
        if (col < p.N) store4(p, r0 + row, col, acc[i][0], sa, *reinterpret_cast<const float4*>(sw + col));
    }
  }
}

// Largest tile: 2 x 4 waves, 256 channels, blocks of up to 288 rows.
typedef Shape<2, 4, 4, 2, 1> Big;
constexpr int kBigFM = 9;
// 128 rows x 128 channels, 8 waves for a group of k. Up to one tile per CU: four
// stages (Mid), or for a long k two groups with two stages each (MidK). More
// tiles: two stages and two workgroups per CU, so that one streams while the
// other starts or ends a tile (Mid2).
typedef Shape<2, 4, 2, 4, 1> Mid;
typedef Shape<2, 4, 2, 2, 2> MidK;
typedef Shape<2, 4, 2, 2, 1> Mid2;
constexpr int kMidFM = 4;
// Fewer tiles, whose time is the number of stages one after another: 64 x 128 in
// two groups of 4 waves, 64 x 64 in four.
typedef Shape<2, 2, 4, 3, 2> Mid64;
typedef Shape<2, 2, 2, 2, 4> Small;
constexpr int kSmallFM = 2;

// Few rows, where only the weight stream counts: 16 or 32 rows x 64 channels,
// two groups of k and two workgroups per CU, so that one streams while the
// other starts or ends a tile (Stream; 64 rows: Stream64); with few tiles, 16
// rows x 32 channels with eight groups (Narrow), or x 64 with four for gate/up.
typedef Shape<1, 2, 2, 3, 2> Stream;
typedef Shape<1, 2, 2, 2, 2> Stream64;  // 64 rows
constexpr int kStreamLocal = 256;  // local experts (two workgroups fill the LDS)
typedef Shape<1, 2, 1, 3, 8> Narrow;
typedef Shape<1, 2, 2, 3, 4> NarrowGU;    // 16 or 32 rows
typedef Shape<1, 2, 1, 2, 8> Narrow32;    // 32 rows x 32 channels
typedef Shape<2, 2, 1, 3, 4> Narrow64;    // 64 rows x 32 channels

// Row caps of the largest tile (the fewest rounds of the grid win, weighted by
// the tallest block, as in the bf16 grouped GEMM); the others have one.
constexpr int kRowCaps = 6;
__device__ constexpr int kRowCap[kRowCaps] = {288, 256, 224, 192, 160, 128};
constexpr int kRowCapMin = 128;

// MAXE: local experts its tables hold.
template <typename T, int FMMAX, int MAXE, bool SWIGLU, bool TAIL>
__global__ void __launch_bounds__(64 * T::W * T::KG) tile_kernel(GemmArgs p) {
  constexpr int kThreads = 64 * T::W * T::KG;
  constexpr bool kVary = FMMAX == kBigFM;  // block heights vary: a row cap is chosen
  constexpr int kBM = 16 * FMMAX * T::WR;
  __shared__ __attribute__((aligned(1024))) char smem[T::KG * T::S * stage_bytes<T, FMMAX>()];
  __shared__ int s_off[MAXE + 1];
  __shared__ int s_tpre[MAXE];
  __shared__ int s_tmp[T::W * T::KG];
  __shared__ unsigned long long s_ntile[kRowCaps];
  __shared__ int s_cand[kRowCaps];
  MOE_LDS char* lds = (MOE_LDS char*)smem;
  constexpr int kCols = SWIGLU ? T::BN / 2 : T::BN;
  const int ntn = (p.N + kCols - 1) / kCols;
  constexpr int kPerT = (MAXE + kThreads - 1) / kThreads;
  int row_cap = kBM, total = 0;
  int only0 = 0, only_rows = 0;  // the one segment of a launch without tables
  const bool tables = p.E_local > 1;
  if (!tables) {
    int end;
    segment(p, 0, only0, end);
    only_rows = end - only0;
    if constexpr (kVary) {
      unsigned long long best = ~0ull;
#pragma unroll
      for (int c = 0; c < kRowCaps; ++c) {
        const int nrt = max(1, (only_rows + kRowCap[c] - 1) / kRowCap[c]);
        const unsigned long long tl = (unsigned long long)nrt * (unsigned long long)ntn;
        const int hm = (((only_rows + nrt - 1) / nrt) + 15) & ~15;
        const unsigned long long est = (tl + gridDim.x - 1) / gridDim.x * (unsigned long long)(hm + T::BN);
        if (tl < (1ull << 31) && est < best) {
          best = est;
          row_cap = kRowCap[c];
        }
      }
    }
    total = (only_rows + row_cap - 1) / row_cap * ntn;
  } else {
  int me[kPerT];
#pragma unroll
  for (int q = 0; q < kPerT; ++q) {
    const int i = int(threadIdx.x) * kPerT + q;
    me[q] = 0;
    if (i < p.E_local) {
      int a, b;
      segment(p, i, a, b);
      s_off[i] = a;
      me[q] = b - a;
      if (i == p.E_local - 1) s_off[p.E_local] = b;
    }
  }
  if constexpr (kVary) {
    if (threadIdx.x < kRowCaps) {
      s_ntile[threadIdx.x] = 0;
      s_cand[threadIdx.x] = 0;
    }
    __syncthreads();
#pragma unroll
    for (int c = 0; c < kRowCaps; ++c) {
      unsigned long long tl = 0;
      int hm = 0;
#pragma unroll
      for (int q = 0; q < kPerT; ++q) {
        if (me[q] > 0) {
          const int nrt = (me[q] + kRowCap[c] - 1) / kRowCap[c];
          tl += (unsigned long long)nrt * (unsigned long long)ntn;
          hm = max(hm, (((me[q] + nrt - 1) / nrt) + 15) & ~15);
        }
      }
      if (tl > 0) atomicAdd(&s_ntile[c], tl);
      if (hm > 0) atomicMax(&s_cand[c], hm);
    }
    __syncthreads();
    unsigned long long best = ~0ull;
    row_cap = kRowCap[0];
#pragma unroll
    for (int c = 0; c < kRowCaps; ++c) {
      const unsigned long long tl = s_ntile[c];
      if (tl >= (1ull << 31)) continue;
      const unsigned long long est = (tl + gridDim.x - 1) / gridDim.x * (unsigned long long)(s_cand[c] + T::BN);
      if (est < best) {
        best = est;
        row_cap = kRowCap[c];
      }
    }
  }
  int mt[kPerT];
  int sum = 0;
#pragma unroll
  for (int q = 0; q < kPerT; ++q) {
    mt[q] = (me[q] + row_cap - 1) / row_cap * ntn;
    sum += mt[q];
  }
  int pre = block_exclusive_scan<kThreads>(sum, s_tmp, total);
#pragma unroll
  for (int q = 0; q < kPerT; ++q) {
    const int i = int(threadIdx.x) * kPerT + q;
    if (i < p.E_local) s_tpre[i] = pre;
    pre += mt[q];
  }
  __syncthreads();
  }

  // each XCD takes a contiguous range of the tiles (workgroup b runs on XCD
  // b % 8); inside an expert, groups of 8 row blocks walk the channel tiles
  // together, so the tiles an XCD works on at a time share both operands
  constexpr int kGroup = 8;
  const int xcd = blockIdx.x % 8, per_xcd = gridDim.x / 8;
  const int lo_t = int((int64_t(total) * xcd) / 8), hi_t = int((int64_t(total) * (xcd + 1)) / 8);
  for (int tile = lo_t + int(blockIdx.x / 8); tile < hi_t; tile += per_xcd) {
    int e = 0, seg0 = only0, m_e = only_rows, first = 0;
    if (tables) {
      int lo = 0, hi = p.E_local - 1;
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (s_tpre[mid] <= tile)
          lo = mid;
        else
          hi = mid - 1;
      }
      e = __builtin_amdgcn_readfirstlane(lo);
      seg0 = __builtin_amdgcn_readfirstlane(s_off[e]);
      m_e = __builtin_amdgcn_readfirstlane(s_off[e + 1]) - seg0;
      first = __builtin_amdgcn_readfirstlane(s_tpre[e]);
    }
    const int nrt = (m_e + row_cap - 1) / row_cap;
    const int local = tile - first;
    const int grp = local / (kGroup * ntn);
    const int in_grp = min(kGroup, nrt - grp * kGroup);
    const int rest = local - grp * kGroup * ntn;
    const int nj = rest / in_grp;
    const int mi = grp * kGroup + rest - nj * in_grp;
    const int height = ((m_e + nrt - 1) / nrt + 15) & ~15;
    const int r0 = seg0 + mi * height;
    const int rows = min(height, seg0 + m_e - r0);
    if (rows <= 0) continue;
    auto go = [&](auto fm_t) {
      constexpr int FM = decltype(fm_t)::value;
      if (p.gather_src != nullptr)
        run_tile<T, FM, SWIGLU, TAIL>(lds, p, p.A, int64_t(p.gather_rows) * p.K,
                                      [&](int r) { return p.gather_src[r0 + r] / p.gather_k; }, rows, r0, e, nj);
      else
        run_tile<T, FM, SWIGLU, TAIL>(lds, p, p.A + int64_t(r0) * p.K, int64_t(rows) * p.K, [](int r) { return r; },
                                      rows, r0, e, nj);
    };
    if constexpr (kVary) {
      switch ((rows + 16 * T::WR - 1) / (16 * T::WR)) {
        case 1: case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: case 4: go(std::integral_constant<int, 4>{}); break;
        case 5: go(std::integral_constant<int, 5>{}); break;
        case 6: go(std::integral_constant<int, 6>{}); break;
        case 7: go(std::integral_constant<int, 7>{}); break;
        case 8: go(std::integral_constant<int, 8>{}); break;
        default: go(std::integral_constant<int, 9>{}); break;
      }
    } else {
      go(std::integral_constant<int, FMMAX>{});
    }
  }
}

// Which tiles a launch takes (names as the shapes above; 16, 32, 64: rows of a
// block), by its sizes and the rows a segment is expected to hold.
enum Tile { kStream16, kStream32, kStream64, kNarrow, kNarrow32, kNarrow64, kSmall, kMid64, kMid, kMidK, kMid2, kBig };

Tile pick_tile(bool swiglu, bool ragged, int E_local, int64_t capacity, int N, int K, int64_t rows_hint, int64_t cus) {
  const int d = swiglu ? 2 : 1;  // channels of an output
  // segments that can have rows
  const int64_t active = std::min<int64_t>(E_local, capacity);
  auto tiles = [&](int bm, int outputs) { return ceil_div(rows_hint, bm) * active * ceil_div(N, outputs); };
  // Ragged segments spread around the expected length: twice as many rows as
  // expected still make one block, and a block in two is a segment's last.
  const int64_t rows = std::min(ragged ? 2 * rows_hint : rows_hint, capacity);
  auto blocks = [&](int bm) {
    const int64_t tall = std::min(ragged ? rows_hint + rows_hint / 4 : rows_hint, capacity);
    return std::min(ceil_div(tall, bm) * active, ceil_div(rows_hint * active, bm) + active / 2);
  };
  // Streams from the first narrow tile (32 outputs) beyond one per CU: a second
  // round of those costs more (us, narrow / stream: 16 experts of 2880 x 768, 61
  // rows 34.4 / 31.2; 5 rows 8.1 / 5.3; 1 x 7168 x 10240 16.7 / 14.3; 17 x 2048 x
  // 16384 14.0 / 8.5).
  const bool streams = E_local <= kStreamLocal;
  if (rows <= 16 && streams && tiles(16, 32) > cus) return kStream16;
  if (rows <= 32 && streams && tiles(32, 32) > cus) return kStream32;
  // blocks of 16 rows also for 17 to 32: twice the tiles, and both blocks of a
  // weight tile read it at the same time (32 x 7168 x 4096: 10.7 -> 8.6 us; two
  // rounds of them, 17 x 7168 x 8192: 14.2, streams 17.1)
  if (rows <= 32) return kNarrow;
  if (rows <= 64 && streams && tiles(64, 64 / d) > cus) return kStream64;
  // The smallest tiles of which each CU gets one at most. (us: 64 x 7168 x 4096
  // Narrow 14.1, Narrow32 11.0, Narrow64 13.6, Small 17.8; 128 x 7168 x 4096 25.3,
  // 18.5, 14.3, 17.7; 128 x 7168 x 1024 8.4, 10.2, 13.8, 16.8; 512 rows 1408 x 2048
  // Small 7.7, Mid64 9.4; 640 rows Small 11.6, Mid64 9.5; 512 rows 7168 x 4096
  // Small 34, Mid64 28, Mid 35; 1024 rows MidK 37; 1280 rows 768 x 2048 Mid 8.7,
  // MidK 9.8.)
  auto once = [&](int bm, int outputs) { return blocks(bm) * ceil_div(N, outputs) <= cus; };
  if (once(16, 32)) return kNarrow;
  if (once(32, 32)) return kNarrow32;
  if (!swiglu && once(64, 32)) return kNarrow64;
  if (once(64, 64 / d)) return kSmall;
  if (once(64, 128 / d)) return kMid64;
  // The largest tiles read the fewest operand bytes, but one at a time per CU:
  // they need rows to fill them and a long k, or very many tiles. (us, Mid2 / Big,
  // 32 experts, K x N: 96 rows 7168 x 4096 192 / 214, 128 rows 273 / 221, 512 rows
  // 595 / 447; 2880 x 2880 68 / 88, 99 / 91, 227 / 167; 1408 x 2048 22 / 33,
  // 32 / 34, 66 / 70; 64 experts 1408 x 2048, 512 rows: 156 / 142.)
  const int64_t mid = blocks(128) * ceil_div(N, 128 / d);
  if (rows_hint >= 128 && mid > 2 * cus && (K >= 2048 || mid * K >= (int64_t(5) << 20))) return kBig;
  // (2048 x 7168 x 4096: Mid 75 us, Mid2 56, Big 58; 1024 x 7168 x 4096: Mid 38, Mid2 40)
  if (mid > cus) return kMid2;
  return K > 2048 ? kMidK : kMid;
}

template <bool SWIGLU>
hipError_t launch_gemm(const GemmArgs& p, int64_t rows_hint, hipStream_t stream) {
  const bool tail = p.K % kRowB != 0;
  const int64_t cus = device_cu_count() / 8 * 8;
  constexpr int d = SWIGLU ? 2 : 1;
  auto go = [&](auto shape, auto fm_t, auto maxe_t, int bm, int per_cu) {
    typedef decltype(shape) T;
    constexpr int FM = decltype(fm_t)::value, MAXE = decltype(maxe_t)::value;
    const int64_t n = (ceil_div(p.capacity, bm) + p.E_local) * ceil_div(p.N, T::BN / d);
    // the kernels index tiles with 31 bits
    if (n >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    const unsigned grid = unsigned(std::max<int64_t>(8, std::min<int64_t>(cus * per_cu, ceil_div(n, 8) * 8)));
    auto* kern = tail ? tile_kernel<T, FM, MAXE, SWIGLU, true> : tile_kernel<T, FM, MAXE, SWIGLU, false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * T::W * T::KG), 0, stream, p);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, kMaxLocal> AnyE;
  typedef std::integral_constant<int, kStreamLocal> StreamE;
  typedef std::integral_constant<int, 1> One;
  typedef std::integral_constant<int, 2> Two;
  typedef std::integral_constant<int, 4> Four;
  typedef std::integral_constant<int, kSmallFM> SmallFM;
  typedef std::integral_constant<int, kMidFM> MidFM;
  typedef std::conditional_t<SWIGLU, NarrowGU, Narrow> Narrow16;
  switch (pick_tile(SWIGLU, p.offsets != nullptr, p.E_local, p.capacity, p.N, p.K, rows_hint, cus)) {
    case kStream16: return go(Stream{}, One{}, StreamE{}, 16, 2);
    case kStream32: return go(Stream{}, Two{}, StreamE{}, 32, 2);
    case kStream64: return go(Stream64{}, Four{}, StreamE{}, 64, 2);
    case kNarrow: return go(Narrow16{}, One{}, AnyE{}, 16, 1);
    case kNarrow32: return go(std::conditional_t<SWIGLU, NarrowGU, Narrow32>{}, Two{}, AnyE{}, 32, 1);
    case kNarrow64:
      if constexpr (!SWIGLU) return go(Narrow64{}, Two{}, AnyE{}, 64, 1);
      return hipErrorInvalidValue;
    case kSmall: return go(Small{}, SmallFM{}, AnyE{}, 64, 1);
    case kMid64: return go(Mid64{}, SmallFM{}, AnyE{}, 64, 1);
    case kMid: return go(Mid{}, MidFM{}, AnyE{}, 128, 1);
    case kMidK: return go(MidK{}, MidFM{}, AnyE{}, 128, 1);
    case kMid2: return go(Mid2{}, MidFM{}, AnyE{}, 128, 2);
    case kBig: return go(Big{}, std::integral_constant<int, kBigFM>{}, AnyE{}, kRowCapMin, 1);
  }
  return hipErrorInvalidValue;
}

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------
// q = 127 v / top rounded to the nearest integer, halves to even. A row whose
// top is below 2^-64 (or above 2^64) is multiplied by 2^64 (2^-64) first, which
// keeps the reciprocal and 127 v finite and normal.
//
// bf16 values: 127 v is exact, and the quotient of the reciprocal estimate is
// corrected once by its exact remainder (fma); it is a half or at least 2^-9
// away from one, so its rounding decides right.
// float32 values: 127 v has 31 bits and the quotient can lie closer to a half
// than its own last bit, so the half is compared exactly: m = floor(127 v / top)
// to within one, and 254 v (as hi + lo) against (2 m + 1) top. hi - (2 m + 1)
// top is exact where it is small, and where it is not, lo does not change its
// sign.
struct RowScale {
  float lift, top, rcp, scale;
  bool zero;  // q = 0 throughout: top is 0, infinite or NaN
  __device__ __forceinline__ explicit RowScale(uint32_t top_bits) {
    const float t = __uint_as_float(top_bits);
    lift = t < 0x1p-64f ? 0x1p64f : t > 0x1p64f ? 0x1p-64f : 1.f;
    top = t * lift;
    rcp = 1.f / top;
    scale = t / 127.f;
    zero = !(t > 0.f) || top_bits >= 0x7F800000u;
  }
  template <bool F32 = false>
  __device__ __forceinline__ int q(float v) const {
    if constexpr (F32) {
      const float vl = v * lift, hi = vl * 254.f, lo = fmaf(vl, 254.f, -hi);
      const float m = floorf(0.5f * hi * rcp);
      const float over = fmaf(-fmaf(2.f, m, 1.f), top, hi) + lo;
      const int f = int(m);
      return zero ? 0 : f + (over > 0.f || (over == 0.f && (f & 1)) ? 1 : 0);
    } else {
      const float n = v * lift * 127.f;
      const float t = n * rcp;
      const float r = fmaf(-t, top, n);
      return zero ? 0 : int(rintf(fmaf(r, rcp, t)));
    }
  }
};

__device__ __forceinline__ uint32_t pack4(int a, int b, int c, int d) {
  return uint32_t(a & 0xFF) | (uint32_t(b & 0xFF) << 8) | (uint32_t(c & 0xFF) << 16) | (uint32_t(d) << 24);
}

// Largest |value| of a row as its bits (NaN above infinity above the rest).
__device__ __forceinline__ uint32_t abs_bits(float f) { return __float_as_uint(f) & 0x7FFFFFFFu; }
__device__ __forceinline__ uint32_t block_max(uint32_t v, uint32_t* s_red) {
#pragma unroll
  for (int m = 32; m >= 1; m >>= 1) v = max(v, uint32_t(__shfl_xor(int(v), m, 64)));
  if (lane_id() == 0) s_red[threadIdx.x >> 6] = v;
  __syncthreads();
  const int nw = blockDim.x >> 6;
  uint32_t t = 0;
  for (int i = 0; i < nw; ++i) t = max(t, s_red[i]);
  return t;
}

template <bool F32>
__device__ __forceinline__ void load8(float (&o)[8], const void* base, int64_t vec) {
  if constexpr (F32) {
    const float4* p = static_cast<const float4*>(base) + 2 * vec;
    const float4 a = p[0], b = p[1];
    o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
    o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
  } else {
    const u32x4 v = static_cast<const u32x4*>(base)[vec];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      o[2 * i] = bf16_lo(v[i]);
      o[2 * i + 1] = bf16_hi(v[i]);
    }
  }
}

// One workgroup per row: its NV vectors of 8 per thread are read once and kept
// (NV = 0: a row wider than 4 vectors of 1024 threads is read twice). END: rows
// at and past *end (device memory) are left alone, and not read either, but for
// `ahead`, a call of few rows, where the first row is asked for before *end
// arrives. (One kernel with and without an end takes 37.0 us for 8192 x 7168,
// this one 36.4.)
template <bool F32, int NV, bool END>
__global__ void __launch_bounds__(1024) quantize_rows_kernel(const void* x, const int32_t* end, int M, int nvec,
                                                             bool ahead, int8_t* q, float* scale) {
  __shared__ uint32_t s_red[16];
  constexpr int kKeep = NV ? NV : 1;
  float v[kKeep][8];
  auto load_row = [&](int64_t m) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = int(threadIdx.x) + i * int(blockDim.x);
      if (c < nvec) load8<F32>(v[i], x, m * nvec + c);
    }
  };
  int64_t m = blockIdx.x;
  if (!END || ahead) load_row(m);  // (m < M: in the array even if it lies past *end)
  const int64_t rows = END ? min(M, *end) : M;
  if (END && !ahead && m < rows) load_row(m);
  while (m < rows) {
    uint32_t top = 0;
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i)
        if (int(threadIdx.x) + i * int(blockDim.x) < nvec)
#pragma unroll
          for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[i][j]));
    } else {
      for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
        load8<F32>(v[0], x, m * nvec + c);
#pragma unroll
        for (int j = 0; j < 8; ++j) top = max(top, abs_bits(v[0][j]));
      }
    }
    const RowScale rs(block_max(top, s_red));
    if (threadIdx.x == 0) scale[m] = rs.scale;
    auto put = [&](const float (&f)[8], int c) {
      int n[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) n[j] = rs.template q<F32>(f[j]);
      reinterpret_cast<uint2*>(q)[m * nvec + c] = make_uint2(pack4(n[0], n[1], n[2], n[3]), pack4(n[4], n[5], n[6], n[7]));
    };
    if constexpr (NV > 0) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = int(threadIdx.x) + i * int(blockDim.x);
        if (c < nvec) put(v[i], c);
      }
    } else {
      for (int c = threadIdx.x; c < nvec; c += blockDim.x) {
        load8<F32>(v[0], x, m * nvec + c);
        put(v[0], c);
      }
    }
    m += gridDim.x;
    if (m < rows) load_row(m);
    __syncthreads();  // s_red is free again
  }
}

template <bool F32>
hipError_t launch_quantize(const void* x, const int32_t* end, int64_t M, int K, int8_t* q, float* scale,
                           hipStream_t stream) {
  const int nvec = K / 8;
  // one vector per thread for few rows (the shortest chain), two up to 1024
  // vectors for many, so that several rows share a CU
  const bool many = M > 2 * device_cu_count();
  // Of a large capacity's rows most can lie past *end, so none is asked for ahead
  // and the workgroups are 16 per CU, not one per row (MLPs, us, with both / with
  // a workgroup per row / with its row asked for ahead too: 16 rows of 65536, 32
  // experts of 4096 x 4096: 225 / 249 / 464; 16384 rows of 131072, 7168 x 2048:
  // 800 / 854 / 1187; all 16384 rows there: 802 / 804 / 805).
  const bool bounded = end != nullptr && many, ahead = !bounded;
  const int nv = nvec <= (many ? 256 : 1024) ? 1 : nvec <= 1024 ? 2 : nvec <= 4096 ? 4 : 0;
  const int nt = nv ? int(ceil_div(ceil_div(nvec, nv), 64) * 64) : 1024;
  const dim3 grid(unsigned(std::min<int64_t>(M, bounded ? 16 * device_cu_count() : kMaxGrid)));
  const dim3 block(static_cast<unsigned>(nt));
  auto go = [&](auto nv_t) {
    constexpr int NV = decltype(nv_t)::value;
    auto* kern = quantize_rows_kernel<F32, NV, true>;
    if constexpr (!F32)  // (float32 rows are h, whose count is always on the device)
      if (end == nullptr) kern = quantize_rows_kernel<F32, NV, false>;
    hipLaunchKernelGGL(kern, grid, block, 0, stream, x, end, int(M), nvec, ahead, q, scale);
  };
  if (nv == 1)
    go(std::integral_constant<int, 1>{});
  else if (nv == 2)
    go(std::integral_constant<int, 2>{});
  else if (nv == 4)
    go(std::integral_constant<int, 4>{});
  else
    go(std::integral_constant<int, 0>{});
  return hipGetLastError();
}

// Weights [K, N] bf16 of one expert -> [N, K] int8 and a scale per channel.
// A workgroup takes 64 channels: the largest |w| of each over all k, then the
// values again (from L2 mostly), turned 64 k x 64 channels at a time in LDS so
// that both sides move in 16-byte vectors. Run once per checkpoint.
__global__ void __launch_bounds__(256) quantize_weights_kernel(const uint16_t* w, int E_local, int K, int N,
                                                               int8_t* q, float* scale) {
  __shared__ uint32_t s_top[32][64 + 1];
  __shared__ uint32_t s_max[64];
  __shared__ __attribute__((aligned(16))) int8_t s_t[64][64 + 16];
  const int panels = (N + 63) / 64;
  for (int64_t panel = blockIdx.x; panel < int64_t(E_local) * panels; panel += gridDim.x) {
  const int e = int(panel / panels), n0 = int(panel - int64_t(e) * panels) * 64;
  const uint16_t* we = w + int64_t(e) * K * N;
  const int cg = threadIdx.x & 7, kr = threadIdx.x >> 3;  // 8 channel groups of 8 x 32 k rows
  const int n = n0 + 8 * cg;                              // N is a multiple of 8: a group is inside or outside
  uint32_t top[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (n < N)
    for (int k = kr; k < K; k += 32) {
      float v[8];
      load8<false>(v, we + int64_t(k) * N + n, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) top[j] = max(top[j], abs_bits(v[j]));
    }
#pragma unroll
  for (int j = 0; j < 8; ++j) s_top[kr][8 * cg + j] = top[j];
  __syncthreads();
  if (threadIdx.x < 64) {
    uint32_t t = 0;
    for (int r = 0; r < 32; ++r) t = max(t, s_top[r][threadIdx.x]);
    s_max[threadIdx.x] = t;
    if (n0 + int(threadIdx.x) < N) scale[int64_t(e) * N + n0 + threadIdx.x] = RowScale(t).scale;
  }
  __syncthreads();
  const RowScale rs[8] = {RowScale(s_max[8 * cg]),     RowScale(s_max[8 * cg + 1]), RowScale(s_max[8 * cg + 2]),
                          RowScale(s_max[8 * cg + 3]), RowScale(s_max[8 * cg + 4]), RowScale(s_max[8 * cg + 5]),
                          RowScale(s_max[8 * cg + 6]), RowScale(s_max[8 * cg + 7])};
  for (int k0 = 0; k0 < K; k0 += 64) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int k = k0 + kr + 32 * h;
      float v[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
      if (n < N && k < K) load8<false>(v, we + int64_t(k) * N + n, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) s_t[8 * cg + j][kr + 32 * h] = int8_t(rs[j].q(v[j]));
    }
    __syncthreads();
    // channel threadIdx.x / 4, 16 k each (K is a multiple of 16)
    const int c = threadIdx.x >> 2, kk = 16 * (threadIdx.x & 3);
    if (n0 + c < N && k0 + kk < K)
      *reinterpret_cast<u32x4*>(q + (int64_t(e) * N + n0 + c) * K + k0 + kk) =
          *reinterpret_cast<const u32x4*>(&s_t[c][kk]);
    __syncthreads();
  }
  }
}

}  // namespace i8

int i8_tile(bool swiglu, bool ragged, int E_local, int64_t capacity, int N, int K, int64_t rows_hint, int cus) {
  return int(i8::pick_tile(swiglu, ragged, E_local, capacity, N, K, rows_hint, cus));
}

hipError_t launch_quantize_rows(const void* x, bool x_f32, const int32_t* end, int64_t M, int K, int8_t* q,
                                float* scale, hipStream_t stream) {
  return x_f32 ? i8::launch_quantize<true>(x, end, M, K, q, scale, stream)
               : i8::launch_quantize<false>(x, end, M, K, q, scale, stream);
}

hipError_t launch_quantize_weights(const uint16_t* w, int E_local, int K, int N, int8_t* q, float* scale,
                                   hipStream_t stream) {
  hipLaunchKernelGGL(i8::quantize_weights_kernel, dim3(unsigned(std::min<int64_t>(E_local * ceil_div(N, 64), i8::kMaxGrid))),
                     dim3(256), 0, stream, w, E_local, K, N, q, scale);
  return hipGetLastError();
}

hipError_t launch_gemm_i8(const int8_t* A, const float* sa, const int32_t* offsets, int E_local, int64_t capacity,
                          const int8_t* W, const float* sw, int K, int N, uint16_t* C, int64_t rows_hint,
                          hipStream_t stream) {
  return i8::launch_gemm<false>({A, sa, nullptr, 1, 0, offsets, E_local, capacity, W, sw, N, K, N, 0, C}, rows_hint,
                                stream);
}

hipError_t launch_gate_up_i8(const int8_t* A, const float* sa, const int32_t* gather_src, int gather_k,
                             int gather_rows, const int32_t* offsets, int E_local, int64_t capacity, const int8_t* W,
                             const float* sw, int H, int I, float* h, int64_t rows_hint, hipStream_t stream) {
  return i8::launch_gemm<true>({A, sa, gather_src, gather_k, gather_rows, offsets, E_local, capacity, W, sw, 2 * I, H,
                                I, I, h},
                               rows_hint, stream);
}

}  // namespace moe

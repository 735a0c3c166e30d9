// bf16 products with bias, activation and residual in the epilogue, for one
// weight matrix or for ragged expert segments:
//
//   C[m] = act(A[m] W_e + bias_e) + residual[m]
//
// float32 sums and epilogue, one rounding at the end.
//
// The weights are [k][n] as the share's are. Both operands come through LDS by
// direct-to-LDS loads in stages of 64 k: rows of A as 128-byte lines with
// swizzled 16-byte chunks, W as 4 x 16 blocks of 128 bytes that
// ds_read_b64_tr_b16 hands out transposed (gemm_dma.h has both layouts). The weights
// are the first operand of v_mfma_f32_16x16x32_bf16, so a lane ends with 4
// consecutive columns of one row.
//
// One kernel in a dozen tile shapes, from 16 x 32 (few rows: the weight stream
// is the whole cost) to 288 x 256.
#include "gemm_dma.h"
#include "gemm_tile.h"
#include "moe_kernels.h"
#include "moe_row.h"

namespace moe {
namespace bfgemm {

using dma::dma16;
using dma::panel::b_swz;
using dma::panel::f32x4v;
using dma::panel::mfma16x16x32;
typedef dma::i32x4 i32x4;

constexpr int kMaxLocal = 1024;
constexpr int kSK = 64;          // k per stage
constexpr int kRowB = 2 * kSK;   // bytes of a row of A in it

__device__ __forceinline__ void segment(const GemmBf16& p, int e, int& a, int& b) {
  if (p.offsets == nullptr) {
    a = 0;
    b = int(p.capacity);
    return;
  }
  const int64_t lo = min<int64_t>(max<int64_t>(p.offsets[e], 0), p.capacity);
  a = int(lo);
  b = int(max<int64_t>(lo, min<int64_t>(p.offsets[e + 1], p.capacity)));
}

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ float activate(int kind, float z) {
  switch (kind) {
    case 1: return z > 0.f ? z : z == z ? 0.f : z;
    case 2: return silu(z);
    // 1 + erf and 1 + tanh cancel for z < 0
    case 3: return 0.5f * z * erfcf(z * -0.70710678f);
    default: return z / (1.f + expf(-1.5957691f * (z + 0.044715f * z * z * z)));
  }
}

// ---------------------------------------------------------------------------
// Tiles through LDS
// ---------------------------------------------------------------------------
__device__ __forceinline__ int chunk_pos(int r, int c) { return c ^ ((r >> 1) & 7); }

// ROWS rows of A x 64 k: load i W + w (8 rows, 8 lanes each) is wave w's. Row r
// sits at 128 r, its 16-byte chunk c at c ^ ((r >> 1) & 7) (conflict-free for
// 16 lanes reading one chunk of 16 consecutive rows).
template <int ROWS, int W>
struct LoaderA {
  static constexpr int kLoads = ROWS / 8;
  static constexpr int kPer = (kLoads + W - 1) / W;
  static_assert(W % 2 == 0, "a lane's chunk does not depend on the load");
  i32x4 rsrc;
  uint32_t voff[kPer];
  __device__ __forceinline__ static int count(int w) { return (kLoads - w + W - 1) / W; }
  // the chunk this lane fetches in every load
  __device__ __forceinline__ static int chunk(int w) {
    const int lane = lane_id();
    return (lane & 7) ^ ((4 * (w & 1) + (lane >> 4)) & 7);
  }
  __device__ __forceinline__ void init(const uint16_t* base, int K, int rows, int w) {
    rsrc = dma::buffer_rsrc(base, int64_t(rows) * K * 2);
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      voff[i] = uint32_t(min(8 * (i * W + w) + (lane_id() >> 3), rows - 1)) * uint32_t(K) * 2u + 16u * uint32_t(chunk(w));
  }
  // valid: chunks of the stage that lie before the end of K; the lanes of the
  // others read its first chunk instead, inside their row
  template <bool TAIL>
  __device__ __forceinline__ void issue(MOE_LDS char* dst, int w, int stage, int valid) const {
    const uint32_t back = TAIL && chunk(w) >= valid ? 16u * uint32_t(chunk(w)) : 0u;
#pragma unroll
    for (int i = 0; i < kPer; ++i)
      if (kLoads % W == 0 || i * W + w < kLoads)
        dma16(rsrc, voff[i] - back, uint32_t(stage) * kRowB, dst + 1024 * (i * W + w));
  }
};

// 64 k x BN columns of W: block (kq, nq) = k 4 kq .. +3, columns 16 nq .. +15 at
// position kq BN / 16 + (nq ^ b_swz(kq)); load j W + w fills 8 positions.
template <int BN, int W>
struct LoaderB {
  static constexpr int kNQ = BN / 16;
  static constexpr int kLoads = BN / 8;
  static constexpr int kPer = (kLoads + W - 1) / W;
  static_assert(kNQ % 2 == 0, "pairs of blocks take the two halves of the banks");
  i32x4 rsrc;
  uint32_t voff[kPer];
  uint32_t ld;  // bytes of a row
  __device__ __forceinline__ static int count(int w) { return (kLoads - w + W - 1) / W; }
  __device__ __forceinline__ static int block(int j, int w) { return 8 * (j * W + w) + (lane_id() >> 3); }
  __device__ __forceinline__ static int row(int j, int w) { return 4 * (block(j, w) / kNQ) + ((lane_id() & 7) >> 1); }
  template <typename ColOf>
  __device__ __forceinline__ void init(const uint16_t* mat, int K, int cols, int w, ColOf col_of) {
    rsrc = dma::buffer_rsrc(mat, int64_t(K) * cols * 2);
    ld = 2u * uint32_t(cols);
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
      const int b = block(j, w), nq = (b % kNQ) ^ b_swz(b / kNQ);
      voff[j] = uint32_t(row(j, w)) * ld + 2u * uint32_t(col_of(16 * nq + 8 * (lane_id() & 1)));
    }
  }
  // (past the end of K a lane reads one of the stage's first 8 rows instead)
  template <bool TAIL>
  __device__ __forceinline__ void issue(MOE_LDS char* dst, int w, int stage, int valid) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (kLoads % W == 0 || j * W + w < kLoads) {
        const int r = row(j, w);
        const uint32_t back = TAIL && r >= 8 * valid ? uint32_t(r & ~7) * ld : 0u;
        dma16(rsrc, voff[j] - back, uint32_t(stage) * kSK * ld, dst + 1024 * (j * W + w));
      }
  }
};

// Ask the scheduler for one LDS read after each MFMA while reads remain.
template <int NM, int NR>
__device__ __forceinline__ void alternate_mfma_reads() {
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
    if (i < NR) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
  }
#pragma unroll
  for (int i = NM; i < NR; ++i) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
}

// KG groups of WR x WC waves; a tile is 16 FM WR rows x 16 FN WC columns, S
// stages in LDS per group. Group q takes k stages q, q + KG, ..; the groups'
// sums meet in LDS, in the order of the groups. 16-row fragment f belongs to wave
// row f % WR; wave column wn holds columns 16 FN wn .. (SwiGLU: 8 FN of gate,
// then the matching up).
template <int WR_, int WC_, int FN_, int S_, int KG_>
struct Shape {
  static constexpr int WR = WR_, WC = WC_, FN = FN_, S = S_, KG = KG_;
  static constexpr int W = WR * WC, BN = 16 * FN * WC;
};

template <typename T, int FM>
constexpr int stage_bytes() { return (16 * FM * T::WR + T::BN) * kRowB; }

__device__ __forceinline__ void wave_sync() {  // LDS of one wave, written before, read after
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// A wave's sums -> bias, activation, residual, store. Up to three rows of
// fragments at a time go through the wave's part of LDS, so that a lane gets 8
// consecutive outputs of a row, the loads and stores are whole vectors, and the
// activation is a loop instead of a copy of its code per register. The
// residual is asked for before the sums are turned.
// LDS: bytes there are.
template <typename T, int FM, bool SWIGLU, int LDS>
__device__ __forceinline__ void epilogue(MOE_LDS char* lds, const GemmBf16& p, const f32x4v (&acc)[FM][T::FN], int w,
                                         int e, int r0, int rows, int c0) {
  constexpr int FN = T::FN, WR = T::WR;
  constexpr int CW = 16 * FN, OW = SWIGLU ? CW / 2 : CW;  // columns, outputs of a wave
  constexpr int kPitch = CW + 4;                          // (16 rows x 4 words: all banks)
  constexpr int VPR = OW / 8, RPP = 64 / VPR;             // lanes of a row, rows of a pass
  constexpr int NI = FM < 3 ? FM : 3;
  static_assert(T::W * 16 * NI * kPitch * 4 <= LDS, "the sums fit");
  const int wm = w % WR, wn = w / WR;
  const int lane = lane_id(), g = lane >> 4, l16 = lane & 15;
  MOE_LDS float* const slab = (MOE_LDS float*)lds + w * 16 * NI * kPitch;
  const int rl = lane / VPR, v0 = 8 * (lane % VPR);
  const int col = c0 + OW * wn + v0;
  const bool col_ok = col < p.N;  // N is a multiple of 8
  float b[8], bu[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) b[i] = bu[i] = 0.f;
  if (p.bias != nullptr && col_ok) {
    const float* pb = p.bias + int64_t(e) * (SWIGLU ? 2 : 1) * p.N + col;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const float4 f = reinterpret_cast<const float4*>(pb)[h];
      b[4 * h] = f.x; b[4 * h + 1] = f.y; b[4 * h + 2] = f.z; b[4 * h + 3] = f.w;
      if constexpr (SWIGLU) {
        const float4 u = reinterpret_cast<const float4*>(pb + p.N)[h];
        bu[4 * h] = u.x; bu[4 * h + 1] = u.y; bu[4 * h + 2] = u.z; bu[4 * h + 3] = u.w;
      }
    }
  }
  auto tile_row = [&](int s0, int r) { return 16 * (WR * (s0 + (r >> 4)) + wm) + (r & 15); };
#pragma unroll
  for (int s0 = 0; s0 < FM; s0 += NI) {
    constexpr int kPass = (16 * NI + RPP - 1) / RPP;
    const int have = 16 * (FM - s0 < NI ? FM - s0 : NI);  // rows of this slab
    if (16 * (WR * s0 + wm) >= rows) break;               // (the later fragments hold no rows either)
    u32x4 res[kPass][2];
    if (p.res != nullptr) {
#pragma unroll
      for (int ps = 0; ps < kPass; ++ps) {
        const int r = ps * RPP + rl, row = tile_row(s0, r);
        if (r < have && row < rows && col_ok) {
          const int64_t at = int64_t(r0 + row) * p.N + col;
          if (p.res_f32) {
            const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p.res) + at);
            res[ps][0] = q[0];
            res[ps][1] = q[1];
          } else {
            res[ps][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.res) + at);
          }
        }
      }
    }
#pragma unroll
    for (int ii = 0; ii < NI; ++ii)
      if (s0 + ii < FM)
#pragma unroll
        for (int j = 0; j < FN; ++j)
          *reinterpret_cast<MOE_LDS f32x4v*>(slab + (16 * ii + l16) * kPitch + 16 * j + 4 * g) = acc[s0 + ii < FM ? s0 + ii : 0][j];
    wave_sync();
    if (SWIGLU || p.act != 0) {
#pragma unroll 1
      for (int r = rl; r < have; r += RPP) {
        MOE_LDS float* q = slab + r * kPitch + v0;
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          f32x4v z = *reinterpret_cast<MOE_LDS f32x4v*>(q + 4 * h);
          if constexpr (SWIGLU) {
            const f32x4v u = *reinterpret_cast<MOE_LDS f32x4v*>(q + OW + 4 * h);
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = silu(z[i] + b[4 * h + i]) * (u[i] + bu[4 * h + i]);
          } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) z[i] = activate(p.act, z[i] + b[4 * h + i]);
          }
          *reinterpret_cast<MOE_LDS f32x4v*>(q + 4 * h) = z;
        }
      }
      wave_sync();
    }
#pragma unroll
    for (int ps = 0; ps < kPass; ++ps) {
      const int r = ps * RPP + rl, row = tile_row(s0, r);
      if (r < have && row < rows && col_ok) {
        float o[8];
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          const f32x4v z = *reinterpret_cast<MOE_LDS f32x4v*>(slab + r * kPitch + v0 + 4 * h);
#pragma unroll
          for (int i = 0; i < 4; ++i) o[4 * h + i] = SWIGLU || p.act != 0 ? z[i] : z[i] + b[4 * h + i];
        }
        if (p.res != nullptr) {
#pragma unroll
          for (int i = 0; i < 8; ++i)
            o[i] += p.res_f32 ? __uint_as_float(res[ps][i >> 2][i & 3])
                              : (i & 1 ? bf16_hi(res[ps][0][i >> 1]) : bf16_lo(res[ps][0][i >> 1]));
        }
        const int64_t at = int64_t(r0 + row) * p.N + col;
        if (p.out_f32) {
          u32x4* q = reinterpret_cast<u32x4*>(static_cast<float*>(p.C) + at);
#pragma unroll
          for (int h = 0; h < 2; ++h)
            q[h] = u32x4{__float_as_uint(o[4 * h]), __float_as_uint(o[4 * h + 1]), __float_as_uint(o[4 * h + 2]),
                         __float_as_uint(o[4 * h + 3])};
        } else {
          *reinterpret_cast<u32x4*>(static_cast<uint16_t*>(p.C) + at) =
              u32x4{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3]), cvt_bf16x2(o[4], o[5]), cvt_bf16x2(o[6], o[7])};
        }
      }
    }
    wave_sync();
  }
}

// TAIL: K is no multiple of 64, so the last stage holds fewer chunks of 8 k.
template <typename T, int FM, bool SWIGLU, bool TAIL, int LDS>
__device__ __forceinline__ void run_tile(MOE_LDS char* lds, const GemmBf16& p, int e, int r0, int rows, int nj) {
  constexpr int WR = T::WR, FN = T::FN, S = T::S, W = T::W, BN = T::BN, KG = T::KG;
  constexpr int BM = 16 * FM * WR;
  constexpr int kA = BM * kRowB, kStage = stage_bytes<T, FM>();
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kg = KG == 1 ? 0 : wave / W, w = wave % W, wm = w % WR, wn = w / WR;
  const int lane = lane_id();
  const int g = lane >> 4, l16 = lane & 15;
  const int nk_all = (p.K + kSK - 1) / kSK;
  const int nvalid = (p.K - (nk_all - 1) * kSK) / 8;  // chunks of the last stage (TAIL: fewer than 8)
  const int nk = (nk_all + KG - 1) / KG;              // iterations of every group
  const int mine = (nk_all - kg + KG - 1) / KG;       // stages of this one
  constexpr int kCols = SWIGLU ? BN / 2 : BN;         // outputs of a tile
  constexpr int kFrags = SWIGLU ? FN / 2 : FN;        // fragments of a wave's outputs
  const int c0 = nj * kCols;
  const int cols = SWIGLU ? 2 * p.N : p.N;
  MOE_LDS char* const ring = lds + kg * S * kStage;

  typedef LoaderA<BM, W> LA;
  typedef LoaderB<BN, W> LB;
  LA la;
  LB lb;
  la.init(p.A + int64_t(r0) * p.K, p.K, rows, w);
  lb.init(p.W + int64_t(e) * p.K * cols, p.K, cols, w, [&](int s) {
    const int col = s / (16 * FN), j = s / 16 % FN, r = s % 16;  // wave column, fragment, column in it
    const int o = c0 + 16 * kFrags * col + 16 * (j % kFrags) + r;
    return o >= p.N ? 0 : j < kFrags ? o : p.N + o;  // (columns past the end are not stored)
  });
  const int nl = LA::count(w) + LB::count(w);
  auto issue = [&](int st) {
    if (st < mine) {
      MOE_LDS char* d = ring + st % S * kStage;
      const int at = kg + KG * st;
      if (TAIL && at == nk_all - 1) {
        la.template issue<true>(d, w, at, nvalid);
        lb.template issue<true>(d + kA, w, at, nvalid);
      } else {
        la.template issue<false>(d, w, at, 8);
        lb.template issue<false>(d + kA, w, at, 8);
      }
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
    dma::wait_vm_barrier_dyn<kMaxAhead>(max(0, min(last, mine - 1) - s) * nl);
  };
  // fragment addresses: row 16 (WR i + wm) + l16 of A, chunk 4 q + g in k step q
  // (the swizzle does not depend on i); column block FN wn + j of W, blocks kq =
  // 8 q + 2 g and + 1, whose swizzle is that of g
  uint32_t fa[2], fb[2];
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const int ra = 16 * wm + l16;
    fa[q] = uint32_t(ra * kRowB + 16 * chunk_pos(ra, 4 * q + g));
    const uint32_t b = uint32_t(kA + (2 * g * LB::kNQ + FN * wn) * 128 + 8 * l16);
    fb[q] = (FN * wn + q) & 1 ? b - 128u * uint32_t(g & 1) : b + 128u * uint32_t(g & 1);  // of even and odd j
  }
  auto read_a = [&](const MOE_LDS char* st, int q, int i) {
    return *reinterpret_cast<const MOE_LDS u32x4*>(st + fa[q] + 16 * WR * kRowB * i);
  };
  auto read_b = [&](const MOE_LDS char* st, int q, int j) {
    const MOE_LDS char* at = st + fb[j & 1] + (8 * q * LB::kNQ + j) * 128;
    const auto lo = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS dma::i16x4*)(at));
    const auto hi = __builtin_amdgcn_ds_read_tr16_b64_v4i16((MOE_LDS dma::i16x4*)(at + LB::kNQ * 128));
    const u32x2 l = __builtin_bit_cast(u32x2, lo), h = __builtin_bit_cast(u32x2, hi);
    return u32x4{l.x, l.y, h.x, h.y};
  };

  f32x4v acc[FM][FN];
#pragma unroll
  for (int i = 0; i < FM; ++i)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[i][j] = f32x4v{0.f, 0.f, 0.f, 0.f};
  u32x4 a[FM], b[FN];
  // k beyond K, or beyond the group's stages, counts as zeros on both sides
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i) a[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = u32x4{0, 0, 0, 0};
  };

  for (int st = 0; st < S; ++st) issue(st);
  wait_stage(0, S - 1);
#pragma unroll
  for (int j = 0; j < FN; ++j) b[j] = read_b(ring, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) a[i] = read_a(ring, 0, i);

  constexpr int kH1 = (FM + 1) / 2;
  for (int kt = 0; kt < nk; ++kt) {
    const MOE_LDS char* cur = ring + kt % S * kStage;
    const int have = TAIL || KG > 1 ? chunks(kt) : 8;
    if ((TAIL || KG > 1) && have < 8 && g >= have) clear();
    u32x4 bs[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bs[j] = read_b(cur, 1, j);
#pragma unroll
    for (int i = 0; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16x16x32(b[j], a[i], acc[i][j]);
      a[i] = read_a(cur, 1, i);
    }
    alternate_mfma_reads<FM * FN, 2 * FN + FM>();
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = bs[j];
    if ((TAIL || KG > 1) && have < 8 && 4 + g >= have) clear();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kH1; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16x16x32(b[j], a[i], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's reads of stage kt returned; after the barrier every wave's
    // have, and stage kt + 1 is in LDS: stage kt's buffer takes stage kt + S
    dma::wait_lgkm0();
    wait_stage(min(kt + 1, nk - 1), kt + S - 1);
    issue(kt + S);
    const MOE_LDS char* nxt = ring + (kt + 1) % S * kStage;
    u32x4 bn[FN];
#pragma unroll
    for (int j = 0; j < FN; ++j) bn[j] = read_b(nxt, 0, j);
#pragma unroll
    for (int i = 0; i < kH1; ++i) a[i] = read_a(nxt, 0, i);
#pragma unroll
    for (int i = kH1; i < FM; ++i) {
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16x16x32(b[j], a[i], acc[i][j]);
      a[i] = read_a(nxt, 0, i);
    }
    alternate_mfma_reads<(FM - kH1) * FN, 2 * FN + FM>();
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = bn[j];
    __builtin_amdgcn_sched_barrier(0);
  }
  dma::wait_lds_barrier();  // the stages are free

  if constexpr (KG > 1) {
    // the other groups' sums into the first: [group - 1][wave][fragment][lane]
    static_assert((KG - 1) * W * FM * FN * 1024 <= KG * S * kStage, "the sums fit the stages");
    MOE_LDS f32x4v* const sums = (MOE_LDS f32x4v*)lds;
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
  }
  if (kg == 0) epilogue<T, FM, SWIGLU, LDS>(lds, p, acc, w, e, r0, rows, c0);
  dma::wait_lds_barrier();  // the next tile's loads may overwrite the stages
}

// Largest tile: 2 x 4 waves, 256 columns, blocks of up to 288 rows.
typedef Shape<2, 4, 4, 2, 1> Big;
constexpr int kBigFM = 9;
// 128 rows x 128 columns, 8 waves for a group of k. Up to one tile per CU: four
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

// Few rows, where only the weight stream counts: 16 or 32 rows x 64 columns,
// two groups of k and two workgroups per CU, so that one streams while the
// other starts or ends a tile (Stream; 64 rows: Stream64); with few tiles, 16
// rows x 32 columns with eight groups (Narrow), or x 64 with four for SwiGLU.
typedef Shape<1, 2, 2, 3, 2> Stream;
typedef Shape<1, 2, 2, 2, 2> Stream64;  // 64 rows
constexpr int kStreamLocal = 256;  // local experts (two workgroups fill the LDS)
typedef Shape<1, 2, 1, 3, 8> Narrow;
typedef Shape<1, 2, 2, 3, 4> NarrowGU;    // 16 or 32 rows
typedef Shape<1, 2, 1, 2, 8> Narrow32;    // 32 rows x 32 columns
typedef Shape<2, 2, 1, 3, 4> Narrow64;    // 64 rows x 32 columns

// Row caps of the largest tile (the fewest rounds of the grid win, weighted by
// the tallest block, as in the share's grouped GEMM); the others have one.
constexpr int kRowCaps = 6;
__device__ constexpr int kRowCap[kRowCaps] = {288, 256, 224, 192, 160, 128};
constexpr int kRowCapMin = 128;

// MAXE: local experts its tables hold.
template <typename T, int FMMAX, int MAXE, bool SWIGLU, bool TAIL>
__global__ void __launch_bounds__(64 * T::W * T::KG) tile_kernel(GemmBf16 p) {
  constexpr int kThreads = 64 * T::W * T::KG;
  constexpr bool kVary = FMMAX == kBigFM;  // block heights vary: a row cap is chosen
  constexpr int kBM = 16 * FMMAX * T::WR;
  constexpr int kLds = T::KG * T::S * stage_bytes<T, FMMAX>();
  __shared__ __attribute__((aligned(1024))) char smem[kLds];
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
  // rounds of the grid for `tl` tiles of up to `hm` rows, weighted
  auto estimate = [&](unsigned long long tl, int hm) {
    return (tl + gridDim.x - 1) / gridDim.x * (unsigned long long)(hm + T::BN);
  };
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
        const unsigned long long est = estimate(tl, (((only_rows + nrt - 1) / nrt) + 15) & ~15);
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
        const unsigned long long est = estimate(tl, s_cand[c]);
        if (tl < (1ull << 31) && est < best) {
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
  // b % 8); inside an expert, groups of 8 row blocks walk the column tiles
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
    auto go = [&](auto fm_t) { run_tile<T, decltype(fm_t)::value, SWIGLU, TAIL, kLds>(lds, p, e, r0, rows, nj); };
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

Tile pick_tile(bool swiglu, bool ragged, int E_local, int64_t capacity, int N, int K, int64_t cus) {
  const int d = swiglu ? 2 : 1;  // columns of an output
  const int64_t rows_hint = ceil_div(capacity, E_local);
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
  const bool streams = E_local <= kStreamLocal;
  if (rows <= 16 && streams && tiles(16, 32) > cus) return kStream16;
  if (rows <= 32 && streams && tiles(32, 32) > cus) return kStream32;
  if (rows <= 32) return kNarrow;
  if (rows <= 64 && streams && tiles(64, 64 / d) > cus) return kStream64;
  auto once = [&](int bm, int outputs) { return blocks(bm) * ceil_div(N, outputs) <= cus; };
  if (once(16, 32)) return kNarrow;
  if (once(32, 32)) return kNarrow32;
  if (!swiglu && once(64, 32)) return kNarrow64;
  if (once(64, 64 / d)) return kSmall;
  if (once(64, 128 / d)) return kMid64;
  const int64_t mid = blocks(128) * ceil_div(N, 128 / d);
  if (rows_hint >= 128 && mid > 2 * cus && (K >= 1024 || mid * K >= (int64_t(5) << 19))) return kBig;
  if (mid > cus) return kMid2;
  return K > 1024 ? kMidK : kMid;
}

template <bool SWIGLU>
hipError_t launch(const GemmBf16& p, int forced, hipStream_t stream) {
  const bool tail = p.K % kSK != 0;
  const int64_t cus = device_cu_count() / 8 * 8;
  constexpr int d = SWIGLU ? 2 : 1;
  auto go = [&](auto shape, auto fm_t, auto maxe_t, int bm, int per_cu) {
    typedef decltype(shape) T;
    constexpr int FM = decltype(fm_t)::value, MAXE = decltype(maxe_t)::value;
    if (p.E_local > MAXE) return hipErrorInvalidValue;
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
  switch (forced >= 0 ? forced : pick_tile(SWIGLU, p.offsets != nullptr, p.E_local, p.capacity, p.N, p.K, cus)) {
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

}  // namespace bfgemm

hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t stream, int tile) {
  return p.act == 5 ? bfgemm::launch<true>(p, tile, stream) : bfgemm::launch<false>(p, tile, stream);
}

int gemm_bf16_tile(bool swiglu, bool ragged, int E_local, int64_t capacity, int N, int K, int cus) {
  return bfgemm::pick_tile(swiglu, ragged, E_local, capacity, N, K, cus);
}

}  // namespace moe

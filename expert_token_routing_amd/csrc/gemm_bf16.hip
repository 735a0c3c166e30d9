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
// One kernel in five tile shapes, from 32 x 256 and 64 x 64 to 288 x 256. Where the tiles are
// fewer than the CUs, k is cut into ranges whose sums a second kernel adds.
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

// dma16 past the caches, for bytes that no other workgroup reads.
__device__ __forceinline__ void dma16_stream(const i32x4& rsrc, uint32_t voff, uint32_t soff,
                                             const MOE_LDS char* lds_base) {
  const uint32_t lds_addr = uint32_t(reinterpret_cast<uintptr_t>(lds_base));
  asm volatile("" : "+s"(soff));
  uint32_t s;
  // (the scalar move keeps a wait state between the write of M0 and the load, and
  // the load off a scalar that a vector instruction may have written just before)
  asm volatile("s_mov_b32 %0, %3\n\tbuffer_load_dwordx4 %1, %2, %0 offen nt lds"
               : "=&s"(s)
               : "v"(voff), "s"(rsrc), "s"(soff), "{m0}"(lds_addr)
               : "memory");
}

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
  __device__ __forceinline__ void issue(MOE_LDS char* dst, int w, int stage, int valid, bool once) const {
#pragma unroll
    for (int j = 0; j < kPer; ++j)
      if (kLoads % W == 0 || j * W + w < kLoads) {
        const int r = row(j, w);
        const uint32_t back = TAIL && r >= 8 * valid ? uint32_t(r & ~7) * ld : 0u;
        if (once)
          dma16_stream(rsrc, voff[j] - back, uint32_t(stage) * kSK * ld, dst + 1024 * (j * W + w));
        else
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

// WR x WC waves; a tile is 16 FM WR rows x 16 FN WC columns, S stages in LDS.
// 16-row fragment f belongs to wave row f % WR; wave column wn holds columns 16 FN
// wn .. (SwiGLU: 8 FN of gate, then the matching up).
// KG groups of such waves take every KG-th stage and meet in LDS at the end.
template <int WR_, int WC_, int FN_, int S_, int KG_ = 1>
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
// activation is a loop instead of a copy of its code per register. The residual of
// the next slab is asked for before this one's sums are turned (8192 x 2048 x 7168,
// bf16 residual: 269 -> 257 us).
// LDS: bytes there are.
template <typename T, int FM, bool SWIGLU, int LDS>
__device__ __forceinline__ void epilogue(MOE_LDS char* lds, const GemmBf16& p, const f32x4v (&acc)[FM][T::FN], int w,
                                         int e, int r0, int rows, int c0) {
  constexpr int FN = T::FN, WR = T::WR;
  constexpr int CW = 16 * FN, OW = SWIGLU ? CW / 2 : CW;  // columns, outputs of a wave
  constexpr int kPitch = CW + 4;                          // (16 rows x 4 words: all banks)
  constexpr int VPR = OW / 8, RPP = 64 / VPR;             // lanes of a row, rows of a pass
  constexpr int NI = FM < 3 ? FM : FM < 8 ? 3 : 2;
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
  constexpr int kPass = (16 * NI + RPP - 1) / RPP;
  constexpr int kSlabs = (FM + NI - 1) / NI;
  auto rows_of = [&](int s0) { return 16 * (FM - s0 < NI ? FM - s0 : NI); };
  constexpr int kAhead = FM < 9 ? 1 : 0;  // (the tallest tile has no registers for two slabs)
  u32x4 res[kAhead + 1][kPass][2];
  auto ask = [&](int sl) {
    const int s0 = sl * NI;
#pragma unroll
    for (int ps = 0; ps < kPass; ++ps) {
      const int r = ps * RPP + rl, row = tile_row(s0, r);
      if (r < rows_of(s0) && row < rows && col_ok) {
        const int64_t at = int64_t(r0 + row) * p.N + col;
        if (p.res_f32) {
          const u32x4* q = reinterpret_cast<const u32x4*>(static_cast<const float*>(p.res) + at);
          res[sl & kAhead][ps][0] = q[0];
          res[sl & kAhead][ps][1] = q[1];
        } else {
          res[sl & kAhead][ps][0] = *reinterpret_cast<const u32x4*>(static_cast<const uint16_t*>(p.res) + at);
        }
      }
    }
  };
  if (kAhead != 0 && p.res != nullptr) ask(0);
#pragma unroll
  for (int sl = 0; sl < kSlabs; ++sl) {
    const int s0 = sl * NI, have = rows_of(s0);
    if (16 * (WR * s0 + wm) >= rows) break;  // (the later fragments hold no rows either)
    if (sl + kAhead < kSlabs && p.res != nullptr) ask(sl + kAhead);
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
            o[i] += p.res_f32 ? __uint_as_float(res[sl & kAhead][ps][i >> 2][i & 3])
                              : (i & 1 ? bf16_hi(res[sl & kAhead][ps][0][i >> 1])
                                          : bf16_lo(res[sl & kAhead][ps][0][i >> 1]));
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

// A wave's sums of one k range as they are, for join_kernel.
template <typename T, int FM, bool SWIGLU>
__device__ __forceinline__ void store_part(const GemmBf16& p, const f32x4v (&acc)[FM][T::FN], int w, int r0, int rows,
                                           int c0, int z) {
  constexpr int FN = T::FN, WR = T::WR, kFrags = SWIGLU ? FN / 2 : FN;
  const int wm = w % WR, wn = w / WR;
  const int g = lane_id() >> 4, l16 = lane_id() & 15;
  const int cols = SWIGLU ? 2 * p.N : p.N;
#pragma unroll
  for (int i = 0; i < FM; ++i) {
    const int row = 16 * (WR * i + wm) + l16;
    if (row < rows) {
      float* to = p.part + (int64_t(z) * p.capacity + r0 + row) * cols;
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        const int o = c0 + 16 * kFrags * wn + 16 * (j % kFrags) + 4 * g;
        if (o < p.N) *reinterpret_cast<f32x4v*>(to + (j < kFrags ? o : p.N + o)) = acc[i][j];
      }
    }
  }
}

// TAIL: K is no multiple of 64, so the last stage holds fewer chunks of 8 k.
// once: no other tile reads these columns, so they pass the caches by (32 experts
// of 7168 x 4096, 64 rows: 282 -> 251 us; 1 x 7168 x 4096: 15.5 -> 14.6).
// SPLIT: z is one of several k ranges; without, the tile is of all k, and its weights
// take the caches.
template <typename T, int FM, bool SWIGLU, bool TAIL, bool SPLIT, int LDS>
__device__ __forceinline__ void run_tile(MOE_LDS char* lds, const GemmBf16& p, int e, int r0, int rows, int nj,
                                         int z, bool once) {
  constexpr int WR = T::WR, FN = T::FN, S = T::S, W = T::W, BN = T::BN;
  constexpr int BM = 16 * FM * WR;
  constexpr int kA = BM * kRowB, kStage = stage_bytes<T, FM>();
  constexpr int KG = T::KG;
  const int wv = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), grp = KG > 1 ? wv / W : 0;
  const int w = KG > 1 ? wv % W : wv, wm = w % WR, wn = w / WR;
  const int lane = lane_id();
  const int g = lane >> 4, l16 = lane & 15;
  static_assert(KG <= 2, "their sums meet in pairs");
  MOE_LDS char* const all = lds;
  lds += grp * S * kStage;
  const int last_stage = (p.K + kSK - 1) / kSK - 1;
  const int nvalid = (p.K - last_stage * kSK) / 8;  // its chunks (TAIL: fewer than 8)
  const int s0 = (SPLIT ? z * p.per : 0) + grp;     // the k range's stages, the group's first
  const int n_st = SPLIT ? min(p.per, last_stage + 1 - (s0 - grp)) : last_stage + 1;
  const int turns = (n_st + KG - 1) / KG;           // of the first group
  const int nk = KG > 1 ? (n_st - grp + KG - 1) / KG : n_st;
  constexpr int kCols = SWIGLU ? BN / 2 : BN;         // outputs of a tile
  constexpr int kFrags = SWIGLU ? FN / 2 : FN;        // fragments of a wave's outputs
  const int c0 = nj * kCols;
  const int cols = SWIGLU ? 2 * p.N : p.N;

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
    if (st < nk) {
      MOE_LDS char* d = lds + st % S * kStage;
      const int at = s0 + st * KG;
      if (TAIL && at == last_stage) {
        la.template issue<true>(d, w, at, nvalid);
        lb.template issue<true>(d + kA, w, at, nvalid, SPLIT && once);
      } else {
        la.template issue<false>(d, w, at, 8);
        lb.template issue<false>(d + kA, w, at, 8, SPLIT && once);
      }
    }
  };
  // stage s landed for this wave; up to `last` were issued
  constexpr int kMaxAhead = (S - 1) * (LA::kPer + LB::kPer);
  auto wait_stage = [&](int s, int last) {
    dma::wait_vm_barrier_dyn<kMaxAhead>(max(0, min(last, nk - 1) - s) * nl);
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
  // k beyond K counts as zeros on both sides
  auto clear = [&] {
#pragma unroll
    for (int i = 0; i < FM; ++i) a[i] = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < FN; ++j) b[j] = u32x4{0, 0, 0, 0};
  };

  for (int st = 0; st < S; ++st) issue(st);
  wait_stage(0, S - 1);
#pragma unroll
  for (int j = 0; j < FN; ++j) b[j] = read_b(lds, 0, j);
#pragma unroll
  for (int i = 0; i < FM; ++i) a[i] = read_a(lds, 0, i);

  constexpr int kH1 = (FM + 1) / 2;
  for (int kt = 0; kt < turns; ++kt) {
    const MOE_LDS char* cur = lds + kt % S * kStage;
    const bool none = KG > 1 && kt >= nk;  // this group has no stage left
    const bool tail = TAIL && s0 + kt * KG == last_stage;
    if (none || (tail && g >= nvalid)) clear();
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
    if (none || (tail && 4 + g >= nvalid)) clear();
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int i = 0; i < kH1; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[i][j] = mfma16x16x32(b[j], a[i], acc[i][j]);
    __builtin_amdgcn_sched_barrier(0);
    // this wave's reads of stage kt returned; after the barrier every wave's
    // have, and stage kt + 1 is in LDS: stage kt's buffer takes stage kt + S
    dma::wait_lgkm0();
    wait_stage(min(kt + 1, turns - 1), kt + S - 1);
    issue(kt + S);
    const MOE_LDS char* nxt = lds + (kt + 1) % S * kStage;
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
  // Two groups: each adds up and ends half of the rows (the first all of one fragment).
  if constexpr (KG == 2) {
    constexpr int HM = FM / KG == 0 ? 1 : FM / KG;
    static_assert(FM == 1 || FM % KG == 0, "halves");
    static_assert(KG * W * HM * FN * 1024 <= LDS, "a half's sums fit");
    MOE_LDS f32x4v* const area = (MOE_LDS f32x4v*)all + w * HM * FN * 64 + lane;
    constexpr int kArea = W * HM * FN * 64;
    const bool ends = FM > 1 || grp == 0;
    f32x4v half[HM][FN];
#pragma unroll
    for (int i = 0; i < HM; ++i)
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        if (FM > 1 || grp > 0) area[grp * kArea + 64 * (i * FN + j)] = FM > 1 && grp == 0 ? acc[FM > 1 ? HM + i : 0][j] : acc[i][j];
        half[i][j] = FM > 1 && grp > 0 ? acc[FM > 1 ? HM + i : 0][j] : acc[i][j];
      }
    dma::wait_lds_barrier();
    if (ends)
#pragma unroll
      for (int i = 0; i < HM; ++i)
#pragma unroll
        for (int j = 0; j < FN; ++j) half[i][j] += area[(1 - grp) * kArea + 64 * (i * FN + j)];
    dma::wait_lds_barrier();
    const int skip = 16 * WR * HM * grp;
    if (ends && skip < rows) {
      if (SPLIT && p.ranges > 1)
        store_part<T, HM, SWIGLU>(p, half, w, r0 + skip, rows - skip, c0, z);
      else
        epilogue<T, HM, SWIGLU, LDS / KG>(all + grp * (LDS / KG), p, half, w, e, r0 + skip, rows - skip, c0);
    }
    if (!(SPLIT && p.ranges > 1)) dma::wait_lds_barrier();  // the next tile's loads may overwrite it
    return;
  }

  if (SPLIT && p.ranges > 1) {
    store_part<T, FM, SWIGLU>(p, acc, w, r0, rows, c0, z);
    return;
  }
  epilogue<T, FM, SWIGLU, LDS>(lds, p, acc, w, e, r0, rows, c0);
  dma::wait_lds_barrier();  // the next tile's loads may overwrite the stages
}

// 128 x 128, eight waves, four stages: blocks of 65 to 128 rows, or a few where the
// weights are the most of it. (16 x 32 tiles for one row, half lines of two XCDs
// each, 1 x 7168 x 4096: 32 us, ranges of this 16.6. Four waves of 64 x 64 for
// 1024 x 7168 x 4096: 85 us, eight of 64 x 32: 72.)
typedef Shape<2, 4, 2, 4> Mid;
constexpr int kMidFM = 4;
// 64 x 64 in two groups of four waves, four stages each: where larger tiles would need
// k ranges, and so a second kernel, to be as many as the CUs, or few columns leave few
// tiles (333 x 2880 x 1536: 17.0 us, Mid in seven ranges 19.2; 1000 x 2880 x 768: 17.4,
// Mid 20.8; 700 x 1408 x 640: 9.6, Mid 14.8; 128 x 4096 x 1024 in 8 ranges: 11.1, Mid
// 15.3). Four groups of two stages take 22.4 us for 512 x 2880 x 1536, three of three
// 19.4, these 18.7.
typedef Shape<2, 2, 2, 4, 2> Small;
constexpr int kSmallFM = 2;
// 256 x 128: fewer operand bytes per product, for about one such tile per CU
// (2048 x 7168 x 4096: 124 us, Mid 146, Big 150). Its blocks of up to 64 rows
// stream weights as well as Mid's (1 x 7168 x 4096 in 8 ranges: 16.3, Mid 16.6).
typedef Shape<4, 2, 4, 3> Tall;
constexpr int kTallFM = 4;
// Largest tile: 256 columns, blocks of up to 288 rows.
typedef Shape<2, 4, 4, 2> Big;
constexpr int kBigFM = 9;
// Few rows and many tiles, where only the weight stream counts: 32 x 256, two
// workgroups per CU, so that one streams while the other starts or ends a tile
// (32 experts of 7168 x 4096, 64 / 256 rows: 254 / 300 us, 6.4 / 6.3 TB/s; Mid
// 311 / 338).
typedef Big Few;
constexpr int kFewLocal = 256;  // local experts (two workgroups fill the LDS)

// Row caps of the largest tile (the fewest rounds of the grid win, weighted by
// the tallest block, as in the share's grouped GEMM); the others have one.
constexpr int kRowCaps = 6;
__device__ constexpr int kRowCap[kRowCaps] = {288, 256, 224, 192, 160, 128};
constexpr int kRowCapMin = 128;

// MAXE: local experts its tables hold.
template <typename T, int FMMAX, int MAXE, bool SWIGLU, bool TAIL>
__global__ void __launch_bounds__(64 * T::W * T::KG) tile_kernel(GemmBf16 p) {
  constexpr int kThreads = 64 * T::W * T::KG;
  static_assert(FMMAX == 1 || FMMAX == 2 || FMMAX == 4 || FMMAX == kBigFM, "fragments per wave row");
  constexpr bool kVary = FMMAX == kBigFM;  // a row cap is chosen; one k range
  constexpr bool kHalves = kVary && MAXE == 1;
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
  const bool tables = MAXE > 1 && p.E_local > 1;
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
        const int nrt = max(1, row_blocks(only_rows, kRowCap[c]));
        const unsigned long long tl = (unsigned long long)nrt * (unsigned long long)ntn;
        const unsigned long long est = estimate(tl, block_height(only_rows, nrt));
        if (tl < (1ull << 31) && est < best) {
          best = est;
          row_cap = kRowCap[c];
        }
      }
    }
    total = row_blocks(only_rows, row_cap) * ntn;
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
            const int nrt = row_blocks(me[q], kRowCap[c]);
            tl += (unsigned long long)nrt * (unsigned long long)ntn;
            hm = max(hm, block_height(me[q], nrt));
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
      mt[q] = row_blocks(me[q], row_cap) * ntn;
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
  const int64_t items = kVary ? int64_t(total) : int64_t(total) * p.ranges;
  const int lo_t = int(items * xcd / 8), n_t = int(items * (xcd + 1) / 8) - lo_t;
  // kHalves: a last round of no more tiles than half the CUs goes in halves of their
  // rows (8192 x 2048 x 7168, 3.5 rounds: 231 -> 224 us, with a residual 263 -> 250.
  // Ragged segments gain nothing and their loop grows by it: 853 -> 863 us.)
  const int last = n_t % per_xcd;
  const bool halves = kHalves && 2 * last <= per_xcd;
  const int end_t = halves ? n_t + last : n_t;
  for (int i_t = int(blockIdx.x / 8); i_t < end_t; i_t += per_xcd) {
    const bool half = halves && i_t >= n_t - last;
    const int item = lo_t + (half ? (n_t - last + i_t) >> 1 : i_t);
    const int z = !kVary && p.ranges > 1 ? item / total : 0, tile = item - z * total;
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
    const int nrt = row_blocks(m_e, row_cap);
    const int local = tile - first;
    const int grp = local / (kGroup * ntn);
    const int in_grp = min(kGroup, nrt - grp * kGroup);
    const int rest = local - grp * kGroup * ntn;
    const int nj = rest / in_grp;
    const int mi = grp * kGroup + rest - nj * in_grp;
    const int height = block_height(m_e, nrt);
    int r0 = seg0 + mi * height;
    int rows = min(height, seg0 + m_e - r0);
    if (half) {
      const int upper = min(rows, (rows / 2 + 31) & ~31);
      if ((n_t - last + i_t) & 1) {
        r0 += upper;
        rows -= upper;
      } else {
        rows = upper;
      }
    }
    if (rows <= 0) continue;
    auto go = [&](auto fm_t) { run_tile<T, decltype(fm_t)::value, SWIGLU, TAIL, !kVary, kLds>(lds, p, e, r0, rows, nj, z, nrt == 1); };
    // fragments that a wave row needs (a shorter last block runs the others' code where
    // there is little to save: fetching code of its own takes 2 us)
    const int fm = ((kVary ? rows : height) + 16 * T::WR - 1) / (16 * T::WR);
    if constexpr (FMMAX == 1) {
      go(std::integral_constant<int, 1>{});
    } else if constexpr (FMMAX == 2) {
      if (fm == 1)
        go(std::integral_constant<int, 1>{});
      else
        go(std::integral_constant<int, 2>{});
    } else if constexpr (FMMAX == 4) {
      switch (fm) {
        case 1: go(std::integral_constant<int, 1>{}); break;
        case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: go(std::integral_constant<int, 3>{}); break;
        default: go(std::integral_constant<int, 4>{}); break;
      }
    } else {
      switch (fm) {
        case 1: case 2: go(std::integral_constant<int, 2>{}); break;
        case 3: case 4: go(std::integral_constant<int, 4>{}); break;
        case 5: go(std::integral_constant<int, 5>{}); break;
        case 6: go(std::integral_constant<int, 6>{}); break;
        case 7: go(std::integral_constant<int, 7>{}); break;
        case 8: go(std::integral_constant<int, 8>{}); break;
        default: go(std::integral_constant<int, 9>{}); break;
      }
    }
  }
}

// The ranges' sums added in order, then the epilogue. 4 outputs a thread.
template <bool SWIGLU>
__global__ void __launch_bounds__(256) join_kernel(GemmBf16 p) {
  const int nv = p.N / 4;
  const int64_t v = int64_t(blockIdx.x) * 256 + threadIdx.x;
  const int64_t row = v / nv;
  if (row >= p.capacity) return;
  const int col = 4 * int(v - row * nv);
  // the row's segment: the last one that starts at or before it
  int e = 0;
  if (p.offsets != nullptr) {
    int lo = 0, hi = p.E_local - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (p.offsets[mid] <= row)
        lo = mid;
      else
        hi = mid - 1;
    }
    e = lo;
    int a, b;
    segment(p, e, a, b);
    if (row < a || row >= b) return;
  }
  constexpr int D = SWIGLU ? 2 : 1;
  const int cols = D * p.N;
  const float* from = p.part + row * cols + col;
  const int64_t step = p.capacity * cols;
  f32x4v z[D];
#pragma unroll
  for (int d = 0; d < D; ++d) z[d] = f32x4v{0.f, 0.f, 0.f, 0.f};
  for (int q0 = 0; q0 < p.ranges; q0 += 8) {
    f32x4v t[8][D];
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (q0 + q < p.ranges) t[q][d] = *reinterpret_cast<const f32x4v*>(from + (q0 + q) * step + d * p.N);
#pragma unroll
    for (int q = 0; q < 8; ++q)
#pragma unroll
      for (int d = 0; d < D; ++d)
        if (q0 + q < p.ranges) z[d] += t[q][d];
  }
  if (p.bias != nullptr)
#pragma unroll
    for (int d = 0; d < D; ++d) z[d] += *reinterpret_cast<const f32x4v*>(p.bias + int64_t(e) * cols + d * p.N + col);
  float o[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (SWIGLU)
      o[i] = silu(z[0][i]) * z[D - 1][i];
    else
      o[i] = p.act != 0 ? activate(p.act, z[0][i]) : z[0][i];
  }
  const int64_t at = row * p.N + col;
  if (p.res != nullptr) {
    if (p.res_f32) {
      const f32x4v r = *reinterpret_cast<const f32x4v*>(static_cast<const float*>(p.res) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += r[i];
    } else {
      const u32x2 r = *reinterpret_cast<const u32x2*>(static_cast<const uint16_t*>(p.res) + at);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] += i & 1 ? bf16_hi(r[i >> 1]) : bf16_lo(r[i >> 1]);
    }
  }
  if (p.out_f32)
    *reinterpret_cast<f32x4v*>(static_cast<float*>(p.C) + at) = f32x4v{o[0], o[1], o[2], o[3]};
  else
    *reinterpret_cast<u32x2*>(static_cast<uint16_t*>(p.C) + at) = u32x2{cvt_bf16x2(o[0], o[1]), cvt_bf16x2(o[2], o[3])};
}

// Which tiles a launch takes (names as the shapes above), and into how many
// ranges k is cut.
enum Tile { kFew, kMid, kTall, kBig, kSmall };
struct Plan {
  Tile tile;
  int ranges;
};

// The plan of the shortest time by this model, from the sizes and the rows that a
// segment is expected to hold (microseconds; stages of 64 k):
//   a round of the CUs: stages x a time by tile and fragments, and a start and end
//   k ranges: 1.6 for the second kernel, 0.05 for each, and the sums' bytes, written
//   and read, at 4.4 TB/s
//   no less than the operands' bytes at 6 TB/s, and the second kernel
// (184 sizes of 1 to 16384 rows, every tile and up to 28 ranges of each timed: 2%
// behind the best of them on average, one by more than 20%.)
Plan pick(bool swiglu, int E_local, int64_t capacity, int N, int K, int64_t cus) {
  const int64_t cols = swiglu ? 2 * int64_t(N) : N, stages = ceil_div(K, kSK);
  const bool ragged = E_local > 1;
  const int64_t rows = ceil_div(capacity, E_local);  // expected of a segment
  const int64_t active = std::min<int64_t>(E_local, capacity);  // segments that can have rows
  // Ragged segments spread around the expected length; a block in two is a segment's
  // last.
  const int64_t tall = ragged ? std::min(rows + rows / 4, capacity) : rows;
  auto blocks = [&](int64_t bm) {
    const int64_t most = ceil_div(tall, bm) * active;
    return tall <= bm ? most : std::min(most, ceil_div(rows * active, bm) + active / 2);
  };
  const double least = (double(active) * K * cols + double(capacity) * K) * 2 / 6e6;
  Plan best{kMid, 1};
  double best_us = 1e30;
  auto consider = [&](Tile tile, int64_t tiles, int64_t places, double per_stage, double ends, int64_t ranges) {
    const int64_t per = ceil_div(stages, ranges), z = ceil_div(stages, per);
    double us = double(ceil_div(tiles * z, places)) * (double(per) * per_stage + ends);
    if (z > 1) us += 1.6 + 0.05 * double(z) + double(z) * double(capacity) * double(cols) * 8 / 4.4e6;
    us = std::max(us, z > 1 ? least + 1.6 : least) + 0.05 * us;
    if (us < best_us) {
      best_us = us;
      best = {tile, int(z)};
    }
  };
  auto ranged = [&](Tile tile, int64_t tiles, int64_t places, double per_stage, double ends) {
    // (a range has two stages at least)
    for (const int64_t z : {1, 2, 3, 4, 5, 6, 8, 12, 16, 28})
      if (z == 1 || z <= stages / 2) consider(tile, tiles, places, per_stage, ends, z);
  };
  // fragments of a wave row in blocks of up to `most` rows
  auto frags = [&](int64_t most) { return ceil_div(std::min(tall, most), most / 4); };
  ranged(kMid, blocks(128) * ceil_div(cols, 128), cus, frags(128) == 1 ? 0.40 : frags(128) == 2 ? 0.48 : 0.65, 2.2);
  ranged(kSmall, blocks(64) * ceil_div(cols, 64), cus, 0.28, 1.9);
  ranged(kTall, blocks(256) * ceil_div(cols, 128), cus, frags(256) == 1 ? 0.42 : frags(256) < 4 ? 0.85 : 1.05, 1.75);
  if (tall <= 128 && E_local <= kFewLocal) ranged(kFew, blocks(32) * ceil_div(cols, 256), 2 * cus, 1.1, 2.2);
  if (tall > 128)
    for (const int64_t cap : {288, 256, 224, 192, 160, 128}) {
      const int64_t height = std::min<int64_t>(cap, (ceil_div(tall, ceil_div(tall, cap)) + 15) / 16 * 16);
      consider(kBig, blocks(cap) * ceil_div(cols, 256), cus, 1.75 * double(height + 256) / 512, 3.8, 1);
    }
  return best;
}

Plan plan_of(const GemmBf16& p, int tile, int ranges) {
  if (tile >= 0) return {Tile(tile), ranges};
  return pick(p.act == 5, p.E_local, p.capacity, p.N, p.K, device_cu_count() / 8 * 8);
}

// Stages of a range, and so many ranges.
void cut(int K, int ranges, int& per, int& n) {
  const int stages = int(ceil_div(K, kSK));
  per = int(ceil_div(stages, std::max(1, std::min(ranges, stages))));
  n = int(ceil_div(stages, per));
}

template <bool SWIGLU>
hipError_t launch(GemmBf16 p, Plan plan, hipStream_t stream) {
  cut(p.K, plan.ranges, p.per, p.ranges);
  const bool tail = p.K % kSK != 0;
  const int64_t cus = device_cu_count() / 8 * 8;
  constexpr int d = SWIGLU ? 2 : 1;
  auto go = [&](auto shape, auto fm_t, auto maxe_t, int bm, int per_cu) {
    typedef decltype(shape) T;
    constexpr int FM = decltype(fm_t)::value, MAXE = decltype(maxe_t)::value;
    if (p.E_local > MAXE) return hipErrorInvalidValue;
    const int64_t n = (ceil_div(p.capacity, bm) + p.E_local) * ceil_div(p.N, T::BN / d) * p.ranges;
    // the kernels index tiles with 31 bits
    if (n >= (int64_t(1) << 31)) return hipErrorInvalidValue;
    const unsigned grid = unsigned(std::max<int64_t>(8, std::min<int64_t>(cus * per_cu, ceil_div(n, 8) * 8)));
    auto* kern = tail ? tile_kernel<T, FM, MAXE, SWIGLU, true> : tile_kernel<T, FM, MAXE, SWIGLU, false>;
    hipLaunchKernelGGL(kern, dim3(grid), dim3(64 * T::W * T::KG), 0, stream, p);
    return hipGetLastError();
  };
  typedef std::integral_constant<int, kMaxLocal> AnyE;
  typedef std::integral_constant<int, 1> OneE;
  hipError_t err = hipErrorInvalidValue;
  switch (plan.tile) {
    case kFew:
      err = go(Few{}, std::integral_constant<int, 1>{}, std::integral_constant<int, kFewLocal>{}, 32, 2);
      break;
    case kMid: err = go(Mid{}, std::integral_constant<int, kMidFM>{}, AnyE{}, 128, 1); break;
    case kSmall: err = go(Small{}, std::integral_constant<int, kSmallFM>{}, AnyE{}, 64, 1); break;
    case kTall: err = go(Tall{}, std::integral_constant<int, kTallFM>{}, AnyE{}, 256, 1); break;
    case kBig:
      if (p.ranges == 1)
        err = p.E_local == 1 ? go(Big{}, std::integral_constant<int, kBigFM>{}, OneE{}, kRowCapMin, 1)
                             : go(Big{}, std::integral_constant<int, kBigFM>{}, AnyE{}, kRowCapMin, 1);
      break;
  }
  if (err == hipSuccess && p.ranges > 1) {
    const int64_t threads = p.capacity * (p.N / 4);
    hipLaunchKernelGGL(join_kernel<SWIGLU>, dim3(unsigned(ceil_div(threads, 256))), dim3(256), 0, stream, p);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace bfgemm

hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t stream, int tile, int ranges) {
  const bfgemm::Plan plan = bfgemm::plan_of(p, tile, ranges);
  return p.act == 5 ? bfgemm::launch<true>(p, plan, stream) : bfgemm::launch<false>(p, plan, stream);
}

size_t gemm_bf16_part_bytes(const GemmBf16& p, int tile, int ranges) {
  int per, n;
  bfgemm::cut(p.K, bfgemm::plan_of(p, tile, ranges).ranges, per, n);
  return n > 1 ? size_t(n) * size_t(p.capacity) * size_t(p.act == 5 ? 2 * int64_t(p.N) : p.N) * sizeof(float) : 0;
}

int gemm_bf16_plan(bool swiglu, int E_local, int64_t capacity, int N, int K, int cus, int* ranges) {
  const bfgemm::Plan plan = bfgemm::pick(swiglu, E_local, capacity, N, K, cus);
  *ranges = plan.ranges;
  return plan.tile;
}

}  // namespace moe

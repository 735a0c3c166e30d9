// Norms before and after a block, fused with the block's gate, the scaled
// residual and the norm before the next block.
//
//   pre:   n  = rms(r) * w                        rms(v) = v / sqrt(mean(v^2) + eps)
//   post:  z  = rms(y) * w_post                   (w_post absent: z = y)
//          r' = residual_scale * r + gate * z     (gate absent: 1)
//          n' = rms(r') * w_next                  (w_next absent: not written)
//
// Every value is read once, kept in registers as float32 until it is rounded
// for its store, and n' is formed from the float32 r', before r' is rounded:
// rounding once per output loses nothing, and the two reductions of a row
// (of y, then of r') need the whole row on chip anyway.
//
// Bound: HBM. One workgroup holds a row, NV vectors of 8 values per thread,
// and walks the rows with a stride of the grid, so that the norm weights and a
// channel gate stay in registers for all of its rows (NV <= 2; wider rows read
// them again from L2) and the next row's loads are issued before the current
// row's reductions. 16384 x 7168 with a float32 y: 200-207 us, 5.7-5.9 TB/s.
#include "moe_kernels.h"
#include "moe_row.h"

namespace moe {
namespace norm {

// Threads of a row: one vector of 8 each up to 1024 vectors (few rows) or up
// to 512 (many), two each (NV = 2) for 513 .. 1024 vectors, four above.
template <int NV>
constexpr int kThreadsMax = NV == 2 ? 512 : 1024;

struct Args {
  const void* y;
  const void* r;
  const float* w_post;
  const float* gate;
  const float* w_next;
  void* out;
  uint16_t* normed;
  int T, nvec, H, gate_kind;
  float scale, eps, inv_h;
};

// 8 consecutive values as stored (bf16: 16 bytes, float32: 32)
template <bool F32>
struct Raw {
  u32x4 v[F32 ? 2 : 1];
  template <bool NT>
  __device__ __forceinline__ void load(const void* base, int64_t vec) {
    const u32x4* p = static_cast<const u32x4*>(base) + vec * (F32 ? 2 : 1);
#pragma unroll
    for (int i = 0; i < (F32 ? 2 : 1); ++i) v[i] = NT ? __builtin_nontemporal_load(p + i) : p[i];
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (F32)
      return __uint_as_float(v[i >> 2][i & 3]);
    else
      return (i & 1) ? bf16_hi(v[0][i >> 1]) : bf16_lo(v[0][i >> 1]);
  }
};

__device__ __forceinline__ void load8(float (&o)[8], const float* p) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  o[0] = a.x; o[1] = a.y; o[2] = a.z; o[3] = a.w;
  o[4] = b.x; o[5] = b.y; o[6] = b.z; o[7] = b.w;
}

template <bool NT>
__device__ __forceinline__ void store16(u32x4* p, const u32x4& v) {
  if constexpr (NT)
    __builtin_nontemporal_store(v, p);
  else
    *p = v;
}
template <bool NT>
__device__ __forceinline__ void store8_bf16(void* base, int64_t vec, const float (&f)[8]) {
  store16<NT>(static_cast<u32x4*>(base) + vec, u32x4{cvt_bf16x2(f[0], f[1]), cvt_bf16x2(f[2], f[3]),
                                                     cvt_bf16x2(f[4], f[5]), cvt_bf16x2(f[6], f[7])});
}

// Sum over the workgroup, the same on every thread. Consecutive calls take
// different halves of s_red, so one barrier each is enough: a wave can write
// half b again only after the barrier of the call in between, which every
// wave reaches after its reads of half b.
__device__ __forceinline__ float block_sum(float v, float* s_red, int half) {
  v = wave_sum(v);
  const int nw = blockDim.x >> 6;
  float* s = s_red + 16 * half;
  if (lane_id() == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  float t = 0.f;
  for (int i = 0; i < nw; ++i) t += s[i];
  return t;
}

// Y: 0 no block output (norm before the block: r alone), 1 bf16, 2 float32.
// NT: the rows go past the caches (more of them than the caches hold).
template <int Y, bool RF32, int NV, bool NT>
__global__ void __launch_bounds__(kThreadsMax<NV>) block_norm_kernel(Args a) {
  constexpr bool kKeep = NV <= 2;  // weights in registers, next row prefetched
  constexpr bool YF32 = Y == 2;
  __shared__ float s_red[32];
  const int nt = blockDim.x;
  int vec[NV];
  bool in[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int v = int(threadIdx.x) + i * nt;
    in[i] = v < a.nvec;
    vec[i] = in[i] ? v : 0;  // idle lanes read vector 0 and neither add nor store it
  }
  float wp[kKeep ? NV : 1][8], wn[kKeep ? NV : 1][8], gc[kKeep ? NV : 1][8];
  if constexpr (kKeep) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if (Y != 0 && a.w_post) load8(wp[i], a.w_post + 8 * vec[i]);
      if (a.w_next) load8(wn[i], a.w_next + 8 * vec[i]);
      if (Y != 0 && a.gate_kind == 1) load8(gc[i], a.gate + 8 * vec[i]);
    }
  }
  int64_t t = blockIdx.x;
  Raw<YF32> qy[NV];
  Raw<RF32> qr[NV];
  auto load_row = [&](int64_t row) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      if constexpr (Y != 0) qy[i].template load<NT>(a.y, row * a.nvec + vec[i]);
      qr[i].template load<NT>(a.r, row * a.nvec + vec[i]);
    }
  };
  if constexpr (kKeep) load_row(t);
  int half = 0;
  for (; t < a.T; t += gridDim.x) {
    if constexpr (!kKeep) load_row(t);
    float v[NV][8];
    float tok_gate = 1.f;
    float ss = 0.f;
    if constexpr (Y != 0) {
      if (a.gate_kind == 2) tok_gate = a.gate[t];
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float f = qy[i].get(j);
          v[i][j] = f;
          if (in[i]) ss = fmaf(f, f, ss);
        }
    }
    float rr[NV][8];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
      for (int j = 0; j < 8; ++j) rr[i][j] = qr[i].get(j);
    if constexpr (kKeep) {
      const int64_t tn = t + gridDim.x;
      if (tn < a.T) load_row(tn);
    }
    if constexpr (Y != 0) {
      if (a.w_post) {
        const float inv = rsqrtf(fmaf(block_sum(ss, s_red, half), a.inv_h, a.eps));
        half ^= 1;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          if constexpr (!kKeep) load8(wp[0], a.w_post + 8 * vec[i]);
#pragma unroll
          for (int j = 0; j < 8; ++j) v[i][j] = v[i][j] * inv * wp[kKeep ? i : 0][j];
        }
      }
      ss = 0.f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float g[8];
        if (a.gate_kind == 3)
          load8(g, a.gate + (t * a.nvec + vec[i]) * 8);
        else if (a.gate_kind == 1 && !kKeep)
          load8(g, a.gate + 8 * vec[i]);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float gj = a.gate_kind == 0 ? 1.f
                           : a.gate_kind == 2 ? tok_gate
                           : (a.gate_kind == 1 && kKeep) ? gc[kKeep ? i : 0][j]
                                                         : g[j];
          v[i][j] = fmaf(gj, v[i][j], a.scale * rr[i][j]);
          if (in[i]) ss = fmaf(v[i][j], v[i][j], ss);
        }
        if (in[i]) {
          const int64_t at = t * a.nvec + vec[i];
          if constexpr (RF32) {
            u32x4* o = static_cast<u32x4*>(a.out) + 2 * at;
#pragma unroll
            for (int h = 0; h < 2; ++h)
              store16<NT>(o + h, u32x4{__float_as_uint(v[i][4 * h]), __float_as_uint(v[i][4 * h + 1]),
                                       __float_as_uint(v[i][4 * h + 2]), __float_as_uint(v[i][4 * h + 3])});
          } else {
            store8_bf16<NT>(a.out, at, v[i]);
          }
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[i][j] = rr[i][j];
          if (in[i]) ss = fmaf(rr[i][j], rr[i][j], ss);
        }
    }
    if (a.w_next) {
      const float inv = rsqrtf(fmaf(block_sum(ss, s_red, half), a.inv_h, a.eps));
      half ^= 1;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if constexpr (!kKeep) load8(wn[0], a.w_next + 8 * vec[i]);
        float n[8];
#pragma unroll
        for (int j = 0; j < 8; ++j) n[j] = v[i][j] * inv * wn[kKeep ? i : 0][j];
        if (in[i]) store8_bf16<NT>(a.normed, t * a.nvec + vec[i], n);
      }
    }
  }
}

template <int Y, bool RF32, bool NT>
hipError_t launch_as(const Args& a, hipStream_t stream) {
  const int cus = device_cu_count();
  // Few rows: one vector per thread, the shortest chain of a row. Many rows:
  // two vectors per thread from 513 vectors on, so that two or more rows are
  // in flight per CU beside the prefetched ones. (Not so with float32 on both
  // sides: 136 registers leave room for one row of more than 6 waves, 16384 x
  // 7168 332 us, 5.0 TB/s, and the kernels of four vectors with a float32 residual
  // keep 12 to 20 bytes a lane in scratch, 2048 x 16384 100 us, 4.7 TB/s.)
  const bool many = a.T > 2 * cus;
  const int nv = a.nvec <= (many ? 512 : 1024) ? 1 : a.nvec <= 1024 ? 2 : 4;
  const int nt = int(ceil_div(ceil_div(a.nvec, nv), 64) * 64);
  const int per_cu = std::max(1, std::min(16, 2048 / nt));
  const unsigned grid = unsigned(std::min<int64_t>(a.T, int64_t(cus) * per_cu));
  if (nv == 1)
    hipLaunchKernelGGL((block_norm_kernel<Y, RF32, 1, NT>), dim3(grid), dim3(nt), 0, stream, a);
  else if (nv == 2)
    hipLaunchKernelGGL((block_norm_kernel<Y, RF32, 2, NT>), dim3(grid), dim3(nt), 0, stream, a);
  else
    hipLaunchKernelGGL((block_norm_kernel<Y, RF32, 4, NT>), dim3(grid), dim3(nt), 0, stream, a);
  return hipGetLastError();
}

// Rows of more than the 256 MB of the last-level cache in all are not there any
// more when the next kernel reads them: they pass by (16384 x 7168 after a
// float32 block output: 201 us against 228; norm before it: 84 against 89).
// Fewer stay cached (16384 x 512: 16.7 us cached, 18.4 passed by).
constexpr int64_t kPassBy = int64_t(256) << 20;

template <int Y, bool RF32>
hipError_t launch(const Args& a, hipStream_t stream) {
  const int64_t per = (Y == 0 ? 0 : Y == 1 ? 2 : 4) + (RF32 ? 4 : 2) + (a.out ? (RF32 ? 4 : 2) : 0) + (a.normed ? 2 : 0);
  return int64_t(a.T) * a.H * per > kPassBy ? launch_as<Y, RF32, true>(a, stream) : launch_as<Y, RF32, false>(a, stream);
}

}  // namespace norm

hipError_t launch_block_norm(const void* y, int y_type, const void* r, bool r_f32, const float* w_post,
                             const float* gate, int gate_kind, float scale, const float* w_next, float eps, int T,
                             int H, void* out, uint16_t* normed, hipStream_t stream) {
  const norm::Args a{y, r, w_post, gate, w_next, out, normed, T, H / 8, H, gate_kind, scale, eps, 1.f / float(H)};
  if (y_type == 0)
    return r_f32 ? norm::launch<0, true>(a, stream) : norm::launch<0, false>(a, stream);
  if (y_type == 1)
    return r_f32 ? norm::launch<1, true>(a, stream) : norm::launch<1, false>(a, stream);
  return r_f32 ? norm::launch<2, true>(a, stream) : norm::launch<2, false>(a, stream);
}

}  // namespace moe

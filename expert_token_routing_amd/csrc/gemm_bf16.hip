// bf16 products with bias, activation and residual in the epilogue, for one
// weight matrix or for ragged expert segments:
//
//   C[m] = act(A[m] W_e + bias_e) + residual[m]
//
// float32 sums and epilogue, one rounding at the end.
#include "gemm_tile.h"
#include "moe_kernels.h"
#include "moe_row.h"

namespace moe {
namespace bf16gemm {

constexpr int kMaxLocal = 1024;
constexpr int kBM = 128, kBN = 256;

__device__ __forceinline__ float silu(float z) { return z / (1.f + expf(-z)); }
__device__ __forceinline__ float act(int kind, float z) {
  switch (kind) {
    case 1: return z > 0.f ? z : z == z ? 0.f : z;
    case 2: return silu(z);
    // 1 + erf and 1 + tanh cancel for z < 0
    case 3: return 0.5f * z * erfcf(z * -0.70710678f);
    case 4: return z / (1.f + expf(-1.5957691f * (z + 0.044715f * z * z * z)));
    default: return z;
  }
}

template <bool SWIGLU>
__global__ void __launch_bounds__(kThreads) simple_kernel(GemmBf16 p) {
  constexpr int FM = kBM / 64, FN = 4;
  __shared__ __attribute__((aligned(16))) uint16_t As[kBM * kLdk];
  __shared__ __attribute__((aligned(16))) uint16_t Bs[kBN * kLdk];
  const int cols = SWIGLU ? 2 * p.N : p.N;
  const int ntn = (cols + kBN - 1) / kBN;
  const int w = threadIdx.x >> 6, wm = w >> 1, wn = w & 1;
  const int lane = lane_id();
  for (int e = blockIdx.y; e < p.E_local; e += gridDim.y) {
    int64_t lo = 0, hi = p.capacity;
    if (p.offsets != nullptr) {
      lo = min<int64_t>(max<int64_t>(p.offsets[e], 0), p.capacity);
      hi = max<int64_t>(lo, min<int64_t>(p.offsets[e + 1], p.capacity));
    }
    const int64_t total = (hi - lo + kBM - 1) / kBM * ntn;
    const uint16_t* We = p.W + int64_t(e) * p.K * cols;
    const float* bias = p.bias == nullptr ? nullptr : p.bias + int64_t(e) * cols;
    for (int64_t tile = blockIdx.x; tile < total; tile += gridDim.x) {
      const int nj = int(tile % ntn);
      const int64_t r0 = lo + tile / ntn * kBM;
      const int rows = int(min<int64_t>(kBM, hi - r0));
      auto row_ptr = [&](int r) { return p.A + (r0 + min(r, rows - 1)) * p.K; };
      auto col_of = [&](int s0) -> int {
        if (SWIGLU) {
          const int q = s0 & 127, oc = nj * 128 + (s0 >> 7) * 64 + (q & 63);
          return oc >= p.N ? -1 : q < 64 ? oc : p.N + oc;
        }
        const int oc = nj * 256 + s0;
        return oc < p.N ? oc : -1;
      };
      f32x16 acc[FM][FN];
      zero_acc(acc);
      KRowsLoader<kBM> la;
      NColsTransposeLoader lb;
      for (int k0 = 0; k0 < p.K; k0 += kBK) {
        la.load(row_ptr, k0, p.K);
        lb.load(We, cols, col_of, k0, p.K);
        __syncthreads();
        la.store(As);
        lb.store(Bs);
        __syncthreads();
        mma_stage<FM, FN, 1, kBN>(As, Bs, wm * (kBM / 2), wn * 128, acc);
      }
      constexpr int FO = SWIGLU ? 2 : 4;
#pragma unroll
      for (int fm = 0; fm < FM; ++fm)
#pragma unroll
        for (int fn = 0; fn < FO; ++fn) {
          const int col = nj * (SWIGLU ? 128 : 256) + wn * (SWIGLU ? 64 : 128) + fn * 32 + (lane & 31);
#pragma unroll
          for (int v = 0; v < 16; ++v) {
            const int row = wm * (kBM / 2) + fm * 32 + mfma_c_row(v, lane);
            if (row < rows && col < p.N) {
              float z = acc[fm][fn][v] + (bias ? bias[col] : 0.f);
              if constexpr (SWIGLU)
                z = silu(z) * (acc[fm][fn + 2][v] + (bias ? bias[p.N + col] : 0.f));
              else
                z = act(p.act, z);
              const int64_t at = (r0 + row) * p.N + col;
              if (p.res != nullptr)
                z += p.res_f32 ? static_cast<const float*>(p.res)[at]
                               : bf16_to_f32(static_cast<const uint16_t*>(p.res)[at]);
              if (p.out_f32)
                static_cast<float*>(p.C)[at] = z;
              else
                static_cast<uint16_t*>(p.C)[at] = cvt_bf16(z);
            }
          }
        }
    }
  }
}

}  // namespace bf16gemm

hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t stream) {
  const bool swiglu = p.act == 5;
  const int64_t tiles = (ceil_div(p.capacity, bf16gemm::kBM)) * ceil_div(swiglu ? 2 * int64_t(p.N) : p.N, bf16gemm::kBN);
  const dim3 grid(unsigned(std::min<int64_t>(tiles, 1024)), unsigned(p.E_local));
  hipLaunchKernelGGL(swiglu ? bf16gemm::simple_kernel<true> : bf16gemm::simple_kernel<false>, grid, dim3(kThreads), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace moe

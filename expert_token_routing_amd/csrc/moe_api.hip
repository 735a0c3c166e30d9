// C-ABI of the MoE rank-share library: argument checks, workspace layout and
// the one-stream forward pass. Every check runs on the host before any launch.
#include <cmath>
#include <initializer_list>
#include <mutex>

#include "moe.h"
#include "moe_kernels.h"

namespace moe {

namespace {
constexpr int kMaxE = 1024;
constexpr int kMaxK = 32;
constexpr size_t kAlign = 256;

size_t align_up(size_t v) { return (v + kAlign - 1) / kAlign * kAlign; }

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

std::mutex g_dev_mu;
int g_cu_count[64] = {0};
void* g_scratch_ptr[64] = {nullptr};
}  // namespace

// The forward workspace of moe_forward_noalloc, for callers that cannot
// allocate. Each GPU the library runs on holds its own copy, from the load
// of the library's code on that GPU until the process ends.
static __device__ __align__(256) unsigned char scratch[MOE_NOALLOC_SCRATCH_BYTES];

// This device's address of `scratch`, looked up once per device with the
// device current (the array's name is not a device address in host code).
static int scratch_address(void** out) {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return MOE_ERR_HIP;
  if (dev >= 64) return MOE_ERR_UNSUPPORTED;
  std::lock_guard<std::mutex> lk(g_dev_mu);
  if (g_scratch_ptr[dev] == nullptr) {
    void* p = nullptr;
    if (hipGetSymbolAddress(&p, HIP_SYMBOL(scratch)) != hipSuccess || p == nullptr) return MOE_ERR_HIP;
    g_scratch_ptr[dev] = p;
  }
  *out = g_scratch_ptr[dev];
  return MOE_OK;
}

int device_cu_count() {
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0) return 256;
  if (dev < 64) {
    std::lock_guard<std::mutex> lk(g_dev_mu);
    if (g_cu_count[dev] == 0) {
      int cus = 0;
      if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
      g_cu_count[dev] = cus;
    }
    return g_cu_count[dev];
  }
  int cus = 0;
  if (hipDeviceGetAttribute(&cus, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || cus <= 0) cus = 256;
  return cus;
}

// Common checks of the problem statement (T, H, E, k, local block).
static int check_route_dims(int T, int H, int E, int k) {
  if (T < 0 || H <= 0 || (H % 8) != 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || k > kMaxK) return MOE_ERR_UNSUPPORTED;
  if (int64_t(T) * k >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static int check_local(int E, int e0, int E_local) {
  if (E_local < 1 || e0 < 0 || int64_t(e0) + E_local > E) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}
static int64_t min_capacity(int T, int k, int E_local) { return int64_t(T) * std::min(k, E_local); }
// Rows of the grouped GEMMs, which round them up to blocks in an int.
static bool rows_fit(int64_t rows) { return rows < (int64_t(1) << 31) - 1024; }
// The GEMMs address one expert's weight matrix through a buffer resource
// whose range and offsets are 32-bit: gate_up (H x 2I bf16, the larger of the
// two) must stay below 2 GiB, i.e. H * I < 2^29.
static bool expert_weights_fit(int H, int I) { return int64_t(H) * I * 4 < (int64_t(1) << 31); }
static int hip_status(hipError_t e) { return e == hipSuccess ? MOE_OK : MOE_ERR_HIP; }

// Workspace layout of moe_forward.
struct ForwardLayout {
  size_t planes, part, logits, topk_idx, topk_w, counts, offsets, perm_src, inv, chunks, x_perm, h, out, row_info,
      total;
};
static ForwardLayout forward_layout(int T, int H, int I, int E, int k, int E_local) {
  ForwardLayout L{};
  const int64_t cap = min_capacity(T, k, E_local);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  L.planes = take(size_t(3) * E * H * sizeof(uint16_t));
  L.part = take(size_t(route_k_parts(T, H, E) - 1) * T * E * sizeof(float));
  L.logits = take(size_t(T) * E * sizeof(float));
  L.topk_idx = take(size_t(T) * k * sizeof(int32_t));
  L.topk_w = take(size_t(T) * k * sizeof(float));
  L.counts = take(size_t(E) * sizeof(int32_t));
  L.offsets = take(size_t(E_local + 1) * sizeof(int32_t));
  L.perm_src = take(size_t(cap) * sizeof(int32_t));
  L.inv = take(size_t(T) * k * sizeof(int32_t));
  L.chunks = take(dispatch_table_bytes(T, E));
  // the dispatched rows: only when GEMM1 cannot read the token vectors in place
  L.x_perm = take(expert_gemm1_can_gather(T, H) ? 0 : size_t(cap) * H * sizeof(uint16_t));
  L.h = take(size_t(cap) * I * sizeof(uint16_t));
  L.out = take(size_t(cap) * H * sizeof(uint16_t));
  L.row_info = take(size_t(cap) * sizeof(int2));
  L.total = o;
  return L;
}

}  // namespace moe

using namespace moe;

extern "C" {

const char* moe_status_string(int status) {
  switch (status) {
    case MOE_OK: return "MOE_OK";
    case MOE_ERR_INVALID_ARG:
      return "MOE_ERR_INVALID_ARG: invalid size, value or index range, or a null or misaligned pointer";
    case MOE_ERR_UNSUPPORTED:
      return "MOE_ERR_UNSUPPORTED: outside the supported sizes (E <= 1024, k <= 32, T*k < 2^31, H*I < 2^29; "
             "moe_forward_few: T <= 32; 8-bit products: K < 131072, N*K < 2^31; norms: H <= 32768; "
             "moe_select: n_group <= 64; moe_gemm: K*columns < 2^30; "
             "the others stand at the entry point's declaration in moe.h)";
    case MOE_ERR_WORKSPACE: return "MOE_ERR_WORKSPACE: workspace missing, misaligned or too small";
    case MOE_ERR_HIP: return "MOE_ERR_HIP: a HIP launch failed";
    default: return "unknown moe_status";
  }
}

size_t moe_route_workspace_size(int T, int H, int E, int k) {
  (void)k;
  if (H <= 0 || E <= 0 || T < 0) return 0;
  return align_up(size_t(3) * E * H * sizeof(uint16_t)) +
         align_up(size_t(route_k_parts(T, H, E) - 1) * T * E * sizeof(float));
}

int moe_route(const moe_bf16* x, const float* w_router, const float* bias, int T, int H, int E, int k,
              int renormalize, float* logits, int32_t* topk_idx, float* topk_w, void* workspace,
              size_t workspace_bytes, hipStream_t stream) {
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !logits || !topk_idx || !topk_w || !aligned16(x) || !aligned16(w_router))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < moe_route_workspace_size(T, H, E, k))
    return MOE_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  return hip_status(launch_route(x, w_router, bias, T, H, E, k, renormalize, logits, topk_idx, topk_w,
                                 reinterpret_cast<uint16_t*>(ws),
                                 reinterpret_cast<float*>(ws + align_up(size_t(3) * E * H * sizeof(uint16_t))),
                                 stream));
}

size_t moe_dispatch_workspace_size(int T, int E, int k) {
  (void)k;
  if (T < 0 || E <= 0) return 0;
  return align_up(dispatch_table_bytes(T, E));
}

int moe_dispatch(const moe_bf16* x, const int32_t* topk_idx, int T, int H, int E, int k, int e0, int E_local,
                 int64_t capacity, int32_t* counts, int32_t* offsets, int32_t* perm_src, int32_t* inv,
                 moe_bf16* x_perm, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if (capacity < min_capacity(T, k, E_local)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!x || !topk_idx || !counts || !offsets || !perm_src || !inv || !x_perm) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(x_perm)) return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < moe_dispatch_workspace_size(T, E, k))
    return MOE_ERR_WORKSPACE;
  return hip_status(launch_dispatch(x, topk_idx, T, H, E, k, e0, E_local, counts, offsets, perm_src, inv, x_perm,
                                    static_cast<int32_t*>(workspace), stream));
}

int moe_expert_ffn(const moe_bf16* x_perm, const int32_t* offsets, const moe_bf16* w_gate_up,
                   const moe_bf16* w_down, int H, int I, int E_local, int64_t capacity, moe_bf16* h,
                   moe_bf16* out, hipStream_t stream) {
  if (H <= 0 || I <= 0 || (H % 8) != 0 || (I % 8) != 0 || E_local < 1 || capacity < 0) return MOE_ERR_INVALID_ARG;
  if (E_local > kMaxE || !expert_weights_fit(H, I)) return MOE_ERR_UNSUPPORTED;
  if (!rows_fit(capacity)) return MOE_ERR_UNSUPPORTED;
  if (capacity == 0) return MOE_OK;
  if (!x_perm || !offsets || !w_gate_up || !w_down || !h || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_perm) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(h) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  return hip_status(launch_expert_ffn(x_perm, offsets, w_gate_up, w_down, H, I, E_local, capacity, h, out, stream));
}

static int combine_impl(const moe_bf16* expert_out, const int32_t* inv, const float* topk_w, int T, int H, int k,
                        void* y, bool y_f32, hipStream_t stream) {
  if (T < 0 || H <= 0 || (H % 8) != 0 || k < 1) return MOE_ERR_INVALID_ARG;
  if (k > kMaxK) return MOE_ERR_UNSUPPORTED;
  if (int64_t(T) * k >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!expert_out || !inv || !topk_w || !y || !aligned16(expert_out) || !aligned16(y)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_combine(expert_out, inv, topk_w, T, H, k, y, y_f32, stream));
}

int moe_combine(const moe_bf16* expert_out, const int32_t* inv, const float* topk_w, int T, int H, int k,
                moe_bf16* y, hipStream_t stream) {
  return combine_impl(expert_out, inv, topk_w, T, H, k, y, false, stream);
}

int moe_combine_f32(const moe_bf16* expert_out, const int32_t* inv, const float* topk_w, int T, int H, int k,
                    float* y, hipStream_t stream) {
  return combine_impl(expert_out, inv, topk_w, T, H, k, y, true, stream);
}

size_t moe_forward_workspace_size(int T, int H, int I, int E, int k, int E_local) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || E_local <= 0) return 0;
  return forward_layout(T, H, I, E, k, E_local).total;
}

int moe_forward_workspace_layout(int T, int H, int I, int E, int k, int E_local, size_t* offsets_out) {
  if (!offsets_out || T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || E_local <= 0) return MOE_ERR_INVALID_ARG;
  const ForwardLayout L = forward_layout(T, H, I, E, k, E_local);
  const size_t v[9] = {L.logits, L.topk_idx, L.topk_w, L.counts, L.offsets, L.perm_src, L.inv, L.x_perm, L.out};
  for (int i = 0; i < 9; ++i) offsets_out[i] = v[i];
  return MOE_OK;
}

// The router's logits, and the choice by their scores.
static hipError_t route_scored(const moe_bf16* x, const float* w_router, const float* bias, const float* choice_bias,
                               int T, int H, int E, int k, const Choice& choice, float* logits, int32_t* topk_idx,
                               float* topk_w, uint16_t* planes, float* part, hipStream_t stream) {
  bool split;
  const hipError_t err = launch_route_logits(x, w_router, bias, T, H, E, logits, planes, part, &split, stream);
  if (err != hipSuccess) return err;
  return launch_select(logits, split ? part : nullptr, route_k_parts(T, H, E) - 1, bias, choice_bias, T, E, k, choice,
                       topk_idx, topk_w, stream);
}

// The launches of a share: selection (by router logits, or with `choice` by scores), dispatch,
// expert MLPs, combine. ws: forward_layout's.
static hipError_t share_steps(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                              const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                              int renormalize, const Choice* choice, const float* choice_bias, void* y, bool y_f32,
                              char* ws, hipEvent_t* events, hipStream_t stream, bool fuse_combine = false) {
  const ForwardLayout L = forward_layout(T, H, I, E, k, E_local);
  auto at = [&](size_t off) { return static_cast<void*>(ws + off); };
  const int64_t cap = min_capacity(T, k, E_local);
  float* logits = static_cast<float*>(at(L.logits));
  float* part = static_cast<float*>(at(L.part));
  uint16_t* planes = static_cast<uint16_t*>(at(L.planes));
  int32_t* topk_idx = static_cast<int32_t*>(at(L.topk_idx));
  float* topk_w = static_cast<float*>(at(L.topk_w));
  int32_t* counts = static_cast<int32_t*>(at(L.counts));
  int32_t* offsets = static_cast<int32_t*>(at(L.offsets));
  int32_t* perm_src = static_cast<int32_t*>(at(L.perm_src));
  int32_t* inv = static_cast<int32_t*>(at(L.inv));
  int32_t* chunks = static_cast<int32_t*>(at(L.chunks));
  uint16_t* x_perm = static_cast<uint16_t*>(at(L.x_perm));
  uint16_t* h = static_cast<uint16_t*>(at(L.h));
  uint16_t* out = static_cast<uint16_t*>(at(L.out));
  int2* row_info = static_cast<int2*>(at(L.row_info));
  // the combine of single-selection tokens runs in the down GEMM's epilogue
  const bool fuse = fuse_combine && !y_f32 && expert_gemm2_can_fuse(I);
  auto mark = [&](int i) { return events ? hipEventRecord(events[i], stream) : hipSuccess; };

  hipError_t err = mark(0);
  if (err == hipSuccess && choice)
    err = route_scored(x, w_router, bias, choice_bias, T, H, E, k, *choice, logits, topk_idx, topk_w, planes, part, stream);
  else if (err == hipSuccess)
    err = launch_route(x, w_router, bias, T, H, E, k, renormalize, logits, topk_idx, topk_w, planes, part, stream);
  if (err == hipSuccess) err = mark(1);
  // GEMM1 reads the token vectors in place when it can, so dispatch only
  // builds the tables; otherwise the rows are copied out first.
  const bool gather = expert_gemm1_can_gather(T, H);
  // rows a local expert holds when the T k selections spread evenly over
  // the E experts (the GEMMs take the grouped GEMV when that is small)
  const int64_t rows_hint = ceil_div(int64_t(T) * k, E);
  if (err == hipSuccess)
    err = gather ? launch_dispatch_index(topk_idx, T, E, k, e0, E_local, counts, offsets, perm_src, inv, chunks, stream)
                 : launch_dispatch(x, topk_idx, T, H, E, k, e0, E_local, counts, offsets, perm_src, inv, x_perm,
                                   chunks, stream);
  if (err == hipSuccess && fuse) err = launch_single_rows(inv, topk_w, T, k, row_info, stream);
  if (err == hipSuccess) err = mark(2);
  if (err == hipSuccess)
    err = gather ? launch_expert_gemm1_gather(x, perm_src, T, k, offsets, w_gate_up, H, I, E_local, cap, h, stream,
                                              rows_hint)
                 : launch_expert_gemm1(x_perm, offsets, w_gate_up, H, I, E_local, cap, h, stream, rows_hint);
  if (err == hipSuccess) err = mark(3);
  if (err == hipSuccess)
    err = fuse ? launch_expert_gemm2_fused(h, offsets, w_down, H, I, E_local, cap, row_info, out,
                                           static_cast<uint16_t*>(y), stream, rows_hint)
               : launch_expert_gemm2(h, offsets, w_down, H, I, E_local, cap, out, stream, rows_hint);
  if (err == hipSuccess) err = mark(4);
  if (err == hipSuccess) err = launch_combine(out, inv, topk_w, T, H, k, y, y_f32, stream, fuse);
  if (err == hipSuccess) err = mark(5);
  return err;
}

static int forward_impl(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                        const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                        int renormalize, void* y, bool y_f32, void* workspace, size_t workspace_bytes,
                        hipEvent_t* events, hipStream_t stream, bool fuse_combine = false) {
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if (I <= 0 || (I % 8) != 0) return MOE_ERR_INVALID_ARG;
  if (!expert_weights_fit(H, I)) return MOE_ERR_UNSUPPORTED;
  if (!rows_fit(min_capacity(T, k, E_local))) return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !w_gate_up || !w_down || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < forward_layout(T, H, I, E, k, E_local).total)
    return MOE_ERR_WORKSPACE;
  return hip_status(share_steps(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, nullptr,
                                nullptr, y, y_f32, static_cast<char*>(workspace), events, stream, fuse_combine));
}

int moe_forward(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                moe_bf16* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false,
                      workspace, workspace_bytes, nullptr, stream);
}

int moe_forward_noalloc(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                        const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                        moe_bf16* y, hipStream_t stream) {
  // the argument checks first, so that a rejected call has no side effect
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if (I <= 0 || (I % 8) != 0) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (forward_layout(T, H, I, E, k, E_local).total > size_t(MOE_NOALLOC_SCRATCH_BYTES)) return MOE_ERR_WORKSPACE;
  void* ws = nullptr;
  if ((st = scratch_address(&ws)) != MOE_OK) return st;
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false, ws,
                      size_t(MOE_NOALLOC_SCRATCH_BYTES), nullptr, stream);
}

int moe_forward_f32(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                    const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                    float* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, true,
                      workspace, workspace_bytes, nullptr, stream);
}

int moe_forward_profiled(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                         const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                         int renormalize, moe_bf16* y, void* workspace, size_t workspace_bytes,
                         hipEvent_t* events, hipStream_t stream) {
  if (!events) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i)
    if (!events[i]) return MOE_ERR_INVALID_ARG;
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false,
                      workspace, workspace_bytes, events, stream);
}

int moe_forward_fused(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                      const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                      int renormalize, moe_bf16* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false,
                      workspace, workspace_bytes, nullptr, stream, true);
}

int moe_forward_fused_profiled(const moe_bf16* x, const float* w_router, const float* bias,
                               const moe_bf16* w_gate_up, const moe_bf16* w_down, int T, int H, int I, int E, int k,
                               int e0, int E_local, int renormalize, moe_bf16* y, void* workspace,
                               size_t workspace_bytes, hipEvent_t* events, hipStream_t stream) {
  if (!events) return MOE_ERR_INVALID_ARG;
  for (int i = 0; i < 6; ++i)
    if (!events[i]) return MOE_ERR_INVALID_ARG;
  return forward_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false,
                      workspace, workspace_bytes, events, stream, true);
}

size_t moe_few_workspace_size(int T, int H, int I, int E, int k, int E_local) {
  if (T < 0 || T > MOE_FEW_TOKENS || H <= 0 || I <= 0 || E <= 0 || k <= 0 || E_local <= 0) return 0;
  return few_workspace_bytes(T, H, I, E, k, E_local);
}

static int few_impl(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                    const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                    void* y, bool y_f32, void* workspace, size_t workspace_bytes, hipStream_t stream,
                    int workgroups = 0, int polls = kFewPolls) {
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if (I <= 0 || (I % 8) != 0 || workgroups < 0 || polls < 1) return MOE_ERR_INVALID_ARG;
  if (T > MOE_FEW_TOKENS || !expert_weights_fit(H, I) || !few_supported(T, H, I, k, E_local))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !w_gate_up || !w_down || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate_up) || !aligned16(w_down) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 ||
      workspace_bytes < few_workspace_bytes(T, H, I, E, k, E_local))
    return MOE_ERR_WORKSPACE;
  return hip_status(launch_few(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, y_f32,
                               workgroups, polls, static_cast<char*>(workspace), stream));
}

int moe_forward_few(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                    const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                    moe_bf16* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return few_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, false, workspace,
                  workspace_bytes, stream);
}

int moe_forward_few_f32(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                        const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                        int renormalize, float* y, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return few_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, true, workspace,
                  workspace_bytes, stream);
}

// moe_forward_few_f32 with another number of workgroups (at least 8; 0: two per
// CU) and of polls before a waiting workgroup puts its item aside for others'
// work. That work is there only where workgroups wait while queues still hold
// earlier items, which two per CU hardly leave (at most 5 items of a call even
// with one poll): the tests call this one with few workgroups, where up to 700
// items of a call are taken that way. Not part of moe.h.
int moe_internal_forward_few(const moe_bf16* x, const float* w_router, const float* bias, const moe_bf16* w_gate_up,
                             const moe_bf16* w_down, int T, int H, int I, int E, int k, int e0, int E_local,
                             int renormalize, float* y, void* workspace, size_t workspace_bytes, int workgroups,
                             int polls, hipStream_t stream) {
  return few_impl(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, y, true, workspace,
                  workspace_bytes, stream, workgroups, polls);
}

// Sizes of the 8-bit products: an exact int32 sum needs K < 2^17; 32-bit
// offsets into one expert's matrix need rows * K < 2^31.
static int check_i8(int K, int64_t channels) {
  if (K <= 0 || (K % 16) != 0 || channels <= 0 || (channels % 8) != 0) return MOE_ERR_INVALID_ARG;
  if (K >= (1 << 17) || channels * K >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Rows and tiles of a grouped product are counted with 31 bits: at the smallest
// blocks (16 rows) and narrowest tiles (32 channels).
static bool i8_rows_fit(int64_t capacity, int E_local, int64_t channels) {
  return rows_fit(capacity) &&
         (ceil_div(capacity, 16) + E_local) * ceil_div(channels, 32) < (int64_t(1) << 31);
}

int moe_quantize_rows(const moe_bf16* x, int64_t M, int K, int8_t* q, float* scale, hipStream_t stream) {
  if (M < 0 || K <= 0 || (K % 16) != 0) return MOE_ERR_INVALID_ARG;
  if (M >= (int64_t(1) << 31)) return MOE_ERR_UNSUPPORTED;
  if (M == 0) return MOE_OK;
  if (!x || !q || !scale || !aligned16(x) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_quantize_rows(x, false, nullptr, M, K, q, scale, stream));
}

int moe_quantize_weights(const moe_bf16* w, int E_local, int K, int N, int8_t* q, float* scale, hipStream_t stream) {
  if (E_local < 1) return MOE_ERR_INVALID_ARG;
  const int st = check_i8(K, N);
  if (st != MOE_OK) return st;
  if (E_local > kMaxE) return MOE_ERR_UNSUPPORTED;
  if (!w || !q || !scale || !aligned16(w) || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_quantize_weights(w, E_local, K, N, q, scale, stream));
}

int moe_gemm_i8(const int8_t* a, const float* a_scale, const int32_t* offsets, const int8_t* w, const float* w_scale,
                int64_t capacity, int N, int K, int E_local, moe_bf16* out, hipStream_t stream) {
  if (E_local < 1 || capacity < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_i8(K, N);
  if (st != MOE_OK) return st;
  if (E_local > kMaxE || !i8_rows_fit(capacity, E_local, N)) return MOE_ERR_UNSUPPORTED;
  if (!offsets && E_local != 1) return MOE_ERR_INVALID_ARG;
  if (capacity == 0) return MOE_OK;
  if (!a || !a_scale || !w || !w_scale || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(w) || !aligned16(w_scale) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_gemm_i8(a, a_scale, offsets, E_local, capacity, w, w_scale, K, N, out,
                                   ceil_div(capacity, E_local), stream));
}

}  // extern "C"

namespace moe {
// The grouped MLPs' intermediates: quantised rows in, h, quantised h.
struct FfnI8Layout {
  size_t xq, xs, h, hq, hs, total;
};
static FfnI8Layout ffn_i8_layout(size_t at, int64_t x_rows, int64_t cap, int H, int I) {
  FfnI8Layout L{};
  auto take = [&](size_t bytes) {
    const size_t o = at;
    at = align_up(at + bytes);
    return o;
  };
  L.xq = take(size_t(x_rows) * H);
  L.xs = take(size_t(x_rows) * sizeof(float));
  L.h = take(size_t(cap) * I * sizeof(float));
  L.hq = take(size_t(cap) * I);
  L.hs = take(size_t(cap) * sizeof(float));
  L.total = at;
  return L;
}

// quantise -> gate/up -> quantise -> down. x: x_rows rows, of which row n of a
// segment is gather_src[n] / gather_k (gather_src given) or row n.
static hipError_t ffn_i8(const moe_bf16* x, int64_t x_rows, const int32_t* gather_src, int gather_k,
                         const int32_t* offsets, const int8_t* w_gate_up, const float* s_gate_up,
                         const int8_t* w_down, const float* s_down, int H, int I, int E_local, int64_t cap,
                         const FfnI8Layout& L, char* ws, moe_bf16* out, int64_t rows_hint, hipStream_t stream) {
  int8_t* xq = reinterpret_cast<int8_t*>(ws + L.xq);
  float* xs = reinterpret_cast<float*>(ws + L.xs);
  float* h = reinterpret_cast<float*>(ws + L.h);
  int8_t* hq = reinterpret_cast<int8_t*>(ws + L.hq);
  float* hs = reinterpret_cast<float*>(ws + L.hs);
  const int32_t* end = offsets + E_local;
  hipError_t err = launch_quantize_rows(x, false, gather_src ? nullptr : end, x_rows, H, xq, xs, stream);
  if (err == hipSuccess)
    err = launch_gate_up_i8(xq, xs, gather_src, gather_k, int(x_rows), offsets, E_local, cap, w_gate_up, s_gate_up, H,
                            I, h, rows_hint, stream);
  if (err == hipSuccess) err = launch_quantize_rows(h, true, end, cap, I, hq, hs, stream);
  if (err == hipSuccess)
    err = launch_gemm_i8(hq, hs, offsets, E_local, cap, w_down, s_down, I, H, out, rows_hint, stream);
  return err;
}

static int check_ffn_i8(int H, int I) {
  const int st = check_i8(H, int64_t(2) * I);
  if (st != MOE_OK) return st;
  return check_i8(I, H);
}

struct ForwardI8Layout {
  size_t planes, part, logits, topk_idx, topk_w, counts, offsets, perm_src, inv, chunks, out;
  FfnI8Layout ffn;
};
static ForwardI8Layout forward_i8_layout(int T, int H, int I, int E, int k, int E_local) {
  ForwardI8Layout L{};
  const int64_t cap = min_capacity(T, k, E_local);
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  L.planes = take(size_t(3) * E * H * sizeof(uint16_t));
  L.part = take(size_t(route_k_parts(T, H, E) - 1) * T * E * sizeof(float));
  L.logits = take(size_t(T) * E * sizeof(float));
  L.topk_idx = take(size_t(T) * k * sizeof(int32_t));
  L.topk_w = take(size_t(T) * k * sizeof(float));
  L.counts = take(size_t(E) * sizeof(int32_t));
  L.offsets = take(size_t(E_local + 1) * sizeof(int32_t));
  L.perm_src = take(size_t(cap) * sizeof(int32_t));
  L.inv = take(size_t(T) * k * sizeof(int32_t));
  L.chunks = take(dispatch_table_bytes(T, E));
  L.out = take(size_t(cap) * H * sizeof(uint16_t));
  L.ffn = ffn_i8_layout(o, T, cap, H, I);
  return L;
}
}  // namespace moe

extern "C" {

// The row blocks of the grouped products, for the tests of sizes next to 2^31. Not part
// of moe.h.
int moe_internal_row_blocks(int rows, int cap, int* height) {
  const int n = row_blocks(rows, cap);
  *height = block_height(rows, std::max(n, 1));
  return n;
}

// The tiles of a product, for the tests of the rule. Not part of moe.h.
int moe_internal_i8_tile(int swiglu, int ragged, int E_local, int64_t capacity, int N, int K, int64_t rows_hint,
                         int cus) {
  return i8_tile(swiglu != 0, ragged != 0, E_local, capacity, N, K, rows_hint, cus);
}

size_t moe_expert_ffn_i8_workspace_size(int H, int I, int64_t capacity) {
  if (H <= 0 || I <= 0 || capacity < 0) return 0;
  return ffn_i8_layout(0, capacity, capacity, H, I).total;
}

int moe_expert_ffn_i8(const moe_bf16* x_perm, const int32_t* offsets, const int8_t* w_gate_up,
                      const float* s_gate_up, const int8_t* w_down, const float* s_down, int H, int I, int E_local,
                      int64_t capacity, moe_bf16* out, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  if (E_local < 1 || capacity < 0) return MOE_ERR_INVALID_ARG;
  const int st = check_ffn_i8(H, I);
  if (st != MOE_OK) return st;
  if (E_local > kMaxE || !i8_rows_fit(capacity, E_local, std::max(H, I))) return MOE_ERR_UNSUPPORTED;
  if (capacity == 0) return MOE_OK;
  if (!x_perm || !offsets || !w_gate_up || !s_gate_up || !w_down || !s_down || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x_perm) || !aligned16(w_gate_up) || !aligned16(s_gate_up) || !aligned16(w_down) ||
      !aligned16(s_down) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  const FfnI8Layout L = ffn_i8_layout(0, capacity, capacity, H, I);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 || workspace_bytes < L.total)
    return MOE_ERR_WORKSPACE;
  return hip_status(ffn_i8(x_perm, capacity, nullptr, 1, offsets, w_gate_up, s_gate_up, w_down, s_down, H, I, E_local,
                           capacity, L, static_cast<char*>(workspace), out, ceil_div(capacity, E_local), stream));
}

size_t moe_forward_i8_workspace_size(int T, int H, int I, int E, int k, int E_local) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0 || E_local <= 0) return 0;
  return forward_i8_layout(T, H, I, E, k, E_local).ffn.total;
}

int moe_forward_i8(const moe_bf16* x, const float* w_router, const float* bias, const int8_t* w_gate_up,
                   const float* s_gate_up, const int8_t* w_down, const float* s_down, int T, int H, int I, int E,
                   int k, int e0, int E_local, int renormalize, moe_bf16* y, void* workspace,
                   size_t workspace_bytes, hipStream_t stream) {
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if ((st = check_ffn_i8(H, I)) != MOE_OK) return st;
  if (!i8_rows_fit(min_capacity(T, k, E_local), E_local, std::max(H, I)) || int64_t(T) * H >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !w_gate_up || !s_gate_up || !w_down || !s_down || !y) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(w_router) || !aligned16(w_gate_up) || !aligned16(s_gate_up) || !aligned16(w_down) ||
      !aligned16(s_down) || !aligned16(y))
    return MOE_ERR_INVALID_ARG;
  const ForwardI8Layout L = forward_i8_layout(T, H, I, E, k, E_local);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 || workspace_bytes < L.ffn.total)
    return MOE_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  auto at = [&](size_t off) { return static_cast<void*>(ws + off); };
  int32_t* topk_idx = static_cast<int32_t*>(at(L.topk_idx));
  float* topk_w = static_cast<float*>(at(L.topk_w));
  int32_t* offsets = static_cast<int32_t*>(at(L.offsets));
  int32_t* perm_src = static_cast<int32_t*>(at(L.perm_src));
  int32_t* inv = static_cast<int32_t*>(at(L.inv));
  uint16_t* out = static_cast<uint16_t*>(at(L.out));
  hipError_t err = launch_route(x, w_router, bias, T, H, E, k, renormalize, static_cast<float*>(at(L.logits)),
                                topk_idx, topk_w, static_cast<uint16_t*>(at(L.planes)),
                                static_cast<float*>(at(L.part)), stream);
  if (err == hipSuccess)
    err = launch_dispatch_index(topk_idx, T, E, k, e0, E_local, static_cast<int32_t*>(at(L.counts)), offsets,
                                perm_src, inv, static_cast<int32_t*>(at(L.chunks)), stream);
  if (err == hipSuccess)
    err = ffn_i8(x, T, perm_src, k, offsets, w_gate_up, s_gate_up, w_down, s_down, H, I, E_local,
                 min_capacity(T, k, E_local), L.ffn, ws, out, ceil_div(int64_t(T) * k, E), stream);
  if (err == hipSuccess) err = launch_combine(out, inv, topk_w, T, H, k, y, false, stream, false);
  return hip_status(err);
}

static int check_norm(int T, int H, float eps) {
  if (T < 0 || H <= 0 || (H % 8) != 0 || !(eps >= 0.f) || !std::isfinite(eps)) return MOE_ERR_INVALID_ARG;
  if (H > MOE_NORM_MAX_H) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}
static bool type_ok(int t) { return t == MOE_TYPE_BF16 || t == MOE_TYPE_F32; }

// moe_norm_post's sizes, types and optional arguments.
static int check_post(int r_type, int y_type, const float* gate, int gate_kind, const float* w_next,
                      const moe_bf16* normed, int T, int H, float eps) {
  const int st = check_norm(T, H, eps);
  if (st != MOE_OK) return st;
  if (!type_ok(y_type) || !type_ok(r_type) || gate_kind < MOE_GATE_NONE || gate_kind > MOE_GATE_FULL)
    return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;  // (empty arrays may be NULL)
  if ((gate_kind == MOE_GATE_NONE) != (gate == nullptr) || (w_next == nullptr) != (normed == nullptr))
    return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

int moe_norm_pre(const void* r, int r_type, const float* w, float eps, int T, int H, moe_bf16* out,
                 hipStream_t stream) {
  const int st = check_norm(T, H, eps);
  if (st != MOE_OK) return st;
  if (!type_ok(r_type)) return MOE_ERR_INVALID_ARG;
  if (T == 0) return MOE_OK;
  if (!r || !w || !out || !aligned16(r) || !aligned16(w) || !aligned16(out)) return MOE_ERR_INVALID_ARG;
  return hip_status(launch_block_norm(nullptr, 0, r, r_type == MOE_TYPE_F32, nullptr, nullptr, MOE_GATE_NONE, 1.f, w,
                                      eps, T, H, nullptr, out, stream));
}

int moe_norm_post(const void* y, int y_type, const void* residual, int r_type, const float* w_post,
                  const float* gate, int gate_kind, float residual_scale, const float* w_next, float eps, int T,
                  int H, void* out, moe_bf16* normed, hipStream_t stream) {
  const int st = check_post(r_type, y_type, gate, gate_kind, w_next, normed, T, H, eps);
  if (st != MOE_OK || T == 0) return st;
  if (!y || !residual || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(y) || !aligned16(residual) || !aligned16(out) || !aligned16(w_post) || !aligned16(w_next) ||
      !aligned16(normed) || (gate_kind != MOE_GATE_TOKEN && !aligned16(gate)))
    return MOE_ERR_INVALID_ARG;
  return hip_status(launch_block_norm(y, y_type == MOE_TYPE_F32 ? 2 : 1, residual, r_type == MOE_TYPE_F32, w_post,
                                      gate, gate_kind, residual_scale, w_next, eps, T, H, out, normed, stream));
}

// The block's own buffers, then the layer's workspace. Up to 16 tokens the
// two-kernel layer is the faster one at every shape measured (DeepSeek-R1 EP=8
// share 34 us against 134 at one token, 204 against 257 at 16); at 24 to 32 the
// two are within 10% of each other either way.
static bool block_is_few(int T, int H, int I, int E, int k) { return T <= 16 && few_supported(T, H, I, k, E); }
struct BlockLayout {
  size_t x, y, layer, total;
};
static BlockLayout block_layout(int T, int H, int I, int E, int k) {
  BlockLayout L{};
  L.y = align_up(size_t(T) * H * sizeof(uint16_t));
  L.layer = L.y + align_up(size_t(T) * H * sizeof(float));
  L.total = L.layer + (block_is_few(T, H, I, E, k) ? few_workspace_bytes(T, H, I, E, k, E)
                                                : forward_layout(T, H, I, E, k, E).total);
  return L;
}

size_t moe_block_workspace_size(int T, int H, int I, int E, int k) {
  if (T < 0 || H <= 0 || I <= 0 || E <= 0 || k <= 0) return 0;
  return block_layout(T, H, I, E, k).total;
}

int moe_block_forward(const void* residual, int r_type, const float* w_pre, const float* w_router,
                      const float* bias, const moe_bf16* w_gate_up, const moe_bf16* w_down, const float* w_post,
                      const float* gate, int gate_kind, float residual_scale, const float* w_next, float eps, int T,
                      int H, int I, int E, int k, int renormalize, void* out, moe_bf16* normed, void* workspace,
                      size_t workspace_bytes, hipStream_t stream) {
  // every step's checks before the first launch
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if (I <= 0 || (I % 8) != 0) return MOE_ERR_INVALID_ARG;
  if (!expert_weights_fit(H, I) || !rows_fit(min_capacity(T, k, E))) return MOE_ERR_UNSUPPORTED;
  if ((st = check_post(r_type, MOE_TYPE_F32, gate, gate_kind, w_next, normed, T, H, eps)) != MOE_OK) return st;
  if (T == 0) return MOE_OK;
  if (!residual || !w_pre || !w_router || !w_gate_up || !w_down || !out) return MOE_ERR_INVALID_ARG;
  for (const void* q : {residual, static_cast<const void*>(w_pre), static_cast<const void*>(w_router),
                        static_cast<const void*>(w_gate_up), static_cast<const void*>(w_down),
                        static_cast<const void*>(w_post), static_cast<const void*>(w_next),
                        static_cast<const void*>(out), static_cast<const void*>(normed)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (gate_kind != MOE_GATE_TOKEN && !aligned16(gate)) return MOE_ERR_INVALID_ARG;
  const BlockLayout L = block_layout(T, H, I, E, k);
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) % kAlign) != 0 || workspace_bytes < L.total)
    return MOE_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  moe_bf16* x = reinterpret_cast<moe_bf16*>(ws + L.x);
  float* y = reinterpret_cast<float*>(ws + L.y);
  st = moe_norm_pre(residual, r_type, w_pre, eps, T, H, x, stream);
  if (st == MOE_OK)
    st = block_is_few(T, H, I, E, k)
             ? moe_forward_few_f32(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, 0, E, renormalize, y,
                                   ws + L.layer, workspace_bytes - L.layer, stream)
             : moe_forward_f32(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, 0, E, renormalize, y,
                               ws + L.layer, workspace_bytes - L.layer, stream);
  if (st == MOE_OK)
    st = moe_norm_post(y, MOE_TYPE_F32, residual, r_type, w_post, gate, gate_kind, residual_scale, w_next, eps, T, H,
                       out, normed, stream);
  return st;
}

}  // extern "C"

namespace moe {
static bool aligned256(const void* p) { return (reinterpret_cast<uintptr_t>(p) % kAlign) == 0; }

// moe_select's sizes and kinds (T, E and k are check_route_dims').
static int check_choice(int T, int E, int k, const Choice& c) {
  if (T < 0 || E < 1 || k < 1 || k > E) return MOE_ERR_INVALID_ARG;
  if ((c.score != MOE_SCORE_SOFTMAX && c.score != MOE_SCORE_SIGMOID) ||
      (c.group_rule != MOE_GROUP_MAX && c.group_rule != MOE_GROUP_TOP2) || !std::isfinite(c.scale))
    return MOE_ERR_INVALID_ARG;
  if (c.n_group < 1 || E % c.n_group != 0 || c.topk_group < 1 || c.topk_group > c.n_group ||
      k > c.topk_group * (E / c.n_group))
    return MOE_ERR_INVALID_ARG;
  if (E > kMaxE || k > kMaxK || c.n_group > MOE_MAX_GROUPS || int64_t(T) * k >= (int64_t(1) << 31))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// Products of moe_gemm: 32-bit byte offsets into one expert's matrix, tiles
// counted with 31 bits.
static int check_gemm(int64_t capacity, int N, int K, int E_local, int activation) {
  if (capacity < 0 || N <= 0 || K <= 0 || (N % 8) != 0 || (K % 8) != 0 || E_local < 1 || activation < MOE_ACT_NONE ||
      activation > MOE_ACT_SWIGLU)
    return MOE_ERR_INVALID_ARG;
  const int64_t cols = activation == MOE_ACT_SWIGLU ? 2 * int64_t(N) : N;
  if (cols * K >= (int64_t(1) << 30) || K >= (1 << 20) || E_local > kMaxE || !i8_rows_fit(capacity, E_local, cols))
    return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

// The layer's own buffers (for a few tokens the selection; where the shared expert is a
// product of its own, the float32 share, h and the products' sums) and behind them the
// share's, in the form that the sizes take. Up to 32 tokens that is the share for a few
// tokens, with the shared expert among the local ones: all hidden values stay float32, and
// it is the faster one (us, the other form first: DeepSeek-R1 TP=8 share, 1 token 58 and 43,
// EP=8, 24 tokens 316 and 236, 32 tokens 332 and 270; 17 tokens, H 5336, I 208, I_shared
// 1936: 384 and 97). Layers whose experts are next to nothing (17 tokens, H 136, I 40: 51
// and 28) keep the bits of the separate calls from 17 tokens on.
static bool layer_is_few(int T, int H, int I, int k, int E_local) {
  return T <= (int64_t(H) * I < 8192 ? 16 : MOE_FEW_TOKENS) && few_supported(T, H, I, k, E_local);
}
static int layer_few_shared(int T, int H, int I, int k, int E_local, int I_shared) {
  return layer_is_few(T, H, I, k, E_local) ? few_shared(T, H, I, k, E_local, I_shared) : 0;
}
struct LayerLayout {
  size_t topk_idx, topk_w, share, h, part, part_bytes, rest, total;
};
static LayerLayout layer_layout(int T, int H, int I, int I_shared, int E, int k, int E_local) {
  LayerLayout L{};
  size_t o = 0;
  auto take = [&](size_t bytes) {
    const size_t at = o;
    o = align_up(o + bytes);
    return at;
  };
  const int inside = layer_few_shared(T, H, I, k, E_local, I_shared);
  const bool few = layer_is_few(T, H, I, k, E_local), apart = I_shared > 0 && inside == 0 && T > 0;
  L.topk_idx = take(few ? size_t(T) * k * sizeof(int32_t) : 0);
  L.topk_w = take(few ? size_t(T) * k * sizeof(float) : 0);
  L.share = take(apart ? size_t(T) * H * sizeof(float) : 0);
  L.h = take(apart ? size_t(T) * I_shared * sizeof(uint16_t) : 0);
  if (apart)
    L.part_bytes = std::max(moe_gemm_workspace_size(T, I_shared, H, 1, MOE_ACT_SWIGLU),
                            moe_gemm_workspace_size(T, H, I_shared, 1, MOE_ACT_NONE));
  L.part = take(L.part_bytes);
  L.rest = o;
  L.total = o + (few ? few_workspace_bytes(T, H, I, E, k, E_local, inside) : forward_layout(T, H, I, E, k, E_local).total);
  return L;
}
}  // namespace moe

extern "C" {

int moe_select(const float* logits, const float* bias, int T, int E, int k, int score, int n_group, int topk_group,
               int group_rule, int renormalize, float scale, int32_t* topk_idx, float* topk_w, hipStream_t stream) {
  const Choice c{score, n_group, topk_group, group_rule, renormalize, scale};
  const int st = check_choice(T, E, k, c);
  if (st != MOE_OK || T == 0) return st;
  if (!logits || !topk_idx || !topk_w) return MOE_ERR_INVALID_ARG;
  // (without parts the logits are only read)
  return hip_status(launch_select(const_cast<float*>(logits), nullptr, 0, nullptr, bias, T, E, k, c, topk_idx, topk_w,
                                  stream));
}

int moe_route_scored(const moe_bf16* x, const float* w_router, const float* bias, const float* choice_bias, int T,
                     int H, int E, int k, int score, int n_group, int topk_group, int group_rule, int renormalize,
                     float scale, float* logits, int32_t* topk_idx, float* topk_w, void* workspace,
                     size_t workspace_bytes, hipStream_t stream) {
  const Choice c{score, n_group, topk_group, group_rule, renormalize, scale};
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_choice(T, E, k, c)) != MOE_OK || T == 0) return st;
  if (!x || !w_router || !logits || !topk_idx || !topk_w || !aligned16(x) || !aligned16(w_router))
    return MOE_ERR_INVALID_ARG;
  if (!workspace || !aligned256(workspace) || workspace_bytes < moe_route_workspace_size(T, H, E, k))
    return MOE_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  float* part = reinterpret_cast<float*>(ws + align_up(size_t(3) * E * H * sizeof(uint16_t)));
  return hip_status(route_scored(x, w_router, bias, choice_bias, T, H, E, k, c, logits, topk_idx, topk_w,
                                 reinterpret_cast<uint16_t*>(ws), part, stream));
}

static int gemm_impl(const moe_bf16* a, const moe_bf16* w, const float* bias, const void* residual, int res_type,
                     const int32_t* offsets, int64_t capacity, int N, int K, int E_local, int activation, void* out,
                     int out_type, void* workspace, size_t workspace_bytes, hipStream_t stream, int tile = -1,
                     int ranges = 1) {
  const int st = check_gemm(capacity, N, K, E_local, activation);
  if (st != MOE_OK) return st;
  if (!type_ok(out_type) || (residual && !type_ok(res_type)) || (!offsets && E_local != 1)) return MOE_ERR_INVALID_ARG;
  if (capacity == 0) return MOE_OK;
  if (!a || !w || !out) return MOE_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(w) || !aligned16(bias) || !aligned16(residual) || !aligned16(out))
    return MOE_ERR_INVALID_ARG;
  const GemmBf16 p{a, w, bias, residual, out, offsets, capacity, E_local, K, N, activation, res_type == MOE_TYPE_F32,
                   out_type == MOE_TYPE_F32, static_cast<float*>(workspace)};
  const size_t need = gemm_bf16_part_bytes(p, tile, ranges);
  if (need > 0 && (!workspace || !aligned256(workspace) || workspace_bytes < need)) return MOE_ERR_WORKSPACE;
  return hip_status(launch_gemm_bf16(p, stream, tile, ranges));
}

size_t moe_gemm_workspace_size(int64_t capacity, int N, int K, int E_local, int activation) {
  if (check_gemm(capacity, N, K, E_local, activation) != MOE_OK || capacity == 0) return 0;
  GemmBf16 p{};
  p.capacity = capacity;
  p.E_local = E_local;
  p.K = K;
  p.N = N;
  p.act = activation;
  return gemm_bf16_part_bytes(p);
}

int moe_gemm(const moe_bf16* a, const moe_bf16* w, const float* bias, const void* residual, int res_type,
             const int32_t* offsets, int64_t capacity, int N, int K, int E_local, int activation, void* out,
             int out_type, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return gemm_impl(a, w, bias, residual, res_type, offsets, capacity, N, K, E_local, activation, out, out_type,
                   workspace, workspace_bytes, stream);
}

// moe_gemm on given tiles and k ranges, and those that a call takes, for the tests
// of every kind at sizes that the rule gives to another. Not part of moe.h.
int moe_internal_gemm(const moe_bf16* a, const moe_bf16* w, const float* bias, const void* residual, int res_type,
                      const int32_t* offsets, int64_t capacity, int N, int K, int E_local, int activation, void* out,
                      int out_type, int tile, int ranges, void* workspace, size_t workspace_bytes,
                      hipStream_t stream) {
  if (tile < 0 || ranges < 1) return MOE_ERR_INVALID_ARG;
  return gemm_impl(a, w, bias, residual, res_type, offsets, capacity, N, K, E_local, activation, out, out_type,
                   workspace, workspace_bytes, stream, tile, ranges);
}
int moe_internal_gemm_plan(int swiglu, int E_local, int64_t capacity, int N, int K, int cus, int* ranges) {
  return gemm_bf16_plan(swiglu != 0, E_local, capacity, N, K, cus, ranges);
}

size_t moe_layer_workspace_size(int T, int H, int I, int I_shared, int E, int k, int E_local) {
  if (T < 0 || H <= 0 || I <= 0 || I_shared < 0 || E <= 0 || k <= 0 || E_local <= 0) return 0;
  return layer_layout(T, H, I, I_shared, E, k, E_local).total;
}

static int layer_impl(const moe_bf16* x, const float* w_router, const float* bias, const float* choice_bias,
                      const moe_bf16* w_gate_up, const moe_bf16* w_down, const moe_bf16* w_shared_gate_up,
                      const moe_bf16* w_shared_down, int T, int H, int I, int I_shared, int E, int k, int e0,
                      int E_local, int score, int n_group, int topk_group, int group_rule, int renormalize,
                      float scale, void* y, int y_type, void* workspace, size_t workspace_bytes, hipStream_t stream,
                      int workgroups = 0, int polls = kFewPolls) {
  const Choice c{score, n_group, topk_group, group_rule, renormalize, scale};
  // every step's checks before the first launch
  int st = check_route_dims(T, H, E, k);
  if (st != MOE_OK) return st;
  if ((st = check_choice(T, E, k, c)) != MOE_OK || (st = check_local(E, e0, E_local)) != MOE_OK) return st;
  if (I <= 0 || (I % 8) != 0 || I_shared < 0 || (I_shared % 8) != 0 || !type_ok(y_type) || workgroups < 0 || polls < 1)
    return MOE_ERR_INVALID_ARG;
  if (!expert_weights_fit(H, I) || !expert_weights_fit(H, I_shared) || !rows_fit(min_capacity(T, k, E_local)))
    return MOE_ERR_UNSUPPORTED;
  if (I_shared > 0) {
    if ((st = check_gemm(T, I_shared, H, 1, MOE_ACT_SWIGLU)) != MOE_OK) return st;
    if ((st = check_gemm(T, H, I_shared, 1, MOE_ACT_NONE)) != MOE_OK) return st;
  }
  if (T == 0) return MOE_OK;
  if (!x || !w_router || !w_gate_up || !w_down || !y || (I_shared > 0) != (w_shared_gate_up != nullptr) ||
      (I_shared > 0) != (w_shared_down != nullptr))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {static_cast<const void*>(x), static_cast<const void*>(w_router),
                        static_cast<const void*>(w_gate_up), static_cast<const void*>(w_down),
                        static_cast<const void*>(w_shared_gate_up), static_cast<const void*>(w_shared_down),
                        static_cast<const void*>(y)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  const LayerLayout L = layer_layout(T, H, I, I_shared, E, k, E_local);
  if (!workspace || !aligned256(workspace) || workspace_bytes < L.total) return MOE_ERR_WORKSPACE;
  char* ws = static_cast<char*>(workspace);
  const int inside = layer_few_shared(T, H, I, k, E_local, I_shared);
  const bool y_f32 = y_type == MOE_TYPE_F32, shared = I_shared > 0 && inside == 0;
  // the share, float32 where the shared expert is added to it
  void* share = shared ? static_cast<void*>(ws + L.share) : y;
  const bool share_f32 = shared || y_f32;
  hipError_t err;
  if (layer_is_few(T, H, I, k, E_local)) {
    const FewScored scored{c, choice_bias, reinterpret_cast<int32_t*>(ws + L.topk_idx),
                           reinterpret_cast<float*>(ws + L.topk_w), inside, I_shared, w_shared_gate_up, w_shared_down};
    err = launch_few(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, share, share_f32,
                     workgroups, polls, ws + L.rest, stream, &scored);
  } else {
    err = share_steps(x, w_router, bias, w_gate_up, w_down, T, H, I, E, k, e0, E_local, renormalize, &c, choice_bias,
                      share, share_f32, ws + L.rest, nullptr, stream);
  }
  if (err == hipSuccess && shared) {
    uint16_t* h = reinterpret_cast<uint16_t*>(ws + L.h);
    float* gemm_part = reinterpret_cast<float*>(ws + L.part);
    err = launch_gemm_bf16({x, w_shared_gate_up, nullptr, nullptr, h, nullptr, T, 1, H, I_shared, MOE_ACT_SWIGLU, 0, 0,
                            gemm_part}, stream);
    if (err == hipSuccess)
      err = launch_gemm_bf16({h, w_shared_down, nullptr, share, y, nullptr, T, 1, I_shared, H, MOE_ACT_NONE, 1, y_f32,
                              gemm_part}, stream);
  }
  return hip_status(err);
}

int moe_layer_forward(const moe_bf16* x, const float* w_router, const float* bias, const float* choice_bias,
                      const moe_bf16* w_gate_up, const moe_bf16* w_down, const moe_bf16* w_shared_gate_up,
                      const moe_bf16* w_shared_down, int T, int H, int I, int I_shared, int E, int k, int e0,
                      int E_local, int score, int n_group, int topk_group, int group_rule, int renormalize,
                      float scale, void* y, int y_type, void* workspace, size_t workspace_bytes, hipStream_t stream) {
  return layer_impl(x, w_router, bias, choice_bias, w_gate_up, w_down, w_shared_gate_up, w_shared_down, T, H, I,
                    I_shared, E, k, e0, E_local, score, n_group, topk_group, group_rule, renormalize, scale, y, y_type,
                    workspace, workspace_bytes, stream);
}

// moe_layer_forward with another number of workgroups and of polls in the kernel of a few
// tokens, as moe_internal_forward_few. Not part of moe.h.
int moe_internal_layer_forward(const moe_bf16* x, const float* w_router, const float* bias, const float* choice_bias,
                               const moe_bf16* w_gate_up, const moe_bf16* w_down, const moe_bf16* w_shared_gate_up,
                               const moe_bf16* w_shared_down, int T, int H, int I, int I_shared, int E, int k, int e0,
                               int E_local, int score, int n_group, int topk_group, int group_rule, int renormalize,
                               float scale, void* y, int y_type, void* workspace, size_t workspace_bytes,
                               int workgroups, int polls, hipStream_t stream) {
  return layer_impl(x, w_router, bias, choice_bias, w_gate_up, w_down, w_shared_gate_up, w_shared_down, T, H, I,
                    I_shared, E, k, e0, E_local, score, n_group, topk_group, group_rule, renormalize, scale, y, y_type,
                    workspace, workspace_bytes, stream, workgroups, polls);
}

}  // extern "C"

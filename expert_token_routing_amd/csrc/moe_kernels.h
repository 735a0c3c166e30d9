// Host-side launchers of the MoE kernels (internal; the public C-ABI is moe.h).
// Every launcher only enqueues on `stream` and returns the launch status.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <algorithm>

namespace moe {

constexpr int kChunk = 64;  // tokens per dispatch chunk (one wave)

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// A segment of `rows` rows in blocks of at most `cap`, a multiple of 16: so many, of such
// a height, a multiple of 16 too (the last is shorter, or empty). No sum passes an int,
// whatever the rows.
__host__ __device__ inline int row_blocks(int rows, int cap) { return rows > 0 ? (rows - 1) / cap + 1 : 0; }
__host__ __device__ inline int block_height(int rows, int blocks) { return ((rows - 1) / blocks + 16) & ~15; }

// How experts are chosen from scores (select.hip); the numbers are MOE_SCORE_*
// and MOE_GROUP_*.
struct Choice {
  int score, n_group, topk_group, group_rule, renormalize;
  float scale;
};

// Router: planes must hold 3*E*H bf16.
// planes: 3 x E x H bf16 scratch; part: T x E float32 scratch (second k half)
// Parts the router's k range is split into (1: no split); the workspace holds
// parts - 1 float32 [T, E] partials besides the logits.
int route_k_parts(int T, int H, int E);

hipError_t launch_route(const uint16_t* x, const float* w_router, const float* bias, int T, int H, int E, int k,
                        int renormalize, float* logits, int32_t* topk_idx, float* topk_w, uint16_t* planes, float* part,
                        hipStream_t stream);

// The router's logits alone: logits [T, E] hold the sums with the bias, or, with
// *split set, the first of route_k_parts(T, H, E) partial sums, the others being
// in part and the bias not added yet.
hipError_t launch_route_logits(const uint16_t* x, const float* w_router, const float* bias, int T, int H, int E,
                               float* logits, uint16_t* planes, float* part, bool* split, hipStream_t stream);

// Dispatch: chunk_table must hold E * ceil(T/64) int32.
hipError_t launch_dispatch(const uint16_t* x, const int32_t* topk_idx, int T, int H, int E, int k, int e0,
                           int E_local, int32_t* counts, int32_t* offsets, int32_t* perm_src, int32_t* inv,
                           uint16_t* x_perm, int32_t* chunk_table, hipStream_t stream);

// Grouped SwiGLU expert MLPs over the segments given by device `offsets`.
hipError_t launch_expert_ffn(const uint16_t* x_perm, const int32_t* offsets, const uint16_t* w_gate_up,
                             const uint16_t* w_down, int H, int I, int E_local, int64_t capacity, uint16_t* h,
                             uint16_t* out, hipStream_t stream);

// The two grouped GEMMs on their own (what launch_expert_ffn runs in order).
// rows_hint: the rows a local expert is expected to hold; few select the
// grouped GEMV (any routing gives correct results either way).
hipError_t launch_expert_gemm1(const uint16_t* x_perm, const int32_t* offsets, const uint16_t* w_gate_up, int H,
                               int I, int E_local, int64_t capacity, uint16_t* h, hipStream_t stream,
                               int64_t rows_hint);
hipError_t launch_expert_gemm2(const uint16_t* h, const int32_t* offsets, const uint16_t* w_down, int H, int I,
                               int E_local, int64_t capacity, uint16_t* out, hipStream_t stream, int64_t rows_hint);

// GEMM1 reading the token vectors of x in place (row n of a segment is token
// perm_src[n] / k) instead of a dispatched copy; usable when
// expert_gemm1_can_gather(T, H).
bool expert_gemm1_can_gather(int T, int H);
hipError_t launch_expert_gemm1_gather(const uint16_t* x, const int32_t* perm_src, int T, int k, const int32_t* offsets,
                                      const uint16_t* w_gate_up, int H, int I, int E_local, int64_t capacity,
                                      uint16_t* h, hipStream_t stream, int64_t rows_hint);

// Down GEMM with the combine of single-selection tokens in its epilogue:
// row_info[n] = {token, bits of its combine weight} when row n's token has
// exactly one local selection, else {-1, 0}; such rows are written to y [T, H]
// as w * out (rounded as the combine rounds a one-term sum), the others to
// out. Usable when expert_gemm2_can_fuse(I).
bool expert_gemm2_can_fuse(int I);
hipError_t launch_expert_gemm2_fused(const uint16_t* h, const int32_t* offsets, const uint16_t* w_down, int H, int I,
                                     int E_local, int64_t capacity, const int2* row_info, uint16_t* out, uint16_t* y,
                                     hipStream_t stream, int64_t rows_hint);

// Grouped GEMV for few rows per expert: each wave streams one weight panel
// of one expert for up to 32 of its rows (an expert with more gets more
// waves). Usable when K (H for the gate/up GEMM, I for the down GEMM) is a
// multiple of 32; chosen when the expected rows per local expert
// (rows_hint) are at most 32 (gate/up GEMM with 512 panels or more: 16).
// N: outputs (I for the gate/up GEMM, H for the down GEMM).
bool grouped_gemv_usable(int64_t rows_hint, int K, int N, int E_local, bool gate_up);
// gate/up + SwiGLU: rows from A [.., H] (row n of a segment is row
// gather_src[n] / gather_k of A when gather_src is given) into h [capacity, I]
hipError_t launch_grouped_gemv1(const uint16_t* A, int lda, const int32_t* gather_src, int gather_k, int gather_rows,
                                const int32_t* offsets, int E_local, int64_t capacity, const uint16_t* w_gate_up,
                                int H, int I, uint16_t* h, hipStream_t stream);
// down: h [capacity, I] into out [capacity, H]; with row_info, rows of
// single-selection tokens go to y as launch_expert_gemm2_fused writes them
hipError_t launch_grouped_gemv2(const uint16_t* h, const int32_t* offsets, int E_local, int64_t capacity,
                                const uint16_t* w_down, int H, int I, const int2* row_info, uint16_t* out,
                                uint16_t* y, hipStream_t stream);

// row_info of launch_expert_gemm2_fused from inv and topk_w (one thread per
// token); rows of tokens with two or more local selections get {-1, 0}.
hipError_t launch_single_rows(const int32_t* inv, const float* topk_w, int T, int k, int2* row_info,
                              hipStream_t stream);

// Bytes of the dispatch tables in the workspace: the per-chunk histogram
// table [E][ceil(T/64)] i32, then the per-chunk lane sets (at most E per
// chunk) u64.
size_t dispatch_table_bytes(int T, int E);

// Dispatch without the row copy (counts, offsets, perm_src, inv only).
hipError_t launch_dispatch_index(const int32_t* topk_idx, int T, int E, int k, int e0, int E_local, int32_t* counts,
                                 int32_t* offsets, int32_t* perm_src, int32_t* inv, int32_t* chunk_table,
                                 hipStream_t stream);

// Weighted top-k sum in token order; y is bf16, or float32 when y_f32. With
// skip_single, tokens with exactly one local selection are left untouched
// (the fused down GEMM wrote them; bf16 y only).
hipError_t launch_combine(const uint16_t* expert_out, const int32_t* inv, const float* topk_w, int T, int H, int k,
                          void* y, bool y_f32, hipStream_t stream, bool skip_single = false);

// Norms around a block (norm.hip). y_type: 0 none (norm of r alone into
// normed), 1 bf16, 2 float32; gate_kind: 0 none, 1 per channel [H], 2 per
// token [T], 3 per value [T, H].
hipError_t launch_block_norm(const void* y, int y_type, const void* r, bool r_f32, const float* w_post,
                             const float* gate, int gate_kind, float scale, const float* w_next, float eps, int T,
                             int H, void* out, uint16_t* normed, hipStream_t stream);

// The whole share for T <= 32 tokens in two kernels (few.hip). workgroups of the
// second (0: two per CU), and polls: how often a waiting one looks before it
// turns to other work. The results depend on neither.
constexpr int kFewPolls = 4096;
bool few_supported(int T, int H, int I, int k, int E_local);
// With `scored`, a kernel between the two chooses by it into topk_idx and topk_w [T, k]
// (the choice's renormalize counts), and the expert that every token shares goes with
// the local ones, as few_shared(..) > 0 more of them (0: none).
struct FewScored {
  Choice choice;
  const float* choice_bias;
  int32_t* topk_idx;
  float* topk_w;
  int shared, I_shared;
  const uint16_t* s_gate_up;
  const uint16_t* s_down;
};
int few_shared(int T, int H, int I, int k, int E_local, int I_shared);
size_t few_workspace_bytes(int T, int H, int I, int E, int k, int E_local, int shared = 0);
hipError_t launch_few(const uint16_t* x, const float* w_router, const float* bias, const uint16_t* w_gate_up,
                      const uint16_t* w_down, int T, int H, int I, int E, int k, int e0, int E_local, int renormalize,
                      void* y, bool y_f32, int workgroups, int polls, char* ws, hipStream_t stream,
                      const FewScored* scored = nullptr);

// 8-bit integer products (gemm_i8.hip). Rows of x quantised with a scale each;
// rows at and past *end (device memory; NULL, for bf16 rows: none) are left alone.
hipError_t launch_quantize_rows(const void* x, bool x_f32, const int32_t* end, int64_t M, int K, int8_t* q,
                                float* scale, hipStream_t stream);
// w [E_local, K, N] bf16 -> q [E_local, N, K] and a scale per channel.
hipError_t launch_quantize_weights(const uint16_t* w, int E_local, int K, int N, int8_t* q, float* scale,
                                   hipStream_t stream);
// C [capacity, N] bf16 over the segments of offsets (NULL: one segment).
// rows_hint: rows a segment is expected to hold; it picks the kernel, any
// segment lengths give the same bits.
hipError_t launch_gemm_i8(const int8_t* A, const float* sa, const int32_t* offsets, int E_local, int64_t capacity,
                          const int8_t* W, const float* sw, int K, int N, uint16_t* C, int64_t rows_hint,
                          hipStream_t stream);
// The tiles that a product takes on a device of `cus` CUs (an i8::Tile); ragged:
// segments by offsets.
int i8_tile(bool swiglu, bool ragged, int E_local, int64_t capacity, int N, int K, int64_t rows_hint, int cus);
// h [capacity, I] float32 = silu(gate) * up, W [E_local, 2 I, H]; row n of a
// segment is row gather_src[n] / gather_k of A when gather_src is given.
hipError_t launch_gate_up_i8(const int8_t* A, const float* sa, const int32_t* gather_src, int gather_k,
                             int gather_rows, const int32_t* offsets, int E_local, int64_t capacity, const int8_t* W,
                             const float* sw, int H, int I, float* h, int64_t rows_hint, hipStream_t stream);

// logits [T, E]; with part, logits hold the first of nparts + 1 partial sums and
// take the whole ones, logit_bias included (which is read only then).
hipError_t launch_select(float* logits, const float* part, int nparts, const float* logit_bias, const float* bias, int T,
                         int E, int k, const Choice& c, int32_t* topk_idx, float* topk_w, hipStream_t stream);

// C = act(A W_e + bias_e) + res over the segments of offsets (NULL: one segment,
// all capacity rows); gemm_bf16.hip. act: MOE_ACT_*.
struct GemmBf16 {
  const uint16_t* A;       // [capacity, K]
  const uint16_t* W;       // [E_local][K, N], or [K, 2 N] for SwiGLU
  const float* bias;       // [E_local][columns of W], or NULL
  const void* res;         // [capacity, N], or NULL
  void* C;                 // [capacity, N]
  const int32_t* offsets;
  int64_t capacity;
  int E_local, K, N, act, res_f32, out_f32;
  float* part;             // gemm_bf16_part_bytes: [k range][capacity, columns of W]
  int ranges = 1, per = 0; // set by the launch: k ranges, and the stages of one
};
// tile, ranges: gemm_bf16_plan's (tile -1: its choice).
hipError_t launch_gemm_bf16(const GemmBf16& p, hipStream_t stream, int tile = -1, int ranges = 1);
size_t gemm_bf16_part_bytes(const GemmBf16& p, int tile = -1, int ranges = 1);
int gemm_bf16_plan(bool swiglu, int E_local, int64_t capacity, int N, int K, int cus, int* ranges);

// Cached device facts of the current device.
int device_cu_count();

}  // namespace moe

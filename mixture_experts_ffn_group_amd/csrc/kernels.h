// Launch entry points of the gfx950 kernels (host side). Shapes and buffers
// are validated by the C-ABI layer before any of these is called; each
// returns the HIP status of its launches.
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

namespace moe {

constexpr int kPermuteBlock = 64;  // tokens per histogram block

// Number of compute units of the current device (cached per device).
int device_cu_count();

hipError_t launch_route(int64_t T, int emb, int E, int k, const uint16_t* x, const float* wr, const float* bias,
                        const float* logits_in, int32_t* topk_idx, float* topk_w, hipStream_t stream);

// masks: [nblk, E] uint64, base: [nblk, E] int32, nblk = ceil(T / 64).
hipError_t launch_permute(int64_t T, int emb, int E, int k, const uint16_t* x, const int32_t* topk_idx,
                          int32_t* group_sizes, int32_t* group_offsets, int32_t* sorted_slot, int32_t* slot_row,
                          uint16_t* xs, uint64_t* masks, int32_t* base, hipStream_t stream);

// The same permute on the library's fixed per-GPU scratch (kPermuteScratchBytes): no workspace argument,
// no allocation. The masks and bases ([nblk, E] uint64, [nblk, E] int32, each rounded up to 256 bytes) must
// fit; concurrent calls on one GPU share the scratch and race.
constexpr size_t kPermuteScratchBytes = size_t(4) << 20;
hipError_t launch_permute_noalloc(int64_t T, int emb, int E, int k, const uint16_t* x, const int32_t* topk_idx,
                                  int32_t* group_sizes, int32_t* group_offsets, int32_t* sorted_slot,
                                  int32_t* slot_row, uint16_t* xs, hipStream_t stream);

// grid: workgroups of the persistent grid (a multiple of 8); 0 = persistent_grid().
// row_slot (nullable): output row r reads A row row_slot[r] / slot_div, row_slot values in [0, n_slots).
// slot_scale (nullable): output row r is scaled by slot_scale[row_slot[r]] (or slot_scale[r]).
hipError_t launch_grouped_gemm(int op, int epi, const uint16_t* A, const uint16_t* B, const float* aux_in,
                               float* aux_out, const int32_t* group_offsets, int E, int64_t M, int K, int N,
                               const int32_t* row_slot, int n_slots, int slot_div, const float* slot_scale,
                               uint16_t* C, hipStream_t stream, int grid = 0);

// GEMM 1 with the SwiGLU epilogue on gathered rows, keeping h as an 8-bit checkpoint.
hipError_t launch_gemm_swiglu_ckpt(const uint16_t* A, const uint16_t* B, const int32_t* group_offsets, int E, int64_t M,
                                   int K, int N, const int32_t* row_slot, int n_slots, int slot_div, uint16_t* C,
                                   int8_t* h_codes, uint8_t* h_scales, hipStream_t stream);

hipError_t launch_wgrad(const uint16_t* A, const uint16_t* D, const int32_t* group_offsets, int E, int64_t M, int P,
                        int Q, uint16_t* C, hipStream_t stream, int grid = 0);

// Workgroups of the persistent GEMM grid: one per compute unit, rounded down to a multiple of 8 (at least 8).
int persistent_grid();

hipError_t launch_combine(int64_t T, int emb, int k, const uint16_t* ys, const int32_t* slot_row, const float* w,
                          uint16_t* y, hipStream_t stream);

hipError_t launch_combine_bwd(int64_t T, int emb, int k, const uint16_t* dy, const uint16_t* ys,
                              const int32_t* slot_row, const float* w, uint16_t* dys, float* dw, hipStream_t stream);

// Router backward, picks held fixed. dl: [T*k] fp32 scratch; wrt: [E, emb] fp32 scratch (used when dx != NULL).
hipError_t launch_mx_quantize_rows(const uint16_t* src, int64_t src_rows, int K, const int32_t* row_index, int row_div,
                                   int64_t M, uint8_t* codes, uint8_t* scales, hipStream_t stream);
hipError_t launch_mx_quantize_weight(const uint16_t* w, int E, int K, int N, uint8_t* codes, uint8_t* scales,
                                     hipStream_t stream);
hipError_t launch_grouped_gemm_mx(int epilogue, const uint8_t* A, const uint8_t* As, int64_t a_rows,
                                  const int32_t* row_slot, int slot_div, const uint8_t* B, const uint8_t* Bs,
                                  const int32_t* group_offsets, int E, int64_t M, int K, int N, uint16_t* C,
                                  uint8_t* Cq, uint8_t* Cqs, hipStream_t stream);
hipError_t launch_route_bwd(int64_t T, int emb, int E, int k, const uint16_t* x, const float* wr,
                            const int32_t* topk_idx, const float* topk_w, const float* dtopk_w,
                            const int32_t* sorted_slot, const int32_t* group_offsets, float* dwr, float* dbias,
                            uint16_t* dx, float* dl, float* dls, int32_t* tok, float* wrt, float* dwrt,
                            hipStream_t stream);

// Routing by scores and its gradient (route_scored.hip); score 0 softmax, 1 sigmoid.
hipError_t launch_route_scored(int64_t T, int E, int k, int score, int n_group, int topk_group, int group_top,
                               int renorm, float scale, const void* logits, bool logits_bf16, const float* bias,
                               int32_t* topk_idx, float* topk_w, hipStream_t stream);
hipError_t launch_route_scored_bwd(int64_t T, int E, int k, int score, int renorm, float scale, const void* logits,
                                   bool logits_bf16, const int32_t* topk_idx, const float* topk_w,
                                   const float* dtopk_w, void* dlogits, hipStream_t stream);

// 8-bit activation checkpoints (ckpt.hip).
hipError_t launch_ckpt_quantize(const void* src, bool src_bf16, int64_t M, int K, int8_t* codes, uint8_t* scales,
                                hipStream_t stream);
hipError_t launch_ckpt_dequantize(const int8_t* codes, const uint8_t* scales, int64_t src_rows, int K,
                                  const int32_t* row_index, int row_div, int64_t M, void* dst, bool dst_bf16,
                                  hipStream_t stream);
hipError_t launch_swiglu_bwd_ckpt(int64_t M, int mlp, const uint16_t* da, const int8_t* h_codes,
                                  const uint8_t* h_scales, const int32_t* row_slot, const float* slot_scale,
                                  uint16_t* dh, uint16_t* a, float* dslot_scale, hipStream_t stream);
size_t wgrad_ckpt_workspace(int E, int64_t M, int P, int Q);
hipError_t launch_wgrad_ckpt(const int8_t* A_codes, const uint8_t* A_scales, int64_t a_rows, const int32_t* row_slot,
                             int slot_div, const uint16_t* D, const int32_t* group_offsets, int E, int64_t M, int P,
                             int Q, uint16_t* C, void* ws, size_t ws_bytes, hipStream_t stream);

// The layer for a few tokens (few.hip). T <= kFewMaxTokens; wr NULL: topk_idx and topk_w are given.
constexpr int kFewMaxTokens = 64;
struct FewWeights {
  const uint16_t *wi, *wo;               // bf16 [E, emb, 2*mlp], [E, mlp, emb], or NULL:
  const uint8_t *wic, *wis, *woc, *wos;  // MXFP8 codes [E, N, K] and scales [E][K/64][N][4]
};
size_t few_workspace(int64_t T, int emb, int mlp, int E, int k);
int64_t few_blocks(int64_t T, int emb, int mlp, int E, int k);  // workgroups (256 lanes) of the experts' kernel
hipError_t launch_few(int64_t T, int emb, int mlp, int E, int k, const uint16_t* x, const float* wr, const float* bias,
                      int32_t* topk_idx, float* topk_w, const FewWeights& wt, uint16_t* y, void* ws,
                      hipStream_t stream);

// The norms around the layer (norm.hip). emb <= kNormMaxEmb, a multiple of 8.
constexpr int kNormMaxEmb = 16384;
enum { kGateNone = 0, kGateChannel = 1, kGateToken = 2, kGateFull = 3 };
struct BlockArgs {
  bool x_f32, w_f32, gate_f32, post;
  int gate_mode;
  float offset, eps, scale, res_scale;
  const void *post_weight, *next_weight, *gate;
};
// y and ys NULL: the norm of res alone, into xn. xn NULL: no next norm.
hipError_t launch_block_out(int64_t T, int emb, const BlockArgs& b, const void* res, const uint16_t* y, int k,
                            const uint16_t* ys, const int32_t* slot_row, const float* topk_w, void* out, uint16_t* xn,
                            uint16_t* y_out, hipStream_t st);
// part NULL: no column sums. `sums`: how many the call can take (next norm, post norm, channel gate). has_y false: the next norm's gradient alone.
size_t block_bwd_workspace(int64_t T, int emb, int sums);
hipError_t launch_block_out_bwd(int64_t T, int emb, const BlockArgs& b, bool has_y, const void* dout, const uint16_t* y,
                                const void* out, const uint16_t* dxn, void* dres, uint16_t* dy, float* dpost,
                                float* dnext, void* dgate, float* part, hipStream_t st);

}  // namespace moe

// launch.h — host-side launch helpers shared by the library's .cu files (internal; not part of
// the C ABI).  Each validates nothing: the extern "C" entry points check their arguments first.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "../../include/nvfp4_moe.h"

namespace nvfp4 {

// Whether any of `rows` rows of `row` bytes, `pitch` bytes apart from `p` on, shares a byte with the `n`
// bytes at `q`.  (What lies between the rows of a strided array is not part of it.)
inline bool rows_overlap(const void* p, int64_t rows, int64_t pitch, int64_t row, const void* q, int64_t n) {
  if (p == nullptr || q == nullptr || rows <= 0 || row <= 0 || n <= 0) return false;
  const int64_t d = static_cast<int64_t>(reinterpret_cast<uintptr_t>(q) - reinterpret_cast<uintptr_t>(p));
  // the first row that ends behind q, and whether it begins before q's end
  const int64_t first = d < row ? 0 : (d - row) / pitch + 1;
  return first < rows && first * pitch < d + n;
}

nvfp4_status_t quantize_launch(const void* x, int64_t rows, int64_t cols, int64_t ld,
                               const int32_t* dst_row, int k, int64_t out_rows, uint8_t* codes,
                               uint8_t* sf, float* gs, int compute_gs, void* ws,
                               int32_t* dev_status, cudaStream_t s);
nvfp4_status_t rmsnorm_quantize_launch(const void* x, int64_t rows, int64_t cols, int64_t ld,
                                       const void* gamma, float eps, const int32_t* dst_row,
                                       int k, int64_t out_rows, uint8_t* codes, uint8_t* sf,
                                       float* gs, int compute_gs, void* ws, int32_t* dev_status,
                                       cudaStream_t s);
nvfp4_status_t permute_launch(const float* logits, int T, int E, int k, int renorm,
                              int32_t* topk_ids, float* topk_w, int32_t* offs, int32_t* dst_row,
                              int32_t* row_slot, float* row_w, int64_t R_max, int32_t* hist_ws,
                              int32_t* dev_status, cudaStream_t s);
size_t permute_workspace_bytes(int T, int E, int k);

nvfp4_status_t gemm_dense(const uint8_t* a, const uint8_t* sfa, const float* gs_a,
                          const uint8_t* b, const uint8_t* sfb, const float* gs_b, int64_t M, int N,
                          int K, void* out_bf16, float* part, int64_t part_floats, int32_t* status,
                          cudaStream_t s);
int dense_k_splits(int64_t M, int N, int K, int sms, int64_t part_floats);
int device_sms();
// 2D byte tensor [rows][row_bytes] in boxes of 128 rows x 128 bytes, 128-byte swizzle.
bool byte_tensor_map(CUtensorMap* m, const void* base, uint64_t row_bytes, uint64_t rows);
nvfp4_status_t gemm_dense_parts(const uint8_t* a, const uint8_t* sfa, const float* gs_a,
                                const uint8_t* b, const uint8_t* sfb, const float* gs_b,
                                int64_t M, int N, int K, int ks, float* part, int32_t* status,
                                cudaStream_t s);

// L1 grouped GEMM + SwiGLU + NVFP4 re-quantization.  h32 (optional): the FP32 h values before
// quantization, [R_max][I].  h_stats (optional, device uint32[3], accumulated): amax bits of |h|
// over real rows (atomicMax), block scales saturated above 448, block scales underflowed to 0.
nvfp4_status_t gemm_l1(const uint8_t* a, const uint8_t* sfa, const float* gs_a, const uint8_t* w1,
                       const uint8_t* sfw1, const float* gs_w1, const int32_t* offs,
                       const int32_t* row_slot, int E, int H, int I, int64_t R_max,
                       const float* gs_h, uint8_t* h, uint8_t* sfh, float* h32,
                       uint32_t* h_stats, int32_t* status, cudaStream_t s);
// L2 grouped GEMM + routing weight + scatter to token order.  atomic = false: each slot's
// weighted row goes to ys [T*k][H] and a combine kernel sums a token's rows in slot order
// (bitwise reproducible).  atomic = true: the rows are added into an FP32 [T][H] accumulator
// (out_f32 if given, else ys) as they are produced, then rounded to bf16; the order of the
// additions, and so the last bits of the sum, may change from run to run.
nvfp4_status_t gemm_l2(const uint8_t* h, const uint8_t* sfh, const float* gs_h, const uint8_t* w2,
                       const uint8_t* sfw2, const float* gs_w2, const int32_t* offs,
                       const int32_t* row_slot, const float* row_w, const int32_t* dst_row, int E,
                       int H, int I, int T, int k, int64_t R_max, float* ys, float* out_f32,
                       void* out_bf16, bool atomic, int32_t* status, cudaStream_t s);
bool l2_use_atomic(int T, int k, int E, bool deterministic);

}  // namespace nvfp4

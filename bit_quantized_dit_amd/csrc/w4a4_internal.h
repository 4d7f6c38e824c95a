// Internal launchers shared between the C-ABI front end and the kernel files.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "../../include/w4a4.h"

namespace w4a4 {

hipError_t launch_column_absmax(const void* X, int x_dtype, int64_t rows, int64_t cols,
                                uint32_t* out_bits, hipStream_t st);

hipError_t launch_pack(const float* W, const w4a4_packed& d, hipStream_t st);

hipError_t launch_actprep(const void* X, int x_dtype, int64_t T, const w4a4_packed& d,
                          uint8_t* Aq, uint8_t* As, uint16_t* XO, hipStream_t st);

// out: fp32 Y [T][d_out], or bf16 H = bf16(gelu_tanh(bf16(Y))) when gelu_bf16
// Destination of the FFN up projection's epilogue that quantizes for the down layer:
// the down layer's A_q / A_s / X_O (workspace order) and RN64(1 / s_j) of its J columns
// in compacted order.
struct QuantDst {
    uint8_t* aq;
    uint8_t* as;
    uint16_t* xo;
    const double* rinv;
    int64_t k_j, k_pad, k_ld;
    int32_t k;
};
// Down-layer preparation that the fused epilogue leaves to a separate pass: rinv from
// the down layer's s and J, zero codes and scales for the 32-blocks past the J columns
// (up to k_pad), zero X_O columns k .. k_ld-1.
hipError_t launch_ffn_prologue(const w4a4_packed& down, int64_t T, const QuantDst& q, hipStream_t st);
// The up projection with GELU and the down layer's activation quantization fused into
// the epilogue: the up layer's output feature f is the down layer's compacted J
// position f for f < k_j and its outlier slot f - k_j above.
hipError_t launch_gemm_quant(const uint8_t* Aq, const uint8_t* As, const uint16_t* XO, int64_t T,
                             const w4a4_packed& up, const QuantDst& q, float* part, hipStream_t st);
hipError_t launch_gemm(const uint8_t* Aq, const uint8_t* As, const uint16_t* XO, int64_t T,
                       const w4a4_packed& d, void* out, bool gelu_bf16, float* part, hipStream_t st);
// Split-K plan of the GEMM for T tokens and N outputs (host logic): tiles [0, full)
// run whole, each later tile as `split` K ranges whose fp32 partial sums take
// part_bytes of workspace (`part`, 256-byte aligned; unused and may be null when
// split == 1), or, with half set, as two 256 x 128 half tiles in a launch of their own.
struct GemmSplit {
    int64_t full;
    int32_t split;
    int32_t half;
    size_t part_bytes;
};
GemmSplit gemm_split_plan(int64_t T, int64_t N, int64_t k_pad, int64_t k_ld);

hipError_t launch_gelu(const float* Y, int64_t n, uint16_t* H, hipStream_t st);

// alpha / k search: the unquantized fp32 product Y = X W^T, and per-block sums of
// (Yq - Yr)^2 and Yr^2 (partials[2b], partials[2b + 1])
hipError_t launch_ref_linear(const void* X, int x_dtype, int64_t T, int64_t d_in, const float* W, int64_t d_out,
                             float* Y, hipStream_t st);
hipError_t launch_sq_err(const float* yq, const float* yr, int64_t n, double* partials, int blocks,
                         hipStream_t st);

// per-call outliers: top-k of the scores into O (ascending) and the column map, and
// the W_O gather from the bf16 copy of W
hipError_t launch_dyn_select(const uint32_t* colmax_bits, const float* s, int64_t d_in, int32_t k, int32_t* O,
                             int32_t* colmap, hipStream_t st);
// W_O[n][i] = W_t[O[i]][n] for i < k, zero for k <= i < k_ld (k_ld a multiple of 32)
hipError_t launch_dyn_gather(const uint16_t* W_t, const int32_t* O, int64_t d_in, int64_t d_out, int32_t k,
                             int64_t k_ld, uint16_t* WO, hipStream_t st);
// W_t[j][n] = bf16_rne(W[n][j]), W fp32 [d_out][d_in]
hipError_t launch_dyn_transpose(const float* W, int64_t d_in, int64_t d_out, uint16_t* W_t, hipStream_t st);

// FP8 block-scaled layer (fp8.hip, fp8gemm.hip): activation codes and scales ([k_pad/128]
// rows of t_ld scales; `count`, where given: counters to clear), weight quantization, the
// reordering of a checkpoint's codes, the product
hipError_t launch_fp8_actquant(const void* X, int x_dtype, int64_t T, int64_t d_in, int kind, uint8_t* aq, float* as,
                               int64_t t_ld, int32_t* count, hipStream_t st);
hipError_t launch_fp8_pack(const void* W, int w_dtype, const w4a4_fp8_packed& d, uint8_t* codes, float* scales,
                           hipStream_t st);
hipError_t launch_fp8_reorder(const uint8_t* src, const void* src_scales, const w4a4_fp8_packed& d, uint8_t* codes,
                              float* scales, hipStream_t st);
// row-major bytes [n_mat][d_out][d_in] into the packed order (any 8-bit codes)
hipError_t launch_reorder_codes(const uint8_t* src, int64_t n_mat, int64_t d_in, int64_t d_out, uint8_t* codes, hipStream_t st);
// Plan of the product (host logic): tiles [0, full) whole, each later one as `split` ranges of the
// inputs, whose fp32 sums take part_bytes of workspace.  `few`: the few-token kernel, which splits all
// its tiles or none and counts the ranges done in FP8_COUNTERS counters.
constexpr int FP8_COUNTERS = 512;
struct Fp8Plan {
    int64_t tiles, full;
    int32_t split, rt;
    bool few, big;
    size_t part_bytes;
};
Fp8Plan fp8_plan(int64_t T, int64_t N, int64_t k_pad);
hipError_t launch_fp8_clear(int32_t* count, hipStream_t st);
// `count` has to be zero where the plan has counters
hipError_t launch_fp8_gemm(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                           int y_dtype, float* part, int32_t* count, hipStream_t st);

// mixture of experts (moe.hip): the arrays of w4a4_moe_ws_layout
struct MoeBuffers {
    float *logits, *p, *part;
    uint16_t *xb, *h;
    int32_t *ids, *place, *count;
};
hipError_t launch_moe(const void* X, int x_dtype, int64_t T, const w4a4_moe& m, const MoeBuffers& b, void* Y, int y_dtype,
                      hipStream_t st);

// INT8 layer (int8.hip, int8gemm.hip): codes and scales of rows (tokens, or weight rows with the
// rows and scales past the last one zeroed up to a multiple of 16), the product
hipError_t launch_int8_quant(const void* X, int x_dtype, int64_t rows, int64_t d_in, bool zero_past, uint8_t* q, float* s,
                             int32_t* count, hipStream_t st);
hipError_t launch_int8_scales(const float* src, int64_t n, int64_t n_pad, float* dst, hipStream_t st);
constexpr int INT8_COUNTERS = 512;
struct Int8Plan {
    int64_t tiles, full;
    int32_t split, rt;
    bool few, big;
    size_t part_bytes;
};
Int8Plan int8_plan(int64_t T, int64_t N, int64_t k_pad);
// What the plans of up to T tokens take at most, so that a workspace for T tokens serves fewer.
struct Int8Room {
    size_t part_bytes;
    bool counters;
};
Int8Room int8_room(int64_t T, int64_t N, int64_t k_pad);
hipError_t launch_int8_clear(int32_t* count, hipStream_t st);
hipError_t launch_int8_gemm(const uint8_t* aq, const float* as, int64_t T, const w4a4_int8_packed& d, void* out, int y_dtype,
                            int32_t* part, int32_t* count, hipStream_t st);

// 4-bit key/value cache (kv.hip, kvattn.hip)
hipError_t launch_kv_append(const w4a4_kv_rows& K, const w4a4_kv_rows& V, int64_t n_rows, const w4a4_kv_batch& b,
                            const w4a4_kv_cache& c, hipStream_t st);
hipError_t launch_kv_read(int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, void* K, void* V, int y_dtype, hipStream_t st);
size_t kv_attention_ws(int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads);
hipError_t launch_kv_attention(const w4a4_kv_rows& Q, int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads,
                               float scale, bool causal, int64_t window, uint16_t* O, void* ws, hipStream_t st);

}  // namespace w4a4

// C-ABI front end of the FP8 block-scaled layer and the mixture-of-experts layer: argument
// validation, size queries, blob and workspace layout, kernel dispatch.  The operations are
// documented in include/w4a4.h.
#include <hip/hip_runtime.h>

#include "capi_util.h"
#include "w4a4_internal.h"

using namespace w4a4;

namespace {

constexpr int64_t kMaxRuns = ((int64_t)1 << 31) - 1;      // runs of 16 rows x 128 inputs: 4 TiB of codes
constexpr int64_t kMaxT = (int64_t)1 << 33;
// 256 x 256 tiles of outputs: a launch counts its work items, 512 a tile, in 32 bits (4096: room for
// the parts of a last round)
constexpr int64_t kMaxTiles = ((int64_t)1 << 23) - 4096;

bool valid_x(int t) { return t == W4A4_X_F32 || t == W4A4_X_BF16; }
bool valid_y(int t) { return t == W4A4_Y_F32 || t == W4A4_Y_BF16; }
bool valid_kind(int k) { return k == W4A4_FP8_SCALE_F32 || k == W4A4_FP8_SCALE_E8M0; }

int check_dims(int64_t n_mat, int64_t d_in, int64_t d_out) {
    if (n_mat <= 0 || d_in <= 0 || d_out <= 0) return W4A4_ERR_INVALID;
    if (d_in > W4A4_FP8_MAX_D || d_out > W4A4_FP8_MAX_D || n_mat > 65535) return W4A4_ERR_SHAPE;
    if (n_mat * (round_up(d_out, 16) / 16) * (round_up(d_in, 128) / 128) > kMaxRuns) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}

size_t codes_bytes(int64_t n_mat, int64_t d_in, int64_t d_out) {
    return (size_t)n_mat * (size_t)round_up(d_out, 16) * (size_t)round_up(d_in, 128);
}
size_t scales_bytes(int64_t n_mat, int64_t d_in, int64_t d_out) {
    return (size_t)n_mat * (size_t)((d_out + 127) / 128) * (size_t)((d_in + 127) / 128) * 4;
}
size_t blob_bytes_of(int64_t n_mat, int64_t d_in, int64_t d_out) {
    return align_up(codes_bytes(n_mat, d_in, d_out)) + align_up(scales_bytes(n_mat, d_in, d_out));
}

int check_packed(const w4a4_fp8_packed* d) {
    if (!d) return W4A4_ERR_INVALID;
    const int st = check_dims(d->n_mat, d->d_in, d->d_out);
    if (st) return st;
    if (!valid_kind(d->scale_kind) || d->k_pad != round_up(d->d_in, 128) || d->n_pad != round_up(d->d_out, 16) || !d->codes ||
        !d->scales)
        return W4A4_ERR_INVALID;
    if (misaligned(d->codes) || misaligned(d->scales)) return W4A4_ERR_ALIGN;
    return W4A4_OK;
}
// a linear layer's descriptor and token count
int check_layer(int64_t T, const w4a4_fp8_packed* d) {
    if (T < 0) return W4A4_ERR_INVALID;
    const int st = check_packed(d);
    if (st) return st;
    if (d->n_mat != 1) return W4A4_ERR_INVALID;
    if (T > kMaxT || (T + 255) / 256 * ((d->d_out + 255) / 256) > kMaxTiles) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}

int64_t t_ld_of(int64_t T) { return round_up(T, 32); }

w4a4_fp8_ws_layout ws_layout(int64_t T, const w4a4_fp8_packed* d) {
    w4a4_fp8_ws_layout w;
    size_t off = 0;
    w.a_q = off;     off = align_up(off + (size_t)(round_up(T, 16) * d->k_pad));
    w.a_s = off;     off = align_up(off + (size_t)(d->k_pad / 128 * t_ld_of(T)) * 4);
    const Fp8Plan plan = fp8_plan(T, d->d_out, d->k_pad);
    w.partial = off; off = align_up(off + plan.part_bytes);
    w.count = off;   off = align_up(off + (plan.few && plan.split > 1 ? FP8_COUNTERS * 4 : 0));
    w.total = off;
    return w;
}

int check_quantize(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* d, const void* ws, size_t ws_bytes,
                   w4a4_fp8_ws_layout* w) {
    const int st = check_layer(T, d);
    if (st) return st;
    if (!X || !ws || !valid_x(x_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(X) || misaligned(ws)) return W4A4_ERR_ALIGN;
    *w = ws_layout(T, d);
    return ws_bytes < w->total ? W4A4_ERR_SHAPE : W4A4_OK;
}

// The product's counters, which have to be zero when it starts; null where its plan has none.
int32_t* counters(const w4a4_fp8_ws_layout& w, void* ws) {
    return w.total > w.count ? (int32_t*)((uint8_t*)ws + w.count) : nullptr;
}
// The codes and scales of checked arguments; clears `count` too.
int quantize(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* d, const w4a4_fp8_ws_layout& w, void* ws, int32_t* count,
             hipStream_t stream) {
    uint8_t* b = (uint8_t*)ws;
    return dev_status(launch_fp8_actquant(X, x_dtype, T, d->d_in, d->scale_kind, b + w.a_q, (float*)(b + w.a_s), t_ld_of(T), count, stream));
}
// The product of checked arguments.
int multiply(const w4a4_fp8_ws_layout& w, void* ws, int64_t T, const w4a4_fp8_packed* d, void* Y, int y_dtype, hipStream_t stream) {
    uint8_t* b = (uint8_t*)ws;
    return dev_status(launch_fp8_gemm(b + w.a_q, (const float*)(b + w.a_s), T, t_ld_of(T), *d, Y, y_dtype, (float*)(b + w.partial),
                                      counters(w, ws), stream));
}

int describe(int64_t n_mat, int64_t d_in, int64_t d_out, int kind, void* blob, size_t blob_bytes, w4a4_fp8_packed* out) {
    const int st = check_dims(n_mat, d_in, d_out);
    if (st) return st;
    if (!valid_kind(kind)) return W4A4_ERR_INVALID;
    if (misaligned(blob)) return W4A4_ERR_ALIGN;
    if (blob_bytes < blob_bytes_of(n_mat, d_in, d_out)) return W4A4_ERR_SHAPE;
    out->n_mat = n_mat;
    out->d_in = d_in;
    out->d_out = d_out;
    out->k_pad = round_up(d_in, 128);
    out->n_pad = round_up(d_out, 16);
    out->scale_kind = kind;
    out->reserved = 0;
    out->codes = (const uint8_t*)blob;
    out->scales = (const float*)((uint8_t*)blob + align_up(codes_bytes(n_mat, d_in, d_out)));
    return W4A4_OK;
}

int check_moe(int64_t T, const w4a4_moe* m) {
    if (T < 0 || !m || !m->router) return W4A4_ERR_INVALID;
    if (!valid_x(m->router_dtype)) return W4A4_ERR_INVALID;
    if (m->activation != W4A4_MOE_SILU_GATED && m->activation != W4A4_MOE_GELU_TANH) return W4A4_ERR_INVALID;
    int st = check_packed(&m->up);
    if (!st) st = check_packed(&m->down);
    if (!st && m->activation == W4A4_MOE_SILU_GATED) st = check_packed(&m->gate);
    if (st) return st;
    const w4a4_fp8_packed &u = m->up, &d = m->down, &g = m->gate;
    if (u.n_mat > W4A4_MOE_MAX_E || u.d_in > W4A4_MOE_MAX_D || u.d_out > W4A4_MOE_MAX_D) return W4A4_ERR_SHAPE;
    if (d.n_mat != u.n_mat || d.d_in != u.d_out || d.d_out != u.d_in) return W4A4_ERR_SHAPE;
    if (m->activation == W4A4_MOE_SILU_GATED && (g.n_mat != u.n_mat || g.d_in != u.d_in || g.d_out != u.d_out))
        return W4A4_ERR_SHAPE;
    if (m->top_k <= 0 || m->top_k > u.n_mat) return W4A4_ERR_INVALID;
    if (m->top_k > W4A4_MOE_MAX_K || T > W4A4_MOE_MAX_T) return W4A4_ERR_SHAPE;
    if (misaligned(m->router)) return W4A4_ERR_ALIGN;
    return W4A4_OK;
}

w4a4_moe_ws_layout moe_layout(int64_t T, const w4a4_moe* m) {
    w4a4_moe_ws_layout w;
    const int64_t E = m->up.n_mat, pairs = T * m->top_k;
    size_t off = 0;
    w.logits = off; off = align_up(off + (size_t)(T * round_up(E, 4)) * 4);
    w.xb = off;     off = align_up(off + (size_t)(T * m->up.k_pad) * 2);
    w.ids = off;    off = align_up(off + (size_t)pairs * 4);
    w.p = off;      off = align_up(off + (size_t)pairs * 4);
    w.h = off;      off = align_up(off + (size_t)(pairs * m->down.k_pad) * 2);
    w.place = off;  off = align_up(off + (size_t)pairs * 4);
    w.count = off;  off = align_up(off + (size_t)((m->down.d_out + 15) / 16) * 4);
    w.part = off;   off = align_up(off + (size_t)T * (2 * 512 * 16 * 4));   // two of 16 outputs for each of 512 workgroups
    w.total = off;
    return w;
}

}  // namespace

extern "C" {

int w4a4_fp8_packed_size(int64_t n_mat, int64_t d_in, int64_t d_out, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    const int st = check_dims(n_mat, d_in, d_out);
    if (st) return st;
    *bytes = blob_bytes_of(n_mat, d_in, d_out);
    return W4A4_OK;
}

int w4a4_fp8_pack_weights(const void* W, int w_dtype, int64_t n_mat, int64_t d_in, int64_t d_out, int scale_kind, void* blob,
                          size_t blob_bytes, w4a4_fp8_packed* desc, void* stream) {
    if (!W || !blob || !desc || !valid_x(w_dtype)) return W4A4_ERR_INVALID;
    w4a4_fp8_packed d;
    const int st = describe(n_mat, d_in, d_out, scale_kind, blob, blob_bytes, &d);
    if (st) return st;
    if (misaligned(W)) return W4A4_ERR_ALIGN;
    const hipError_t e = launch_fp8_pack(W, w_dtype, d, (uint8_t*)d.codes, (float*)d.scales, (hipStream_t)stream);
    if (e == hipSuccess) *desc = d;
    return dev_status(e);
}

int w4a4_fp8_pack_codes(const uint8_t* codes, const void* scales, int64_t n_mat, int64_t d_in, int64_t d_out, int scale_kind,
                        void* blob, size_t blob_bytes, w4a4_fp8_packed* desc, void* stream) {
    if (!codes || !scales || !blob || !desc) return W4A4_ERR_INVALID;
    w4a4_fp8_packed d;
    const int st = describe(n_mat, d_in, d_out, scale_kind, blob, blob_bytes, &d);
    if (st) return st;
    if (misaligned(codes) || misaligned(scales)) return W4A4_ERR_ALIGN;
    const hipError_t e = launch_fp8_reorder(codes, scales, d, (uint8_t*)d.codes, (float*)d.scales, (hipStream_t)stream);
    if (e == hipSuccess) *desc = d;
    return dev_status(e);
}

int w4a4_fp8_workspace_layout(int64_t T, const w4a4_fp8_packed* desc, w4a4_fp8_ws_layout* out) {
    if (!out) return W4A4_ERR_INVALID;
    const int st = check_layer(T, desc);
    if (st) return st;
    *out = ws_layout(T, desc);
    return W4A4_OK;
}

int w4a4_fp8_workspace_size(int64_t T, const w4a4_fp8_packed* desc, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    w4a4_fp8_ws_layout w;
    const int st = w4a4_fp8_workspace_layout(T, desc, &w);
    if (st) return st;
    *bytes = w.total;
    return W4A4_OK;
}

int w4a4_fp8_quantize_activations(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* desc, void* ws, size_t ws_bytes,
                                  void* stream) {
    w4a4_fp8_ws_layout w;
    const int st = check_quantize(X, x_dtype, T, desc, ws, ws_bytes, &w);
    if (st || T == 0) return st;
    return quantize(X, x_dtype, T, desc, w, ws, nullptr, (hipStream_t)stream);
}

int w4a4_fp8_gemm_prequantized(void* ws, size_t ws_bytes, int64_t T, const w4a4_fp8_packed* desc, void* Y, int y_dtype,
                               void* stream) {
    const int st = check_layer(T, desc);
    if (st) return st;
    if (!Y || !ws || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(Y) || misaligned(ws)) return W4A4_ERR_ALIGN;
    const w4a4_fp8_ws_layout w = ws_layout(T, desc);
    if (ws_bytes < w.total) return W4A4_ERR_SHAPE;
    if (T == 0) return W4A4_OK;
    // the codes may come from a call for another layer, whose workspace has its counters elsewhere or none
    if (int32_t* const count = counters(w, ws)) {
        const hipError_t e = launch_fp8_clear(count, (hipStream_t)stream);
        if (e != hipSuccess) return dev_status(e);
    }
    return multiply(w, ws, T, desc, Y, y_dtype, (hipStream_t)stream);
}

int w4a4_fp8_linear(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* desc, void* Y, int y_dtype, void* ws,
                    size_t ws_bytes, void* stream) {
    if (!Y || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(Y)) return W4A4_ERR_ALIGN;
    w4a4_fp8_ws_layout w;
    const int st = check_quantize(X, x_dtype, T, desc, ws, ws_bytes, &w);
    if (st || T == 0) return st;
    const int q = quantize(X, x_dtype, T, desc, w, ws, counters(w, ws), (hipStream_t)stream);
    return q ? q : multiply(w, ws, T, desc, Y, y_dtype, (hipStream_t)stream);
}

int w4a4_moe_workspace_layout(int64_t T, const w4a4_moe* moe, w4a4_moe_ws_layout* out) {
    if (!out) return W4A4_ERR_INVALID;
    const int st = check_moe(T, moe);
    if (st) return st;
    *out = moe_layout(T, moe);
    return W4A4_OK;
}

int w4a4_moe_workspace_size(int64_t T, const w4a4_moe* moe, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    w4a4_moe_ws_layout w;
    const int st = w4a4_moe_workspace_layout(T, moe, &w);
    if (st) return st;
    *bytes = w.total;
    return W4A4_OK;
}

int w4a4_moe_forward(const void* X, int x_dtype, int64_t T, const w4a4_moe* moe, void* Y, int y_dtype, void* ws,
                     size_t ws_bytes, void* stream) {
    const int st = check_moe(T, moe);
    if (st) return st;
    if (!X || !Y || !ws || !valid_x(x_dtype) || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(X) || misaligned(Y) || misaligned(ws)) return W4A4_ERR_ALIGN;
    const w4a4_moe_ws_layout w = moe_layout(T, moe);
    if (ws_bytes < w.total) return W4A4_ERR_SHAPE;
    if (T == 0) return W4A4_OK;
    uint8_t* b = (uint8_t*)ws;
    MoeBuffers m;
    m.logits = (float*)(b + w.logits);
    m.p = (float*)(b + w.p);
    m.xb = (uint16_t*)(b + w.xb);
    m.h = (uint16_t*)(b + w.h);
    m.part = (float*)(b + w.part);
    m.place = (int32_t*)(b + w.place);
    m.count = (int32_t*)(b + w.count);
    m.ids = (int32_t*)(b + w.ids);
    return dev_status(launch_moe(X, x_dtype, T, *moe, m, Y, y_dtype, (hipStream_t)stream));
}

}  // extern "C"

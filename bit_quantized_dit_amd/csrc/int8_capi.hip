// C-ABI front end of the INT8 layer: argument validation, size queries, blob and workspace layout,
// kernel dispatch.  The operations are documented in include/w4a4.h.
#include <hip/hip_runtime.h>

#include "capi_util.h"
#include "w4a4_internal.h"

using namespace w4a4;

namespace {

// 16 tokens a workgroup of up to 1024 work items, which a launch counts in 32 bits
constexpr int64_t kMaxT = ((int64_t)1 << 26) - 16;
// 256 x 256 tiles of outputs: a launch counts its work items, 512 a tile (and up to 512 ranges' besides), in 32 bits
constexpr int64_t kMaxTiles = W4A4_INT8_MAX_TILES;
static_assert((kMaxTiles + 512) * 512 < (int64_t)1 << 32, "work items of a launch");

bool valid_x(int t) { return t == W4A4_X_F32 || t == W4A4_X_BF16; }
bool valid_y(int t) { return t == W4A4_Y_F32 || t == W4A4_Y_BF16; }

int check_dims(int64_t d_in, int64_t d_out) {
    if (d_in <= 0 || d_out <= 0) return W4A4_ERR_INVALID;
    return d_in > W4A4_INT8_MAX_D_IN || d_out > W4A4_INT8_MAX_D_OUT ? W4A4_ERR_SHAPE : W4A4_OK;
}
size_t codes_bytes(int64_t d_in, int64_t d_out) { return (size_t)round_up(d_out, 16) * (size_t)round_up(d_in, 128); }
size_t blob_bytes_of(int64_t d_in, int64_t d_out) {
    return align_up(codes_bytes(d_in, d_out)) + align_up((size_t)round_up(d_out, 16) * 4);
}

int check_layer(int64_t T, const w4a4_int8_packed* d) {
    if (T < 0 || !d) return W4A4_ERR_INVALID;
    const int st = check_dims(d->d_in, d->d_out);
    if (st) return st;
    if (d->k_pad != round_up(d->d_in, 128) || d->n_pad != round_up(d->d_out, 16) || !d->codes || !d->scales) return W4A4_ERR_INVALID;
    if (misaligned(d->codes) || misaligned(d->scales)) return W4A4_ERR_ALIGN;
    if (T > kMaxT || (T + 255) / 256 * ((d->d_out + 255) / 256) > kMaxTiles) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}

w4a4_int8_ws_layout ws_layout(int64_t T, const w4a4_int8_packed* d) {
    w4a4_int8_ws_layout w;
    size_t off = 0;
    w.a_q = off;     off = align_up(off + (size_t)(round_up(T, 16) * d->k_pad));
    w.a_s = off;     off = align_up(off + (size_t)T * 4);
    const Int8Room room = int8_room(T, d->d_out, d->k_pad);
    w.partial = off; off = align_up(off + room.part_bytes);
    w.count = off;   off = align_up(off + (room.counters ? INT8_COUNTERS * 4 : 0));
    w.total = off;
    return w;
}

int check_quantize(const void* X, int x_dtype, int64_t T, const w4a4_int8_packed* d, const void* ws, size_t ws_bytes,
                   w4a4_int8_ws_layout* w) {
    const int st = check_layer(T, d);
    if (st) return st;
    if (!X || !ws || !valid_x(x_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(X) || misaligned(ws)) return W4A4_ERR_ALIGN;
    *w = ws_layout(T, d);
    return ws_bytes < w->total ? W4A4_ERR_SHAPE : W4A4_OK;
}

// The product's counters, which have to be zero when it starts; null where its plan has none.
int32_t* counters(const w4a4_int8_ws_layout& w, void* ws, int64_t T, const w4a4_int8_packed* d) {
    const Int8Plan plan = int8_plan(T, d->d_out, d->k_pad);
    return plan.few && plan.split > 1 ? (int32_t*)((uint8_t*)ws + w.count) : nullptr;
}
int quantize(const void* X, int x_dtype, int64_t T, const w4a4_int8_packed* d, const w4a4_int8_ws_layout& w, void* ws, int32_t* count,
             hipStream_t stream) {
    uint8_t* b = (uint8_t*)ws;
    return dev_status(launch_int8_quant(X, x_dtype, T, d->d_in, false, b + w.a_q, (float*)(b + w.a_s), count, stream));
}
int multiply(const w4a4_int8_ws_layout& w, void* ws, int64_t T, const w4a4_int8_packed* d, void* Y, int y_dtype, hipStream_t stream) {
    uint8_t* b = (uint8_t*)ws;
    return dev_status(launch_int8_gemm(b + w.a_q, (const float*)(b + w.a_s), T, *d, Y, y_dtype, (int32_t*)(b + w.partial),
                                       counters(w, ws, T, d), stream));
}

int describe(int64_t d_in, int64_t d_out, void* blob, size_t blob_bytes, w4a4_int8_packed* out) {
    const int st = check_dims(d_in, d_out);
    if (st) return st;
    if (misaligned(blob)) return W4A4_ERR_ALIGN;
    if (blob_bytes < blob_bytes_of(d_in, d_out)) return W4A4_ERR_SHAPE;
    out->d_in = d_in;
    out->d_out = d_out;
    out->k_pad = round_up(d_in, 128);
    out->n_pad = round_up(d_out, 16);
    out->codes = (const uint8_t*)blob;
    out->scales = (const float*)((uint8_t*)blob + align_up(codes_bytes(d_in, d_out)));
    return W4A4_OK;
}

}  // namespace

extern "C" {

int w4a4_int8_packed_size(int64_t d_in, int64_t d_out, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    const int st = check_dims(d_in, d_out);
    if (st) return st;
    *bytes = blob_bytes_of(d_in, d_out);
    return W4A4_OK;
}

int w4a4_int8_pack_weights(const void* W, int w_dtype, int64_t d_in, int64_t d_out, void* blob, size_t blob_bytes,
                           w4a4_int8_packed* desc, void* stream) {
    if (!W || !blob || !desc || !valid_x(w_dtype)) return W4A4_ERR_INVALID;
    w4a4_int8_packed d;
    const int st = describe(d_in, d_out, blob, blob_bytes, &d);
    if (st) return st;
    if (misaligned(W)) return W4A4_ERR_ALIGN;
    const hipError_t e = launch_int8_quant(W, w_dtype, d_out, d_in, true, (uint8_t*)d.codes, (float*)d.scales, nullptr, (hipStream_t)stream);
    if (e == hipSuccess) *desc = d;
    return dev_status(e);
}

int w4a4_int8_pack_codes(const int8_t* codes, const float* scales, int64_t d_in, int64_t d_out, void* blob, size_t blob_bytes,
                         w4a4_int8_packed* desc, void* stream) {
    if (!codes || !scales || !blob || !desc) return W4A4_ERR_INVALID;
    w4a4_int8_packed d;
    const int st = describe(d_in, d_out, blob, blob_bytes, &d);
    if (st) return st;
    if (misaligned(codes) || misaligned(scales)) return W4A4_ERR_ALIGN;
    hipError_t e = launch_reorder_codes((const uint8_t*)codes, 1, d_in, d_out, (uint8_t*)d.codes, (hipStream_t)stream);
    if (e == hipSuccess) e = launch_int8_scales(scales, d_out, d.n_pad, (float*)d.scales, (hipStream_t)stream);
    if (e == hipSuccess) *desc = d;
    return dev_status(e);
}

int w4a4_int8_workspace_layout(int64_t T, const w4a4_int8_packed* desc, w4a4_int8_ws_layout* out) {
    if (!out) return W4A4_ERR_INVALID;
    const int st = check_layer(T, desc);
    if (st) return st;
    *out = ws_layout(T, desc);
    return W4A4_OK;
}

int w4a4_int8_workspace_size(int64_t T, const w4a4_int8_packed* desc, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    w4a4_int8_ws_layout w;
    const int st = w4a4_int8_workspace_layout(T, desc, &w);
    if (st) return st;
    *bytes = w.total;
    return W4A4_OK;
}

int w4a4_int8_quantize_activations(const void* X, int x_dtype, int64_t T, const w4a4_int8_packed* desc, void* ws, size_t ws_bytes,
                                   void* stream) {
    w4a4_int8_ws_layout w;
    const int st = check_quantize(X, x_dtype, T, desc, ws, ws_bytes, &w);
    if (st || T == 0) return st;
    return quantize(X, x_dtype, T, desc, w, ws, nullptr, (hipStream_t)stream);
}

int w4a4_int8_gemm_prequantized(void* ws, size_t ws_bytes, int64_t T, const w4a4_int8_packed* desc, void* Y, int y_dtype, void* stream) {
    const int st = check_layer(T, desc);
    if (st) return st;
    if (!Y || !ws || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(Y) || misaligned(ws)) return W4A4_ERR_ALIGN;
    const w4a4_int8_ws_layout w = ws_layout(T, desc);
    if (ws_bytes < w.total) return W4A4_ERR_SHAPE;
    if (T == 0) return W4A4_OK;
    // the codes may come from a call for another layer, whose workspace has its counters elsewhere or none
    if (int32_t* const count = counters(w, ws, T, desc)) {
        const hipError_t e = launch_int8_clear(count, (hipStream_t)stream);
        if (e != hipSuccess) return dev_status(e);
    }
    return multiply(w, ws, T, desc, Y, y_dtype, (hipStream_t)stream);
}

int w4a4_int8_linear(const void* X, int x_dtype, int64_t T, const w4a4_int8_packed* desc, void* Y, int y_dtype, void* ws, size_t ws_bytes,
                     void* stream) {
    if (!Y || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(Y)) return W4A4_ERR_ALIGN;
    w4a4_int8_ws_layout w;
    const int st = check_quantize(X, x_dtype, T, desc, ws, ws_bytes, &w);
    if (st || T == 0) return st;
    const int q = quantize(X, x_dtype, T, desc, w, ws, counters(w, ws, T, desc), (hipStream_t)stream);
    return q ? q : multiply(w, ws, T, desc, Y, y_dtype, (hipStream_t)stream);
}

}  // extern "C"

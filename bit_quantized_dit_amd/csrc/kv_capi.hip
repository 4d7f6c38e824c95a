// C-ABI front end of the 4-bit key/value cache and of attention over it: argument validation, size
// queries, kernel dispatch.  The operations are documented in include/w4a4.h.
#include <hip/hip_runtime.h>

#include <cmath>

#include "capi_util.h"
#include "w4a4_internal.h"

using namespace w4a4;

namespace {

constexpr int64_t kMaxRows = (int64_t)1 << 26, kMaxSeqs = 65535, kMaxHeads = 4096, kMaxPageTokens = (int64_t)1 << 20;
constexpr int64_t kMaxTokens = 0x7FFFFF00;                  // of a sequence
constexpr int64_t kMaxGroups = ((int64_t)1 << 23) - 1;      // workgroups of a launch, up to 512 work items each

bool valid_x(int t) { return t == W4A4_X_F32 || t == W4A4_X_BF16; }
bool valid_y(int t) { return t == W4A4_Y_F32 || t == W4A4_Y_BF16; }

int64_t pad_of(int64_t d) { return d <= 128 ? round_up(d, 32) : round_up(d, 64); }
int64_t block_bytes_of(int64_t d) {
    const int64_t g = pad_of(d) / 32, sg = g <= 2 ? g : round_up(g, 4);
    return 512 * g + 32 * sg;
}

int check_dims(int64_t n_pages, int64_t page_tokens, int64_t n_heads, int64_t head_dim) {
    if (n_pages <= 0 || page_tokens <= 0 || n_heads <= 0 || head_dim <= 0 || page_tokens % 16) return W4A4_ERR_INVALID;
    if (n_pages > 0x7FFFFFFF || page_tokens > kMaxPageTokens || n_heads > kMaxHeads || head_dim > 256) return W4A4_ERR_SHAPE;
    // (2^31 pages of 2^20 tokens, 4096 heads and 4352 bytes a block of 16 stay below 2^72, not 2^63)
    if ((__int128)n_pages * n_heads * (page_tokens / 16) * block_bytes_of(head_dim) > ((__int128)1 << 62)) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}
size_t cache_bytes(int64_t n_pages, int64_t page_tokens, int64_t n_heads, int64_t head_dim) {
    return (size_t)(n_pages * n_heads * (page_tokens / 16) * block_bytes_of(head_dim));
}

int check_cache(const w4a4_kv_cache* c) {
    if (!c || !c->data) return W4A4_ERR_INVALID;
    const int st = check_dims(c->n_pages, c->page_tokens, c->n_heads, c->head_dim);
    if (st) return st;
    if (c->d_pad != pad_of(c->head_dim) || c->block_bytes != block_bytes_of(c->head_dim)) return W4A4_ERR_INVALID;
    return misaligned(c->data) ? W4A4_ERR_ALIGN : W4A4_OK;
}

int check_batch(int64_t n_rows, const w4a4_kv_batch* b, const w4a4_kv_cache* c) {
    if (n_rows < 0 || !b || b->n_seqs < 0 || b->max_rows < 0 || b->max_pages <= 0) return W4A4_ERR_INVALID;
    const int st = check_cache(c);
    if (st) return st;
    if (b->n_seqs && (!b->q_start || !b->lens || !b->pages)) return W4A4_ERR_INVALID;      // (empty arrays may have no address)
    if (((uintptr_t)b->q_start | (uintptr_t)b->lens | (uintptr_t)b->pages) & 3u) return W4A4_ERR_ALIGN;
    if (n_rows > kMaxRows || b->max_rows > kMaxRows || b->n_seqs > kMaxSeqs || b->max_pages > kMaxTokens / c->page_tokens)
        return W4A4_ERR_SHAPE;
    // a launch counts its workgroups: blocks of 16 rows x 4 heads
    if (b->n_seqs * ((b->max_rows + 14) / 16 + 1) * ((c->n_heads + 3) / 4) > kMaxGroups) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}

int check_rows(const w4a4_kv_rows* x) {
    if (!x || !x->data || !valid_x(x->dtype)) return W4A4_ERR_INVALID;
    return (uintptr_t)x->data & (x->dtype == W4A4_X_F32 ? 3u : 1u) ? W4A4_ERR_ALIGN : W4A4_OK;
}

bool nothing(int64_t n_rows, const w4a4_kv_batch* b) { return n_rows == 0 || b->n_seqs == 0 || b->max_rows == 0; }

int check_heads(const w4a4_kv_batch* b, const w4a4_kv_cache* c, int32_t n_q_heads) {
    if (n_q_heads <= 0 || n_q_heads % c->n_heads) return W4A4_ERR_INVALID;
    if (n_q_heads > kMaxHeads) return W4A4_ERR_SHAPE;
    const int64_t rows = b->max_rows * (n_q_heads / c->n_heads);
    if (rows > 0x7FFFFFFF - 256 || b->n_seqs * c->n_heads * ((rows + 127) / 128 + 1) > kMaxGroups) return W4A4_ERR_SHAPE;
    return W4A4_OK;
}

}  // namespace

extern "C" {

int w4a4_kv_cache_size(int64_t n_pages, int32_t page_tokens, int32_t n_heads, int32_t head_dim, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    const int st = check_dims(n_pages, page_tokens, n_heads, head_dim);
    if (st) return st;
    *bytes = cache_bytes(n_pages, page_tokens, n_heads, head_dim);
    return W4A4_OK;
}

int w4a4_kv_cache_describe(int64_t n_pages, int32_t page_tokens, int32_t n_heads, int32_t head_dim, void* data, size_t data_bytes,
                           w4a4_kv_cache* out) {
    if (!data || !out) return W4A4_ERR_INVALID;
    const int st = check_dims(n_pages, page_tokens, n_heads, head_dim);
    if (st) return st;
    if (misaligned(data)) return W4A4_ERR_ALIGN;
    if (data_bytes < cache_bytes(n_pages, page_tokens, n_heads, head_dim)) return W4A4_ERR_SHAPE;
    out->n_pages = n_pages;
    out->page_tokens = page_tokens;
    out->n_heads = n_heads;
    out->head_dim = head_dim;
    out->d_pad = (int32_t)pad_of(head_dim);
    out->block_bytes = block_bytes_of(head_dim);
    out->data = (uint8_t*)data;
    return W4A4_OK;
}

int w4a4_kv_append(const w4a4_kv_rows* K, const w4a4_kv_rows* V, int64_t n_rows, const w4a4_kv_batch* batch, const w4a4_kv_cache* cache,
                   void* stream) {
    int st = check_batch(n_rows, batch, cache);
    if (!st) st = check_rows(K);
    if (!st) st = check_rows(V);
    if (st) return st;
    if (K->dtype != V->dtype) return W4A4_ERR_INVALID;
    if (nothing(n_rows, batch)) return W4A4_OK;
    return dev_status(launch_kv_append(*K, *V, n_rows, *batch, *cache, (hipStream_t)stream));
}

int w4a4_kv_read(int64_t n_rows, const w4a4_kv_batch* batch, const w4a4_kv_cache* cache, void* K, void* V, int y_dtype, void* stream) {
    const int st = check_batch(n_rows, batch, cache);
    if (st) return st;
    if (!K || !V || !valid_y(y_dtype)) return W4A4_ERR_INVALID;
    if (misaligned(K) || misaligned(V)) return W4A4_ERR_ALIGN;
    if (nothing(n_rows, batch)) return W4A4_OK;
    return dev_status(launch_kv_read(n_rows, *batch, *cache, K, V, y_dtype, (hipStream_t)stream));
}

int w4a4_kv_attention_workspace_size(int64_t n_rows, const w4a4_kv_batch* batch, const w4a4_kv_cache* cache, int32_t n_q_heads, size_t* bytes) {
    if (!bytes) return W4A4_ERR_INVALID;
    int st = check_batch(n_rows, batch, cache);
    if (!st) st = check_heads(batch, cache, n_q_heads);
    if (st) return st;
    *bytes = kv_attention_ws(n_rows, *batch, *cache, n_q_heads);
    return W4A4_OK;
}

int w4a4_kv_attention(const w4a4_kv_rows* Q, int64_t n_rows, const w4a4_kv_batch* batch, const w4a4_kv_cache* cache, int32_t n_q_heads,
                      float scale, int causal, int64_t window, uint16_t* O, void* ws, size_t ws_bytes, void* stream) {
    int st = check_batch(n_rows, batch, cache);
    if (!st) st = check_heads(batch, cache, n_q_heads);
    if (!st) st = check_rows(Q);
    if (st) return st;
    if (!O || !ws || !(scale > 0.0f) || !std::isfinite(scale * 1.44269504088896340736f) || (causal != 0 && causal != 1) || window < 0 || (window && !causal))
        return W4A4_ERR_INVALID;
    if (misaligned(O) || misaligned(ws)) return W4A4_ERR_ALIGN;
    if (ws_bytes < kv_attention_ws(n_rows, *batch, *cache, n_q_heads)) return W4A4_ERR_SHAPE;
    if (nothing(n_rows, batch)) return W4A4_OK;
    if (window > kMaxTokens) window = 0;      // no sequence is longer
    return dev_status(launch_kv_attention(*Q, n_rows, *batch, *cache, n_q_heads, scale, causal != 0, window, O, ws, (hipStream_t)stream));
}

}  // extern "C"

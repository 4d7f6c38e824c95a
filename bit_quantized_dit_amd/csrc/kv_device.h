// Device helpers of the 4-bit key/value cache: where a token stands, block layout, E2M1 codes.
#pragma once

#include <type_traits>

#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

// A call's batch and cache as the kernels take them.
struct KvArgs {
    const int32_t *q_start, *lens, *pages;
    int64_t n_seqs, max_rows, max_pages, n_rows;
    uint8_t* data;
    int64_t n_pages, block_bytes;
    int32_t page_blocks, n_heads, head_dim;      // page_blocks: blocks of 16 tokens in a page
};
inline KvArgs kv_args(int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c) {
    return KvArgs{b.q_start, b.lens, b.pages, b.n_seqs, b.max_rows, b.max_pages, n_rows, c.data, c.n_pages, c.block_bytes,
                  c.page_tokens / 16, c.n_heads, c.head_dim};
}

// Block layout for G groups of 32 channels (d_pad = 32 G).
template <int G> struct KvBlock {
    static constexpr int SG = G <= 2 ? G : (G + 3) / 4 * 4;      // bytes of a token's scales
    static constexpr int V = 256 * G, KS = 512 * G, VS = KS + 16 * SG, BYTES = VS + 16 * SG;
};

// f with the number of groups as a constant: d_pad is 32, 64, 96, 128, 192 or 256.
template <typename F>
hipError_t kv_groups(int d_pad, const F& f) {
    switch (d_pad) {
        case 32: return f(std::integral_constant<int, 1>());
        case 64: return f(std::integral_constant<int, 2>());
        case 96: return f(std::integral_constant<int, 3>());
        case 128: return f(std::integral_constant<int, 4>());
        case 192: return f(std::integral_constant<int, 6>());
        case 256: return f(std::integral_constant<int, 8>());
    }
    return hipErrorInvalidValue;
}

// A sequence: its first row, rows (as given, and as many as are computed), cached tokens, the
// position of its first row.
struct KvSeq {
    int64_t row0;
    int32_t rows, done, len, first;
};
__device__ __forceinline__ KvSeq kv_seq(const KvArgs& a, int64_t b) {
    const int64_t lo = a.q_start[b], hi = a.q_start[b + 1], cap = a.max_pages * a.page_blocks * 16, len = a.lens[b];
    KvSeq s;
    s.row0 = lo < 0 ? 0 : lo > a.n_rows ? a.n_rows : lo;
    const int64_t end = hi > a.n_rows ? a.n_rows : hi;
    s.rows = (int32_t)(end > s.row0 ? end - s.row0 : 0);
    s.done = (int32_t)(s.rows < a.max_rows ? s.rows : a.max_rows);
    s.len = (int32_t)(len < 0 ? 0 : len > cap ? cap : len);
    s.first = s.len - s.rows;
    return s;
}

// The block of head h that holds tokens 16 q .. of sequence b; null where its page is not there.
__device__ __forceinline__ uint8_t* kv_block(const KvArgs& a, int64_t b, uint32_t q, int h) {
    const uint32_t pi = q / (uint32_t)a.page_blocks, r = q - pi * (uint32_t)a.page_blocks;
    if ((int64_t)pi >= a.max_pages) return nullptr;
    const int32_t page = a.pages[b * a.max_pages + pi];
    if (page < 0 || page >= a.n_pages) return nullptr;
    return a.data + (((int64_t)page * a.n_heads + h) * a.page_blocks + r) * a.block_bytes;
}

}  // namespace w4a4

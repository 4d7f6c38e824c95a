// 4-bit key/value cache on gfx950: rows quantized as they are written, and read back.
//
//   c = max(floor(log2 amax) - 2 + 127, 0) of 32 channels (0xFF for a NaN or Inf), code =
//   e2m1(x / 2^(c - 127)), nearest, ties to even, saturating at 6
//
// Bound by memory (a prompt of 57600 rows, 40 heads of 128, bf16: written in 274 us, read back in 257, 1.49 GB each, 5.4 and
// 5.8 TB/s) or by the launch (64 rows of 8 heads: 4.5 and 3.5 us).  A wavefront owns a block of 16 tokens
// of one head, keys and values, and goes through its rows in items of 8 channels, neighbouring lanes on
// neighbouring items, so that rows are read and written in whole lines.  The block's bytes, which lie in the
// attention's order (value codes four tokens to a dword), pass through LDS.  Blocks that the call covers in
// part are stored item by item.
#include "kv_device.h"

namespace w4a4 {

namespace {

// Eight nibbles of finite values whose group has scale code `code` (zeros for 0xFF).
__device__ __forceinline__ uint32_t e2m1_word(const float* v, uint32_t code) {
    // 2^(code - 127): the exponent field, or the subnormal 2^-127 for code 0
    const float scale = __uint_as_float(max(code << 23, 0x00400000u));
    uint32_t w = 0;
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[0], v[1], scale, 0);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[2], v[3], scale, 1);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[4], v[5], scale, 2);
    w = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(w, v[6], v[7], scale, 3);
    return code == 0xFFu ? 0u : w;
}

// Four nibbles spread to the low halves of four bytes.
__device__ __forceinline__ uint32_t spread4(uint32_t n) {
    n = (n | (n << 8)) & 0x00FF00FFu;
    return (n | (n << 4)) & 0x0F0F0F0Fu;
}

template <typename X> struct KvIn {
    const X* p;
    int64_t row, head;
};

// The value of the lane two further on in its group of four, and the group's largest.
__device__ __forceinline__ uint32_t quad_swap2(uint32_t v) { return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x4E, 0xF, 0xF, false); }
__device__ __forceinline__ uint32_t quad_max(uint32_t v) {
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0xB1, 0xF, 0xF, false));
    return max(v, quad_swap2(v));
}
template <typename T> __device__ __forceinline__ void put(uint8_t* p, T v) { __builtin_memcpy(__builtin_assume_aligned(p, sizeof(T)), &v, sizeof(T)); }
template <typename T> __device__ __forceinline__ T get(const uint8_t* p) {
    T v;
    __builtin_memcpy(&v, __builtin_assume_aligned(p, sizeof(T)), sizeof(T));
    return v;
}

// A workgroup's wavefronts take four heads of one (sequence, block) pair.
template <typename X, int G>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs a, KvIn<X> K, KvIn<X> V, uint32_t blocks, uint32_t head_groups) {
    typedef KvBlock<G> L;
    __shared__ __attribute__((aligned(16))) uint8_t images[4][L::BYTES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t hg = blockIdx.x % head_groups, rest = blockIdx.x / head_groups;
    const uint32_t rr = rest % blocks;
    const int64_t b = rest / blocks;
    const KvSeq s = kv_seq(a, b);
    const int32_t start = s.first > 0 ? s.first : 0, end = s.first + s.done;      // positions written
    const int32_t q = start / 16 + (int32_t)rr, h = (int32_t)hg * 4 + wave;
    if (q * 16 >= end || h >= a.n_heads) return;      // wave-uniform; no barrier below
    uint8_t* const blk = kv_block(a, b, (uint32_t)q, h);
    if (!blk) return;
    const bool whole = q * 16 >= start && q * 16 + 16 <= end;

    // item i of this lane: token r, channels 32 d + 8 c .. + 7
    Row8<X> x[2][G];
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int it = i * 64 + lane, r = it / (4 * G), ch = it % (4 * G);
        const int32_t pos = q * 16 + r;
        if (pos >= start && pos < end) {
            const int64_t row = s.row0 + (pos - s.first);
            x[0][i].load(K.p + row * K.row + h * K.head, 8 * ch, a.head_dim);
            x[1][i].load(V.p + row * V.row + h * V.head, 8 * ch, a.head_dim);
        } else {
            x[0][i].load(nullptr, 0, 0);      // zeros
            x[1][i].load(nullptr, 0, 0);
        }
    }
    uint8_t* const img = images[wave];
    if constexpr (L::SG > G) {      // scale bytes past the last group
        if (lane < L::SG) put(img + L::KS + 16 * lane, make_uint4(0, 0, 0, 0));
        if (lane < L::SG) put(img + L::VS + 16 * lane, make_uint4(0, 0, 0, 0));
        __builtin_amdgcn_wave_barrier();
    }
#pragma unroll
    for (int i = 0; i < G; ++i) {
        const int it = i * 64 + lane, r = it / (4 * G), ch = it % (4 * G), c = ch & 3, d = ch >> 2;
        uint32_t code[2], w[2];
#pragma unroll
        for (int t = 0; t < 2; ++t) {
            float v[8];
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                v[j] = x[t][i].at(j);
                m = max(m, abs_bits(v[j]));
            }
            code[t] = e8m0_from_absbits(quad_max(m));
            w[t] = e2m1_word(v, code[t]);
        }
        // bytes of (channel, channel + 16): items c and c + 2 hold the halves; each makes four of the eight
        const uint32_t other = quad_swap2(w[1]), lo = c < 2 ? w[1] : other, hi = c < 2 ? other : w[1];
        const int j0 = c < 2 ? 0 : 4;
        const uint32_t bytes = spread4((lo >> (4 * j0)) & 0xFFFFu) | spread4((hi >> (4 * j0)) & 0xFFFFu) << 4;
        const int key_at = ((c * 16 + r) * G + d) * 4, val_at = L::V + ((r >> 2) * 16 + 8 * (c & 1) + j0) * 4 * G + 4 * d + (r & 3);
        const int ks_at = L::KS + r * L::SG + d, vs_at = L::VS + (r >> 2) * 4 * L::SG + d * 4 + (r & 3);
        const int32_t pos = q * 16 + r;
        if (whole) {
            put(img + key_at, w[0]);
#pragma unroll
            for (int j = 0; j < 4; ++j) img[val_at + j * 4 * G] = (uint8_t)(bytes >> (8 * j));
            if (c == 0) img[ks_at] = (uint8_t)code[0];
            if (c == 1) img[vs_at] = (uint8_t)code[1];
        } else if (pos >= start && pos < end) {
            put(blk + key_at, w[0]);
#pragma unroll
            for (int j = 0; j < 4; ++j) blk[val_at + j * 4 * G] = (uint8_t)(bytes >> (8 * j));
            if (c == 0) blk[ks_at] = (uint8_t)code[0];
            if (c == 1) blk[vs_at] = (uint8_t)code[1];
            if constexpr (L::SG > G)      // the padding of this token's scales
                if (c >= 2 && d == 0)
                    for (int e = G; e < L::SG; ++e) blk[c == 2 ? ks_at + e : vs_at + 4 * e] = 0;
        }
    }
    if (!whole) return;
    __builtin_amdgcn_wave_barrier();      // the wavefront's own LDS, in order
#pragma unroll
    for (int i = 0; i < (L::BYTES + 1023) / 1024; ++i) {
        const int at = i * 1024 + lane * 16;
        if (at < L::BYTES) put(blk + at, get<uint4>(img + at));
    }
}

// 16 bytes of a row at channel p, rows of any alignment.  Where rows are whole lines they go past the
// caches: a prompt's values do not stay in them, and what they push out has to be written first (57600 x 40 x 128,
// append and read back: 570 to 537 us); lines in parts are joined in the L2 (9000 x 6 x 72 in fp32: 46 us, past it 57).
template <bool LINES> __device__ __forceinline__ void store16(float* row, int p, int cols, const float* x) {
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    const v4 v = {x[0], x[1], x[2], x[3]};
    if (p + 4 <= cols) {
        if constexpr (LINES) __builtin_nontemporal_store(v, reinterpret_cast<v4*>(row + p));
        else *reinterpret_cast<v4*>(row + p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (p + i < cols) row[p + i] = x[i];
}
template <bool LINES> __device__ __forceinline__ void store16(uint16_t* row, int p, int cols, const float* x) {
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
    const v4 v = {pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
    if (p + 8 <= cols) {
        if constexpr (LINES) __builtin_nontemporal_store(v, reinterpret_cast<v4*>(row + p));
        else *reinterpret_cast<v4*>(row + p) = v;
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (p + i < cols) row[p + i] = (uint16_t)(v[i / 2] >> (16 * (i & 1)));
}

// EL nibbles times the scale of `code`: exact in binary32 and in bf16.
template <int EL> __device__ __forceinline__ void values(uint32_t w, uint32_t code, float* x) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(code == 0xFFu ? 0x7FC00000u : max(code << 23, 0x00400000u));
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
    for (int j = 0; j < EL; ++j) x[j] = v[j] * s;
}

// An item is 16 bytes of output: EL channels.
template <typename Y, int G, bool LINES>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, Y* __restrict__ K, Y* __restrict__ V, uint32_t blocks, uint32_t head_groups) {
    typedef KvBlock<G> L;
    constexpr int EL = 16 / sizeof(Y), ITEMS = 32 * G / EL;
    __shared__ __attribute__((aligned(16))) uint8_t images[4][L::BYTES];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    const uint32_t hg = blockIdx.x % head_groups, rest = blockIdx.x / head_groups;
    const uint32_t rr = rest % blocks;
    const int64_t b = rest / blocks;
    const KvSeq s = kv_seq(a, b);
    // blocks from the first row's on; positions below zero come first (their rows read as zero)
    const int32_t q0 = s.first >= 0 ? s.first / 16 : -((15 - s.first) / 16);
    const int32_t q = q0 + (int32_t)rr, h = (int32_t)hg * 4 + wave, end = s.first + s.done;
    if (q * 16 >= end || h >= a.n_heads) return;
    const uint8_t* const blk = q >= 0 ? kv_block(a, b, (uint32_t)q, h) : nullptr;
    uint8_t* const img = images[wave];
#pragma unroll
    for (int i = 0; i < (L::BYTES + 1023) / 1024; ++i) {
        const int at = i * 1024 + lane * 16;
        if (at < L::BYTES) put(img + at, blk ? __builtin_nontemporal_load(reinterpret_cast<const v4i*>(blk + at)) : v4i{0, 0, 0, 0});
    }
    __builtin_amdgcn_wave_barrier();      // the wavefront's own LDS, in order
#pragma unroll
    for (int i = 0; i < ITEMS / 4; ++i) {
        const int it = i * 64 + lane, r = it / ITEMS, p = it % ITEMS * EL, d = p >> 5, c = p >> 3 & 3;
        const int32_t pos = q * 16 + r;
        if (pos < s.first || pos >= end || p >= a.head_dim) continue;
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < EL; ++j)
            w |= (((uint32_t)img[L::V + ((r >> 2) * 16 + (p & 15) + j) * 4 * G + 4 * d + (r & 3)] >> (4 * (c >> 1))) & 15u) << (4 * j);
        const int64_t at = ((s.row0 + (pos - s.first)) * a.n_heads + h) * a.head_dim;
        float x[8];
        values<EL>(get<uint32_t>(img + ((c * 16 + r) * G + d) * 4) >> (p & 4 ? 16 : 0), img[L::KS + r * L::SG + d], x);
        store16<LINES>(K + at, p, a.head_dim, x);
        values<EL>(w, img[L::VS + (r >> 2) * 4 * L::SG + d * 4 + (r & 3)], x);
        store16<LINES>(V + at, p, a.head_dim, x);
    }
}

// Blocks that max_rows rows touch at most, and the launch's size.
struct Grid {
    uint32_t blocks, head_groups;
    dim3 n;
};
Grid grid_of(const w4a4_kv_batch& b, const w4a4_kv_cache& c) {
    Grid g;
    g.blocks = (uint32_t)((b.max_rows + 14) / 16 + 1);
    g.head_groups = (uint32_t)((c.n_heads + 3) / 4);
    g.n = dim3((uint32_t)(b.n_seqs * g.blocks * g.head_groups));
    return g;
}

template <typename X, int G>
hipError_t run_append(const w4a4_kv_rows& K, const w4a4_kv_rows& V, const KvArgs& a, const Grid& g, hipStream_t st) {
    const KvIn<X> k = {(const X*)K.data, K.row_stride, K.head_stride}, v = {(const X*)V.data, V.row_stride, V.head_stride};
    hipLaunchKernelGGL((kv_append_kernel<X, G>), g.n, dim3(256), 0, st, a, k, v, g.blocks, g.head_groups);
    return hipGetLastError();
}
template <typename Y, int G>
hipError_t run_read(void* K, void* V, const KvArgs& a, const Grid& g, hipStream_t st) {
    if (a.head_dim * sizeof(Y) % 128 == 0) hipLaunchKernelGGL((kv_read_kernel<Y, G, true>), g.n, dim3(256), 0, st, a, (Y*)K, (Y*)V, g.blocks, g.head_groups);
    else hipLaunchKernelGGL((kv_read_kernel<Y, G, false>), g.n, dim3(256), 0, st, a, (Y*)K, (Y*)V, g.blocks, g.head_groups);
    return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_append(const w4a4_kv_rows& K, const w4a4_kv_rows& V, int64_t n_rows, const w4a4_kv_batch& b,
                            const w4a4_kv_cache& c, hipStream_t st) {
    const KvArgs a = kv_args(n_rows, b, c);
    const Grid g = grid_of(b, c);
    return kv_groups(c.d_pad, [&](auto G) {
        return K.dtype == W4A4_X_BF16 ? run_append<uint16_t, G()>(K, V, a, g, st) : run_append<float, G()>(K, V, a, g, st);
    });
}

hipError_t launch_kv_read(int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, void* K, void* V, int y_dtype, hipStream_t st) {
    const KvArgs a = kv_args(n_rows, b, c);
    const Grid g = grid_of(b, c);
    return kv_groups(c.d_pad, [&](auto G) {
        return y_dtype == W4A4_Y_BF16 ? run_read<uint16_t, G()>(K, V, a, g, st) : run_read<float, G()>(K, V, a, g, st);
    });
}

}  // namespace w4a4

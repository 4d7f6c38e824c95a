// 4-bit key/value cache on gfx950: rows quantized as they are written, and read back.
//
//   c = max(floor(log2 amax) - 2 + 127, 0) of 32 channels (0xFF for a NaN or Inf), code =
//   e2m1(x / 2^(c - 127)), nearest, ties to even, saturating at 6
//
// Bound by memory (a prompt) or by the launch (a few rows).  A wavefront owns a block of 16 tokens
// of one head, keys and values: lane 16 g + r loads channels 32 b + 8 g .. + 7 of token r by
// 16-byte loads, and its eight nibbles are a dword of the key codes as they lie in memory.  The value
// codes lie four tokens to a dword, since the attention multiplies with values along the tokens;
// they are turned through LDS.  Blocks that the call covers in part are stored token by token.
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

// Codes and scale codes of this lane's channels; the scale codes, one a byte, in sc.
template <typename X, int G>
__device__ __forceinline__ void quantize(const X* row, bool live, int g, int D, uint32_t (&w)[G], uint32_t (&sc)[2]) {
    float v[G][8];
    sc[0] = sc[1] = 0;
#pragma unroll
    for (int b = 0; b < G; ++b) {
        if (live) {
            load8(row, 32 * b + 8 * g, D, v[b]);
        } else {
#pragma unroll
            for (int j = 0; j < 8; ++j) v[b][j] = 0.0f;
        }
    }
#pragma unroll
    for (int b = 0; b < G; ++b) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[b][j]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        const uint32_t c = e8m0_from_absbits(m);
        w[b] = e2m1_word(v[b], c);
        sc[b / 4] |= c << (8 * (b & 3));
    }
}

// A workgroup's wavefronts take four heads of one (sequence, block) pair.
template <typename X, int G>
__global__ __launch_bounds__(256) void kv_append_kernel(KvArgs a, KvIn<X> K, KvIn<X> V, uint32_t blocks, uint32_t head_groups) {
    typedef KvBlock<G> L;
    __shared__ __attribute__((aligned(16))) uint8_t turn[4][256 * G];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
    const uint32_t hg = blockIdx.x % head_groups, rest = blockIdx.x / head_groups;
    const uint32_t rr = rest % blocks;
    const int64_t b = rest / blocks;
    const KvSeq s = kv_seq(a, b);
    const int32_t start = s.first > 0 ? s.first : 0, end = s.first + s.done;      // positions written
    const int32_t q = start / 16 + (int32_t)rr, h = (int32_t)hg * 4 + wave;
    if (q * 16 >= end || h >= a.n_heads) return;      // wave-uniform; no barrier below
    uint8_t* const blk = kv_block(a, b, (uint32_t)q, h);
    if (!blk) return;
    const int32_t pos = q * 16 + r;
    const bool live = pos >= start && pos < end;
    const int64_t row = s.row0 + (pos - s.first);
    const uint32_t mask = (uint32_t)__ballot(live && g == 0);      // bit t: token t is written

    uint32_t kw[G], vw[G], ks[2], vs[2];
    quantize<X, G>(K.p + (live ? row * K.row + h * K.head : 0), live, g, a.head_dim, kw, ks);
    quantize<X, G>(V.p + (live ? row * V.row + h * V.head : 0), live, g, a.head_dim, vw, vs);

    if (live) {
        uint32_t* const kd = reinterpret_cast<uint32_t*>(blk) + lane * G;
#pragma unroll
        for (int c = 0; c < G; ++c) kd[c] = kw[c];
        if (g == 0) {
            uint8_t* const sd = blk + L::KS + r * L::SG;
            if constexpr (G == 1) sd[0] = (uint8_t)ks[0];
            else if constexpr (G == 2) *reinterpret_cast<uint16_t*>(sd) = (uint16_t)ks[0];
            else {
                reinterpret_cast<uint32_t*>(sd)[0] = ks[0];
                if constexpr (G > 4) reinterpret_cast<uint32_t*>(sd)[1] = ks[1];
            }
        }
        uint8_t* const sv = blk + L::VS + (r >> 2) * 4 * L::SG + (r & 3);
#pragma unroll
        for (int c = 0; c < L::SG; ++c)
            if ((c & 3) == g) sv[c * 4] = (uint8_t)(vs[c / 4] >> (8 * (c & 3)));
    }
    // Bytes of (d, d + 16): lanes g < 2 hold d = 8 g + j, lanes g + 2 the other half; each of the two
    // makes four of the eight bytes.
    uint8_t* const t = turn[wave];
#pragma unroll
    for (int c = 0; c < G; ++c) {
        const uint32_t other = (uint32_t)__shfl_xor((int)vw[c], 32);
        const uint32_t lo = g < 2 ? vw[c] : other, hi = g < 2 ? other : vw[c];
        const int j0 = g < 2 ? 0 : 4;
        const uint32_t bytes = spread4((lo >> (4 * j0)) & 0xFFFFu) | spread4((hi >> (4 * j0)) & 0xFFFFu) << 4;
#pragma unroll
        for (int j = 0; j < 4; ++j) t[((r >> 2) * 16 + 8 * (g & 1) + j0 + j) * 4 * G + 4 * c + (r & 3)] = (uint8_t)(bytes >> (8 * j));
    }
    __builtin_amdgcn_wave_barrier();      // the wavefront's own LDS, in order
    const uint32_t m4 = (mask >> (4 * g)) & 15u;      // this lane's dwords hold tokens 4 g .. + 3
#pragma unroll
    for (int c = 0; c < G; ++c) {
        const uint32_t v = *reinterpret_cast<const uint32_t*>(t + lane * 4 * G + 4 * c);
        uint8_t* const d = blk + L::V + lane * 4 * G + 4 * c;
        if (m4 == 15u) {
            *reinterpret_cast<uint32_t*>(d) = v;
        } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
                if (m4 >> j & 1) d[j] = (uint8_t)(v >> (8 * j));
        }
    }
}

// 8 values of a row at channel p, rows of any alignment.
__device__ __forceinline__ void store8(float* row, int p, int cols, const float* x) {
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    if (p + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < 2; ++i) *reinterpret_cast<v4*>(row + p + 4 * i) = v4{x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (p + i < cols) row[p + i] = x[i];
}
__device__ __forceinline__ void store8(uint16_t* row, int p, int cols, const float* x) {
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
    const uint32_t w[4] = {pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])};
    if (p + 8 <= cols) {
        *reinterpret_cast<v4*>(row + p) = v4{w[0], w[1], w[2], w[3]};
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (p + i < cols) row[p + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

// Eight nibbles times the scale of `code`: exact in binary32 and in bf16.
__device__ __forceinline__ void values8(uint32_t w, uint32_t code, float* x) {
    typedef float v2f __attribute__((ext_vector_type(2)));
    const float s = __uint_as_float(code == 0xFFu ? 0x7FC00000u : max(code << 23, 0x00400000u));
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = v[j] * s;
}

template <typename Y, int G>
__global__ __launch_bounds__(256) void kv_read_kernel(KvArgs a, Y* __restrict__ K, Y* __restrict__ V, uint32_t blocks, uint32_t head_groups) {
    typedef KvBlock<G> L;
    __shared__ __attribute__((aligned(16))) uint8_t turn[4][256 * G];
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
    const uint32_t hg = blockIdx.x % head_groups, rest = blockIdx.x / head_groups;
    const uint32_t rr = rest % blocks;
    const int64_t b = rest / blocks;
    const KvSeq s = kv_seq(a, b);
    // blocks from the first row's on; positions below zero come first (their rows read as zero)
    const int32_t q0 = s.first >= 0 ? s.first / 16 : -((15 - s.first) / 16);
    const int32_t q = q0 + (int32_t)rr, h = (int32_t)hg * 4 + wave, end = s.first + s.done;
    if (q * 16 >= end || h >= a.n_heads) return;
    const int32_t pos = q * 16 + r;
    const bool live = pos >= s.first && pos < end;
    const uint8_t* const blk = q >= 0 ? kv_block(a, b, (uint32_t)q, h) : nullptr;
    const int64_t at = ((s.row0 + (pos - s.first)) * a.n_heads + h) * a.head_dim;
    uint32_t kw[G], ks[2] = {0, 0}, vs[2] = {0, 0}, vd[G];
#pragma unroll
    for (int c = 0; c < G; ++c) kw[c] = vd[c] = 0;
    if (blk) {
#pragma unroll
        for (int c = 0; c < G; ++c) {
            kw[c] = reinterpret_cast<const uint32_t*>(blk)[lane * G + c];
            vd[c] = reinterpret_cast<const uint32_t*>(blk + L::V)[lane * G + c];
            ks[c / 4] |= (uint32_t)blk[L::KS + r * L::SG + c] << (8 * (c & 3));
            vs[c / 4] |= (uint32_t)blk[L::VS + (r >> 2) * 4 * L::SG + c * 4 + (r & 3)] << (8 * (c & 3));
        }
    }
    uint8_t* const t = turn[wave];
#pragma unroll
    for (int c = 0; c < G; ++c) *reinterpret_cast<uint32_t*>(t + lane * 4 * G + 4 * c) = vd[c];
    __builtin_amdgcn_wave_barrier();
#pragma unroll
    for (int c = 0; c < G; ++c) {
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j)
            w |= (((uint32_t)t[((r >> 2) * 16 + 8 * (g & 1) + j) * 4 * G + 4 * c + (r & 3)] >> (4 * (g >> 1))) & 15u) << (4 * j);
        if (!live) continue;
        float x[8];
        values8(kw[c], ks[c / 4] >> (8 * (c & 3)) & 0xFFu, x);
        store8(K + at, 32 * c + 8 * g, a.head_dim, x);
        values8(w, vs[c / 4] >> (8 * (c & 3)) & 0xFFu, x);
        store8(V + at, 32 * c + 8 * g, a.head_dim, x);
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
    hipLaunchKernelGGL((kv_read_kernel<Y, G>), g.n, dim3(256), 0, st, a, (Y*)K, (Y*)V, g.blocks, g.head_groups);
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

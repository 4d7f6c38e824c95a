// FP8 block quantization on gfx950: activations (one scale per token and 128 inputs) and
// weights (one scale per 128 x 128 block) into E4M3 codes, in the order in which the
// products of fp8gemm.hip and moe.hip read them.
//
//   s = max(fl32(amax / 448), 2^-60), or the smallest power of two >= 2^-60 with
//   amax <= 448 s;  q = e4m3_rne(fl32(x / s)).
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

// The 16 values of one 16-byte piece of the packed order: inputs p .. + 7 and p + 32 .. + 39
// (p = 64 half + 8 chunk of the block).
template <typename X>
__device__ __forceinline__ void load_piece(const X* row, int64_t p, int64_t cols, float* x) {
    load8(row, p, cols, x);
    load8(row, p + 32, cols, x + 8);
}

template <typename Inv>
__device__ __forceinline__ uint4 encode_piece(const float* x, float s, const Inv& inv) {
    const uint2 a = encode8(x, s, inv), b = encode8(x + 8, s, inv);
    return make_uint4(a.x, a.y, b.x, b.y);
}

// A launch counts its work items in 32 bits, which 64 GiB of codes already exceed; longer work runs
// as launches of this many workgroups, which the kernels number from `first` on (a GiB of codes or
// more each, so that their starts do not count).
constexpr int64_t SLICE = 1 << 18;
template <typename F>
hipError_t in_slices(int64_t workgroups, const F& launch) {
    for (int64_t first = 0; first < workgroups; first += SLICE) {
        launch(dim3((uint32_t)(workgroups - first < SLICE ? workgroups - first : SLICE)), first);
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess) return e;
    }
    return hipSuccess;
}

// Activations.  A wavefront takes 16 tokens x one block of 128 inputs, one run of the packed order:
// lane l holds the 32 inputs that it has in the matrix instructions (token l % 16, inputs
// 32 q + 8 (l / 16) .. + 7), so that the two stores write one KiB each.
template <typename X>
__global__ __launch_bounds__(256) void fp8_actquant_kernel(const X* __restrict__ x, int64_t T, int64_t d_in, int64_t nkb,
                                                           int64_t first, int64_t items, int kind, uint8_t* __restrict__ aq,
                                                           float* __restrict__ as, int64_t t_ld, int32_t* __restrict__ count) {
    if (count && first + blockIdx.x == 0)   // the product's counters
        for (int i = threadIdx.x; i < FP8_COUNTERS; i += 256) count[i] = 0;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    const int64_t item = (first + blockIdx.x) * 4 + (threadIdx.x >> 6);
    if (item >= items) return;
    const int64_t tg = item / nkb, kb = item - tg * nkb;
    const int64_t t = tg * 16 + r;
    const bool live = t < T;
    const X* const row = x + (live ? t : T - 1) * d_in;
    float v[2][16];
    uint32_t m = 0;
#pragma unroll
    for (int h = 0; h < 2; ++h) load_piece(row, kb * 128 + h * 64 + g * 8, d_in, v[h]);
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[h][j]));
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    const float s = block_scale(m, kind);
    const typename InverseOf<X>::type inv(s);
    if (!live) return;
    uint8_t* const dst = aq + item * 2048 + lane * 16;
#pragma unroll
    for (int h = 0; h < 2; ++h) *reinterpret_cast<uint4*>(dst + h * 1024) = encode_piece(v[h], s, inv);
    if (g == 0) as[kb * t_ld + t] = s;
}

// The product's counters, where the quantization of the same call does not clear them.
__global__ __launch_bounds__(FP8_COUNTERS) void fp8_clear_kernel(int32_t* __restrict__ count) { count[threadIdx.x] = 0; }

// Weights: one workgroup per 128 x 128 block; thread = (row, half of the block's inputs).
template <typename W>
__global__ __launch_bounds__(256) void fp8_pack_kernel(const W* __restrict__ w, int64_t d_in, int64_t d_out, int64_t nkb,
                                                       int64_t nnb, int64_t n_pad, int64_t first, int kind,
                                                       uint8_t* __restrict__ codes, float* __restrict__ scales) {
    __shared__ uint32_t wmax[4];
    const int64_t b = first + blockIdx.x;
    const int64_t mat = b / (nnb * nkb), nb = (b / nkb) % nnb, kb = b % nkb;
    const int64_t row = nb * 128 + (threadIdx.x >> 1);
    const int64_t p0 = kb * 128 + (threadIdx.x & 1) * 64;
    float v[4][16];
    uint32_t m = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (row < d_out) {
            load_piece(w + (mat * d_out + row) * d_in, p0 + 8 * i, d_in, v[i]);
        } else {
#pragma unroll
            for (int j = 0; j < 16; ++j) v[i][j] = 0.0f;
        }
#pragma unroll
        for (int j = 0; j < 16; ++j) m = max(m, abs_bits(v[i][j]));
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
    m = max(max(wmax[0], wmax[1]), max(wmax[2], wmax[3]));
    const float s = block_scale(m, kind);
    if (threadIdx.x == 0) scales[b] = s;
    if (row >= n_pad) return;
    const typename InverseOf<W>::type inv(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        uint8_t* dst = codes + ((mat * (n_pad / 16) + row / 16) * nkb + kb) * 2048 + (threadIdx.x & 1) * 1024 + i * 256 +
                       (row & 15) * 16;
        *reinterpret_cast<uint4*>(dst) = encode_piece(v[i], s, inv);
    }
}

// Codes of a checkpoint, row-major, into the packed order: one thread per 16-byte piece.
__global__ __launch_bounds__(256) void fp8_reorder_kernel(const uint8_t* __restrict__ src, int64_t d_in, int64_t d_out,
                                                          int64_t nkb, int64_t n_pad, int64_t first, int64_t pieces,
                                                          int vec, uint8_t* __restrict__ codes) {
    const int64_t q = (first + blockIdx.x) * 256 + threadIdx.x;
    if (q >= pieces) return;
    const int l = (int)(q & 63), h = (int)((q >> 6) & 1);
    const int64_t run = q >> 7;                       // 16 rows x 128 inputs
    const int64_t rb = run / nkb, kb = run - rb * nkb;
    const int64_t mat = rb / (n_pad / 16), row = (rb - mat * (n_pad / 16)) * 16 + (l & 15);
    uint2 v[2] = {make_uint2(0, 0), make_uint2(0, 0)};
    if (row < d_out) {
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            const int64_t p = kb * 128 + h * 64 + c * 32 + (l >> 4) * 8;
            const uint8_t* s = src + (mat * d_out + row) * d_in + p;
            if (vec && p + 8 <= d_in) {
                v[c] = *reinterpret_cast<const uint2*>(s);
            } else {
                uint32_t w[2] = {0, 0};
#pragma unroll
                for (int i = 0; i < 8; ++i) w[i / 4] |= (p + i < d_in ? (uint32_t)s[i] : 0u) << (8 * (i & 3));
                v[c] = make_uint2(w[0], w[1]);
            }
        }
    }
    *reinterpret_cast<uint4*>(codes + q * 16) = make_uint4(v[0].x, v[0].y, v[1].x, v[1].y);
}

__global__ __launch_bounds__(256) void fp8_scales_kernel(const void* __restrict__ src, int64_t first, int64_t n, int kind,
                                                         float* __restrict__ scales) {
    const int64_t i = (first + blockIdx.x) * 256 + threadIdx.x;
    if (i >= n) return;
    if (kind == W4A4_FP8_SCALE_F32) {
        scales[i] = reinterpret_cast<const float*>(src)[i];
    } else {
        const uint32_t c = reinterpret_cast<const uint8_t*>(src)[i];
        scales[i] = __uint_as_float(c == 0xFFu ? 0x7FC00000u : c == 0 ? 0x00400000u : c << 23);
    }
}

}  // namespace

hipError_t launch_fp8_actquant(const void* X, int x_dtype, int64_t T, int64_t d_in, int kind, uint8_t* aq, float* as,
                               int64_t t_ld, int32_t* count, hipStream_t st) {
    const int64_t nkb = (d_in + 127) / 128, items = (T + 15) / 16 * nkb;
    return in_slices((items + 3) / 4, [&](dim3 grid, int64_t first) {
        if (x_dtype == W4A4_X_BF16)
            hipLaunchKernelGGL(fp8_actquant_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)X, T, d_in, nkb, first, items, kind,
                               aq, as, t_ld, count);
        else
            hipLaunchKernelGGL(fp8_actquant_kernel<float>, grid, dim3(256), 0, st, (const float*)X, T, d_in, nkb, first, items, kind, aq, as,
                               t_ld, count);
    });
}

hipError_t launch_fp8_clear(int32_t* count, hipStream_t st) {
    hipLaunchKernelGGL(fp8_clear_kernel, dim3(1), dim3(FP8_COUNTERS), 0, st, count);
    return hipGetLastError();
}

hipError_t launch_fp8_pack(const void* W, int w_dtype, const w4a4_fp8_packed& d, uint8_t* codes, float* scales,
                           hipStream_t st) {
    const int64_t nkb = d.k_pad / 128, nnb = (d.d_out + 127) / 128;
    return in_slices(d.n_mat * nnb * nkb, [&](dim3 grid, int64_t first) {
        if (w_dtype == W4A4_X_BF16)
            hipLaunchKernelGGL(fp8_pack_kernel<uint16_t>, grid, dim3(256), 0, st, (const uint16_t*)W, d.d_in, d.d_out, nkb, nnb, d.n_pad,
                               first, d.scale_kind, codes, scales);
        else
            hipLaunchKernelGGL(fp8_pack_kernel<float>, grid, dim3(256), 0, st, (const float*)W, d.d_in, d.d_out, nkb, nnb, d.n_pad, first,
                               d.scale_kind, codes, scales);
    });
}

hipError_t launch_reorder_codes(const uint8_t* src, int64_t n_mat, int64_t d_in, int64_t d_out, uint8_t* codes, hipStream_t st) {
    const int64_t nkb = (d_in + 127) / 128, n_pad = (d_out + 15) / 16 * 16, pieces = n_mat * n_pad * nkb * 8;
    return in_slices((pieces + 255) / 256, [&](dim3 grid, int64_t first) {
        hipLaunchKernelGGL(fp8_reorder_kernel, grid, dim3(256), 0, st, src, d_in, d_out, nkb, n_pad, first, pieces,
                           d_in % 8 == 0 ? 1 : 0, codes);
    });
}

hipError_t launch_fp8_reorder(const uint8_t* src, const void* src_scales, const w4a4_fp8_packed& d, uint8_t* codes,
                              float* scales, hipStream_t st) {
    const hipError_t e = launch_reorder_codes(src, d.n_mat, d.d_in, d.d_out, codes, st);
    if (e != hipSuccess) return e;
    const int64_t n = d.n_mat * ((d.d_out + 127) / 128) * (d.k_pad / 128);
    return in_slices((n + 255) / 256, [&](dim3 grid, int64_t first) {
        hipLaunchKernelGGL(fp8_scales_kernel, grid, dim3(256), 0, st, src_scales, first, n, d.scale_kind, scales);
    });
}

}  // namespace w4a4

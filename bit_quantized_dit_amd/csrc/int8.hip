// INT8 quantization of rows (tokens, or weight rows) on gfx950 into two's complement codes, in
// the packed order of the FP8 layer: runs of 16 rows x 128 inputs, lane 16 g + r of a run holding
// inputs 32 q + 8 g .. + 7 (q < 4) of row r.
//
//   s = max(fl32(amax / 127), 2^-60);  q = rne(fl32(x / s))
//
// Bound by memory: one read of X, one write of codes.  A workgroup owns 16 rows, because a run's
// stores are whole KiB then; its wavefronts take every NW-th block of 128 inputs.  The scale needs
// the whole row before the first code, so up to HB blocks a wavefront stay in registers between
// the two passes, and wider rows are read again.
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

// 8 neighbouring values of a row of any alignment, as they lie in memory; zero past its end.
template <typename X> struct Row8;
template <> struct Row8<float> {
    float v[8];
    __device__ void load(const float* row, int64_t p, int64_t cols) { load8(row, p, cols, v); }
    __device__ float at(int i) const { return v[i]; }
};
template <> struct Row8<uint16_t> {
    uint32_t w[4];
    __device__ void load(const uint16_t* row, int64_t p, int64_t cols) {
        typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
        if (p + 8 <= cols) {
            const v4 v = *reinterpret_cast<const v4*>(row + p);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[j] = v[j];
            return;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            w[j] = (p + 2 * j < cols ? (uint32_t)row[p + 2 * j] : 0u) | (p + 2 * j + 1 < cols ? (uint32_t)row[p + 2 * j + 1] << 16 : 0u);
    }
    __device__ float at(int i) const { return __uint_as_float(i & 1 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16); }
};

// The 32 values of a lane in a block: chunk c holds inputs 32 c + 8 g .. + 7.
template <typename X>
__device__ __forceinline__ void load_block(Row8<X> (&v)[4], const X* row, int64_t p, int64_t cols) {
#pragma unroll
    for (int c = 0; c < 4; ++c) v[c].load(row, p + 32 * c, cols);
}
template <typename X>
__device__ __forceinline__ uint32_t block_amax(const Row8<X> (&v)[4], uint32_t m) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, abs_bits(v[c].at(j)));
    return m;
}
// Adding 1.5 * 2^23 rounds a quotient of at most 127 (and a rounding) to the nearest integer, ties
// to even, and leaves its two's complement in the low byte.
template <typename X, typename Inv>
__device__ __forceinline__ uint32_t encode4(const Row8<X>& v, int j, float s, const Inv& inv) {
    uint32_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) b[i] = __float_as_uint(inv.of(v.at(j + i), s) + 12582912.0f);
    const uint32_t lo = __builtin_amdgcn_perm(b[1], b[0], 0x0C0C0400u), hi = __builtin_amdgcn_perm(b[3], b[2], 0x04000C0Cu);
    return lo | hi;
}
template <typename X, typename Inv>
__device__ __forceinline__ void store_block(const Row8<X> (&v)[4], float s, const Inv& inv, uint8_t* dst) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
        uint4 o = make_uint4(encode4(v[2 * h], 0, s, inv), encode4(v[2 * h], 4, s, inv), encode4(v[2 * h + 1], 0, s, inv),
                             encode4(v[2 * h + 1], 4, s, inv));
        if (s != s) o = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + h * 1024) = o;
    }
}

template <typename X, int NW, int HB>
__global__ __launch_bounds__(NW * 64) void int8_quant_kernel(const X* __restrict__ x, int64_t rows, int64_t d_in, int nkb, int zero_past,
                                                             uint8_t* __restrict__ q, float* __restrict__ sc, int32_t* __restrict__ count) {
    __shared__ uint32_t wmax[NW][16];
    if (count && blockIdx.x == 0)   // the product's counters
        for (int i = threadIdx.x; i < INT8_COUNTERS; i += NW * 64) count[i] = 0;
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4, wave = threadIdx.x >> 6;
    const int64_t t = (int64_t)blockIdx.x * 16 + r;
    const bool live = t < rows;
    const X* const row = x + (live ? t : rows - 1) * d_in;
    uint8_t* const dst = q + (int64_t)blockIdx.x * nkb * 2048 + lane * 16;
    uint32_t m = 0;
    Row8<X> v[HB > 0 ? HB : 1][4];
    if constexpr (HB > 0) {
#pragma unroll
        for (int i = 0; i < HB; ++i)
            if (wave + i * NW < nkb) load_block(v[i], row, (int64_t)(wave + i * NW) * 128 + g * 8, d_in);
#pragma unroll
        for (int i = 0; i < HB; ++i)
            if (wave + i * NW < nkb) m = block_amax(v[i], m);
    } else {
        for (int kb = wave; kb < nkb; kb += NW) {
            load_block(v[0], row, (int64_t)kb * 128 + g * 8, d_in);
            m = block_amax(v[0], m);
        }
    }
    m = max(m, (uint32_t)__shfl_xor((int)m, 16));
    m = max(m, (uint32_t)__shfl_xor((int)m, 32));
    if (g == 0) wmax[wave][r] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NW; ++w) m = max(m, wmax[w][r]);
    float s = m >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __builtin_fmaxf(__uint_as_float(m) / 127.0f, 0x1p-60f);
    if (!live) {      // rows past the last one: zeros where asked for
        if (!zero_past) return;
        s = __uint_as_float(0x7FC00000u);
    }
    const typename InverseOf<X>::type inv(s);
    if constexpr (HB > 0) {
#pragma unroll
        for (int i = 0; i < HB; ++i)
            if (wave + i * NW < nkb) store_block(v[i], s, inv, dst + (int64_t)(wave + i * NW) * 2048);
    } else {
        for (int kb = wave; kb < nkb; kb += NW) {
            load_block(v[0], row, (int64_t)kb * 128 + g * 8, d_in);
            store_block(v[0], s, inv, dst + (int64_t)kb * 2048);
        }
    }
    if (wave == 0 && g == 0) sc[t] = live ? s : 0.0f;
}

__global__ __launch_bounds__(INT8_COUNTERS) void int8_clear_kernel(int32_t* __restrict__ count) { count[threadIdx.x] = 0; }

__global__ __launch_bounds__(256) void int8_scales_kernel(const float* __restrict__ src, int64_t n, int64_t n_pad, float* __restrict__ dst) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i < n_pad) dst[i] = i < n ? src[i] : 0.0f;
}

template <typename X, int NW, int HB>
hipError_t run_quant(const void* x, int64_t rows, int64_t d_in, bool zero_past, uint8_t* q, float* s, int32_t* count, hipStream_t st) {
    hipLaunchKernelGGL((int8_quant_kernel<X, NW, HB>), dim3((uint32_t)((rows + 15) / 16)), dim3(NW * 64), 0, st, (const X*)x, rows, d_in,
                       (int)((d_in + 127) / 128), zero_past ? 1 : 0, q, s, count);
    return hipGetLastError();
}

}  // namespace

// The held blocks' registers: 16 a block of bf16, 32 of fp32; 8 wavefronts have 256 registers each,
// 16 have 128.
hipError_t launch_int8_quant(const void* X, int x_dtype, int64_t rows, int64_t d_in, bool zero_past, uint8_t* q, float* s,
                             int32_t* count, hipStream_t st) {
    const int64_t nkb = (d_in + 127) / 128;
    if (x_dtype == W4A4_X_BF16) {
        if (nkb <= 40 && rows > 4096) return run_quant<uint16_t, 8, 5>(X, rows, d_in, zero_past, q, s, count, st);
        if (nkb <= 80) return run_quant<uint16_t, 16, 5>(X, rows, d_in, zero_past, q, s, count, st);
        return run_quant<uint16_t, 16, 0>(X, rows, d_in, zero_past, q, s, count, st);
    }
    if (nkb <= 32) return run_quant<float, 16, 2>(X, rows, d_in, zero_past, q, s, count, st);
    if (nkb <= 40) return run_quant<float, 8, 5>(X, rows, d_in, zero_past, q, s, count, st);
    return run_quant<float, 16, 0>(X, rows, d_in, zero_past, q, s, count, st);
}

hipError_t launch_int8_clear(int32_t* count, hipStream_t st) {
    hipLaunchKernelGGL(int8_clear_kernel, dim3(1), dim3(INT8_COUNTERS), 0, st, count);
    return hipGetLastError();
}

hipError_t launch_int8_scales(const float* src, int64_t n, int64_t n_pad, float* dst, hipStream_t st) {
    hipLaunchKernelGGL(int8_scales_kernel, dim3((uint32_t)((n_pad + 255) / 256)), dim3(256), 0, st, src, n, n_pad, dst);
    return hipGetLastError();
}

}  // namespace w4a4

// INT8 quantization of rows (tokens, or weight rows) on gfx950 into two's complement codes, in
// the packed order of the FP8 layer: runs of 16 rows x 128 inputs, lane 16 g + r of a run holding
// inputs 32 q + 8 g .. + 7 (q < 4) of row r.
//
//   s = max(fl32(amax / 127), 2^-60);  q = rne(fl32(x / s))
//
// Bound by memory: one read of X, one write of codes.  A workgroup owns 16 rows, because a run's
// stores are whole KiB then (57600 x 5120 bf16: 156 us, 0.89 GB, 5.7 TB/s, above the rate of a copy); its wavefronts take every NW-th block of 128 inputs.  The scale needs
// the whole row before the first code, so up to HB blocks a wavefront stay in registers between
// the two passes, and wider rows are read again.
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

// Scale of a row from the bit pattern of its largest |x|.
__device__ __forceinline__ float scale_of(uint32_t amax_bits) {
    return amax_bits >= 0x7F800000u ? __uint_as_float(0x7FC00000u) : __builtin_fmaxf(__uint_as_float(amax_bits) / 127.0f, 0x1p-60f);
}

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
    float s = scale_of(m);
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

// Few rows: a workgroup a row, its lanes a 16-byte piece of codes each (inputs 64 h + 8 g .. + 7 and the
// same 32 further on), HP pieces held between the passes.
template <typename X, int NT, int HP>
__global__ __launch_bounds__(NT) void int8_quant_row_kernel(const X* __restrict__ x, int64_t d_in, int pieces, uint8_t* __restrict__ q,
                                                            float* __restrict__ sc, int32_t* __restrict__ count) {
    __shared__ uint32_t wmax[NT / 64];
    if (count && blockIdx.x == 0)   // the product's counters
        for (int i = threadIdx.x; i < INT8_COUNTERS; i += NT) count[i] = 0;
    const int64_t t = blockIdx.x;
    const X* const row = x + t * d_in;
    uint8_t* const dst = q + (t >> 4) * pieces * 256 + (t & 15) * 16;      // (8 pieces of 256 bytes a block of 16 rows)
    Row8<X> v[HP][2];
    uint32_t m = 0;
    auto input_of = [](int p) { return (int64_t)(p >> 3) * 128 + (p & 4) * 16 + (p & 3) * 8; };
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int p = threadIdx.x + i * NT;
        if (p >= pieces) break;
        v[i][0].load(row, input_of(p), d_in);
        v[i][1].load(row, input_of(p) + 32, d_in);
    }
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        if ((int)threadIdx.x + i * NT >= pieces) break;
#pragma unroll
        for (int j = 0; j < 8; ++j) m = max(m, max(abs_bits(v[i][0].at(j)), abs_bits(v[i][1].at(j))));
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, o));
    if ((threadIdx.x & 63) == 0) wmax[threadIdx.x >> 6] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 64; ++w) m = max(m, wmax[w]);
    const float s = scale_of(m);
    const typename InverseOf<X>::type inv(s);
#pragma unroll
    for (int i = 0; i < HP; ++i) {
        const int p = threadIdx.x + i * NT;
        if (p >= pieces) break;
        uint4 o = make_uint4(encode4(v[i][0], 0, s, inv), encode4(v[i][0], 4, s, inv), encode4(v[i][1], 0, s, inv), encode4(v[i][1], 4, s, inv));
        if (s != s) o = make_uint4(0, 0, 0, 0);
        *reinterpret_cast<uint4*>(dst + (int64_t)p * 256) = o;
    }
    if (threadIdx.x == 0) sc[t] = s;
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

template <typename X, int NT, int HP>
hipError_t run_rows(const void* x, int64_t rows, int64_t d_in, uint8_t* q, float* s, int32_t* count, hipStream_t st) {
    hipLaunchKernelGGL((int8_quant_row_kernel<X, NT, HP>), dim3((uint32_t)rows), dim3(NT), 0, st, (const X*)x, d_in, (int)((d_in + 127) / 128 * 8), q,
                       s, count);
    return hipGetLastError();
}
template <typename X>
hipError_t run_few(const void* x, int64_t rows, int64_t d_in, uint8_t* q, float* s, int32_t* count, hipStream_t st) {
    const int64_t pieces = (d_in + 127) / 128 * 8;
    if (pieces <= 256) return run_rows<X, 256, 1>(x, rows, d_in, q, s, count, st);
    if (pieces <= 512) return run_rows<X, 512, 1>(x, rows, d_in, q, s, count, st);
    if (pieces <= 1024) return run_rows<X, 1024, 1>(x, rows, d_in, q, s, count, st);
    return run_rows<X, 1024, 2>(x, rows, d_in, q, s, count, st);
}

}  // namespace

// A row a workgroup, up to this many rows (us, bf16, a row against 16 rows a workgroup: 1 x 5120 2.4 and 7.6,
// 333 x 4999 5.0 and 17.4, 1024 x 5120 7.2 and 10.2, 2048 11.5 and 11.8, 4096 21.6 and 14.2; 24 x 13824 in fp32 3.8
// and 50): its 16-byte stores of one row lie 256 bytes apart.
constexpr int64_t ROWS_FEW = 1024;
// The held blocks' registers: 16 a block of bf16, 32 of fp32; 8 wavefronts have 256 registers each,
// 16 have 128.
hipError_t launch_int8_quant(const void* X, int x_dtype, int64_t rows, int64_t d_in, bool zero_past, uint8_t* q, float* s,
                             int32_t* count, hipStream_t st) {
    const int64_t nkb = (d_in + 127) / 128;
    if (rows <= ROWS_FEW && nkb <= 256 && !zero_past)
        return x_dtype == W4A4_X_BF16 ? run_few<uint16_t>(X, rows, d_in, q, s, count, st) : run_few<float>(X, rows, d_in, q, s, count, st);
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

// Device helpers of the FP8 kernels: block scales and E4M3 codes, buffer loads.
#pragma once

#include "w4a4_device.h"
#include "../../include/w4a4.h"

namespace w4a4 {

// Scale of a block from the bit pattern of its largest |x|.
__device__ __forceinline__ float block_scale(uint32_t amax_bits, int kind) {
    if (amax_bits >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    if (kind == W4A4_FP8_SCALE_F32) return __builtin_fmaxf(__uint_as_float(amax_bits) / 448.0f, 0x1p-60f);
    // amax = (1 + m / 2^23) 2^(e - 127), 448 = 1.75 * 2^8
    const int e = (int)(amax_bits >> 23) - 8 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)(e < 127 - 60 ? 127 - 60 : e) << 23);
}

// fl32(x / s) without a division per element.  Binary32 x: the double product x * RN64(1 / s)
// rounded to binary32; it lies within 2^-52 (relative) of x / s, and a quotient of two binary32
// numbers stays further than that from every binary32 rounding midpoint, so the rounding lands on
// the same value.  bf16 x: q = x r, then q - (q s - x) r with r = RN32(1 / s), three full-rate
// operations; equal to the quotient for every bf16 significand and every significand of s (2^30
// pairs, compared at two exponents each).  The remainder is taken as q s - x, because x - q s is +0
// for a zero of either sign and would turn a quotient of -0 into +0.  Quotients below 2^-11 may
// differ where a remainder leaves the normal range; they are the code of a zero of their sign either
// way, as s >= 2^-60.
struct InverseF32 {
    double r;
    __device__ explicit InverseF32(float s) : r(1.0 / (double)s) {}
    __device__ float of(float x, float) const { return (float)((double)x * r); }
};
struct InverseBf16 {
    float r;
    __device__ explicit InverseBf16(float s) : r(1.0f / s) {}
    __device__ float of(float x, float s) const {
        const float q = x * r;
        return __builtin_fmaf(-__builtin_fmaf(q, s, -x), r, q);
    }
};
template <typename X> struct InverseOf { typedef InverseF32 type; };
template <> struct InverseOf<uint16_t> { typedef InverseBf16 type; };

// 8 values to 8 codes; a block whose scale is NaN has zero codes.
template <typename Inv>
__device__ __forceinline__ uint2 encode8(const float* x, float s, const Inv& inv) {
    uint32_t w[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        float q[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = inv.of(x[4 * i + j], s);
        const int r = __builtin_amdgcn_cvt_pk_fp8_f32(q[0], q[1], 0, false);
        w[i] = s != s ? 0u : (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(q[2], q[3], r, true);
    }
    return make_uint2(w[0], w[1]);
}

// Values p .. p + 7 of a row of `cols`, zero past its end.  Rows of any alignment: the loads are
// marked as aligned to an element only (the hardware takes unaligned vector loads).
__device__ __forceinline__ void load8(const float* row, int64_t p, int64_t cols, float* x) {
    typedef float v4 __attribute__((ext_vector_type(4), aligned(4)));
    if (p + 8 <= cols) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const v4 v = *reinterpret_cast<const v4*>(row + p + 4 * i);
#pragma unroll
            for (int j = 0; j < 4; ++j) x[4 * i + j] = v[j];
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p + i < cols ? row[p + i] : 0.0f;
}
__device__ __forceinline__ void load8(const uint16_t* row, int64_t p, int64_t cols, float* x) {
    typedef uint32_t v4 __attribute__((ext_vector_type(4), aligned(2)));
    if (p + 8 <= cols) {
        const v4 v = *reinterpret_cast<const v4*>(row + p);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = __uint_as_float(v[j] << 16);
            x[2 * j + 1] = __uint_as_float(v[j] & 0xFFFF0000u);
        }
        return;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = p + i < cols ? bf16_to_f32(row[p + i]) : 0.0f;
}
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

// Values that workgroups of different XCDs pass each other go past the XCDs' caches, value by value: a
// release or acquire fence would write back or drop a whole L2 (and made these kernels up to 8
// times slower).
__device__ __forceinline__ void put_shared(float* p, float v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ float get_shared(const float* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

// Buffer loads: a uniform descriptor, a lane offset that stays in one register for a whole stream
// and a uniform offset that walks it (flat addresses cost two registers a load in flight).
typedef __amdgpu_buffer_rsrc_t Rsrc;
__device__ __forceinline__ Rsrc rsrc(const void* p, uint32_t bytes) {
    return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
__device__ __forceinline__ uint4 load_at(Rsrc p, uint32_t lane_off, uint32_t off) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(p, (int)lane_off, (int)off, 0));
}
// The same for codes, which a call reads once: marked non-temporal, they do not push what is read
// again (tokens, h, routing) out of the L2 (the experts' up step of 64 tokens, 64 experts of 5120 x
// 1536: 190 to 176 us).
__device__ __forceinline__ uint4 load_once(Rsrc p, uint32_t lane_off, uint32_t off) {
    return __builtin_bit_cast(uint4, __builtin_amdgcn_raw_buffer_load_b128(p, (int)lane_off, (int)off, 2));
}
__device__ __forceinline__ float load_word(Rsrc p, uint32_t lane_off) {
    return __uint_as_float((uint32_t)__builtin_amdgcn_raw_buffer_load_b32(p, (int)lane_off, 0, 0));
}
// Added to the lane offset of a load that nothing needs: past every descriptor's range (which is
// below 2^31 bytes), it reads zeros and no memory.
constexpr uint32_t NO_LOAD = 0x80000000u;

}  // namespace w4a4

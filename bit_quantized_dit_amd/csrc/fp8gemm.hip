// FP8 block-scaled product on gfx950:
//
//   Y[t][n] = sum_b s_x[t][b] s_w[n / 128][b] sum_{p in block b} q_x[t][p] q_w[n][p]
//
// over blocks b of 128 inputs, E4M3 codes, binary32 sums.  Operand roles as in gemm.hip:
// src0 = weight rows, src1 = token rows, so a lane of the result holds one token and its
// activation scale is one value per lane.
//
// Both operands lie in memory in runs of 16 rows x 128 inputs (2 KiB), in the order in which a
// wavefront of a 16-row matrix instruction reads them: lane l takes row l % 16 and the 32 inputs
// 32 q + 8 (l / 16) .. + 7, q < 4, its two 16-byte halves at 16 l and 1024 + 16 l.  (Which inputs
// a lane takes is free as long as both operands agree; these let the unquantized operand of
// moe.hip be read in 64-byte pieces of its rows.)  Runs of a row block
// follow each other along the inputs, so that whoever streams 16 rows reads one contiguous
// range; copies to LDS are linear; and a 32-row fragment takes 16 rows from each of two runs
// in 256-byte pieces that no two of 16 neighbouring lanes' banks share.
//
// Precision.  The FP8 matrix instructions (all of them, whatever their shape) line the
// products of a few inputs up with the largest one and drop what falls about 13 bits below
// it: on Gaussian codes a block's sum is off by 1.4e-5 of its norm, with one heavy input by
// 4e-5 (measured against exact sums).  For bf16 outputs that is a fiftieth of the final
// rounding and the FP8 instructions run.  fp32 outputs, and few tokens (where the arithmetic
// is free), take the codes widened to bf16, which is exact: bf16 products are exact in
// binary32 and their sums are off by 1e-8.
//
// Scales.  The MFMAs of a block start from zero, and acc += (s_x s_w) * sum is one fused
// multiply-add per output and block.  E8M0 scales with bf16 outputs: the instruction's own
// scale operands apply both scales and the accumulators run through.
#include "w4a4_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));

// How a tile computes: FP8 MFMA and scaling after each block, FP8 MFMA with scale operands,
// or bf16 MFMA on widened codes and scaling after each block.
constexpr int MUL_FP8 = 0, MUL_FP8_E8M0 = 1, MUL_BF16 = 2;

__device__ __forceinline__ v8i join(const uint4& a, const uint4& b) {
    return v8i{(int)a.x, (int)a.y, (int)a.z, (int)a.w, (int)b.x, (int)b.y, (int)b.z, (int)b.w};
}

// Linear tile id -> (token tile, feature tile).  Workgroups go to the 8 XCDs in turn, each
// with an L2 of its own: ids that share an XCD get a contiguous range of tiles, ordered in
// groups of GROUP_M token panels, so that they share operand panels in that L2.
// 32-bit arithmetic: the launcher keeps the tile count below 2^31.
constexpr int XCDS = 8;
template <int GROUP_M>
__device__ __forceinline__ void tile_at(uint32_t bid, uint32_t nt_m, uint32_t nt_n, uint32_t& tm, uint32_t& tn) {
    const uint32_t total = nt_m * nt_n;
    const uint32_t q = total / XCDS, r = total % XCDS;
    const uint32_t x = bid % XCDS, j = bid / XCDS;
    const uint32_t id = (x < r ? x * (q + 1) : r * (q + 1) + (x - r) * q) + j;
    const uint32_t per_group = GROUP_M * nt_n;
    const uint32_t g = id / per_group;
    const uint32_t first_m = g * GROUP_M;
    const uint32_t gsize = nt_m - first_m < (uint32_t)GROUP_M ? nt_m - first_m : (uint32_t)GROUP_M;
    const uint32_t in_g = id - g * per_group;
    tn = in_g / gsize;
    tm = first_m + (in_g - tn * gsize);
}

// ---------------------------------------------------------------- many tokens
//
// A workgroup of WT x WF wavefronts owns (WT FT 32) tokens x (WF FF 32) features, a
// wavefront FT x FF tiles of 32 x 32.  The K loop walks blocks of 128 inputs through
// two LDS slots filled by global -> LDS copies: block b + 1 arrives while b is computed.
template <int FT, int FF, int WT, int WF, int MUL, int OUT>
__global__ __launch_bounds__(WT * WF * 64, 1) void fp8_gemm_kernel(
    const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T, int64_t t_ld, const uint8_t* __restrict__ Bq,
    const float* __restrict__ Bs, int64_t N, int64_t nkb64, void* __restrict__ out, int vec_store) {
    constexpr int BT = WT * FT * 32, BF = WF * FF * 32, NW = WT * WF;
    constexpr int NFB = (BF + 127) / 128;                 // weight scale blocks across the tile
    constexpr int PIECES = (BT + BF) / 32 * 4;            // 1 KiB copies per block
    constexpr int B_OFF = BT * 128, AS_OFF = (BT + BF) * 128, BS_OFF = AS_OFF + BT * 4;
    constexpr int SLOT = BS_OFF + NFB * 256;
    static_assert(PIECES % NW == 0 && BT / 64 + NFB <= NW && 32 * 128 * NW <= 2 * SLOT, "tile geometry");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * SLOT];

    const int tid = threadIdx.x, lane = tid & 63;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = wave % WT, wf = wave / WT, l32 = lane & 31, lh = lane >> 5;
    const int nkb = (int)nkb64;
    uint32_t tm, tn;
    tile_at<4>(blockIdx.x, (uint32_t)((T + BT - 1) / BT), (uint32_t)((N + BF - 1) / BF), tm, tn);
    const int64_t t0 = (int64_t)tm * BT, f0 = (int64_t)tn * BF;
    const int64_t rows_a = T - t0 < BT ? T - t0 : BT, rows_b = N - f0 < BF ? N - f0 : BF;
    const int64_t blk = nkb64 * 2048;                     // bytes of 16 rows
    const v4i srd_a = make_srd(Aq + t0 / 16 * blk, (uint32_t)((rows_a + 15) / 16 * blk));
    const v4i srd_b = make_srd(Bq + f0 / 16 * blk, (uint32_t)((rows_b + 15) / 16 * blk));
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    // copy the operands and scales of block kb into slot kb & 1
    auto issue = [&](int kb) __attribute__((always_inline)) {
        const uint32_t slot = lds0 + (uint32_t)(kb & 1) * SLOT;
#pragma unroll
        for (int i = 0; i < PIECES / NW; ++i) {
            const int q = wave * (PIECES / NW) + i;       // wave-uniform
            const int rb = q >> 1, sub = q & 1;
            const bool is_a = rb < BT / 16;
            const int r = is_a ? rb : rb - BT / 16;
            dma16(is_a ? srd_a : srd_b, slot + q * 1024, (int)(r * blk) + sub * 1024 + lane * 16, kb * 2048);
        }
        if (wave < BT / 64) {
            dma4(make_srd(As + (int64_t)kb * t_ld + t0, (uint32_t)(rows_a * 4)), slot + AS_OFF + wave * 256,
                 wave * 256 + lane * 4, 0);
        } else if (wave < BT / 64 + NFB) {
            const int fb = wave - BT / 64;
            const bool in = fb * 128 < rows_b;
            dma4(make_srd(Bs + (in ? (f0 / 128 + fb) * nkb64 : 0) + kb, in ? 4u : 0u), slot + BS_OFF + fb * 256, 0, 0);
        }
    };

    v16f acc[FF][FT];
#pragma unroll
    for (int i = 0; i < FF; ++i)
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.f;

    issue(0);
    for (int kb = 0; kb < nkb; ++kb) {
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        __syncthreads();
        if (kb + 1 < nkb) issue(kb + 1);
        const uint8_t* slot = smem + (kb & 1) * SLOT;
        auto frag = [&](int off, int rb, int half) __attribute__((always_inline)) {
            const uint8_t* p = slot + off + (rb * 2 + (l32 >> 4)) * 2048 + half * 512 + lh * 256 + (lane & 15) * 16;
            return join(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024));
        };
        v8i b[FF][2];
#pragma unroll
        for (int i = 0; i < FF; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[i][h] = frag(B_OFF, wf * FF + i, h);
        const float sb = *reinterpret_cast<const float*>(slot + BS_OFF + (wf * FF * 32 / 128) * 256 + lane * 4);
        static_assert(FF * 32 <= 128 && 128 % (FF * 32) == 0, "one weight scale per wavefront");
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            const v8i a0 = frag(0, wt * FT + j, 0), a1 = frag(0, wt * FT + j, 1);
            const float sa = *reinterpret_cast<const float*>(slot + AS_OFF + ((wt * FT + j) * 32 + l32) * 4);
            if constexpr (MUL != MUL_FP8_E8M0) {
                const float s = sa * sb;
#pragma unroll
                for (int i = 0; i < FF; ++i) {
                    v16f t = v16f{};
                    if constexpr (MUL == MUL_FP8) {
                        t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[i][0], a0, t, 0, 0, 0, 0, 0, 0);
                        t = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[i][1], a1, t, 0, 0, 0, 0, 0, 0);
                    } else {
                        // a lane's 32 inputs in four steps of 8: any order of inputs, the same on both sides
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int q = 0; q < 4; ++q)
                                t = __builtin_amdgcn_mfma_f32_32x32x16_bf16(widen_e4m3(b[i][h][2 * q], b[i][h][2 * q + 1]),
                                                                            h ? widen_e4m3(a1[2 * q], a1[2 * q + 1])
                                                                              : widen_e4m3(a0[2 * q], a0[2 * q + 1]), t, 0, 0, 0);
                    }
#pragma unroll
                    for (int r = 0; r < 16; ++r) acc[i][j][r] = __builtin_fmaf(t[r], s, acc[i][j][r]);
                }
            } else {
                // exponent field of a power of two; a NaN scale gives 0xFF, the E8M0 NaN
                const int ea = (int)((__float_as_uint(sa) >> 23) & 0xFFu), eb = (int)((__float_as_uint(sb) >> 23) & 0xFFu);
#pragma unroll
                for (int i = 0; i < FF; ++i) {
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[i][0], a0, acc[i][j], 0, 0, 0, eb, 0, ea);
                    acc[i][j] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(b[i][1], a1, acc[i][j], 0, 0, 0, eb, 0, ea);
                }
            }
        }
    }
    __syncthreads();   // the slots are free: each wavefront stages its tiles through 4 KiB of its own

    // Lane l holds token l32 and features 8q + 4 lh + e of each tile; tiles are restaged
    // so that stores write whole 128-byte lines (16-byte chunk c of row r at c ^ (r % 8)).
    uint8_t* const stage = smem + wave * 4096;
    const int rr = lane >> 3, cc = lane & 7;
    if constexpr (OUT == W4A4_Y_F32) {
        float* const Y = reinterpret_cast<float*>(out);
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < FF; ++i) {
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    *reinterpret_cast<v4f*>(stage + l32 * 128 + (((2 * q + lh) ^ (l32 & 7)) << 4)) =
                        v4f{acc[i][j][4 * q], acc[i][j][4 * q + 1], acc[i][j][4 * q + 2], acc[i][j][4 * q + 3]};
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = rr + 8 * k;
                    const v4f v = *reinterpret_cast<const v4f*>(stage + r * 128 + ((cc ^ (r & 7)) << 4));
                    const int64_t t = t0 + (wt * FT + j) * 32 + r, n = f0 + (wf * FF + i) * 32 + cc * 4;
                    if (t >= T) continue;
                    if (vec_store && n + 3 < N) {
                        __builtin_nontemporal_store(v, reinterpret_cast<v4f*>(Y + t * N + n));
                    } else {
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            if (n + e < N) Y[t * N + n + e] = v[e];
                    }
                }
            }
    } else {
        static_assert(FF % 2 == 0, "bf16 staging takes two feature tiles");
        uint16_t* const Y = reinterpret_cast<uint16_t*>(out);
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int ip = 0; ip < FF; ip += 2) {
#pragma unroll
                for (int i = 0; i < 2; ++i)
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        *reinterpret_cast<uint2*>(stage + l32 * 128 + (((4 * i + q) ^ (l32 & 7)) << 4) + lh * 8) =
                            make_uint2(pk_bf16(acc[ip + i][j][4 * q], acc[ip + i][j][4 * q + 1]),
                                       pk_bf16(acc[ip + i][j][4 * q + 2], acc[ip + i][j][4 * q + 3]));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int r = rr + 8 * k;
                    const v4i v = *reinterpret_cast<const v4i*>(stage + r * 128 + ((cc ^ (r & 7)) << 4));
                    const int64_t t = t0 + (wt * FT + j) * 32 + r, n = f0 + (wf * FF + ip) * 32 + cc * 8;
                    if (t >= T) continue;
                    if (vec_store && n + 7 < N) {
                        __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(Y + t * N + n));
                    } else {
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            if (n + e < N) Y[t * N + n + e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                    }
                }
            }
    }
}

// ---------------------------------------------------------------- few tokens
//
// Bound by reading the weight codes once.  A workgroup owns 16 weight rows; its eight
// wavefronts take every eighth block of 128 inputs, read codes straight from memory, widen them to bf16 and multiply
// them with up to NT tiles of 16 tokens by v_mfma_f32_16x16x32_bf16; the eight partial sums
// meet in LDS and are added in wavefront order.
template <int NT, int OUT>
__global__ __launch_bounds__(512) void fp8_gemv_kernel(const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T,
                                                       int64_t t_ld, const uint8_t* __restrict__ Bq,
                                                       const float* __restrict__ Bs, int64_t N, int64_t nkb,
                                                       void* __restrict__ out, int vec_store) {
    constexpr int LD = 20;                                 // staged row stride in floats
    __shared__ __attribute__((aligned(16))) float red[8 * NT * 16 * LD];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * 16;
    const int64_t blk = nkb * 2048;
    const uint8_t* const bp = Bq + blockIdx.x * blk + lane * 16;
    const float* const sp = Bs + n0 / 128 * nkb;
    const uint8_t* ap[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) ap[i] = Aq + (i * 16 < T ? i : 0) * blk + lane * 16;

    v4f acc[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) acc[i] = v4f{0, 0, 0, 0};
    for (int64_t kb = wave; kb < nkb; kb += 8) {
        const uint8_t* const p = bp + kb * 2048;
        const v8i b = join(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024));
        const float sb = sp[kb];
        v8bf wb[4];
#pragma unroll
        for (int q = 0; q < 4; ++q) wb[q] = widen_e4m3(b[2 * q], b[2 * q + 1]);
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint8_t* const x = ap[i] + kb * 2048;
            const v8i a = join(*reinterpret_cast<const uint4*>(x), *reinterpret_cast<const uint4*>(x + 1024));
            const float s = As[kb * t_ld + i * 16 + r] * sb;
            v4f t = v4f{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q)
                t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[q], widen_e4m3(a[2 * q], a[2 * q + 1]), t, 0, 0, 0);
#pragma unroll
            for (int e = 0; e < 4; ++e) acc[i][e] = __builtin_fmaf(t[e], s, acc[i][e]);
        }
    }
    // lane: token r of tile i, rows 4 g .. 4 g + 3
#pragma unroll
    for (int i = 0; i < NT; ++i)
        *reinterpret_cast<v4f*>(red + (wave * NT * 16 + i * 16 + r) * LD + 4 * g) = acc[i];
    __syncthreads();
    if (tid >= NT * 64) return;
    const int tok = tid >> 2, c = tid & 3;
    v4f y = v4f{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 8; ++w) {
        const v4f v = *reinterpret_cast<const v4f*>(red + (w * NT * 16 + tok) * LD + 4 * c);
#pragma unroll
        for (int e = 0; e < 4; ++e) y[e] += v[e];
    }
    if (tok >= T) return;
    const int64_t n = n0 + 4 * c;
    if constexpr (OUT == W4A4_Y_F32) {
        float* const Y = reinterpret_cast<float*>(out) + (int64_t)tok * N + n;
        if (vec_store && n + 3 < N) {
            *reinterpret_cast<v4f*>(Y) = y;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) Y[e] = y[e];
        }
    } else {
        uint16_t* const Y = reinterpret_cast<uint16_t*>(out) + (int64_t)tok * N + n;
        const uint32_t lo = pk_bf16(y[0], y[1]), hi = pk_bf16(y[2], y[3]);
        if (vec_store && n + 3 < N) {
            *reinterpret_cast<uint2*>(Y) = make_uint2(lo, hi);
        } else {
            const uint32_t w[2] = {lo, hi};
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) Y[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
    }
}

template <int FT, int FF, int WT, int WF, int MUL, int OUT>
hipError_t run_tiles(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                     hipStream_t st) {
    constexpr int BT = WT * FT * 32, BF = WF * FF * 32;
    const int64_t tiles = ((T + BT - 1) / BT) * ((d.d_out + BF - 1) / BF);
    hipLaunchKernelGGL((fp8_gemm_kernel<FT, FF, WT, WF, MUL, OUT>), dim3((uint32_t)tiles), dim3(WT * WF * 64), 0, st, aq, as, T,
                       t_ld, d.codes, d.scales, d.d_out, d.k_pad / 128, out, d.d_out % (OUT == W4A4_Y_F32 ? 4 : 8) == 0 ? 1 : 0);
    return hipGetLastError();
}

template <int MUL, int OUT>
hipError_t run_many(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                    hipStream_t st) {
    if (((T + 255) / 256) * ((d.d_out + 255) / 256) >= 192)
        return run_tiles<4, 2, 2, 4, MUL, OUT>(aq, as, T, t_ld, d, out, st);
    return run_tiles<2, 2, 2, 2, MUL, OUT>(aq, as, T, t_ld, d, out, st);
}

template <int NT, int OUT>
hipError_t run_few(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                   hipStream_t st) {
    hipLaunchKernelGGL((fp8_gemv_kernel<NT, OUT>), dim3((uint32_t)((d.d_out + 15) / 16)), dim3(512), 0, st, aq, as, T, t_ld,
                       d.codes, d.scales, d.d_out, d.k_pad / 128, out, d.d_out % 4 == 0 ? 1 : 0);
    return hipGetLastError();
}

template <int OUT>
hipError_t run_out(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                   hipStream_t st) {
    if (T <= 16) return run_few<1, OUT>(aq, as, T, t_ld, d, out, st);
    if (T <= 32) return run_few<2, OUT>(aq, as, T, t_ld, d, out, st);
    if (T <= 64) return run_few<4, OUT>(aq, as, T, t_ld, d, out, st);
    if constexpr (OUT == W4A4_Y_F32) return run_many<MUL_BF16, OUT>(aq, as, T, t_ld, d, out, st);
    else if (d.scale_kind == W4A4_FP8_SCALE_F32) return run_many<MUL_FP8, OUT>(aq, as, T, t_ld, d, out, st);
    else return run_many<MUL_FP8_E8M0, OUT>(aq, as, T, t_ld, d, out, st);
}

}  // namespace

hipError_t launch_fp8_gemm(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                           int y_dtype, hipStream_t st) {
    return y_dtype == W4A4_Y_F32 ? run_out<W4A4_Y_F32>(aq, as, T, t_ld, d, out, st)
                                 : run_out<W4A4_Y_BF16>(aq, as, T, t_ld, d, out, st);
}

}  // namespace w4a4

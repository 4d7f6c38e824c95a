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
// range, and copies to LDS and fragment reads are linear.
//
// Precision.  The FP8 matrix instructions (all of them, whatever their shape) line the
// products of a few inputs up with the largest one and drop what falls about 13 bits below
// it: on Gaussian codes a block's sum is off by 1.4e-5 of its norm, with one heavy input by
// 4e-5 (measured against exact sums).  For bf16 outputs that is a fiftieth of the final
// rounding and the FP8 instructions run: 1 to 3% of the outputs round to a neighbour of the bf16
// number nearest to the exact sum, no more where E8M0's accumulators run through 108 blocks.  fp32 outputs, and few tokens (where the arithmetic
// is free), take the codes widened to bf16, which is exact: bf16 products are exact in
// binary32 and their sums are off by 1e-8.
//
// Scales.  The MFMAs of a block start from zero, and acc += (s_x s_w) * sum is one fused
// multiply-add per output and block.  E8M0 scales with bf16 outputs: the instruction's own
// scale operands apply both scales and the accumulators run through.
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef float v4f __attribute__((ext_vector_type(4)));

// How a tile computes: FP8 MFMA and scaling after each block, FP8 MFMA with scale operands,
// or bf16 MFMA on widened codes and scaling after each block.
constexpr int MUL_FP8 = 0, MUL_FP8_E8M0 = 1, MUL_BF16 = 2;

// Whether the few-token kernel runs: up to 64 tokens, and small layers, whose tiles would fill few
// CUs for many latencies (256 x 512 -> 1024: 9.9 us in tiles, 4.0 here; whole calls, tiles against
// this kernel: 333 x 4999 -> 1111 21.9 and 18.7, 512 x 2048 -> 2048 18.7 and 16.2, 256 x 5120 -> 3000 24.6 and 22.0;
// even at 256 x 2048 -> 8192, 24.2 and 24.0).  Short inputs leave more to the writes: 1000 x 512 -> 4096 15.9 and 25.2.
bool fp8_few(int64_t T, int64_t N, int64_t k_pad) {
    return T <= 64 || (T <= 1024 && (T + 63) / 64 * ((N + 15) / 16) * (k_pad / 128) <= (k_pad < 1024 ? 8192 : 32768));
}

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

// The outputs of a wavefront's FT x FF tiles, the first at token t0 and feature f0, through 4 KiB of
// LDS of its own.
template <int FT, int FF, int OUT>
__device__ __forceinline__ void store_tiles(const v4f (&acc)[FT][FF], uint8_t* stage, int64_t t0, int64_t f0, int64_t T,
                                            int64_t N, void* __restrict__ out, int vec_store) {
    // Lane l holds token l % 16 and features 4 (l / 16) .. + 3 of each tile; 32 tokens are
    // restaged so that stores write whole 128-byte lines (16-byte chunk c of row r at c ^ (r % 8)).
    const int lane = threadIdx.x & 63, r16 = lane & 15, g = lane >> 4;
    const int rr = lane >> 3, cc = lane & 7;
#pragma unroll
    for (int j = 0; j < FT; j += 2) {
        constexpr int FP = OUT == W4A4_Y_F32 ? 2 : 4;      // feature tiles of a 128-byte row
#pragma unroll
        for (int ip = 0; ip < FF; ip += FP) {
#pragma unroll
            for (int h = 0; h < 2; ++h)
#pragma unroll
                for (int i = 0; i < FP; ++i) {
                    const v4f v = acc[j + h][ip + i];
                    uint8_t* const row = stage + (h * 16 + r16) * 128;
                    if constexpr (OUT == W4A4_Y_F32)
                        *reinterpret_cast<v4f*>(row + (((i * 4 + g) ^ (r16 & 7)) << 4)) = v;
                    else
                        *reinterpret_cast<uint2*>(row + (((i * 2 + (g >> 1)) ^ (r16 & 7)) << 4) + (g & 1) * 8) =
                            make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]));
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int r = rr + 8 * k;
                const v4i v = *reinterpret_cast<const v4i*>(stage + r * 128 + ((cc ^ (r & 7)) << 4));
                constexpr int EL = OUT == W4A4_Y_F32 ? 4 : 8;
                const int64_t tt = t0 + j * 16 + r, n = f0 + ip * 16 + cc * EL;
                if (tt >= T) continue;
                if (vec_store && n + EL - 1 < N) {
                    __builtin_nontemporal_store(v, reinterpret_cast<v4i*>(reinterpret_cast<uint8_t*>(out) + (tt * N + n) * (16 / EL)));
                } else {
#pragma unroll
                    for (int e = 0; e < EL; ++e) {
                        if (n + e >= N) continue;
                        if constexpr (OUT == W4A4_Y_F32) reinterpret_cast<int*>(out)[tt * N + n + e] = v[e];
                        else reinterpret_cast<uint16_t*>(out)[tt * N + n + e] = (uint16_t)((uint32_t)v[e / 2] >> (16 * (e & 1)));
                    }
                }
            }
        }
    }
}

// A workgroup of WT x WF wavefronts owns (WT FT 16) tokens x (WF FF 16) features, a
// wavefront FT x FF tiles of 16 x 16: with the 16-row instructions a block's sum takes four
// registers until it is scaled, with the 32-row ones sixteen, which do not fit beside the
// accumulators and the fragments.  The K loop walks blocks of 128 inputs through two LDS
// slots filled by global -> LDS copies.  A wavefront has read all of a slot when it starts
// its last token tile of the block; the block's one barrier sits there: behind it the slot's
// refill (block b + 2) is issued, and the next block's first fragments are read from the
// other slot while the last tiles' MFMAs run.  A tile is scaled LAG tiles later, across
// block boundaries too, so that nothing waits for an MFMA's result.
//
// Tiles that would leave most CUs idle in a last round run as sp.n ranges of their blocks, whose
// sums go to memory; fp8_reduce_kernel adds them in order.
//
// Measured (this kernel alone, traced, clocks settled: the first twenty calls after a pause take a tenth
// longer): 57600 x 5120 -> 13824, bf16 outputs, 3.39 ms (2.40 PFLOP/s; the library's product with one
// scale for each whole operand takes 2.75).  What shares a CU's LDS bounds it: the same loop took 2.7 ms of
// 3.4 without the copies into LDS, 2.1 without the fragment reads, 3.25 with a quarter of the scaling.
// A second barrier and the copies in two halves changed nothing (0.5%).  E8M0 scales in the
// instruction: 4096 x 13824 -> 5120 in 216 us (library 210).  fp32 outputs: 4096 x 5120 -> 13824 in
// 457 us, 1.27 PFLOP/s, which is what the 16-row bf16 instruction gives alone (1.3; the 32-row form gives 2.3,
// the library's bf16 product 1.24).  Registers: 222 with fp32 scales, 201 with E8M0; 256 and 12
// bytes of scratch a lane with fp32 outputs.
struct Split {
    float* part;
    uint32_t full, n;
};
template <int FT, int FF, int WT, int WF, int MUL, int OUT>
__global__ __launch_bounds__(WT * WF * 64, 1) void fp8_gemm_kernel(
    const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T, int64_t t_ld, const uint8_t* __restrict__ Bq,
    const float* __restrict__ Bs, int64_t N, int64_t nkb64, void* __restrict__ out, int vec_store, Split sp) {
    constexpr int BT = WT * FT * 16, BF = WF * FF * 16, NW = WT * WF, NT = FT * FF, LAG = 3;
    constexpr int NFB = (BF + 127) / 128;                 // weight scale blocks across the tile
    constexpr int PIECES = (BT + BF) / 16 * 2;            // 1 KiB copies per block
    constexpr int B_OFF = BT * 128, AS_OFF = (BT + BF) * 128, BS_OFF = AS_OFF + BT * 4;
    constexpr int SLOT = BS_OFF + NFB * 256;
    static_assert(PIECES % NW == 0 && BT / 64 + NFB <= NW && 32 * 128 * NW <= 2 * SLOT, "tile geometry");
    static_assert(FT % 2 == 0 && NT % 4 == 0 && FF == 4, "buffers by parity; 64 features a wavefront");
    // the slots, then 256 bytes that wavefronts without scales to copy fill with zeros
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * SLOT + 256];

    const int tid = threadIdx.x, lane = tid & 63, r16 = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wt = wave % WT, wf = wave / WT;
    // a whole tile, or one of sp.n ranges of a later tile's blocks
    const uint32_t late = blockIdx.x < sp.full ? 0 : blockIdx.x - sp.full;
    const uint32_t id = blockIdx.x < sp.full ? blockIdx.x : sp.full + late / sp.n;
    const int part = blockIdx.x < sp.full ? 0 : (int)(late % sp.n), parts = blockIdx.x < sp.full ? 1 : (int)sp.n;
    const int kb0 = (int)(nkb64 * part / parts), nkb = (int)(nkb64 * (part + 1) / parts) - kb0;
    uint32_t tm, tn;
    tile_at<4>(id, (uint32_t)((T + BT - 1) / BT), (uint32_t)((N + BF - 1) / BF), tm, tn);
    const int64_t t0 = (int64_t)tm * BT, f0 = (int64_t)tn * BF;
    const int64_t rows_a = T - t0 < BT ? T - t0 : BT, rows_b = N - f0 < BF ? N - f0 : BF;
    const int64_t blk = nkb64 * 2048;                     // bytes of 16 rows
    // (a range's first block goes into the bases; a row block then still passes the range check
    // exactly when it is valid, as kb0 * 2048 is less than one row block)
    const v4i srd_a = make_srd(Aq + t0 / 16 * blk + kb0 * 2048, (uint32_t)((rows_a + 15) / 16 * blk - kb0 * 2048));
    const v4i srd_b = make_srd(Bq + f0 / 16 * blk + kb0 * 2048, (uint32_t)((rows_b + 15) / 16 * blk - kb0 * 2048));
    const uint32_t lds0 = (uint32_t)(uintptr_t)smem;

    // What this wavefront copies of a block's scales: 64 tokens', or one 128-feature block's (the same
    // word into 64 places), or nothing.
    const bool sc_a = wave < BT / 64, sc_b = !sc_a && wave < BT / 64 + NFB && (wave - BT / 64) * 128 < rows_b;
    const float* const sc_p = sc_a ? As + (int64_t)kb0 * t_ld + t0 : Bs + (sc_b ? (f0 / 128 + wave - BT / 64) * nkb64 + kb0 : 0);
    const int64_t sc_step = sc_a ? t_ld : sc_b ? 1 : 0;
    const uint32_t sc_bytes = sc_a ? (uint32_t)(rows_a * 4) : sc_b ? 4u : 0u;
    const int sc_off = sc_a ? wave * 256 + lane * 4 : 0;
    // Copy the operands and scales of block kb into slot kb & 1.  Past the last block the same
    // copies run with empty ranges (they write zeros): without branches, every wait below counts the
    // same number of copies, and the compiler cannot move the tiles' arithmetic past one.
    constexpr int COPIES = PIECES / NW + 1;
    auto issue = [&](int kb) __attribute__((always_inline)) {
        const bool on = kb < nkb;
        const uint32_t slot = lds0 + (uint32_t)(kb & 1) * SLOT;
        v4i a = srd_a, b = srd_b;
        a[2] = on ? a[2] : 0;
        b[2] = on ? b[2] : 0;
#pragma unroll
        for (int i = 0; i < PIECES / NW; ++i) {
            constexpr int PA = BT / 16 * 2 / NW, PB = BF / 16 * 2 / NW;   // pieces of each operand a wavefront copies
            static_assert(PA * NW == BT / 8 && PB * NW == BF / 8, "pieces divide evenly");
            const bool is_a = i < PA;
            const int q = is_a ? wave * PA + i : wave * PB + i - PA;      // wave-uniform
            dma16(is_a ? a : b, slot + (is_a ? 0 : B_OFF) + q * 1024, (int)((q >> 1) * blk) + (q & 1) * 1024 + lane * 16, kb * 2048);
        }
        dma4(make_srd(sc_p + (on ? kb : 0) * sc_step, on ? sc_bytes : 0u),
             sc_a ? slot + AS_OFF + wave * 256 : sc_b ? slot + BS_OFF + (wave - BT / 64) * 256 : lds0 + 2 * SLOT, sc_off, 0);
    };

    v4f acc[FT][FF];
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int i = 0; i < FF; ++i) acc[j][i] = v4f{0, 0, 0, 0};
    v8i fb[FF], fa[2];             // weight fragments; token fragments of tiles j, j + 1
    float sa[2], sb = 0.f;
    const uint8_t* const pa = smem + wt * FT * 2048 + lane * 16;
    const uint8_t* const pb = smem + B_OFF + wf * FF * 2048 + lane * 16;
    const uint8_t* const ps = smem + AS_OFF + (wt * FT * 16 + r16) * 4;
    const uint8_t* const pw = smem + BS_OFF + (wf * FF * 16 / 128) * 256 + lane * 4;
    auto frag = [&](const uint8_t* p) __attribute__((always_inline)) {
        return join(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024));
    };
    auto load_a = [&](int slot, int j) __attribute__((always_inline)) {
        fa[j & 1] = frag(pa + slot * SLOT + j * 2048);
        sa[j & 1] = *reinterpret_cast<const float*>(ps + slot * SLOT + j * 64);
    };
    auto load_b = [&](int slot, int i) __attribute__((always_inline)) {
        fb[i] = frag(pb + slot * SLOT + i * 2048);
        if (i == FF - 1) sb = *reinterpret_cast<const float*>(pw + slot * SLOT);
    };
    v4f t[4];                      // sums of the last tiles
    float st[2] = {0.f, 0.f};      // scales of the current and the last token tile
#pragma unroll
    for (int i = 0; i < 4; ++i) t[i] = v4f{0, 0, 0, 0};
    auto scale = [&](int n) __attribute__((always_inline)) {   // the tile LAG tiles before tile n
        if constexpr (MUL != MUL_FP8_E8M0) {
            const int q = (n + NT - LAG) % NT;
#pragma unroll
            for (int r = 0; r < 4; ++r)
                acc[q / FF][q % FF][r] = __builtin_fmaf(t[q & 3][r], st[(q / FF) & 1], acc[q / FF][q % FF][r]);
        }
    };

    issue(0);
    issue(1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(COPIES) : "memory");   // block 0 is there
    __syncthreads();
    load_a(0, 0);
#pragma unroll
    for (int i = 0; i < FF; ++i) load_b(0, i);
    for (int kb = 0; kb < nkb; ++kb) {
        const int slot = kb & 1;
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            if (j + 1 < FT) {
                load_a(slot, j + 1);
            } else {
                // every read of this slot is in registers; the other slot's copies have landed
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                issue(kb + 2);
            }
            const int ea = (int)((__float_as_uint(sa[j & 1]) >> 23) & 0xFFu), eb = (int)((__float_as_uint(sb) >> 23) & 0xFFu);
            st[j & 1] = sa[j & 1] * sb;
            v8bf wa[4];
            if constexpr (MUL == MUL_BF16) {
#pragma unroll
                for (int q = 0; q < 4; ++q) wa[q] = widen_e4m3(fa[j & 1][2 * q], fa[j & 1][2 * q + 1]);
            }
#pragma unroll
            for (int i = 0; i < FF; ++i) {
                const int n = j * FF + i;
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (MUL == MUL_FP8) {
                    t[n & 3] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i], fa[j & 1], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
                } else if constexpr (MUL == MUL_FP8_E8M0) {
                    // exponent field of a power of two; a NaN scale gives 0xFF, the E8M0 NaN
                    acc[j][i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[i], fa[j & 1], acc[j][i], 0, 0, 0, eb, 0, ea);
                } else {
                    t[n & 3] = v4f{0, 0, 0, 0};
#pragma unroll
                    for (int q = 0; q < 4; ++q)
                        t[n & 3] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_e4m3(fb[i][2 * q], fb[i][2 * q + 1]), wa[q], t[n & 3], 0, 0, 0);
                }
                __builtin_amdgcn_sched_barrier(0);
                scale(n);
                if (j + 1 == FT) {   // fragments of the next block, as theirs are used up (after the last: not used)
                    if (i == 0) load_a(slot ^ 1, 0);
                    load_b(slot ^ 1, i);
                }
            }
        }
    }
#pragma unroll
    for (int n = 0; n < LAG; ++n) scale(n);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (blockIdx.x >= sp.full) {   // a range's sums as they lie in the registers, 1 KiB a store
        v4f* const p = reinterpret_cast<v4f*>(sp.part) + ((int64_t)late * NW + wave) * NT * 64 + lane;
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < FF; ++i) p[(j * FF + i) * 64] = acc[j][i];
        return;
    }
    __syncthreads();   // the slots are free: each wavefront stages its tiles through 4 KiB of its own

    store_tiles<FT, FF, OUT>(acc, smem + wave * 4096, t0 + wt * FT * 16, f0 + wf * FF * 16, T, N, out, vec_store);
}

// One wavefront per two token tiles x FF of a split tile: its ranges' sums, in order, then the outputs.
template <int FT, int FF, int WT, int WF, int OUT>
__global__ __launch_bounds__(64) void fp8_reduce_kernel(int64_t T, int64_t N, void* __restrict__ out, int vec_store, Split sp) {
    constexpr int BT = WT * FT * 16, BF = WF * FF * 16, NW = WT * WF, NT = FT * FF;
    __shared__ __attribute__((aligned(1024))) uint8_t stage[4096];
    const uint32_t jp = blockIdx.x % (FT / 2) * 2, sub = blockIdx.x / (FT / 2), tile = sub / NW, wave = sub % NW;
    uint32_t tm, tn;
    tile_at<4>(sp.full + tile, (uint32_t)((T + BT - 1) / BT), (uint32_t)((N + BF - 1) / BF), tm, tn);
    const int64_t t0 = (int64_t)tm * BT + (wave % WT * FT + jp) * 16, f0 = (int64_t)tn * BF + wave / WT * FF * 16;
    if (t0 >= T || f0 >= N) return;
    const v4f* p = reinterpret_cast<const v4f*>(sp.part) + (((int64_t)tile * sp.n * NW + wave) * NT + jp * FF) * 64 + threadIdx.x;
    v4f acc[2][FF];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < FF; ++i) acc[j][i] = v4f{0, 0, 0, 0};
    for (uint32_t c = 0; c < sp.n; c += 4) {   // four ranges' loads in flight
        v4f v[4][2][FF];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const v4f* const q = p + (int64_t)(c + u < sp.n ? c + u : c) * NW * NT * 64;
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
                for (int i = 0; i < FF; ++i) v[u][j][i] = q[(j * FF + i) * 64];
        }
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (c + u < sp.n) {
#pragma unroll
                for (int j = 0; j < 2; ++j)
#pragma unroll
                    for (int i = 0; i < FF; ++i)
#pragma unroll
                        for (int r = 0; r < 4; ++r) acc[j][i][r] += v[u][j][i][r];
            }
    }
    store_tiles<2, FF, OUT>(acc, stage, t0, f0, T, N, out, vec_store);
}

// ---------------------------------------------------------------- few tokens
//
// Bound by reading the weight codes once.  A workgroup owns RT tiles of 16 weight rows; its eight
// wavefronts take every eighth block of 128 inputs, read codes straight from memory, widen
// them to bf16 and multiply them with up to NT tiles of 16 tokens by v_mfma_f32_16x16x32_bf16;
// the eight partial sums meet in LDS and are added in wavefront order.
//
// The loop is as simple as it looks on purpose: at 40 registers all 864 workgroups of a 13824-row
// layer are resident and cover each other's waits (one token, 5120 -> 13824: 12.6 us for 71 MB; a
// kernel that only reads as much takes 14.4 from memory).  A ring of
// blocks in flight per wavefront with the registers that it takes was slower (16.8), so was
// quantizing the token in the same kernel (17.9, against 3.3 more for the quantization's launch),
// and non-temporal loads lose a layer that stays in the 256 MB memory-side cache (24 tokens,
// 13824 -> 5120: 29 against 19 us).
//
// With several token tiles the vector memory path, not the memory, is what the reads of both operands
// wait for: two row tiles use a token fragment once more, and the inputs split over gridDim.z
// workgroups keep the CUs evenly filled.  Both pay from a layer that the L2s do not hold on
// (24 tokens, 13824 -> 5120: 22.8 to 20.4 us a call, 64 tokens 32.5 to 25.6; but 32 tokens, 5120 -> 5120:
// 12.7 to 14.5).  One row tile splits only where few workgroups would walk far (one token, 13824 ->
// 5120, split in 3: 18.4 to 19.8 us; 32768 -> 512, in 8: 20.1 to 15.0).
template <int NT, int RT, int OUT>
__global__ __launch_bounds__(512, RT == 1 ? 1 : NT == 2 ? 4 : 2) void fp8_gemv_kernel(const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T,
                                                       int64_t t_ld, const uint8_t* __restrict__ Bq,
                                                       const float* __restrict__ Bs, int64_t N, int64_t nkb,
                                                       void* __restrict__ out, int vec_store, float* __restrict__ part,
                                                       int32_t* __restrict__ count) {
    constexpr int LD = 20;                                 // staged row stride in floats
    __shared__ __attribute__((aligned(16))) float red[8 * RT * NT * 16 * LD];
    __shared__ int done;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * RT * 16, t0 = (int64_t)blockIdx.y * NT * 16;
    const int64_t blk = nkb * 2048;
    const uint8_t* bp[RT];
#pragma unroll
    for (int m = 0; m < RT; ++m) bp[m] = Bq + (n0 + m * 16 < N ? n0 + m * 16 : n0) / 16 * blk + lane * 16;
    const float* const sp = Bs + n0 / 128 * nkb;
    const uint8_t* ap[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) ap[i] = Aq + (t0 + i * 16 < T ? t0 + i * 16 : t0) / 16 * blk + lane * 16;

    v4f acc[RT][NT];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i] = v4f{0, 0, 0, 0};
    const int kb1 = (int)(nkb * (blockIdx.z + 1) / gridDim.z);
    for (int kb = (int)(nkb * blockIdx.z / gridDim.z) + wave; kb < kb1; kb += 8) {
        const float sb = sp[kb];
        v8bf wb[RT][4];
#pragma unroll
        for (int m = 0; m < RT; ++m) {
            const uint8_t* const p = bp[m] + kb * 2048;
            const v8i b = join(*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024));
#pragma unroll
            for (int q = 0; q < 4; ++q) wb[m][q] = widen_e4m3(b[2 * q], b[2 * q + 1]);
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            const uint8_t* const x = ap[i] + kb * 2048;
            const v8i a = join(*reinterpret_cast<const uint4*>(x), *reinterpret_cast<const uint4*>(x + 1024));
            const float s = As[kb * t_ld + min(t0 + i * 16 + r, t_ld - 1)] * sb;
            v4f t[RT];
#pragma unroll
            for (int m = 0; m < RT; ++m) t[m] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v8bf wa = widen_e4m3(a[2 * q], a[2 * q + 1]);
#pragma unroll
                for (int m = 0; m < RT; ++m) t[m] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(wb[m][q], wa, t[m], 0, 0, 0);
            }
#pragma unroll
            for (int m = 0; m < RT; ++m)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[m][i][e] = __builtin_fmaf(t[m][e], s, acc[m][i][e]);
        }
    }
    // lane: token r of tile i, rows 4 g .. 4 g + 3
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
            *reinterpret_cast<v4f*>(red + (((wave * RT + m) * NT + i) * 16 + r) * LD + 4 * g) = acc[m][i];
    __syncthreads();
    const int c = tid & 3, m = RT == 2 ? tid / (NT * 64) & 1 : 0;
    const int64_t tok = t0 + tid % (NT * 64) / 4;
    v4f y = v4f{0, 0, 0, 0};
    if (tid < RT * NT * 64)
#pragma unroll
        for (int w = 0; w < 8; ++w) {
            const v4f v = *reinterpret_cast<const v4f*>(red + (w * RT * NT * 16 + (tid >> 2)) * LD + 4 * c);
#pragma unroll
            for (int e = 0; e < 4; ++e) y[e] += v[e];
        }
    if (gridDim.z > 1) {   // the last of the tile's ranges to be done adds them all, in order
        const uint32_t tile = blockIdx.y * gridDim.x + blockIdx.x, step = gridDim.x * gridDim.y * RT * NT * 256;
        float* const p = part + tile * RT * NT * 256 + tid * 4;
        if (tid < RT * NT * 64)
#pragma unroll
            for (int e = 0; e < 4; ++e) put_shared(p + blockIdx.z * step + e, y[e]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the range is where every XCD sees it
        __syncthreads();
        if (tid == 0) done = __hip_atomic_fetch_add(count + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (done != (int)gridDim.z - 1) return;
        y = v4f{0, 0, 0, 0};
        if (tid < RT * NT * 64)
            for (uint32_t u = 0; u < gridDim.z; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += get_shared(p + u * step + e);
    }
    if (tid >= RT * NT * 64) return;
    if (tok >= T) return;
    const int64_t n = n0 + m * 16 + 4 * c;
    if constexpr (OUT == W4A4_Y_F32) {
        float* const Y = reinterpret_cast<float*>(out) + tok * N + n;
        if (vec_store && n + 3 < N) {
            *reinterpret_cast<v4f*>(Y) = y;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) Y[e] = y[e];
        }
    } else {
        uint16_t* const Y = reinterpret_cast<uint16_t*>(out) + tok * N + n;
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
hipError_t run_tiles(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out, float* part,
                     const Fp8Plan& plan, hipStream_t st) {
    const int vec = d.d_out % (OUT == W4A4_Y_F32 ? 4 : 8) == 0 ? 1 : 0;
    const Split sp = {part, (uint32_t)plan.full, (uint32_t)plan.split};
    const int64_t tail = plan.tiles - plan.full;
    hipLaunchKernelGGL((fp8_gemm_kernel<FT, FF, WT, WF, MUL, OUT>), dim3((uint32_t)(plan.full + tail * plan.split)), dim3(WT * WF * 64),
                       0, st, aq, as, T, t_ld, d.codes, d.scales, d.d_out, d.k_pad / 128, out, vec, sp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !tail) return e;
    hipLaunchKernelGGL((fp8_reduce_kernel<FT, FF, WT, WF, OUT>), dim3((uint32_t)(tail * WT * WF * (FT / 2))), dim3(64), 0, st, T, d.d_out, out,
                       vec, sp);
    return hipGetLastError();
}

template <int MUL, int OUT>
hipError_t run_many(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out, float* part,
                    const Fp8Plan& plan, hipStream_t st) {
    if (plan.big) return run_tiles<8, 4, 2, 4, MUL, OUT>(aq, as, T, t_ld, d, out, part, plan, st);
    return run_tiles<4, 4, 2, 2, MUL, OUT>(aq, as, T, t_ld, d, out, part, plan, st);
}

template <int NT, int RT, int OUT>
hipError_t run_few(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out, float* part,
                   int32_t* count, const Fp8Plan& plan, hipStream_t st) {
    const dim3 grid((uint32_t)((d.d_out + RT * 16 - 1) / (RT * 16)), (uint32_t)((T + NT * 16 - 1) / (NT * 16)), (uint32_t)plan.split);
    hipLaunchKernelGGL((fp8_gemv_kernel<NT, RT, OUT>), grid, dim3(512), 0, st, aq, as, T, t_ld, d.codes, d.scales, d.d_out,
                       d.k_pad / 128, out, d.d_out % 4 == 0 ? 1 : 0, part, count);
    return hipGetLastError();
}

template <int OUT>
hipError_t run_out(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out, float* part,
                   int32_t* count, hipStream_t st) {
    const Fp8Plan plan = fp8_plan(T, d.d_out, d.k_pad);
    if (plan.few && T <= 16) return run_few<1, 1, OUT>(aq, as, T, t_ld, d, out, part, count, plan, st);
    if (plan.few && T <= 32) return plan.rt == 2 ? run_few<2, 2, OUT>(aq, as, T, t_ld, d, out, part, count, plan, st)
                            : run_few<2, 1, OUT>(aq, as, T, t_ld, d, out, part, count, plan, st);
    if (plan.few) return plan.rt == 2 ? run_few<4, 2, OUT>(aq, as, T, t_ld, d, out, part, count, plan, st)
                            : run_few<4, 1, OUT>(aq, as, T, t_ld, d, out, part, count, plan, st);
    if constexpr (OUT == W4A4_Y_F32) return run_many<MUL_BF16, OUT>(aq, as, T, t_ld, d, out, part, plan, st);
    else if (d.scale_kind == W4A4_FP8_SCALE_F32) return run_many<MUL_FP8, OUT>(aq, as, T, t_ld, d, out, part, plan, st);
    else return run_many<MUL_FP8_E8M0, OUT>(aq, as, T, t_ld, d, out, part, plan, st);
}

}  // namespace

// Big tiles are 256 x 256, one workgroup a CU, from 64 of them on (at 54, 128 x 5120 -> 13824, 43 us against
// 34 with small tiles; at 40, 512 x 13824 -> 5120, 64 against 68); small ones 128 x 128, two a CU.  The tiles that fill
// whole rounds of the CUs run whole; the rest are cut along the inputs into as many ranges as there
// are free CUs, at least MIN_BLOCKS blocks each (4096 x 13824 -> 5120, 64 of 320 tiles in four ranges:
// 346 to 286 us).
Fp8Plan fp8_plan(int64_t T, int64_t N, int64_t k_pad) {
    Fp8Plan p = {0, 0, 1, 1, false, false, 0};
    constexpr int64_t CUS = 256, MIN_BLOCKS = 4, MAX_SPLIT = 16, FEW_CODES = 1 << 25;
    const int64_t nkb = k_pad / 128;
    p.few = fp8_few(T, N, k_pad);
    if (T == 0 || N == 0) return p;
    if (p.few) {
        const int64_t nt = T <= 16 ? 1 : T <= 32 ? 2 : 4;   // token tiles of a workgroup
        p.rt = nt > 1 && N * k_pad > FEW_CODES ? 2 : 1;
        p.tiles = ((N + 16 * p.rt - 1) / (16 * p.rt)) * ((T + nt * 16 - 1) / (nt * 16));
        int64_t s = 2 * CUS / p.tiles, least = p.rt == 2 ? 16 : 32;   // ranges; blocks of each
        if (s > nkb / least) s = nkb / least;
        if (s > MAX_SPLIT) s = MAX_SPLIT;
        if (s >= 2) {
            p.split = (int32_t)s;
            p.part_bytes = (size_t)(p.tiles * s * nt * p.rt) * 1024;
        }
        return p;
    }
    const int64_t big = ((T + 255) / 256) * ((N + 255) / 256);
    p.big = big >= 64;
    p.tiles = p.big ? big : ((T + 127) / 128) * ((N + 127) / 128);
    const int64_t round = p.big ? CUS : 2 * CUS, tail = p.tiles % round;
    p.full = p.tiles;
    if (tail) {
        int64_t s = round / tail < MAX_SPLIT ? round / tail : MAX_SPLIT;
        if (s > nkb / MIN_BLOCKS) s = nkb / MIN_BLOCKS;
        if (s >= 2) {
            p.full -= tail;
            p.split = (int32_t)s;
            p.part_bytes = (size_t)(tail * s) * (p.big ? 256 * 256 : 128 * 128) * 4;
        }
    }
    return p;
}

hipError_t launch_fp8_gemm(const uint8_t* aq, const float* as, int64_t T, int64_t t_ld, const w4a4_fp8_packed& d, void* out,
                           int y_dtype, float* part, int32_t* count, hipStream_t st) {
    return y_dtype == W4A4_Y_F32 ? run_out<W4A4_Y_F32>(aq, as, T, t_ld, d, out, part, count, st)
                                 : run_out<W4A4_Y_BF16>(aq, as, T, t_ld, d, out, part, count, st);
}

}  // namespace w4a4

// INT8 product on gfx950:
//
//   Y[t][n] = (s_x[t] s_w[n]) sum_p q_x[t][p] q_w[n][p]
//
// integer codes, exact 32-bit sums, one scaling at the end.  Operand roles as in gemm.hip: src0 =
// weight rows, src1 = token rows, so a lane of the result holds one token and its scale.
//
// Both operands lie in runs of 16 rows x 128 inputs (2 KiB), as in the FP8 layer: 16-byte pieces,
// piece p of row r at 256 p + 16 r.  A 16-row instruction of 64 inputs takes one piece a lane
// (lane 16 g + r: piece 4 h + g), a 32-row one of 32 inputs too (lane 32 h + 16 u + r: row r of run
// u, piece 2 s + h).  Which inputs a piece holds is free, as both operands agree.
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef int v16i __attribute__((ext_vector_type(16)));

// Whether the few-token kernel runs: up to 64 tokens, and layers whose tiles would leave most CUs idle (us a call,
// tiles and this kernel: 333 x 4999 -> 1111 26.6 and 18.4, 256 x 5120 -> 3000 27.5 and 20.9, 1024 x 2048 -> 2048 27.4 and
// 22.0; even at 256 x 5120 -> 5120, 26.3 and 27.1; 512 x 5120 -> 5120 31.3 and 45.5).  Short inputs: 300 x 800 -> 2000 13.6
// and 8.7, 1000 x 512 -> 4096 18.5 and 18.8.
bool int8_few(int64_t T, int64_t N, int64_t k_pad) {
    return T <= 64 || (T <= 1024 && (T + 63) / 64 * ((N + 15) / 16) * (k_pad / 128) <= (k_pad < 1024 ? 16000 : 45000));
}

// Linear tile id -> (token tile, feature tile): ids that share an XCD get a contiguous range of
// tiles, in groups of GROUP_M token panels, so that they share operand panels in its L2.
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

// The outputs of a wavefront's FT x FF tiles of 32 x 32, the first at token t0 and feature f0,
// through 4 KiB of LDS of its own: lane 32 h + r holds token r and features 8 (i / 4) + 4 h + i % 4;
// 32 tokens are restaged so that stores write whole 128-byte lines (16-byte chunk c of row r at c ^ (r % 8)).
template <int FT, int FF, int OUT>
__device__ __forceinline__ void store_tiles(const v16i (&acc)[FT][FF], uint8_t* stage, int64_t t0, int64_t f0, int64_t T, int64_t N,
                                            const float* __restrict__ As, const float* __restrict__ Bs, int64_t n_pad,
                                            void* __restrict__ out, int vec_store) {
    constexpr int FP = OUT == W4A4_Y_F32 ? 1 : 2;      // feature tiles of a 128-byte row
    constexpr int EL = OUT == W4A4_Y_F32 ? 4 : 8;
    static_assert(FF % FP == 0, "whole lines");
    const int lane = threadIdx.x & 63, r = lane & 31, h = lane >> 5;
    const int rr = lane >> 3, cc = lane & 7;
#pragma unroll
    for (int ip = 0; ip < FF; ip += FP) {
        v4f sw[FP][4];
#pragma unroll
        for (int i = 0; i < FP; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const int64_t n = f0 + (ip + i) * 32 + 8 * q + 4 * h;
                sw[i][q] = n < n_pad ? *reinterpret_cast<const v4f*>(Bs + n) : v4f{0, 0, 0, 0};
            }
#pragma unroll
        for (int j = 0; j < FT; ++j) {
            const int64_t t = t0 + j * 32 + r;
            const float sx = t < T ? As[t] : 0.0f;
#pragma unroll
            for (int i = 0; i < FP; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    v4f y;
#pragma unroll
                    for (int e = 0; e < 4; ++e) y[e] = (sx * sw[i][q][e]) * (float)acc[j][ip + i][4 * q + e];
                    uint8_t* const row = stage + r * 128;
                    if constexpr (OUT == W4A4_Y_F32)
                        *reinterpret_cast<v4f*>(row + (((2 * q + h) ^ (r & 7)) << 4)) = y;
                    else
                        *reinterpret_cast<uint2*>(row + (((4 * i + q) ^ (r & 7)) << 4) + h * 8) =
                            make_uint2(pk_bf16(y[0], y[1]), pk_bf16(y[2], y[3]));
                }
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int row = rr + 8 * k;
                const v4i v = *reinterpret_cast<const v4i*>(stage + row * 128 + ((cc ^ (row & 7)) << 4));
                const int64_t tt = t0 + j * 32 + row, n = f0 + ip * 32 + cc * EL;
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

// Bound by the board's power: 57600 x 5120 -> 5120 settles at 1264 us, 2.39 PO/s, with the matrix unit busy in 65% of the
// cycles (1316 on another card, where the library's product of the same size took 1324).  Tiles of 128 x 128 a wavefront, four
// wavefronts a workgroup, have fewer fragment reads and took 1484 there: one wavefront a SIMD does not cover its own waits.
//
// A workgroup of WT x WF wavefronts owns (WT FT 32) tokens x (WF FF 32) features, a wavefront FT x FF
// tiles of 32 x 32 whose sums stay in its accumulators.  The K loop walks blocks of 128 inputs
// through two LDS slots filled by global -> LDS copies, each block as four steps of 32 inputs; a
// step's fragments are read while the step before it multiplies.  The block's one barrier sits
// before its last step, whose fragments are in registers by then: behind it the slot's refill (block b + 2) is
// issued and the next block's first fragments are read from the other slot.
//
// Tiles that would leave most CUs idle in a last round run as sp.n ranges of their blocks, whose
// sums go to memory; int8_reduce_kernel adds them.
struct Split {
    int32_t* part;
    uint32_t full, n;
};
template <int FT, int FF, int WT, int WF, int OUT>
__global__ __launch_bounds__(WT * WF * 64, 1) void int8_gemm_kernel(
    const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T, const uint8_t* __restrict__ Bq,
    const float* __restrict__ Bs, int64_t N, int64_t n_pad, int64_t nkb64, void* __restrict__ out, int vec_store, Split sp) {
    constexpr int BT = WT * FT * 32, BF = WF * FF * 32, NW = WT * WF;
    constexpr int PA = BT / 8 / NW, PB = BF / 8 / NW;     // 1 KiB copies of each operand a wavefront makes per block
    constexpr int B_OFF = BT * 128, SLOT = (BT + BF) * 128;
    static_assert(PA * NW == BT / 8 && PB * NW == BF / 8 && NW * 4096 <= 2 * SLOT, "tile geometry");
    __shared__ __attribute__((aligned(1024))) uint8_t smem[2 * SLOT];

    const int tid = threadIdx.x, lane = tid & 63;
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

    // Copy block kb into slot kb & 1.  Past the last block the same copies run with empty ranges
    // (they write zeros), so that no branch stands in the loop.
    constexpr int COPIES = PA + PB;
    auto issue = [&](int kb) __attribute__((always_inline)) {
        const bool on = kb < nkb;
        const uint32_t slot = lds0 + (uint32_t)(kb & 1) * SLOT;
        v4i a = srd_a, b = srd_b;
        a[2] = on ? a[2] : 0;
        b[2] = on ? b[2] : 0;
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
            const bool is_a = i < PA;
            const int q = is_a ? wave * PA + i : wave * PB + i - PA;      // wave-uniform
            dma16(is_a ? a : b, slot + (is_a ? 0 : B_OFF) + q * 1024, (int)((q >> 1) * blk) + (q & 1) * 1024 + lane * 16, kb * 2048);
        }
    };

    v16i acc[FT][FF];
#pragma unroll
    for (int j = 0; j < FT; ++j)
#pragma unroll
        for (int i = 0; i < FF; ++i)
#pragma unroll
            for (int e = 0; e < 16; ++e) acc[j][i][e] = 0;
    v4i fa[2][FT], fb[2][FF];
    const int in_frag = ((lane >> 4) & 1) * 2048 + (lane >> 5) * 256 + (lane & 15) * 16;
    const uint8_t* const pa = smem + wt * FT * 4096 + in_frag;
    const uint8_t* const pb = smem + B_OFF + wf * FF * 4096 + in_frag;
    auto load = [&](int slot, int s) __attribute__((always_inline)) {
#pragma unroll
        for (int i = 0; i < FF; ++i) fb[s & 1][i] = *reinterpret_cast<const v4i*>(pb + slot * SLOT + i * 4096 + s * 512);
#pragma unroll
        for (int j = 0; j < FT; ++j) fa[s & 1][j] = *reinterpret_cast<const v4i*>(pa + slot * SLOT + j * 4096 + s * 512);
    };

    issue(0);
    issue(1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"i"(COPIES) : "memory");   // block 0 is there
    __syncthreads();
    load(0, 0);
    for (int kb = 0; kb < nkb; ++kb) {
        const int slot = kb & 1;
#pragma unroll
        for (int s = 0; s < 4; ++s) {
            if (s < 3) {
                load(slot, s + 1);
            } else {
                // every read of this slot is in registers; the other slot's copies have landed
                asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                issue(kb + 2);
                load(slot ^ 1, 0);
            }
#pragma unroll
            for (int j = 0; j < FT; ++j)
#pragma unroll
                for (int i = 0; i < FF; ++i)
                    acc[j][i] = __builtin_amdgcn_mfma_i32_32x32x32_i8(fb[s & 1][i], fa[s & 1][j], acc[j][i], 0, 0, 0);
        }
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    if (blockIdx.x >= sp.full) {   // a range's sums as they lie in the registers
        v4i* const p = reinterpret_cast<v4i*>(sp.part) + ((int64_t)late * NW + wave) * FT * FF * 256 + lane;
#pragma unroll
        for (int j = 0; j < FT; ++j)
#pragma unroll
            for (int i = 0; i < FF; ++i)
#pragma unroll
                for (int q = 0; q < 4; ++q)
                    p[((j * FF + i) * 4 + q) * 64] = v4i{acc[j][i][4 * q], acc[j][i][4 * q + 1], acc[j][i][4 * q + 2], acc[j][i][4 * q + 3]};
        return;
    }
    __syncthreads();   // the slots are free: each wavefront stages its tiles through 4 KiB of its own
    store_tiles<FT, FF, OUT>(acc, smem + wave * 4096, t0 + wt * FT * 32, f0 + wf * FF * 32, T, N, As, Bs, n_pad, out, vec_store);
}

// One wavefront per token tile x FF of a split tile: its ranges' sums, then the outputs.
template <int FT, int FF, int WT, int WF, int OUT>
__global__ __launch_bounds__(64) void int8_reduce_kernel(const float* __restrict__ As, int64_t T, const float* __restrict__ Bs, int64_t N,
                                                         int64_t n_pad, void* __restrict__ out, int vec_store, Split sp) {
    constexpr int BT = WT * FT * 32, BF = WF * FF * 32, NW = WT * WF;
    __shared__ __attribute__((aligned(1024))) uint8_t stage[4096];
    const uint32_t j = blockIdx.x % FT, sub = blockIdx.x / FT, tile = sub / NW, wave = sub % NW;
    uint32_t tm, tn;
    tile_at<4>(sp.full + tile, (uint32_t)((T + BT - 1) / BT), (uint32_t)((N + BF - 1) / BF), tm, tn);
    const int64_t t0 = (int64_t)tm * BT + (wave % WT * FT + j) * 32, f0 = (int64_t)tn * BF + wave / WT * FF * 32;
    if (t0 >= T || f0 >= N) return;
    v16i acc[1][FF];
#pragma unroll
    for (int i = 0; i < FF; ++i)
#pragma unroll
        for (int e = 0; e < 16; ++e) acc[0][i][e] = 0;
    for (uint32_t c = 0; c < sp.n; ++c) {
        const v4i* const p = reinterpret_cast<const v4i*>(sp.part) + (((int64_t)(tile * sp.n + c) * NW + wave) * FT + j) * FF * 256 + threadIdx.x;
#pragma unroll
        for (int i = 0; i < FF; ++i)
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const v4i v = p[(i * 4 + q) * 64];
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[0][i][4 * q + e] += v[e];
            }
    }
    store_tiles<1, FF, OUT>(acc, stage, t0, f0, T, N, As, Bs, n_pad, out, vec_store);
}

// ---------------------------------------------------------------- few tokens
//
// Bound by reading the weight codes once (one token, 5120 -> 13824: 71 MB in 13.8 us, 5.1 TB/s with the start), for
// 65 to 1024 tokens of middling layers by the CUs' load path, as every 16 weight rows read all tokens' codes.  A workgroup owns RT tiles of 16 weight rows; its eight
// wavefronts take every eighth block of 128 inputs and multiply codes straight from memory with
// up to NT tiles of 16 tokens; the eight partial sums meet in LDS.  gridDim.z ranges of the inputs
// keep the CUs filled where there are few row tiles; the last one done adds them.  (33 to 64 tokens by two row tiles: sums and
// flag are 81924 bytes of LDS, so that a CU has one workgroup; 64 tokens 5120 -> 13824 25 us a call, 32 tokens 16.)
__device__ __forceinline__ void put_int(int32_t* p, int32_t v) { __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }
__device__ __forceinline__ int32_t get_int(const int32_t* p) { return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT); }

template <int NT, int RT, int OUT>
__global__ __launch_bounds__(512, RT == 1 ? 1 : NT == 2 ? 4 : 2) void int8_gemv_kernel(
    const uint8_t* __restrict__ Aq, const float* __restrict__ As, int64_t T, const uint8_t* __restrict__ Bq, const float* __restrict__ Bs,
    int64_t N, int64_t nkb, void* __restrict__ out, int vec_store, int32_t* __restrict__ part, int32_t* __restrict__ count) {
    constexpr int LD = 20;                                 // staged row stride
    __shared__ __attribute__((aligned(16))) int32_t red[8 * RT * NT * 16 * LD];
    __shared__ int done;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int64_t n0 = (int64_t)blockIdx.x * RT * 16, t0 = (int64_t)blockIdx.y * NT * 16;
    const int64_t blk = nkb * 2048;
    const uint8_t *bp[RT], *ap[NT];
#pragma unroll
    for (int m = 0; m < RT; ++m) bp[m] = Bq + (n0 + m * 16 < N ? n0 + m * 16 : n0) / 16 * blk + lane * 16;
#pragma unroll
    for (int i = 0; i < NT; ++i) ap[i] = Aq + (t0 + i * 16 < T ? t0 + i * 16 : t0) / 16 * blk + lane * 16;

    v4i acc[RT][NT];
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i] = v4i{0, 0, 0, 0};
    const int kb1 = (int)(nkb * (blockIdx.z + 1) / gridDim.z);
    for (int kb = (int)(nkb * blockIdx.z / gridDim.z) + wave; kb < kb1; kb += 8) {
        v4i b[RT][2];
#pragma unroll
        for (int m = 0; m < RT; ++m)
#pragma unroll
            for (int h = 0; h < 2; ++h) b[m][h] = *reinterpret_cast<const v4i*>(bp[m] + kb * 2048 + h * 1024);
#pragma unroll
        for (int i = 0; i < NT; ++i)
#pragma unroll
            for (int h = 0; h < 2; ++h) {
                const v4i a = *reinterpret_cast<const v4i*>(ap[i] + kb * 2048 + h * 1024);
#pragma unroll
                for (int m = 0; m < RT; ++m) acc[m][i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(b[m][h], a, acc[m][i], 0, 0, 0);
            }
    }
    // lane: token r of tile i, rows 4 g .. 4 g + 3
#pragma unroll
    for (int m = 0; m < RT; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) *reinterpret_cast<v4i*>(red + (((wave * RT + m) * NT + i) * 16 + r) * LD + 4 * g) = acc[m][i];
    __syncthreads();
    const int c = tid & 3, m = RT == 2 ? tid / (NT * 64) & 1 : 0;
    const int64_t tok = t0 + tid % (NT * 64) / 4, n = n0 + m * 16 + 4 * c;
    v4i y = v4i{0, 0, 0, 0};
    if (tid < RT * NT * 64)
#pragma unroll
        for (int w = 0; w < 8; ++w) y += *reinterpret_cast<const v4i*>(red + (w * RT * NT * 16 + (tid >> 2)) * LD + 4 * c);
    if (gridDim.z > 1) {   // the last of the tile's ranges to be done adds them all
        const uint32_t tile = blockIdx.y * gridDim.x + blockIdx.x, step = gridDim.x * gridDim.y * RT * NT * 256;
        int32_t* const p = part + tile * RT * NT * 256 + tid * 4;
        if (tid < RT * NT * 64)
#pragma unroll
            for (int e = 0; e < 4; ++e) put_int(p + blockIdx.z * step + e, y[e]);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // the range is where every XCD sees it
        __syncthreads();
        if (tid == 0) done = __hip_atomic_fetch_add(count + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        if (done != (int)gridDim.z - 1) return;
        y = v4i{0, 0, 0, 0};
        if (tid < RT * NT * 64)
            for (uint32_t u = 0; u < gridDim.z; ++u)
#pragma unroll
                for (int e = 0; e < 4; ++e) y[e] += get_int(p + u * step + e);
    }
    if (tid >= RT * NT * 64 || tok >= T || n >= N) return;
    const float sx = As[tok];
    const v4f sw = *reinterpret_cast<const v4f*>(Bs + n);
    v4f o;
#pragma unroll
    for (int e = 0; e < 4; ++e) o[e] = (sx * sw[e]) * (float)y[e];
    if constexpr (OUT == W4A4_Y_F32) {
        float* const Y = reinterpret_cast<float*>(out) + tok * N + n;
        if (vec_store && n + 3 < N) {
            *reinterpret_cast<v4f*>(Y) = o;
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) Y[e] = o[e];
        }
    } else {
        uint16_t* const Y = reinterpret_cast<uint16_t*>(out) + tok * N + n;
        const uint32_t w[2] = {pk_bf16(o[0], o[1]), pk_bf16(o[2], o[3])};
        if (vec_store && n + 3 < N) {
            *reinterpret_cast<uint2*>(Y) = make_uint2(w[0], w[1]);
        } else {
#pragma unroll
            for (int e = 0; e < 4; ++e)
                if (n + e < N) Y[e] = (uint16_t)(w[e / 2] >> (16 * (e & 1)));
        }
    }
}

template <int FT, int FF, int WT, int WF, int OUT>
hipError_t run_tiles(const uint8_t* aq, const float* as, int64_t T, const w4a4_int8_packed& d, void* out, int32_t* part, const Int8Plan& plan,
                     hipStream_t st) {
    const int vec = d.d_out % (OUT == W4A4_Y_F32 ? 4 : 8) == 0 ? 1 : 0;
    const Split sp = {part, (uint32_t)plan.full, (uint32_t)plan.split};
    const int64_t tail = plan.tiles - plan.full;
    hipLaunchKernelGGL((int8_gemm_kernel<FT, FF, WT, WF, OUT>), dim3((uint32_t)(plan.full + tail * plan.split)), dim3(WT * WF * 64), 0, st, aq,
                       as, T, d.codes, d.scales, d.d_out, d.n_pad, d.k_pad / 128, out, vec, sp);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess || !tail) return e;
    hipLaunchKernelGGL((int8_reduce_kernel<FT, FF, WT, WF, OUT>), dim3((uint32_t)(tail * WT * WF * FT)), dim3(64), 0, st, as, T, d.scales,
                       d.d_out, d.n_pad, out, vec, sp);
    return hipGetLastError();
}

template <int NT, int RT, int OUT>
hipError_t run_few(const uint8_t* aq, const float* as, int64_t T, const w4a4_int8_packed& d, void* out, int32_t* part, int32_t* count,
                   const Int8Plan& plan, hipStream_t st) {
    const dim3 grid((uint32_t)((d.d_out + RT * 16 - 1) / (RT * 16)), (uint32_t)((T + NT * 16 - 1) / (NT * 16)), (uint32_t)plan.split);
    hipLaunchKernelGGL((int8_gemv_kernel<NT, RT, OUT>), grid, dim3(512), 0, st, aq, as, T, d.codes, d.scales, d.d_out, d.k_pad / 128, out,
                       d.d_out % 4 == 0 ? 1 : 0, part, count);
    return hipGetLastError();
}

template <int OUT>
hipError_t run_out(const uint8_t* aq, const float* as, int64_t T, const w4a4_int8_packed& d, void* out, int32_t* part, int32_t* count,
                   hipStream_t st) {
    const Int8Plan plan = int8_plan(T, d.d_out, d.k_pad);
    if (plan.few && T <= 16) return run_few<1, 1, OUT>(aq, as, T, d, out, part, count, plan, st);
    if (plan.few && T <= 32)
        return plan.rt == 2 ? run_few<2, 2, OUT>(aq, as, T, d, out, part, count, plan, st)
                            : run_few<2, 1, OUT>(aq, as, T, d, out, part, count, plan, st);
    if (plan.few)
        return plan.rt == 2 ? run_few<4, 2, OUT>(aq, as, T, d, out, part, count, plan, st)
                            : run_few<4, 1, OUT>(aq, as, T, d, out, part, count, plan, st);
    if (plan.big) return run_tiles<4, 2, 2, 4, OUT>(aq, as, T, d, out, part, plan, st);
    return run_tiles<2, 2, 2, 2, OUT>(aq, as, T, d, out, part, plan, st);
}

}  // namespace

// Big tiles are 256 x 256, one workgroup a CU, from 64 of them on; small ones 128 x 128, two a CU.
// The tiles that fill whole rounds of the CUs run whole; the rest are cut along the inputs into as
// many ranges as there are free CUs, at least MIN_BLOCKS blocks each.
Int8Plan int8_plan(int64_t T, int64_t N, int64_t k_pad) {
    Int8Plan p = {0, 0, 1, 1, false, false, 0};
    constexpr int64_t CUS = 256, MIN_BLOCKS = 4, MAX_SPLIT = 16, FEW_CODES = 1 << 25;
    const int64_t nkb = k_pad / 128;
    p.few = int8_few(T, N, k_pad);
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

// Few tokens have a plan of their own for 16, 32 and every 64 tokens: looked at one by one.  Tiles have one for
// every 128 or 256: of many tokens, what tails leave at most, s ranges of each of min(tiles, a round's) tiles.
Int8Room int8_room(int64_t T, int64_t N, int64_t k_pad) {
    Int8Room r = {0, false};
    auto most = [&](int64_t n, const Int8Plan& p) {
        if ((size_t)n > r.part_bytes) r.part_bytes = (size_t)n;
        r.counters |= p.few && p.split > 1;
    };
    for (int64_t t : {16, 32}) {
        const Int8Plan p = int8_plan(T < t ? T : t, N, k_pad);
        most((int64_t)p.part_bytes, p);
    }
    for (int64_t t = 64; t - 64 < T && t <= 1024; t += 64) {
        const Int8Plan p = int8_plan(T < t ? T : t, N, k_pad);
        most((int64_t)p.part_bytes, p);
    }
    const int64_t s = k_pad / 128 / 4 < 16 ? k_pad / 128 / 4 : 16, nb = (N + 255) / 256;
    if (T <= 1024 || s < 2) return r;
    const int64_t big = (T + 255) / 256 * nb, small_T = 63 / nb * 256 < T ? 63 / nb * 256 : T;
    if (small_T > 1024) {
        const int64_t tiles = (small_T + 127) / 128 * ((N + 127) / 128);
        most((tiles * s < 512 ? tiles * s : 512) * 128 * 128 * 4, Int8Plan{});
    }
    if (big >= 64) most((big * s < 256 ? big * s : 256) * 256 * 256 * 4, Int8Plan{});
    return r;
}

hipError_t launch_int8_gemm(const uint8_t* aq, const float* as, int64_t T, const w4a4_int8_packed& d, void* out, int y_dtype, int32_t* part,
                            int32_t* count, hipStream_t st) {
    return y_dtype == W4A4_Y_F32 ? run_out<W4A4_Y_F32>(aq, as, T, d, out, part, count, st)
                                 : run_out<W4A4_Y_BF16>(aq, as, T, d, out, part, count, st);
}

}  // namespace w4a4

// Mixture-of-experts layer for a few tokens on gfx950 (declared and defined in
// include/w4a4.h: w4a4_moe_forward).  Three launches:
//
//   1. router logits l = X router^T, and the bf16 copy of X;
//   2. per (expert, 16 columns of h): which tokens chose the expert, gate and up products,
//      activation, h;
//   3. per 16 output columns: every chosen expert's down product, weighted and summed.
//
// The layer is bound by reading the chosen experts' codes once.  Wavefronts read codes
// straight from memory in the packed order (lane l of a run: row l % 16, inputs
// 32 q + 8 (l / 16) .. + 7 for q < 4), widen them to bf16 (exact) and feed
// v_mfma_f32_16x16x32_bf16 with 16 tokens on the other side, whose operand of step q is 64
// contiguous bytes of each token's row; a block's sum of 128 products is scaled by the block's
// weight scale in fp32.
//
// No kernel waits for another workgroup and no sum depends on who comes first: who chose what is
// recomputed where it is needed by counting, for one expert, how many experts rank before
// it (a total order, so every token's ranks 0 .. top_k - 1 are taken exactly once), and where
// workgroups share a tile of outputs, the last one to finish adds all parts in their order.
//
// Measured (us a call; "codes" is the time that the chosen experts' codes alone take at the 6.4 TB/s that a kernel
// which only reads reaches on long arrays):
//   1 token,   5120 x 1536 gated, 8 of 64 experts        42   (codes 30)
//   8 tokens,  2048 x 768 gated, 8 of 128 experts        61   (codes 38)
//   16 tokens, 5120 x 13824 GELU, 2 of 8 experts        184   (codes 175)
//   64 tokens, 5120 x 1536 gated, 6 of 64 experts       259   (codes 236)
// (on a slower card of the same kind 43, 64, 196, 258).  In the first two the three launches' starts and
// the first loads' latencies are the rest; in the last two the up kernel reads at 99% of that
// rate and the down kernel at 86 to 95%.
#include "fp8_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int MAX_T = W4A4_MOE_MAX_T;
constexpr int SLOT_E = 256;   // experts that the up kernel's slot search holds in a wavefront's registers
constexpr int WAVES = 4;   // of the up kernel: together a workgroup's rs x ks

// Order of logits as integers: larger first, a NaN before every number, -0 = +0.
__device__ __forceinline__ uint32_t rank_key(float l) {
    const uint32_t u = __float_as_uint(l + 0.0f);
    if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
    return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
// Whether expert e2 with key k2 comes before expert e with key k.
__device__ __forceinline__ bool before(uint32_t k2, int e2, uint32_t k, int e) { return k2 > k || (k2 == k && e2 < e); }

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const uint16_t* p) { return bf16_to_f32(*p); }
__device__ __forceinline__ void row8(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void row8(const uint16_t* p, float* v) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// ---------------------------------------------------------------- 1. router

__host__ __device__ constexpr int logits_ld(int E) { return (E + 3) / 4 * 4; }   // row stride of the logits

constexpr int LE = 2;   // experts per workgroup
// Workgroup: LE experts x LT tokens, the inputs dealt over its 256 lanes.  Workgroups past the
// experts' write the bf16 copy of X (zero padded to d_pad), 2048 inputs of LT tokens each; there
// are none where X itself is bf16 without padding.
template <int LT, typename X, typename R>
__global__ __launch_bounds__(256) void moe_logits_kernel(const X* __restrict__ x, const R* __restrict__ router, int T, int d,
                                                         int d_pad, int E, int vec, float* __restrict__ logits,
                                                         uint16_t* __restrict__ xb, int32_t* __restrict__ count) {
    __shared__ float part[4][LE * LT];
    const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
    const int t0 = blockIdx.y * LT;
    const int ne = (E + LE - 1) / LE;
    if (blockIdx.x + blockIdx.y == 0)   // the down step's counters
        for (int i = tid; i < (d + 15) / 16; i += 256) count[i] = 0;
    if ((int)blockIdx.x >= ne) {
        const int p = ((int)blockIdx.x - ne) * 2048 + tid * 8;
        if (p >= d_pad) return;
        for (int t = t0; t < t0 + LT && t < T; ++t) {
            const X* const r = x + (int64_t)t * d;
            float v[8];
            if (vec && p + 8 <= d) {
                row8(r + p, v);
            } else {
#pragma unroll
                for (int q = 0; q < 8; ++q) v[q] = p + q < d ? load1(r + p + q) : 0.0f;
            }
            *reinterpret_cast<uint4*>(xb + (int64_t)t * d_pad + p) =
                make_uint4(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3]), pk_bf16(v[4], v[5]), pk_bf16(v[6], v[7]));
        }
        return;
    }
    const int e0 = blockIdx.x * LE;
    float acc[LE][LT];
    const R* wr[LE];
    const X* xr[LT];
#pragma unroll
    for (int j = 0; j < LE; ++j) wr[j] = router + (int64_t)(e0 + j < E ? e0 + j : E - 1) * d;
#pragma unroll
    for (int i = 0; i < LT; ++i) {
        xr[i] = x + (int64_t)(t0 + i < T ? t0 + i : T - 1) * d;
#pragma unroll
        for (int j = 0; j < LE; ++j) acc[j][i] = 0.0f;
    }
    if (vec) {
#pragma unroll 2
        for (int p = tid * 8; p < d; p += 2048) {
            float a[LE][8], b[8];
#pragma unroll
            for (int j = 0; j < LE; ++j) row8(wr[j] + p, a[j]);
#pragma unroll
            for (int i = 0; i < LT; ++i) {
                row8(xr[i] + p, b);
#pragma unroll
                for (int j = 0; j < LE; ++j)
#pragma unroll
                    for (int q = 0; q < 8; ++q) acc[j][i] = __builtin_fmaf(a[j][q], b[q], acc[j][i]);
            }
        }
    } else {
        for (int p = tid; p < d; p += 256) {
#pragma unroll
            for (int i = 0; i < LT; ++i) {
                const float b = load1(xr[i] + p);
#pragma unroll
                for (int j = 0; j < LE; ++j) acc[j][i] = __builtin_fmaf(load1(wr[j] + p), b, acc[j][i]);
            }
        }
    }
#pragma unroll
    for (int j = 0; j < LE; ++j)
#pragma unroll
        for (int i = 0; i < LT; ++i) {
#pragma unroll
            for (int o = 32; o; o >>= 1) acc[j][i] += __shfl_xor(acc[j][i], o);
            if (lane == 0) part[wave][j * LT + i] = acc[j][i];
        }
    __syncthreads();
    if (tid < LE * LT) {
        const int e = e0 + tid / LT, t = t0 + tid % LT;
        if (e < E && t < T) logits[(int64_t)t * logits_ld(E) + e] = (part[0][tid] + part[1][tid]) + (part[2][tid] + part[3][tid]);
    }
}

// ---------------------------------------------------------------- products

struct Codes {
    uint4 lo, hi;   // a lane's 32 codes of one block
};
// (16 rows x 128 inputs of codes) . (128 inputs x 16 tokens); x: this lane's four pieces of its
// token.
__device__ __forceinline__ v4f block_mma(const Codes& c, const uint4* x) {
    const uint32_t w[8] = {c.lo.x, c.lo.y, c.lo.z, c.lo.w, c.hi.x, c.hi.y, c.hi.z, c.hi.w};
    v4f t = v4f{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_e4m3(w[2 * j], w[2 * j + 1]), __builtin_bit_cast(v8bf, x[j]), t, 0, 0, 0);
    return t;
}

// The vector memory path moves about 30 bytes a cycle into a CU's registers, whatever the addresses:
// with 2 KiB of codes a block it is the bound where the other operand is read for 16 tokens (4 KiB)
// and only a few are there.  So a wavefront reads the rows of 4 XI tokens, one KiB for each four
// (lane: row lane / 16, 16-byte chunk lane % 16), and passes them through LDS of its own to the
// lanes that the matrix instruction wants them in.  XI == 4: 16 tokens, read in place.
constexpr int tokens_of(int xi) { return xi == 4 ? 16 : 4 * xi; }
// Where row `row`'s chunk c lies (16-byte units): four rows' chunks of one column in four bank groups.
__device__ __forceinline__ int xs_at(int row, int c) { return row * 16 + (c ^ ((row & 3) * 4)); }
template <int XI>
__device__ __forceinline__ void spread(uint4 (&x)[4], const uint4 (&v)[XI], uint4* xs) {
    if constexpr (XI == 4) {
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = v[q];
    } else {
        const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
        const int row = r < 4 * XI ? r : 0;
#pragma unroll
        for (int i = 0; i < XI; ++i) xs[xs_at(i * 4 + g, r)] = v[i];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
#pragma unroll
        for (int q = 0; q < 4; ++q) x[q] = xs[xs_at(row, q * 4 + g)];
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    }
}

// acc[m][i] += the scaled blocks kb0, kb0 + step, ... (n of them) of NM row tiles (wp, sp: codes and
// scales of the row tiles' nkb blocks, uniform) on NT token tiles, whose operand of block b is read
// at x0 + b * 256 + xoff (XI == 4: in pieces 64 bytes apart).  A ring of D blocks per wavefront: a
// block's registers are refilled as soon as they are used, so D - 1 blocks are always in flight.
// A lane holds one block's scale of a group of D.  The code is kept short: these kernels run for a
// few microseconds from a cold instruction cache.
template <int D, int NM, int NT, int XI>
__device__ __forceinline__ void stream_blocks(v4f (&acc)[NM][NT], const uint8_t* const (&wp)[NM], const float* const (&sp)[NM],
                                              Rsrc x0, const uint32_t (&xoff)[NT * (XI == 4 ? 1 : XI)], uint4* xs, int nkb,
                                              int kb0, int n, int step) {
    static_assert(NT == 1 || XI == 4, "several token tiles are read in place");
    if (n <= 0) return;
    const int lane = threadIdx.x & 63;
    Rsrc wr[NM], sr[NM];
#pragma unroll
    for (int m = 0; m < NM; ++m) {
        wr[m] = rsrc(wp[m], (uint32_t)nkb * 2048u);
        sr[m] = rsrc(sp[m], (uint32_t)nkb * 4u);
    }
    Codes w[D][NM];
    float s[NM], next[NM];
    uint4 x[D][NT][XI];
    auto load = [&](int j, int i) __attribute__((always_inline)) {
        const uint32_t b = (uint32_t)(kb0 + (i < n ? i : 0) * step), off = i < n ? 0 : NO_LOAD;
#pragma unroll
        for (int m = 0; m < NM; ++m)
            w[j][m] = Codes{load_once(wr[m], lane * 16 + off, b * 2048), load_once(wr[m], lane * 16 + off + 1024, b * 2048)};
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int q = 0; q < XI; ++q)
                x[j][t][q] = load_at(x0, XI == 4 ? xoff[t] + off + q * 64 : xoff[q] + off, b * 256);
    };
    auto load_scales = [&](int i) __attribute__((always_inline)) {   // of blocks i .. i + D - 1, one a lane
        const uint32_t at = i + lane < n && lane < D ? (uint32_t)(kb0 + (i + lane) * step) * 4u : NO_LOAD;
#pragma unroll
        for (int m = 0; m < NM; ++m) next[m] = load_word(sr[m], at);
    };
    load_scales(0);
#pragma unroll
    for (int j = 0; j < D; ++j) {
        load(j, j);
        __builtin_amdgcn_sched_barrier(0);
    }
    for (int i = 0; i < n; i += D) {
#pragma unroll
        for (int m = 0; m < NM; ++m) s[m] = next[m];
        load_scales(i + D);
#pragma unroll
        for (int j = 0; j < D; ++j) {
            const bool in = i + j < n;   // uniform; past the end the sums stay as they are
#pragma unroll
            for (int t = 0; t < NT; ++t) {
                uint4 op[4];
                spread<XI>(op, x[j][t], xs);
#pragma unroll
                for (int m = 0; m < NM; ++m) {
                    const float sm = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(s[m]), j));
                    const v4f v = block_mma(w[j][m], op);
#pragma unroll
                    for (int r = 0; r < 4; ++r) acc[m][t][r] = in ? __builtin_fmaf(v[r], sm, acc[m][t][r]) : acc[m][t][r];
                }
            }
            load(j, i + j + D);
            __builtin_amdgcn_sched_barrier(0);   // each block waits for its own loads only
        }
    }
}

// Sum over the eight lanes of an aligned group.
__device__ __forceinline__ int sum8(int c) {
#pragma unroll
    for (int o = 1; o < 8; o *= 2) c += __shfl_xor(c, o);
    return c;
}

// Maximum over the wavefront (in every lane).
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
    // row_shr 1, 2, 4, 8, then lane 15 of each row to the next row and lane 31 to the upper half;
    // lanes without a source keep the identity 0
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x111, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x112, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x114, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x118, 0xF, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x142, 0xA, 0xF, false));
    v = max(v, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x143, 0xC, 0xF, false));
    return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

struct UpArgs {
    const float* logits;
    const uint16_t* xb;
    int32_t *ids, *place;
    float* p;
    uint16_t* h;
    int T, E, k, renorm, f, by_slot;
    int rs, ks;                              // wavefronts along the rows (16 each) and along d
    int nkb_d, f_pad, n_pad;                 // d blocks of 128, roundup(f, 128), roundup(f, 16)
    const uint8_t *gate, *up;
    const float *gate_s, *up_s;
    int64_t mat_codes, mat_scales;           // bytes / scales per expert
};

// ---------------------------------------------------------------- 2. up

// A list entry: token, and the rank that the expert has there.
__device__ __forceinline__ int entry(int t, int rank) { return t << 8 | rank; }
__device__ __forceinline__ int entry_pair(int v, int k) { return (v >> 8) * k + (v & 255); }

// A pass over the codes takes NT tiles of 16 tokens, or, NT == 1, 4 XI tokens.  The workgroup computes
// rs row tiles, each summed over ks wavefronts.
template <bool GATED, int NT, int XI>
__global__ __launch_bounds__(WAVES * 64, NT == 1 ? 4 : NT == 2 ? 3 : 2) void moe_up_kernel(UpArgs a) {
    constexpr int NM = GATED ? 2 : 1, LD = 20;
    constexpr int D = NT == 4 ? 1 : NT == 2 ? 2 : GATED ? (XI == 4 ? 2 : 3) : (XI == 1 ? 6 : XI == 2 ? 5 : 4);
    constexpr int TP = NT == 1 ? tokens_of(XI) : NT * 16, NX = XI == 4 ? NT : XI;
    __shared__ int32_t list[MAX_T];
    __shared__ int32_t rank[MAX_T];
    __shared__ uint32_t top[MAX_T];          // key of the token's largest logit
    __shared__ int32_t count;                // tokens of the expert
    __shared__ __attribute__((aligned(16))) float red[NM * WAVES * NT * 16 * LD];
    __shared__ uint4 xs[XI == 4 ? 1 : WAVES * XI * 64];
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int ld = logits_ld(a.E);

    // Which expert: the grid's second dimension counts experts, or, where the tokens choose
    // fewer than there are, slots t * k + rank; a slot whose expert an earlier token chose too is
    // left to that token's slot.
    int e = blockIdx.y, n = 1;
    if (a.by_slot) {
        // the (want + 1)-th of the token's logits, by every wavefront for itself: logit j * 64 + lane
        // in a lane's j-th register, the largest taken want times
        const int t = blockIdx.y / a.k, want = blockIdx.y - t * a.k;
        const float* l = a.logits + t * ld;
        uint32_t key[SLOT_E / 64];
#pragma unroll
        for (int j = 0; j < SLOT_E / 64; ++j) key[j] = j * 64 + lane < a.E ? rank_key(l[j * 64 + lane]) : 0u;   // 0: no logit's key
        for (int i = 0; i <= want; ++i) {
            uint32_t m = 0;
#pragma unroll
            for (int j = 0; j < SLOT_E / 64; ++j) m = max(m, key[j]);
            m = wave_max(m);
            if (i == 0) top[t] = m;
            e = -1;
#pragma unroll
            for (int j = 0; j < SLOT_E / 64; ++j) {
                const uint64_t b = __ballot(key[j] == m);
                const bool here = e < 0 && b;
                const int at = __builtin_ctzll(b | 1ull << 63);
                e = here ? j * 64 + at : e;
                key[j] = here && lane == at ? 0u : key[j];
            }
        }
        e = __builtin_amdgcn_readfirstlane(e);
        list[0] = entry(t, want);   // every lane writes what it reads: one token needs no barrier
    }
    if (!a.by_slot || a.T > 1) {
        if (a.by_slot) __syncthreads();
        // the rank of e in every token: eight lanes a token
        for (int t = tid >> 3; t < a.T; t += WAVES * 8) {
            const float* l = a.logits + t * ld;
            const uint32_t key = rank_key(l[e]);
            int c = 0;
            uint32_t m = 0;
#pragma unroll 2
            for (int j = (tid & 7) * 4; j < a.E; j += 32) {
                const float4 v = *reinterpret_cast<const float4*>(l + j);
                const float lv[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    const uint32_t kj = j + q < a.E ? rank_key(lv[q]) : 0u;
                    c += before(kj, j + q, key, e) ? 1 : 0;
                    m = max(m, kj);
                }
            }
            c = sum8(c);
#pragma unroll
            for (int o = 1; o < 8; o *= 2) m = max(m, (uint32_t)__shfl_xor((int)m, o));
            if ((tid & 7) == 0) {
                rank[t] = c;
                top[t] = m;
            }
        }
        __syncthreads();
        if (tid < 64) {
            n = 0;
            for (int t0 = 0; t0 < a.T; t0 += 64) {
                const int t = t0 + lane;
                const bool in = t < a.T && rank[t < a.T ? t : 0] < a.k;
                const uint64_t b = __ballot(in);
                if (in) list[n + __popcll(b & ((1ull << lane) - 1))] = entry(t, rank[t]);
                n += __popcll(b);
            }
            if (lane == 0) count = n;
        }
        __syncthreads();
        n = __builtin_amdgcn_readfirstlane(count);
        if (n == 0 || (a.by_slot && entry_pair(list[0], a.k) < (int)blockIdx.y)) return;
    }

    const int wk = wave % a.ks, row0 = (blockIdx.x * a.rs + wave / a.ks) * 16;
    const int nkb = row0 < a.n_pad ? a.nkb_d : 0;   // past the packed rows: only h's padding
    const int64_t cofs = (int64_t)e * a.mat_codes + (int64_t)(row0 / 16) * a.nkb_d * 2048;
    const int64_t sofs = (int64_t)e * a.mat_scales + (int64_t)(row0 / 128) * a.nkb_d;
    const Rsrc xr = rsrc(a.xb, (uint32_t)a.T * (uint32_t)a.nkb_d * 256u);
    const int nb = nkb > wk ? (nkb - wk + a.ks - 1) / a.ks : 0;
    for (int c0 = 0; c0 < n; c0 += TP) {
        uint32_t xoff[NX];
#pragma unroll
        for (int i = 0; i < NX; ++i) {
            const int q = c0 + (XI == 4 ? i * 16 + r : i * 4 + g);
            xoff[i] = (uint32_t)(list[q < n ? q : c0] >> 8) * (uint32_t)a.nkb_d * 256u + (XI == 4 ? g : r) * 16;
        }
        v4f acc[NM][NT];
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i) acc[m][i] = v4f{0, 0, 0, 0};
        if constexpr (GATED) {
            const uint8_t* const wp[2] = {a.up + cofs, a.gate + cofs};
            const float* const sp[2] = {a.up_s + sofs, a.gate_s + sofs};
            stream_blocks<D, 2, NT, XI>(acc, wp, sp, xr, xoff, xs + wave * XI * 64, a.nkb_d, wk, nb, a.ks);
        } else {
            const uint8_t* const wp[1] = {a.up + cofs};
            const float* const sp[1] = {a.up_s + sofs};
            stream_blocks<D, 1, NT, XI>(acc, wp, sp, xr, xoff, xs + wave * XI * 64, a.nkb_d, wk, nb, a.ks);
        }
        if (c0) __syncthreads();
        // lane: token r of tile i, rows 4 g .. 4 g + 3
#pragma unroll
        for (int m = 0; m < NM; ++m)
#pragma unroll
            for (int i = 0; i < NT; ++i)
                *reinterpret_cast<v4f*>(red + (((m * WAVES + wave) * NT + i) * 16 + r) * LD + 4 * g) = acc[m][i];
        __syncthreads();
        for (int q = tid; q < a.rs * NT * 256; q += WAVES * 64) {
            const int tile = q / (NT * 256), at = q / 16 % (NT * 16), row = q & 15;
            const int hr = (blockIdx.x * a.rs + tile) * 16 + row;
            if (at >= TP || c0 + at >= n || hr >= a.f_pad) continue;
            float u = 0.0f, v = 0.0f;
            for (int w = tile * a.ks; w < (tile + 1) * a.ks; ++w) {
                u += red[(w * NT * 16 + at) * LD + row];
                if constexpr (GATED) v += red[((WAVES + w) * NT * 16 + at) * LD + row];
            }
            if constexpr (GATED) u = v / (1.0f + expf(-v)) * u;
            else u = gelu_tanh_f32(u);
            a.h[(int64_t)entry_pair(list[c0 + at], a.k) * a.f_pad + hr] = hr < a.f ? bf16_rne(u) : 0;
        }
    }

    if (blockIdx.x == 0) {   // what the down step reads of the routing, once per expert
        for (int q = tid >> 3; q < n; q += WAVES * 8) {
            const int t = list[q] >> 8, pair = entry_pair(list[q], a.k);
            const float* l = a.logits + t * ld;
            const uint32_t mk = top[t];
            const float mx = mk == 0xFFFFFFFFu ? __uint_as_float(0x7FC00000u)
                                               : __uint_as_float(mk ^ ((mk >> 31) ? 0x80000000u : 0xFFFFFFFFu));
            float v = expf(l[e] - mx);
            if (!a.renorm) {
                float sum = 0.0f;
                for (int j = tid & 7; j < a.E; j += 8) sum += expf(l[j] - mx);
#pragma unroll
                for (int o = 1; o < 8; o *= 2) sum += __shfl_xor(sum, o);
                v /= sum;
            }
            if ((tid & 7) == 0) {
                a.ids[pair] = e;
                a.place[pair] = q;
                a.p[pair] = v;
            }
        }
    }
}

// ---------------------------------------------------------------- 3. down

struct DownArgs {
    const int32_t *ids, *place;
    const float* p;
    const uint16_t* h;
    int T, E, k, renorm, d, y_dtype;
    int nkb_f;                               // f blocks of 128
    const uint8_t* codes;
    const float* scales;
    int64_t mat_codes, mat_scales;
    void* out;
    float* part;                             // [two a workgroup][T][16 RT]
    int32_t* count;                          // by tile of 16 RT outputs: parts that are done
};

__device__ __forceinline__ void store_y(const DownArgs& a, int t, int row, float y) {
    if (row >= a.d) return;
    if (a.y_dtype == W4A4_Y_F32) reinterpret_cast<float*>(a.out)[(int64_t)t * a.d + row] = y;
    else reinterpret_cast<uint16_t*>(a.out)[(int64_t)t * a.d + row] = bf16_rne(y);
}

constexpr int DOWN_MIN = 2;   // groups a wavefront, below which tiles stay whole (1 and 4: the same within 2%)

// TB: tokens the sums are laid out for; RT: row tiles (16 outputs) of a workgroup's tile.  A tile's
// work is one sequence of groups of D blocks: segment by segment (up to S tokens of one expert),
// the segment's nkb_f blocks, the last group of a segment cut short.  All tiles' groups are dealt
// evenly over as many workgroups as the CUs hold (one workgroup a tile left CUs idle or doubly loaded:
// 64 tokens, 1536 -> 5120: 125 against 101 us; 16 tokens, 13824 -> 5120: 123 against 97), so a workgroup
// has parts of one or more tiles.  The W wavefronts take equal consecutive ranges of a part; a
// wavefront's ring of D blocks in flight runs on from segment to segment, and where a segment ends its
// sums, times the tokens' probabilities, go to the wavefront's own sums in LDS, which are added in
// wavefront order at the end.  Segments have to be the same in every workgroup: the up step gives
// each pair its place in its expert's list.
template <int TB, int W, int XI, int RT>
__global__ __launch_bounds__(W * 64, TB < MAX_T ? 4 : 2) void moe_down_kernel(DownArgs a) {
    constexpr int S = tokens_of(XI), NX = XI == 4 ? 1 : XI, RL = 16 * RT;
    constexpr int PB = TB * W4A4_MOE_MAX_K, SEGS = W4A4_MOE_MAX_E + PB / S;
    constexpr int D = XI == 1 ? 6 : XI == 2 ? 4 : RT == 2 ? 2 : 3;
    __shared__ __attribute__((aligned(16))) float sums[W * TB * RL];
    __shared__ uint4 xs[XI == 4 ? 1 : W * XI * 64];
    __shared__ float den[TB], prob[PB];
    __shared__ uint16_t list[PB];              // pairs, expert by expert
    __shared__ int32_t first[W4A4_MOE_MAX_E];  // by expert: pairs, then where its list starts
    __shared__ uint16_t seg_e[SEGS], seg_l[SEGS];   // by segment: expert, place in list
    __shared__ uint8_t seg_n[SEGS];                 // its tokens
    __shared__ int n_seg, done;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int pairs = a.T * a.k, nkb = a.nkb_f;
    if (a.T == 1) {   // every pair is a segment
        for (int i = tid; i < pairs; i += W * 64) {
            prob[i] = a.p[i];
            list[i] = seg_l[i] = (uint16_t)i;
            seg_e[i] = (uint16_t)a.ids[i];
            seg_n[i] = 1;
        }
        if (tid == 0) n_seg = pairs;
        __syncthreads();
    } else {
        for (int i = tid; i < a.E; i += W * 64) first[i] = 0;
        __syncthreads();
        for (int i = tid; i < pairs; i += W * 64) {
            prob[i] = a.p[i];
            atomicAdd(&first[a.ids[i]], 1);
        }
        __syncthreads();
        if (tid < 64) {
            int at = 0, seg = 0;
            for (int e0 = 0; e0 < a.E; e0 += 64) {
                const int e = e0 + lane, c = e < a.E ? first[e] : 0;
                int v = c | ((c + S - 1) / S) << 16;       // pairs and segments, summed over the lanes before
#pragma unroll
                for (int o = 1; o < 64; o *= 2) {
                    const int u = __shfl_up(v, o);
                    v += lane >= o ? u : 0;
                }
                const int l0 = at + (v & 0xFFFF) - c;
                int s = seg + (v >> 16) - (c + S - 1) / S;
                if (e < a.E) first[e] = l0;
                for (int q = 0; q * S < c; ++q, ++s) {
                    seg_e[s] = (uint16_t)e;
                    seg_l[s] = (uint16_t)(l0 + q * S);
                    seg_n[s] = (uint8_t)(c - q * S < S ? c - q * S : S);
                }
                const int all = __shfl(v, 63);
                at += all & 0xFFFF;
                seg += all >> 16;
            }
            if (lane == 0) n_seg = seg;
        }
        __syncthreads();
        for (int i = tid; i < pairs; i += W * 64) list[first[a.ids[i]] + a.place[i]] = (uint16_t)i;
    }
    for (int t = tid; t < a.T; t += W * 64) {
        float s = 1.0f;
        if (a.renorm) {
            s = 0.0f;
            for (int j = 0; j < a.k; ++j) s += prob[t * a.k + j];
        }
        den[t] = s;
    }
    __syncthreads();

    const int groups = (nkb + D - 1) / D;          // of a segment
    // all groups of all tiles, dealt evenly; 32 bits hold them (4096 tiles, 1500 segments, 171 groups)
    const int per = __builtin_amdgcn_readfirstlane(n_seg) * groups, tiles = (a.d + RL - 1) / RL, all = tiles * per;
    const int wgs = min(max(tiles, all / (DOWN_MIN * W)), (int)gridDim.x), q = blockIdx.x;
    if (q >= wgs) return;
    const int share = all / wgs, extra = all - share * wgs;   // the first `extra` workgroups take one more
    auto start = [&](int u) { return share * u + min(u, extra); };
    auto owner = [&](int x) { return x < extra * (share + 1) ? x / (share + 1) : extra + (x - extra * (share + 1)) / share; };
    const int q_at = start(q), q_end = start(q + 1);
    for (int at = q_at; at < q_end;) {
        const int tile = at / per, stop = min(q_end, (tile + 1) * per);
        const int row0 = tile * RL, from = at - tile * per, size = stop - at;
        const int begin = from + size * wave / W, len = from + size * (wave + 1) / W - begin;
        const int rts = min((a.d + 15) / 16 - tile * RT, RT);
        float* const mine = sums + wave * TB * RL;
        for (int i = lane; i < TB * RL; i += 64) mine[i] = 0.0f;
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
        if (len > 0) {
            int seg = begin / groups, lkb = (begin - seg * groups) * D;   // the group that is loaded
            const Rsrc xr = rsrc(a.h, (uint32_t)pairs * (uint32_t)nkb * 256u);
            Rsrc wr, sr;
            uint32_t xoff[NX];
            auto open = [&](int sg) __attribute__((always_inline)) {
                const int e = __builtin_amdgcn_readfirstlane(seg_e[sg]), n = __builtin_amdgcn_readfirstlane(seg_n[sg]);
                wr = rsrc(a.codes + (int64_t)e * a.mat_codes + (int64_t)tile * RT * nkb * 2048, (uint32_t)rts * nkb * 2048u);
                sr = rsrc(a.scales + (int64_t)e * a.mat_scales + (int64_t)(row0 / 128) * nkb, (uint32_t)nkb * 4u);
                // rows past the segment's tokens read the first one's h
    #pragma unroll
                for (int i = 0; i < NX; ++i) {
                    const int q = XI == 4 ? r : i * 4 + g;
                    xoff[i] = (uint32_t)list[seg_l[sg] + (q < n ? q : 0)] * (uint32_t)nkb * 256u + (XI == 4 ? g : r) * 16;
                }
            };
            Codes w[D][RT];
            uint4 x[D][XI];
            float sc, next;
            auto load = [&](int j) __attribute__((always_inline)) {
                const uint32_t b = (uint32_t)(lkb + j), off = lkb + j < nkb ? 0 : NO_LOAD;
    #pragma unroll
                for (int t = 0; t < RT; ++t) {
                    const uint32_t at = off + lane * 16 + t * (uint32_t)nkb * 2048u;
                    w[j][t] = Codes{load_once(wr, at, b * 2048u), load_once(wr, at + 1024, b * 2048u)};
                }
    #pragma unroll
                for (int q = 0; q < XI; ++q) x[j][q] = load_at(xr, XI == 4 ? xoff[0] + off + q * 64 : xoff[q] + off, b * 256u);
            };
            auto load_scales = [&]() __attribute__((always_inline)) {   // of the group, one a lane
                const uint32_t at = lane < D && lkb + lane < nkb ? (uint32_t)(lkb + lane) * 4u : NO_LOAD;
                next = load_word(sr, at);
            };
            open(seg);
            load_scales();
    #pragma unroll
            for (int j = 0; j < D; ++j) {
                load(j);
                __builtin_amdgcn_sched_barrier(0);
            }
            v4f acc[RT];
    #pragma unroll
            for (int t = 0; t < RT; ++t) acc[t] = v4f{0, 0, 0, 0};
            for (int i = 0; i < len; ++i) {
                const int kb = lkb, sg = seg;          // the group that is used
                lkb += D;
                const bool ends = lkb >= nkb;
                if (i + 1 == len) {
                    lkb = nkb;                         // nothing left to load
                } else if (ends) {
                    lkb = 0;
                    open(++seg);
                }
                sc = next;
                load_scales();
    #pragma unroll
                for (int j = 0; j < D; ++j) {
                    const bool in = kb + j < nkb;      // uniform; past the end the sums stay as they are
                    uint4 op[4];
                    spread<XI>(op, x[j], xs + wave * XI * 64);
                    const float s = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(sc), j));
    #pragma unroll
                    for (int t = 0; t < RT; ++t) {
                        const v4f v = block_mma(w[j][t], op);
    #pragma unroll
                        for (int q = 0; q < 4; ++q) acc[t][q] = in ? __builtin_fmaf(v[q], s, acc[t][q]) : acc[t][q];
                    }
                    load(j);
                    __builtin_amdgcn_sched_barrier(0);   // each block waits for its own loads only
                }
                if (ends || i + 1 == len) {            // the segment, or the wavefront's part of it, ends
                    if (r < seg_n[sg]) {               // tokens of one expert are distinct: no two lanes meet
                        const int pair = list[seg_l[sg] + r], t = pair / a.k;
                        const float pw = a.renorm ? prob[pair] / den[t] : prob[pair];
    #pragma unroll
                        for (int u = 0; u < RT; ++u) {
                            v4f* const s = reinterpret_cast<v4f*>(mine + t * RL + u * 16 + 4 * g);
                            v4f v = *s;
    #pragma unroll
                            for (int q = 0; q < 4; ++q) v[q] = __builtin_fmaf(acc[u][q], pw, v[q]);
                            *s = v;
                        }
                    }
    #pragma unroll
                    for (int u = 0; u < RT; ++u) acc[u] = v4f{0, 0, 0, 0};
                }
            }
        }
        __syncthreads();
        const bool whole = size == per;
        // the first of the workgroup's parts, or the last one
        float* const part = a.part + (2 * q + (at != q_at)) * a.T * RL;
        for (int i = tid; i < a.T * RL; i += W * 64) {
            float y = 0.0f;
#pragma unroll
            for (int w = 0; w < W; ++w) y += sums[w * TB * RL + i];
            if (whole) store_y(a, i / RL, row0 + i % RL, y);
            else put_shared(part + i, y);
        }
        if (!whole) {
            const int q0 = owner(tile * per), q1 = owner((tile + 1) * per - 1);
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // this part is where every XCD sees it
            __syncthreads();
            if (tid == 0) done = __hip_atomic_fetch_add(a.count + tile, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
            __syncthreads();
            if (done == q1 - q0) {          // the last part to be done adds them all, in order
                const float* const p0 = a.part + (2 * q0 + (start(q0) < tile * per)) * a.T * RL;
                for (int i = tid; i < a.T * RL; i += W * 64) {
                    float y = get_shared(p0 + i);
                    for (int u = q0 + 1; u <= q1; ++u) y += get_shared(a.part + 2 * u * a.T * RL + i);
                    store_y(a, i / RL, row0 + i % RL, y);
                }
            }
        }
        __syncthreads();
        at = stop;
    }
}

template <int LT, typename X>
void run_logits(const void* X_, const w4a4_moe& m, int T, bool copy, float* logits, uint16_t* xb, int32_t* count, hipStream_t st) {
    const int d = (int)m.up.d_in, d_pad = (int)m.up.k_pad, E = (int)m.up.n_mat;
    const dim3 grid((uint32_t)((E + LE - 1) / LE + (copy ? (d_pad + 2047) / 2048 : 0)), (uint32_t)((T + LT - 1) / LT));
    const int vec = d % 8 == 0 ? 1 : 0;
    if (m.router_dtype == W4A4_X_BF16)
        hipLaunchKernelGGL((moe_logits_kernel<LT, X, uint16_t>), grid, dim3(256), 0, st, (const X*)X_, (const uint16_t*)m.router, T,
                           d, d_pad, E, vec, logits, xb, count);
    else
        hipLaunchKernelGGL((moe_logits_kernel<LT, X, float>), grid, dim3(256), 0, st, (const X*)X_, (const float*)m.router, T, d,
                           d_pad, E, vec, logits, xb, count);
}

// Tokens of an expert that a pass over its codes takes (xi and, above 16, nt tiles), from the number
// that it has on average: a second pass reads the codes again, a wider one reads more of the other
// operand than there is.  Passes of 4, 8, 16 and 32 tokens, us a call, 2048 x 768 gated, 8 of 64 experts:
//   8 tokens 58, 56, 57, 62;  16: 70, 62, 62, 67;  32: 95, 73, 67, 72;  64: 146, 104, 77, 80;
// 64 tokens, 8 of 32 experts: 125, 86, 65, 58.  Between three and four tokens an expert, 8 or 16 a pass:
// above 16 tokens, where the down step then has 16 wavefronts a workgroup, 16 (24 tokens, 2048 x 768, 9 of 64 experts: 69, 63; 32 tokens, 8 of 64: 75, 65; 40 tokens,
// 5120 x 1536, 6 of 64: 252, 246; 20 tokens, 4096 x 1024, 3 of 16: 52, 48; but 40 tokens, 1024 x 512, 3
// of 32: 32, 35, and 32 tokens, 2880 x 2880, 4 of 32: 150, 158), up to 16 tokens, where it has 8
// either way, 8 (16 tokens, 5120 x 13824 GELU, 2 of 8: 196, 223; 16 tokens, 5120 x 1536, 8 of 32:
// 133, 140; 10 tokens, 5120 x 13824, 3 of 8: 274, 285; but 16 tokens, 2048 x 768, 4 of 16: 32, 30).
struct Pass {
    int xi, nt;
};
Pass pass_of(int64_t T, int64_t k, int64_t E) {
    const int64_t pairs = T * k;
    if (T <= 4 || pairs <= E) return {1, 1};
    if (T <= 8 || pairs <= (T <= 16 ? 4 : 3) * E) return {2, 1};
    if (T <= 16 || pairs <= 10 * E) return {4, 1};
    return {4, pairs <= 24 * E ? 2 : 4};
}

template <bool GATED>
void run_up(const UpArgs& a, Pass p, dim3 grid, hipStream_t st) {
    const dim3 block(WAVES * 64);
    if (p.xi == 1) hipLaunchKernelGGL((moe_up_kernel<GATED, 1, 1>), grid, block, 0, st, a);
    else if (p.xi == 2) hipLaunchKernelGGL((moe_up_kernel<GATED, 1, 2>), grid, block, 0, st, a);
    else if (p.nt == 1) hipLaunchKernelGGL((moe_up_kernel<GATED, 1, 4>), grid, block, 0, st, a);
    else if (p.nt == 2) hipLaunchKernelGGL((moe_up_kernel<GATED, 2, 4>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((moe_up_kernel<GATED, 4, 4>), grid, block, 0, st, a);
}

// One workgroup of 16 wavefronts or two of 8 fit a CU.
template <int TB, int W, int XI, int RT>
void down(const DownArgs& a, int wgs, hipStream_t st) {
    hipLaunchKernelGGL((moe_down_kernel<TB, W, XI, RT>), dim3((uint32_t)wgs), dim3(W * 64), 0, st, a);
}
template <int XI>
void run_down(const DownArgs& a, hipStream_t st) {
    if (a.T <= 16) return down<16, 8, XI, 1>(a, 512, st);
    if (a.T > 64) return down<MAX_T, 8, XI, 1>(a, 256, st);
    if constexpr (XI == 4) {
        // two row tiles for one read of h, where its 16 tokens' rows are twice the codes of one (64
        // tokens, 6 of 64 experts, 1536 -> 5120: 145 to 120 us), where there are more tiles than workgroups
        // (37 tokens, 333 -> 1000: 11.4 us with two, 10.0 with one)
        if (a.d > 4096) return down<64, 16, XI, 2>(a, 256, st);
        down<64, 16, XI, 1>(a, 256, st);
    } else {
        down<64, 8, XI, 1>(a, 512, st);
    }
}

}  // namespace

hipError_t launch_moe(const void* X, int x_dtype, int64_t T, const w4a4_moe& m, const MoeBuffers& b, void* Y, int y_dtype,
                      hipStream_t st) {
    // X itself serves the products where it is bf16 and its rows need no padding
    const bool copy = x_dtype != W4A4_X_BF16 || m.up.d_in != m.up.k_pad;
    if (x_dtype == W4A4_X_BF16) {
        if (T == 1) run_logits<1, uint16_t>(X, m, (int)T, copy, b.logits, b.xb, b.count, st);
        else run_logits<4, uint16_t>(X, m, (int)T, copy, b.logits, b.xb, b.count, st);
    } else {
        if (T == 1) run_logits<1, float>(X, m, (int)T, copy, b.logits, b.xb, b.count, st);
        else run_logits<4, float>(X, m, (int)T, copy, b.logits, b.xb, b.count, st);
    }
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;

    const bool gated = m.activation == W4A4_MOE_SILU_GATED;
    UpArgs u;
    u.logits = b.logits; u.xb = copy ? b.xb : (const uint16_t*)X; u.ids = b.ids; u.place = b.place; u.p = b.p; u.h = b.h;
    u.T = (int)T; u.E = (int)m.up.n_mat; u.k = m.top_k; u.renorm = m.renormalize != 0; u.f = (int)m.up.d_out;
    u.by_slot = T * m.top_k < m.up.n_mat && m.up.n_mat <= SLOT_E ? 1 : 0;
    u.nkb_d = (int)(m.up.k_pad / 128); u.f_pad = (int)m.down.k_pad; u.n_pad = (int)m.up.n_pad;
    u.gate = gated ? m.gate.codes : nullptr; u.gate_s = gated ? m.gate.scales : nullptr;
    u.up = m.up.codes; u.up_s = m.up.scales;
    u.mat_codes = m.up.n_pad * m.up.k_pad; u.mat_scales = (m.up.d_out + 127) / 128 * (m.up.k_pad / 128);
    const int64_t ny = u.by_slot ? T * m.top_k : m.up.n_mat, tiles = u.f_pad / 16;
    // 16 wavefronts fit a CU at this kernel's registers: d is split over as many as keep all
    // of them resident
    u.ks = ny * tiles <= 1024 ? 4 : ny * tiles <= 2048 ? 2 : 1;
    u.rs = WAVES / u.ks;
    const dim3 grid((uint32_t)((tiles + u.rs - 1) / u.rs), (uint32_t)ny);
    const Pass pass = pass_of(T, m.top_k, m.up.n_mat);
    if (gated) run_up<true>(u, pass, grid, st);
    else run_up<false>(u, pass, grid, st);
    e = hipGetLastError();
    if (e != hipSuccess) return e;

    DownArgs d;
    d.ids = b.ids; d.place = b.place; d.p = b.p; d.h = b.h;
    d.T = u.T; d.E = u.E; d.k = u.k; d.renorm = u.renorm; d.d = (int)m.down.d_out;
    d.nkb_f = (int)(m.down.k_pad / 128);
    d.codes = m.down.codes; d.scales = m.down.scales;
    d.mat_codes = m.down.n_pad * m.down.k_pad; d.mat_scales = (m.down.d_out + 127) / 128 * (m.down.k_pad / 128);
    d.out = Y;
    d.part = b.part; d.count = b.count;
    d.y_dtype = y_dtype;
    if (pass.xi == 1) run_down<1>(d, st);
    else if (pass.xi == 2) run_down<2>(d, st);
    else run_down<4>(d, st);
    return hipGetLastError();
}

}  // namespace w4a4

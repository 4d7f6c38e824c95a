// Mixture-of-experts layer for a few tokens on gfx950 (declared and defined in
// include/w4a4.h: w4a4_moe_forward).  Three launches:
//
//   1. router logits l = X router^T, and the bf16 copy of X;
//   2. per (expert, 16 columns of h): which tokens chose the expert, gate and up products,
//      activation, h;
//   3. per 16 output columns: every chosen expert's down product, weighted and summed.
//
// The layer is bound by reading the chosen experts' codes once.  Wavefronts read codes
// straight from memory in the packed order (lane l of a 16-row half block: row l % 16,
// inputs 32 (l / 16) .. + 31), widen them to bf16 (exact) and feed
// v_mfma_f32_16x16x32_bf16 with 16 tokens on the other side; a block's sum of 128 products
// is scaled by the block's weight scale in fp32.
//
// No kernel waits for another workgroup and nothing is added by atomics: who chose what is
// recomputed where it is needed by counting, for one expert, how many experts rank before
// it (a total order, so every token's ranks 0 .. top_k - 1 are taken exactly once).
#include "w4a4_device.h"
#include "w4a4_internal.h"

namespace w4a4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int MAX_T = W4A4_MOE_MAX_T;
constexpr int WAVES = 8;

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
__device__ __forceinline__ void load8(const float* p, float* v) {
    const float4 a = *reinterpret_cast<const float4*>(p), b = *reinterpret_cast<const float4*>(p + 4);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void load8(const uint16_t* p, float* v) {
    const uint4 a = *reinterpret_cast<const uint4*>(p);
    const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
}

// ---------------------------------------------------------------- 1. router

constexpr int LT = 4;   // tokens per wavefront
// Wavefront: one expert x LT tokens.  The last column of workgroups writes the bf16 copy of
// its tokens (zero padded to d_pad) and clears the experts' counts.
template <typename X, typename R>
__global__ __launch_bounds__(256) void moe_logits_kernel(const X* __restrict__ x, const R* __restrict__ router, int T, int d,
                                                         int d_pad, int E, int vec, float* __restrict__ logits,
                                                         uint16_t* __restrict__ xb, int32_t* __restrict__ count) {
    const int lane = threadIdx.x & 63;
    const int t0 = blockIdx.y * LT;
    if (blockIdx.x == gridDim.x - 1) {
        for (int i = threadIdx.x; i < LT * d_pad; i += 256) {
            const int t = t0 + i / d_pad, p = i % d_pad;
            if (t < T) xb[(int64_t)t * d_pad + p] = p < d ? bf16_rne(load1(x + (int64_t)t * d + p)) : 0;
        }
        if (blockIdx.y == 0)
            for (int e = threadIdx.x; e < E; e += 256) count[e] = 0;
        return;
    }
    const int e = blockIdx.x * 4 + (threadIdx.x >> 6);
    if (e >= E) return;
    const R* const w = router + (int64_t)e * d;
    float acc[LT];
    const X* xr[LT];
#pragma unroll
    for (int i = 0; i < LT; ++i) {
        acc[i] = 0.0f;
        xr[i] = x + (int64_t)(t0 + i < T ? t0 + i : T - 1) * d;
    }
    int p = 0;
    if (vec) {
        for (p = lane * 8; p + 8 <= d; p += 512) {
            float a[8], b[8];
            load8(w + p, a);
#pragma unroll
            for (int i = 0; i < LT; ++i) {
                load8(xr[i] + p, b);
#pragma unroll
                for (int j = 0; j < 8; ++j) acc[i] = __builtin_fmaf(a[j], b[j], acc[i]);
            }
        }
    } else {
        for (p = lane; p < d; p += 64) {
            const float a = load1(w + p);
#pragma unroll
            for (int i = 0; i < LT; ++i) acc[i] = __builtin_fmaf(a, load1(xr[i] + p), acc[i]);
        }
    }
#pragma unroll
    for (int i = 0; i < LT; ++i) {
#pragma unroll
        for (int o = 32; o; o >>= 1) acc[i] += __shfl_xor(acc[i], o);
        if (lane == 0 && t0 + i < T) logits[(int64_t)(t0 + i) * E + e] = acc[i];
    }
}

// ---------------------------------------------------------------- products

// Byte offset of this lane's first 16 codes of the 16-row half block `half` of a 32-row run.
__device__ __forceinline__ int lane_off(int half) {
    const int lane = threadIdx.x & 63, r = lane & 15, g = lane >> 4;
    return (g >> 1) * 2048 + ((g & 1) * 32 + half * 16 + r) * 16;
}

struct Codes {
    uint4 lo, hi;   // a lane's 32 codes of one block
};
__device__ __forceinline__ Codes load_codes(const uint8_t* p) {
    return Codes{*reinterpret_cast<const uint4*>(p), *reinterpret_cast<const uint4*>(p + 1024)};
}
// acc += scale * (16 rows x 128 inputs of codes) . (128 inputs x 16 tokens); x: this lane's
// 32 consecutive bf16 values of its token.
__device__ __forceinline__ void block_mma(v4f& acc, const Codes& c, const uint4* x, float scale) {
    const uint32_t w[8] = {c.lo.x, c.lo.y, c.lo.z, c.lo.w, c.hi.x, c.hi.y, c.hi.z, c.hi.w};
    v4f t = v4f{0, 0, 0, 0};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(widen_e4m3(w[2 * j], w[2 * j + 1]), __builtin_bit_cast(v8bf, x[j]), t, 0, 0, 0);
#pragma unroll
    for (int r = 0; r < 4; ++r) acc[r] = __builtin_fmaf(t[r], scale, acc[r]);
}

struct UpArgs {
    const float* logits;
    const uint16_t* xb;
    int32_t *ids, *count, *pairs;
    float* p;
    uint16_t* h;
    int T, E, k, renorm, f, by_slot;
    int nkb_d, f_pad, n_pad;                 // d blocks of 128, roundup(f, 128), roundup(f, 32)
    const uint8_t *gate, *up;
    const float *gate_s, *up_s;
    int64_t mat_codes, mat_scales;           // bytes / scales per expert
};

// ---------------------------------------------------------------- 2. up

template <bool GATED, int NT>
__device__ __forceinline__ void up_chunk(const UpArgs& a, int e, int row0, const int32_t* list, int c0, int n, float* red) {
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    constexpr int NM = GATED ? 2 : 1, LD = 20;
    const int64_t cofs = (int64_t)e * a.mat_codes + (int64_t)(row0 / 32) * a.nkb_d * 4096 + lane_off((row0 >> 4) & 1);
    const int64_t sofs = (int64_t)e * a.mat_scales + (int64_t)(row0 / 128) * a.nkb_d;
    const uint16_t* xp[NT];
#pragma unroll
    for (int i = 0; i < NT; ++i) {
        const int q = c0 + i * 16 + r;
        xp[i] = a.xb + (int64_t)(list[q < n ? q : c0] / a.k) * a.nkb_d * 128 + g * 32;
    }
    v4f acc[NM][NT];
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i) acc[m][i] = v4f{0, 0, 0, 0};
    for (int kb = wave; kb < a.nkb_d; kb += WAVES) {
        Codes w[NM];
        float s[NM];
        w[0] = load_codes(a.up + cofs + (int64_t)kb * 4096);
        s[0] = a.up_s[sofs + kb];
        if constexpr (GATED) {
            w[1] = load_codes(a.gate + cofs + (int64_t)kb * 4096);
            s[1] = a.gate_s[sofs + kb];
        }
#pragma unroll
        for (int i = 0; i < NT; ++i) {
            uint4 x[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4*>(xp[i] + kb * 128 + 8 * j);
#pragma unroll
            for (int m = 0; m < NM; ++m) block_mma(acc[m][i], w[m], x, s[m]);
        }
    }
    // lane: token r of tile i, rows 4 g .. 4 g + 3
#pragma unroll
    for (int m = 0; m < NM; ++m)
#pragma unroll
        for (int i = 0; i < NT; ++i)
            *reinterpret_cast<v4f*>(red + (((m * WAVES + wave) * NT + i) * 16 + r) * LD + 4 * g) = acc[m][i];
    __syncthreads();
    for (int i = tid; i < NT * 256; i += WAVES * 64) {
        const int tok = i >> 4, row = i & 15;
        if (c0 + tok < n) {
            float u = 0.0f, v = 0.0f;
#pragma unroll
            for (int w = 0; w < WAVES; ++w) {
                u += red[(w * NT * 16 + tok) * LD + row];
                if constexpr (GATED) v += red[((WAVES + w) * NT * 16 + tok) * LD + row];
            }
            float y;
            if constexpr (GATED) y = v / (1.0f + expf(-v)) * u;
            else y = gelu_tanh_f32(u);
            a.h[(int64_t)list[c0 + tok] * a.f_pad + row0 + row] = row0 + row < a.f ? bf16_rne(y) : 0;
        }
    }
    __syncthreads();
}

template <bool GATED>
__global__ __launch_bounds__(WAVES * 64) void moe_up_kernel(UpArgs a) {
    __shared__ int32_t list[MAX_T];
    __shared__ int32_t rank[MAX_T];
    __shared__ uint32_t top[MAX_T];          // key of the token's largest logit
    __shared__ int32_t head[2];              // expert, tokens of it
    __shared__ uint32_t keys[W4A4_MOE_MAX_E];
    __shared__ __attribute__((aligned(16))) float red[(GATED ? 2 : 1) * WAVES * 4 * 16 * 20];
    const int tid = threadIdx.x, lane = tid & 63;
    const int row0 = blockIdx.x * 16;

    // Which expert: the grid's second dimension counts experts, or, where the tokens choose
    // fewer than there are, slots t * k + rank; a slot whose expert an earlier token chose too is
    // left to that token's slot.
    int e = blockIdx.y;
    if (a.by_slot) {
        const int t = blockIdx.y / a.k, want = blockIdx.y - t * a.k;
        for (int i = tid; i < a.E; i += WAVES * 64) keys[i] = rank_key(a.logits[(int64_t)t * a.E + i]);
        __syncthreads();
        for (int i = tid; i < a.E; i += WAVES * 64) {
            const uint32_t key = keys[i];
            int c = 0;
            for (int j = 0; j < a.E; ++j) c += before(keys[j], j, key, i) ? 1 : 0;
            if (c == want) head[0] = i;
        }
        __syncthreads();
        e = head[0];
    }
    // The rank of e in every token: eight lanes a token.
    for (int t = tid >> 3; t < a.T; t += WAVES * 8) {
        const float* l = a.logits + (int64_t)t * a.E;
        const uint32_t key = rank_key(l[e]);
        int c = 0;
        uint32_t m = 0;
        for (int j = tid & 7; j < a.E; j += 8) {
            const uint32_t kj = rank_key(l[j]);
            c += before(kj, j, key, e) ? 1 : 0;
            m = max(m, kj);
        }
#pragma unroll
        for (int o = 1; o < 8; o *= 2) {
            c += __shfl_xor(c, o);
            m = max(m, (uint32_t)__shfl_xor((int)m, o));
        }
        if ((tid & 7) == 0) {
            rank[t] = c;
            top[t] = m;
        }
    }
    __syncthreads();
    if (tid < 64) {
        int n = 0;
        for (int t0 = 0; t0 < a.T; t0 += 64) {
            const int t = t0 + lane;
            const bool in = t < a.T && rank[t < a.T ? t : 0] < a.k;
            const uint64_t b = __ballot(in);
            if (in) list[n + __popcll(b & ((1ull << lane) - 1))] = t * a.k + rank[t];
            n += __popcll(b);
        }
        if (lane == 0) head[1] = n;
    }
    __syncthreads();
    const int n = head[1];
    if (n == 0 || (a.by_slot && list[0] < (int)blockIdx.y)) return;

    if (blockIdx.x == 0) {   // what the down step reads of the routing, once per expert
        if (tid == 0) a.count[e] = n;
        for (int q = tid >> 3; q < n; q += WAVES * 8) {
            const int pair = list[q], t = pair / a.k;
            const float* l = a.logits + (int64_t)t * a.E;
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
                a.p[pair] = v;
                a.pairs[(int64_t)e * a.T + q] = pair;
            }
        }
    }
    if (row0 >= a.n_pad) {   // past the packed rows: only h's padding
        for (int i = tid; i < n * 16; i += WAVES * 64) a.h[(int64_t)list[i >> 4] * a.f_pad + row0 + (i & 15)] = 0;
        return;
    }
    for (int c0 = 0; c0 < n;) {
        const int left = n - c0;
        if (left <= 16) {
            up_chunk<GATED, 1>(a, e, row0, list, c0, n, red);
            c0 += 16;
        } else if (left <= 32) {
            up_chunk<GATED, 2>(a, e, row0, list, c0, n, red);
            c0 += 32;
        } else {
            up_chunk<GATED, 4>(a, e, row0, list, c0, n, red);
            c0 += 64;
        }
    }
}

// ---------------------------------------------------------------- 3. down

struct DownArgs {
    const int32_t *count, *pairs;
    const float* p;
    const uint16_t* h;
    int T, E, k, renorm, d;
    int nkb_f;                               // f blocks of 128
    const uint8_t* codes;
    const float* scales;
    int64_t mat_codes, mat_scales;
    void* out;
};

// TB: tokens the sums are laid out for.  The wavefronts share the (expert, block) sequence in
// equal consecutive ranges; each adds to sums of its own, which are added in wavefront order.
template <int TB, int OUT>
__global__ __launch_bounds__(WAVES * 64) void moe_down_kernel(DownArgs a) {
    __shared__ __attribute__((aligned(16))) float sums[WAVES * TB * 16];
    __shared__ float den[TB];
    __shared__ uint16_t active[W4A4_MOE_MAX_E];
    __shared__ int n_active;
    const int tid = threadIdx.x, lane = tid & 63, r = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int row0 = blockIdx.x * 16;
    for (int i = tid; i < WAVES * TB * 16; i += WAVES * 64) sums[i] = 0.0f;
    for (int t = tid; t < a.T; t += WAVES * 64) {
        float s = 1.0f;
        if (a.renorm) {
            s = 0.0f;
            for (int j = 0; j < a.k; ++j) s += a.p[t * a.k + j];
        }
        den[t] = s;
    }
    if (tid < 64) {
        int n = 0;
        for (int e0 = 0; e0 < a.E; e0 += 64) {
            const bool in = e0 + lane < a.E && a.count[e0 + lane] > 0;
            const uint64_t b = __ballot(in);
            if (in) active[n + __popcll(b & ((1ull << lane) - 1))] = (uint16_t)(e0 + lane);
            n += __popcll(b);
        }
        if (lane == 0) n_active = n;
    }
    __syncthreads();
    const int total = n_active * a.nkb_f;
    int pos = (int)((int64_t)total * wave / WAVES);
    const int end = (int)((int64_t)total * (wave + 1) / WAVES);
    float* const mine = sums + wave * TB * 16;
    while (pos < end) {
        const int ai = pos / a.nkb_f, kb0 = pos - ai * a.nkb_f;
        const int kb1 = end - pos < a.nkb_f - kb0 ? kb0 + (end - pos) : a.nkb_f;
        pos += kb1 - kb0;
        const int e = active[ai];
        const int n = a.count[e];
        const int32_t* const list = a.pairs + (int64_t)e * a.T;
        const uint8_t* const wp = a.codes + (int64_t)e * a.mat_codes + (int64_t)(row0 / 32) * a.nkb_f * 4096 + lane_off((row0 >> 4) & 1);
        const float* const sp = a.scales + (int64_t)e * a.mat_scales + (int64_t)(row0 / 128) * a.nkb_f;
        for (int c0 = 0; c0 < n; c0 += 16) {
            const int q = c0 + r;
            const int pair = list[q < n ? q : c0];
            const uint16_t* const hp = a.h + (int64_t)pair * a.nkb_f * 128 + g * 32;
            v4f acc = v4f{0, 0, 0, 0};
            for (int kb = kb0; kb < kb1; ++kb) {
                const Codes w = load_codes(wp + (int64_t)kb * 4096);
                uint4 x[4];
#pragma unroll
                for (int j = 0; j < 4; ++j) x[j] = *reinterpret_cast<const uint4*>(hp + kb * 128 + 8 * j);
                block_mma(acc, w, x, sp[kb]);
            }
            if (q < n) {   // tokens of one expert are distinct: no two lanes meet
                const int t = pair / a.k;
                const float pw = a.renorm ? a.p[pair] / den[t] : a.p[pair];
                v4f* const s = reinterpret_cast<v4f*>(mine + t * 16 + 4 * g);
                v4f v = *s;
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i] = __builtin_fmaf(acc[i], pw, v[i]);
                *s = v;
            }
        }
    }
    __syncthreads();
    for (int i = tid; i < a.T * 16; i += WAVES * 64) {
        const int t = i >> 4, row = row0 + (i & 15);
        if (row >= a.d) continue;
        float y = 0.0f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) y += sums[w * TB * 16 + i];
        if constexpr (OUT == W4A4_Y_F32) reinterpret_cast<float*>(a.out)[(int64_t)t * a.d + row] = y;
        else reinterpret_cast<uint16_t*>(a.out)[(int64_t)t * a.d + row] = bf16_rne(y);
    }
}

template <typename X>
void run_logits(const void* X_, const w4a4_moe& m, int T, float* logits, uint16_t* xb, int32_t* count, hipStream_t st) {
    const int d = (int)m.up.d_in, d_pad = (int)m.up.k_pad, E = (int)m.up.n_mat;
    const dim3 grid((uint32_t)((E + 3) / 4 + 1), (uint32_t)((T + LT - 1) / LT));
    const int vec = d % 8 == 0 ? 1 : 0;
    if (m.router_dtype == W4A4_X_BF16)
        hipLaunchKernelGGL((moe_logits_kernel<X, uint16_t>), grid, dim3(256), 0, st, (const X*)X_, (const uint16_t*)m.router, T, d,
                           d_pad, E, vec, logits, xb, count);
    else
        hipLaunchKernelGGL((moe_logits_kernel<X, float>), grid, dim3(256), 0, st, (const X*)X_, (const float*)m.router, T, d,
                           d_pad, E, vec, logits, xb, count);
}

template <int OUT>
void run_down(const DownArgs& a, dim3 grid, hipStream_t st) {
    const dim3 block(WAVES * 64);
    if (a.T <= 16) hipLaunchKernelGGL((moe_down_kernel<16, OUT>), grid, block, 0, st, a);
    else if (a.T <= 64) hipLaunchKernelGGL((moe_down_kernel<64, OUT>), grid, block, 0, st, a);
    else hipLaunchKernelGGL((moe_down_kernel<MAX_T, OUT>), grid, block, 0, st, a);
}

}  // namespace

hipError_t launch_moe(const void* X, int x_dtype, int64_t T, const w4a4_moe& m, const MoeBuffers& b, void* Y, int y_dtype,
                      hipStream_t st) {
    if (x_dtype == W4A4_X_BF16) run_logits<uint16_t>(X, m, (int)T, b.logits, b.xb, b.count, st);
    else run_logits<float>(X, m, (int)T, b.logits, b.xb, b.count, st);
    hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;

    const bool gated = m.activation == W4A4_MOE_SILU_GATED;
    UpArgs u;
    u.logits = b.logits; u.xb = b.xb; u.ids = b.ids; u.count = b.count; u.pairs = b.pairs; u.p = b.p; u.h = b.h;
    u.T = (int)T; u.E = (int)m.up.n_mat; u.k = m.top_k; u.renorm = m.renormalize != 0; u.f = (int)m.up.d_out;
    u.by_slot = T * m.top_k < m.up.n_mat ? 1 : 0;
    u.nkb_d = (int)(m.up.k_pad / 128); u.f_pad = (int)m.down.k_pad; u.n_pad = (int)m.up.n_pad;
    u.gate = gated ? m.gate.codes : nullptr; u.gate_s = gated ? m.gate.scales : nullptr;
    u.up = m.up.codes; u.up_s = m.up.scales;
    u.mat_codes = m.up.n_pad * m.up.k_pad; u.mat_scales = (m.up.d_out + 127) / 128 * (m.up.k_pad / 128);
    const dim3 grid((uint32_t)(u.f_pad / 16), (uint32_t)(u.by_slot ? T * m.top_k : m.up.n_mat));
    if (gated) hipLaunchKernelGGL(moe_up_kernel<true>, grid, dim3(WAVES * 64), 0, st, u);
    else hipLaunchKernelGGL(moe_up_kernel<false>, grid, dim3(WAVES * 64), 0, st, u);
    e = hipGetLastError();
    if (e != hipSuccess) return e;

    DownArgs d;
    d.count = b.count; d.pairs = b.pairs; d.p = b.p; d.h = b.h;
    d.T = u.T; d.E = u.E; d.k = u.k; d.renorm = u.renorm; d.d = (int)m.down.d_out;
    d.nkb_f = (int)(m.down.k_pad / 128);
    d.codes = m.down.codes; d.scales = m.down.scales;
    d.mat_codes = m.down.n_pad * m.down.k_pad; d.mat_scales = (m.down.d_out + 127) / 128 * (m.down.k_pad / 128);
    d.out = Y;
    const dim3 gd((uint32_t)((d.d + 15) / 16));
    if (y_dtype == W4A4_Y_F32) run_down<W4A4_Y_F32>(d, gd, st);
    else run_down<W4A4_Y_BF16>(d, gd, st);
    return hipGetLastError();
}

}  // namespace w4a4

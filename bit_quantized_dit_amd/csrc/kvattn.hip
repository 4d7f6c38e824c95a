// Attention over the 4-bit key/value cache on gfx950:
//
//   O[row][j] = sum_t p_t v_t / sum_t p_t,  p_t = exp(scale (q . k_t) - m)
//
// in one pass over the cache with a running maximum and sum.  Rows of the heads that share a
// key/value head are stacked (row m = i * ratio + j), so every block of codes is read and
// widened once for all of them.  Scores are computed transposed, S^T = K Q^T: a lane of the result
// holds one row and a few tokens, so the softmax runs in the lane's own registers, and P^T is in the
// operand order of the second product O^T = V^T P^T as it stands, with the tokens of a value operand
// taken in the same order (which the cache's layout of the value codes provides).  Codes times a power
// of two are bf16 numbers, exactly: one conversion widens and scales two of them.
//
// The running maximum moves lazily: p_t = 2^(x_t - m) with m a maximum that is renewed only when
// a score passes it by more than 2^8, which leaves the result as it is (numerator and denominator
// carry the same factor) and spares most steps the exchange between lanes and the rescaling of O.
#include "kv_device.h"

namespace w4a4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float M_NONE = -3.0e38f;       // below every score that counts
constexpr float M_SLACK = 8.0f;

struct AttnArgs {
    KvArgs kv;
    const void* q;
    int64_t q_row, q_head;
    uint16_t* out;
    float *part_o, *part_ml;      // [unit][split][rows_cap][d_pad], [unit][split][rows_cap][2]
    int64_t window;
    float scale;                  // scale * log2(e)
    int32_t ratio, causal, nsplit, rows_cap;
};

// The steps of ST tokens that rows m0 .. m1 - 1 of a sequence see, cut into equal ranges.
template <int ST> struct Steps {
    int32_t start, n, chunk, active;
    __device__ Steps(const AttnArgs& a, const KvSeq& s, int32_t m0, int32_t m1) {
        const int64_t i0 = m0 / a.ratio, i1 = (m1 - 1) / a.ratio;
        int64_t lo = a.causal && a.window ? s.first + i0 - a.window + 1 : 0, hi = a.causal ? s.first + i1 + 1 : s.len;
        lo = lo < 0 ? 0 : lo / ST * ST;
        n = m1 > m0 && hi > lo ? (int32_t)((hi - lo + ST - 1) / ST) : 0;
        start = (int32_t)lo;
        constexpr int LEAST = 256 / ST;
        chunk = (n + a.nsplit - 1) / a.nsplit;
        chunk = chunk < LEAST ? LEAST : chunk;
        active = n > chunk ? (n + chunk - 1) / chunk : 1;
    }
};

template <int N> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    __builtin_memcpy(w, __builtin_assume_aligned(p, N % 4 == 0 ? 16 : N % 2 == 0 ? 8 : 4), 4 * N);
}
__device__ __forceinline__ float scale_of(uint32_t word, int byte) {
    return __uint_as_float(byte == 3 ? (word >> 1) & 0x7F800000u : (word << (23 - 8 * byte)) & 0x7F800000u);
}
template <int J> __device__ __forceinline__ uint32_t widen2(uint32_t w, float s) {
    return __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, J));
}
__device__ __forceinline__ v8bf join8(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __builtin_bit_cast(v8bf, make_uint4(a, b, c, d));
}
// 8 key channels of one token.
__device__ __forceinline__ v8bf widen_key(uint32_t w, float s) { return join8(widen2<0>(w, s), widen2<1>(w, s), widen2<2>(w, s), widen2<3>(w, s)); }
// 8 tokens (two dwords of four) of channels d and d + 16.
__device__ __forceinline__ void widen_value(uint32_t w0, uint32_t s0, uint32_t w1, uint32_t s1, v8bf& d, v8bf& d16) {
    uint32_t p[8] = {widen2<0>(w0, scale_of(s0, 0)), widen2<1>(w0, scale_of(s0, 1)), widen2<2>(w0, scale_of(s0, 2)), widen2<3>(w0, scale_of(s0, 3)),
                     widen2<0>(w1, scale_of(s1, 0)), widen2<1>(w1, scale_of(s1, 1)), widen2<2>(w1, scale_of(s1, 2)), widen2<3>(w1, scale_of(s1, 3))};
    uint32_t lo[4], hi[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        lo[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x05040100u);
        hi[i] = __builtin_amdgcn_perm(p[2 * i + 1], p[2 * i], 0x07060302u);
    }
    d = join8(lo[0], lo[1], lo[2], lo[3]);
    d16 = join8(hi[0], hi[1], hi[2], hi[3]);
}
// Scale codes of tokens that no row may multiply with: codes above 252 (a NaN's 0xFF, or memory that
// was never written) become 0, so that zero times the value is zero.  `nan` gets a bit per 0xFF.
__device__ __forceinline__ uint32_t tame(uint32_t w, uint32_t& nan) {
    uint32_t o = 0;
    nan = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        const uint32_t c = w >> (8 * j) & 0xFFu;
        o |= (c > 252u ? 0u : c) << (8 * j);
        nan |= (c == 0xFFu ? 1u : 0u) << j;
    }
    return o;
}
// Whether any byte of w is above 251 (tame may have something to do).
__device__ __forceinline__ bool wild(uint32_t w) {
    const uint32_t t = ~w & 0xFCFCFCFCu;
    return ((t - 0x01010101u) & ~t & 0x80808080u) != 0;
}

__device__ __forceinline__ void load_q8(const AttnArgs& a, int64_t at, int p, bool bf16, float* x) {
    if (bf16) load8((const uint16_t*)a.q + at, p, a.kv.head_dim, x);
    else load8((const float*)a.q + at, p, a.kv.head_dim, x);
}
__device__ __forceinline__ v8bf pack_q(const float* x) { return join8(pk_bf16(x[0], x[1]), pk_bf16(x[2], x[3]), pk_bf16(x[4], x[5]), pk_bf16(x[6], x[7])); }

// Four outputs of a row from channel d on.
__device__ __forceinline__ void store_out4(uint16_t* row, int d, int D, v4f v) {
    const uint32_t w[2] = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
    if (d + 4 <= D && (D & 3) == 0) {
        *reinterpret_cast<uint2*>(row + d) = make_uint2(w[0], w[1]);
        return;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < D) row[d + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

// ---------------------------------------------------------------- few rows
//
// Up to 16 MT stacked rows: bound by reading the cache.  A wavefront takes every fourth step of
// 32 tokens of its workgroup's range, codes straight from memory into registers with the next
// step's in flight; the wavefronts' results meet in LDS.
template <int G, int MT, bool QB>
__global__ __launch_bounds__(256) void kv_few_kernel(AttnArgs a) {
    typedef KvBlock<G> L;
    constexpr int DP = 32 * G, LD = DP + 4, NW = 4;
    __shared__ __attribute__((aligned(16))) float red[NW][16][LD];
    __shared__ float red_m[NW][MT][16], red_l[NW][MT][16];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int64_t unit = blockIdx.x / a.nsplit;
    const int sp = blockIdx.x % a.nsplit;
    const int64_t b = unit / a.kv.n_heads;
    const int h = (int)(unit - b * a.kv.n_heads);
    const KvSeq s = kv_seq(a.kv, b);
    const int rows = s.done * a.ratio;
    const Steps<32> st(a, s, 0, rows);
    if (rows == 0 || sp >= st.active) return;
    const int s0 = sp * st.chunk, s1 = s0 + st.chunk < st.n ? s0 + st.chunk : st.n;

    // this lane's rows: the operand of each block of 32 channels, and the tokens they see
    v8bf q[MT][G];
    int32_t lo[MT], hi[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        const int m = mt * 16 + c, i = m / a.ratio, j = m - i * a.ratio;
        const bool on = m < rows;
        const int64_t at = on ? (s.row0 + i) * a.q_row + (int64_t)(h * a.ratio + j) * a.q_head : 0;
#pragma unroll
        for (int d = 0; d < G; ++d) {
            float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (on) load_q8(a, at, 32 * d + 8 * g, QB, x);
            q[mt][d] = pack_q(x);
        }
        const int64_t pos = (int64_t)s.first + i, from = a.causal && a.window ? pos - a.window + 1 : 0;
        lo[mt] = from < 0 ? 0 : (int32_t)from;
        hi[mt] = on && a.causal ? (int32_t)pos : s.len - 1;
    }
    // tokens that every row sees
    const int32_t all_hi = a.causal ? s.first : s.len - 1;
    const int64_t last_from = a.causal && a.window ? (int64_t)s.first + s.done - a.window : 0;

    v4f acc[MT][2 * G];
    float mx[MT], sum[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        mx[mt] = M_NONE;
        sum[mt] = 0.0f;
#pragma unroll
        for (int t = 0; t < 2 * G; ++t) acc[mt][t] = v4f{0, 0, 0, 0};
    }

    struct Codes {
        uint32_t k[2][G], v[2][G], ks[2][(G + 3) / 4], vs[2][G];
        bool there[2];
    };
    Codes buf[2];
    // block addresses of 32 steps at a time, two a step, one a lane
    for (int k0 = s0 + wave; k0 < s1; k0 += 32 * NW) {
        const int mine = k0 + (lane >> 1) * NW;
        uint64_t addr = 0;
        if (mine < s1) addr = (uint64_t)(uintptr_t)kv_block(a.kv, b, (uint32_t)(st.start / 16 + 2 * mine + (lane & 1)), h);
        auto fetch = [&](Codes& x, int k) __attribute__((always_inline)) {
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const uint32_t al = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)addr, 2 * k + u);
                const uint32_t ah = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(addr >> 32), 2 * k + u);
                const uint8_t* p = (const uint8_t*)(uintptr_t)((uint64_t)ah << 32 | al);
                x.there[u] = p != nullptr;
                p = p ? p : a.kv.data;
                load_words<G>(p + lane * 4 * G, x.k[u]);
                load_words<G>(p + L::V + lane * 4 * G, x.v[u]);
                load_words<G>(p + L::VS + g * 4 * L::SG, x.vs[u]);
                if constexpr (G == 1) x.ks[u][0] = p[L::KS + c];
                else if constexpr (G == 2) x.ks[u][0] = *reinterpret_cast<const uint16_t*>(p + L::KS + c * 2);
                else load_words<(G + 3) / 4>(p + L::KS + c * L::SG, x.ks[u]);
            }
        };
        auto compute = [&](Codes& x, int pos) __attribute__((always_inline)) {      // pos: the step's first token
            const bool full = pos + 31 <= all_hi && pos >= last_from && x.there[0] && x.there[1];
            v4f sc[MT][2];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) sc[mt][0] = sc[mt][1] = v4f{0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < G; ++d) {
                    const v8bf kf = widen_key(x.k[u][d], scale_of(x.ks[u][d / 4], d & 3));
#pragma unroll
                    for (int mt = 0; mt < MT; ++mt) sc[mt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[mt][d], sc[mt][u], 0, 0, 0);
                }
            uint32_t bad[MT];      // groups whose values are NaN for this lane's row
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) bad[mt] = 0;
            if (!full) {
                uint32_t seen[MT][2];      // bit i: token 4 g + i of the block is seen by the row
#pragma unroll
                for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        seen[mt][u] = 0;
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            const int t = pos + 16 * u + 4 * g + i;
                            const bool see = t >= lo[mt] && t <= hi[mt] && x.there[u];
                            seen[mt][u] |= see ? 1u << i : 0u;
                            sc[mt][u][i] = see ? sc[mt][u][i] : -__builtin_inff();
                        }
                    }
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int d = 0; d < G; ++d) {
                        uint32_t nan;
                        x.vs[u][d] = tame(x.vs[u][d], nan);
#pragma unroll
                        for (int mt = 0; mt < MT; ++mt) bad[mt] |= (nan & seen[mt][u]) ? 1u << d : 0u;
                    }
            }
            v8bf ph[MT], pl[MT];
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                float top = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(sc[mt][0][0], sc[mt][0][1]), __builtin_fmaxf(sc[mt][0][2], sc[mt][0][3])),
                                            __builtin_fmaxf(__builtin_fmaxf(sc[mt][1][0], sc[mt][1][1]), __builtin_fmaxf(sc[mt][1][2], sc[mt][1][3])));
                top *= a.scale;
                if (__any(top > mx[mt] + M_SLACK)) {
                    top = __builtin_fmaxf(top, __shfl_xor(top, 16));
                    top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                    const float m = __builtin_fmaxf(mx[mt], top), f = __builtin_amdgcn_exp2f(mx[mt] - m);
                    mx[mt] = m;
                    sum[mt] *= f;
#pragma unroll
                    for (int t = 0; t < 2 * G; ++t) acc[mt][t] *= f;
                }
                float p[8];
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[mt][i >> 2][i & 3], a.scale, -mx[mt]));
                    sum[mt] += p[i];
                }
                uint32_t ph_[4], pl_[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    ph_[i] = pk_bf16(p[2 * i], p[2 * i + 1]);
                    pl_[i] = pk_bf16(p[2 * i] - __uint_as_float(ph_[i] << 16), p[2 * i + 1] - __uint_as_float(ph_[i] & 0xFFFF0000u));
                }
                ph[mt] = join8(ph_[0], ph_[1], ph_[2], ph_[3]);
                pl[mt] = join8(pl_[0], pl_[1], pl_[2], pl_[3]);
            }
#pragma unroll
            for (int d = 0; d < G; ++d) {
                v8bf v0, v1;
                widen_value(x.v[0][d], x.vs[0][d], x.v[1][d], x.vs[1][d], v0, v1);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    acc[mt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, ph[mt], acc[mt][2 * d], 0, 0, 0);
                    acc[mt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[mt], acc[mt][2 * d], 0, 0, 0);
                    acc[mt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, ph[mt], acc[mt][2 * d + 1], 0, 0, 0);
                    acc[mt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[mt], acc[mt][2 * d + 1], 0, 0, 0);
                }
            }
            if (!full) {
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    bad[mt] |= (uint32_t)__shfl_xor((int)bad[mt], 16);
                    bad[mt] |= (uint32_t)__shfl_xor((int)bad[mt], 32);
#pragma unroll
                    for (int d = 0; d < G; ++d)
                        if (bad[mt] >> d & 1) acc[mt][2 * d] = acc[mt][2 * d + 1] = acc[mt][2 * d] + __uint_as_float(0x7FC00000u);
                }
            }
        };
        const int left = (s1 - k0 + NW - 1) / NW, steps = left < 32 ? left : 32;
        fetch(buf[0], 0);
        for (int k = 0; k < steps; k += 2) {
            if (k + 1 < steps) fetch(buf[1], k + 1);
            compute(buf[0], st.start + (k0 + k * NW) * 32);
            if (k + 1 < steps) {
                if (k + 2 < steps) fetch(buf[0], k + 2);
                compute(buf[1], st.start + (k0 + (k + 1) * NW) * 32);
            }
        }
    }

    // the wavefronts' results: one maximum, then the sums of 16 rows at a time
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        sum[mt] += __shfl_xor(sum[mt], 16);
        sum[mt] += __shfl_xor(sum[mt], 32);
        if (g == 0) {
            red_m[wave][mt][c] = mx[mt];
            red_l[wave][mt][c] = sum[mt];
        }
    }
    __syncthreads();
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        if (mt * 16 >= rows) break;      // uniform over the workgroup
        float m = red_m[0][mt][c];
#pragma unroll
        for (int w = 1; w < NW; ++w) m = __builtin_fmaxf(m, red_m[w][mt][c]);
        const float f = __builtin_amdgcn_exp2f(mx[mt] - m);
#pragma unroll
        for (int t = 0; t < 2 * G; ++t) *reinterpret_cast<v4f*>(&red[wave][c][16 * t + 4 * g]) = acc[mt][t] * f;
        __syncthreads();
        for (int e = threadIdx.x; e < 16 * (DP / 4); e += 256) {
            const int col = e / (DP / 4), d = e % (DP / 4) * 4, row = mt * 16 + col;
            if (row >= rows) continue;
            float top = red_m[0][mt][col], l = 0.0f;
#pragma unroll
            for (int w = 1; w < NW; ++w) top = __builtin_fmaxf(top, red_m[w][mt][col]);
            v4f o = v4f{0, 0, 0, 0};
#pragma unroll
            for (int w = 0; w < NW; ++w) {
                l += red_l[w][mt][col] * __builtin_amdgcn_exp2f(red_m[w][mt][col] - top);
                o += *reinterpret_cast<const v4f*>(&red[w][col][d]);
            }
            if (st.active == 1) {
                const int i = row / a.ratio, j = row - i * a.ratio;
                const float r = l == 0.0f ? 0.0f : 1.0f / l;
                store_out4(a.out + ((s.row0 + i) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + j) * a.kv.head_dim, d, a.kv.head_dim, o * r);
            } else {
                const int64_t at = (unit * a.nsplit + sp) * a.rows_cap + row;
                *reinterpret_cast<v4f*>(a.part_o + at * DP + d) = o;
                if (d == 0) {
                    a.part_ml[2 * at] = top;
                    a.part_ml[2 * at + 1] = l;
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- many rows
//
// A workgroup owns 32 rows a wavefront and walks tiles of 64 tokens.  The tile's codes are widened
// once, a block of 16 tokens a wavefront, into two LDS buffers that take turns; the codes of the tile after
// are in flight meanwhile.  Rows of LDS are 16 bytes longer than their data, so that the
// operand reads of 16 lanes touch every bank once.
template <int G, int NW, bool QB>
__global__ __launch_bounds__(NW * 64) void kv_many_kernel(AttnArgs a, uint32_t row_tiles) {
    typedef KvBlock<G> L;
    constexpr int DP = 32 * G, KLD = 64 * G + 16, VLD = 144, KB = 64 * KLD, VB = DP * VLD, BUF = KB + VB, ROWS = 32 * NW;
    constexpr int NB = (G + 1) / 2;                        // value groups a lane converts
    static_assert(NW == 4, "a wavefront widens one of the tile's four blocks");
    __shared__ __attribute__((aligned(16))) uint8_t lds[2][BUF];
    __shared__ uint32_t flags[2][4];                       // of a block: 1 values that are NaN, 2 not there
    __shared__ uint8_t nans[2][64];                        // a token's groups that are NaN
    const int lane = threadIdx.x & 63, c = lane & 31, h2 = lane >> 5, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const int sp = blockIdx.x % a.nsplit;
    const uint32_t rest = blockIdx.x / a.nsplit;
    const int tile = (int)(row_tiles - 1 - rest % row_tiles);      // the rows that see most first
    const int64_t unit = rest / row_tiles;
    const int64_t b = unit / a.kv.n_heads;
    const int h = (int)(unit - b * a.kv.n_heads);
    const KvSeq s = kv_seq(a.kv, b);
    const int64_t all_rows = (int64_t)s.done * a.ratio;
    const int64_t m0 = (int64_t)tile * ROWS;
    if (m0 >= all_rows) return;
    const int rows = (int)(all_rows - m0 < ROWS ? all_rows - m0 : ROWS);
    const Steps<64> st(a, s, (int32_t)m0, (int32_t)(m0 + rows));
    if (sp >= st.active) return;
    const int s0 = sp * st.chunk, s1 = s0 + st.chunk < st.n ? s0 + st.chunk : st.n;

    const int m = (int)m0 + wave * 32 + c, qi = m / a.ratio, qj = m - qi * a.ratio;
    const bool on = wave * 32 + c < rows;
    v8bf q[2 * G];
    {
        const int64_t at = on ? (s.row0 + qi) * a.q_row + (int64_t)(h * a.ratio + qj) * a.q_head : 0;
#pragma unroll
        for (int d = 0; d < 2 * G; ++d) {
            float x[8] = {0, 0, 0, 0, 0, 0, 0, 0};
            if (on) load_q8(a, at, 16 * d + 8 * h2, QB, x);
            q[d] = pack_q(x);
        }
    }
    const int64_t pos = (int64_t)s.first + qi, from = a.causal && a.window ? pos - a.window + 1 : 0;
    const int32_t lo = from < 0 ? 0 : (int32_t)from, hi = !on ? -1 : a.causal ? (int32_t)pos : s.len - 1;
    // the wavefront's rows: tokens that any of them sees, and that all of them see
    const int w0 = wave * 32, w1 = w0 + 32 < rows ? w0 + 32 : rows;
    const bool idle = w0 >= rows;
    const int64_t i0 = ((int)m0 + w0) / a.ratio, i1 = ((int)m0 + (idle ? w0 : w1 - 1)) / a.ratio;
    const int64_t any_hi = idle ? -1 : a.causal ? s.first + i1 : s.len - 1, all_hi = a.causal ? s.first + i0 : s.len - 1;
    const int64_t any_lo = a.causal && a.window ? s.first + i0 - a.window + 1 : 0, all_lo = a.causal && a.window ? s.first + i1 - a.window + 1 : 0;

    v16f acc[G];
#pragma unroll
    for (int d = 0; d < G; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float mx = M_NONE, sum = 0.0f;

    // codes of one block: keys of token r16; values of tokens 4 hh .. and 8 + 4 hh .., groups from gb on
    const int hh = g & 1, gb = (g >> 1) * NB;
    uint32_t kw[G], ks[(G + 3) / 4], vw[2][NB], vs[2][NB];
    bool there;
    auto fetch = [&](int step) __attribute__((always_inline)) {
        const uint8_t* p = kv_block(a.kv, b, (uint32_t)(st.start / 16 + 4 * step + wave), h);
        there = p != nullptr;
        p = p ? p : a.kv.data;
        load_words<G>(p + lane * 4 * G, kw);
        if constexpr (G == 1) ks[0] = p[L::KS + r16];
        else if constexpr (G == 2) ks[0] = *reinterpret_cast<const uint16_t*>(p + L::KS + r16 * 2);
        else load_words<(G + 3) / 4>(p + L::KS + r16 * L::SG, ks);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < NB; ++d) {
                const int gd = gb + d < G ? gb + d : G - 1;
                vw[u][d] = *reinterpret_cast<const uint32_t*>(p + L::V + ((hh + 2 * u) * 16 + r16) * 4 * G + 4 * gd);
                vs[u][d] = *reinterpret_cast<const uint32_t*>(p + L::VS + (hh + 2 * u) * 4 * L::SG + 4 * gd);
            }
    };
    auto widen = [&](int slot) __attribute__((always_inline)) {
        uint8_t* const kd = lds[slot] + (wave * 16 + r16) * KLD + g * 16;
#pragma unroll
        for (int d = 0; d < G; ++d) *reinterpret_cast<v8bf*>(kd + d * 64) = widen_key(kw[d], scale_of(ks[d / 4], d & 3));
        bool odd = false;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < NB; ++d) odd |= wild(vs[u][d]);
        uint32_t flag = there ? 0u : 2u;
        if (__any(odd)) {      // rare: values that are NaN go by a list of their own
            uint32_t bits[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < NB; ++d) {
                    uint32_t nan;
                    vs[u][d] = tame(vs[u][d], nan);
#pragma unroll
                    for (int j = 0; j < 4; ++j) bits[4 * u + j] |= gb + d < G && (nan >> j & 1) ? 1u << (gb + d) : 0u;
                }
#pragma unroll
            for (int k = 0; k < 8; ++k) bits[k] |= (uint32_t)__shfl_xor((int)bits[k], 32);      // the other half of the groups
            if (r16 == 0 && g < 2)
#pragma unroll
                for (int k = 0; k < 8; ++k) nans[slot][wave * 16 + 4 * hh + (k >> 2) * 8 + (k & 3)] = (uint8_t)bits[k];
            flag |= 1u;
        }
        if (lane == 0) flags[slot][wave] = flag;
        uint8_t* const vd = lds[slot] + KB + r16 * VLD + (2 * wave + hh) * 16;
#pragma unroll
        for (int d = 0; d < NB; ++d) {
            if (gb + d >= G) continue;
            v8bf v0, v1;
            widen_value(vw[0][d], vs[0][d], vw[1][d], vs[1][d], v0, v1);
            *reinterpret_cast<v8bf*>(vd + (gb + d) * 32 * VLD) = v0;
            *reinterpret_cast<v8bf*>(vd + ((gb + d) * 32 + 16) * VLD) = v1;
        }
    };

    if (s0 < s1) {
        fetch(s0);
        widen(0);
        if (s0 + 1 < s1) fetch(s0 + 1);
    }
    for (int k = s0; k < s1; ++k) {
        const int slot = (k - s0) & 1;
        __syncthreads();
        const int64_t t0 = st.start + (int64_t)k * 64;
        const uint32_t fl = flags[slot][0] | flags[slot][1] | flags[slot][2] | flags[slot][3];
#pragma unroll
        for (int half = 0; half < 2; ++half) {      // 32 tokens
            const int64_t p0 = t0 + 32 * half;
            if (p0 > any_hi || p0 + 31 < any_lo) continue;
            v16f sc;
#pragma unroll
            for (int i = 0; i < 16; ++i) sc[i] = 0.0f;
            const uint8_t* const kp = lds[slot] + (half * 32 + c) * KLD + h2 * 16;
#pragma unroll
            for (int d = 0; d < 2 * G; ++d)
                sc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const v8bf*>(kp + d * 32), q[d], sc, 0, 0, 0);
            if (p0 + 31 > all_hi || p0 < all_lo || (fl & 2)) {
#pragma unroll
                for (int i = 0; i < 16; ++i) {
                    const int32_t t = (int32_t)p0 + 8 * (i >> 2) + 4 * h2 + (i & 3);
                    const bool see = t >= lo && t <= hi && !(flags[slot][2 * half + (i >> 3)] & 2);
                    sc[i] = see ? sc[i] : -__builtin_inff();
                }
            }
            float top = sc[0];
#pragma unroll
            for (int i = 1; i < 16; ++i) top = __builtin_fmaxf(top, sc[i]);
            top *= a.scale;
            if (__any(top > mx + M_SLACK)) {
                top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                const float mn = __builtin_fmaxf(mx, top), f = __builtin_amdgcn_exp2f(mx - mn);
                mx = mn;
                sum *= f;
#pragma unroll
                for (int d = 0; d < G; ++d) acc[d] *= f;
            }
            uint32_t pw[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float pa = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i], a.scale, -mx));
                const float pb = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[2 * i + 1], a.scale, -mx));
                sum += pa;
                sum += pb;
                pw[i] = pk_bf16(pa, pb);
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const v8bf pf = join8(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]);
                const uint8_t* const vp = lds[slot] + KB + c * VLD + ((half * 2 + u) * 2 + h2) * 16;
#pragma unroll
                for (int d = 0; d < G; ++d)
                    acc[d] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(*reinterpret_cast<const v8bf*>(vp + d * 32 * VLD), pf, acc[d], 0, 0, 0);
            }
            if (fl & 1) {
                uint32_t bad = 0;
                for (int t = 0; t < 32; ++t) {
                    if (!(flags[slot][2 * half + (t >> 4)] & 1)) continue;
                    const int32_t tp = (int32_t)p0 + t;
                    bad |= tp >= lo && tp <= hi && !(flags[slot][2 * half + (t >> 4)] & 2) ? nans[slot][half * 32 + t] : 0u;
                }
#pragma unroll
                for (int d = 0; d < G; ++d)
                    if (bad >> d & 1) {
#pragma unroll
                        for (int i = 0; i < 16; ++i) acc[d][i] = __uint_as_float(0x7FC00000u);
                    }
            }
        }
        if (k + 1 < s1) {
            widen(slot ^ 1);
            if (k + 2 < s1) fetch(k + 2);
        }
    }
    sum += __shfl_xor(sum, 32);
    if (!on) return;
    const float r = st.active > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = (unit * a.nsplit + sp) * a.rows_cap + m;
    uint16_t* const out = a.out + ((s.row0 + qi) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + qj) * a.kv.head_dim;
#pragma unroll
    for (int d = 0; d < G; ++d)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const v4f v = v4f{acc[d][4 * u] * r, acc[d][4 * u + 1] * r, acc[d][4 * u + 2] * r, acc[d][4 * u + 3] * r};
            const int ch = 32 * d + 8 * u + 4 * h2;
            if (st.active == 1) store_out4(out, ch, a.kv.head_dim, v);
            else *reinterpret_cast<v4f*>(a.part_o + at * DP + ch) = v;
        }
    if (st.active > 1 && h2 == 0) {
        a.part_ml[2 * at] = mx;
        a.part_ml[2 * at + 1] = sum;
    }
}

// The ranges' results of one row a wavefront: the common maximum, then the weighted sums.
template <int G, int ST, int ROWS>
__global__ __launch_bounds__(256) void kv_join_kernel(AttnArgs a) {
    constexpr int DP = 32 * G;
    const int lane = threadIdx.x & 63;
    const int64_t id = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
    const int64_t unit = id / a.rows_cap, b = unit / a.kv.n_heads;
    const int m = (int)(id - unit * a.rows_cap), h = (int)(unit - b * a.kv.n_heads);
    if (b >= a.kv.n_seqs) return;
    const KvSeq s = kv_seq(a.kv, b);
    const int rows = s.done * a.ratio;
    if (m >= rows) return;
    const int m0 = ROWS ? m / (ROWS ? ROWS : 1) * ROWS : 0, m1 = ROWS && m0 + ROWS < rows ? m0 + ROWS : rows;
    const Steps<ST> st(a, s, m0, m1);
    if (st.active == 1) return;
    const int64_t at = unit * a.nsplit * a.rows_cap + m;
    float top = M_NONE, l = 0.0f;
    for (int k = 0; k < st.active; ++k) top = __builtin_fmaxf(top, a.part_ml[2 * (at + (int64_t)k * a.rows_cap)]);
    v4f o = v4f{0, 0, 0, 0};
    for (int k = 0; k < st.active; ++k) {
        const int64_t p = at + (int64_t)k * a.rows_cap;
        const float f = __builtin_amdgcn_exp2f(a.part_ml[2 * p] - top);
        l += a.part_ml[2 * p + 1] * f;
        if (lane < DP / 4) o += *reinterpret_cast<const v4f*>(a.part_o + p * DP + 4 * lane) * f;
    }
    if (4 * lane >= a.kv.head_dim) return;
    const int i = m / a.ratio, j = m - i * a.ratio;
    store_out4(a.out + ((s.row0 + i) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + j) * a.kv.head_dim, 4 * lane, a.kv.head_dim,
               o * (l == 0.0f ? 0.0f : 1.0f / l));
}

// How a call runs: the kernel for few rows (16 mt of them at most) or the other one, and the ranges
// that a sequence's tokens are cut into, so that there are workgroups for every CU.
struct Plan {
    int mt;                 // 0: many rows
    int64_t units, row_tiles;
    int32_t nsplit, rows_cap;
    size_t o_bytes, ml_bytes;
};
constexpr int MANY_WAVES = 4;
Plan plan_of(const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads) {
    Plan p;
    const int64_t ratio = n_q_heads / c.n_heads, rows = b.max_rows * ratio, cap = b.max_pages * c.page_tokens;
    p.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= W4A4_KV_FEW_ROWS ? 4 : 0;
    p.units = b.n_seqs * c.n_heads;
    p.rows_cap = (int32_t)rows;
    p.row_tiles = p.mt ? 1 : (rows + 32 * MANY_WAVES - 1) / (32 * MANY_WAVES);
    const int64_t groups = p.units * p.row_tiles, target = p.mt ? 2048 : 512;
    int64_t n = groups ? target / groups : 1;
    if (n > cap / 256) n = cap / 256;
    p.nsplit = (int32_t)(n < 1 ? 1 : n > 256 ? 256 : n);
    p.o_bytes = p.nsplit > 1 ? (size_t)(p.units * p.nsplit * rows) * c.d_pad * 4 : 0;
    p.ml_bytes = p.nsplit > 1 ? (size_t)(p.units * p.nsplit * rows) * 8 : 0;
    return p;
}

template <int G, int MT>
void run_few(const AttnArgs& a, const Plan& p, bool qb, hipStream_t st) {
    const dim3 grid((uint32_t)(p.units * p.nsplit));
    if (qb) hipLaunchKernelGGL((kv_few_kernel<G, MT, true>), grid, dim3(256), 0, st, a);
    else hipLaunchKernelGGL((kv_few_kernel<G, MT, false>), grid, dim3(256), 0, st, a);
}

}  // namespace

size_t kv_attention_ws(int64_t, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads) {
    const Plan p = plan_of(b, c, n_q_heads);
    return (p.o_bytes + 255) / 256 * 256 + (p.ml_bytes + 255) / 256 * 256;
}

hipError_t launch_kv_attention(const w4a4_kv_rows& Q, int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads,
                               float scale, bool causal, int64_t window, uint16_t* O, void* ws, hipStream_t stream) {
    const Plan p = plan_of(b, c, n_q_heads);
    AttnArgs a;
    a.kv = kv_args(n_rows, b, c);
    a.q = Q.data;
    a.q_row = Q.row_stride;
    a.q_head = Q.head_stride;
    a.out = O;
    a.part_o = (float*)ws;
    a.part_ml = (float*)((uint8_t*)ws + (p.o_bytes + 255) / 256 * 256);
    a.window = window;
    a.scale = scale * 1.44269504088896340736f;
    a.ratio = n_q_heads / c.n_heads;
    a.causal = causal ? 1 : 0;
    a.nsplit = p.nsplit;
    a.rows_cap = p.rows_cap;
    const bool qb = Q.dtype == W4A4_X_BF16;
    return kv_groups(c.d_pad, [&](auto gc) {
        constexpr int G = gc();
        const dim3 join((uint32_t)((p.units * p.rows_cap + 3) / 4));
        if (p.mt) {
            if (p.mt == 1) run_few<G, 1>(a, p, qb, stream);
            else if (p.mt == 2) run_few<G, 2>(a, p, qb, stream);
            else run_few<G, 4>(a, p, qb, stream);
        } else {
            const dim3 grid((uint32_t)(p.units * p.row_tiles * p.nsplit));
            if (qb) hipLaunchKernelGGL((kv_many_kernel<G, MANY_WAVES, true>), grid, dim3(64 * MANY_WAVES), 0, stream, a, (uint32_t)p.row_tiles);
            else hipLaunchKernelGGL((kv_many_kernel<G, MANY_WAVES, false>), grid, dim3(64 * MANY_WAVES), 0, stream, a, (uint32_t)p.row_tiles);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || p.nsplit == 1) return e;
        if (p.mt) hipLaunchKernelGGL((kv_join_kernel<G, 32, 0>), join, dim3(256), 0, stream, a);
        else hipLaunchKernelGGL((kv_join_kernel<G, 64, 32 * MANY_WAVES>), join, dim3(256), 0, stream, a);
        return hipGetLastError();
    });
}

}  // namespace w4a4

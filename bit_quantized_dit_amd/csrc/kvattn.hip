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
// a weight passes 2^8 (many rows: a tile's weights 2^16), which leaves the result as it is (numerator and denominator
// carry the same factor) and spares most steps the exchange between lanes and the rescaling of O.  Every row renews
// by its own scores alone, so that its bits do not depend on the rows beside it.
#include "kv_device.h"

namespace w4a4 {

namespace {

typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v16f __attribute__((ext_vector_type(16)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

constexpr float M_NONE = -3.40282347e38f;      // no score yet: the lowest number
constexpr float M_SLACK = 8.0f;
// A weight's exponent is scale s - m, one rounding at the end, with m the rounded scale s of some token: the rounding
// of m is a factor that all weights share.  It is 2^(1/2) at most while |m| <= 2^24, and past 2^31 it could be
// infinity or zero.  Rows with maxima past 2^24 therefore round scale s as m was rounded, before m is taken off
// (calls without such rows: the same times within 1%).
constexpr float M_FAR = 16777216.0f;

struct AttnArgs {
    KvArgs kv;
    const void* q;
    int64_t q_row, q_head;
    uint16_t* out;
    float *part_o, *part_ml;      // [slot][rows_cap][d_pad], [slot][rows_cap][2]
    int64_t* joins;               // [n_seqs]: a sequence's first slot * 2^20 + its number of ranges
    struct Range* ranges;         // by number, of many sequences
    int64_t window;
    float scale;                  // scale * log2(e)
    int32_t ratio, causal, target, rows_cap;
};

// The steps of ST tokens that rows m0 .. m1 - 1 of a sequence see.
template <int ST> struct Steps {
    int32_t start, n;
    __device__ Steps(const AttnArgs& a, const KvSeq& s, int32_t m0, int32_t m1) {
        const int64_t i0 = m0 / a.ratio, i1 = (m1 - 1) / a.ratio;
        int64_t lo = a.causal && a.window ? s.first + i0 - a.window + 1 : 0, hi = a.causal ? s.first + i1 + 1 : s.len;
        lo = lo < 0 ? 0 : lo / ST * ST;
        n = m1 > m0 && hi > lo ? (int32_t)((hi - lo + ST - 1) / ST) : 0;
        start = (int32_t)lo;
    }
};

// Long sequences are cut into ranges of about the same number of steps, whatever sequence they
// belong to, so that a ragged batch keeps all CUs busy to the end: with `target` workgroups in mind a
// range has total / target steps, at least FEW_LEAST.  The lengths are the device's: up to 64 sequences every
// wavefront sums their steps, one a lane, and looks its number up among their ranges; for more a small kernel does it
// first, for all (500 sequences of 300 tokens in a long table, 8 heads: 53 us, with every wavefront looking 112).  Ranges of
// sequences that have several leave their results in slots, of which there are fewer than 2 target (a sequence of
// n steps > C has at most n / C + 1 < 2 n / C).
constexpr int FEW_LEAST = 16;      // steps of a range: 512 tokens
struct alignas(16) Range {
    int32_t b, slot;      // slot of the sequence's first range (heads lie side by side)
    int32_t k, count;     // which of how many ranges; count 0: there is nothing to do
};
__device__ __forceinline__ int32_t scan64(int32_t v) {      // inclusive, over the wavefront
    const int lane = threadIdx.x & 63;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) {
        const int32_t u = __shfl_up(v, o);
        v += lane >= o ? u : 0;
    }
    return v;
}
// Steps of a sequence, -1 for one without rows (or past the last one); its ranges of `chunk` steps.
__device__ __forceinline__ int32_t few_steps(const AttnArgs& a, int64_t b) {
    if (b >= a.kv.n_seqs) return -1;
    const KvSeq s = kv_seq(a.kv, b);
    return s.done > 0 ? Steps<32>(a, s, 0, s.done * a.ratio).n : -1;
}
__device__ __forceinline__ int32_t chunk_of(const AttnArgs& a, int64_t total) {
    const int64_t c = (total * a.kv.n_heads + a.target - 1) / a.target;
    return (int32_t)(c < FEW_LEAST ? FEW_LEAST : c);
}
__device__ __forceinline__ int32_t count_of(int32_t n, int32_t chunk) { return n < 0 ? 0 : n > chunk ? (n + chunk - 1) / chunk : 1; }

__device__ __forceinline__ Range find_range(const AttnArgs& a, uint32_t item) {
    if (!a.target) return Range{(int32_t)item, 0, 0, item < a.kv.n_seqs ? 1 : 0};
    if (a.kv.n_seqs > 64) return a.ranges[item];
    const int lane = threadIdx.x & 63;
    const int32_t n = few_steps(a, lane);
    int64_t total = n > 0 ? n : 0;
#pragma unroll
    for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
    const int32_t c = count_of(n, chunk_of(a, total)), m = c > 1 ? c : 0, sc = scan64(c), sm = scan64(m);
    const uint64_t hit = __ballot((int32_t)item < sc);
    Range r = {0, 0, 0, 0};
    if (hit) {
        r.b = __builtin_ctzll(hit);
        r.count = __shfl(c, r.b);
        r.k = (int32_t)item - (__shfl(sc, r.b) - r.count);
        r.slot = __shfl(sm, r.b) - (r.count > 1 ? r.count : 0);
    }
    return r;
}

// The same for many sequences: every item's range, and what the join reads.
__global__ __launch_bounds__(1024) void kv_plan_kernel(AttnArgs a, int32_t items) {
    __shared__ int64_t part[16];
    __shared__ int32_t part_c[16], part_m[16];
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    int64_t total = 0;
    for (int64_t b = threadIdx.x; b < a.kv.n_seqs; b += 1024) {
        const int32_t n = few_steps(a, b);
        total += n > 0 ? n : 0;
    }
#pragma unroll
    for (int o = 1; o < 64; o *= 2) total += __shfl_xor(total, o);
    if (lane == 0) part[wave] = total;
    __syncthreads();
    total = 0;
    for (int w = 0; w < 16; ++w) total += part[w];
    const int32_t chunk = chunk_of(a, total);
    int32_t before = 0, slots = 0;      // items and slots of the sequences before these 1024
    for (int64_t b0 = 0; b0 < a.kv.n_seqs; b0 += 1024) {
        const int64_t b = b0 + threadIdx.x;
        const int32_t c = count_of(few_steps(a, b), chunk), m = c > 1 ? c : 0, sc = scan64(c), sm = scan64(m);
        __syncthreads();
        if (lane == 63) {
            part_c[wave] = sc;
            part_m[wave] = sm;
        }
        __syncthreads();
        int32_t at = before + sc - c, slot = slots + sm - m;
        for (int w = 0; w < 16; ++w) {
            at += w < wave ? part_c[w] : 0;
            slot += w < wave ? part_m[w] : 0;
            before += part_c[w];
            slots += part_m[w];
        }
        for (int k = 0; k < c && at + k < items; ++k) a.ranges[at + k] = Range{(int32_t)b, slot, k, c};
        if (b < a.kv.n_seqs) a.joins[b] = (int64_t)slot << 20 | c;
    }
    for (int i = before + threadIdx.x; i < items; i += 1024) a.ranges[i] = Range{0, 0, 0, 0};
}

template <int N> __device__ __forceinline__ void load_words(const uint8_t* p, uint32_t (&w)[N]) {
    __builtin_memcpy(w, __builtin_assume_aligned(p, N % 4 == 0 ? 16 : N % 2 == 0 ? 8 : 4), 4 * N);
}
// A scale code's byte where a binary32 has its exponent.  The neighbouring bytes stay beside it: the
// conversions read the exponent field only (compared for every code and several other bits).
__device__ __forceinline__ float scale_of(uint32_t word, int byte) {
    return __uint_as_float(byte == 3 ? word >> 1 : word << (23 - 8 * byte));
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
__device__ __forceinline__ void store_quad(uint16_t* p, v4f v) { *reinterpret_cast<uint2*>(p) = make_uint2(pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])); }
__device__ __forceinline__ void store_out4(uint16_t* row, int d, int D, v4f v) {
    if ((D & 3) == 0) {
        if (d < D) store_quad(row + d, v);
        return;
    }
    const uint32_t w[2] = {pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (d + i < D) row[d + i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
}

// ---------------------------------------------------------------- few rows
//
// Up to 16 MT stacked rows: bound by reading the cache (kernel times: 64 ragged sequences of 8 heads and 1.16 GB 201 us, 5.8 TB/s;
// one row of 40 heads over 57600 tokens, 313 MB, 58 us, 5.4 TB/s; a kernel that only reads reaches 6.1), or, for a
// few hundred tokens, by the latency of its dependent loads (9 us).  The tiles are those of the 16-row instruction,
// as a sequence's one row and its ratio of heads seldom fill more.  The matrix unit has time to spare, so weights are
// multiplied as two bf16 terms (16 bits) and their rounding does not show.  A wavefront takes every NW-th step of
// 32 tokens of its workgroup's range.  Its two blocks go into a ring of R steps in LDS by copies that
// need no registers, so that many steps are in flight beside the accumulators, and go past the caches, as no one
// reads them twice (through them: 227 and 64 us); rings of 4 steps, of which fewer wavefronts fit, are slower, and so
// are workgroups of 8 wavefronts.  The copies past the last step run with empty ranges, so that every wait counts the same number.  The wavefronts'
// results meet in LDS.
// (One wavefront a SIMD has its sums copied between register files at every use: 64 rows of 40 heads of 72 over 57600 tokens 170 us,
// with two and 52 bytes in scratch 133; 20 rows of 192 channels 143 and 103.  Heads of 256 do not fit: 20 rows 326, with two 363,
// and 140 bytes of 32 rows are in scratch.  Four wavefronts a SIMD put 152 bytes of 64 rows of up to 32 channels into scratch, and 16
// of 32 rows of up to 64; not measured against fewer.)
template <int G, int MT> struct Few {      // wavefronts of a workgroup, steps of a ring, wavefronts a SIMD (for the register budget)
    static constexpr int NW = 4, R = 2, OCC = G * MT <= 4 ? 4 : G * MT <= 12 ? 2 : 1;
    static constexpr int COPIES = (KvBlock<G>::BYTES + 1023) / 1024, STEP = 2 * KvBlock<G>::BYTES, LD = 32 * G + 4;
    static constexpr int64_t ROUND = 256 * OCC;      // workgroups at a time
    static constexpr int RING = NW * R * STEP, RED = NW * 16 * LD * 4, LDS = RING > RED ? RING : RED;
};

template <int G, int MT, bool QB>
__global__ __launch_bounds__((Few<G, MT>::NW * 64), (Few<G, MT>::OCC)) void kv_few_kernel(AttnArgs a) {
    typedef KvBlock<G> L;
    typedef Few<G, MT> F;
    constexpr int DP = 32 * G, LD = F::LD, NW = F::NW, R = F::R;
    __shared__ __attribute__((aligned(1024))) uint8_t smem[F::LDS];      // the rings, then the wavefronts' sums
    __shared__ float red_m[NW][MT][16], red_l[NW][MT][16];
    const int lane = threadIdx.x & 63, c = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t item = blockIdx.x / (uint32_t)a.kv.n_heads;
    const int h = (int)(blockIdx.x - item * (uint32_t)a.kv.n_heads);
    Range rg = find_range(a, item);
    rg.k = __builtin_amdgcn_readfirstlane(rg.k);
    rg.count = __builtin_amdgcn_readfirstlane(rg.count);
    if (rg.count == 0) return;
    const int64_t b = __builtin_amdgcn_readfirstlane(rg.b);
    const KvSeq s = kv_seq(a.kv, b);
    const int rows = s.done * a.ratio;
    const Steps<32> st(a, s, 0, rows);
    if (rows == 0) return;
    if (a.target && rg.k == 0 && h == 0 && threadIdx.x == 0) a.joins[b] = (int64_t)rg.slot << 20 | rg.count;
    // equal parts of the sequence's steps; this wavefront's are s0 + wave, + NW, ..
    const int s0 = (int)((int64_t)st.n * rg.k / rg.count), s1 = (int)((int64_t)st.n * (rg.k + 1) / rg.count);
    const int mine = s1 - s0 > wave ? (s1 - s0 - wave + NW - 1) / NW : 0;

    // Block addresses of 32 steps, two a step, one a lane (zero where a block is not there).
    uint64_t addr = 0;
    auto lookup = [&](int k) __attribute__((always_inline)) {
        const int mk = k + (lane >> 1);
        addr = mk < mine ? (uint64_t)(uintptr_t)kv_block(a.kv, b, (uint32_t)(st.start / 16 + 2 * (s0 + wave + mk * NW) + (lane & 1)), h) : 0;
    };
    const uint32_t ring = (uint32_t)(uintptr_t)smem + (uint32_t)wave * R * F::STEP;
    uint64_t there_bits = 0;      // whether each block of these steps is there
    auto copy = [&](int k, uint32_t slot) __attribute__((always_inline)) {      // step k of this wavefront into a slot of its ring
        if ((k & 31) == 0) {
            lookup(k);
            there_bits = __ballot(addr != 0);
        }
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            const int from = 2 * (k & 31) + u;
            const uint32_t al = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)addr, from);
            const uint32_t ah = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(addr >> 32), from);
            const uint64_t p = (uint64_t)ah << 32 | al;
            const v4i srd = make_srd((const void*)(uintptr_t)p, p ? L::BYTES : 0u);
#pragma unroll
            for (int i = 0; i < F::COPIES; ++i) {
                const int off = i * 1024 + lane * 16;
                if (off < L::BYTES) dma16_once(srd, ring + slot * F::STEP + u * L::BYTES + i * 1024, off, 0);
            }
        }
    };
    uint64_t there = 0;      // of the steps whose copies are under way, two bits a step, the next one lowest
    auto there_of = [&](int k) { return (uint32_t)(there_bits >> (2 * (k & 31))) & 3u; };
#pragma unroll
    for (int k = 0; k < R - 1; ++k) {      // on their way while the queries are read
        copy(k, k);
        there |= (uint64_t)there_of(k) << (2 * k);
    }

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
    uint64_t far_rows = 0;      // lanes whose maxima are past M_FAR
    float mx[MT], sum[MT];
#pragma unroll
    for (int mt = 0; mt < MT; ++mt) {
        mx[mt] = M_NONE;
        sum[mt] = 0.0f;
#pragma unroll
        for (int t = 0; t < 2 * G; ++t) acc[mt][t] = v4f{0, 0, 0, 0};
    }

    // One step from token `pos` on; `there` tells which of its two blocks are in the cache.  Where some row
    // does not see all of its tokens, their scores become -Inf; value scale codes that no weight
    // of zero may be multiplied with are made harmless first, and values that are NaN go by a list of their own.
    auto step = [&](uint8_t* x, int pos, uint32_t there) __attribute__((always_inline)) {
        const bool full = there == 3u && pos + 31 <= all_hi && pos >= last_from;      // uniform
        uint32_t nan = 0;
        if (!full) {
            constexpr int WORDS = 4 * L::SG;      // of a block's value scales: tokens 4 (i / sg) .., group i % sg
            if (lane < 2 * WORDS) {
                uint32_t* const w = reinterpret_cast<uint32_t*>(x + lane / WORDS * L::BYTES + L::VS) + lane % WORDS;
                if (wild(*w)) {
                    *w = tame(*w, nan);
                    const int left = s.len - (pos + lane / WORDS * 16 + lane % WORDS / L::SG * 4);      // tokens that were written
                    nan &= left >= 4 ? 15u : left <= 0 ? 0u : (1u << left) - 1u;
                }
            }
            asm volatile("" ::: "memory");
        }
        v4f sc[MT][2];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) sc[mt][0] = sc[mt][1] = v4f{0, 0, 0, 0};
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            uint32_t kw[G], ks[(G + 3) / 4];
            const uint8_t* const p = x + u * L::BYTES;
            load_words<G>(p + lane * 4 * G, kw);
            if constexpr (G == 1) ks[0] = p[L::KS + c];
            else if constexpr (G == 2) ks[0] = *reinterpret_cast<const uint16_t*>(p + L::KS + c * 2);
            else load_words<(G + 3) / 4>(p + L::KS + c * L::SG, ks);
#pragma unroll
            for (int d = 0; d < G; ++d) {
                const v8bf kf = widen_key(kw[d], scale_of(ks[d / 4], d & 3));
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) sc[mt][u] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(kf, q[mt][d], sc[mt][u], 0, 0, 0);
            }
        }
        uint32_t vw[2][G], vs[2][G];
#pragma unroll
        for (int u = 0; u < 2; ++u) {
            load_words<G>(x + u * L::BYTES + L::V + lane * 4 * G, vw[u]);
            load_words<G>(x + u * L::BYTES + L::VS + g * 4 * L::SG, vs[u]);
        }
        if (!full) {
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const int t = pos + 16 * u + 4 * g + i;
                        if (t < lo[mt] || t > hi[mt] || !(there >> u & 1)) sc[mt][u][i] = -__builtin_inff();
                    }
        }
        v8bf ph[MT], pl[MT];
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            float top = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(sc[mt][0][0], sc[mt][0][1]), __builtin_fmaxf(sc[mt][0][2], sc[mt][0][3])),
                                        __builtin_fmaxf(__builtin_fmaxf(sc[mt][1][0], sc[mt][1][1]), __builtin_fmaxf(sc[mt][1][2], sc[mt][1][3])));
            top *= a.scale;
            float k = a.scale;
            if (far_rows | __ballot(top > mx[mt] + M_SLACK)) {
                top = __builtin_fmaxf(top, __shfl_xor(top, 16));
                top = __builtin_fmaxf(top, __shfl_xor(top, 32));
                // (a row's own scores decide: other rows' tokens must not move its rounding)
                const float m = top > mx[mt] + M_SLACK ? top : mx[mt], f = __builtin_amdgcn_exp2f(mx[mt] - m);
                const bool far = __builtin_fabsf(m) > M_FAR && m != M_NONE;
                mx[mt] = m;
                far_rows |= __ballot(far);
                sum[mt] *= f;
#pragma unroll
                for (int t = 0; t < 2 * G; ++t) acc[mt][t] *= f;
                if (far_rows) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) sc[mt][i >> 2][i & 3] *= far ? a.scale : 1.0f;
                    k = far ? 1.0f : a.scale;
                }
            }
            float p[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[mt][i >> 2][i & 3], k, -mx[mt]));
                sum[mt] += p[i];
            }
            uint32_t wh[4], wl[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                wh[i] = pk_bf16(p[2 * i], p[2 * i + 1]);
                wl[i] = pk_bf16(p[2 * i] - __uint_as_float(wh[i] << 16), p[2 * i + 1] - __uint_as_float(wh[i] & 0xFFFF0000u));
            }
            ph[mt] = join8(wh[0], wh[1], wh[2], wh[3]);
            pl[mt] = join8(wl[0], wl[1], wl[2], wl[3]);
        }
#pragma unroll
        for (int d = 0; d < G; ++d) {
            v8bf v0, v1;
            widen_value(vw[0][d], vs[0][d], vw[1][d], vs[1][d], v0, v1);
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                acc[mt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, ph[mt], acc[mt][2 * d], 0, 0, 0);
                acc[mt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, ph[mt], acc[mt][2 * d + 1], 0, 0, 0);
                acc[mt][2 * d] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v0, pl[mt], acc[mt][2 * d], 0, 0, 0);
                acc[mt][2 * d + 1] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v1, pl[mt], acc[mt][2 * d + 1], 0, 0, 0);
            }
        }
        if (!full) {      // rare: for every NaN that a row sees, its group of channels
            for (uint64_t left = __ballot(nan != 0); left; left &= left - 1) {
                const int from = __builtin_ctzll(left), w = from % (4 * L::SG), u = from / (4 * L::SG);
                const uint32_t bits = (uint32_t)__builtin_amdgcn_readlane((int)nan, from);
                const int t0 = pos + 16 * u + 4 * (w / L::SG), d = w % L::SG;
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    bool hit = false;
                    for (int j = 0; j < 4; ++j) hit |= (bits >> j & 1) && (there >> u & 1) && t0 + j >= lo[mt] && t0 + j <= hi[mt];
#pragma unroll
                    for (int e = 0; e < G; ++e)
                        if (hit && e == d) acc[mt][2 * e][0] = acc[mt][2 * e][1] = acc[mt][2 * e][2] = acc[mt][2 * e][3] = acc[mt][2 * e + 1][0] =
                            acc[mt][2 * e + 1][1] = acc[mt][2 * e + 1][2] = acc[mt][2 * e + 1][3] = __uint_as_float(0x7FC00000u);
                }
            }
        }
    };
    uint32_t slot = 0;
    for (int k = 0; k < mine; ++k) {
        // the slot read last is free: its reads are in registers
        asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        copy(k + R - 1, slot == 0 ? R - 1 : slot - 1);
        there |= (uint64_t)there_of(k + R - 1) << (2 * (R - 1));
        asm volatile("s_waitcnt vmcnt(%0)" ::"i"((R - 1) * 2 * F::COPIES) : "memory");
        step(smem + (wave * R + slot) * F::STEP, st.start + (s0 + wave + k * NW) * 32, (uint32_t)there & 3u);
        there >>= 2;
        slot = slot == R - 1 ? 0 : slot + 1;
    }
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __syncthreads();      // the rings are free
    float(*const red)[16][LD] = reinterpret_cast<float(*)[16][LD]>(smem);

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
        for (int e = threadIdx.x; e < 16 * (DP / 4); e += NW * 64) {
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
            if (rg.count == 1) {
                const int i = row / a.ratio, j = row - i * a.ratio;
                const float r = l == 0.0f ? 0.0f : 1.0f / l;
                store_out4(a.out + ((s.row0 + i) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + j) * a.kv.head_dim, d, a.kv.head_dim, o * r);
            } else {
                const int64_t at = ((int64_t)(rg.slot + rg.k) * a.kv.n_heads + h) * a.rows_cap + row;
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
// Bound by the matrix unit, the vector unit's softmax and widening beside it, and the board's power: 4096 rows of 40
// heads over 57600 tokens 4.27 to 4.33 ms, 1.12 PFLOP/s, matrix unit 52% of the cycles (a large bf16 product
// of the library: 1.24; of 4.28, without the widening 3.86, without the exponentials 4.04, without either 3.29).  So weights are one
// bf16 term here: two would double the second product.  TWO: of up to 64 stacked rows of heads of 97 to 128 channels, which
// the few-row kernel has no registers for, they are two terms as there (64 rows of 40 heads over 57600 tokens 212 us, with one
// 196; 64 sequences of 40 rows, 8 heads, 2048 tokens 94; error against 64 bits 0.0016 and 0.0023).
//
// A workgroup owns 32 rows a wavefront and walks tiles of 64 tokens.  A tile's codes are widened once,
// every wavefront its share, into LDS; rows of LDS are 16 bytes longer than their data, so that the
// operand reads of 16 lanes touch every bank once.  The loop is a pipeline with one barrier a tile: while the
// matrix unit multiplies tile k's keys, the codes of tile k + 1 are widened; while it multiplies tile
// k - 1's weights with its values, tile k's scores become weights, a quarter of them as soon as that quarter of the
// old ones has been used.  The codes of tile k + 2 are on their way meanwhile.  The order of instructions is written
// out: a matrix instruction, the read of an operand FR steps ahead, a few vector instructions.
//
// Weights are taken with the maximum of the tiles before; where their sum shows that a score passed it by
// far, the maximum is renewed and they are taken again.
template <int G, int WAVES> struct Many {
    static constexpr int NW = WAVES, ROWS = 32 * NW, PARTS = NW / 4;      // wavefronts; those that share a block's widening
    static constexpr int KG = (G + PARTS - 1) / PARTS, VG = (G + 2 * PARTS - 1) / (2 * PARTS);      // groups that a lane widens
    static constexpr int KLD = 64 * G + 16, VLD = 144, KB = 64 * KLD, VB = 32 * G * VLD;
    // value buffers: widened a tile ahead and read a tile behind, without a barrier between the two.  Wide heads,
    // for which four do not fit, and small workgroups, of which two share a CU, take keys and values in turn.
    static constexpr int VSLOTS = G <= 4 && NW == 8 ? 4 : 2;
    static constexpr int OCC = G <= 4 ? 2 : 1;
};
// (a row at a time renews its maximum: with 2^8 the ragged windowed prompts are settled often enough to take 17.6 us, with 2^16 17.0)
constexpr float P_MOST = 65536.0f;
// The ranges that a row tile's steps are cut into, out of nsplit that there is room for.
constexpr int MANY_LEAST = 8;
__device__ __forceinline__ int many_parts(int n, int nsplit) { return n / MANY_LEAST < 1 ? 1 : n / MANY_LEAST < nsplit ? n / MANY_LEAST : nsplit; }

// The item'th of all sequences' tiles of ROWS rows, a sequence's last ones, which see most, first.  Of up to 64
// sequences every wavefront counts their tiles, one a lane, so that no workgroup without rows stands between the others
// and two of them share a CU only when all CUs have one (5 prompts of 1 to 777 rows: 19.1 us, with gaps 21.2).  More sequences have room
// for row_tiles tiles each.
struct TileAt {
    KvSeq s;
    int32_t b, tile;      // tile -1: there is none
};
template <int ROWS> __device__ __forceinline__ TileAt find_tile(const AttnArgs& a, uint32_t item, uint32_t row_tiles) {
    TileAt t;
    if (a.kv.n_seqs > 64) {
        const uint32_t n = (uint32_t)a.kv.n_seqs, behind = item / n;
        t.b = (int32_t)(item - behind * n);
        t.tile = (int32_t)(row_tiles - 1 - behind);
        t.s = kv_seq(a.kv, t.b);
        return t;
    }
    const int lane = threadIdx.x & 63;
    KvSeq s = {0, 0, 0, 0, 0};
    if (lane < a.kv.n_seqs) s = kv_seq(a.kv, lane);
    const int32_t c = (int32_t)(((int64_t)s.done * a.ratio + ROWS - 1) / ROWS), sc = scan64(c);
    const uint64_t hit = __ballot((int32_t)item < sc);
    t.b = hit ? __builtin_ctzll(hit) : 0;
    auto of = [&](int32_t v) { return __builtin_amdgcn_readlane(v, t.b); };
    t.s.row0 = (int64_t)((uint64_t)(uint32_t)of((int32_t)(s.row0 >> 32)) << 32 | (uint32_t)of((int32_t)s.row0));
    t.s.rows = of(s.rows);
    t.s.done = of(s.done);
    t.s.len = of(s.len);
    t.s.first = of(s.first);
    t.tile = hit ? of(sc) - 1 - (int32_t)item : -1;
    return t;
}

template <int G, int WAVES, bool TWO, bool QB>
__global__ __launch_bounds__((WAVES * 64), (Many<G, WAVES>::OCC)) void kv_many_kernel(AttnArgs a, uint32_t row_tiles, int32_t nsplit) {
    typedef KvBlock<G> L;
    typedef Many<G, WAVES> M;
    constexpr int DP = 32 * G, ROWS = M::ROWS, KG = M::KG, VG = M::VG, KLD = M::KLD, VLD = M::VLD, N = 4 * G, FR = TWO ? 2 : 4;
    __shared__ __attribute__((aligned(16))) uint8_t keys[2][M::KB];
    __shared__ __attribute__((aligned(16))) uint8_t vals[M::VSLOTS][M::VB];
    __shared__ uint4 flags[M::VSLOTS][M::PARTS];           // by share and block: 1 values that are NaN, 2 not there
    __shared__ uint8_t nans[M::VSLOTS][M::PARTS][64];      // a token's groups that are NaN
    const int lane = threadIdx.x & 63, c = lane & 31, h2 = lane >> 5, r16 = lane & 15, g = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const uint32_t sp = blockIdx.x % (uint32_t)nsplit, rest = blockIdx.x / (uint32_t)nsplit;
    const uint32_t item = rest / (uint32_t)a.kv.n_heads;
    const int h = (int)(rest - item * (uint32_t)a.kv.n_heads);
    const TileAt at_tile = find_tile<ROWS>(a, item, row_tiles);
    const KvSeq s = at_tile.s;
    const int64_t b = at_tile.b, unit = b * a.kv.n_heads + h;
    const int tile = at_tile.tile;
    if (tile < 0) return;
    const int64_t all_rows = (int64_t)s.done * a.ratio;
    const int64_t m0 = (int64_t)tile * ROWS;
    if (m0 >= all_rows) return;
    const int rows = (int)(all_rows - m0 < ROWS ? all_rows - m0 : ROWS);
    const Steps<64> st(a, s, (int32_t)m0, (int32_t)(m0 + rows));
    const int parts = many_parts(st.n, nsplit);
    if ((int)sp >= parts) return;
    int s0 = 0, s1 = st.n;
    if (parts > 1) {
        s0 = (int)((int64_t)st.n * sp / parts);
        s1 = (int)((int64_t)st.n * (sp + 1) / parts);
    }

    const int row = wave * 32 + c, m = (int)m0 + row, qi = m / a.ratio, qj = m - qi * a.ratio;
    const bool on = row < rows;
    // tokens that the row sees
    const int64_t pos = (int64_t)s.first + qi, from = a.causal && a.window ? pos - a.window + 1 : 0;
    const int32_t lo = from < 0 ? 0 : (int32_t)from, hi = !on ? -1 : a.causal ? (int32_t)pos : s.len - 1;
    const uint32_t from_lo = (uint32_t)lo, span = hi < lo ? 0u : (uint32_t)(hi - lo) + 1u;
    // tokens that all of the wavefront's rows see (where some row is missing: none)
    const int64_t i0 = ((int)m0 + wave * 32) / a.ratio, i1 = ((int)m0 + wave * 32 + 31) / a.ratio;
    const int64_t all_hi = wave * 32 + 32 > rows ? -1 : a.causal ? s.first + i0 : s.len - 1;
    const int64_t all_lo = a.causal && a.window ? s.first + i1 - a.window + 1 : 0;

    v16f acc[G];
#pragma unroll
    for (int d = 0; d < G; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[d][i] = 0.0f;
    float mx = M_NONE, sum = 0.0f;
    uint64_t far_rows = 0;      // lanes whose maxima are past M_FAR

    // This wavefront's share of a tile: of block `blk` the keys of token r16, groups from k0 on, and of the values
    // of tokens 4 hh .. and 8 + 4 hh .. the groups from v0 on (shares that do not divide overlap).
    const int blk = wave / M::PARTS, share = wave % M::PARTS, hh = g & 1;
    const int k0 = share * KG < G - KG ? share * KG : G - KG;
    const int vi = (2 * share + (g >> 1)) * VG, v0 = vi < G - VG ? vi : G - VG;
    uint32_t kw[KG], ks[(G + 3) / 4], vw[2][VG], vs[2][VG];
    bool there = false;
    uint64_t addr = 0;      // the block's address in 64 tiles, one a lane (zero: not there, or past the last tile)
    auto fetch = [&](int k) __attribute__((always_inline)) {
        const int j = (k - s0) & 63;
        if (j == 0) addr = k + lane < s1 ? (uint64_t)(uintptr_t)kv_block(a.kv, b, (uint32_t)(st.start / 16 + 4 * (k + lane) + blk), h) : 0;
        const uint32_t al = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)addr, j), ah = (uint32_t)__builtin_amdgcn_readlane((int)(uint32_t)(addr >> 32), j);
        const uint8_t* p = (const uint8_t*)(uintptr_t)((uint64_t)ah << 32 | al);
        there = p != nullptr;
        p = p ? p : a.kv.data;
#pragma unroll
        for (int d = 0; d < KG; ++d) kw[d] = *reinterpret_cast<const uint32_t*>(p + lane * 4 * G + 4 * (k0 + d));
        if constexpr (G == 1) ks[0] = p[L::KS + r16];
        else if constexpr (G == 2) ks[0] = *reinterpret_cast<const uint16_t*>(p + L::KS + r16 * 2);
        else load_words<(G + 3) / 4>(p + L::KS + r16 * L::SG, ks);
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < VG; ++d) {
                vw[u][d] = *reinterpret_cast<const uint32_t*>(p + L::V + ((hh + 2 * u) * 16 + r16) * 4 * G + 4 * (v0 + d));
                vs[u][d] = *reinterpret_cast<const uint32_t*>(p + L::VS + (hh + 2 * u) * 4 * L::SG + 4 * (v0 + d));
            }
    };
    if (s0 < s1) fetch(s0);      // on its way while the queries are read
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
    // Before a fetched block is widened: its flag, and scale codes that a weight of zero may not be multiplied with.
    auto prepare = [&](int slot) __attribute__((always_inline)) {
        uint32_t flag = there ? 0u : 2u;
        bool odd = false;
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
            for (int d = 0; d < VG; ++d) odd |= wild(vs[u][d]);
        if (__any(odd)) {      // rare: values that are NaN go by a list of their own
            uint32_t bits[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int d = 0; d < VG; ++d) {
                    uint32_t nan;
                    vs[u][d] = tame(vs[u][d], nan);
#pragma unroll
                    for (int j = 0; j < 4; ++j) bits[4 * u + j] |= (nan >> j & 1) ? 1u << (v0 + d) : 0u;
                }
#pragma unroll
            for (int k = 0; k < 8; ++k) bits[k] |= (uint32_t)__shfl_xor((int)bits[k], 32);      // the other half's groups
            if (r16 == 0 && g < 2)
#pragma unroll
                for (int k = 0; k < 8; ++k) nans[slot][share][blk * 16 + 4 * hh + (k >> 2) * 8 + (k & 3)] = (uint8_t)bits[k];
            flag |= 1u;
        }
        if (lane == 0) reinterpret_cast<uint32_t*>(&flags[slot][share])[blk] = flag;
    };
    // The widening in UNITS parts: a group of keys each, then two tokens of a group of values each.
    constexpr int UNITS = KG + 4 * VG;
    uint32_t vlo[4], vhi[4];
    auto widen = [&](int n, int kslot, int vslot) __attribute__((always_inline)) {
        if (n < KG) {
            const int kg = k0 + n;
            const float f = __uint_as_float((G > 4 && kg >= 4 ? ks[(G + 3) / 4 - 1] : ks[0]) >> (8 * (kg & 3)) << 23);
            *reinterpret_cast<v8bf*>(keys[kslot] + (blk * 16 + r16) * KLD + g * 16 + kg * 64) = widen_key(kw[n], f);
            return;
        }
        const int d = (n - KG) / 4, i = (n - KG) & 3, u = i >> 1, j = 2 * (i & 1);
        const uint32_t w = vw[u][d], x = vs[u][d];
        const uint32_t p0 = j ? widen2<2>(w, scale_of(x, 2)) : widen2<0>(w, scale_of(x, 0));
        const uint32_t p1 = j ? widen2<3>(w, scale_of(x, 3)) : widen2<1>(w, scale_of(x, 1));
        vlo[i] = __builtin_amdgcn_perm(p1, p0, 0x05040100u);
        vhi[i] = __builtin_amdgcn_perm(p1, p0, 0x07060302u);
        if (i == 3) {
            uint8_t* const vd = vals[vslot] + ((v0 + d) * 32 + r16) * VLD + (2 * blk + hh) * 16;
            *reinterpret_cast<v8bf*>(vd) = join8(vlo[0], vlo[1], vlo[2], vlo[3]);
            *reinterpret_cast<v8bf*>(vd + 16 * VLD) = join8(vhi[0], vhi[1], vhi[2], vhi[3]);
        }
    };

    v16f sc[2];           // a tile's scores, 32 tokens each
    uint32_t pw[16], pl[TWO ? 16 : 1];      // weights, and what their rounding left
    float tile_sum = 0.0f;
    // weights 2 i, 2 i + 1
    auto weigh = [&](int i, float k) __attribute__((always_inline)) {
        const float pa = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i >> 3][2 * (i & 7)], k, -mx));
        const float pb = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[i >> 3][2 * (i & 7) + 1], k, -mx));
        tile_sum = i == 0 ? pa + pb : tile_sum + (pa + pb);
        pw[i] = pk_bf16(pa, pb);
        if constexpr (TWO) pl[i] = pk_bf16(pa - __uint_as_float(pw[i] << 16), pb - __uint_as_float(pw[i] & 0xFFFF0000u));
        asm volatile("" : "+v"(pw[i]), "+v"(tile_sum));      // here, between the matrix instructions
    };
    // Whether the weights just taken may be used; if not, they are taken again with a new maximum.
    auto settle = [&]() __attribute__((always_inline)) {
        const uint64_t over = __ballot(!(tile_sum <= P_MOST));
        if (far_rows | over) {
            float top = sc[0][0];
#pragma unroll
            for (int i = 1; i < 32; ++i) top = __builtin_fmaxf(top, sc[i >> 4][i & 15]);
            top *= a.scale;
            top = __builtin_fmaxf(top, __shfl_xor(top, 32));
            // a row's own weights decide, those of both its lanes: other rows' must not move its rounding
            const bool own = __builtin_amdgcn_inverse_ballot_w64(far_rows | over | over >> 32 | over << 32);
            const float n = own ? __builtin_fmaxf(mx, top) : mx, f = __builtin_amdgcn_exp2f(mx - n);
            mx = n;
            sum *= f;
#pragma unroll
            for (int d = 0; d < G; ++d) acc[d] *= f;
            const bool far = __builtin_fabsf(mx) > M_FAR && mx != M_NONE;
            far_rows |= __ballot(far);
            float k = a.scale;
            if (far_rows) {
#pragma unroll
                for (int i = 0; i < 32; ++i) sc[i >> 4][i & 15] *= far ? a.scale : 1.0f;
                k = far ? 1.0f : a.scale;
            }
#pragma unroll
            for (int i = 0; i < 16; ++i) weigh(i, k);
        }
        sum += tile_sum;
    };
    v8bf fr[FR];
    const int key_at = c * KLD + h2 * 16, val_at = c * VLD + h2 * 16;
    auto key_operand = [&](int kslot, int i) __attribute__((always_inline)) {      // step i: channels 16 (i / 2) .., tokens 32 (i % 2) ..
        return *reinterpret_cast<const v8bf*>(keys[kslot] + key_at + (i & 1) * 32 * KLD + (i >> 1) * 32);
    };
    auto value_operand = [&](int slot, int i) __attribute__((always_inline)) {      // step i: tokens 16 (i / G) .., channels 32 (i % G) ..
        return *reinterpret_cast<const v8bf*>(vals[slot] + val_at + (i % G) * 32 * VLD + i / G * 32);
    };
    auto key_step = [&](int i) __attribute__((always_inline)) {
        if (i < 2) {
#pragma unroll
            for (int e = 0; e < 16; ++e) sc[i][e] = 0.0f;
        }
        sc[i & 1] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % FR], q[i >> 1], sc[i & 1], 0, 0, 0);
    };
    auto value_step = [&](int i) __attribute__((always_inline)) {
        const int u = i / G;
        acc[i % G] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % FR], join8(pw[4 * u], pw[4 * u + 1], pw[4 * u + 2], pw[4 * u + 3]), acc[i % G], 0, 0, 0);
        if constexpr (TWO)
            acc[i % G] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(fr[i % FR], join8(pl[4 * u], pl[4 * u + 1], pl[4 * u + 2], pl[4 * u + 3]), acc[i % G], 0, 0, 0);
    };
    // A tile's flags by block; bit 0 of any, bit 1 of any.
    auto flags_of = [&](int slot) __attribute__((always_inline)) {
        uint4 f = flags[slot][0];
        if constexpr (M::PARTS > 1) {
            const uint4 o = flags[slot][1];
            f = make_uint4(f.x | o.x, f.y | o.y, f.z | o.z, f.w | o.w);
        }
        return f;
    };
    // rare: for every NaN that the lane's row sees, its group of channels
    auto spread_nans = [&](int slot, int64_t p0) __attribute__((always_inline)) {
        const uint4 f = flags_of(slot);
        if (!((f.x | f.y | f.z | f.w) & 1)) return;
        // one token a lane; those past the sequence, which were never written, are left out (a last page of random
        // bytes, ragged prompts: 17.6 us, looked through token by token 19.1)
        uint32_t bits = 0, bad = 0;
        bool gone = (int32_t)p0 + lane >= s.len;
#pragma unroll
        for (int w = 0; w < M::PARTS; ++w) {
            const uint32_t fb = reinterpret_cast<const uint32_t*>(&flags[slot][w])[lane >> 4];
            if (fb & 1) bits |= nans[slot][w][lane];
            gone |= (fb & 2) != 0;
        }
        for (uint64_t left = __ballot(bits != 0 && !gone); left; left &= left - 1) {
            const int t = __builtin_ctzll(left);
            const int32_t tp = (int32_t)p0 + t;
            const uint32_t group = (uint32_t)__builtin_amdgcn_readlane((int)bits, t);
            if (tp >= lo && tp <= hi) bad |= group;
        }
#pragma unroll
        for (int d = 0; d < G; ++d)
            if (bad >> d & 1) {
#pragma unroll
                for (int i = 0; i < 16; ++i) acc[d][i] = __uint_as_float(0x7FC00000u);
            }
    };
    // The scores of tokens that a row does not see.
    auto hide = [&](int k, int slot) __attribute__((always_inline)) {
        const int64_t p0 = st.start + (int64_t)k * 64;
        const uint4 f = flags_of(slot);
        if (p0 + 63 <= all_hi && p0 >= all_lo && !((f.x | f.y | f.z | f.w) & 2)) return;
        const uint32_t off = (uint32_t)((int32_t)p0 + 4 * h2) - from_lo;      // of the first score, from the row's first token on
#pragma unroll
        for (int i = 0; i < 32; ++i)
            if (off + 8 * (i >> 2) + (i & 3) >= span) sc[i >> 4][i & 15] = -__builtin_inff();
        const uint32_t gone[4] = {f.x & 2, f.y & 2, f.z & 2, f.w & 2};
#pragma unroll
        for (int u = 0; u < 4; ++u)
            if (gone[u]) {
#pragma unroll
                for (int i = 0; i < 8; ++i) sc[u >> 1][8 * (u & 1) + i] = -__builtin_inff();
            }
    };
    auto widen_all = [&](int kslot, int slot) __attribute__((always_inline)) {
        prepare(slot);
#pragma unroll
        for (int e = 0; e < UNITS; ++e) widen(e, kslot, slot);
    };
    constexpr int VS = M::VSLOTS - 1;      // a mask
    if (s0 < s1) {
        widen_all(0, 0);
        fetch(s0 + 1);
        __syncthreads();
    }
    if constexpr (M::VSLOTS == 4) {
        // Tile s0 + j: its scores, then its weights, beside them (unless it is the first) tile j - 1's weights and values.
        auto body = [&](auto first, int j) __attribute__((always_inline)) {
            constexpr bool FIRST = first();
            prepare((j + 1) & VS);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                key_step(i);
                if (i + FR < N) fr[i % FR] = key_operand(j & 1, i + FR);
                else if constexpr (!FIRST) fr[i % FR] = value_operand((j - 1) & VS, i + FR - N);
#pragma unroll
                for (int e = UNITS * i / N; e < UNITS * (i + 1) / N; ++e) widen(e, (j + 1) & 1, (j + 1) & VS);
            }
            __builtin_amdgcn_sched_barrier(0);
            fetch(s0 + j + 2);
            __syncthreads();
            hide(s0 + j, j & VS);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                __builtin_amdgcn_sched_barrier(0);
                if constexpr (!FIRST) {
                    value_step(i);
                    if (i + FR < N) fr[i % FR] = value_operand((j - 1) & VS, i + FR);
                }
                if (i + FR >= N) fr[i % FR] = key_operand((j + 1) & 1, i + FR - N);
                // the weights of 16 tokens are free after their G steps
                if (i >= G) {
#pragma unroll
                    for (int e = 4 * (i - G) / G; e < 4 * (i + 1 - G) / G; ++e) weigh(e, a.scale);
                }
            }
            __builtin_amdgcn_sched_barrier(0);
#pragma unroll
            for (int e = 12; e < 16; ++e) weigh(e, a.scale);
            if constexpr (!FIRST) spread_nans((j - 1) & VS, st.start + (int64_t)(s0 + j - 1) * 64);
            settle();
        };
        if (s0 < s1) {
#pragma unroll
            for (int i = 0; i < FR; ++i) fr[i] = key_operand(0, i);
            body(std::true_type(), 0);
            const int n = s1 - s0;
            for (int j = 1; j < n; ++j) body(std::false_type(), j);
#pragma unroll
            for (int i = 0; i < N; ++i) {
                fr[i % FR] = value_operand((n - 1) & VS, i);
                value_step(i);
            }
            spread_nans((n - 1) & VS, st.start + (int64_t)(s1 - 1) * 64);
        }
    } else {
        // of at most 64 rows: wavefronts without any widen only
        const bool live = !TWO || wave * 32 < rows;
        for (int j = 0; j < s1 - s0; ++j) {
            if (j) __syncthreads();
            if (live) {
#pragma unroll
                for (int i = 0; i < FR; ++i) fr[i] = key_operand(j & 1, i);
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    key_step(i);
                    if (i + FR < N) fr[i % FR] = key_operand(j & 1, i + FR);
                    else fr[i % FR] = value_operand(j & VS, i + FR - N);
                }
                hide(s0 + j, j & VS);
#pragma unroll
                for (int e = 0; e < 16; ++e) weigh(e, a.scale);
                settle();
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    value_step(i);
                    if (i + FR < N) fr[i % FR] = value_operand(j & VS, i + FR);
                }
                spread_nans(j & VS, st.start + (int64_t)(s0 + j) * 64);
            }
            widen_all((j + 1) & 1, (j + 1) & VS);
            fetch(s0 + j + 2);
        }
    }
    sum += __shfl_xor(sum, 32);
    if (!on) return;
    const float f = parts > 1 ? 1.0f : sum == 0.0f ? 0.0f : 1.0f / sum;
    const int64_t at = (unit * nsplit + sp) * a.rows_cap + m;
    uint16_t* const out = a.out + ((s.row0 + qi) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + qj) * a.kv.head_dim;
    auto each = [&](auto put) __attribute__((always_inline)) {
#pragma unroll
        for (int d = 0; d < G; ++d)
#pragma unroll
            for (int u = 0; u < 4; ++u)
                put(32 * d + 8 * u + 4 * h2, v4f{acc[d][4 * u] * f, acc[d][4 * u + 1] * f, acc[d][4 * u + 2] * f, acc[d][4 * u + 3] * f});
    };
    // (one branch for all: the elements' stores are many instructions)
    if (parts > 1) each([&](int ch, v4f v) { *reinterpret_cast<v4f*>(a.part_o + at * DP + ch) = v; });
    else if ((a.kv.head_dim & 3) == 0) each([&](int ch, v4f v) { if (ch < a.kv.head_dim) store_quad(out + ch, v); });
    else each([&](int ch, v4f v) { store_out4(out, ch, a.kv.head_dim, v); });
    if (parts > 1 && h2 == 0) {
        a.part_ml[2 * at] = mx;
        a.part_ml[2 * at + 1] = sum;
    }
}

// The ranges' results of a row: the common maximum, and the weighted sums.  `step` lies between two ranges' rows.
template <int DP>
__device__ __forceinline__ void join_ranges(const AttnArgs& a, int64_t at, int64_t step, int from, int count, int stride, int q, float& top, float& l, v4f& o) {
    top = M_NONE;
    l = 0.0f;
    o = v4f{0, 0, 0, 0};
#pragma unroll 4
    for (int k = from; k < count; k += stride) {
        const int64_t p = at + k * step;
        const float2 ml = *reinterpret_cast<const float2*>(a.part_ml + 2 * p);
        const v4f v = *reinterpret_cast<const v4f*>(a.part_o + p * DP + 4 * q);
        const float t = __builtin_fmaxf(top, ml.x), f0 = __builtin_amdgcn_exp2f(top - t), f1 = __builtin_amdgcn_exp2f(ml.x - t);
        l = l * f0 + ml.y * f1;
        o = o * f0 + v * f1;
        top = t;
    }
}
__device__ __forceinline__ void store_joined(const AttnArgs& a, const KvSeq& s, int h, int m, int q, float l, v4f o) {
    if (4 * q >= a.kv.head_dim) return;
    const int i = m / a.ratio, j = m - i * a.ratio;
    store_out4(a.out + ((s.row0 + i) * a.kv.n_heads * a.ratio + (int64_t)h * a.ratio + j) * a.kv.head_dim, 4 * q, a.kv.head_dim,
               o * (l == 0.0f ? 0.0f : 1.0f / l));
}

// Of few rows, a sequence and head a workgroup: d_pad / 4 lanes take four channels each of every GR-th
// range of a row, GR groups of them a row.
template <int G>
__global__ __launch_bounds__(512) void kv_join_kernel(AttnArgs a) {
    constexpr int DP = 32 * G, QL = DP / 4, NG = 512 / QL;
    __shared__ __attribute__((aligned(16))) float red[NG][DP];
    __shared__ float red_m[NG], red_l[NG];
    const int64_t b = blockIdx.x / (uint32_t)a.kv.n_heads;
    const int h = (int)(blockIdx.x - (uint32_t)b * (uint32_t)a.kv.n_heads);
    const int64_t r = a.joins[b];      // (undefined where the sequence has no rows)
    const KvSeq s = kv_seq(a.kv, b);
    const int rows = s.done * a.ratio, count = (int)(r & 0xFFFFF);
    if (rows == 0 || count <= 1) return;
    const int GR = rows >= NG ? 1 : NG / rows, pass = NG / GR;      // groups of a row, rows at a time
    const int q = threadIdx.x % QL, group = threadIdx.x / QL, sub = group % GR;
    for (int m0 = 0; m0 < rows; m0 += pass) {
        const int m = m0 + group / GR;
        const bool on = group < pass * GR && m < rows;
        float top = M_NONE, l = 0.0f;
        v4f o = v4f{0, 0, 0, 0};
        if (on) join_ranges<DP>(a, ((r >> 20) * a.kv.n_heads + h) * a.rows_cap + m, (int64_t)a.kv.n_heads * a.rows_cap, sub, count, GR, q, top, l, o);
        if (GR > 1) {      // uniform
            __syncthreads();
            if (on) {
                *reinterpret_cast<v4f*>(&red[group][4 * q]) = o;
                if (q == 0) {
                    red_m[group] = top;
                    red_l[group] = l;
                }
            }
            __syncthreads();
            if (!on || sub) continue;
            for (int k = 1; k < GR; ++k) {
                const float m1 = red_m[group + k], t = __builtin_fmaxf(top, m1), f0 = __builtin_amdgcn_exp2f(top - t), f1 = __builtin_amdgcn_exp2f(m1 - t);
                l = l * f0 + red_l[group + k] * f1;
                o = o * f0 + *reinterpret_cast<const v4f*>(&red[group + k][4 * q]) * f1;
                top = t;
            }
        }
        if (on) store_joined(a, s, h, m, q, l, o);
    }
}

// Of many rows, tiles of ROWS of them, KK a workgroup: d_pad / 4 lanes take a row's few ranges.
template <int G, int ROWS>
__global__ __launch_bounds__(256) void kv_join_many_kernel(AttnArgs a, int32_t nsplit) {
    constexpr int DP = 32 * G, QL = DP / 4, KK = 256 / QL;
    const uint32_t groups = ((uint32_t)a.rows_cap + KK - 1) / KK, unit = blockIdx.x / groups;
    const int q = threadIdx.x % QL, m = (int)((blockIdx.x - unit * groups) * KK + threadIdx.x / QL);
    const int64_t b = unit / (uint32_t)a.kv.n_heads;
    const int h = (int)(unit - (uint32_t)b * (uint32_t)a.kv.n_heads);
    const KvSeq s = kv_seq(a.kv, b);
    const int64_t rows = (int64_t)s.done * a.ratio;
    if (m >= rows || threadIdx.x / QL >= KK) return;
    const int m0 = m / ROWS * ROWS, m1 = (int)(m0 + ROWS < rows ? m0 + ROWS : rows);
    const Steps<64> st(a, s, m0, m1);
    const int count = many_parts(st.n, nsplit);
    if (count <= 1) return;
    float top, l;
    v4f o;
    join_ranges<DP>(a, (int64_t)unit * nsplit * a.rows_cap + m, a.rows_cap, 0, count, 1, q, top, l, o);
    store_joined(a, s, h, m, q, l, o);
}

// How a call runs: the kernel for few rows (16 mt of them at most) or the other one, and room for the
// ranges that sequences are cut into, so that there are workgroups for every CU.
struct Plan {
    int mt, waves;          // mt 0: many rows, of a workgroup of so many wavefronts
    bool two;               // many rows: weights of two terms
    int64_t units, row_tiles, groups, slots;
    int32_t target, nsplit, rows_cap;
    size_t o_bytes, ml_bytes, join_bytes, bytes;
};
int64_t few_round(int g, int mt) {
    int64_t r = 0;
    (void)kv_groups(32 * g, [&](auto gc) {
        r = mt == 1 ? Few<gc(), 1>::ROUND : mt == 2 ? Few<gc(), 2>::ROUND : Few<gc(), 4>::ROUND;
        return hipSuccess;
    });
    return r;
}
size_t up256(size_t n) { return (n + 255) / 256 * 256; }
// (a window leaves less to cut: never more ranges than without)
Plan plan_of(const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads, int64_t window) {
    Plan p = {};
    const int64_t ratio = n_q_heads / c.n_heads, rows = b.max_rows * ratio, all = b.max_pages * c.page_tokens;
    const int64_t cap = window && window + b.max_rows < all ? window + b.max_rows : all;
    // Four tiles of rows up to 96 channels (40 rows, 8 heads, 8 sequences of 8192 tokens, us a call: 64 channels 38, the other kernel
    // 39; 72: 48 and 47; 64 rows of 40 heads over 57600 tokens 102 and 140, 133 and 172), whose sums wider heads would not
    // leave in registers (128: 143 and, with weights of two terms as well, 57; 469 and 212).  Two tiles at any width (32 rows, 8 heads,
    // 32 sequences of 4096 tokens: 128 channels 52 and 139, 256: 147 and 208).
    p.mt = rows <= 16 ? 1 : rows <= 32 ? 2 : rows <= W4A4_KV_FEW_ROWS && c.d_pad <= 96 ? 4 : 0;
    p.two = !p.mt && rows <= W4A4_KV_FEW_ROWS && c.d_pad == 128;
    p.units = b.n_seqs * c.n_heads;
    p.rows_cap = (int32_t)rows;
    // eight wavefronts share a tile's widening where that leaves every CU a workgroup
    p.waves = !p.two && c.d_pad <= 128 && p.units * ((rows + 255) / 256) >= 256 ? 8 : 4;
    const int64_t tile = 32 * p.waves;
    p.row_tiles = p.mt ? 1 : (rows + tile - 1) / tile;
    p.nsplit = 1;
    if (p.mt) {
        // (tokens that start and end inside a step: two steps more)
        const int64_t most = p.units * ((cap / 32 + 2 + FEW_LEAST - 1) / FEW_LEAST), round = few_round(c.d_pad / 32, p.mt);
        // One round of workgroups where few sequences leave most of it to full ranges (one row over 57600
        // tokens, 40 heads: least kernel time of 90 calls 55 us, in two rounds 58); else about two, whose ranges are shorter, so that
        // the last ones end closer together (64 ragged sequences: least 194 us, in one round 213).  Sequences that fill the CUs by
        // themselves stay whole.
        const int64_t target = p.units <= round / 4 ? round - p.units : p.units < round ? 2 * round - p.units : round;
        p.groups = p.units;
        if (cap > 32 * FEW_LEAST && p.units < 4 * round) {
            p.target = (int32_t)target;
            p.groups = most < target + p.units ? most : target + p.units;
            p.slots = most < 2 * target ? most : 2 * target;
        }
    } else {
        // as many ranges as leave the last round of workgroups fullest
        const int64_t groups = p.units * p.row_tiles, seen = window ? window + tile / ratio + 1 : all;
        const int64_t most = (seen < all ? seen : all) / (64 * MANY_LEAST), round = p.waves == 4 && c.d_pad <= 128 ? 512 : 256;
        int64_t best = 1;
        for (int64_t n = 2; n <= most && n <= 64 && groups * n <= 2048; ++n)
            if (((groups * n + round - 1) / round) * best * 20 < ((groups * best + round - 1) / round) * n * 19) best = n;      // worth the join: 5%
        p.nsplit = (int32_t)best;
        p.groups = p.units * p.row_tiles * p.nsplit;
        p.slots = p.nsplit > 1 ? p.units * p.nsplit : 0;
    }
    // At most W4A4_KV_ATTENTION_WS_MOST: slots * rows are up to 2048 tiles of 256 rows (few rows: 4096 slots of 16, or of up
    // to 64 in 32 channels), 2^21 d_pad bytes and 2^22; joins and ranges of up to 4096 sequences below 2^18.
    p.o_bytes = up256((size_t)(p.slots * rows) * c.d_pad * 4);
    p.ml_bytes = up256((size_t)(p.slots * rows) * 8);
    p.join_bytes = p.target ? up256((size_t)b.n_seqs * 8) : 0;
    p.bytes = p.o_bytes + p.ml_bytes + p.join_bytes + (p.target && b.n_seqs > 64 ? up256((size_t)((p.groups + c.n_heads - 1) / c.n_heads) * sizeof(Range)) : 0);
    return p;
}

template <int G, int MT>
void run_few(const AttnArgs& a, const Plan& p, bool qb, hipStream_t st) {
    const dim3 grid((uint32_t)p.groups), threads(Few<G, MT>::NW * 64);
    if (qb) hipLaunchKernelGGL((kv_few_kernel<G, MT, true>), grid, threads, 0, st, a);
    else hipLaunchKernelGGL((kv_few_kernel<G, MT, false>), grid, threads, 0, st, a);
}

template <int G, int WAVES, bool TWO>
void run_many(const AttnArgs& a, const Plan& p, bool qb, hipStream_t st) {
    const dim3 grid((uint32_t)p.groups), threads(64 * WAVES);
    if (qb) hipLaunchKernelGGL((kv_many_kernel<G, WAVES, TWO, true>), grid, threads, 0, st, a, (uint32_t)p.row_tiles, p.nsplit);
    else hipLaunchKernelGGL((kv_many_kernel<G, WAVES, TWO, false>), grid, threads, 0, st, a, (uint32_t)p.row_tiles, p.nsplit);
}

}  // namespace

size_t kv_attention_ws(int64_t, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads) {
    return plan_of(b, c, n_q_heads, 0).bytes;
}

hipError_t launch_kv_attention(const w4a4_kv_rows& Q, int64_t n_rows, const w4a4_kv_batch& b, const w4a4_kv_cache& c, int32_t n_q_heads,
                               float scale, bool causal, int64_t window, uint16_t* O, void* ws, hipStream_t stream) {
    const Plan p = plan_of(b, c, n_q_heads, window);
    AttnArgs a;
    a.kv = kv_args(n_rows, b, c);
    a.q = Q.data;
    a.q_row = Q.row_stride;
    a.q_head = Q.head_stride;
    a.out = O;
    a.part_o = (float*)ws;
    a.part_ml = (float*)((uint8_t*)ws + p.o_bytes);
    a.joins = (int64_t*)((uint8_t*)ws + p.o_bytes + p.ml_bytes);
    a.ranges = (Range*)((uint8_t*)ws + p.o_bytes + p.ml_bytes + p.join_bytes);
    a.window = window;
    a.scale = scale * 1.44269504088896340736f;
    a.ratio = n_q_heads / c.n_heads;
    a.causal = causal ? 1 : 0;
    a.target = p.target;
    a.rows_cap = p.rows_cap;
    const bool qb = Q.dtype == W4A4_X_BF16;
    return kv_groups(c.d_pad, [&](auto gc) {
        constexpr int G = gc();
        if (p.target && b.n_seqs > 64)
            hipLaunchKernelGGL(kv_plan_kernel, dim3(1), dim3(1024), 0, stream, a, (int32_t)((p.groups + c.n_heads - 1) / c.n_heads));
        if (p.mt) {
            if (p.mt == 1) run_few<G, 1>(a, p, qb, stream);
            else if (p.mt == 2) run_few<G, 2>(a, p, qb, stream);
            else if constexpr (G <= 3) run_few<G, 4>(a, p, qb, stream);
        } else {
            if constexpr (G <= 4) {
                if (p.waves == 8) run_many<G, 8, false>(a, p, qb, stream);
            }
            if constexpr (G == 4) {
                if (p.two) run_many<G, 4, true>(a, p, qb, stream);
            }
            if (p.waves == 4 && !p.two) run_many<G, 4, false>(a, p, qb, stream);
        }
        const hipError_t e = hipGetLastError();
        if (e != hipSuccess || !p.slots) return e;
        constexpr int KK = 256 / (8 * G);      // rows of a workgroup
        const dim3 join((uint32_t)(p.mt ? p.units : p.units * ((p.rows_cap + KK - 1) / KK)));
        if (p.mt) hipLaunchKernelGGL((kv_join_kernel<G>), join, dim3(512), 0, stream, a);
        else if (p.waves == 4) hipLaunchKernelGGL((kv_join_many_kernel<G, 128>), join, dim3(256), 0, stream, a, p.nsplit);
        else if constexpr (G <= 4) hipLaunchKernelGGL((kv_join_many_kernel<G, 256>), join, dim3(256), 0, stream, a, p.nsplit);
        return hipGetLastError();
    });
}

}  // namespace w4a4

/*
 * w4a4.h -- C ABI of the MI355X (gfx950) W4A4 dual-branch linear library.
 *
 * The layer (page "W4A4 Quantization for Inference on Wan2.2-I2V-A14B (ICME 2026
 * Challenge)", xllm-io paper review, sec. 3.2-3.4):
 *
 *     Y = Q(X_J / s_J) . Q(s_J * W_J)  +  X_O . W_O
 *
 *   - SmoothQuant smoothing s_j = act_scale_j^alpha / weight_scale_j^(1-alpha)
 *     (sec. 3.2), folded into the weights offline; activations are divided by s
 *     at inference time and then quantized.
 *   - A static set O of k outlier input columns, the top-k of
 *     score_j = max_t |x_tj / s_j| over calibration tokens (sec. 3.3, scored
 *     after the fold per sec. 3.5), runs as a narrow BF16 branch on the raw
 *     (unsmoothed) columns; the rest, J, runs as strict MXFP4.
 *   - MXFP4 (named in sec. 1-2; OCP MX definition): E2M1 codes
 *     {0,+-0.5,+-1,+-1.5,+-2,+-3,+-4,+-6}, two per byte with the even K index
 *     in the low nibble, one E8M0 scale 2^(code-127) per group;
 *     E = floor(log2 amax) - 2 clamped at -127, amax = 0 -> code 0, a NaN/Inf
 *     in the group -> code 0xFF with all its nibbles 0; elements round to
 *     nearest, ties to the even code, saturating at 6, sign kept.
 *   - Weight scale groups (sec. 3.4): 1x32 along K, 32x32 tiles, or 128x1
 *     K-major stripes.  Activation scales are always 1x32 per token.
 *   - The J columns are compacted in ascending order and zero padded to
 *     K_pad = roundup(K_J, 128), K_J = d_in - k.
 *
 * Conventions for every entry point:
 *   - Return value: a w4a4_status; no exception or abort crosses the ABI.
 *   - "device" pointers are HIP device memory on the current device; "host"
 *     pointers are ordinary host memory.  The caller owns every buffer.
 *   - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *     Calls marked async only enqueue work on it; kernel faults surface at the
 *     caller's next synchronisation as HIP errors.
 *   - Shapes are validated before anything is enqueued.  T = 0 is a no-op.
 *   - Device pointers handed to the per-call entry points must be 16-byte
 *     aligned; buffers sized by the size queries are 256-byte aligned inside.
 *   - Calls on different streams that share a workspace race; the library keeps
 *     no global state and is otherwise reentrant (the one exception is the fixed
 *     device scratch array of w4a4_linear_noalloc).
 *   - The async per-call entry points enqueue kernels only: no allocation, no
 *     memset or copy, no synchronisation (memory that must start at zero is
 *     cleared by a kernel).  They may be captured into a HIP graph once the same
 *     call has run eagerly on the device (the first call sets kernel attributes).
 */
#ifndef W4A4_H
#define W4A4_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum w4a4_status {
    W4A4_OK = 0,
    W4A4_ERR_INVALID = 1,   /* null pointer, bad dtype/layout, k not in [0,d_in], alpha not in [0,1], negative size */
    W4A4_ERR_SHAPE = 2,     /* size beyond the supported range, or a blob/workspace that is too small */
    W4A4_ERR_ALIGN = 3,     /* a device pointer that is not 16-byte aligned */
    W4A4_ERR_DEVICE = 4,    /* a HIP runtime error from a launch, copy or synchronisation */
    W4A4_ERR_NONFINITE = 5, /* calibration data holds NaN or Inf */
    W4A4_ERR_SCRATCH = 6    /* w4a4_linear_noalloc: the call needs more workspace than
                               W4A4_NOALLOC_SCRATCH_BYTES */
} w4a4_status;

enum { W4A4_X_F32 = 0, W4A4_X_BF16 = 1 };

/* Weight scale-group layouts (page above, sec. 3.4). */
enum {
    W4A4_WS_1X32 = 0,          /* B_s [d_out][K_pad/32]: one scale per row per 32 K          */
    W4A4_WS_32X32_TILE = 1,    /* B_s [K_pad/32][ceil(d_out/32)]: 32 K x 32 rows per scale   */
    W4A4_WS_128X1_STRIPE = 2   /* B_s [d_out][K_pad/128]: 128 K x 1 row, K-major stripes      */
};

/* Largest supported input width (act-prep stages smoothed rows, K_pad fp32 each,
 * in LDS). */
#define W4A4_MAX_D_IN 32768
/* Largest d_in of the per-call outlier path (its top-k holds every column's score
 * in the registers of one 1024-lane workgroup, 16 per lane). */
#define W4A4_DYN_MAX_D_IN 16384

/* Packed layer descriptor, filled by w4a4_pack_weights.  Plain data: copy it
 * freely; it points into the caller's blob and owns nothing. */
typedef struct w4a4_packed {
    int64_t d_in, d_out;
    int32_t k;              /* |O|, number of BF16 outlier columns                        */
    int32_t layout;         /* W4A4_WS_*                                                  */
    int64_t k_j;            /* d_in - k                                                   */
    int64_t k_pad;          /* roundup(k_j, 128)                                          */
    int64_t k_ld;           /* row stride in elements of W_O and X_O: roundup(k, 32)      */
    const int32_t* colmap;  /* device [d_in]: p >= 0 = J column at compacted position p;
                               -(i+1) = outlier column O[i]                               */
    const float* s;         /* device [d_in] smoothing factors                            */
    const int32_t* O;       /* device [k], ascending                                      */
    const int32_t* J;       /* device [k_j], ascending                                    */
    const uint8_t* B_q;     /* device [d_out][k_pad/2] E2M1 codes of fl32(s_j * W[n][j])  */
    const uint8_t* B_s;     /* device, E8M0 codes in the layout's shape (see enum)        */
    const uint8_t* B_s_rows;/* device [k_pad/128][d_out][4]: the same codes, one per row per
                               32-block, step-major (the four codes of a 128-code step of
                               one row are adjacent, and consecutive rows follow), a
                               derived copy that the GEMM streams                         */
    const uint16_t* W_O;    /* device bf16 [d_out][k_ld], raw W[n][O[i]], zero padded     */
    const uint8_t* B_q_tiles;/* device, the codes of B_q re-laid for the GEMM's DMA (a derived
                               copy): [ceil(d_out/16)][k_pad/128][16][64] -- for each block of
                               16 rows and each 128-code step one contiguous 1 KiB run, row r
                               of the block at r*64, its 16-byte chunk c at chunk position
                               c ^ ((r >> 2) & 3); rows past d_out are zero                 */
} w4a4_packed;

/* Offsets (bytes) of the quantized activations inside a workspace. */
/* Layer packed for per-call outlier selection (w4a4_pack_weights_dyn): `base` is the
 * layer packed over all d_in columns (k = 0: J = every column, s folded in, B_q, B_s,
 * B_s_rows, B_q_tiles over K_pad = roundup(d_in, 128)); W_t = bf16_rne(W) transposed
 * keeps every column of W, contiguous, for the per-call W_O gather; k columns are
 * chosen per call. */
typedef struct w4a4_packed_dyn {
    w4a4_packed base;
    int32_t k;              /* outlier columns chosen per call, 0 <= k <= d_in             */
    int32_t reserved;
    const uint16_t* W_t;    /* device bf16 [d_in][d_out]: W_t[j][n] = bf16_rne(W[n][j])   */
} w4a4_packed_dyn;

typedef struct w4a4_ws_layout {
    size_t a_q;       /* uint8 activation E2M1 codes in the GEMM's tiled order,
                         [ceil(T/16)][k_pad/128][16][64]: the byte holding codes
                         p, p+1 (p even) of token t sits at
                           ((t/16)*(k_pad/128) + p/128)*1024 + (t%16)*64
                           + (c ^ ((t%16)/4))*16 + ((p%128)/2)%16,
                         c = (p%128)/32 -- the order of B_q_tiles; rows past T
                         inside the last 16-row block are left unwritten     */
    size_t a_s;       /* uint8 [k_pad/128][T][4] activation E8M0 scales (1x32),
                         step-major: for each 128-code step the four codes of
                         token t sit at [(step*T + t)*4 .. +3]                 */
    size_t x_o;       /* bf16  [T][k_ld] outlier columns, zero padded         */
    size_t partial;   /* fp32 partial sums of the GEMM's split-K tail tiles
                         (scratch the GEMM writes and reads back within one
                         call; empty when the tiles fill whole rounds of 256
                         workgroups or too few would be split)              */
    size_t total;     /* bytes needed                                         */
} w4a4_ws_layout;

/* Human-readable name of a status code (static storage). */
const char* w4a4_status_string(int status);

/* Column-wise max |x| of a row-major [rows][cols] device matrix (fp32 or bf16),
 * the per-channel magnitudes of sec. 3.2.  out_bits (device, [cols]) receives the
 * binary32 bit pattern of each maximum; a pattern >= 0x7F800000 means the
 * column holds NaN or Inf.  Async; out_bits is overwritten. */
int w4a4_column_absmax(const void* X, int x_dtype, int64_t rows, int64_t cols,
                       uint32_t* out_bits, void* stream);

/* Offline calibration (sec. 3.2-3.3, order per sec. 2 / 3.5): per-channel maxima of
 * X_cal (device [T_cal][d_in], fp32 or bf16) and of W (device fp32 [d_out][d_in],
 * nn.Linear orientation, reduced over d_out), then on the host in double:
 *   s_j = max(a_j,1e-5)^alpha / max(w_j,1e-5)^(1-alpha), rounded once to fp32,
 *   score_j = fl32(a_j / s_j), O = top-k scores (ties -> smaller j), ascending.
 * s_out [d_in] and O_out [k] are HOST buffers; act_scale_out / weight_scale_out
 * (host [d_in]) may be NULL.  Blocking: synchronises `stream`.  Allocates a
 * small device scratch (8*d_in bytes) internally.  Returns W4A4_ERR_NONFINITE if
 * either input holds NaN/Inf. */
int w4a4_calibrate_scales(const void* X_cal, int x_dtype, int64_t T_cal, int64_t d_in,
                          const float* W, int64_t d_out, float alpha, int32_t k,
                          float* s_out, int32_t* O_out,
                          float* act_scale_out, float* weight_scale_out, void* stream);

/* Bytes of the device blob that w4a4_pack_weights fills. */
int w4a4_packed_size(int64_t d_in, int64_t d_out, int32_t k, int layout, size_t* bytes);

/* Offline fold + split + pack (sec. 3.2 fold, 3.3 split, 3.4 block packing):
 * W device fp32 [d_out][d_in]; s (host [d_in], s_j > 0 finite) and O (host [k],
 * strictly ascending, in [0,d_in)) as produced by calibration (s = 1, k = 0 gives
 * naive W4A4).  Writes B_q = E2M1(fl32(s_j * W[n][J[p]])) with E8M0 scales in
 * `layout`, W_O = bf16_rne(W[n][O[i]]), plus s, O, J and the column map, into
 * `blob` (device, blob_bytes >= w4a4_packed_size), and fills *desc.  Blocking:
 * synchronises `stream` (host inputs are staged before return). */
int w4a4_pack_weights(const float* W, int64_t d_in, int64_t d_out, const float* s,
                      const int32_t* O, int32_t k, int layout, void* blob,
                      size_t blob_bytes, w4a4_packed* desc, void* stream);

/* Workspace offsets and size for T tokens with this layer. */
int w4a4_workspace_layout(int64_t T, const w4a4_packed* desc, w4a4_ws_layout* out);
int w4a4_workspace_size(int64_t T, const w4a4_packed* desc, size_t* bytes);

/* Act-prep (sec. 3.2 "divide by s, then quantize", sec. 3.3 split): X device
 * [T][d_in] fp32 or bf16, row-major contiguous.  For each token: x~ = fl32(x / s_j)
 * (IEEE binary32 division, subnormals kept) over the J columns in ascending order,
 * 1x32 E8M0 + E2M1 codes into A_q/A_s (A_s step-major, see w4a4_ws_layout);
 * X_O = bf16_rne(x) over the O columns.
 * Async on `stream`; never allocates. */
int w4a4_quantize_activations(const void* X, int x_dtype, int64_t T, const w4a4_packed* desc,
                              void* ws, size_t ws_bytes, void* stream);

/* Dual-branch GEMM (sec. 3.3) on quantized activations already in `ws`:
 * Y[t][n] = sum_b 2^(Ea+Eb) sum_{p in b} a.b  (block-scaled FP4 MFMA)
 *         + sum_i X_O[t][i] W_O[n][i]         (BF16 MFMA, same fp32 accumulator)
 * Y device fp32 [T][d_out].  Reads A_q, A_s and X_O of `ws`; writes its `partial`
 * region when the plan splits the last round of 256 x 256 output tiles along K
 * (results then sum the K ranges' fp32 partials in a fixed order, so a given shape
 * is bit-reproducible).  Async; never allocates. */
int w4a4_gemm_prequantized(void* ws, size_t ws_bytes, int64_t T, const w4a4_packed* desc,
                           float* Y, void* stream);

/* The per-call path: act-prep then the dual-branch GEMM.  Async; never allocates. */
int w4a4_linear(const void* X, int x_dtype, int64_t T, const w4a4_packed* desc, float* Y,
                void* ws, size_t ws_bytes, void* stream);

/* Per-call outlier selection, the online variant that sec. 3.3 / sec. 4 attribute to
 * MixQ and that the page's method replaces with a static top-k.  Each call scores its
 * own tokens, score_j = fl32(max_t |x_tj| / s_j), compared as binary32 bit patterns of
 * |score| (numeric order for finite values and +Inf, a NaN above +Inf), larger first,
 * ties to the smaller column; O = the top k, ascending.  The J branch keeps every
 * column at its own K position (K_pad = roundup(d_in, 128)) with the chosen columns'
 * activations set to zero, so its 32-blocks are the column blocks of X rather than
 * blocks of the compacted J; the O branch is bf16 X_O . bf16 W_O with W_O gathered per
 * call from W_t.  d_in <= W4A4_DYN_MAX_D_IN and even; s as for w4a4_pack_weights.
 *
 * w4a4_packed_dyn_size / w4a4_pack_weights_dyn: one device blob (blocking,
 * like w4a4_pack_weights).  w4a4_workspace_dyn_layout / _size: for T tokens, the static
 * workspace of the k-column layer over K_pad = roundup(d_in, 128) followed by the
 * per-call column maxima (uint32 bit patterns [d_in]), O (int32 [k]), the column map
 * (int32 [d_in]: j for a J column, -(i+1) for the i-th outlier) and W_O (bf16
 * [d_out][roundup(k, 32)]).  w4a4_linear_dyn: X device [T][d_in] fp32 or bf16, Y
 * device fp32 [T][d_out]; async, never allocates; a call reuses its workspace, so
 * concurrent calls need one each. */
typedef struct w4a4_ws_dyn_layout {
    w4a4_ws_layout base;    /* a_q, a_s, x_o as for the static path, k_pad over all columns */
    size_t colmax, O, colmap, W_O, total;
} w4a4_ws_dyn_layout;
int w4a4_packed_dyn_size(int64_t d_in, int64_t d_out, int32_t k, int layout, size_t* bytes);
int w4a4_pack_weights_dyn(const float* W, int64_t d_in, int64_t d_out, const float* s, int32_t k,
                          int layout, void* blob, size_t blob_bytes, w4a4_packed_dyn* desc,
                          void* stream);
int w4a4_workspace_dyn_layout(int64_t T, const w4a4_packed_dyn* desc, w4a4_ws_dyn_layout* out);
int w4a4_workspace_dyn_size(int64_t T, const w4a4_packed_dyn* desc, size_t* bytes);
int w4a4_linear_dyn(const void* X, int x_dtype, int64_t T, const w4a4_packed_dyn* desc, float* Y,
                    void* ws, size_t ws_bytes, void* stream);

/* FFN block with the down layer's activation prep fused into the up projection
 * (sec. 3.1 / 3.5: up projection, GELU-tanh, down projection; sec. 3.2-3.4 for the
 * down layer's smoothing, outlier split and MXFP4 codes).  H = bf16(gelu_tanh(bf16(
 * X W_up^T))) never goes to memory: the up GEMM's epilogue writes the down layer's
 * A_q, A_s and X_O directly, bit-identical to w4a4_quantize_activations(H, down).
 *
 * Precondition on the packing: output feature f of `up` must be the down layer's
 * input column P[f], with P = (the down layer's J columns, ascending, then its O
 * columns, ascending), i.e. `up` is packed from the rows W_up[P[f]].  Permuting the
 * rows of W_up does not change its calibration (the per-input-column maxima), and
 * GELU is elementwise.  With 1x32 or 128x1 weight scales (one row per scale group)
 * the permuted layer is the same layer with its outputs reordered; with 32x32 tiles
 * the permutation also regroups the rows that share a tile scale, so the permuted
 * layer is a different, equally valid quantization of W_up.  The up layer's output
 * feature f < k_j is the down layer's compacted J position f and f >= k_j its outlier
 * slot f - k_j.  The library cannot check the permutation.
 *
 * w4a4_ffn_workspace_layout / _size: for T tokens, the up layer's workspace (offsets
 * in `up` relative to up_base), the down layer's (relative to down_base) and
 * RN64(1 / s_j) of the down layer's J columns (double [down.k_j]).
 * w4a4_ffn_up_quantize: act-prep of X for `up`, then the up GEMM with GELU and the
 * down layer's act-prep in its epilogue; afterwards the down layer's A_q, A_s, X_O sit
 * in the workspace at down_base + down.{a_q, a_s, x_o}, in the layout
 * w4a4_ws_layout documents.  w4a4_ffn_forward: the same, then the down GEMM into Y
 * (fp32 [T][down.d_out]).  Errors: INVALID (null pointer, bad dtype, T < 0, a bad
 * descriptor), SHAPE (up.d_out != down.d_in, workspace too small), ALIGN (pointers
 * not 16-byte aligned), DEVICE.  Async; never allocates. */
typedef struct w4a4_ffn_ws_layout {
    w4a4_ws_layout up;     /* relative to up_base                                   */
    w4a4_ws_layout down;   /* relative to down_base                                 */
    size_t up_base, down_base;
    size_t rinv;           /* double [down.k_j]                                     */
    size_t total;
} w4a4_ffn_ws_layout;

int w4a4_ffn_workspace_layout(int64_t T, const w4a4_packed* up, const w4a4_packed* down,
                              w4a4_ffn_ws_layout* out);
int w4a4_ffn_workspace_size(int64_t T, const w4a4_packed* up, const w4a4_packed* down, size_t* bytes);
int w4a4_ffn_up_quantize(const void* X, int x_dtype, int64_t T, const w4a4_packed* up,
                         const w4a4_packed* down, void* ws, size_t ws_bytes, void* stream);
int w4a4_ffn_forward(const void* X, int x_dtype, int64_t T, const w4a4_packed* up,
                     const w4a4_packed* down, float* Y, void* ws, size_t ws_bytes, void* stream);

/* Layer-wise choice of alpha and k (sec. 3.2 gives alpha in [0.5, 0.7] for the FFN up
 * projection; sec. 4 lists per-layer alpha and k, and sec. 6 names tuning them per
 * layer as the next step; the pages give no selection rule, so the rule here is the
 * smallest output error on calibration tokens).  For every pair (alphas[a], ks[b]):
 * calibrate s and O on X_cal (as w4a4_calibrate_scales), pack W in `layout` (as
 * w4a4_pack_weights), run the layer on X_cal (as w4a4_linear), and score it by the
 * relative Frobenius error ||Y_q - Y_ref||_F / ||Y_ref||_F against the unquantized
 * product Y_ref = X_cal W^T (fp32 inputs and accumulation; the sums of squares in
 * fp64, added in a fixed order, so the result is deterministic).
 *   X_cal  device [T_cal][d_in] fp32 or bf16; W device fp32 [d_out][d_in];
 *   alphas host [n_alpha] in [0,1]; ks host [n_k] in [0,d_in];
 *   scratch device, scratch_bytes >= w4a4_search_scratch_size (16-byte aligned);
 *   err_out host [n_alpha * n_k]: err_out[a * n_k + b];
 *   best_out host [2]: (a, b) of the smallest finite error, first on ties, (-1, -1)
 *   if none is finite.
 * Blocking (synchronises `stream` once per candidate); never allocates.  Errors as
 * the calls it composes (W4A4_ERR_NONFINITE for non-finite calibration data). */
int w4a4_search_scratch_size(int64_t T_cal, int64_t d_in, int64_t d_out, const int32_t* ks, int n_k,
                             int layout, size_t* bytes);
int w4a4_search_alpha_k(const void* X_cal, int x_dtype, int64_t T_cal, int64_t d_in, const float* W,
                        int64_t d_out, const float* alphas, int n_alpha, const int32_t* ks, int n_k,
                        int layout, void* scratch, size_t scratch_bytes, double* err_out,
                        int32_t* best_out, void* stream);

/* The FFN up projection with its activation fused (sec. 3.1 / 3.5: ffn.0 is followed
 * by GELU-tanh, whose bf16 output feeds ffn.2): the dual-branch GEMM of
 * w4a4_gemm_prequantized / w4a4_linear, with every fp32 output y stored as
 * H = bf16_rne(gelu_tanh(bf16_rne(y))) -- bit-identical to w4a4_gelu_tanh_bf16 over
 * the fp32 Y of the unfused call, without writing or re-reading Y.
 * H device bf16 [T][d_out] (16-byte aligned).  Async; never allocate. */
int w4a4_gemm_prequantized_gelu_bf16(void* ws, size_t ws_bytes, int64_t T,
                                     const w4a4_packed* desc, uint16_t* H, void* stream);
int w4a4_linear_gelu_bf16(const void* X, int x_dtype, int64_t T, const w4a4_packed* desc,
                          uint16_t* H, void* ws, size_t ws_bytes, void* stream);

/* GELU-tanh between the FFN up (ffn.0) and down (ffn.2) projections named in
 * sec. 3.1 / 3.5: H = bf16_rne(gelu_tanh(bf16_rne(Y))), gelu_tanh(x) =
 * 0.5x(1+tanh(sqrt(2/pi)(x+0.044715x^3))) in fp32.  Y device fp32 [n], H device
 * bf16 [n].  Async. */
int w4a4_gelu_tanh_bf16(const float* Y, int64_t n, uint16_t* H, void* stream);

/* For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): w4a4_linear with its
 * workspace in a fixed device array that the library holds on every GPU it runs on,
 * W4A4_NOALLOC_SCRATCH_BYTES long, until the process ends.  The caller still passes X
 * and Y (as for w4a4_linear).  The call makes no allocation and frees nothing; its
 * first call on a device looks up that device's copy of the array.
 *   - T tokens need w4a4_workspace_size(T, desc) bytes of it; a larger need returns
 *     W4A4_ERR_SCRATCH before anything is enqueued.
 *   - The results are those of w4a4_linear, bit for bit (same kernels, same plan).
 *   - Every call on one GPU uses that GPU's one array: calls that overlap in time on
 *     one GPU (other streams, other host threads) race and give undefined results.
 *     Nothing in the array needs to start at zero; it keeps the last call's contents.
 * Async on `stream`. */
#define W4A4_NOALLOC_SCRATCH_BYTES ((size_t)128 << 20)
int w4a4_linear_noalloc(const void* X, int x_dtype, int64_t T, const w4a4_packed* desc, float* Y,
                        void* stream);

/* ------------------------------------------------------------------------------------
 * FP8 linear layer with block scales: the 8-bit layer for the projections that four bits
 * cannot carry (the page keeps up to five blocks at a higher precision, sec. 2).
 *
 *     Y[t][n] = sum_b s_x[t][b] s_w[n / 128][b] sum_{p in block b} q_x[t][p] q_w[n][p]
 *
 *   - Codes are OCP E4M3 (largest value 448), blocks b are 128 inputs; activations have
 *     one scale per token and block, weights one per 128 outputs x 128 inputs.
 *   - Scale of a block with largest magnitude a:
 *       W4A4_FP8_SCALE_F32:  s = max(fl32(a / 448), 2^-60)
 *       W4A4_FP8_SCALE_E8M0: s = the smallest power of two >= 2^-60 with a <= 448 s
 *     (the floor keeps products of two scales normal numbers; blocks below 448 * 2^-60
 *     lose codes to it).  A NaN or Inf in the block gives s = NaN and zero codes (every
 *     output that reads the block is NaN).  A zero block has s = 2^-60.
 *   - Codes: e4m3_rne(fl32(x / s)), nearest, ties to the even mantissa, signs kept.
 *   - Sums, and the products with the scales, are binary32, and fp32 outputs are those
 *     sums.  For bf16 outputs of more than 64 tokens the matrix instructions may take the
 *     codes as FP8 and drop what is 13 bits below the largest product beside it: 1.4e-5 to 4e-5
 *     of the outputs' root mean square, a fiftieth of their own rounding (1 to 3% of the
 *     outputs round to a neighbour of the nearest bf16 number).  The product of two scales
 *     s_x s_w is taken first: with scales of a checkpoint it has to be a normal number.
 *   - The inputs are zero padded to k_pad = roundup(d_in, 128); 1 <= d_in <=
 *     W4A4_FP8_MAX_D, 1 <= d_out <= W4A4_FP8_MAX_D, any number of tokens whose outputs a
 *     launch can count (2^33 tokens, 2^39 outputs; W4A4_ERR_SHAPE above).
 * The conventions at the top of this file hold: caller-owned buffers, 16-byte aligned
 * device pointers, T = 0 a no-op, no allocation or synchronisation, graph capture.
 * Calls are bit-reproducible for a given shape. */
enum { W4A4_FP8_SCALE_F32 = 0, W4A4_FP8_SCALE_E8M0 = 1 };
enum { W4A4_Y_F32 = 0, W4A4_Y_BF16 = 1 };
#define W4A4_FP8_MAX_D 1048576

/* n_mat weight matrices of one shape (one for a linear layer, one per expert for a
 * mixture of experts).  Plain data that points into the caller's blob. */
typedef struct w4a4_fp8_packed {
    int64_t n_mat, d_in, d_out;
    int64_t k_pad;           /* roundup(d_in, 128)                                          */
    int64_t n_pad;           /* roundup(d_out, 16)                                          */
    int32_t scale_kind;      /* W4A4_FP8_SCALE_*: also the kind of the activations' scales  */
    int32_t reserved;
    const uint8_t* codes;    /* device E4M3 [n_mat][n_pad/16][k_pad/128][2][64][16]: each run
                                of 16 rows x 128 inputs is 2 KiB in the order the matrix
                                instructions read it; the byte of row r, input p sits at
                                  ((r/16)*(k_pad/128) + p/128)*2048 + ((p/64)%2)*1024
                                  + ((p/8)%4)*256 + (r%16)*16 + ((p/32)%2)*8 + p%8;
                                rows past d_out and inputs past d_in are zero              */
    const float* scales;     /* device [n_mat][ceil(d_out/128)][k_pad/128], as binary32 for
                                both kinds                                                 */
} w4a4_fp8_packed;

/* Bytes of the device blob of n_mat packed matrices. */
int w4a4_fp8_packed_size(int64_t n_mat, int64_t d_in, int64_t d_out, size_t* bytes);

/* Quantize W (device [n_mat][d_out][d_in], fp32 or bf16: w_dtype is W4A4_X_F32 or
 * W4A4_X_BF16) into `blob` (device, blob_bytes >= w4a4_fp8_packed_size) and fill *desc.
 * A 128 x 128 block that the matrix's edge cuts takes its scale from the part inside.
 * Async on `stream`. */
int w4a4_fp8_pack_weights(const void* W, int w_dtype, int64_t n_mat, int64_t d_in, int64_t d_out,
                          int scale_kind, void* blob, size_t blob_bytes, w4a4_fp8_packed* desc,
                          void* stream);

/* The same from weights that are quantized already (a checkpoint): codes device uint8
 * [n_mat][d_out][d_in] E4M3, scales device [n_mat][ceil(d_out/128)][ceil(d_in/128)], fp32
 * for W4A4_FP8_SCALE_F32, uint8 E8M0 codes for W4A4_FP8_SCALE_E8M0 (value 2^(c-127); 0xFF
 * is NaN).  Values are taken as they are.  Async on `stream`. */
int w4a4_fp8_pack_codes(const uint8_t* codes, const void* scales, int64_t n_mat, int64_t d_in,
                        int64_t d_out, int scale_kind, void* blob, size_t blob_bytes,
                        w4a4_fp8_packed* desc, void* stream);

/* Offsets (bytes) inside a workspace for T tokens. */
typedef struct w4a4_fp8_ws_layout {
    size_t a_q;       /* activation codes in the order of w4a4_fp8_packed.codes, tokens as
                         rows: [ceil(T/16)][k_pad/128][2][64][16]; rows past T unwritten   */
    size_t a_s;       /* fp32 [k_pad/128][roundup(T, 32)] activation scales; tokens past T
                         unwritten                                                         */
    size_t partial;   /* fp32 partial sums of K ranges (written and read back within a
                         call; empty when the plan does not split)                         */
    size_t count;     /* int32 ranges done (of a few tokens' plan that splits; cleared by
                         every call that multiplies)                                       */
    size_t total;
} w4a4_fp8_ws_layout;
int w4a4_fp8_workspace_layout(int64_t T, const w4a4_fp8_packed* desc, w4a4_fp8_ws_layout* out);
int w4a4_fp8_workspace_size(int64_t T, const w4a4_fp8_packed* desc, size_t* bytes);

/* Activation codes and scales of X (device [T][d_in] fp32 or bf16, row-major contiguous)
 * into ws.  desc->n_mat must be 1, here and in the calls below.  Where they lie depends on T
 * and d_in only, and they on scale_kind too: one call serves every layer of that d_in and
 * scale_kind (gate and up, or query, key and value projections), in a workspace that is large
 * enough for each of them.  Async. */
int w4a4_fp8_quantize_activations(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* desc,
                                  void* ws, size_t ws_bytes, void* stream);
/* The product on quantized activations in ws.  Y device [T][d_out], fp32 or bf16 (the
 * fp32 sums rounded once to nearest even): y_dtype is W4A4_Y_F32 or W4A4_Y_BF16.  Async. */
int w4a4_fp8_gemm_prequantized(void* ws, size_t ws_bytes, int64_t T, const w4a4_fp8_packed* desc,
                               void* Y, int y_dtype, void* stream);
/* Both.  Async. */
int w4a4_fp8_linear(const void* X, int x_dtype, int64_t T, const w4a4_fp8_packed* desc, void* Y,
                    int y_dtype, void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------------------
 * Mixture-of-experts layer for a few tokens (decoding), weights in the FP8 block format
 * above.  For each token t of X [T][d], with E experts of width f:
 *
 *     l[e]  = sum_i X[t][i] router[e][i]                            (fp32 sums)
 *     S     = the top_k experts by l: larger first, ties to the lower index, a NaN before
 *             every number
 *     p[e]  = exp(l[e] - max l) / sum of the same over S (renormalize != 0) or over all
 *             experts (renormalize == 0)
 *     g, u  = gate_e . x, up_e . x     with x = bf16_rne(X[t]),     (fp32 sums)
 *     h     = bf16_rne(silu(g) u)      or, W4A4_MOE_GELU_TANH: h = bf16_rne(gelu_tanh(u))
 *     Y[t]  = sum_{e in S} p[e] (down_e . h)                        (fp32 sums)
 *
 * The experts' products are bound by reading the codes of the chosen experts, so the
 * activations stay bf16 (the matrix instructions take E4M3 weights widened to bf16, which
 * is exact): no activation quantization error at no cost in time.
 * Limits: 1 <= T <= W4A4_MOE_MAX_T tokens a call (W4A4_ERR_SHAPE above), E <=
 * W4A4_MOE_MAX_E, top_k <= W4A4_MOE_MAX_K and <= E, d and f <= W4A4_MOE_MAX_D. */
enum { W4A4_MOE_SILU_GATED = 0, W4A4_MOE_GELU_TANH = 1 };
#define W4A4_MOE_MAX_T 128
#define W4A4_MOE_MAX_E 1024
#define W4A4_MOE_MAX_K 32
#define W4A4_MOE_MAX_D 65536

typedef struct w4a4_moe {
    w4a4_fp8_packed gate;    /* n_mat = E, d -> f; not read for W4A4_MOE_GELU_TANH          */
    w4a4_fp8_packed up;      /* n_mat = E, d -> f                                           */
    w4a4_fp8_packed down;    /* n_mat = E, f -> d                                           */
    const void* router;      /* device [E][d], row-major contiguous                         */
    int32_t router_dtype;    /* W4A4_X_F32 or W4A4_X_BF16                                   */
    int32_t top_k;
    int32_t renormalize;
    int32_t activation;      /* W4A4_MOE_*                                                  */
} w4a4_moe;

/* Offsets (bytes) inside a workspace for T tokens: what a call leaves there. */
typedef struct w4a4_moe_ws_layout {
    size_t logits;    /* fp32 [T][roundup(E, 4)]                                            */
    size_t xb;        /* bf16 [T][roundup(d, 128)], zero padded (left alone where X itself is
                         bf16 and d a multiple of 128)                                      */
    size_t ids;       /* int32 [T][top_k]: the chosen experts, largest logit first          */
    size_t p;         /* fp32 [T][top_k]: exp(l - max), divided by the sum over all experts
                         when renormalize == 0 (otherwise the down step divides by the sum
                         over the row)                                                      */
    size_t h;         /* bf16 [T * top_k][roundup(f, 128)], zero padded                     */
    size_t place;     /* int32 [T][top_k]: which of its expert's tokens it is, in their order */
    size_t count;     /* int32 [roundup(d, 16) / 16]: the down step's parts that are done   */
    size_t part;      /* fp32: their sums                                                   */
    size_t total;
} w4a4_moe_ws_layout;
int w4a4_moe_workspace_layout(int64_t T, const w4a4_moe* moe, w4a4_moe_ws_layout* out);
int w4a4_moe_workspace_size(int64_t T, const w4a4_moe* moe, size_t* bytes);

/* The whole layer: X device [T][d] fp32 or bf16, Y device [T][d] fp32 or bf16.  Async;
 * never allocates.  Three launches: router logits, the chosen experts' up projections, their
 * down projections with the weighted sum. */
int w4a4_moe_forward(const void* X, int x_dtype, int64_t T, const w4a4_moe* moe, void* Y, int y_dtype,
                     void* ws, size_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* W4A4_H */

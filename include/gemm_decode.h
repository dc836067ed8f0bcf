/*
 * gemm_decode.h -- C ABI of libgemm_decode.so: block-quantized weight x
 * activation products for LLM decode (batch-1 GEMV) and prefill (small-M /
 * M-token GEMM) on AMD Instinct MI355X (gfx950).
 *
 * Conventions for every entry point below
 * ---------------------------------------
 *  - Pointers named in a "device" argument are HIP device (or host-coherent)
 *    memory owned by the caller; the library never allocates, frees or keeps
 *    a pointer after returning. Inputs are read only; outputs are fully
 *    overwritten (never accumulated into).
 *  - `stream` is a hipStream_t passed as void* (NULL = the null stream).
 *    Calls only enqueue work: results are valid once the caller has
 *    synchronised with `stream`.
 *  - Sizes are int64_t element counts. Every argument is validated on the
 *    host before any HIP call; on a validation failure nothing is launched
 *    and a negative status is returned, so every status except GD_EHIP can
 *    be produced on a machine without a GPU.
 *  - No entry point aborts, throws, or silently switches to another code
 *    path: a shape a kernel cannot run is an error.
 *  - gemm_decode_last_error() returns a thread-local description of the last
 *    non-zero status raised on the calling thread.
 *
 * Page citations name the page's title and the section on it:
 *   "browseml-gpu.js" (browseML on the GPU, exactly),
 *   "block_q8_matmul_nt.wgsl" (kopitiam-gpu),
 *   "BonsaiのWebGPUカーネルを読み解く" (habakan blog, on PrismML's Bonsai
 *    WebGPU demo),
 *   "web-xpu-ops" (package README),
 *   "roofline.html" (Decode roofline — your GPU).
 */
#ifndef GEMM_DECODE_H
#define GEMM_DECODE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ------------------------------------------------------------------ status */
#define GD_OK       0
#define GD_EINVAL  (-1) /* null pointer, non-positive or overflowing size     */
#define GD_ESHAPE  (-2) /* a size is not a multiple of the format's block      */
#define GD_EALIGN  (-3) /* a pointer is not aligned as the layout requires     */
#define GD_EHIP    (-4) /* HIP reported an error (launch, configuration)        */
#define GD_ERANGE  (-5) /* a size exceeds a documented kernel limit            */

/* Short constant name of a status code ("GD_OK", "GD_EINVAL", ...). */
const char *gemm_decode_status_string(int status);
/* Thread-local text describing the last failure on this thread ("" if none). */
const char *gemm_decode_last_error(void);
/* ABI version of this header (incremented on incompatible changes). */
int gemm_decode_abi_version(void);
#define GEMM_DECODE_ABI_VERSION 4

/* ====================================================================
 * Q1_0 . q8_0  ("browseml-gpu.js": header comment "The arithmetic, as the
 * reference does it", Q1_DOT_WGSL, Q1_MM_WGSL, packQ1, packQ8)
 * ====================================================================
 * Wire formats (as the page defines them):
 *  - Q1_0 weight block, 18 bytes per 128 weights: f16 d0 little-endian,
 *    then 128 sign bits, element j in byte 2 + j/8, bit j%8; bit 1 means
 *    +d0, bit 0 means -d0. A row of K weights is K/128 consecutive blocks;
 *    rows follow each other ("AoS" weights).
 *  - q8_0 activation block, 34 bytes per 32 activations: f16 d1, then 32
 *    int8. Activation column c is K/32 consecutive blocks starting at byte
 *    c*(K/32)*34.
 *
 * Result (bit-exact, one correct bit pattern per output): for each row and
 * accumulation lane l = 0..7 over blocks i in order,
 *   s      = sum_{e=4l}^{4l+3} (bit(32k+e) ? q_e : -q_e)   (int8 negation
 *            wraps: -(-128) = -128), k = sub-block 0..3 (activation block 4i+k)
 *   ab_l   = d1_k*s for k = 0, then ab_l = ab_l + d1_k*s for k = 1..3
 *   acc_l  = fma(d0_i, ab_l, acc_l)       (acc_l starts at +0)
 *   y      = ((acc0+acc4)+(acc2+acc6)) + ((acc1+acc5)+(acc3+acc7)).
 * f16 scales are decoded exactly, subnormals included.
 *
 * Q1 planes (the library's resident weight layout, written once by
 * q1_repack and read by the GEMV; the page's packQ1 repacks for the same
 * reason). With R64 = rows rounded up to 64, nb = K/128 and nb8 = nb rounded
 * up to 8:
 *  - bits plane, R64*nb*16 bytes, 16-byte aligned: u32 index
 *    ((((r/64)*nb + i)*2 + h)*64 + r%64)*2 + m holds, for half h (lanes
 *    4h..4h+3) and word m (sub-blocks 2m, 2m+1) of block i of row r, the sign
 *    bits of elements 32k + 4l + j with l = 4h + jj (jj = 0..3),
 *    k = 2m + kk (kk = 0..1), j = 0..3, at bit (8*jj + 2 + 4*kk + j) mod 32.
 *    (Each 4-bit group, pre-shifted by 2, indexes a 16-entry table of 4-byte
 *    products; the two halves are read by two different waves.)
 *  - scale plane, R64*nb8*2 bytes, 16-byte aligned: u16 index
 *    ((r/64)*(nb8/8) + i/8)*512 + (r%64)*8 + i%8 holds the f16 bits of d0
 *    of block i of row r.
 *  - Padding rows (r >= rows) and padding blocks (i >= nb) are zero.
 * ==================================================================== */

/* Sizes in bytes of the two Q1 planes for a rows x K weight (host only, no
 * GPU needed). Errors: GD_EINVAL (null out pointer, rows < 1, K < 1,
 * overflow), GD_ESHAPE (K % 128 != 0). */
int q1_planes_bytes(int64_t rows, int64_t K, size_t *bits_bytes, size_t *scale_bytes);

/* One-time repack of AoS Q1_0 weights into the Q1 planes (integer byte
 * moves; "browseml-gpu.js", packQ1).
 *   w_aos       device, rows*(K/128)*18 bytes, 2-byte aligned.
 *   bits_plane  device, q1_planes_bytes(...).bits_bytes, 16-byte aligned.
 *   scale_plane device, q1_planes_bytes(...).scale_bytes, 16-byte aligned.
 * Every byte of both planes is written (padding with zeros). Errors:
 * GD_EINVAL, GD_ESHAPE (K % 128), GD_EALIGN, GD_EHIP. */
int q1_repack(const void *w_aos, int64_t rows, int64_t K,
              void *bits_plane, void *scale_plane, void *stream);

/* y = W . a for n_act q8_0 activation columns, bit-exact as above.
 *   bits_plane, scale_plane  device Q1 planes of a rows x K weight (q1_repack).
 *   a_q8   device, n_act*(K/32)*34 bytes of q8_0 blocks, 2-byte aligned.
 *   y      device f32 [n_act][rows] (column c at y + c*rows, as Q1_MM_WGSL's
 *          O[col*rows + row]), 4-byte aligned.
 * n_act = 1 is the batch-1 decode GEMV; n_act > 1 (the small-M product)
 * keeps every column's bits: one launch runs every column as its own GEMV
 * (each re-reads the weights, mostly from cache).
 * Limits: rows <= 2^31 - 64, n_act <= 65535. Errors: GD_EINVAL, GD_ESHAPE
 * (K % 128), GD_EALIGN, GD_ERANGE, GD_EHIP. */
int q1_q8_gemv(const void *bits_plane, const void *scale_plane, const void *a_q8,
               float *y, int64_t rows, int64_t K, int64_t n_act, void *stream);

/* One independent batch-1 problem of a grouped launch. */
typedef struct gd_q1_problem {
    const void *bits_plane;   /* device Q1 bits plane, 16-byte aligned     */
    const void *scale_plane;  /* device Q1 scale plane, 16-byte aligned    */
    const void *a_q8;         /* device q8_0 activation (one column)       */
    float *y;                 /* device f32 [its rows]                      */
    int64_t rows;             /* its rows, 1 .. the launch's rows; 0 (or a
                                 value outside that range) means the
                                 launch's rows. Planes are sized for it.   */
} gd_q1_problem;

/* `count` independent batch-1 Q1_0 . q8_0 GEMVs with a common K in one
 * launch, each with its own weights, row count, activation and output; the
 * same kernel body and the same bits as q1_q8_gemv with n_act = 1.
 *   problems  device array of `count` gd_q1_problem, 8-byte aligned. The
 *             pointers and row counts inside it are read by the kernel and
 *             cannot be validated by the host: they must satisfy
 *             q1_q8_gemv's rules for that problem's rows.
 *   rows      the largest row count of the problems (sets the grid).
 * Limits: 1 <= count <= 65535. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN,
 * GD_ERANGE, GD_EHIP. */
int q1_q8_gemv_grouped(const gd_q1_problem *problems, int64_t count,
                       int64_t rows, int64_t K, void *stream);

/* ====================================================================
 * Sign-bit prefill GEMM  ("BonsaiのWebGPUカーネルを読み解く", figure on
 * PrismML's decode/prefill kernels: q1_bits holds the sign bits of 32
 * weights per u32, q1_scales one scale per 32 weights, bit 1 -> +1.0,
 * bit 0 -> -1.0; prefill is the compute-bound M-token case)
 * ====================================================================
 *   y[m][n] = sum_g scales[n][g] * sum_{j<32} x[m][32g+j] * (bit_j ? +1 : -1)
 *   x       device f32 [M][K] row-major, 16-byte aligned, finite. The
 *           product runs on fp16 matrix cores: each row of x is scaled, in
 *           each eighth of K (ceil(K/256) groups), by the power of two that
 *           brings its largest |x| there into [2^14, 2^15), each output's
 *           scales by the power of two that does the same for its largest
 *           |scale|, and both are split into a high and a low
 *           fp16 part (x = xh + xl, s = sh + sl, each within 2^-22 of its
 *           value while normal in fp16); a 32-weight group contributes
 *           xh*sh + xl*sh + xh*sl of its signed products, accumulated in
 *           f32 on the matrix cores per eighth of K; each eighth's sum is
 *           unscaled exactly and the eight are added in a fixed order.
 *           Error within 1e-5 of ||y||_inf (about 5e-7 on N(0,1)
 *           activations and |N(0,0.02)| scales at K = 4096).
 *   w_bits  device u32 [N][K/32], bit j of word g = weight 32g+j (LSB
 *           first), 4-byte aligned.
 *   w_scales device f32 [N][K/32], 4-byte aligned.
 *   y       device f32 [M][N], 4-byte aligned.
 *   workspace  device scratch of at least q1_sign_gemm_workspace_bytes(M,
 *           N, K) bytes, 16-byte aligned, owned by the caller. A first
 *           kernel writes the split activations and the weights in the
 *           matrix-core layout (see q1_sign_pack) into it for the second;
 *           calls that share it must be ordered on one stream. Its contents
 *           on entry do not matter and on return are unspecified.
 * Requires K % 32 == 0. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE
 * (M, N or K above 2^31 - 1, workspace too small), GD_EHIP. */
int q1_sign_gemm(const float *x, const uint32_t *w_bits, const float *w_scales,
                 float *y, int64_t M, int64_t N, int64_t K,
                 void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes q1_sign_gemm needs: 4*K per token (tokens padded to a
 * multiple of 16) plus 32 per padded token (an exponent per eighth of K),
 * plus 16 per output and pair of 32-weight groups (ceil(K/64) pairs), plus
 * 4 per output. Host only.
 * Errors: GD_EINVAL, GD_ESHAPE (K % 32 != 0), GD_ERANGE. */
int q1_sign_gemm_workspace_bytes(int64_t M, int64_t N, int64_t K, size_t *bytes);

/* Bytes of the packed sign-bit weights written by q1_sign_pack:
 * 32 * N * ceil(K/64) + 4 * N. Host only. Errors: GD_EINVAL, GD_ESHAPE,
 * GD_ERANGE. */
int q1_sign_packed_bytes(int64_t N, int64_t K, size_t *bytes);

/* One-time repack of the page's sign words and scales (the layouts
 * q1_sign_gemm takes) for the calls below, in three sections (P = 16 * N *
 * ceil(K/64) bytes each for the first two):
 *   [0, P)      for the table kernels (q1_sign_gemv, q1_sign_gemm_lut4):
 *               for each output n and pair of 32-weight groups (g, g+1),
 *               g even, the u32x4 {bits[n][g], bits[n][g+1], scale[n][g],
 *               scale[n][g+1]} (scales as f32 bit patterns) at index
 *               (g/2)*N + n, a missing group g+1 = K/32 having bits 0 and
 *               scale 0, so the words of one group pair for consecutive
 *               outputs are contiguous;
 *   [P, 2P)     for the matrix-core GEMM: for each group g and output n the
 *               u32x2 {bits[n][g], sh | sl << 16} at index g*N + n, sh and
 *               sl the fp16 high and low parts of scale[n][g] * 2^c_n;
 *   [2P, 2P+4N) the int32 c_n per output: the exponent that puts the
 *               output's largest |scale| in [2^14, 2^15) (0 if all are 0).
 *   w_bits, w_scales  as for q1_sign_gemm, 4-byte aligned.
 *   w_packed          device, q1_sign_packed_bytes(N, K) bytes, 16-byte
 *                     aligned; written whole.
 * Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int q1_sign_pack(const uint32_t *w_bits, const float *w_scales, int64_t N, int64_t K,
                 void *w_packed, void *stream);

/* q1_sign_gemm on weights packed once by q1_sign_pack (no per-call
 * regrouping launch); same numerics and bits as q1_sign_gemm. The workspace
 * holds only the split activations and row exponents: at least
 * 4*K*M16 + 32*M16 bytes (M16 = M rounded up to 16), so any size
 * q1_sign_gemm_workspace_bytes(M, N, K) returns is enough. x, w_packed and
 * workspace 16-byte aligned, y 4-byte. Errors: GD_EINVAL, GD_ESHAPE,
 * GD_EALIGN, GD_ERANGE, GD_EHIP. */
int q1_sign_gemm_packed(const float *x, const void *w_packed, float *y,
                        int64_t M, int64_t N, int64_t K,
                        void *workspace, size_t workspace_bytes, void *stream);

/* Sign-bit decode GEMV (the page's decode kernel, one token at a time):
 * y[m][n] = sum_g scale[n][g] * sum_{j<32} s(n, 32g+j) x[m][32g+j] for each
 * of M activation rows, from packed weights. Each workgroup turns the row
 * into LDS tables of the signed sums of every 4 consecutive elements (16
 * per 4), so a nibble of signs costs one table read and one add; partial
 * sums round in f32 (within 1e-5 of ||y||_inf of the exact sum).
 *   x  device f32 [M][K], 16-byte aligned; y device f32 [M][N], 4-byte.
 * Requires K % 32 == 0, 1 <= M <= 65535. Every row reads the weights once
 * more: meant for a few tokens (use q1_sign_gemm(_packed) for prefill).
 * Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int q1_sign_gemv(const float *x, const void *w_packed, float *y,
                 int64_t M, int64_t N, int64_t K, void *stream);

/* The page's LUT4 prefill GEMM (binary-lut4-matmul: 16 partial sums of
 * every 4 activations in workgroup memory, one read per nibble, reused over
 * a 16-token x 512-output tile), kept as the comparator of the matrix-core
 * GEMM: same y and contract as q1_sign_gemv, for any M. */
int q1_sign_gemm_lut4(const float *x, const void *w_packed, float *y,
                      int64_t M, int64_t N, int64_t K, void *stream);

/* ====================================================================
 * Block-scaled int8 matmul_nt  ("block_q8_matmul_nt.wgsl": PACKING,
 * ACCUMULATION ORDER, quant_at, main)
 * ====================================================================
 *   y[r][c] = sum_b scales[c][b] * sum_{t<32} x[r][32b+t] * q[c][32b+t]
 *   x       device f32 [m][k] row-major, 16-byte aligned.
 *   quants  device u32 [n][k/4]: element t of row c in byte t%4 of word
 *           c*k/4 + t/4 (little-endian), two's-complement int8; 16-byte
 *           aligned.
 *   scales  device f32 [n][k/32], 4-byte aligned.
 *   y       device f32 [m][n], 4-byte aligned.
 * Requires k % 32 == 0 (an error, where the page's kernel would silently
 * drop a tail) and k % 16 == 0 rows of quants on 16-byte boundaries (implied
 * by k % 32 == 0). x must be finite. Results agree with the page's order
 * within 1e-5 of ||y||_inf. For 2 <= m <= 16 and k <= 1024 the block
 * sub-totals run on fp16 matrix cores: each activation row is scaled by a
 * power of two that brings its largest |x| into [2^14, 2^15), split into
 * high and low fp16 parts, and the sub-total is scaled back exactly, so
 * rows of any finite magnitude keep ~22 bits. Limits: m <= 16 and
 * m*k <= 16384 (the activation rows are staged whole in LDS). Errors:
 * GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int blockq8_matmul_nt(const float *x, const uint32_t *quants, const float *scales,
                      float *y, int64_t m, int64_t k, int64_t n, void *stream);

/* ====================================================================
 * Ternary bitplane GEMV  ("BonsaiのWebGPUカーネルを読み解く", section on
 * Bonsai: P bit set where w = +1, N bit set where w = -1, and
 * dot = 2(pc(P&X) - pc(N&X)) - pc(P) + pc(N) for a binary plane X)
 * ====================================================================
 * The int8 activation enters as its eight two's-complement bit planes B_b
 * (x = sum_{b<7} 2^b B_b - 128 B_7), so the integer dot is a weighted sum of
 * per-plane popcount identities and is exact.
 * ==================================================================== */

/* Bit planes of an int8 activation vector (or `count` vectors).
 *   x_q     device int8 [count][K], 16-byte aligned.
 *   planes  device u32 [count][8][K/32]: word m of plane b holds bit b of
 *           the two's-complement bytes x_q[32m .. 32m+31], element 32m+j at
 *           bit j. 16-byte aligned.
 * Requires K % 32 == 0, 1 <= count <= 65535. Errors: GD_EINVAL, GD_ESHAPE,
 * GD_EALIGN, GD_ERANGE, GD_EHIP. */
int ternary_act_bitplanes(const int8_t *x_q, int64_t count, int64_t K,
                          uint32_t *planes, void *stream);

/* dot[r] = sum_k w[r][k] * x[k] (exact int32) and y[r] = (float)dot[r] * s
 * with s = w_scale * x_scale rounded once to f32.
 *   w_pos, w_neg  device u32 [rows][K/32], bit j of word m = element 32m+j;
 *                 16-byte aligned. An element with both bits set counts as 0.
 *   x_planes      device u32 [8][K/32] from ternary_act_bitplanes, 16-byte
 *                 aligned.
 *   y             device f32 [rows]; dot_out device int32 [rows] or NULL.
 * Requires K % 32 == 0 and K <= 65536 (so |dot| <= 128*K < 2^24 and
 * f32(dot) is exact; the planes, 8*K/8 bytes, are staged whole in LDS). Errors: GD_EINVAL,
 * GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int ternary_gemv(const uint32_t *w_pos, const uint32_t *w_neg, float w_scale,
                 const uint32_t *x_planes, float x_scale, float *y, int32_t *dot_out,
                 int64_t rows, int64_t K, void *stream);

typedef struct gd_ternary_problem {
    const uint32_t *w_pos;     /* device u32 [rows][K/32]  */
    const uint32_t *w_neg;     /* device u32 [rows][K/32]  */
    const uint32_t *x_planes;  /* device u32 [8][K/32]     */
    float *y;                  /* device f32 [rows]        */
    int32_t *dot_out;          /* device int32 [rows] or NULL */
    float w_scale;
    float x_scale;             /* used when x_scale_dev is NULL */
    const float *x_scale_dev;  /* device f32 (e.g. from ternary_quantize_act) or NULL;
                                  when set, the activation scale is read from it */
} gd_ternary_problem;

/* `count` independent ternary GEMVs of one shape in one launch (one decode
 * step's projections of a given shape); same kernel body and bits as
 * ternary_gemv, the scale product w_scale * x_scale taken with the scale
 * read from x_scale_dev where that is set. `problems` is a device array (8-byte aligned) whose inner
 * pointers must satisfy ternary_gemv's rules. Limits: 1 <= count <= 65535.
 * Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int ternary_gemv_grouped(const gd_ternary_problem *problems, int64_t count,
                         int64_t rows, int64_t K, void *stream);

/* ====================================================================
 * Activation quantization  ("web-xpu-ops", operator table: quantize, and
 * the reciprocal and rounding rows of its q4 format table, which state the
 * same convention)
 * ====================================================================
 * The step before each GEMV. Per group (a token for the ternary path, a
 * 32-element block for q8_0): absmax = max |x|; codes are Math.round of
 * x * (127/absmax), the reciprocal formed in f64, ties toward +infinity
 * (floor(v) + (v - floor(v) >= 0.5) in f64), clamped to [-127, 127]; the
 * scale is the f64 quotient absmax/127 rounded to f32. A group whose absmax
 * is 0 gets scale 0 and zero codes. Inputs must be finite (NaN or infinity
 * give unspecified codes). Codes and scales are bit-exact with this rule.
 * ==================================================================== */

/* f32 activations -> q8_0 blocks in the layout q1_q8_gemv reads
 * ("browseml-gpu.js", packQ8: 34 bytes, f16 d then 32 int8 codes). The
 * pages fix the block, not its quantizer: the rule above is applied to each
 * block of 32, and d is the f32 scale rounded to f16 (nearest even).
 *   x     device f32 [n][K], 16-byte aligned.
 *   a_q8  device, n * (K/32) * 34 bytes (column c at byte c * (K/32) * 34),
 *         2-byte aligned; written whole.
 * Requires K % 32 == 0, n >= 1, n * K/32 <= 2^34. Errors: GD_EINVAL,
 * GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int q8_0_quantize(const float *x, void *a_q8, int64_t n, int64_t K, void *stream);

/* f32 activations -> per-token int8 codes (the rule above over each token's
 * K values), written as the bit planes ternary_gemv reads, and the scales.
 *   x        device f32 [count][K], 16-byte aligned.
 *   planes   device u32 [count][8][K/32], the layout of
 *            ternary_act_bitplanes; 4-byte aligned (ternary_gemv itself
 *            needs 16).
 *   x_scale  device f32 [count] (for gd_ternary_problem.x_scale_dev).
 * Requires K % 32 == 0, 1 <= count <= 2^31 - 1, K <= 2^30. Errors:
 * GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int ternary_quantize_act(const float *x, int64_t count, int64_t K, uint32_t *planes,
                         float *x_scale, void *stream);

/* ====================================================================
 * Split-K decode attention  ("BonsaiのWebGPUカーネルを読み解く", section on
 * split-K flash decode attention: per split a running maximum, denominator
 * and rescaled output; a merge that rescales every split to the global
 * maximum)
 * ====================================================================
 * One decode token: for query head h and its KV head kv = h / (n_heads /
 * n_kv_heads), s_j = scale * q[h] . k[kv][j] over positions j < kv_len, and
 * out[h] = sum_j exp(s_j - max s) v[kv][j] / sum_j exp(s_j - max s). The
 * pages leave the score scale to the caller (1/sqrt(head_dim) is usual).
 * f32 throughout; within 1e-5 of ||out||_inf of the f64 definition.
 * ==================================================================== */

/* Workspace bytes attn_decode_splitk needs: num_splits * n_heads *
 * (head_dim + 2) * 4, num_splits = 0 meaning the split count the call picks
 * for that shape. Host only. Errors as attn_decode_splitk's validation. */
int attn_decode_workspace_bytes(int64_t n_heads, int64_t n_kv_heads, int64_t head_dim,
                                int64_t kv_len, int64_t num_splits, size_t *bytes);

/*   q         device f32 [n_heads][head_dim], 16-byte aligned.
 *   k_cache,  device f32 [n_kv_heads][kv_stride][head_dim]: position j of KV
 *   v_cache   head kv at row kv * kv_stride + j; rows j < kv_len are read.
 *             16-byte aligned.
 *   out       device f32 [n_heads][head_dim], 4-byte aligned.
 *   num_splits  number of key ranges run in parallel (each ceil(kv_len /
 *             num_splits) keys, trailing splits may be empty); 0 picks about
 *             512 workgroups in all, at least 64 keys each.
 *   workspace device, attn_decode_workspace_bytes(...) bytes, 16-byte
 *             aligned: per split and head the running output, maximum and
 *             denominator, read by the merge launch of the same call.
 * Requires head_dim == 128, n_heads % n_kv_heads == 0 with n_heads /
 * n_kv_heads in {1, 2, 4, 8}, kv_len >= 1, kv_stride >= kv_len,
 * num_splits <= 65535. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE,
 * GD_EHIP. */
int attn_decode_splitk(const float *q, const float *k_cache, const float *v_cache, float *out,
                       int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, int64_t kv_len,
                       int64_t kv_stride, float scale, int64_t num_splits,
                       void *workspace, size_t workspace_bytes, void *stream);

/* attn_decode_splitk without a workspace, for callers that cannot allocate
 * device memory (code under HIP graph capture, serving loops or harnesses
 * that forbid hipMalloc). Same arguments, validation, kernels and results
 * as attn_decode_splitk; the split partials go to a scratch array inside the
 * library (GD_ATTN_NOALLOC_MAX_BYTES per device, held from the first call on
 * that device until the process ends). The call allocates nothing. Requires
 * num_splits * n_heads * (head_dim + 2) * 4 <= GD_ATTN_NOALLOC_MAX_BYTES
 * (num_splits = 0: the split count the call picks), else GD_ERANGE before
 * any launch. Calls on one device share its scratch: calls that overlap on
 * one device (several streams, several host threads) race; order them.
 * Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
#define GD_ATTN_NOALLOC_MAX_BYTES (4 * 1024 * 1024)
int attn_decode_splitk_noalloc(const float *q, const float *k_cache, const float *v_cache, float *out,
                               int64_t n_heads, int64_t n_kv_heads, int64_t head_dim, int64_t kv_len,
                               int64_t kv_stride, float scale, int64_t num_splits, void *stream);

/* ====================================================================
 * Norm with an 8-bit output, and readers of the activation formats
 * ====================================================================
 * The step between the residual stream and a product. With
 *   h = x + residual                (rounded to the stream's type)
 *   p = h * weight,  rstd = 1 / sqrt(mean over the row of h^2 + eps)
 * the norm is y = rstd * p, quantized as above but for the factor (below). rstd
 * divides out of y * factor, so the codes are Math.round(p * (127 * (1 / max|p|)))
 * (each step rounded in f64, where p is exact) and the scale is max|p| * rstd
 * / 127, evaluated in f64 from left to right and rounded to f32. A group whose
 * products are all 0 gets scale 0 and zero codes. Sums are f64; inputs and h
 * must be finite.
 *
 * The factor. The norms and the cache write form it as 127 * (1 / absmax), each
 * step rounded in f64, where q8_0_quantize and ternary_quantize_act form the
 * quotient 127 / absmax: that is how torch evaluates `127 / tensor`, and rows
 * quantized by such code are reproduced bit for bit. The two factors differ by at
 * most 2^-52 of themselves, so a code of one value can differ between the entry
 * points only where value * 127 / absmax is an exact half (for the norms, whose
 * products have 48 bits, or within 2^-45 of one): it is then one of the two whole
 * numbers beside the half, which are equally near. Scales are the same. f32 data
 * hardly meet that; of random blocks of bf16 values about one in ninety has such
 * a code.
 *
 * Element types of the entry points from here on that take a `dtype`: */
#define GD_F32  0
#define GD_F16  1
#define GD_BF16 2

/* h = x + residual, and the norm of h as q8_0 blocks (what q1_q8_gemv reads;
 * one scale per 32 elements, the f32 scale rounded to f16).
 *   x         device dtype [n][K].
 *   residual  device dtype [n][K] or NULL (h = x).
 *   weight    device f32 [K].
 *   h_out     device dtype [n][K], the sum h, or NULL. May be x or residual
 *             itself (the stream updated in place); must not overlap them
 *             otherwise.
 *   a_q8      device, n * (K/32) * 34 bytes, 2-byte aligned; written whole.
 * x, residual, weight and h_out 16-byte aligned. Requires K % 32 == 0,
 * K <= 2^30, 1 <= n < 2^23, finite eps >= 0. Errors: GD_EINVAL, GD_ESHAPE,
 * GD_EALIGN, GD_ERANGE, GD_EHIP. */
int rmsnorm_q8_0(const void *x, const void *residual, const float *weight, void *h_out,
                 void *a_q8, int64_t n, int64_t K, float eps, int32_t dtype, void *stream);

/* The same with one scale per row, as the bit planes and scale that
 * ternary_gemv reads (the outputs of ternary_quantize_act).
 *   planes   device u32 [n][8][K/32], 4-byte aligned (ternary_gemv itself
 *            needs 16).
 *   x_scale  device f32 [n].
 * Limits and errors as rmsnorm_q8_0. */
int rmsnorm_ternary_act(const void *x, const void *residual, const float *weight, void *h_out,
                        uint32_t *planes, float *x_scale, int64_t n, int64_t K, float eps,
                        int32_t dtype, void *stream);

/* The values that activations stand for: f32(code) * scale in f32, rounded
 * to dtype. y device dtype [n][K], 16-byte aligned. Requires K % 32 == 0 and
 * n * K < 2^34 - 1024. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE,
 * GD_EHIP. */
int q8_0_dequantize(const void *a_q8, void *y, int64_t n, int64_t K, int32_t dtype, void *stream);
int ternary_dequantize_act(const uint32_t *planes, const float *x_scale, void *y, int64_t n, int64_t K,
                           int32_t dtype, void *stream);

/* ====================================================================
 * 8-bit cache of keys and values
 * ====================================================================
 * A pool of pages, each of page_size positions of every KV head. A row (one
 * position of one head) is head_dim int8 codes with an f16 scale per 32 dims,
 * quantized as q8_0_quantize does but for the factor, which is the norms' (a code
 * can differ by one, and only where it falls on an exact half); it stands for
 * code * scale. Position p of page g of head h is row (g * n_kv_heads + h) * page_size + p of each plane;
 * slot s names position s % page_size of page s / page_size. A cache without
 * paging is a pool whose page b holds all of sequence b.
 * The struct is read on the host during the call; the planes are device
 * memory, 16-byte aligned. head_dim is 64, 128 or 256, page_size a multiple
 * of 16, n_kv_heads <= 4096. Scales are finite and not negative in rows that
 * are used; rows that were never stored are not used (any bytes may be there). */
typedef struct gd_kv_q8 {
    int8_t *k_codes;      /* [n_pages][n_kv_heads][page_size][head_dim]          */
    uint16_t *k_scales;   /* f16 bits, [n_pages][n_kv_heads][page_size][head_dim/32] */
    int8_t *v_codes;
    uint16_t *v_scales;
    int64_t n_pages, page_size, n_kv_heads, head_dim;
} gd_kv_q8;

/* Rotary frequencies f_i = base^(-2i/rot_dim), i < rot_dim/2, for contexts
 * past the trained length (`factor` >= 1 in all kinds but NONE). */
#define GD_ROPE_NONE   0
#define GD_ROPE_LINEAR 1 /* f_i / factor                                       */
#define GD_ROPE_NTK    2 /* base * factor^(rot_dim / (rot_dim - 2)) as base     */
#define GD_ROPE_YARN   3 /* f_i for pairs that turn more than `high` times over
                            original_len, f_i / factor below `low` times, a
                            linear ramp over the pair index between; cos and
                            sin times `attention` (0: 0.1 ln(factor) + 1)      */
#define GD_ROPE_LLAMA3 4 /* as YARN with the ramp linear in the number of turns
                            and no attention factor                            */
typedef struct gd_rope_scaling {
    int32_t kind;
    int32_t reserved;     /* 0 */
    double factor;
    double original_len;  /* YARN, LLAMA3: the trained length                  */
    double low, high;     /* YARN, LLAMA3: turns, 0 < low < high (1 and 32, 1 and 4) */
    double attention;     /* YARN */
} gd_rope_scaling;

/* The table kv_q8_store reads: table[p][i] = (cos, sin) of p * f_i, angles in
 * f64, rounded once to f32. Written once per model.
 *   table    device f32 [n_pos][rot_dim/2][2], 16-byte aligned.
 *   scaling  host struct or NULL (GD_ROPE_NONE).
 * Requires rot_dim % 8 == 0, rot_dim <= 256, base > 1, n_pos * rot_dim/2 <
 * 2^32 - 256. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int rope_table(float *table, int64_t n_pos, int64_t rot_dim, double base,
               const gd_rope_scaling *scaling, void *stream);

/* Rotates q and k by their tokens' positions and writes k and v to the cache.
 * Pair (x1, x2) becomes (x1 cos - x2 sin, x2 cos + x1 sin); the pairs are
 * dims (i, i + rot_dim/2), or (2i, 2i+1) if `interleaved`; dims from rot_dim
 * on stay. For k the sum of the two products is taken to 2^-46 of the larger
 * one and rounded to f32, which the cache quantizes; for q the second product
 * is rounded to f32 and the first fused with the sum, and q_out rounds that to
 * dtype.
 *   q, k, v    device dtype, token t's heads at q + t * q_stride (n_heads head
 *              rows of head_dim), k + t * k_stride, v + t * v_stride
 *              (n_kv_heads): parts of one projection's row, for instance.
 *              Strides in elements, multiples of 16 bytes, at most 2^36. All values
 *              finite, those of v and of the rotated k (a pair can grow by a factor
 *              of sqrt 2, times the table's) below 65504 * 127: the scales are f16.
 *   q_out      device dtype [n_tok][n_heads][head_dim]; may be q itself if
 *              q_stride is n_heads * head_dim or n_tok is 1, must not overlap q
 *              otherwise, nor k or v. n_heads may be 0, with q and q_out NULL
 *              (only the cache is written).
 *   rope       device f32 [n_pos][rot_dim/2][2] from rope_table, with
 *   positions  device int32 [n_tok]; both NULL: nothing is rotated (n_pos and
 *              rot_dim are then ignored). A token whose position is outside
 *              [0, n_pos) is left out: its q_out row and its slot stay as
 *              they were.
 *   slots      device int64 [n_tok], the slot each token is stored at. A token
 *              whose slot is outside the pool (-1: padding) is not stored;
 *              its q is still rotated. Slots of one call must differ: of two
 *              tokens with one slot, the row is left as a mixture.
 * rot_dim a multiple of 8, at most head_dim; n_heads <= 65536; n_tok < 2^24.
 * q, k, v, q_out and rope 16-byte aligned. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE,
 * GD_EHIP. */
int kv_q8_store(const gd_kv_q8 *cache, const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                const void *v, int64_t v_stride, void *q_out, const float *rope, int64_t n_pos,
                int64_t rot_dim, int32_t interleaved, const int32_t *positions, const int64_t *slots,
                int64_t n_tok, int64_t n_heads, int32_t dtype, void *stream);

/* Reads rows back: token t of k_out and v_out is the row that slots[t] names,
 * f32(code) * f32(scale) rounded to dtype; a slot outside the pool reads as
 * zeros.
 *   slots         device int64 [n_tok] (any order, repeats allowed).
 *   k_out, v_out  device dtype [n_tok][n_kv_heads][head_dim], 16-byte aligned;
 *                 one of them may be NULL.
 * n_tok < 2^24. Errors as kv_q8_store. */
int kv_q8_load(const gd_kv_q8 *cache, const int64_t *slots, void *k_out, void *v_out, int64_t n_tok,
               int32_t dtype, void *stream);

/* Attention of the last tokens of each of n_seqs sequences over the cache: one
 * decode token, a chain, or a tree of drafted tokens (at most 64, stored in
 * the cache beforehand). Sequence b has kv_lens[b] keys, its T_b query tokens
 * the last of them. Query token t sees every key before the drafted ones, and
 * drafted key i if bit i of its mask word is set (a tree's token: itself and
 * its ancestors) or, without masks, if i <= t.
 *   s_j = scale * q . k_j, then softcap * tanh(s_j / softcap) if softcap > 0;
 *   out = sum over seen j of exp(s_j - max s) v_j / sum of exp(s_j - max s);
 * scores, without a softcap, lie within f32's range (|s_j| < 2^126). A row that
 * sees no key gets zeros. A drafted key that no row of its sequence
 * sees need not be stored.
 *   q, out      device dtype [n_q][n_heads][head_dim], finite; head h reads KV
 *               head h / (n_heads / n_kv_heads). 16-byte aligned; out must not
 *               overlap q.
 *   page_table  device int32 [n_seqs][max_pages]: page_table[b][i] holds the
 *               positions i * page_size .. of sequence b. Keys on a page
 *               outside the pool are not seen. NULL: sequence b is page b
 *               (needs n_pages >= n_seqs; max_pages is ignored).
 *   kv_lens     device int32 [n_seqs], taken as at most max_kv_len (0: the
 *               sequence's rows get zeros).
 *   q_start     device int32 [n_seqs + 1], increasing: the query rows of
 *               sequence b are q_start[b] .. q_start[b + 1] - 1, at most max_q
 *               (rows past that, and rows of no sequence, stay as they were).
 *               NULL: max_q rows each (needs n_q = n_seqs * max_q).
 *   tree_mask   device u64 [n_q], one word per query row, or NULL.
 *   max_kv_len  the longest kv_lens: sets the split of the keys, at most
 *               max_pages * page_size.
 *   workspace   device, attn_decode_q8_workspace_bytes(...) bytes, 16-byte
 *               aligned; one made for the largest call serves every smaller
 *               one. Calls that share it must be ordered.
 * Accuracy, against the definition without roundings, with V the largest |v| of
 * the sequence, S the largest scale * sum |q_i k_i| (the products' magnitudes: where
 * they cancel, far above |s|) and n its keys:
 *   f32        (1e-5 + 2^-28 n + 2^-19 S) V: q and the weights keep 22 bits, sums
 *              are f32. With a softcap 2^-18 S.
 *   f16, bf16  2^-10 V and half a step of the result more: the weights and the
 *              values (code * scale) are rounded to f16 for their product, and q
 *              loses what lies below 2^-25 of its row's largest value.
 * Requires n_heads % n_kv_heads == 0, max_q <= 64, n_q <= n_seqs * max_q,
 * n_heads <= 4096, n_seqs <= 65535, max_kv_len <= 2^30, finite scale,
 * 0 <= softcap <= 1e30. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int attn_decode_q8(const gd_kv_q8 *cache, const void *q, void *out, const int32_t *page_table,
                   int64_t max_pages, const int32_t *kv_lens, const int32_t *q_start,
                   const uint64_t *tree_mask, int64_t n_seqs, int64_t n_q, int64_t n_heads,
                   int64_t max_q, int64_t max_kv_len, float scale, float softcap, int32_t dtype,
                   void *workspace, size_t workspace_bytes, void *stream);

/* Workspace bytes of such a call: enough for every call of the same head counts
 * and head_dim that is no larger in n_seqs, n_q, max_q and max_kv_len, and never
 * less for a larger call (a call itself may be cut into more parts than a larger
 * one). Host only. Errors as its size checks. */
int attn_decode_q8_workspace_bytes(int64_t n_seqs, int64_t n_q, int64_t n_heads, int64_t n_kv_heads,
                                   int64_t head_dim, int64_t max_q, int64_t max_kv_len, size_t *bytes);

/* ====================================================================
 * Measurement kernels  ("roofline.html": the FILL kernel writes a non-zero,
 * incompressible pattern so reads reach real DRAM; the read kernel streams
 * 16-byte words through an XOR into a sink)
 * ==================================================================== */

/* Fill `bytes` (multiple of 16, 16-byte aligned) with a hash of the 16-byte
 * word index and `seed`. Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_EHIP. */
int gemm_decode_fill(void *buf, size_t bytes, uint32_t seed, void *stream);

/* Read `bytes` (multiple of 16, 16-byte aligned) `passes` times with
 * 16-byte loads, XOR-reducing into sink (device u32 [sink_words], written).
 * Errors: GD_EINVAL, GD_ESHAPE, GD_EALIGN, GD_ERANGE, GD_EHIP. */
int gemm_decode_stream_read(const void *buf, size_t bytes, int32_t passes,
                            uint32_t *sink, int64_t sink_words, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GEMM_DECODE_H */

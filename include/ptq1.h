/*
 * ptq1.h -- C ABI of the MI355X (gfx950) PTQ1_0 ternary linear layer.
 *
 * The method: weights quantised to -1, 0, +1 with a 16-bit scale for every 128
 * weights, five trits packed into a byte in base 3 (1.75 bits per weight),
 * after every weight matrix was multiplied by a 1024-wide Walsh-Hadamard
 * butterfly with a sign pattern; at inference the same rotation is applied to
 * the activations before every folded matmul and undone on embedding rows
 * ("A 27B model in 5.5 GB: Bonsai ternary on Ferrox, locally", section
 * "What Bonsai is").  A trit is read from its byte on the float pipeline as
 * floor(3^(n+1) u) - 3 floor(3^n u), u = byte/256 (same page, section
 * "What Ferrox does with it").  Decode is a matvec, prefill a GEMM, and the
 * feed-forward block is gate and up, SwiGLU, down (section "Speed, and where
 * it goes").
 *
 * Layout of one PTQ1_0 block (28 bytes):
 *   bytes 0..25  trit bytes; weight 5i+n of the block is base-3 digit n of
 *                byte i (n = 0 most significant), digit d means weight d-1;
 *                byte 25 holds weights 125..127 in digits 0..2, digits 3..4
 *                are padding (written as 1, ignored when read);
 *   bytes 26..27 the block scale, IEEE binary16, little-endian.
 * A packed matrix [n][k] is row-major: row r is k/128 consecutive blocks.
 * Weight (r, c) = scale(r, c/128) * trit(r, c).
 *
 * Tiled layout (this library's device layout, not part of the format): the
 * same 28-byte blocks reordered so that each tile of 32 rows x 2 blocks
 * (256 weights of K) is 1792 contiguous bytes, K-slices outermost.  With
 * G = ceil(n/32) row bands, tile (g, t) -- rows 32g.., K-slice t -- starts at
 * byte (t*G + g) * 1792 and holds block j = 2t + b of row r = 32g + i at
 * byte (2i + b) * 28 of the tile; places past the matrix (r >= n or
 * j >= k/128) hold zero bytes.  The
 * matvec, gate/up, GEMM and feed-forward calls read weights in this layout
 * (ptq1_tile makes it from a packed matrix, once, at load time); pack
 * and dequant use the packed layout.
 *
 * Beyond PTQ1_0 with fp32 activations, two more numerics of the same layer:
 * the PQ2_0 format (pq2_*: two bits per weight, described before pq2_packed_bytes)
 * and 8-bit activations (ptq1_matvec_w2a8).
 *
 * Rotation R of a row x of width k (k a multiple of 1024): every 1024-wide
 * chunk c becomes (1/32) H (s * c), with H the natural-order Sylvester
 * Hadamard matrix and s the 1024 signs (one vector for every chunk).
 * R is orthogonal; the inverse applied to embedding rows is s * ((1/32) H c).
 *
 * Conventions for every call:
 *   - pointers are device pointers (hipMalloc'd or equivalent) unless stated;
 *     all memory is owned by the caller; weights are only read;
 *   - work is enqueued on `stream` (0 = the null stream) and the call returns
 *     without waiting; a fault during execution surfaces at the caller's
 *     stream synchronisation, as usual in HIP;
 *   - on any status other than PTQ1_OK nothing has been enqueued (except
 *     PTQ1_ERR_HIP, which reports a failed launch);
 *   - ptq1_last_error() then names the refused argument (thread-local);
 *   - the library allocates no memory; calls that need scratch take a
 *     caller-owned workspace `ws` of at least the size the matching
 *     *_workspace_bytes() returns, 256-byte aligned, with any contents: it
 *     is scratch, written before it is read within each call, so one
 *     workspace may serve calls of any shape and entry point.  Calls that
 *     share a workspace must be ordered on one stream; two calls in flight
 *     at once must not share one.  The decode calls (matvec, gate_up,
 *     ffn_block with m = 1) take at most 2^20 output rows per matrix and
 *     tiled matrices below 2 GiB;
 *   - `float *` buffers must be 16-byte aligned, weights 16-byte aligned;
 *   - sizes are int64_t; products are checked for overflow.
 */
#ifndef PTQ1_H
#define PTQ1_H

#include <stddef.h>
#include <stdint.h>
#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

#define PTQ1_BLOCK_WEIGHTS 128
#define PTQ1_TRIT_BYTES 26
#define PTQ1_BLOCK_BYTES 28
#define PTQ1_HADAMARD 1024
#define PTQ1_TILE_ROWS 32
#define PTQ1_TILE_BLOCKS 2

typedef enum ptq1_status {
    PTQ1_OK = 0,
    PTQ1_ERR_NULL = 1,        /* a required pointer is NULL                        */
    PTQ1_ERR_SHAPE = 2,       /* a size is negative or not a multiple it must be    */
    PTQ1_ERR_ALIGN = 3,       /* a pointer is not aligned as stated above          */
    PTQ1_ERR_OVERFLOW = 4,    /* a derived byte count or index overflows int64     */
    PTQ1_ERR_UNSUPPORTED = 5, /* a well-formed request this library does not run   */
    PTQ1_ERR_WORKSPACE = 6,   /* ws is NULL or smaller than *_workspace_bytes()    */
    PTQ1_ERR_ALIAS = 7,       /* an output overlaps an input it must not overlap   */
    PTQ1_ERR_HIP = 8          /* a HIP runtime call or kernel launch failed        */
} ptq1_status;

/* Human-readable name of a status.  Never NULL. */
const char *ptq1_status_string(ptq1_status s);

/* Message of the last non-OK status returned on this thread ("" if none).
 * Never NULL; valid until the next call on this thread. */
const char *ptq1_last_error(void);

/* Copies the compiled geometry {weights per block, trit bytes, block bytes,
 * Hadamard width, tile rows, tile blocks} into out[0..n) (n <= 6).
 * PTQ1_ERR_NULL / PTQ1_ERR_SHAPE. */
ptq1_status ptq1_geometry(int32_t *out, int32_t n);

/* Bytes of a packed [n][k] matrix: n * (k/128) * 28, or -1 if n < 0, k < 0,
 * k % 128 != 0 or the product overflows. */
int64_t ptq1_packed_bytes(int64_t n, int64_t k);

/* Codec encode ("What Bonsai is": five trits per byte in base 3, one 16-bit
 * scale per 128 weights).
 *   trits      int8 [n][k], values in {-1, 0, +1} (other values are clamped
 *              to the nearest of these);
 *   scales_f16 binary16 bit patterns [n][k/128], copied verbatim;
 *   blocks     output, ptq1_packed_bytes(n, k) bytes.
 * Each byte carries the code v = sum_n (t_n + 1) 3^(4-n) as the smallest
 * byte b with floor(243 b / 256) = v, i.e. b = ceil(256 v / 243).
 * Errors: NULL, SHAPE (k % 128), ALIGN (blocks), OVERFLOW. */
ptq1_status ptq1_pack(const int8_t *trits, const uint16_t *scales_f16, int64_t n, int64_t k,
                      uint8_t *blocks, hipStream_t stream);

/* Bytes of the tiled layout of an [n][k] matrix: ceil(n/32)*32 rows times
 * ceil(k/256)*2 blocks of 28 bytes (equal to ptq1_packed_bytes when n % 32
 * == 0 and k % 256 == 0), or -1 on a bad shape or overflow. */
int64_t ptq1_tiled_bytes(int64_t n, int64_t k);

/* Reorders a packed [n][k] matrix into the tiled layout described above
 * (bytes of every block copied unchanged, padding written as zeros).
 *   blocks  packed, ptq1_packed_bytes(n, k) bytes;
 *   tiled   output, ptq1_tiled_bytes(n, k) bytes, must not overlap blocks.
 * Errors: NULL, SHAPE (k % 128), ALIGN, ALIAS, OVERFLOW. */
ptq1_status ptq1_tile(const uint8_t *blocks, int64_t n, int64_t k, uint8_t *tiled, hipStream_t stream);

/* Codec decode ("What Ferrox does with it": digit n of u = b/256 read on the
 * float pipeline).  w [n][k] fp32 = binary16 scale * (digit - 1), exact.
 * Errors: NULL, SHAPE, ALIGN, OVERFLOW. */
ptq1_status ptq1_dequant(const uint8_t *blocks, int64_t n, int64_t k, float *w, hipStream_t stream);

/* Rotation of activations ("What Bonsai is": the rotation applied to the
 * activations before every matmul of a folded weight).
 *   x, y  fp32 [m][k], k % 1024 == 0; y may equal x (in place), otherwise
 *         they must not overlap;
 *   signs1024  fp32 [1024], +-1.0 (other values are used as given and break
 *         orthogonality).
 * Errors: NULL, SHAPE (k % 1024), ALIGN, ALIAS (partial overlap), OVERFLOW. */
ptq1_status hadamard_rotate(const float *x, float *y, int64_t m, int64_t k, const float *signs1024,
                            hipStream_t stream);

/* Embedding lookup with the rotation undone ("What Bonsai is": undo the
 * rotation on the embedding table after each lookup).
 *   table  fp32 [n_table][d] row-major, rows stored rotated, d % 1024 == 0;
 *   ids    int32 [n_rows] device array of row indices, or NULL for rows
 *          0..n_rows-1; an id outside [0, n_table) yields a row of NaN;
 *   out    fp32 [n_rows][d]: out[i] = s * ((1/32) H table[ids[i]]) per chunk.
 * Errors: NULL, SHAPE (d % 1024, n_rows > n_table without ids), ALIGN,
 * ALIAS, OVERFLOW. */
ptq1_status hadamard_unrotate_rows(const float *table, int64_t n_table, int64_t d,
                                   const int32_t *ids, int64_t n_rows, const float *signs1024,
                                   float *out, hipStream_t stream);

/* Batch-1 decode matvec ("What Ferrox does with it": the decode matvec reads
 * every block once).
 *   y[r] = (residual ? residual[r] : 0) + sum_c W[r][c] * xr[c],
 *   xr = R x when signs1024 != NULL (k % 1024 == 0), else x as given.
 *   tiled   [n][k] in the tiled layout; x fp32 [k]; residual fp32 [n] or
 *   NULL; y fp32 [n] (y may equal residual, must not overlap x or tiled).
 * Trits are decoded through a per-slice table of byte-position x byte-value
 * partial dot products built from xr in 32-bit fixed point: each 256-wide
 * K-slice of xr is scaled by its own power of two so that max|xr| lies in
 * [2^22, 2^23) and rounded to integers once (an error of at most 2^-24 of the
 * slice's max|xr| per element); table entries and each block's sum are exact
 * int32, the block sum is scaled by its fp16 scale in fp32 and the rest is
 * fp32.  A NaN or an infinity in xr makes every output a NaN.  Two launches
 * (split-K partials per slice, then their sum in slice order).
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE. */
size_t ptq1_matvec_workspace_bytes(int64_t n, int64_t k);
ptq1_status ptq1_matvec(const uint8_t *tiled, int64_t n, int64_t k, const float *x,
                        const float *signs1024, const float *residual, float *y, void *ws,
                        size_t ws_bytes, hipStream_t stream);

/* The same matvec with every trit peeled on the float pipeline as the page
 * describes ("What Ferrox does with it": eight lanes share one 128-weight
 * block, each lane owns whole bytes, and a trit is floor(3^(n+1) u) -
 * 3 floor(3^n u), u = byte/256).  Same tiled matrix, results (to rounding
 * order and ptq1_matvec's fixed-point rounding of xr), workspace size and
 * errors as ptq1_matvec (its sums are fp32, so a NaN or an infinity
 * propagates as the float operations make it); kept as the page's own
 * decode, to be measured beside the table lookups. */
ptq1_status ptq1_matvec_float_peel(const uint8_t *tiled, int64_t n, int64_t k, const float *x,
                                   const float *signs1024, const float *residual, float *y, void *ws,
                                   size_t ws_bytes, hipStream_t stream);

/* Gate and up projections of one token in one pass over a shared rotated
 * input ("Speed, and where it goes": paired projections fused into one GPU
 * submission).
 *   w_gate, w_up  tiled [f][d]; x fp32 [d]; g, u fp32 [f]:
 *   g = W_gate R x, u = W_up R x (R skipped when signs1024 == NULL), with
 * the table lookups and numerics of ptq1_matvec.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE. */
size_t ptq1_gate_up_workspace_bytes(int64_t f, int64_t d);
ptq1_status ptq1_gate_up(const uint8_t *w_gate, const uint8_t *w_up, int64_t f, int64_t d,
                         const float *x, const float *signs1024, float *g, float *u, void *ws,
                         size_t ws_bytes, hipStream_t stream);

/* SwiGLU ("Speed, and where it goes": gate, SwiGLU, down):
 * h[i] = g[i] / (1 + exp(-g[i])) * u[i], fp32 [len].  h may equal g or u.
 * Errors: NULL, SHAPE (len < 0), ALIGN. */
ptq1_status ptq1_swiglu(const float *g, const float *u, float *h, int64_t len, hipStream_t stream);

/* Multi-token prefill GEMM ("What Ferrox does with it": a GEMM for prefill).
 *   Y [m][n] fp32 = bf16(R X) . W^T: X fp32 [m][k] is rotated (when
 *   signs1024 != NULL) and rounded to bf16 (nearest even); trits enter bf16
 *   MFMA exactly; each 128-weight block's partial sum is scaled by its fp16
 *   scale in fp32; accumulation is fp32.
 *   tiled [n][k] in the tiled layout; 1 <= m <= 65536; k % 128 == 0
 *   (k % 1024 == 0 with signs).
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED (m). */
size_t ptq1_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k);
ptq1_status ptq1_gemm(const uint8_t *tiled, int64_t n, int64_t k, const float *x, int64_t m,
                      const float *signs1024, float *y, void *ws, size_t ws_bytes,
                      hipStream_t stream);

/* One feed-forward block on m tokens ("Speed, and where it goes": the whole
 * block -- rotation, gate, SwiGLU, down -- enqueued as one sequence; "Why I
 * Am Building Another Inference Engine", Level 4: the layer's norm, with its
 * own weight, ahead of the rotation):
 *   a     = (mean(x^2) + rms_eps)^(-1/2) per token if rms_eps > 0, else 1
 *   xn    = a * rms_gain * x                      (rms_gain fp32 [d], NULL: 1)
 *   g, u  = W_gate R xn, W_up R xn                (W_gate, W_up tiled [f][d])
 *   h     = silu(g) * u
 *   x_out = x + W_down R h                        (W_down tiled [d][f])
 * m == 1 runs the table-lookup matvec path (numerics of ptq1_matvec), m >= 2
 * the bf16-MFMA GEMM path.
 * d % 1024 == 0, f % 1024 == 0; x_out may equal x; rms_gain, if given, is
 * 16-byte aligned and overlaps neither x_out nor ws.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED. */
size_t ptq1_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f);
ptq1_status ptq1_ffn_block(const float *x, float *x_out, int64_t m, int64_t d, int64_t f,
                           const uint8_t *w_gate, const uint8_t *w_up, const uint8_t *w_down,
                           const float *signs1024, float rms_eps, const float *rms_gain, void *ws,
                           size_t ws_bytes, hipStream_t stream);

/* Where ptq1_ffn_block leaves the block's intermediate activations in its
 * workspace, so a caller can inspect each stage after the call ("A 27B model
 * in 5.5 GB: Bonsai ternary on Ferrox, locally", "Accuracy: measured, not
 * eyeballed": every execution path is compared stage by stage):
 *   offsets[0], offsets[1]  byte offsets of g and u, fp32 [m][f] (the gate
 *                           and up projections of the normalised input), for
 *                           m >= 2; -1 for m == 1;
 *   offsets[2]              byte offset of h = silu(g) * u, fp32 [f], for
 *                           m == 1; -1 for m >= 2 (there h is only formed in
 *                           bf16 inside the down projection's input).
 * They hold the values of the last call with this (m, d, f) until the
 * workspace is reused.  Errors: NULL, SHAPE (m < 1, d or f not a multiple of
 * 1024), UNSUPPORTED (m). */
ptq1_status ptq1_ffn_workspace_offsets(int64_t m, int64_t d, int64_t f, int64_t *offsets);

/* ptq1_ffn_block for callers that cannot allocate memory or pass a
 * workspace (code under HIP graph capture, tight serving loops, harnesses
 * that forbid allocation): the same arguments, kernels, results and errors,
 * without ws / ws_bytes.  Its scratch is a buffer of 8 MiB (8388608 bytes)
 * that the library holds statically on every GPU it runs on, until the
 * process ends; a call whose ptq1_ffn_workspace_bytes(m, d, f) exceeds it is
 * refused with PTQ1_ERR_UNSUPPORTED before anything is enqueued (m = 1 up to
 * d = 8192, f = 28672; m <= 8 at d = 5120, f = 17408).  Nothing in it needs
 * to start at zero: every call writes the scratch it reads.  All calls on
 * one GPU share that buffer, so two calls that may overlap on one GPU (on
 * different streams, or from several host threads without ordering) race:
 * order them on one stream, or use ptq1_ffn_block with a workspace each.
 * The stage offsets of ptq1_ffn_workspace_offsets hold for this buffer too,
 * but it is not reachable from outside the library. */
ptq1_status ptq1_ffn_block_noalloc(const float *x, float *x_out, int64_t m, int64_t d, int64_t f,
                                   const uint8_t *w_gate, const uint8_t *w_up, const uint8_t *w_down,
                                   const float *signs1024, float rms_eps, const float *rms_gain,
                                   hipStream_t stream);

/* ---- PQ2_0: the two-bit ternary format ("Why I Am Building Another
 * Inference Engine", Level 2: two bits per weight and a 16-bit scale for every
 * 128 weights, 2.125 bits per weight).  A block is 32 code bytes, weight
 * 4i + f in bits 2f..2f+1 of byte i (code q is the trit q - 1; code 3, never
 * written, reads as 0), then the binary16 scale, little-endian: 34 bytes.
 * The device layout for the matvec is tiled like PTQ1_0's (32 rows x 2
 * blocks per tile, tiles K-slice-major) with each tile holding its 64 code
 * records of 32 bytes first and then its 64 scales: 2176 bytes per tile. */

/* Bytes of a packed [n][k] PQ2_0 matrix: n * (k/128) * 34, or -1 if n < 0,
 * k < 0, k % 128 != 0 or the product overflows. */
int64_t pq2_packed_bytes(int64_t n, int64_t k);

/* Encode.  trits int8 [n][k] ({-1, 0, +1}; others clamped), scales_f16
 * binary16 bit patterns [n][k/128] (copied verbatim), blocks output of
 * pq2_packed_bytes(n, k) bytes, 16-byte aligned.
 * Errors: NULL, SHAPE (k % 128), ALIGN, ALIAS, OVERFLOW. */
ptq1_status pq2_pack(const int8_t *trits, const uint16_t *scales_f16, int64_t n, int64_t k, uint8_t *blocks,
                     hipStream_t stream);

/* Decode: w [n][k] fp32 = binary16 scale * trit, exact.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW. */
ptq1_status pq2_dequant(const uint8_t *blocks, int64_t n, int64_t k, float *w, hipStream_t stream);

/* Bytes of the PQ2_0 tiled layout: ceil(n/32) * ceil(k/256) * 2176, or -1 on
 * a bad shape or overflow. */
int64_t pq2_tiled_bytes(int64_t n, int64_t k);

/* Packed -> tiled reorder (code bytes and scales copied unchanged, padding
 * written as zeros).  Both pointers 16-byte aligned, not overlapping.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW. */
ptq1_status pq2_tile(const uint8_t *blocks, int64_t n, int64_t k, uint8_t *tiled, hipStream_t stream);

/* Batch-1 decode matvec over a PQ2_0 tiled matrix, with the arguments,
 * results, workspace rule and errors of ptq1_matvec:
 *   y[r] = (residual ? residual[r] : 0) + sum_c W[r][c] * xr[c],
 *   xr = R x when signs1024 != NULL (k % 1024 == 0), else x as given.
 * Codes are decoded through a per-slice table of (code byte, byte value)
 * partial dot products over xr in the same 32-bit fixed point as
 * ptq1_matvec (exact int32 block sums; a NaN or infinity in xr makes every
 * output a NaN); split-K partials over 256-wide slices, then their sum in
 * slice order.  The tiled matrix must be below 2 GiB (UNSUPPORTED
 * otherwise). */
size_t pq2_matvec_workspace_bytes(int64_t n, int64_t k);
ptq1_status pq2_matvec(const uint8_t *tiled, int64_t n, int64_t k, const float *x, const float *signs1024,
                       const float *residual, float *y, void *ws, size_t ws_bytes, hipStream_t stream);

/* Multi-token prefill GEMM over a PQ2_0 tiled matrix, with the arguments,
 * numerics, limits and errors of ptq1_gemm: Y [m][n] fp32 = bf16(R X) . W^T,
 * codes entering bf16 MFMA exactly as -1 / 0 / +1 and each block's partial
 * sum scaled by its fp16 scale in fp32. */
size_t pq2_gemm_workspace_bytes(int64_t m, int64_t n, int64_t k);
ptq1_status pq2_gemm(const uint8_t *tiled, int64_t n, int64_t k, const float *x, int64_t m, const float *signs1024,
                     float *y, void *ws, size_t ws_bytes, hipStream_t stream);

/* The feed-forward block of ptq1_ffn_block over PQ2_0 tiled matrices: the
 * same arguments, numerics (m = 1: fixed-point table lookups as in
 * pq2_matvec; m >= 2: bf16 MFMA),
 * workspace rule and errors; every matrix must be below 2 GiB at m = 1. */
size_t pq2_ffn_workspace_bytes(int64_t m, int64_t d, int64_t f);
ptq1_status pq2_ffn_block(const float *x, float *x_out, int64_t m, int64_t d, int64_t f, const uint8_t *w_gate,
                          const uint8_t *w_up, const uint8_t *w_down, const float *signs1024, float rms_eps,
                          const float *rms_gain, void *ws, size_t ws_bytes, hipStream_t stream);

/* The same stage offsets for pq2_ffn_block's workspace. */
ptq1_status pq2_ffn_workspace_offsets(int64_t m, int64_t d, int64_t f, int64_t *offsets);

/* Batch-1 decode matvec with 8-bit activations (W2A8: "Why I Am Building
 * Another Inference Engine", Level 5, the numerics of integer kernels; Level
 * 4, where a BitNet layer rounds its activations to int8 ahead of its ternary
 * matmuls):
 *   c = float(127 / max|x|) (0 when x is all zeros), q[i] = rint(x[i] * c) in
 *   fp32 (integers in [-127, 127], ties to even), step = max|x| / 127;
 *   y[r] = (residual ? residual[r] : 0) + step * sum_b s_rb * sum_{i in b} t_ri q_i.
 * x is used as given (rotate it first with hadamard_rotate for a folded
 * layer).  The per-block integer sums are exact; the block scales, the sum
 * over blocks and the step are fp32.  Same tiled matrix, residual and
 * aliasing rules as ptq1_matvec; k % 128 == 0, k > 0.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED. */
size_t ptq1_matvec_w2a8_workspace_bytes(int64_t n, int64_t k);
ptq1_status ptq1_matvec_w2a8(const uint8_t *tiled, int64_t n, int64_t k, const float *x, const float *residual,
                             float *y, void *ws, size_t ws_bytes, hipStream_t stream);

/* Prefill GEMM with 8-bit activations: each row of X [m][k] quantised as in
 * ptq1_matvec_w2a8 (its own absmax and step), the int8 rows multiplied with
 * the trits as int8 on the matrix cores (every 128-weight block summed
 * exactly in int32), each block sum scaled by its fp16 scale in fp32, and
 * row i of Y multiplied by its step:
 *   Y[i][r] = step_i * sum_b s_rb * sum_{c in b} t_rc q_ic.
 * X is used as given (no rotation).  Limits and errors as ptq1_gemm. */
size_t ptq1_gemm_w2a8_workspace_bytes(int64_t m, int64_t n, int64_t k);
ptq1_status ptq1_gemm_w2a8(const uint8_t *tiled, int64_t n, int64_t k, const float *x, int64_t m, float *y, void *ws,
                           size_t ws_bytes, hipStream_t stream);

/* ---- Attention: the other half of a layer ("Why I Am Building Another
 * Inference Engine", Level 4: a layer's projections, rotary positions,
 * attention and output projection; "Speed, and where it goes": the key-value
 * cache is what long contexts cost).  The calls below take the fp32 rows that
 * the projections above produce (or 16-bit rows), keep keys and values in a
 * paged cache, and return rows for the output projection.
 *
 * The cache is a set of pages that the caller owns; a page holds page_size
 * consecutive tokens of one sequence for every key-value head:
 *   k_pages  [n_pages][n_kv_heads][page_size][head_dim]
 *   v_pages  [n_pages][n_kv_heads][head_dim][page_size]   (dimension-major)
 * in binary16, bfloat16 or int8.  An int8 cache has one fp32 step for every
 * token and head, k_steps and v_steps [n_pages][n_kv_heads][page_size]: the
 * value is step * code (step = max|x| / 127 over the head's row, code =
 * rint(x * float(127 / max|x|)), ties to even, as in ptq1_matvec_w2a8; a row
 * below 2^-119 in magnitude is stored as zeros; a row that holds a NaN or an
 * infinity reads back as NaN; steps that a program writes itself are not
 * negative and below 2^122, or NaN).  V is dimension-major because the attention
 * over one token multiplies whole runs of tokens of one dimension: both
 * operands of both products are then 16 contiguous bytes per lane.  A token's
 * slot is page * page_size + its place in the page.  Cache memory needs no
 * initial contents: what no token was written to is never used. */
typedef enum ptq1_dtype {
    PTQ1_F32 = 0,  /* IEEE binary32 */
    PTQ1_F16 = 1,  /* IEEE binary16 */
    PTQ1_BF16 = 2, /* bfloat16 */
    PTQ1_I8 = 3    /* int8 codes with fp32 steps (cache only) */
} ptq1_dtype;

typedef struct ptq1_kv_cache {
    void *k_pages;       /* device pointers, 16-byte aligned */
    void *v_pages;
    float *k_steps;      /* PTQ1_I8 only, else NULL */
    float *v_steps;
    int64_t n_pages;     /* 1 .. 2^31 - 1 */
    int32_t page_size;   /* 16, 32, 64, 128 or 256 tokens */
    int32_t n_kv_heads;  /* 1 .. 1024 */
    int32_t head_dim;    /* 64, 128 or 256 */
    int32_t dtype;       /* PTQ1_F16, PTQ1_BF16 or PTQ1_I8 */
} ptq1_kv_cache;

/* Writes n_tokens fresh tokens into the cache, with rotary positions on
 * their keys and queries, in one launch.
 *   q, k, v    rows [n_tokens] of n_q_heads, n_kv_heads and n_kv_heads heads
 *              of head_dim elements of src_dtype (F32, F16 or BF16; heads
 *              contiguous, rows q_stride, k_stride, v_stride elements apart,
 *              so they may be parts of one stacked projection's rows).  16-byte
 *              aligned, strides multiples of 16 bytes, at least a row (or
 *              anything when n_tokens <= 1).  n_q_heads = 0: no queries
 *              (q and q_out unused).
 *   cos_sin    fp32 [n_positions][rot_dim]: rot_dim / 2 cosines, then
 *              rot_dim / 2 sines; rot_dim a multiple of 8, <= head_dim; 0 (and
 *              cos_sin NULL): no rotation.  Elements i and i + rot_dim / 2 of
 *              a head turn together: (a cos - b sin, b cos + a sin), each
 *              product and sum rounded to fp32; elements from rot_dim on
 *              stay.
 *   positions  int32 [n_tokens], the row of cos_sin for each token (unused
 *              without rotation).  A position outside [0, n_positions) makes
 *              the elements that would turn NaN, the first rot_dim of the
 *              token's q_out and key (in an int8 cache its whole key).
 *   slots      int64 [n_tokens].  A slot outside [0, n_pages * page_size)
 *              writes nothing to the cache (padding: -1); q_out is written
 *              all the same.  The slots in the cache must differ: of two
 *              tokens with one slot, either may end up there, or parts of
 *              both.
 *   q_out      [n_tokens][n_q_heads][head_dim] of q_dtype (F32, F16, BF16),
 *              16-byte aligned, overlapping neither inputs nor the cache.
 * Values are rounded once, to nearest even, to the cache's and q_out's types.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, UNSUPPORTED (types, head_dim,
 * page_size, more than 2^24 tokens or 2^25 rows of heads). */
ptq1_status ptq1_kv_write(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                          int64_t v_stride, int32_t src_dtype, int64_t n_tokens, int32_t n_q_heads,
                          const int32_t *positions, const float *cos_sin, int64_t n_positions, int32_t rot_dim,
                          const int64_t *slots, void *q_out, int32_t q_dtype, const ptq1_kv_cache *cache,
                          hipStream_t stream);

/* ptq1_kv_write with norms of the query and key heads ahead of the rotation
 * (layers that norm each head of q and k):
 *   x' = a * gain * x,  a = (mean(x^2) + eps)^(-1/2) over the head's
 *   head_dim elements, in fp32;
 * values go into the cache as they are.
 *   q_gain, k_gain  fp32 [head_dim], 16-byte aligned, one for all heads; NULL:
 *        ones.
 *   eps  2^-100 to 2^100.
 * Everything else as in ptq1_kv_write.  Finite rows of any magnitude are
 * normed, also where their squares leave fp32's range.  A NaN in a head makes
 * all of it NaN, an infinity its own element NaN and the others, before the
 * rotation, zero.
 * Errors: as ptq1_kv_write; SHAPE (eps). */
ptq1_status ptq1_kv_write_norm(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                               int64_t v_stride, int32_t src_dtype, int64_t n_tokens, int32_t n_q_heads,
                               const float *q_gain, const float *k_gain, float eps, const int32_t *positions,
                               const float *cos_sin, int64_t n_positions, int32_t rot_dim, const int64_t *slots,
                               void *q_out, int32_t q_dtype, const ptq1_kv_cache *cache, hipStream_t stream);

/* Reads whole sequences back, packed: rows cu_seqlens[b] .. cu_seqlens[b + 1]
 * of k_out and v_out [n_rows][n_kv_heads][head_dim] (out_dtype F32, F16 or
 * BF16) get the first cu_seqlens[b + 1] - cu_seqlens[b] tokens of sequence b,
 * whose pages are block_table[b][0..max_pages) (int32, device).  cu_seqlens
 * int32 [batch + 1], device, not negative, not decreasing.  Rows that belong to no sequence
 * are left as they were, and no row from n_rows on is written.  A token whose
 * page is outside [0, n_pages), or past max_pages, reads as NaN.  An int8
 * value is step * code, rounded once to out_dtype.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, UNSUPPORTED (types, head_dim,
 * page_size, more than 2^24 - 1 tiles of 64 tokens of a head, n_rows >
 * 2^31 - 1). */
ptq1_status ptq1_kv_read(const ptq1_kv_cache *cache, const int32_t *block_table, int64_t max_pages,
                         const int32_t *cu_seqlens, int64_t batch, int64_t n_rows, void *k_out, void *v_out,
                         int32_t out_dtype, hipStream_t stream);

/* Attention of one new token of each of `batch` sequences over the paged
 * cache:
 *   out[b][h] = sum_j p_j V[j],  p = softmax over j < seq_lens[b] of
 *               scale * (q[b][h] . K[j]),
 * query head h reading key-value head h / (n_q_heads / n_kv_heads).
 *   q, out     [batch][n_q_heads][head_dim], q_dtype F32, the cache's own
 *              16-bit type, or any of F32, F16, BF16 over an int8 cache; out
 *              has q's type and must not overlap q.
 *   block_table int32 [batch][max_pages], seq_lens int32 [batch] (device):
 *              sequence b's tokens are 0 .. seq_lens[b] - 1, the new token's own
 *              key among them if it is to be seen.  Length 0 gives zeros.  A
 *              length outside [0, max_len], or a page outside [0, n_pages)
 *              among those the length covers, makes the sequence's rows NaN.
 *   max_len    a bound on the lengths that the caller knows (at most
 *              max_pages * page_size); the work is laid out for it.
 *   scale      positive, 2^126 at most.
 * The products run on the matrix cores.  Over 16-bit caches K and V enter
 * exactly, fp32 queries as three 16-bit terms (over bf16 down to 2^-133, over
 * fp16 down to 2^-38 of the head's largest magnitude) and weights as two or three
 * (bf16 queries: two, 16 bits of a weight; fp16: down to 2^-38 of the row's
 * largest).  Over int8 caches the codes enter exactly; the queries are fixed-point
 * numbers, multiples of 2^-29 (fp32 queries) or 2^-21 of a power of two not
 * above the head's largest magnitude; weight times step enters as three fp16
 * terms (16-bit queries: two), down to 2^-38 of the largest or to 2^-149.  Sums,
 * maxima and accumulators are fp32; values up to fp32's largest, or steps up to
 * the bound above, do not overflow on the way to a row that is in range.  A NaN
 * or an infinity in a query or in a key or value that is read makes the entries
 * of out that it enters NaN or infinite; an infinite key that meets a 16-bit
 * query at a score of -infinity has weight zero instead, as if it were not there
 * (fp32 queries: that or NaN).  Long sequences are cut into pieces that run side
 * by side and are joined by a second launch, in a fixed order.
 * Errors: NULL, SHAPE (n_q_heads not a multiple of n_kv_heads, max_len, scale),
 * ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED (types, head_dim, page_size,
 * batch > 65535, more than 2^24 - 2^14 groups of 16 query heads of a kv head in
 * all sequences together, max_len > 2^22). */
size_t ptq1_attn_decode_workspace_bytes(int64_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                        int64_t max_len);
ptq1_status ptq1_attn_decode(const void *q, int32_t q_dtype, int64_t batch, int32_t n_q_heads,
                             const ptq1_kv_cache *cache, const int32_t *block_table, int64_t max_pages,
                             const int32_t *seq_lens, int64_t max_len, float scale, void *out, void *ws,
                             size_t ws_bytes, hipStream_t stream);

/* ptq1_attn_decode for layers with a sliding window: of a sequence's n =
 * seq_lens[b] tokens the last `window` (the new one among them) and the first
 * `sinks` are seen,
 *   j >= n - window  or  j < sinks.
 * Pages that hold no such token are not read, and their entries of block_table
 * may be anything: a program may give them back.  Everything else as in
 * ptq1_attn_decode (a page outside [0, n_pages) matters among those that hold a
 * token that is seen); the work is laid out for the tokens that are read.
 *   window  1 or more (more than max_len: every token is seen); sinks 0 or more.
 * Errors: as ptq1_attn_decode; SHAPE (window, sinks). */
size_t ptq1_attn_decode_window_workspace_bytes(int64_t batch, int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim,
                                               int64_t max_len, int64_t window, int64_t sinks);
ptq1_status ptq1_attn_decode_window(const void *q, int32_t q_dtype, int64_t batch, int32_t n_q_heads,
                                    const ptq1_kv_cache *cache, const int32_t *block_table, int64_t max_pages,
                                    const int32_t *seq_lens, int64_t max_len, int64_t window, int64_t sinks, float scale,
                                    void *out, void *ws, size_t ws_bytes, hipStream_t stream);

/* Attention of the last tokens of every sequence over the paged cache that
 * holds them already (ptq1_kv_write first): proposed tokens to be verified,
 * prompts that arrive in pieces, and batches of both.  Sequence b's queries are
 * rows cu_q[b] .. cu_q[b + 1] of q; with m of them and n = seq_lens[b] tokens,
 * query i stands at position p = n - m + i and sees the tokens
 *   j <= p  with  window = 0  or  j > p - window  or  j < sinks
 * (window counts the query's own token; sinks: first tokens that stay visible).
 * A query at a negative position sees none and gets zeros.
 *   q    [n_q_rows][n_q_heads][head_dim] (heads contiguous, rows q_stride
 *        elements apart, 16-byte aligned, a multiple of 16 bytes), q_dtype the
 *        cache's own 16-bit type, F16 or BF16 over an int8 cache;
 *   out  [n_q_rows][n_q_heads][head_dim] contiguous, of q's type; must not
 *        overlap q.  Rows that belong to no sequence are left as they were.
 *   cu_q, seq_lens, block_table  int32, device: [batch + 1] (not negative, not
 *        decreasing), [batch], [batch][max_pages].
 *   max_q, max_len  bounds on the sequences' queries and tokens that the caller
 *        knows (max_len at most max_pages * page_size); the work is laid out for
 *        them.  A sequence that exceeds one, or whose length is negative, gets
 *        NaN rows, as does one whose rows lie outside [0, n_q_rows) (those
 *        inside).  A row that sees a token whose page is outside [0, n_pages) is
 *        NaN.
 *   scale  positive, 2^126 at most.
 * What a query does not see does not enter its row, whatever it holds, and pages
 * that hold nothing that a query of their sequence sees are not read: their
 * entries of block_table may be anything.
 * bf16 or fp16 matrix cores, fp32 scores, maxima, sums and accumulators.  K, V,
 * queries and int8 codes enter exactly.  Weights enter the second product in
 * the cache's 16-bit type, over int8 caches times their value's step in fp16:
 *   where max_q * n_q_heads / n_kv_heads is at most 32 (few rows, where K and V
 *        bound the call) as two terms, 16 (bf16) or 22 bits of a weight;
 *   elsewhere as one, 8 (bf16) or 11 bits, and over 16-bit caches it is the
 *        rounded weights that are summed, as in ptq1_attn_prompt.
 * fp16 terms end at 2^-32 of the row's largest weight, over int8 caches at 2^-27
 * of its largest weight times step.  Values up to the type's largest, and steps
 * up to what ptq1_kv_write makes, do not overflow on the way to a row that is in
 * range; over int8 caches log2(e) * scale * step has to be a normal number of
 * fp32, or the keys' scores lose bits.  A NaN or an infinity in a query, or in a
 * key or value that it sees, makes the entries of out that it enters NaN or
 * infinite; an infinite key at a score of -infinity has weight zero instead.
 * Where the tiles of query rows alone would not fill the GPU, the keys are cut
 * into pieces that run side by side and are joined by a second launch, in a
 * fixed order, by the lengths on the device.
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED (types,
 * head_dim, page_size, max_len > 2^22, more than 2^31 - 1025 rows of one kv head
 * or 2^23 tiles of 128 query rows). */
size_t ptq1_attn_chunk_workspace_bytes(int64_t batch, int64_t n_q_rows, int64_t max_q, int32_t n_q_heads,
                                       int32_t n_kv_heads, int32_t head_dim, int64_t max_len, int64_t window,
                                       int64_t sinks);
ptq1_status ptq1_attn_chunk(const void *q, int64_t q_stride, int32_t q_dtype, const int32_t *cu_q, int64_t batch,
                            int64_t n_q_rows, int64_t max_q, int32_t n_q_heads, const ptq1_kv_cache *cache,
                            const int32_t *block_table, int64_t max_pages, const int32_t *seq_lens, int64_t max_len,
                            int64_t window, int64_t sinks, float scale, void *out, void *ws, size_t ws_bytes,
                            hipStream_t stream);

/* Attention over whole prompts, packed without padding: sequence b's queries
 * are rows cu_q[b] .. cu_q[b + 1] of q [n_q_rows][n_q_heads][head_dim], its
 * keys and values rows cu_k[b] .. cu_k[b + 1] of k and v
 * [n_k_rows][n_kv_heads][head_dim] (heads contiguous, rows q_stride,
 * k_stride, v_stride elements apart; 16-byte aligned, strides multiples of 16
 * bytes), all of dtype F16 or BF16; cu_q, cu_k int32 [batch + 1], device, not
 * decreasing.
 *   out  [n_q_rows][n_q_heads][head_dim] contiguous, of dtype; must overlap
 *        no input.  Rows that belong to no sequence are left as they were.
 *   causal != 0: query i of n_q sees the keys j <= i + n_k - n_q (the last
 *        query sees the last key, as when the first n_k - n_q keys come from
 *        a cache: ptq1_kv_read); else every key.  A query that sees no key
 *        gets zeros.  Keys and values that a query does not see do not enter
 *        its row, whatever they hold.
 *   max_q, max_k  bounds on the sequences' query and key counts that the
 *        caller knows; the work is laid out for them.  A sequence that
 *        exceeds one gets NaN rows, as does one whose rows lie outside
 *        [0, n_q_rows) or [0, n_k_rows) (those inside q's range).
 *   scale  positive, 2^126 at most.
 * bf16 or fp16 matrix cores, fp32 scores, maxima, sums and accumulators; the
 * weights enter the second product rounded to dtype (fp16: to 11 bits, down to
 * 2^-32 of the row's largest), and their sum, in fp32, is that of the rounded ones.
 * Where the query rows alone would not fill the GPU, the keys are cut into
 * chunks that run side by side and are joined by a second launch, in a fixed
 * order; the workspace (for max_k as given, or n_k_rows if that is less) holds
 * their parts (the size covers every n_k_rows; a call may need less).
 * Errors: NULL, SHAPE, ALIGN, ALIAS, OVERFLOW, WORKSPACE, UNSUPPORTED (types,
 * head_dim, more than 2^31 - 1025 rows of one kv head or 2^23 tiles of 128
 * query rows, k_stride or v_stride above 2^24). */
size_t ptq1_attn_prompt_workspace_bytes(int64_t batch, int64_t n_q_rows, int64_t max_k, int32_t n_q_heads,
                                        int32_t n_kv_heads, int32_t head_dim);
ptq1_status ptq1_attn_prompt(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                             int64_t v_stride, int32_t dtype, const int32_t *cu_q, const int32_t *cu_k,
                             int64_t batch, int64_t n_q_rows, int64_t n_k_rows, int64_t max_q, int64_t max_k,
                             int32_t n_q_heads, int32_t n_kv_heads, int32_t head_dim, int32_t causal, float scale,
                             void *out, void *ws, size_t ws_bytes, hipStream_t stream);

/* Profiling: attaches start[i] / stop[i] to the dispatch of the i-th of the
 * next `count` launches of one kernel family (hipExtLaunchKernel: they take
 * the kernel's own start and end times on its stream), so a caller can time
 * a kernel inside a composite call (ptq1_ffn_block) with events.  Families: "lut_matvec_2" (the
 * table-lookup matvec over two matrices: gate and up), "lut_matvec_1" (over
 * one matrix: ptq1_matvec, ptq1_matvec_w2a8, the down projection), "gemm" (the MFMA GEMM),
 * "pq2_matvec" (the PQ2_0 table-lookup matvec of pq2_matvec), "peel_matvec"
 * (the float-peel matvec of ptq1_matvec_float_peel); pq2_gemm's kernel
 * counts as "gemm".
 * Events are created and owned by the caller; both arrays must stay valid
 * until `count` launches have happened or the family is re-armed.  count =
 * 0 disarms.  Process-wide; not meant for concurrent use by several
 * threads.  Errors: NULL, SHAPE (count < 0), UNSUPPORTED (unknown name). */
ptq1_status ptq1_profile_arm(const char *kernel, hipEvent_t *start, hipEvent_t *stop, int32_t count);

/* Launches of `kernel` bracketed since it was last armed; -1 for an unknown
 * name. */
int32_t ptq1_profile_count(const char *kernel);

#ifdef __cplusplus
}
#endif

#endif /* PTQ1_H */

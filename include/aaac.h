/*
 * aaac.h -- C ABI of the MI355X (gfx950) activation-aware dual-codebook 4-bit weight quantizer.
 *
 * Method: the gist.science summary page "기술 요약: AAAC (활성화 인식 적응형 코드북)"
 * (arXiv 2605.08692), cited as "AAAC summary" with its section number. Each weight matrix gets two
 * learned scalar tables T0, T1 of n entries (n = 16 for INT4, 15 for NVFP4; §2 mechanism 1); every
 * group of g weights gets a positive scale; every selection group of S weights picks the table with
 * the lower activation-weighted reconstruction error (§2 mechanism 2); the tables are refined as
 * activation-weighted k-means centroids, alternating with the assignment (§2 mechanism 4); the
 * result is stored as 4-bit codes, bf16 tables, and the table choice in the sign bit of the bf16
 * scale or in a separate bitmap (§2 mechanism 3).
 *
 * Conventions for every call:
 *  - W is bf16 [R, C] row-major (out x in), passed as uint16_t bit patterns. A scale group is g
 *    consecutive weights of a row, a selection group S consecutive weights; groups never cross rows.
 *  - Supported shapes: g and S powers of two with 8 <= S <= g <= 512, C % g == 0, R >= 1,
 *    2 <= n <= 16, R * C < 2^40. Device pointers must be 16-byte aligned.
 *  - All data pointers are DEVICE pointers owned by the caller. The library never allocates, frees
 *    or synchronizes; every call checks its arguments on the host, enqueues its kernels on `stream`
 *    (a hipStream_t; NULL means the default stream) and returns. Buffers must stay alive until the
 *    stream work has completed.
 *  - A failed check returns a non-zero status BEFORE anything is launched, so nothing is written.
 *    AAAC_ERR_HIP reports a launch error seen through hipGetLastError; aaac_last_error() returns a
 *    message for the last failure on the calling thread.
 *  - Workspaces are caller-owned device buffers of at least aaac_workspace_bytes(...) bytes, 256-byte
 *    aligned, and ZERO-FILLED before their first use; every call leaves its workspace zero-filled
 *    again where that matters (the counters), so one workspace can be reused call after call on one
 *    stream. Calls that overlap on different streams need different workspaces.
 *  - Weights must be finite. Results are bitwise deterministic for given inputs and device.
 *  - Tables are fp32 [2][n] (T0 then T1) while iterating; bf16 [2][n] bit patterns when packed.
 */
#ifndef AAAC_H
#define AAAC_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t aaac_status;

#define AAAC_OK 0
#define AAAC_ERR_INVALID_ARG 1          /* null pointer, misaligned pointer, bad flag */
#define AAAC_ERR_UNSUPPORTED_SHAPE 2    /* g, S, n, R, C outside the supported set */
#define AAAC_ERR_WORKSPACE_TOO_SMALL 3  /* ws_bytes below aaac_workspace_bytes(...) */
#define AAAC_ERR_HIP 4                  /* the HIP runtime reported an error */

/* Workspace query operations. */
#define AAAC_OP_IMPORTANCE 0
#define AAAC_OP_INIT 1
#define AAAC_OP_ASSIGN 2
#define AAAC_OP_REFINE 3

/* Flags of aaac_refine. */
#define AAAC_REFINE_ROUND_BF16 1        /* round the new tables to bf16 (ties to even), stored as fp32 */
#define AAAC_REFINE_W2_KNOWN 2          /* *w2 already holds sum I w^2 of this matrix (see err) */

/* Static description of a status code. Never NULL. */
const char* aaac_status_string(aaac_status status);

/* Detail of the last failure on the calling thread ("" if none). Valid until the next call on
 * this thread. */
const char* aaac_last_error(void);

/* Workspace bytes needed by one call of operation `op` on an [R, C] matrix (for IMPORTANCE, R is
 * the token count T and C the column count K). Returns 0 for an unknown op or unsupported shape. */
size_t aaac_workspace_bytes(int op, int64_t R, int64_t C, int g, int S, int n);

/*
 * Importance, AAAC summary §2 mechanism 2: I_k = sum_t X[t, k]^2 over the calibration tokens.
 *
 * X      fp32 [T, K] with row stride ldx >= K (elements); one chunk of the token stream.
 * I_acc  fp64 [K], accumulated in place: I_acc[k] += sum_t X[t, k]^2 (fp32 squares are exact in
 *        fp64). Zero it before the first chunk; chunks may follow in any number of calls.
 * I_out  fp32 [K] or NULL; if given, receives I_acc rounded to fp32 after this chunk.
 * ws     workspace of aaac_workspace_bytes(AAAC_OP_IMPORTANCE, T, K, 0, 0, 0) bytes.
 * T == 0 is allowed (I_out is still written). The sum over a chunk is taken in a fixed order.
 */
aaac_status aaac_importance(const float* X, int64_t T, int64_t K, int64_t ldx, double* I_acc,
                            float* I_out, void* ws, size_t ws_bytes, void* stream);

/*
 * Table initialization, AAAC summary §2 mechanism 4: equally spaced quantiles of the normalized
 * weight distribution, T1 shifted half a step. With s = max |w| over the scale group,
 * u = fl32(w / s) (u = +0 when s = 0), V the ascending sort of all N = R*C values of u:
 *   T0[j] = V[floor((2j + 1) N / (2n))],  T1[j] = V[min(N - 1, floor((j + 1) N / n))].
 * Found by an exact radix select; tables fp32 [2][n] (output).
 * ws: aaac_workspace_bytes(AAAC_OP_INIT, R, C, g, 0, n) bytes.
 */
aaac_status aaac_init_quantiles(const uint16_t* W, int64_t R, int64_t C, int g, int n,
                                float* tables, void* ws, size_t ws_bytes, void* stream);

/*
 * Assign, AAAC summary §2 mechanisms 2 and 4. For every weight and table c, q_c is the entry
 * nearest to u = w / s (ties to the lower index); for every selection group H,
 *   E_c(H) = sum_{k in H} I_k (w_k - s T_c[q_c(k)])^2,   sel(H) = 1 iff E_1 < E_0,
 * and the stored code is q_sel. The nearest entry is decided on exactly rounded fp32 residuals
 * w - s T (a differing decision is only possible when the two squared distances agree to 2.4e-7
 * relative); the selection compares E_1 - E_0 accumulated in fp32 over at most four terms and in
 * fp64 beyond (a differing decision needs |E_1 - E_0| < 1e-6 max(E_0, E_1)).
 *
 * I       fp32 [C] importance (finite, >= 0).
 * tables  fp32 [2][n], any order, duplicates allowed.
 * codes   [R * C / 2] bytes, two codes per byte, the low nibble holds the even column.
 * sel     [R * C / S] bytes, 0 = T0, 1 = T1, one per selection group in row-major order.
 * err     NULL, or fp64 [R * C / S][2] receiving (E_0, E_1) per selection group (for checking).
 * err_total  NULL, or one fp64 receiving the total weighted error of the assignment,
 *         sum over H of E_sel(H) (the k-means objective that the alternation never increases, §2
 *         mechanism 4). Summed in a fixed order (lanes in row order, then waves, then workgroups
 *         in order; no floating-point atomics), so it is reproducible call after call. Needs ws.
 * ws      with err_total: aaac_workspace_bytes(AAAC_OP_ASSIGN, R, C, g, S, n) bytes, same
 *         zero-fill rule as the other workspaces; otherwise ignored (may be NULL, ws_bytes 0).
 * One kernel (the lookup structure lives in LDS).
 */
aaac_status aaac_assign(const uint16_t* W, int64_t R, int64_t C, int g, int S, int n,
                        const float* I, const float* tables, uint8_t* codes, uint8_t* sel,
                        double* err, double* err_total, void* ws, size_t ws_bytes, void* stream);

/*
 * Refine, AAAC summary §2 mechanism 4 (activation-weighted k-means). For every table c and entry j,
 * over the cell {weights with sel = c and code = j}:
 *   num = sum I_k s w_k,  den = sum I_k s^2,   T_c[j] <- num / den if den > 0, else unchanged.
 * num / den minimizes sum I (w - s t)^2 over t, i.e. it is the I s^2-weighted centroid of u.
 * Every term is exact in fp64 and is added in fp64, per thread, then across threads and workgroups
 * in a fixed order, so the result is bitwise reproducible.
 * One kernel: the last workgroup to finish a matrix (an integer ticket in the workspace) adds the
 * per-workgroup partials and writes tables_out. The ticket is reset at the end of every call; a call
 * that did not complete (a device fault) leaves the workspace to be zero-filled again.
 *
 * codes, sel   as written by aaac_assign.
 * tables_in    fp32 [2][n];  tables_out fp32 [2][n], may equal tables_in.
 * flags        0, or AAAC_REFINE_ROUND_BF16 (round the new entries to bf16; used on the last
 *              iteration so that the final assign runs against the stored tables) and/or
 *              AAAC_REFINE_W2_KNOWN (see w2; needs err).
 * err          NULL, or two fp64: err[0] receives the total weighted error of the incoming
 *              assignment under tables_in (the codes and selectors as the assign half-step left
 *              them: the quantity aaac_assign's err_total reports), err[1] the same assignment's
 *              error under the tables this call writes (after this half-step; after the bf16
 *              rounding when that flag is set). Both are formed from the cell sums as
 *              E = W2 - 2 sum_cells T num + sum_cells T^2 den with W2 = sum I_k w_k^2 (sums of
 *              exact fp64 terms). Their absolute accuracy is about 1e-15 W2, far below E except
 *              for matrices quantized almost exactly (aaac_assign's err_total has no such limit).
 * w2           with err: one fp64. Without AAAC_REFINE_W2_KNOWN the kernel sums W2 (one more fp64
 *              fma per weight) and writes it here; with the flag it reads W2 from here (the value
 *              an earlier call on the same W and I wrote), at no cost per weight. NULL without err.
 * ws           aaac_workspace_bytes(AAAC_OP_REFINE, R, C, g, S, n) bytes.
 */
aaac_status aaac_refine(const uint16_t* W, int64_t R, int64_t C, int g, int S, int n,
                        const float* I, const uint8_t* codes, const uint8_t* sel,
                        const float* tables_in, float* tables_out, int flags, double* err,
                        double* w2, void* ws, size_t ws_bytes, void* stream);

/*
 * Pack, AAAC summary §2 mechanism 3 and §4: the stored format.
 *   codes_u8  NULL, or codes given one per byte: u8 [R * C], the code of (r, c) in the low nibble
 *             of byte r * C + c (the high nibble is ignored). Then codes_out (u8 [R * C / 2], not
 *             NULL, 4-byte aligned; codes_u8 8-byte aligned) receives them two per byte, the even
 *             column in the low nibble: the layout aaac_assign writes and aaac_dequant reads. Codes
 *             from aaac_assign are already in that layout and need neither (both NULL).
 *   scales    [R * C / g] bf16 bit patterns of s = max |w| over each scale group; when S == g the
 *             sign bit holds the selector (1 = T1), when S < g it is 0.
 *   bitmap    S < g: [ceil(R * C / S / 8)] bytes, bit i (byte i >> 3, bit i & 7) = selector of the
 *             i-th selection group in row-major order (1 / S extra bits per weight). S == g: NULL.
 *   tables_bf16 [2][n] bf16 bit patterns of the tables (ties to even).
 * Errors: AAAC_ERR_INVALID_ARG for codes_u8 without codes_out (or the reverse) or a misaligned
 * pointer; shape errors as for aaac_assign.
 */
aaac_status aaac_pack(const uint16_t* W, int64_t R, int64_t C, int g, int S, int n,
                      const uint8_t* sel, const float* tables, const uint8_t* codes_u8,
                      uint8_t* codes_out, uint16_t* scales, uint8_t* bitmap,
                      uint16_t* tables_bf16, void* stream);

/*
 * Dequantize, AAAC summary §1 (the dequantized values are what inference uses) and §2 mechanism 3:
 *   W_hat = bf16(|s| * T~_sel[q])  (the product of two bf16 values is exact in fp32; one rounding,
 *   ties to even), with the selector read from the scale sign bit (bitmap == NULL, S == g) or from
 *   the bitmap (S < g).
 * W_hat  bf16 [R, C] bit patterns (output).
 */
aaac_status aaac_dequant(const uint8_t* codes, const uint16_t* scales, const uint8_t* bitmap,
                         const uint16_t* tables_bf16, int64_t R, int64_t C, int g, int S, int n,
                         uint16_t* W_hat, void* stream);

/*
 * Pack and dequantize up to AAAC_MAX_BATCH matrices that share g, S and n, in one set of launches
 * (pack: 1, or 2 with bitmaps; dequant: 1): every output as aaac_pack / aaac_dequant give for
 * matrix i, bit for bit. Arrays of count per-matrix arguments, laid out and owned as in the
 * single calls; bitmap may be NULL when S == g (else it and every bitmap[i] must be given).
 * Errors: AAAC_ERR_INVALID_ARG for count outside [1, AAAC_MAX_BATCH], a null array, or any matrix
 * the single call would reject (nothing is launched then).
 */
aaac_status aaac_pack_batch(int count, const uint16_t* const* W, const int64_t* R,
                            const int64_t* C, int g, int S, int n, const uint8_t* const* sel,
                            const float* const* tables, uint16_t* const* scales,
                            uint8_t* const* bitmap, uint16_t* const* tables_bf16, void* stream);
aaac_status aaac_dequant_batch(int count, const uint8_t* const* codes,
                               const uint16_t* const* scales, const uint8_t* const* bitmap,
                               const uint16_t* const* tables_bf16, const int64_t* R,
                               const int64_t* C, int g, int S, int n, uint16_t* const* W_hat,
                               void* stream);

/*
 * Decode GEMV on the packed format, AAAC summary §1 (4-bit weights with 16-bit activations, W4A16;
 * the dequantized values are the weights inference uses) and §2 mechanism 3 (the stored format):
 *   y[b, r] = sum_c |s(r, c)| * T~_sel(r, c)[q(r, c)] * x[b, c]      for b < B
 * The weight is the exact product of the bf16 scale and the bf16 table entry (both are bf16, so the
 * product is exact in fp32); unlike aaac_dequant it is not rounded to bf16 first. Sums run in fp32
 * in a fixed order (bitwise reproducible): within a scale group, then scaled by |s|, then across
 * groups; a code >= n reads entry 0, as in aaac_dequant.
 * codes, scales, bitmap, tables_bf16  as written by aaac_assign / aaac_pack (bitmap NULL iff S == g).
 *                                     codes 16-byte aligned, scales 8-byte aligned.
 * x   bf16 [B, C] bit patterns (row stride C), 16-byte aligned; 1 <= B <= 4.
 * y   fp32 [B, R] (output, row stride R).
 * Shapes as for the other calls, C % 32 == 0, and fewer than 2^24 blocks of 32 rows (of 16 over
 * 4096 columns, 8 over 8192), in aaac_gemv_batch over all matrices together.
 */
aaac_status aaac_gemv(const uint8_t* codes, const uint16_t* scales, const uint8_t* bitmap,
                      const uint16_t* tables_bf16, int64_t R, int64_t C, int g, int S, int n,
                      const uint16_t* x, int B, float* y, void* stream);

/* aaac_gemv over up to AAAC_MAX_BATCH matrices sharing g, S, n and B in one launch (for example
 * every linear of a decoder layer for one decode step). bitmap is an array of count pointers when
 * S < g, else NULL. Results are bitwise identical to one aaac_gemv call per matrix. */
aaac_status aaac_gemv_batch(int count, const uint8_t* const* codes, const uint16_t* const* scales,
                            const uint8_t* const* bitmap, const uint16_t* const* tables_bf16,
                            const int64_t* R, const int64_t* C, int g, int S, int n,
                            const uint16_t* const* x, int B, float* const* y, void* stream);

/*
 * AWQ composition hook, AAAC summary §4 (AAAC on weights that AWQ scaled before quantization; the
 * search for the scales is not part of this library). Given a positive finite per-column scale
 * a [C] (fp32), prepares the inputs that quantize W diag(a) against the importance that matches
 * it, the energy of the inputs x / a that the scaled matrix sees at inference:
 *   W_scaled[r, c] = bf16(W[r, c] * a[c])   exact product, one rounding (ties to even); a product
 *                                           past the bf16 range becomes infinite, so choose a that
 *                                           keeps the weights finite
 *   I_scaled[c]    = fp32(I[c] / a[c]^2)    one fp64 division of exact operands, then fp32
 * W, W_scaled  bf16 [R, C]; W_scaled may be W (in place). 16-byte aligned.
 * a            fp32 [C], 16-byte aligned.
 * I, I_scaled  fp32 [C], both NULL or both given; I_scaled may be I.
 * The rest of the pipeline then runs on (W_scaled, I_scaled) unchanged. Shapes: R >= 1, C >= 8,
 * C % 8 == 0, R * C < 2^40.
 */
aaac_status aaac_awq_prescale(const uint16_t* W, int64_t R, int64_t C, const float* a,
                              const float* I, uint16_t* W_scaled, float* I_scaled, void* stream);

/*
 * Batched assign / refine over up to AAAC_MAX_BATCH matrices that share g, S and n (for example
 * the seven linears of one decoder layer) in one launch each. Element i of every array describes
 * matrix i exactly as the single-matrix call does; the results are bitwise identical to calling
 * the single-matrix entry points one matrix at a time, except where a sum's rounding depends on
 * how the rows are split over workgroups (the refine sums and err_total: the same call gives the
 * same bits every time; against single calls they agree to rounding). refine updates tables[i] in
 * place. The host arrays are read during the call only. The refine workspace holds
 * aaac_batch_workspace_bytes(AAAC_OP_REFINE, count, R, C, g, S, n) bytes, same zero-fill rule as
 * above. assign: err_total is NULL or fp64 [count] (the total of matrix i in err_total[i]), with
 * a workspace of aaac_batch_workspace_bytes(AAAC_OP_ASSIGN, count, R, C, g, S, n) bytes.
 * refine: err is NULL or fp64 [2][count] (matrix i's error before the update at err[i], after it
 * at err[count + i]), w2 NULL or fp64 [count] (matrix i's at index i); as in aaac_refine.
 */
#define AAAC_MAX_BATCH 8

size_t aaac_batch_workspace_bytes(int op, int count, const int64_t* R, const int64_t* C, int g,
                                  int S, int n);

/*
 * Init for up to AAAC_MAX_BATCH matrices sharing g and n, in one set of launches (6 in all, not 6
 * per matrix): tables[i] as aaac_init_quantiles gives for matrix i, bit for bit. The workspace
 * holds aaac_batch_workspace_bytes(AAAC_OP_INIT, count, R, C, g, 8, n) bytes (fixed headers of
 * histograms, then the keys of every matrix), zero-filled before its first use; every call leaves
 * the headers zero again, so one workspace serves any later batch that fits in it.
 */
aaac_status aaac_init_quantiles_batch(int count, const uint16_t* const* W, const int64_t* R,
                                      const int64_t* C, int g, int n, float* const* tables,
                                      void* ws, size_t ws_bytes, void* stream);

aaac_status aaac_assign_batch(int count, const uint16_t* const* W, const int64_t* R,
                              const int64_t* C, int g, int S, int n, const float* const* I,
                              const float* const* tables, uint8_t* const* codes,
                              uint8_t* const* sel, double* err_total, void* ws, size_t ws_bytes,
                              void* stream);

aaac_status aaac_refine_batch(int count, const uint16_t* const* W, const int64_t* R,
                              const int64_t* C, int g, int S, int n, const float* const* I,
                              const uint8_t* const* codes, const uint8_t* const* sel,
                              float* const* tables, int flags, double* err, double* w2, void* ws,
                              size_t ws_bytes, void* stream);

/*
 * aaac_refine_batch without a workspace argument, for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid allocation). The
 * counters and per-workgroup partials live in a fixed array in the library's device memory: each
 * GPU the library runs on holds one copy, of 256 + 8 * 66 * 1024 * 8 bytes (about 4.3 MB), until
 * the process ends; its address on a device is looked up once, on the first call there. Every
 * other argument, and every result, is as for aaac_refine_batch (bit for bit the same). The call
 * allocates nothing and launches a small kernel that clears the counters before the refine.
 * All calls on one GPU share that array, so calls that overlap on one GPU (on different streams,
 * or from different threads) race and must not be issued; calls on one stream are ordered.
 * Errors: as aaac_refine_batch; AAAC_ERR_WORKSPACE_TOO_SMALL if a batch needed more scratch than
 * the array holds (not possible within AAAC_MAX_BATCH matrices); AAAC_ERR_HIP if the array's
 * address cannot be obtained.
 */
aaac_status aaac_refine_batch_noalloc(int count, const uint16_t* const* W, const int64_t* R,
                                      const int64_t* C, int g, int S, int n,
                                      const float* const* I, const uint8_t* const* codes,
                                      const uint8_t* const* sel, float* const* tables, int flags,
                                      double* err, double* w2, void* stream);

/*
 * One iteration of the alternation (AAAC summary §2 mechanism 4) in one launch: the batched assign
 * against tables[i], writing codes[i] and sel[i], then the batched refine from those codes,
 * updating tables[i] in place. flags, err and w2 are as for aaac_refine_batch: err[i] receives the
 * weighted error of the assignment this call makes under the tables it was made with, and
 * err[count + i] under the tables it writes. Codes, selectors, tables and errors are bitwise those
 * of aaac_assign_batch followed by aaac_refine_batch with the same arguments. With S >= 16 one kernel does both: each wave assigns
 * a row and adds its terms into the refine bins at once, so W is read once. With S = 8 the call
 * makes the two launches. Workspace: as aaac_refine_batch.
 * Errors: as aaac_assign_batch and aaac_refine_batch.
 */
aaac_status aaac_assign_refine_batch(int count, const uint16_t* const* W, const int64_t* R,
                                     const int64_t* C, int g, int S, int n,
                                     const float* const* I, float* const* tables,
                                     uint8_t* const* codes, uint8_t* const* sel, int flags,
                                     double* err, double* w2, void* ws, size_t ws_bytes,
                                     void* stream);

/*
 * Element types of the calls below.
 */
#define AAAC_BF16 0
#define AAAC_F16 1
#define AAAC_F32 2
#define AAAC_MXFP4 3                    /* matmul input: codes and scale bytes of aaac_mxfp4_quantize */

/*
 * MXFP4 quantization (OCP Microscaling formats, MXFP4: 4-bit e2m1 elements in blocks of 32 along a
 * row with one power-of-two scale, e8m0), the other 4-bit weight format beside the dual-codebook
 * one, and the format of 4-bit activations. The last block of a row is padded with zeros; with
 * Cp = 32 ceil(C / 32):
 *   e = clamp(floor(log2 max |x|) - 2, -127, 127) over the block, scale byte e + 127;
 *   code = the e2m1 value nearest to x 2^-e, ties to the even code, magnitudes above 6 become 6.
 * A block of zeros has scale byte 0. A block holding an infinity or a NaN has scale byte 255 and
 * zero codes, and reads back as NaN. Code values by bits 0..2: 0, 1/2, 1, 3/2, 2, 3, 4, 6; bit 3 is
 * the sign.
 * X       [M, C] of x_type AAAC_BF16, AAAC_F16 or AAAC_F32, row stride ldx >= C (elements), aligned
 *         to its element; rows of 16-byte multiples on a 16-byte boundary are read fastest.
 * codes   u8 [M, Cp / 2], two codes per byte, the low nibble holds the even column; 16-byte aligned.
 * scales  u8 [M, Cp / 32].
 * Shapes: M >= 0 (0: nothing is written), 1 <= C < 2^21, M * Cp < 2^40. One kernel.
 */
aaac_status aaac_mxfp4_quantize(const void* X, int x_type, int64_t M, int64_t C, int64_t ldx,
                                uint8_t* codes, uint8_t* scales, void* stream);

/*
 * The values of MXFP4 codes: y = e2m1[code] 2^(byte - 127), exact in fp32 up to its range, rounded
 * once to y_type (ties to even); scale byte 255 gives NaN. Y [M, C] with row stride ldy >= C; only
 * the C columns of a row are written. codes 4-byte aligned. Shapes as aaac_mxfp4_quantize.
 */
aaac_status aaac_mxfp4_dequant(const uint8_t* codes, const uint8_t* scales, int64_t M, int64_t C,
                               void* Y, int y_type, int64_t ldy, void* stream);

/* The products below, as aaac_matmul_workspace_bytes names them. */
#define AAAC_MATMUL_PACKED 0            /* aaac_matmul */
#define AAAC_MATMUL_MXFP4 1             /* aaac_mxfp4_matmul, x bf16 */
#define AAAC_MATMUL_MXFP4_X 2           /* aaac_mxfp4_matmul, x in MXFP4 */
#define AAAC_MATMUL_QUANTIZE_X 3        /* aaac_mxfp4_matmul with AAAC_QUANTIZE_X */

/* Flags of aaac_mxfp4_matmul. */
#define AAAC_QUANTIZE_X 1               /* x is quantized to MXFP4 first, in the workspace */

/* Workspace bytes of one product call of the given kind, 0 for an unsupported shape or where the
 * call uses none. The workspace needs no particular contents and keeps none that matter. */
size_t aaac_matmul_workspace_bytes(int kind, int64_t E, int64_t R, int64_t C, int64_t T);

/*
 * How one product call of the given kind runs on the current device, for tests and profiles:
 *   plan[0], plan[1]  weight rows and rows of x in a tile, both 0 for the few-row kernels;
 *   plan[2]           workgroups that share a tile's columns (1 without a workspace);
 *   plan[3] .. [5]    few-row kernels: blocks of 16 weight rows and of 16 rows of x a workgroup,
 *                     chunks of columns a wave at a time; 0 for tiles.
 * AAAC_ERR_UNSUPPORTED_SHAPE where aaac_matmul_workspace_bytes knows no such call.
 */
aaac_status aaac_matmul_plan(int kind, int64_t E, int64_t R, int64_t C, int64_t T, int has_ws,
                             int32_t plan[6]);

/*
 * Matrix products on 4-bit weights for any number of rows of x, grouped by expert:
 *   y[t, r] = sum_c x[t, c] W_e[r, c]   for offsets[e] <= t < offsets[e + 1],
 * W_e the values of the e-th of E stacked [R, C] matrices; sums in fp32 in an order fixed by the
 * call's shapes and by whether it has a workspace (bitwise reproducible), rounded once to y_type.
 * offsets  int32 [E + 1] on the device, ascending: the rows of x sorted by expert; an expert may
 *          have none. Rows of y outside [offsets[0], offsets[E]) are left as they were. Values are
 *          not checked on the host: the kernels clamp them to [0, T] and to ascending order, so a
 *          bad one never leads outside x or y. NULL (then E must be 1): every row belongs to the
 *          one matrix.
 * T        rows of x and y, 0 <= T < 2^31; T = 0 launches nothing.
 * y        [T, R] of y_type AAAC_BF16, AAAC_F16 or AAAC_F32, row stride ldy >= R, aligned to its
 *          element. y must not overlap an input.
 * ws       NULL with ws_bytes 0, or aaac_matmul_workspace_bytes(...) bytes, 256-byte aligned. With
 *          it a product of few output tiles splits its columns over workgroups and adds their fp32
 *          sums in order with a second kernel.
 * Shapes: 1 <= E <= 65535, 1 <= R < 2^31, 1 <= C < 2^21, E * R * C < 2^40, and at most 2^31 output
 * tiles of 16 x 16.
 *
 * aaac_mxfp4_matmul: weights in MXFP4, w_codes [E, R, Cp / 2] (16-byte aligned) and w_scales
 * [E, R, Cp / 32] as aaac_mxfp4_quantize writes them for the stacked rows. x_type:
 *   AAAC_MXFP4  x = codes [T, Cp / 2] (16-byte aligned), x_scales [T, Cp / 32], ldx ignored; products
 *               of codes and scales are exact.
 *   AAAC_BF16   x bf16 [T, C], row stride C <= ldx < 2^21; x 16-byte aligned, C % 8 == 0,
 *               ldx % 8 == 0; x_scales NULL.
 *   with the flag AAAC_QUANTIZE_X: AAAC_BF16, AAAC_F16 or AAAC_F32, x [T, C] of any row stride
 *               ldx >= C, aligned to its element; x_scales NULL. The call runs aaac_mxfp4_quantize
 *               into ws (which it then needs) and multiplies the result: the same bits as the two
 *               calls with a workspace give.
 *
 * aaac_matmul: weights in the packed dual-codebook format, stacked: codes [E, R, C / 2] (16-byte
 * aligned), scales [E, R, C / g], tables_bf16 [E, 2, n], bitmap [E, ceil(R * C / S / 8)] exactly
 * when S < g, each matrix's part as aaac_assign and aaac_pack write it. The weight is aaac_dequant's
 * W_hat = bf16(|s| T~_sel[q]) (a product below 2^-126 may differ from it by its rounding); a code
 * >= n reads entry 0. x bf16 [T, C] as above. g, S, n as for the other calls, and C % 32 == 0.
 *
 * Weights may start where a larger tensor's part starts: scales and tables_bf16 of aaac_matmul on any
 * 2-byte address, its bitmap, and w_scales and x_scales of aaac_mxfp4_matmul, on any byte.
 */
aaac_status aaac_mxfp4_matmul(const uint8_t* w_codes, const uint8_t* w_scales, int64_t E, int64_t R,
                              int64_t C, const int32_t* offsets, const void* x, int x_type,
                              const uint8_t* x_scales, int64_t T, int64_t ldx, int flags, void* y,
                              int y_type, int64_t ldy, void* ws, size_t ws_bytes, void* stream);
aaac_status aaac_matmul(const uint8_t* codes, const uint16_t* scales, const uint8_t* bitmap,
                        const uint16_t* tables_bf16, int64_t E, int64_t R, int64_t C, int g, int S,
                        int n, const int32_t* offsets, const uint16_t* x, int64_t T, int64_t ldx,
                        void* y, int y_type, int64_t ldy, void* ws, size_t ws_bytes, void* stream);

#define AAAC_FP8 4                      /* aaac_fp8_matmul input: codes and scales of aaac_fp8_quantize */

/*
 * 8-bit floating point (OCP FP8 e4m3: largest value 448, 0x7f and 0xff NaN, no infinities) with one
 * fp32 scale for each block of 128: 128 columns of a row (tile 0, activations), or 128 rows by 128
 * columns of a weight matrix (tile 1). Blocks at a row's or a matrix's end may be short.
 *   scale = max(top / 448, 2^-126), top = max |x| over the block, in fp32;
 *   code  = the e4m3 value nearest to the fp32 quotient x / scale, ties to even.
 * A block holding an infinity or a NaN has a NaN scale and NaN codes (0x7f) and reads back as NaN.
 * X       [E, M, C] of x_type AAAC_BF16, AAAC_F16 or AAAC_F32, row stride ldx >= C, matrices stride_x >=
 *         (M - 1) ldx + C elements apart, aligned to its element. tile 0: E = 1.
 * codes   u8 [E, M, ldq], 16-byte aligned, ldq % 16 == 0, ldq >= C; the columns of a row from C to the
 *         next multiple of 16 are zeroed, those behind it left alone.
 * scales  fp32 [M, ceil(C / 128)], or with tile 1 [E, ceil(M / 128), ceil(C / 128)].
 * Shapes: E >= 1, M >= 0 (0: nothing is written), 1 <= C < 2^21, E * M * C < 2^40. One kernel.
 */
aaac_status aaac_fp8_quantize(const void* X, int x_type, int64_t E, int64_t M, int64_t C, int64_t ldx,
                              int64_t stride_x, int tile, uint8_t* codes, int64_t ldq, float* scales,
                              void* stream);

/*
 * The values of FP8 codes: y = code * scale in fp32, rounded to y_type. codes as above but on any
 * address and with any ldq >= C (those on 16 bytes are read fastest); Y [E M, C] with row stride ldy.
 */
aaac_status aaac_fp8_dequant(const uint8_t* codes, int64_t ldq, const float* scales, int64_t E,
                             int64_t M, int64_t C, int tile, void* Y, int y_type, int64_t ldy,
                             void* stream);

/* Workspace bytes of one aaac_fp8_matmul call, 0 for an unsupported shape or where it uses none. The
 * workspace needs no particular contents and keeps none that matter. quantize: x is not FP8. */
size_t aaac_fp8_matmul_workspace_bytes(int64_t E, int64_t R, int64_t C, int64_t T, int64_t Tx,
                                       int quantize, int y_type);

/* How one such call runs on the current device, as aaac_matmul_plan. */
aaac_status aaac_fp8_matmul_plan(int64_t E, int64_t R, int64_t C, int64_t T, int y_type, int has_ws,
                                 int32_t plan[6]);

/*
 * Matrix product on FP8 weights for any number of rows, grouped by expert as the products above:
 *   y[t, r] = sum over blocks b of (sx[i, b] sw_e[r / 128, b]) sum_{c in b} qx[i, c] qw_e[r, c],
 * i = t, or rows[t], in a fixed order, rounded once to y_type. Products of codes are exact, and sums are kept
 * in fp32. Results in AAAC_F32 and AAAC_F16 add as fp32 does; for AAAC_BF16 the matrix unit adds eight products of
 * a block at a time, cut below 2^-13 of the largest of them. The two scales' product is one fp32 number: an
 * infinity where the largest values of the two blocks multiply to more than 2^128 448^2, and of fewer bits
 * where it is below 2^-126.
 * w_codes  [E, R, ldw] (16-byte aligned, ldw % 16 == 0, C <= ldw < 2^22), w_scales fp32
 *          [E, ceil(R / 128), ceil(C / 128)], as aaac_fp8_quantize writes them with tile 1. Bytes of a row
 *          past C are not used.
 * offsets  int32 [E + 1] or NULL, as above.
 * rows     int32 [T] on the device or NULL: the row of x that row t of y multiplies, such as the token of
 *          a routed slot. Values outside [0, Tx) stand for a row of zeros; with Tx = 0 that is every one, and
 *          no workspace is used. NULL: Tx = T.
 * x        AAAC_FP8: codes [Tx, ldx bytes] (16-byte aligned, ldx % 16 == 0, C <= ldx < 2^22) with x_scales
 *          fp32 [Tx, ceil(C / 128)]; else AAAC_BF16, AAAC_F16 or AAAC_F32 [Tx, C], any row stride ldx >= C,
 *          x_scales NULL: the call quantizes x as aaac_fp8_quantize does, into ws where it needs one for
 *          that, and multiplies the result: the same bits as two calls with a workspace give.
 * y, ws    as above. y must not overlap an input.
 * Shapes: 1 <= E <= 65535, 1 <= R < 2^31, 1 <= C < 2^21, E * R * C < 2^40, 0 <= T, Tx < 2^31, at most
 * 2^31 output tiles of 16 x 16; with rows, codes and scales of x below 2^31 bytes each.
 */
aaac_status aaac_fp8_matmul(const uint8_t* w_codes, int64_t ldw, const float* w_scales, int64_t E,
                            int64_t R, int64_t C, const int32_t* offsets, const int32_t* rows,
                            const void* x, int x_type, const float* x_scales, int64_t Tx, int64_t ldx,
                            int64_t T, void* y, int y_type, int64_t ldy, void* ws, size_t ws_bytes,
                            void* stream);

/* Scores of aaac_route. */
#define AAAC_SOFTMAX 0
#define AAAC_SIGMOID 1

/* Workspace bytes of one aaac_route call, 0 where it uses none. */
size_t aaac_route_workspace_bytes(int64_t T, int64_t E);

/*
 * Routing of T tokens to k of E experts, and the order of the chosen slots by expert that the grouped
 * products take.
 * Choice: scores s = softmax(logits) over a token's experts or sigmoid(logits); value v = s + bias. An
 * expert whose logit or bias is -inf is left out, also where the other is a NaN. The experts form `groups`
 * groups of E / groups neighbours; a group's value is its largest v (group_top 1) or the sum of its two largest (group_top 2;
 * one, where a group has only one left), and only the top_groups largest groups take part. The k largest
 * v are chosen, in descending order; the lower index first among equals, of groups too. Values are
 * compared in 64 bits, and where neither a bias nor a sum over a group enters, by the logits themselves.
 * A NaN ranks above every number: a logit's shows in the weights, a bias's puts its expert first and leaves them.
 * Weights: s of the chosen experts, without the bias, divided by their sum with `renormalize` (a sum of
 * zero gives zeros), times `scale`.
 * logits   [T, E] of type AAAC_BF16, AAAC_F16 or AAAC_F32, row stride ldl >= E elements.
 * bias     fp32 [E] or NULL.
 * experts  int32 [T, k]: a token's experts, -1 where none is left; weights fp32 [T, k], 0 there.
 * offsets  int32 [E + 1]: the places of expert e are offsets[e] <= p < offsets[e + 1].
 * places   int32 [T, k]: the place of each slot, places of one expert in the order of their slots
 *          (token by token); -1 for slots without an expert.
 * rows     int32 [T k]: the token of each place, -1 from offsets[E] on.
 * ws       NULL with ws_bytes 0 where the call uses none, else aaac_route_workspace_bytes(...) bytes,
 *          256-byte aligned, no particular contents.
 * Shapes: T >= 0 with T k < 2^31 (T = 0: the offsets are zeroed), 1 <= E <= 512, 1 <= k <= min(64,
 * top_groups E / groups), 1 <= top_groups <= groups <= 64, E % groups == 0. Results are bitwise
 * reproducible. One kernel for few tokens (16 to 64, by E), two above.
 */
aaac_status aaac_route(const void* logits, int type, int64_t T, int64_t E, int64_t ldl,
                       const float* bias, int score, int64_t k, int groups, int top_groups,
                       int group_top, int renormalize, float scale, int32_t* experts, float* weights,
                       int32_t* offsets, int32_t* rows, int32_t* places, void* ws, size_t ws_bytes,
                       void* stream);

/*
 * Rows to their experts: out[places[t, j]] = x[t] for j < k. x [T, C] of any type of `element` bytes (1,
 * 2 or 4), row stride ldx >= C; out [N, C], row stride ldo >= C (elements). places int32 [T, k] on the
 * device; those outside [0, N) are skipped, and rows of out that no place names are left as they were.
 * A place may be named once. out must not overlap x. Shapes: 0 <= T, N < 2^31, 1 <= k <= 64,
 * 1 <= C < 2^31.
 */
aaac_status aaac_rows_to_experts(const void* x, int element, int64_t T, int64_t C, int64_t ldx,
                                 const int32_t* places, int64_t k, void* out, int64_t N, int64_t ldo,
                                 void* stream);

/*
 * And back: out[t] = sum over j of weights[t, j] y[places[t, j]], in fp32 in the order of j, rounded once
 * to out_type; places outside [0, N) add nothing. y [N, C] of y_type, out [T, C] of out_type (AAAC_BF16,
 * AAAC_F16, AAAC_F32); weights fp32 [T, k]; out must not overlap y. Shapes as above.
 */
aaac_status aaac_rows_from_experts(const void* y, int y_type, int64_t N, int64_t C, int64_t ldy,
                                   const int32_t* places, const float* weights, int64_t T, int64_t k,
                                   void* out, int out_type, int64_t ldo, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* AAAC_H */

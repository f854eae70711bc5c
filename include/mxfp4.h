/*
 * libmxfp4 — MXFP4 block quantizer for NVIDIA B200 (sm_100a).
 *
 * C ABI. Every entry point takes plain device pointers, element counts and a
 * CUDA stream passed as `void*` (a cudaStream_t; NULL means the legacy
 * default stream). The caller owns every buffer and the stream. The library
 * allocates no memory, keeps no state between calls and never synchronises:
 * work is enqueued on `stream` and the call returns. Arguments are validated
 * on the host before any launch; a failed check returns a status and launches
 * nothing. Nothing in the library aborts or traps.
 *
 * Format (sources: "ALTO MXFP4 training — Weight de-oscillation — What does it
 * mean?", Jargon: MXFP4, E2M1, Bin; "Unveiling the Potential of Quantization
 * with MXFP4", abstract: power-of-two block scaling):
 *   - A group is 32 consecutive elements along the group axis. ROWS groups are
 *     1x32 (32 consecutive columns of one row); COLS groups are 32x1 (32
 *     consecutive rows of one column).
 *   - Every group shares one power-of-two scale 2^e, stored as an E8M0 byte
 *     e + 127. e = floor(log2(absmax)) - 2, clamped to [-127, 127]; a group of
 *     zeros stores byte 0; a group holding Inf or NaN stores byte 0xFF and all
 *     of its codes are 0.
 *   - Each element x becomes a 4-bit E2M1 code: bit 3 = sign of x, bits 0..2 =
 *     index m of the magnitude G[m] in {0, 0.5, 1, 1.5, 2, 3, 4, 6} nearest to
 *     |x| * 2^-e (RNE: ties go to even m; |x| * 2^-e >= 6 saturates to 6), or
 *     chosen stochastically between the two neighbours (SR, below).
 *   - Two codes per byte: the element with the even index along the group
 *     axis sits in the low nibble.
 *
 * Layouts for an input X of shape [rows, cols], row-major:
 *   ROWS: codes [rows][cols/2],  scales [rows][cols/32]
 *   COLS: codes [cols][rows/2],  scales [cols][rows/32]   (element (r,c) is at
 *         byte c*rows/2 + r/2; the column layout is the transpose, K-major
 *         along rows, which the weight-gradient GEMM consumes)
 *
 * Stochastic rounding (ALTO explainer, Jargon: Stochastic rounding; TetraJet
 * rebuttal, Question 2, point (2): an unbiased quantizer): for a = |x|*2^-e
 * below 6, lo = largest grid value <= a, hi = the next one,
 * frac = (a - lo)/(hi - lo); the result is hi iff (r + 0.5) * 2^-16 < frac,
 * where r is the element's 16-bit random number. a >= 6 gives 6.
 *
 * Random numbers (counter based, no state): mix() is the MurmurHash3 32-bit
 * finalizer. K(seed, s) = mix(lo32(seed) ^ mix(hi32(seed) + s*0x9E3779B9)).
 * For the element with row-major index i = r*cols + c of the INPUT tensor
 * (whatever the axis, tiling or launch shape) and pair p = i >> 1,
 * h = mix(mix(K ^ hi32(p)) + lo32(p)); even i takes h & 0xFFFF, odd i takes
 * h >> 16. Streams s: 0 = stochastic rounding, 1 = Hadamard column signs,
 * 2 = synthetic optimizer updates.
 *
 * Alignment: every tensor pointer (x, codes, y, w, w_snap, d_w, d_q, rotated)
 * must be 16-byte aligned; scale pointers may have any alignment.
 */
#ifndef MXFP4_H
#define MXFP4_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum mxfp4_status {
  MXFP4_OK = 0,
  MXFP4_ERR_NULL = 1,  /* a required pointer is NULL */
  MXFP4_ERR_SHAPE = 2, /* rows or cols <= 0, a group axis that is not a
                          multiple of 32, or a size past the stated limit */
  MXFP4_ERR_ALIGN = 3, /* a tensor pointer is not 16-byte aligned (a
                          status word: not 4-byte aligned) */
  MXFP4_ERR_ENUM = 4,  /* dtype, axis or rounding out of range */
  MXFP4_ERR_CUDA = 5,  /* the launch failed (cudaGetLastError); faults of a
                          kernel that launched surface on the stream */
  MXFP4_ERR_VALUE = 6, /* a number (eps, a factor, a step count) is outside
                          its stated range */
  MXFP4_ERR_WORKSPACE = 7 /* the workspace is smaller than its entry point's
                             _workspace function says */
} mxfp4_status;

typedef enum mxfp4_dtype { MXFP4_F32 = 0, MXFP4_BF16 = 1 } mxfp4_dtype;
typedef enum mxfp4_axis { MXFP4_ROWS = 0, MXFP4_COLS = 1 } mxfp4_axis;
typedef enum mxfp4_rounding { MXFP4_RNE = 0, MXFP4_SR = 1 } mxfp4_rounding;

/* Largest rows and largest cols accepted (each); rows*cols must also stay
 * below 2^46 elements. */
#define MXFP4_MAX_DIM ((int64_t)1 << 31)

/*
 * Device status word of the tensor-core entry points (mxfp4_rht_quantize,
 * mxfp4_rht_quantize_oas, mxfp4_gemm, mxfp4_gemm_quantize_a). Their kernels wait on mbarriers for
 * copies and tensor-core work inside the CTA; every such wait is bounded.
 * When one runs out, the CTA stops waiting, lets its own copies and MMAs in
 * flight finish (again with bounded waits), frees its tensor memory, writes
 * the poison values the entry point states for the tiles it did not
 * complete, and ORs MXFP4_STATUS_WAIT_TIMEOUT into the caller's status word
 * (an int in device memory, 4-byte aligned; NULL: not reported). The bit is
 * never cleared by the library: zero the word before the call and read it
 * once the stream has passed the call. A set bit means the outputs are
 * incomplete; it does not mean the CUDA context is damaged. The paper has no
 * counterpart: this is the library's own error channel.
 */
#define MXFP4_STATUS_WAIT_TIMEOUT 1

/*
 * Block quantize X [rows, cols] (bf16 or fp32) into MXFP4 codes and E8M0
 * scales along `axis`, rounding RNE (deterministic, Q_D) or SR (stochastic,
 * Q_S, keyed by `seed`; ignored for RNE).
 * Sources: ALTO explainer, Jargon (MXFP4, E2M1, Bin, Stochastic rounding);
 * TetraJet rebuttal, Question 2 (Q_D in the forward pass, 1x32 and 32x1
 * group shapes).
 *   x       device, [rows][cols] of dtype, read only
 *   codes   device, rows*cols/2 bytes, written in the layout of `axis`
 *   scales  device, rows*cols/32 bytes, written in the layout of `axis`
 * The group axis (cols for ROWS, rows for COLS) must be a multiple of 32.
 */
mxfp4_status mxfp4_quantize(const void* x, int dtype, int64_t rows,
                            int64_t cols, int axis, int rounding,
                            uint64_t seed, uint8_t* codes, uint8_t* scales,
                            void* stream);

/*
 * mxfp4_quantize with the overflow-aware scale: e is the smallest exponent
 * with absmax * 2^-e <= 6 (instead of floor(log2 absmax) - 2), so no element
 * saturates and stochastic rounding is unbiased for every input; e is the
 * OCP exponent, or one more where the OCP-scaled maximum exceeds 6. Same
 * arguments, layouts, statuses and non-finite handling as mxfp4_quantize.
 * Source: "Unveiling the Potential of Quantization with MXFP4", abstract
 * (overflow-aware scaling under power-of-two block scales); the page gives
 * the idea, not a formula, so the rule above is a reading.
 */
mxfp4_status mxfp4_quantize_oas(const void* x, int dtype, int64_t rows,
                                int64_t cols, int axis, int rounding,
                                uint64_t seed, uint8_t* codes, uint8_t* scales,
                                void* stream);

/*
 * Decode codes and scales back to values: y = (-1)^sign * G[m] * 2^e, exact
 * in bf16 and fp32 (a scale byte of 0xFF decodes to NaN).
 * Source: ALTO explainer, Jargon: MXFP4 (a block of 32 4-bit values sharing
 * one scale).
 *   rows, cols  shape of the tensor that was quantized
 *   codes, scales  device, in the layout of `axis`
 *   y       device, written: [rows][cols] for ROWS, [cols][rows] (the
 *           transpose) for COLS, of out_dtype
 */
mxfp4_status mxfp4_dequantize(const uint8_t* codes, const uint8_t* scales,
                              int64_t rows, int64_t cols, int axis, void* y,
                              int out_dtype, void* stream);

/*
 * TetraJet double quantization Q_S(32x1)(Q_D(1x32)(X)) in one pass over X:
 * the row layout of Q_D along rows (RNE), and the column layout of Q_S
 * (SR, keyed by `seed`) applied to the exactly dequantized row result. The
 * column scales come from Q_D(X), not from X.
 * Source: "Oscillation-Reduced MXFP4 Training for Vision Transformers"
 * rebuttal, Question 2, points (1) and (2).
 *   x                       device, [rows][cols] of dtype
 *   row_codes, row_scales   device, ROWS layout (as mxfp4_quantize)
 *   col_codes, col_scales   device, COLS layout (as mxfp4_quantize)
 * rows and cols must both be multiples of 32.
 */
mxfp4_status mxfp4_double_quantize(const void* x, int dtype, int64_t rows,
                                   int64_t cols, uint64_t seed,
                                   uint8_t* row_codes, uint8_t* row_scales,
                                   uint8_t* col_codes, uint8_t* col_scales,
                                   void* stream);

/*
 * mxfp4_double_quantize with the overflow-aware scale (as mxfp4_quantize_oas)
 * in both passes. The row pass moves where a group maximum would scale above
 * 6; the column pass then sees decoded values with two significant bits,
 * whose maxima never scale above 6, so its scales follow the OCP rule as
 * well. A row scale of 2^126 gives Q_D(X) values of 4 * 2^126 and 6 * 2^126,
 * beyond the fp32 range; the column pass still quantizes them exactly (to
 * codes 4 and 6 at column scale 2^126). Same arguments, layouts and statuses
 * as mxfp4_double_quantize.
 * Source: "Unveiling the Potential of Quantization with MXFP4", abstract
 * (overflow-aware scaling), with the double quantization above.
 */
mxfp4_status mxfp4_double_quantize_oas(const void* x, int dtype, int64_t rows,
                                       int64_t cols, uint64_t seed,
                                       uint8_t* row_codes, uint8_t* row_scales,
                                       uint8_t* col_codes, uint8_t* col_scales,
                                       void* stream);

/*
 * Randomized Hadamard rotation of every 1x32 row group followed by 1x32
 * quantization: y_g = (1/sqrt(32)) * H32 * (s .* x_g), H32 the Sylvester
 * Hadamard matrix (H[j][k] = (-1)^popcount(j&k)), s_c = -1 iff bit 31 of
 * mix(K(sign_seed, 1) + c) is set for column c; fp32 arithmetic (bf16
 * inputs: exact +-1 products summed in fp32 on the tensor cores; fp32
 * inputs: a radix-2 butterfly). y is then quantized along ROWS with
 * `rounding` (SR keyed by sr_seed).
 * Sources: ALTO explainer, Jargon: Randomized Hadamard transform; "Microscaling
 * FP4 Quantization: MR-GPTQ Achieves 6x Speedup", section "FP4 Quantization
 * with Micro-Rotated GPTQ Algorithm" (block-wise Hadamard transforms).
 *   x        device, [rows][cols] of dtype; cols a multiple of 32
 *   codes, scales  device, ROWS layout
 *   rotated  device fp32 [rows][cols] receiving y, or NULL to skip it
 *   status   device int or NULL (MXFP4_STATUS_WAIT_TIMEOUT above); bf16
 *            inputs only (the fp32 path never waits). A group whose
 *            rotation was not read out gets scale byte 0xFF, zero codes and
 *            NaN in `rotated`.
 */
mxfp4_status mxfp4_rht_quantize(const void* x, int dtype, int64_t rows,
                                int64_t cols, uint64_t sign_seed,
                                int rounding, uint64_t sr_seed,
                                uint8_t* codes, uint8_t* scales,
                                float* rotated, int* status, void* stream);

/*
 * mxfp4_rht_quantize with the overflow-aware scale (as mxfp4_quantize_oas)
 * for the rotated values. Same arguments, layouts and statuses.
 */
mxfp4_status mxfp4_rht_quantize_oas(const void* x, int dtype, int64_t rows,
                                    int64_t cols, uint64_t sign_seed,
                                    int rounding, uint64_t sr_seed,
                                    uint8_t* codes, uint8_t* scales,
                                    float* rotated, int* status, void* stream);

/*
 * One step of the weight-oscillation tracker on fp32 master weights w.
 * DQ() is 1x32 RNE quantize-dequantize. Per element, in fp32 with no fused
 * multiply-add:
 *   d_w += |w - w_snap|;  d_q += |DQ(w) - DQ(w_snap)|;  w_snap = w.
 * If window_end != 0, afterwards: an element is flagged iff
 * d_q > threshold * d_w; a flagged w becomes DQ(w) (the centre of its
 * current bin); then d_w = d_q = 0 and w_snap = w for every element, and the
 * number of flagged elements is ADDED to *n_flagged (if not NULL).
 * Source: ALTO explainer, "How does ALTO detect and fix oscillating
 * weights?" and the paragraph on the d_Q/d_w ratio (window P = 200,
 * threshold 4.0, snap to the bin centre; state: two distances and a weight
 * snapshot).
 *   w, w_snap, d_w, d_q  device fp32 [rows][cols], read and written
 *   n_flagged            device, or NULL
 * cols must be a multiple of 32.
 */
mxfp4_status mxfp4_osc_step(float* w, float* w_snap, float* d_w, float* d_q,
                            int64_t rows, int64_t cols, int window_end,
                            float threshold, unsigned long long* n_flagged,
                            void* stream);

/*
 * One iteration of Q-Ramping: oscillation detection in a short tracking
 * window at the start of each epoch, then k2-times-slower updates for the
 * weights it flags. Source: "Oscillation-Reduced MXFP4 Training for Vision
 * Transformers", rebuttal, Weakness 2 (oscillations are tracked only in the
 * first 30 of about 2500 iterations of an epoch) and the hyper-parameter
 * answers (oscillation detection factor k1, 16 recommended; weight update
 * frequency factor k2, 3 to 5, 5 by default). The page gives no formula;
 * this is the reading the library implements (parity against the page
 * unpinned). Per element, in fp32 with no fused multiply-add, at iteration
 * `iter` of the epoch (0-based):
 *   iter == 0:  if flag: w += acc;  acc = 0; flag = 0;
 *               w_snap = w; d_w = d_q = 0          (the window starts)
 *   update:     if flag: acc += delta, and when iter % k2 == k2 - 1:
 *               w += acc, acc = 0;   else: w += delta
 *   iter < track_iters (the window), on the updated w:
 *               d_w += |w - w_snap|; d_q += |DQ(w) - DQ(w_snap)|; w_snap = w
 *               (DQ = 1x32 RNE quantize-dequantize, as mxfp4_osc_step)
 *   iter == track_iters - 1 (the window's end):
 *               flag = d_q > k1 * d_w; d_w = d_q = 0; the number of flagged
 *               elements is ADDED to *n_flagged (if not NULL).
 * Outside the window w_snap, d_w and d_q are neither read nor written.
 *   w, w_snap, d_w, d_q, acc  device fp32 [rows][cols], read and written
 *   delta                     device fp32 [rows][cols], the iteration's
 *                             optimizer update (read only)
 *   flag                      device uint8 [rows][cols] (0 or 1)
 *   n_flagged                 device, or NULL
 * cols must be a multiple of 32; every array 16-byte aligned.
 * MXFP4_ERR_SHAPE also for iter < 0, track_iters < 0 or k2 < 1.
 */
mxfp4_status mxfp4_qramp_step(float* w, const float* delta, float* w_snap,
                              float* d_w, float* d_q, float* acc, uint8_t* flag,
                              int64_t rows, int64_t cols, int64_t iter,
                              int64_t track_iters, float k1, int64_t k2,
                              unsigned long long* n_flagged, void* stream);

/*
 * Synthetic optimizer update that drives the oscillation workload (a stand-in
 * for the AdamW step that the tracker follows; not part of the method):
 * w = w + s * (rel_step * |w|) in fp32 (separate multiply and add), where
 * s = -1 iff bit 31 of mix(mix(K ^ hi32(i)) + lo32(i)) is set, with
 * K = K(seed + (step << 32), 2) and i the row-major element index.
 *   w  device fp32 [rows][cols], read and written
 */
mxfp4_status mxfp4_osc_synthetic_update(float* w, int64_t rows, int64_t cols,
                                        uint64_t seed, uint32_t step,
                                        float rel_step, void* stream);

/*
 * Q-EMA step fused with the forward quantization of the averaged weight:
 * per element, in fp32 with no fused multiply-add,
 *   w_ema = beta * w_ema + (1 - beta) * w        ((1 - beta) rounded first)
 * then the new w_ema is block quantized along 1x32 row groups with RNE, as
 * mxfp4_quantize(w_ema, F32, rows, cols, ROWS, RNE, ...).
 * Source: "Oscillation-Reduced MXFP4 Training for Vision Transformers"
 * rebuttal, Question 4 (an extra EMA weight per linear layer, quantized in
 * the forward pass) and the hyper-parameter answers (beta in
 * [0.997, 0.999], default 0.998).
 *   w       device fp32 [rows][cols], the master weight, read only
 *   w_ema   device fp32 [rows][cols], read and written
 *   codes, scales  device, ROWS layout of the updated w_ema
 * cols must be a multiple of 32.
 */
mxfp4_status mxfp4_qema_quantize(const float* w, float* w_ema, int64_t rows,
                                 int64_t cols, float beta, uint8_t* codes,
                                 uint8_t* scales, void* stream);

/*
 * Scale bytes in the blocked order that block-scaled tensor-core GEMMs read.
 * Source: "Oscillation-Reduced MXFP4 Training for Vision Transformers",
 * abstract (the MX format is supported by the Blackwell architecture); the
 * order itself is NVIDIA's published one-dimensional block-scaling-factor
 * layout of its block-scaled GEMMs (a reading: the pages name the hardware,
 * not the layout). Both GEMM operands of an MXFP4 product are K-major with
 * one scale per 32 elements along K, which is what mxfp4_quantize writes: a
 * ROWS quantization of X [R, C] is an operand with rows = R, groups = C/32;
 * a COLS quantization (and the column output of mxfp4_double_quantize) is
 * the operand X^T with rows = C, groups = R/32.
 *
 * The matrix scales[rows][groups] (row-major) is cut into tiles of 128 rows
 * by 4 groups, zero-padded at the edges; tiles are stored one after another,
 * along the groups first, then for the next 128 rows, 512 bytes each; inside
 * a tile the scale of tile row r and tile group g is byte
 * 16*(r mod 32) + 4*(r div 32) + g.
 *   scales   device, [rows][groups] bytes, any alignment, read only
 *   blocked  device, ceil(rows/128)*128 * ceil(groups/4)*4 bytes, 16-byte
 *            aligned, written entirely (padding included)
 * rows, groups > 0 and within the size limit of the other entry points.
 */
mxfp4_status mxfp4_scales_to_blocked(const uint8_t* scales, int64_t rows,
                                     int64_t groups, uint8_t* blocked,
                                     void* stream);

/*
 * MXFP4 GEMM on the block-scaled tensor cores, consuming quantizer outputs:
 *   C[m][n] = sum_k A[m][k] * B[n][k]      (fp32 accumulate, fp32 out)
 * where A[i][k] = G(a_codes)[i][k] * 2^(a scale of group k/32 of row i - 127)
 * and likewise B. Source: "Oscillation-Reduced MXFP4 Training for Vision
 * Transformers", abstract and rebuttal Question 2 (forward and backward
 * GEMMs on MXFP4 operands quantized along the reduction axis; MX on
 * Blackwell tensor cores).
 *   a_codes   device, [m][k/2], K-major (the ROWS codes of an [m, k] tensor,
 *             or the COLS codes of a [k, m] tensor), 16-byte aligned
 *   a_scales  device, the scales of a_codes in the blocked order of
 *             mxfp4_scales_to_blocked (rows = m, groups = k/32), 16-byte
 *             aligned
 *   b_codes, b_scales  the same for B with n rows
 *   c         device fp32 [m][n], written (every element)
 *   status    device int or NULL (MXFP4_STATUS_WAIT_TIMEOUT above)
 * k must be a multiple of 32; m, n, k > 0 within the size limit. The result
 * equals the exact sum of the products up to fp32 accumulation rounding (the
 * order of the additions is the hardware's). When a bounded wait runs out,
 * the tile it served and the CTA's later tiles are written as NaN.
 */
mxfp4_status mxfp4_gemm(const uint8_t* a_codes, const uint8_t* a_scales,
                        const uint8_t* b_codes, const uint8_t* b_scales,
                        int64_t m, int64_t n, int64_t k, float* c,
                        int* status, void* stream);

/*
 * GEMM with the activation quantized in the GEMM's load stage:
 *   C[m][n] = sum_k Q(X)[m][k] * B[n][k]        (fp32 accumulate, fp32 out)
 * Q(X) is the 1x32 quantization of X along k (ROWS) with `rounding`: RNE
 * (Q_D, the forward GEMM Q_D(X) Q_D(W)^T) or SR (Q_S keyed by `seed`, e.g.
 * a gradient quantized for a backward GEMM), exactly as mxfp4_quantize(x,
 * MXFP4_BF16, m, k, MXFP4_ROWS, rounding, seed, ...) computes it; B is given
 * as in mxfp4_gemm (for the forward GEMM the pre-quantized weight). The
 * result equals that quantization followed by mxfp4_scales_to_blocked and
 * mxfp4_gemm, bit for bit, but Q(X) never passes through global memory:
 * bf16 X tiles are quantized in shared memory into the tensor cores'
 * operand layout. Source: "Oscillation-Reduced MXFP4 Training for Vision
 * Transformers", rebuttal Question 2 (Q_D(X) Q_D(W)^T in the forward pass,
 * Q_S in the backward pass).
 *   x         device bf16 [m][k], 16-byte aligned, read only
 *   rounding  MXFP4_RNE or MXFP4_SR; seed keys SR (ignored for RNE)
 *   b_codes, b_scales  as in mxfp4_gemm, n rows
 *   c         device fp32 [m][n], written (every element)
 *   a_codes   device [m][k/2], 16-byte aligned, or NULL: receives the codes
 *             of Q(X) in the ROWS layout
 *   a_scales  device [m][k/32], or NULL; given exactly when a_codes is
 *   status    device int or NULL, as in mxfp4_gemm; when it is set, the
 *             tiles of C that were not completed hold NaN or were left
 *             unwritten
 * k must be a multiple of 256; m, n > 0 within the size limit. With more
 * than 256 columns of C, clusters of 2 or 4 CTAs (up to 1024 columns) share
 * the quantization of their rows, so X is read and quantized once per 1024
 * columns; the fusion pays where n is small (up to a few hundred to about
 * a thousand columns on B200); for large n the separate quantize +
 * mxfp4_gemm is faster.
 */
mxfp4_status mxfp4_gemm_quantize_a(const void* x, int64_t m, int64_t n, int64_t k,
                                   int rounding, uint64_t seed, const uint8_t* b_codes,
                                   const uint8_t* b_scales, float* c, uint8_t* a_codes,
                                   uint8_t* a_scales, int* status, void* stream);

/* Bytes of workspace mxfp4_gemv needs (0 for m <= 2; about 4 m k else, m
 * rounded up to 8, 16 or a multiple of 32); -1 for a shape it refuses. */
int64_t mxfp4_gemv_workspace(int64_t m, int64_t n, int64_t k);

/*
 * Product of a few unquantized rows with an MXFP4 weight, the step a model
 * answers single tokens with (m = 1 to a few dozen):
 *   Y[m][n] = sum_k X[m][k] * B[n][k]         (fp32 accumulate)
 * X is bf16 and is not quantized; B is given as in mxfp4_gemm. The products
 * run on the block-scaled tensor cores: each x enters as eight base-8 digits
 * (E2M1 values with a power-of-two scale per 32 elements), which add up to x
 * exactly where |x| is at least 2^-16 of the largest magnitude of its group
 * of 32, and are off by at most 2^-23 of that magnitude otherwise (by 2^-128
 * in groups whose largest magnitude is below 2^-104). Sums are fp32; Y is
 * rounded once. The same arguments give the same bits every time.
 *   x        device bf16, row i at x + i * ldx elements; 16-byte aligned,
 *            ldx >= k a multiple of 8
 *   b_codes  device [n][k/2], 16-byte aligned
 *   b_scales device, blocked order (rows = n, groups = k/32), 16-byte aligned
 *   y        device [m][n] of y_dtype, 16-byte aligned, written
 *   workspace  device, 16-byte aligned, workspace_bytes of scratch (at least
 *            mxfp4_gemv_workspace; NULL where that is 0); calls that run at
 *            the same time need workspaces of their own
 *   status   device int or NULL (MXFP4_STATUS_WAIT_TIMEOUT above); the tiles
 *            of a CTA whose wait ran out hold NaN
 * y, workspace and status overlap neither the inputs nor one another.
 * k must be a multiple of 32, m at most 2^19, k at most 2^30. A group of x that holds Inf or
 * NaN makes its row of Y NaN, a scale byte of 0xFF its column.
 * Any m works; from about a hundred rows on, quantizing X (mxfp4_gemm) or
 * decoding B (mxfp4_dequantize) and a dense product are faster.
 * Source: "Microscaling FP4 Quantization: MR-GPTQ Achieves 6x Speedup"
 * (inference with MXFP4 weights).
 */
mxfp4_status mxfp4_gemv(const void* x, int64_t m, int64_t n, int64_t k, int64_t ldx,
                        const uint8_t* b_codes, const uint8_t* b_scales, void* y, int y_dtype,
                        void* workspace, int64_t workspace_bytes, int* status, void* stream);

/* Largest rows and cols of mxfp4_newton_schulz. */
#define MXFP4_NS_MAX_DIM ((int64_t)1 << 20)

/* Bytes of workspace mxfp4_newton_schulz needs (about 6 bytes per element and
 * 4 per element of the smaller square); -1 for a shape it refuses. */
int64_t mxfp4_newton_schulz_workspace(int64_t rows, int64_t cols);

/*
 * A weight's update made nearly orthogonal by Newton-Schulz products (the
 * optimizer step whose result mxfp4_osc_step and mxfp4_qramp_step follow;
 * with scale = minus the step size, OUT in fp32 is mxfp4_qramp_step's delta):
 *   X = G / (|G|_F + eps)
 *   `steps` times:  A = X X^T,  B = b A + c A A,  X = a X + B X
 *   OUT = scale * X
 * (for rows > cols the same with X^T). Each step moves every singular value s
 * of X to a s + b s^3 + c s^5. The products take fp16 operands with fp32
 * sums, X is carried with about 22 bits between steps, the norm is summed in
 * fp64. The result differs from the exact one (before the rounding to
 * out_dtype, relative to its norm, for 3.4445, -4.775, 2.0315 on normal and
 * on nearly low-rank matrices) by at most 3e-3 for up to six steps where the
 * shorter side is 64 or more (measured: 2e-4 to 2.7e-3), and by at most 1e-2
 * for five steps where it is less (measured: up to 6.4e-3); each further step
 * carries the error on (ten steps: measured up to 6e-3, 4e-2 on 2 x 2). The
 * same inputs give the same bits. Values are held times 2^12 in fp16, so the
 * entries of X, A and B must stay below 15.9 in magnitude, which those
 * coefficients do (below 3); a result with Inf or NaN shows where others do
 * not.
 *   g        device, [rows][cols] of dtype, 16-byte aligned, read only
 *   steps    1 to 1000; a, b, c within 1e4 in magnitude; eps >= 0
 *   out      device, [rows][cols] of out_dtype, 16-byte aligned, written; it
 *            may be g itself where the two types are the same
 *   workspace  device, 256-byte aligned, workspace_bytes of scratch (at
 *            least mxfp4_newton_schulz_workspace); calls that run at the same
 *            time need workspaces of their own
 *   status   device int or NULL (MXFP4_STATUS_WAIT_TIMEOUT above); when it is
 *            set, the tiles of OUT that were not completed hold NaN
 * workspace and status overlap neither g nor out nor one another.
 * Any rows, cols up to MXFP4_NS_MAX_DIM. G of zeros gives zeros (eps > 0);
 * Inf or NaN in G gives NaN.
 */
mxfp4_status mxfp4_newton_schulz(const void* g, int dtype, int64_t rows, int64_t cols, int steps,
                                 float a, float b, float c, float eps, float scale, void* out,
                                 int out_dtype, void* workspace, int64_t workspace_bytes,
                                 int* status, void* stream);

/*
 * Layer norm of every row of X, the transform in front of a quantized linear
 * layer (pre-norm blocks of the pages' vision transformers and LLMs):
 *   mean = sum_c X[r][c] / cols,   var = sum_c (X[r][c] - mean)^2 / cols,
 *   rstd = (var + eps)^(-1/2),
 *   Y[r][c] = (X[r][c] - mean) * rstd * weight[c] + bias[c]
 * in fp32 (the squares are summed around the mean, not as E[x^2] - mean^2),
 * rounded once to dtype. The mean is an fp32 sum, off by some 2^-24 of the
 * row's mean |X|, and y by that times rstd * weight: data far from zero beside
 * its spread loses that much, a row of one value its exact zeros with it.
 * Squares and sums are fp32 too: |X - mean| below about 2^63 / sqrt(cols).
 *   x      device, rows of cols elements of dtype, row r at x + r * ldx
 *          elements (ldx >= cols); element alignment suffices, 16-byte
 *          aligned rows are faster
 *   weight, bias  device fp32 [cols] or NULL (1 and 0)
 *   eps    >= 0 and finite
 *   y      device, written: [rows][cols] of dtype
 *   mean, rstd  device fp32 [rows] or NULL: the statistics the backward pass
 *          takes
 * What is written overlaps neither the inputs nor one another.
 * Any rows, cols > 0 within the size limit. A row that holds Inf or NaN
 * gives NaN in that row.
 */
mxfp4_status mxfp4_layernorm(const void* x, int dtype, int64_t rows, int64_t cols,
                             int64_t ldx, const float* weight, const float* bias, float eps,
                             void* y, float* mean, float* rstd, void* stream);

/*
 * mxfp4_layernorm fused with the forward quantization of its output: codes
 * and scales are those of mxfp4_quantize(y, dtype, rows, cols, ROWS, RNE,
 * ...), bit for bit, without y being read back; y itself is written only
 * where it is wanted. y has the bits that mxfp4_layernorm gives, except where
 * x and y lie equally far off a 16-byte boundary and x is dense: the two then
 * sum a row in different orders. Source: "Oscillation-Reduced MXFP4 Training for Vision
 * Transformers", rebuttal Question 2 (Q_D of a linear layer's input in the
 * forward pass).
 *   y       as in mxfp4_layernorm, or NULL
 *   codes, scales  device, ROWS layout; codes 16-byte aligned
 * cols must be a multiple of 32. What is written overlaps neither the inputs
 * nor one another.
 */
mxfp4_status mxfp4_layernorm_quantize(const void* x, int dtype, int64_t rows, int64_t cols,
                                      int64_t ldx, const float* weight, const float* bias,
                                      float eps, void* y, float* mean, float* rstd,
                                      uint8_t* codes, uint8_t* scales, void* stream);

/* Bytes of workspace mxfp4_layernorm_backward needs for dw and db; -1 for a
 * shape it refuses. */
int64_t mxfp4_layernorm_backward_workspace(int64_t rows, int64_t cols);

/*
 * Gradients of mxfp4_layernorm. With h = (x - mean) * rstd and
 * g = dy * weight, per row:
 *   dx = rstd * (g - sum_c(g) / cols - h * sum_c(g * h) / cols)
 * and over the rows, summed in fp32 in a fixed order (the same inputs give
 * the same bits on the same device):
 *   dw[c] = sum_r dy * h,   db[c] = sum_r dy
 *   dy, x   device, of dtype, row strides lddy and ldx (elements)
 *   weight  device fp32 [cols] or NULL (1)
 *   mean, rstd  device fp32 [rows], from the forward pass
 *   dx      device, written: [rows][cols] of dtype
 *   dw, db  device fp32 [cols], written; both NULL to leave them out
 *   workspace  device, 16-byte aligned, workspace_bytes of scratch (at least
 *           mxfp4_layernorm_backward_workspace); not read by a later call.
 *           NULL only where dw and db are. Calls that run at the same time
 *           need workspaces of their own.
 * dx and workspace overlap neither the inputs nor one another; dw and db
 * overlap neither these two nor one another.
 */
mxfp4_status mxfp4_layernorm_backward(const void* dy, const void* x, int dtype, int64_t rows,
                                      int64_t cols, int64_t lddy, int64_t ldx,
                                      const float* weight, const float* mean, const float* rstd,
                                      void* dx, float* dw, float* db, void* workspace,
                                      int64_t workspace_bytes, void* stream);

/* Static text for a status code; never NULL. */
const char* mxfp4_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* MXFP4_H */

/*
 * serq.h -- C ABI of libserq, the SERQ quantized linear layer for MI355X (gfx950).
 *
 * SERQ ("SERQ: Saliency-Aware Low-Rank Error Reconstruction for LLM
 * Quantization") computes a linear layer Y = X W (X: M x K tokens by input
 * channels, W: K x N) as a pure 4-bit GEMM plus one small residual product:
 *
 *     Y  ~  Q(X^) Q(W^)  +  X~_{s,q} Q(R)
 *
 * where, after calibration,
 *   X~ = X diag(s^-1), W~ = diag(s) W          static per-channel flattening
 *   W^ = P W~ = [W~_s; W~_r], X^ = X~ P^-1     rows in descending saliency
 *   R  = W~_s - Q(W~_s)                        r x N compensator of the r
 *                                              most salient rows
 * and X~_{s,q} is the first r columns of the quantized activations.
 * Sources: papernotes.org ICLR 2026 notes on SERQ, sections 核心 idea,
 * 方法详解 / 整体框架 and 关键设计 1-3; gist.science/de/paper/2603.08185,
 * "Technische Zusammenfassung" 2.A-2.C.
 *
 * Conventions for every call
 *   - Sizes are element counts. Matrices are row-major and contiguous.
 *   - 4-bit codes are packed two per byte: byte t of a row holds code 2t in
 *     bits 0-3 and code 2t+1 in bits 4-7, each a 4-bit two's complement
 *     value in [-8, 7]. int8 codes are plain signed bytes.
 *   - Quantizer (weights, R, activations): symmetric, one scale per group,
 *     scale = fl32(m / qmax), code = clamp(rne(fl32(v * fl32(qmax / m)))),
 *     m the group's absolute maximum, qmax 7 (int4) or 127 (int8), rne round
 *     half to even. A group whose fl32(qmax / m) overflows (an all-zero group
 *     in particular) gets scale 0 and zero codes.
 *   - The caller owns every input and output. The library creates no
 *     streams and allocates no memory; the only device memory it holds is
 *     scratch for two paths (serq_linear's K split, chunked activation
 *     quantization) in file-scope device arrays, described at those calls:
 *     calls that take them must not overlap on one device. The attention
 *     calls take a workspace from the caller instead.
 *   - Argument errors are detected on the host and returned before anything
 *     is launched; the output buffers are then untouched.
 *   - Online calls only enqueue work on `stream` (a hipStream_t; NULL is the
 *     null stream) and return without synchronizing. A launch failure
 *     returns SERQ_EHIP.
 */
#ifndef SERQ_H_
#define SERQ_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  SERQ_OK = 0,
  SERQ_EINVAL = -1,       /* bad size, NULL pointer, bad enum value           */
  SERQ_EALIGN = -2,       /* a device pointer is not 16-byte aligned          */
  SERQ_EUNSUPPORTED = -3, /* valid request the library does not implement    */
  SERQ_EHIP = -4          /* the HIP runtime reported an error at launch      */
} serq_status;

typedef enum { SERQ_F32 = 0, SERQ_BF16 = 1 } serq_dtype;

/* Human-readable name of a status code (static string, never NULL). */
const char* serq_strerror(int status);

/* Version of the ABI described by this header (major * 100 + minor). */
int serq_abi_version(void);

/* Bytes per row of the packed Q(R) buffer for r salient rows: r codes
 * padded with zero codes to a multiple of 32 (16 bytes). */
#define SERQ_RQ_ROW_BYTES(r) ((((r) + 31) / 32) * 16)

/* SERQ_RQ_ROW_BYTES as a function (for bindings that cannot use macros);
 * returns -1 for r < 0. */
int serq_rq_row_bytes(int r);

/*
 * serq_calibrate -- offline, host memory, synchronous, deterministic.
 *
 * Follows the calibration phase of the pages (papernotes.org SERQ notes,
 * 方法详解 / 整体框架: calibration fixes the scale factors, the salient rows
 * and the permutation; 关键设计 1: SmoothQuant-style static per-channel s;
 * 关键设计 2: salient rows identified by their scale, rows permuted in
 * descending saliency, compensator R on the first r rows, R itself
 * quantized; 核心 idea: R = W~_s - Q(W~_s)).
 *
 *   W          K x N, dtype w_dtype (SERQ_F32 or SERQ_BF16), Y = X W.
 *   act_absmax K floats: max over the calibration tokens of |X[t, j]|.
 *   alpha      smoothing exponent in [0, 1]:
 *              s_j = fl32( max(a_j,1e-5)^alpha / max(w_j,1e-5)^(1-alpha) ),
 *              a_j = act_absmax[j], w_j = max_n |W[j, n]|, evaluated in
 *              double (for alpha = 0.5 exactly sqrt(a)/sqrt(w)).
 *   r          number of salient rows, 0 <= r <= K, r even.
 * Outputs (caller-allocated host buffers):
 *   perm       K int32: perm[i] = original channel placed at position i,
 *              descending s, equal s keep ascending channel order.
 *   s_hat_inv  K floats: fl32(1 / s[perm[i]]), the activation multiplier
 *              in saliency order.
 *   Wq         N x K/2 bytes: column n of Q(W^) as packed int4 along K
 *              (N-major), W^[i, n] = fl32(s[perm[i]] * W[perm[i], n]).
 *   sw         N floats: per-output-channel weight scale.
 *   Rq         N x SERQ_RQ_ROW_BYTES(r) bytes: column n of Q(R) packed
 *              along r, where R[i, n] = fl32(W^[i, n] - fl32(Wq[n, i] * sw[n])),
 *              i < r; each row is padded with zero codes to a multiple of 32
 *              codes (16 bytes), so rows stay 16-byte aligned.
 *              May be NULL when r == 0.
 *   sr         N floats: per-output-channel scale of R (all 0 when r == 0).
 *              May be NULL when r == 0.
 * Errors: SERQ_EINVAL for NULL inputs/outputs, K or N <= 0, odd K, odd r,
 * r outside [0, K], alpha outside [0, 1], unknown w_dtype.
 */
int serq_calibrate(const void* W, serq_dtype w_dtype, int K, int N,
                   const float* act_absmax, float alpha, int r,
                   int32_t* perm, float* s_hat_inv,
                   uint8_t* Wq, float* sw, uint8_t* Rq, float* sr);

/*
 * serq_calibrate_gptq -- offline, host memory, synchronous, deterministic.
 *
 * serq_calibrate with GPTQ codes for the weights (SERQ(GPTQ); the method
 * works with RTN and with GPTQ: gist.science/de/paper/2603.08185,
 * "Technische Zusammenfassung" 3; the pages' accuracy rows use it:
 * papernotes.org SERQ notes, 实验关键数据). GPTQ (Frantar et al., ICLR 2023)
 * quantizes the rows of W^ one at a time in the saliency order and moves
 * each row's error onto the rows not yet quantized, weighted by the upper
 * Cholesky factor U of H^-1, H = X^^T X^ over calibration inputs. Same
 * arguments and outputs as serq_calibrate, plus:
 *   X_cal      T x K calibration activations in the original channel order,
 *              dtype x_dtype (SERQ_F32 or SERQ_BF16); the Hessian is taken
 *              over the inputs the layer sees, x^ = fl32(X_cal[t, perm[i]] *
 *              s_hat_inv[i]), summed over t in order in double.
 *   T          calibration tokens, T > 0.
 *   damp       dampening: damp * mean(diag H) is added to the diagonal
 *              (0.01 in GPTQ); an all-zero H is replaced by the identity.
 * The r salient rows lead the order and their error is left to the
 * compensator, so their codes, R, Q(R) and every scale equal
 * serq_calibrate's; rows r..K-1 get GPTQ codes on the same per-column grid
 * (scale from the column maximum of W^, codes clamped to [-8, 7]). Every
 * step is one double operation in a fixed order, so the result does not
 * depend on the number of host threads. Cost ~ K^3 / 3 + K^2 (T + N) / 2
 * multiply-adds and 8 (3 K^2 + K N) bytes of host memory.
 * Errors: as serq_calibrate, plus SERQ_EINVAL for NULL X_cal, T <= 0, bad
 * x_dtype, damp negative or not finite, and for a Hessian that is not
 * positive definite (possible only with damp == 0; the outputs then hold
 * serq_calibrate's results).
 */
int serq_calibrate_gptq(const void* W, serq_dtype w_dtype, int K, int N,
                        const float* act_absmax, float alpha, int r,
                        const void* X_cal, serq_dtype x_dtype, int T, float damp,
                        int32_t* perm, float* s_hat_inv,
                        uint8_t* Wq, float* sw, uint8_t* Rq, float* sr);

/*
 * serq_permute_outputs -- offline, host memory, in place.
 *
 * Pushes the next layer's input order into this layer's output channels so
 * that its output already arrives in that order and no layer reorders at run
 * time (papernotes.org SERQ notes, 关键设计 3: the down projection's order P4
 * is propagated into the gate/up weight columns; gist.science/de
 * "Technische Zusammenfassung" 2.C).
 *
 *   perm_next  N int32, a permutation of 0..N-1: new output channel i is old
 *              channel perm_next[i].
 *   K, N, r    this layer's sizes, in serq_calibrate's order (K inputs, N
 *              outputs, r salient rows).
 *   Wq (N x K/2 bytes), sw (N), Rq (N x SERQ_RQ_ROW_BYTES(r)), sr (N) are
 *   reordered in place. Rq and sr may be NULL when r == 0.
 * Errors: SERQ_EINVAL for NULL pointers, bad sizes, or perm_next not a
 * permutation (detected before anything is modified).
 */
int serq_permute_outputs(const int32_t* perm_next, int K, int N, int r,
                         uint8_t* Wq, float* sw, uint8_t* Rq, float* sr);

/*
 * serq_quant_act -- online, device memory, asynchronous on `stream`.
 *
 * Per-token symmetric quantization of the flattened activations
 * (papernotes.org SERQ notes, 方法详解 / 整体框架: the main path runs on
 * Q(X^); output node "W4A4/W4A8"). X arrives already in saliency order
 * (关键设计 3), so no gather is done: x^[m, k] = fl32(X[m, k] * s_hat_inv[k]),
 * then one scale per row over all K columns.
 *
 *   X          M x K, dtype x_dtype (SERQ_F32 or SERQ_BF16), device.
 *   s_hat_inv  K floats, device (from serq_calibrate).
 *   a_bits     4 (W4A4) or 8 (W4A8).
 *   Xq         device, M x K/2 bytes (a_bits 4, packed) or M x K int8.
 *   sx         device, M floats: per-token scale.
 * Scratch: up to 64 rows with K > 8192 are cut into chunks over two
 * launches whose chunk maxima meet in a 32 KB device array the library holds
 * per device (no allocation call); such calls on one device must not overlap.
 * M == 0 is a no-op; X, Xq and sx may then be NULL. Errors: SERQ_EINVAL
 * (NULL pointer, M < 0, K <= 0, odd K, bad a_bits or dtype), SERQ_EALIGN
 * (pointer not 16-byte aligned), SERQ_EHIP.
 */
int serq_quant_act(const void* X, serq_dtype x_dtype, int M, int K,
                   const float* s_hat_inv, int a_bits,
                   void* Xq, float* sx, void* stream);

/*
 * serq_silu_mul_quant_act -- online, device memory, asynchronous on `stream`.
 *
 * The MLP step between gate/up and down, fused with down's activation
 * quantization: h = silu(g) * u elementwise, then exactly serq_quant_act on
 * h (per token: x^ = h * s_hat_inv, absmax, codes, sx). The gate and up
 * outputs arrive already in down's saliency order, the permutation having
 * been pushed into their output channels offline with serq_permute_outputs
 * (papernotes.org SERQ notes, 关键设计 3), so no gather is needed. The pages
 * do not spell out the nonlinearity; silu(g) = g / (1 + e^-g) as in the
 * LLaMA MLP, evaluated by a fixed fp32 recipe so results are reproducible
 * bit for bit: e = exp(-g) with the argument clamped to [-80, 80], by
 * Cody-Waite reduction (e^x = 2^n e^r, n = rne(x log2 e), ln 2 split in a
 * head c_hi = 22713 * 2^-15 of 15 significant bits, so n c_hi is exact for
 * |n| <= 116, and a tail; r by two fused multiply-adds) and the degree-7
 * Taylor polynomial of e^r (Horner, one fused multiply-add per degree); then
 * fl32(fl32(g / fl32(1 + e)) * u) with IEEE division and no other fused op.
 *
 *   G, U       device, row m of gate at G + m * ld, of up at U + m * ld, K
 *              elements each, of x_dtype (a gate/up output stored as one
 *              M x 2K buffer is G = Y, U = Y + K, ld = 2K).
 *   ld         row stride in elements, ld >= K. G and U need only be
 *              aligned to their element; rows that are all 16-byte aligned
 *              (and K % 8 == 0) take the vector path, others a scalar one
 *              with the same results.
 *   s_hat_inv  K floats, device (down's, from serq_calibrate).
 *   a_bits, Xq, sx as for serq_quant_act (so is the scratch rule, here for
 *              up to 64 rows with K > 4096, or 128 with K > 16384).
 * M == 0 is a no-op. Errors: SERQ_EINVAL (NULL pointer, M < 0, K <= 0, odd
 * K, ld < K, bad a_bits or dtype), SERQ_EALIGN (G or U not aligned to its
 * element, Xq or sx not 16-byte aligned), SERQ_EHIP. Subnormal inputs are
 * outside the contract.
 */
int serq_silu_mul_quant_act(const void* G, const void* U, int ld, serq_dtype x_dtype,
                            int M, int K, const float* s_hat_inv, int a_bits,
                            void* Xq, float* sx, void* stream);

/*
 * serq_linear -- online, device memory, asynchronous on `stream`.
 *
 * The SERQ linear: acc_main = Xq . Q(W^) over all K, acc_res = Xq[:, :r] . Q(R)
 * over the r salient channels, reusing the same activation codes (no second
 * quantization; papernotes.org SERQ notes, 关键设计 2: the residual is one
 * (tokens x r)(r x d) product on the salient activation channels, R is
 * quantized, no intermediate quantization), and
 *     Y[m, n] = sx[m] * (sw[n] * acc_main[m, n] + sr[n] * acc_res[m, n])
 * evaluated in fp32 and stored as y_dtype (bf16 with round to nearest even).
 * Integer accumulation is exact (int32) for every K the call accepts (the
 * matrix-core kernels serve K < 2^17, longer rows a plain kernel).
 *
 *   Xq, sx     from serq_quant_act with the same a_bits (device).
 *   Wq, sw     N x K/2 bytes and N floats (device).
 *   Rq, sr     N x SERQ_RQ_ROW_BYTES(r) bytes (the layout serq_calibrate
 *              writes, zero codes in the padding) and N floats (device);
 *              may be NULL when r == 0.
 *   M, K, N, r sizes; 0 <= r <= K, r even, K even. M == 0 is a no-op (the
 *              M-sized buffers Xq, sx, Y and the debug buffers may then be
 *              NULL; the weights are still validated).
 *   Y          device, M x N of y_dtype.
 *   acc_main_dbg, acc_res_dbg
 *              NULL on the hot path; when non-NULL, device M x N int32
 *              buffers that receive the exact integer accumulators (both
 *              must then be given).
 * No allocation, no synchronization: the call only enqueues kernels, so it
 * may be captured into a HIP graph, the first call on a device included.
 * Scratch: for 4..32 tokens whose activation rows exceed the kernel's LDS
 * budget (long K), the K range is split across workgroups whose int32
 * partial sums meet in file-scope device arrays of the library (16 MiB of
 * partial sums and 64 KiB of counters per device, held from the moment the
 * library's code is loaded on the device until the process ends). Sizes
 * whose split would need more take a kernel without a split, so no size is
 * refused for it. Calls that take the split path on one device share the
 * arrays, so they must not overlap in time (e.g. on two streams at once).
 * Errors: SERQ_EINVAL (NULL pointer, bad sizes, bad a_bits or dtype, only one
 * debug buffer), SERQ_EALIGN (pointer not 16-byte aligned), SERQ_EHIP.
 */
int serq_linear(const void* Xq, const float* sx, int a_bits,
                const uint8_t* Wq, const float* sw,
                const uint8_t* Rq, const float* sr,
                int M, int K, int N, int r,
                void* Y, serq_dtype y_dtype,
                int32_t* acc_main_dbg, int32_t* acc_res_dbg,
                void* stream);

/*
 * serq_linear_kernel_name -- which kernel serq_linear would launch for these
 * sizes (static string: "gemv", "decode16", "decode32_ksplit" (the K split
 * with scratch), "tile128x128", ..., "generic"), or NULL for invalid sizes.
 * Host only; launches nothing. For profiling and tests.
 */
const char* serq_linear_kernel_name(int M, int K, int N, int r, int a_bits);

/*
 * The same linear on gfx950's scaled FP6 matrix instruction (bf6 route).
 *
 * The pages run SERQ on integer or microscaling-FP4 matrix hardware alike
 * (gist.science/de/paper/2603.08185, "3. Wichtige Beiträge": the method is
 * compatible with INT4 and MXFP4 formats; "4. Ergebnisse", Performance &
 * Latenz: the fast path is the hardware FP4 product, the residual adding
 * about 1 %). CDNA4 has no int4 matrix instruction, but every int4 code in
 * [-8, 7] is exactly a bf6 (E3M2) value, and a product of two such codes
 * summed in fp32 stays an exact integer while |sum| <= 2^24, i.e. for K up to
 * 2^18. So this route computes bit for bit the accumulators of serq_linear
 * (W4A4 only) at the FP6 instruction rate, on operands re-encoded as bf6:
 *
 * bf6 tile layout of a matrix of `rows` x `k` int4 codes. Rows are padded
 * with zero codes to a multiple of 128 (Rp) and k to a multiple of 128 (Kp).
 * The buffer is a sequence of 3072-byte fragment blocks, block (kt, rb) at
 * byte ((kt * Rp / 32) + rb) * 3072 for k-tile kt (codes [128 kt, +128)) and
 * 32-row block rb; inside a block, step s (0, 1) at +1536 s and lane l
 * (0..63) at +24 l hold the 32 codes of row 32 rb + l % 32 at
 * k = 128 kt + 64 s + 32 (l / 32) + f, f = 0..31, each as the 6-bit E3M2
 * pattern (sign bit 5, exponent bits 4..2 with bias 3, mantissa bits 1..0)
 * in bits [6 f, 6 f + 6) of the 24 bytes read as one little-endian 192-bit
 * integer. Code -> pattern: 0 -> 0x00, 1 -> 0x0C, 2 -> 0x10, 3 -> 0x12,
 * 4 -> 0x14, 5 -> 0x15, 6 -> 0x16, 7 -> 0x17, and -v -> 0x20 | pattern(v),
 * -8 -> 0x38. Size: SERQ_BF6_BYTES(rows, k) bytes.
 */
#define SERQ_BF6_BYTES(rows, k) ((size_t)(((k) + 127) / 128) * (size_t)(((rows) + 127) / 128) * 12288u)

/* SERQ_BF6_BYTES as a function; returns -1 for rows < 0 or k < 0. */
int64_t serq_bf6_bytes(int rows, int k);

/*
 * serq_prepack_bf6 -- offline, host memory, synchronous.
 *
 * Re-encodes a packed int4 matrix (serq_calibrate's Q(W^) with k = K and
 * pitch = K/2, or Q(R) with k = r and pitch = SERQ_RQ_ROW_BYTES(r)) into the
 * bf6 tile layout, writing every byte of `out` (padding included).
 *   codes  rows x pitch bytes, canonical nibble order (host).
 *   rows, k, pitch  rows > 0, 0 < k <= 2 * pitch, k even.
 *   out    SERQ_BF6_BYTES(rows, k) bytes (host), caller-owned.
 * Errors: SERQ_EINVAL (NULL pointer, bad sizes).
 */
int serq_prepack_bf6(const uint8_t* codes, int rows, int k, int pitch, uint8_t* out);

/*
 * serq_act_bf6 -- online, device memory, asynchronous on `stream`.
 *
 * Re-encodes W4A4 activation codes (serq_quant_act's Xq, M x K/2 bytes) into
 * the bf6 tile layout, padding included, for serq_linear_bf6. The token
 * scales sx are used as they are.
 *   Xq   device, M x K/2 bytes, 16-byte aligned.
 *   M, K M >= 0 (0: no-op), K > 0 even, K <= 262144.
 *   X6   device, SERQ_BF6_BYTES(M, K) bytes, 16-byte aligned.
 * Errors: SERQ_EINVAL, SERQ_EALIGN, SERQ_EHIP.
 */
int serq_act_bf6(const void* Xq, int M, int K, void* X6, void* stream);

/*
 * serq_linear_bf6 -- online, device memory, asynchronous on `stream`.
 *
 * serq_linear (W4A4) on bf6 operands: the same acc_main, acc_res (exact
 * integers) and the same fp32 epilogue, so Y and the debug accumulators are
 * bit-identical to serq_linear's on the same codes.
 *   X6         SERQ_BF6_BYTES(M, K) bytes from serq_act_bf6 (device).
 *   sx         M floats from serq_quant_act (device).
 *   W6, sw     SERQ_BF6_BYTES(N, K) bytes from serq_prepack_bf6 of Q(W^),
 *              and N floats (device).
 *   R6, sr     SERQ_BF6_BYTES(N, r) bytes from serq_prepack_bf6 of Q(R),
 *              and N floats (device); may be NULL when r == 0.
 *   M, K, N, r M >= 0 (0: no-op), K > 0 even, K <= 262144, N > 0,
 *              0 <= r <= min(K, 256), r even.
 *   Y, y_dtype, acc_main_dbg, acc_res_dbg  as for serq_linear.
 * Uses no scratch memory. Errors: SERQ_EINVAL (NULL pointer, bad sizes or
 * dtype, only one debug buffer), SERQ_EALIGN (pointer not 16-byte aligned),
 * SERQ_EHIP.
 */
int serq_linear_bf6(const void* X6, const float* sx,
                    const uint8_t* W6, const float* sw,
                    const uint8_t* R6, const float* sr,
                    int M, int K, int N, int r,
                    void* Y, serq_dtype y_dtype,
                    int32_t* acc_main_dbg, int32_t* acc_res_dbg,
                    void* stream);

/*
 * serq_linear_bf6_kernel_name -- which tile serq_linear_bf6 launches for M
 * tokens, N outputs and r salient rows (static string "bf6_tile128x128" or
 * "bf6_tile256x256"), or NULL for M <= 0, N <= 0 or r < 0. Host only;
 * launches nothing. For profiling and tests.
 */
const char* serq_linear_bf6_kernel_name(int M, int N, int r);

/*
 * The MXFP4 variant of the layer.
 *
 * The pages run SERQ on MXFP4 as well as INT4 (gist.science/de/paper/
 * 2603.08185, "Technische Zusammenfassung" 3: compatible with INT4 and
 * MXFP4; 4, Performance & Latenz: measured on hardware FP4 products, the
 * residual adding about 1 %). The format is OCP Microscaling (MX): blocks of
 * 32 consecutive elements along K share an E8M0 exponent e (stored as the
 * byte e + 127; the scale is 2^e), e = floor(log2(max |v|)) - 2 clamped to
 * [-127, 127] (-127 for an all-zero block); each element is the FP4 E2M1
 * value (sign bit 3, exponent bits 2-1 with bias 1, mantissa bit 0:
 * magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6) nearest to v / 2^e, ties to the
 * even mantissa, saturated at 6; a value that rounds to zero is code 0.
 * Codes are packed two per byte, element 2t in the low nibble. In the layer
 * the blocks run along K: per output column of W^, per token row of the
 * activations, per output column of R over its r rows (K and r multiples of
 * 32). s, P and W^ are those of serq_calibrate; R = W~_s - Q(W~_s) with the
 * MX quantizer's own dequantized salient rows, in fp32; Q(R) in MXFP4. The
 * block exponents are the only scales:
 *   Y[m, n] = sum over blocks b of 2^(ex_mb + ew_nb) sum_{k in b} x_mk w_nk
 *           + sum over the first r/32 blocks of 2^(ex_mb + er_nb) sum x_mk rho_nk.
 */

/*
 * serq_calibrate_mx -- offline, host memory, synchronous, deterministic.
 * As serq_calibrate, with MXFP4 outputs:
 *   Wq   N x K/2 bytes: column n of Q(W^), FP4 codes along K.
 *   Wsc  N x K/32 bytes: E8M0 exponent bytes of those blocks.
 *   Rq   N x r/2 bytes, Rsc N x r/32 bytes: Q(R) likewise (NULL when r == 0).
 * Errors: SERQ_EINVAL for NULL pointers, K or N <= 0, K or r not a multiple
 * of 32, r outside [0, K], alpha outside [0, 1], unknown w_dtype.
 */
int serq_calibrate_mx(const void* W, serq_dtype w_dtype, int K, int N,
                      const float* act_absmax, float alpha, int r,
                      int32_t* perm, float* s_hat_inv,
                      uint8_t* Wq, uint8_t* Wsc, uint8_t* Rq, uint8_t* Rsc);

/*
 * serq_quant_act_mx -- online, device memory, asynchronous on `stream`.
 * x^ = fl32(X[m, k] * s_hat_inv[k]) (X already in saliency order), then
 * MXFP4 per token row in blocks of 32 along K.
 *   X      M x K, SERQ_F32 or SERQ_BF16; K a multiple of 32.
 *   Xq     M x K/2 bytes of FP4 codes; Xsc M x K/32 exponent bytes.
 * M == 0 is a no-op. Errors: SERQ_EINVAL (NULL pointer, M < 0, K not a
 * positive multiple of 32, bad dtype), SERQ_EALIGN (X, Xq or s_hat_inv not
 * 16-byte aligned), SERQ_EHIP. Uses no scratch memory.
 */
int serq_quant_act_mx(const void* X, serq_dtype x_dtype, int M, int K,
                      const float* s_hat_inv, uint8_t* Xq, uint8_t* Xsc, void* stream);

/*
 * serq_linear_mx -- online, device memory, asynchronous on `stream`.
 * Y = acc_main + acc_res (the formula above) on gfx950's scaled FP4 matrix
 * instructions, whose operands are these codes and exponent bytes as
 * stored; one token (two when N < 16384) takes a dot-product kernel instead
 * (each 32-element block summed exactly, then scaled and added). Either way
 * accumulation is fp32 with one rounding per block (rounded, unlike the
 * integer layer) plus a fixed-order sum of partial sums; Y is stored as
 * y_dtype (bf16 with round to nearest even).
 *   Xq, Xsc    from serq_quant_act_mx; Wq, Wsc, Rq, Rsc from
 *              serq_calibrate_mx (Rq, Rsc may be NULL when r == 0).
 *   M, K, N, r M >= 0 (0: no-op), K > 0 and 0 <= r <= K multiples of 32,
 *              N > 0.
 *   acc_main_dbg, acc_res_dbg  NULL, or both device M x N floats that
 *              receive the two fp32 accumulators.
 * Uses no scratch memory. Errors: SERQ_EINVAL, SERQ_EALIGN (Xq, Wq, Rq, Y or
 * the debug buffers not 16-byte aligned), SERQ_EHIP.
 */
int serq_linear_mx(const uint8_t* Xq, const uint8_t* Xsc,
                   const uint8_t* Wq, const uint8_t* Wsc,
                   const uint8_t* Rq, const uint8_t* Rsc,
                   int M, int K, int N, int r,
                   void* Y, serq_dtype y_dtype,
                   float* acc_main_dbg, float* acc_res_dbg,
                   void* stream);

/*
 * The linear in 8-bit integers: for the layers that keep 8 bits where others
 * take 4 (down projections, output heads),
 *     Y[m, n] = sx[m] * (sw[n] * sum_k Xq[m, k] Wq[n, k]),
 * a scale for each token and each channel, no compensator and no permutation.
 *
 * serq_calibrate_i8 -- offline, host memory, synchronous, deterministic.
 *   W, w_dtype, alpha  as for serq_calibrate; act_absmax as there, or NULL for
 *              no smoothing (s_j = 1).
 * Outputs: s_hat_inv, K floats fl32(1 / s_j) in channel order, for
 * serq_quant_act and serq_silu_mul_quant_act with a_bits 8; Wq, N x K int8,
 * row n the codes of fl32(s_j W[j, n]) (qmax 127); sw, N floats.
 * Errors: SERQ_EINVAL (NULL W or output, K or N <= 0, alpha outside [0, 1],
 * bad w_dtype), SERQ_EUNSUPPORTED (no host memory for K floats).
 */
int serq_calibrate_i8(const void* W, serq_dtype w_dtype, int K, int N, const float* act_absmax, float alpha,
                      float* s_hat_inv, int8_t* Wq, float* sw);

/*
 * serq_linear_i8 -- online, device memory, asynchronous on `stream`. The sums
 * are exact (int32); the formula's products are fp32, in its order, and Y is
 * stored as y_dtype (bf16 with round to nearest even).
 *   Xq, sx     M x K int8 and M floats (serq_quant_act, a_bits 8).
 *   Wq, sw     N x K int8 and N floats (serq_calibrate_i8).
 *   M, K, N    M >= 0 (0: no-op, the M-sized buffers may then be NULL), 0 < K
 *              < 2^17, 0 < N <= 2^26, M N <= 2^37. K that is no multiple of
 *              16 takes a plain kernel.
 *   Y          M x N of y_dtype.
 *   acc_dbg    NULL, or device M x N int32 that receive the sums.
 *   workspace  serq_linear_i8_workspace(M, K, N) bytes, 16-byte aligned, or NULL
 *              if that is 0 (K is cut in parts where there are few outputs).
 *              Its contents need no preparation and are free again when the
 *              call's work is done; calls that may overlap need one each.
 * Errors: SERQ_EINVAL (NULL pointer, sizes, y_dtype, workspace too small),
 * SERQ_EALIGN (a pointer not 16-byte aligned), SERQ_EHIP.
 */
int serq_linear_i8(const int8_t* Xq, const float* sx, const int8_t* Wq, const float* sw, int M, int K, int N,
                   void* Y, serq_dtype y_dtype, int32_t* acc_dbg, void* workspace, int64_t workspace_bytes,
                   void* stream);

/* Bytes of workspace serq_linear_i8 needs for these sizes (may be 0), or -1 for
 * invalid ones. Host only. */
int64_t serq_linear_i8_workspace(int M, int K, int N);

/* Which kernel serq_linear_i8 launches for these sizes (static string:
 * "stream", "tile64x64", "tile64x128", "tile128x128", "tile256x128",
 * "tile256x256" or "generic"), or NULL for invalid sizes. Host only. */
const char* serq_linear_i8_kernel_name(int M, int K, int N);

/*
 * The attention half of a decoder layer, between the q/k/v linear and the
 * output linear: rotating and storing keys, causal attention of new tokens,
 * and single-token attention of a batch that may share a prefix.
 *
 * The paged cache. Keys and values of all sequences live in two device
 * buffers of n_pages pages each, a page holding page_size tokens of every
 * key/value head:
 *     Kc[page][kv head][token in page][D],  Vc likewise,
 * of one dtype (the calls' `dtype`: SERQ_F32 or SERQ_BF16). page_size is a
 * power of two from 16 to 1024. A slot is page * page_size + token in page.
 * A sequence is a row of page ids in order: its token t lies in page
 * row[t / page_size] at t % page_size. What lies in a page past a sequence's
 * length is never used (it may hold NaN). Page ids outside [0, n_pages) read
 * some page inside the cache: wrong values, no access outside.
 *
 * Heads. Hq query heads share Hkv key/value heads (Hq a multiple of Hkv);
 * query head h reads key/value head h / (Hq / Hkv). D is 64 or 128 (others
 * SERQ_EUNSUPPORTED). Bounds: 16384 heads, rows * Hq of the two attentions
 * and the keys of a sequence at most 2^30, n_pages * page_size below 2^31.
 */

typedef enum { SERQ_ROPE_HALF = 0, SERQ_ROPE_INTERLEAVED = 1 } serq_rope_layout;
typedef enum {
  SERQ_ROPE_PLAIN = 0,  /* f_i                                              */
  SERQ_ROPE_LINEAR = 1, /* f_i / factor: positions interpolated             */
  SERQ_ROPE_BASE = 2,   /* theta * factor^(rot / (rot - 2)) in place of theta */
  SERQ_ROPE_BANDS = 3   /* low frequencies interpolated, high ones kept     */
} serq_rope_scaling;

/*
 * serq_rope_table -- offline, host memory, synchronous.
 *
 * Cosines and sines of the rotary position embedding (Su et al. 2021): for
 * position p and pair i < rot_dim / 2 the angle p * f_i, f_i =
 * theta^(-2 i / rot_dim), in double, rounded once. For contexts longer than
 * the trained one the frequencies are scaled: SERQ_ROPE_LINEAR (position
 * interpolation, Chen et al. 2023), SERQ_ROPE_BASE (a larger base), or
 * SERQ_ROPE_BANDS (by parts, Peng et al. 2023): with n_i = orig_len f_i / 2 pi
 * turns over the trained length and g = clamp((n_i - low) / (high - low), 0,
 * 1) the frequency is (1 - g) f_i / factor + g f_i. Every entry is multiplied
 * by mscale (1, or that method's temperature 0.1 ln(factor) + 1).
 *   rot_dim  even, 2..65536;  max_pos >= 1;  theta > 0;  factor >= 1;
 *            orig_len >= 1 and low < high for SERQ_ROPE_BANDS.
 *   table    max_pos x rot_dim floats: row p holds its rot_dim / 2 cosines,
 *            then its sines.
 * Errors: SERQ_EINVAL (NULL table, a value outside these ranges or not
 * finite; rot_dim 2 with SERQ_ROPE_BASE).
 */
int serq_rope_table(int rot_dim, int max_pos, double theta, serq_rope_scaling scaling,
                    double factor, int orig_len, double low, double high, double mscale,
                    float* table);

/*
 * serq_rope_append -- online, device memory, asynchronous on `stream`.
 *
 * From the q/k/v linear's output to queries and a filled cache in one pass:
 * for token t, every query and key head x (D values) becomes
 *     y = x * w / sqrt(mean(x^2) + eps)          (only where w is given)
 *     (y_a, y_b) -> (y_a c - y_b s, y_b c + y_a s)
 * over the pairs of its first rot_dim values, c and s from row pos[t] of the
 * table: pair i is (i, i + rot_dim / 2) for SERQ_ROPE_HALF and (2 i, 2 i + 1)
 * for SERQ_ROPE_INTERLEAVED; values from rot_dim on are not rotated. All in
 * fp32, rounded once at the end. Keys and the unchanged values then go to
 * slot[t] of the cache.
 *   QKV      M rows of Hq + 2 Hkv heads of D (queries, keys, values), row t
 *            at QKV + t * ld elements, ld >= (Hq + 2 Hkv) D. It need only be
 *            aligned to its element; rows that are all 16-byte aligned take
 *            the vector path, others a scalar one.
 *   q_norm, k_norm  D floats each, or NULL for no norm of that kind.
 *   table    max_pos x rot_dim floats (serq_rope_table); rot_dim even,
 *            0 <= rot_dim <= D; NULL when rot_dim == 0.
 *   pos      M int32. A token whose position is outside [0, max_pos) gets
 *            NaN queries and is not stored (rot_dim > 0 only).
 *   slot     M int32, distinct where they are stored. A token whose slot is
 *            outside [0, n_pages * page_size) gets its queries but is not
 *            stored (-1: padding).
 *   Q        device, M x Hq x D, row stride ldq >= Hq D elements; must not
 *            overlap QKV unless it is its query part (Q == QKV, ldq == ld).
 * M == 0 is a no-op (QKV, pos, slot and Q may then be NULL). Hq may be 0 (Q
 * is then not used). Errors: SERQ_EINVAL (NULL pointer, bad size, eps
 * negative or not finite), SERQ_EUNSUPPORTED (D or page_size),
 * SERQ_EALIGN (QKV or Q not aligned to its element, Kc, Vc, the table or a
 * norm not 16-byte aligned), SERQ_EHIP. Uses no scratch memory.
 */
int serq_rope_append(const void* QKV, serq_dtype dtype, int64_t ld, int M, int Hq, int Hkv, int D,
                     const float* q_norm, const float* k_norm, float eps,
                     const float* table, int rot_dim, int max_pos, serq_rope_layout layout,
                     const int32_t* pos, const int32_t* slot,
                     void* Q, int64_t ldq, void* Kc, void* Vc, int n_pages, int page_size,
                     void* stream);

/*
 * serq_rope_append_axes -- serq_rope_append for tokens with a position on each
 * of several axes (time, height and width of a picture's or clip's patches):
 * pair i of a head is rotated by the position on axis pair_axis[i], by the
 * table's row for that position as before.
 *   n_axes     1 to 4.
 *   pair_axis  host, rot_dim / 2 bytes, each below n_axes; read during the
 *              call. May be NULL when n_axes is 1.
 *   pos        n_axes rows of M int32 (axis a of token t at a * M + t). A
 *              token with a position outside [0, max_pos) on any axis gets NaN
 *              queries and is not stored.
 * All else, errors included, as for serq_rope_append; SERQ_EINVAL for n_axes
 * or an axis outside these ranges.
 */
int serq_rope_append_axes(const void* QKV, serq_dtype dtype, int64_t ld, int M, int Hq, int Hkv, int D,
                          const float* q_norm, const float* k_norm, float eps,
                          const float* table, int rot_dim, int max_pos, serq_rope_layout layout,
                          int n_axes, const uint8_t* pair_axis, const int32_t* pos, const int32_t* slot,
                          void* Q, int64_t ldq, void* Kc, void* Vc, int n_pages, int page_size,
                          void* stream);

/*
 * The paged cache in 8 bits. Kc and Vc hold FP8 codes (OCP E4M3, one byte a
 * value) in the layout above, and each block of 16 tokens of a page and head
 * has a power of two:
 *     k_scale[page][kv head][page_size / 16],  v_scale likewise,
 * bytes e + 127 (OCP E8M0) with -117 <= e <= 120. Both arrays are 4-byte aligned
 * and are read by words of 4 bytes: where their size is no multiple of 4, the
 * memory has to reach to the next one. (What lies there is not used, and never
 * written.)
 * A cache value is code * 2^e, which is a bf16 number; at e = 120 the codes from
 * 256 on, 2^128 and more, are infinities. Half the bytes of a bf16 cache and 1 in
 * 16 D more; a value has 4 significant bits, so it is off by at most 2^-4 of itself
 * (2^-10 * 2^e near 0), and one of 248 * 2^120 (3.297e38) or more in magnitude
 * becomes an infinity, as it would rounded to 4 bits.
 *
 * Storing a block's token 0 begins it anew: its scale then comes from what that
 * call stores in it, and the codes of its other tokens stay as they are, to be
 * stored after it. Later tokens may need a larger scale; the block's other
 * codes are then multiplied by 2^(old e - new e), exactly but for those that fall below
 * 2^-6 (rounded to the nearest multiple of 2^-9, ties to even). One call
 * stores a block's tokens from rows next to one another, in any order; where
 * rows of other blocks, or rows that are not stored, lie between them, that
 * block's values are unspecified.
 *
 * serq_rope_append_f8 -- serq_rope_append_axes onto such a cache. Keys are
 * computed in 64 bits (norm, products and sums) and rounded to fp32 once; then
 * with m the largest finite |y| of a block's new tokens (of one head, of keys or
 * of values)
 *     e = the least integer >= -117 with m <= 448 * 2^e, at least the block's
 *         e of before unless it is begun anew;
 *     code = y * 2^-e rounded to E4M3 (nearest, ties to even).
 * NaN and infinities become the code NaN and do not change the scale. Queries
 * as for serq_rope_append.
 *   dtype      of QKV and Q.
 *   Kc, Vc     n_pages * Hkv * page_size * D bytes each, 16-byte aligned.
 *   k_scale, v_scale  n_pages * Hkv * page_size / 16 bytes each, in memory that
 *              the attention calls can read to the next multiple of 4. Bytes
 *              outside 10..247 of a block that is not begun anew are taken as the
 *              nearest inside.
 * Errors as for serq_rope_append_axes, SERQ_EINVAL and SERQ_EALIGN (4 bytes)
 * for the scales too. Uses no scratch memory.
 */
int serq_rope_append_f8(const void* QKV, serq_dtype dtype, int64_t ld, int M, int Hq, int Hkv, int D,
                        const float* q_norm, const float* k_norm, float eps,
                        const float* table, int rot_dim, int max_pos, serq_rope_layout layout,
                        int n_axes, const uint8_t* pair_axis, const int32_t* pos, const int32_t* slot,
                        void* Q, int64_t ldq, uint8_t* Kc, uint8_t* Vc, uint8_t* k_scale, uint8_t* v_scale,
                        int n_pages, int page_size, void* stream);

/*
 * serq_attn_prefill -- online, device memory, asynchronous on `stream`.
 *
 * Causal attention of the new tokens of B sequences, packed one after
 * another, over the cache that already holds their keys and values: with
 * n_b = cu_q[b + 1] - cu_q[b] new tokens of sequence b and kv_len[b] tokens
 * in the cache (the new ones the last of them), new token i sees the keys
 * j <= kv_len[b] - n_b + i:
 *     O_i = sum_j softmax_j(scale q_i . k_j) v_j .
 * A token that sees no key (kv_len[b] < n_b) gets zeros, and so does one all
 * of whose scores are -inf. A key or value that a token does not see has no
 * influence on it, NaN and infinities included. Scores, softmax statistics
 * and sums are fp32; with SERQ_BF16 each softmax weight is rounded to bf16
 * for the product with the values. Weighted values are summed before they are
 * divided by the weights' sum, with weights of up to 2^8: a value's magnitude
 * times the keys it is summed with has to stay below 2^120.
 *   Q        T rows of Hq heads of D, row stride ldq >= Hq D elements; 16-byte
 *            aligned rows.
 *   cu_q     B + 1 int32, cu_q[0] = 0, not decreasing, cu_q[B] = T (values
 *            outside [0, T] are taken as the nearest inside; rows that no
 *            sequence holds are left untouched).
 *   page_table  B rows of max_pages page ids;  kv_len  B int32 (taken as at
 *            most min(max_len, max_pages * page_size)).
 *   max_len  bound of kv_len, known to the host; sizes the workspace and
 *            the split of the keys (parts of equal size up to max_len, so a
 *            bound far above the lengths leaves fewer parts with keys).
 *   O        T rows of Hq heads of D, row stride ldo >= Hq D, 16-byte
 *            aligned rows; must not overlap Q unless it is Q (same stride).
 *   workspace  serq_attn_prefill_workspace(...) bytes, 16-byte aligned, or
 *            NULL if that is 0. Its contents need no preparation and are
 *            free again when the call's work is done; calls that may overlap
 *            need one each.
 * One launch bounds the rows and sequences of a call further: (T / 256 + B) *
 * Hq below 2^23 with SERQ_BF16 and (T / 32 + B) * Hq below 2^24 with SERQ_F32
 * are always taken, and SERQ_EINVAL says where it is more than that.
 * T == 0 or B == 0 is a no-op. Errors: SERQ_EINVAL (NULL pointer, bad size,
 * scale not finite, workspace too small), SERQ_EUNSUPPORTED (D or
 * page_size), SERQ_EALIGN, SERQ_EHIP.
 */
int serq_attn_prefill(const void* Q, serq_dtype dtype, int64_t ldq, const int32_t* cu_q, int B, int T,
                      int Hq, int Hkv, int D, const void* Kc, const void* Vc, int n_pages, int page_size,
                      const int32_t* page_table, int max_pages, const int32_t* kv_len, int max_len,
                      float scale, void* O, int64_t ldo, void* workspace, int64_t workspace_bytes,
                      void* stream);

/* Bytes of workspace serq_attn_prefill needs for these sizes (may be 0), or
 * -1 for invalid ones. Host only. */
int64_t serq_attn_prefill_workspace(serq_dtype dtype, int B, int T, int Hq, int Hkv, int D, int max_len);

/*
 * serq_attn_decode -- online, device memory, asynchronous on `stream`.
 *
 * One new token of each of B sequences over the cache. The sequences may
 * share a prefix of prefix_len tokens, whose pages are given once; sequence
 * b then continues with kv_len[b] tokens of its own (the new one among
 * them), which begin in pages of its own whatever prefix_len is. Token b
 * attends to the prefix and to its own tokens:
 *     O_b = sum_j softmax_j(scale q_b . k_j) v_j .
 * The prefix is read once for all sequences: their queries form the rows of
 * one matrix product per key/value head. Both parts are cut along the keys,
 * and the parts are joined by their running maxima and sums, in a fixed
 * order. Zeros where there is no key at all; arithmetic as for
 * serq_attn_prefill.
 *   Q, O     B rows of Hq heads of D, strides and alignment as for
 *            serq_attn_prefill.
 *   prefix_table  ceil(prefix_len / page_size) page ids; NULL when
 *            prefix_len == 0.
 *   page_table  B rows of max_pages page ids (may be NULL when max_pages or
 *            max_len is 0: no sequence then has tokens of its own);
 *            kv_len  B int32, taken as at most min(max_len, max_pages *
 *            page_size), negative as 0.
 *   max_len  bound of kv_len, known to the host: sizes the workspace and the
 *            split of the keys, as for serq_attn_prefill.
 *   workspace  serq_attn_decode_workspace(...) bytes, as for
 *            serq_attn_prefill.
 * B == 0 is a no-op. Errors as for serq_attn_prefill.
 */
int serq_attn_decode(const void* Q, serq_dtype dtype, int64_t ldq, int B, int Hq, int Hkv, int D,
                     const void* Kc, const void* Vc, int n_pages, int page_size,
                     const int32_t* prefix_table, int prefix_len,
                     const int32_t* page_table, int max_pages, const int32_t* kv_len, int max_len,
                     float scale, void* O, int64_t ldo, void* workspace, int64_t workspace_bytes,
                     void* stream);

/* Bytes of workspace serq_attn_decode needs for these sizes (may be 0), or
 * -1 for invalid ones. Host only. */
int64_t serq_attn_decode_workspace(serq_dtype dtype, int B, int Hq, int Hkv, int D, int prefix_len,
                                   int max_len);

/*
 * serq_attn_prefill_f8, serq_attn_decode_f8 -- the same attentions over a cache
 * in 8 bits: keys and values are code * 2^e, exactly (bf16 numbers, or at e = 120
 * infinities), and everything else is as for serq_attn_prefill and
 * serq_attn_decode with `dtype` that of Q and O. A code NaN behaves as a NaN does
 * there, and those infinities as infinities. Scales of blocks that no token of a
 * sequence lies in are never used.
 * Errors as there; SERQ_EINVAL (NULL) and SERQ_EALIGN (not 4-byte aligned) for
 * the scales too. Their workspaces are sized by their own functions.
 */
int serq_attn_prefill_f8(const void* Q, serq_dtype dtype, int64_t ldq, const int32_t* cu_q, int B, int T,
                         int Hq, int Hkv, int D, const uint8_t* Kc, const uint8_t* Vc,
                         const uint8_t* k_scale, const uint8_t* v_scale, int n_pages, int page_size,
                         const int32_t* page_table, int max_pages, const int32_t* kv_len, int max_len,
                         float scale, void* O, int64_t ldo, void* workspace, int64_t workspace_bytes,
                         void* stream);
int64_t serq_attn_prefill_f8_workspace(serq_dtype dtype, int B, int T, int Hq, int Hkv, int D, int max_len);

int serq_attn_decode_f8(const void* Q, serq_dtype dtype, int64_t ldq, int B, int Hq, int Hkv, int D,
                        const uint8_t* Kc, const uint8_t* Vc, const uint8_t* k_scale, const uint8_t* v_scale,
                        int n_pages, int page_size, const int32_t* prefix_table, int prefix_len,
                        const int32_t* page_table, int max_pages, const int32_t* kv_len, int max_len,
                        float scale, void* O, int64_t ldo, void* workspace, int64_t workspace_bytes,
                        void* stream);
int64_t serq_attn_decode_f8_workspace(serq_dtype dtype, int B, int Hq, int Hkv, int D, int prefix_len,
                                      int max_len);

#ifdef __cplusplus
}
#endif

#endif /* SERQ_H_ */

/*
 * clef.h -- C ABI of the GB300 (sm_103a) W8A8 quantized projection library.
 *
 * The library computes the quantized decoder linear projections of a
 * Clef-style single-pass decision backbone: a per-token activation
 * quantizer (block-128 Walsh-Hadamard rotation, absmax scale, symmetric INT8
 * codes; FP8-e4m3 dynamic variant), W8A8 GEMMs whose epilogues fuse the
 * row x column scales, the bias and, for packed gate/up weights, the SwiGLU
 * product, and the runtime LoRA add.  For answering token by token it adds
 * linears over 4-bit weights, a paged 8-bit cache of keys and values, and the
 * attention that reads it; between the projections norms whose results are
 * already codes, rotary positions, and linears over e4m3 codes in blocks of 128.  Every step runs in hand-written CUDA kernels on
 * the caller's stream.
 *
 * Conventions shared by every entry point:
 *  - Pointers are DEVICE pointers to memory the caller owns (clef_copy_sm
 *    also takes page-locked host memory); the library never allocates, frees
 *    or synchronises inside these calls.
 *  - Matrices are row-major.  x/activations are [M][K]; weights are [N][K]
 *    (output-channel major, the Linear convention), so the GEMMs contract
 *    both operands along their contiguous K axis.
 *  - bf16 tensors hold IEEE bfloat16 bit patterns (uint16_t storage); e4m3
 *    tensors hold OCP FP8 E4M3 codes (finite variant, max 448).
 *  - `stream` is a cudaStream_t (NULL = legacy default stream).  Calls
 *    launch asynchronously and return; results are ready when the stream is.
 *  - Return value: CLEF_OK, or an error code from argument checks made on
 *    the host before anything is launched (nothing is launched on error),
 *    or CLEF_ERR_CUDA when a launch fails.  Device-side waits that exceed
 *    their time limit record CLEF_ERR_TIMEOUT in a library-owned status word
 *    read by clef_poll_status(); the kernels never trap.
 *  - M = 0 is a valid empty call: it returns CLEF_OK without a launch (its
 *    row-indexed pointers may then be null, as those of empty tensors are).
 *  - Inputs are assumed finite; NaN/Inf inputs give unspecified codes.
 *  - Alignment: every tensor base and every row pitch must be a multiple of
 *    16 bytes (TMA and vector-access rule); the checks below state it per
 *    call as the element counts that satisfy it.
 *
 * Sources (web pages; cited by title and section):
 *  [INT8]  "CLEF Calibrated INT8 ConvRot" model card: Benefits (kernels fuse
 *          calibrated scales, biases and MLP SwiGLU) and the note under the
 *          latency table (a CUDA ConvRot activation quantizer feeds integer
 *          GEMMs).
 *  [USAGE] "Loading CLEF INT8" usage notes: fuse_mlp (paired gate/up epilogue
 *          fusion) and gate/up weights packed during loading.
 *  [FP8]   "clef-flash-FP8" model card, Quantization table and the note below
 *          the recipe (FP8 weights per channel, FP8 activations per token,
 *          dynamic; weight scales computed from the weights).
 *  [LORA]  TensorFold pull request 1364, first bullet of the description:
 *          y = bf16(y + bf16(x A^T) B^T), fp32 sums, bf16 add; A (rank, k),
 *          B (n, rank); ranks zero-padded to whole 64-groups; a row's bits
 *          independent of row count and chunking.
 */
#ifndef CLEF_H
#define CLEF_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum clef_status {
    CLEF_OK = 0,
    CLEF_ERR_INVALID_ARG = 1,   /* null/misaligned pointer, bad size or stride */
    CLEF_ERR_UNSUPPORTED = 2,   /* device is not sm_103, or a mode not built */
    CLEF_ERR_CUDA = 3,          /* a CUDA runtime call or launch failed */
    CLEF_ERR_TIMEOUT = 4,       /* a device-side wait exceeded its limit */
    CLEF_ERR_BAD_PAGE = 5,      /* on the device: a page, sequence, length or row index out of range */
    CLEF_ERR_NO_PAGES = 6       /* on the device: the pool has too few free pages; nothing was changed */
} clef_status;

typedef enum clef_act_mode {
    CLEF_ACT_INT8_H128 = 0,     /* rotate 128-blocks, s = amax/127, int8 codes */
    CLEF_ACT_FP8_E4M3 = 1,      /* no rotation, s = amax/448, e4m3 codes */
    CLEF_ACT_FP8_E4M3_H128 = 2, /* rotate 128-blocks, then the FP8 codes */
    CLEF_ACT_FP8_E4M3_B128 = 3  /* no rotation, a scale for each 128 values of a row
                                   (clef_rms_norm_quant; clef_quant_fp8_block makes the same of any x) */
} clef_act_mode;

/*
 * clef_quant_act -- per-token activation quantizer [INT8: latency-table
 * note, "ConvRot activation quantizer"; FP8: Quantization table,
 * "Activations FP8, per-token, dynamic"].  Also the weight quantizer: run on
 * W's N rows it gives the per-output-channel codes and scales.
 *
 * For each row m of x (bf16 [M][K], row pitch ldx elements):
 *   v = x[m] widened to fp32; for the H128 modes each contiguous 128-block of
 *   v is rotated by the orthonormal Walsh-Hadamard butterfly (strides 1, 2,
 *   4, ..., 64, (a+b, a-b) in fp32, then one multiply by fp32(1/sqrt(128)));
 *   amax = max |v|;
 *   INT8:  scale[m] = amax/127, q = clamp(rne(v * (127/amax)), -127, 127);
 *   FP8:   scale[m] = amax/448, q = e4m3_rn_satfinite(v * (448/amax));
 *   an all-zero row gives scale 0 and codes 0.
 * q: int8 or e4m3 [M][K], dense (row pitch K); scale: fp32 [M].
 * Requirements: K > 0, K % 128 == 0 for H128 modes else K % 32 == 0,
 *   K <= 65536, ldx >= K, ldx % 8 == 0; x and q 16-byte aligned, scale 4-byte.
 */
int clef_quant_act(const void *x, int64_t M, int64_t K, int64_t ldx, int mode,
                   void *q, float *scale, void *stream);

/*
 * clef_quant_act_static -- the quantizer with one static scale s for the
 * whole tensor (a calibrated scale [INT8: "calibrated scales" of the
 * Benefits list]) in place of the per-token amax:
 *   v as in clef_quant_act; r = fp32(1 / s);
 *   INT8:  q = clamp(rne(fp32(v * r)), -127, 127)
 *   FP8:   q = e4m3_rn_satfinite(fp32(v * r))   (saturates at +-448)
 *   scale[m] = s for every row, so the GEMM entry points apply unchanged.
 * s must be positive and finite; other arguments and requirements as for
 * clef_quant_act.
 */
int clef_quant_act_static(const void *x, int64_t M, int64_t K, int64_t ldx, int mode,
                          float s, void *q, float *scale, void *stream);

/*
 * clef_w8a8_linear -- W8A8 INT8 linear with the fused scale/bias epilogue
 * [INT8: Benefits, "fuse calibrated scales, biases"].
 *   acc[m][n] = sum_k qx[m][k] * qw[n][k]        (exact int32)
 *   y[m][n]   = bf16(((float)acc * sx[m]) * sw[n] + bias[n])
 * qx: int8 [M][K] dense; sx: fp32 [M]; qw: int8 [N][K] dense; sw: fp32 [N];
 * bias: bf16 [N] or NULL; y: bf16 [M][N], row pitch ldy elements.
 * Requirements: K % 16 == 0, N % 8 == 0, ldy >= N, ldy % 8 == 0; qx, qw,
 * sw, bias and y 16-byte aligned, sx 4-byte.  The
 * library receives bare pointers and cannot check buffer lengths: sx must
 * hold M values and sw and bias N (the packed gate/up calls: 2N), else the
 * kernels read past their ends.
 */
int clef_w8a8_linear(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw,
                     const void *bias, int64_t M, int64_t N, int64_t K,
                     void *y, int64_t ldy, void *stream);

/*
 * clef_w8a8_gateup_swiglu -- INT8 gate/up projection with the paired SwiGLU
 * epilogue [USAGE: fuse_mlp; gate/up packed during loading; INT8: Benefits,
 * "MLP SwiGLU"].  qw_gu: int8 [2N][K] with the gate rows 0..N-1 followed by
 * the up rows N..2N-1; sw_gu, bias_gu: [2N] in the same order (bias may be
 * NULL).  With g, u the unrounded fp32 epilogue values of rows n and N+n:
 *   h[m][n] = bf16(g / (1 + exp(-g)) * u)
 * evaluated in fp32 with the hardware exp2 and reciprocal approximations
 * (the bf16 result is within one ulp of the correctly rounded value).
 * h: bf16 [M][N], row pitch ldh.  Requirements as clef_w8a8_linear.
 */
int clef_w8a8_gateup_swiglu(const int8_t *qx, const float *sx, const int8_t *qw_gu,
                            const float *sw_gu, const void *bias_gu,
                            int64_t M, int64_t N, int64_t K,
                            void *h, int64_t ldh, void *stream);

/*
 * clef_fp8_linear -- FP8 e4m3 W8A8 dynamic linear [FP8: Quantization table,
 * "Weights FP8, per-channel; Activations FP8, per-token, dynamic"].
 *   acc = sum_k qx[m][k] * qw[n][k] in fp32 (tensor-core accumulation order;
 *         for K >= 8192, K is cut into three fixed parts of ceil(ceil(K/128)
 *         / 3) * 128 elements (the last the rest), each summed apart, the
 *         three added in K order, for every M, so that a row's bits never
 *         depend on the call's row count or on a split)
 *   y[m][n] = bf16(((float)acc * sx[m]) * sw[n] + bias[n])
 * qx: e4m3 [M][K]; qw: e4m3 [N][K]; other arguments as clef_w8a8_linear.
 */
int clef_fp8_linear(const void *qx, const float *sx, const void *qw, const float *sw,
                    const void *bias, int64_t M, int64_t N, int64_t K,
                    void *y, int64_t ldy, void *stream);

/*
 * clef_fp8_gateup_swiglu -- the FP8 counterpart of clef_w8a8_gateup_swiglu
 * (the paired SwiGLU epilogue of [USAGE] over the FP8 scheme of [FP8]); its
 * silu uses CUDA expf and a correctly rounded division.
 */
int clef_fp8_gateup_swiglu(const void *qx, const float *sx, const void *qw_gu,
                           const float *sw_gu, const void *bias_gu,
                           int64_t M, int64_t N, int64_t K,
                           void *h, int64_t ldh, void *stream);

/*
 * clef_lora_add -- runtime LoRA add [LORA: y = bf16(y + bf16(x A^T) B^T),
 * fp32 sums and a bf16 add, rank zero-padded to a 64-group].
 *   t[m][j] = bf16(sum_k x[m][k] * A[j][k])  for j < r, 0 for r <= j < r_pad
 *   y[m][n] = bf16((float)y[m][n] + sum_j t[m][j] * B[n][j])   (in place)
 * with r_pad = r rounded up to a multiple of 64.
 * x: bf16 [M][K], row pitch ldx (the unquantized, unrotated input of the
 * projection); A: bf16 [r][K] dense; B: bf16 [N][r] dense;
 * t_scratch: bf16 [M][r_pad] dense, caller-owned scratch that receives t;
 * y: bf16 [M][N], row pitch ldy, read and written.
 * Requirements: K % 8 == 0, r % 8 == 0, 0 < r <= 1024, N % 8 == 0,
 *   ldx >= K, ldx % 8 == 0, ldy >= N, ldy % 8 == 0.
 */
int clef_lora_add(const void *x, int64_t ldx, const void *A, const void *B,
                  int64_t M, int64_t K, int64_t N, int64_t r,
                  void *t_scratch, void *y, int64_t ldy, void *stream);

/*
 * clef_w8a8_linear_lora -- the INT8 linear with the runtime LoRA expand
 * fused into the same GEMM [LORA; INT8: Benefits].  t = bf16(x A^T) comes
 * from a clef_lora_shrink call made before (t's columns past r must be
 * finite); each output tile accumulates t B^T as a last bf16 tensor-core
 * chunk, and its epilogue adds it to the rounded base value, so y is never
 * written and read back between the two:
 *   y[m][n] = bf16(bf16(((float)acc * sx[m]) * sw[n] + bias[n])
 *                  + sum_{j<r} t[m][tcol(n) + j] * B[n][j])
 * -- the same bytes as clef_w8a8_linear followed by clef_lora_expand_add from
 * t + tcol(n).  B: bf16 [N][r] dense (for packed projections, the adapters'
 * B factors stacked in output-column order; zero rows for columns without
 * an adapter).  nseg (0..4) column segments map output columns to t columns:
 * columns below seg_end[i] (and at or above seg_end[i-1]) read t columns
 * seg_tcol[i] .. seg_tcol[i] + r_pad - 1 (r_pad = r rounded up to 64);
 * nseg = 0 means one segment at t column 0.  seg_end increasing, every end
 * but the last a multiple of 256, the last equal to N; seg_tcol multiples of
 * 8 with seg_tcol + r_pad <= ldt.  t: bf16, row pitch ldt (multiple of 8).
 * Other arguments and requirements as clef_w8a8_linear; 0 < r <= 1024,
 * r % 8 == 0.  This call never splits tiles across SMs (no stream-K
 * workspace is used).
 */
int clef_w8a8_linear_lora(const int8_t *qx, const float *sx, const int8_t *qw, const float *sw,
                          const void *bias, int64_t M, int64_t N, int64_t K, const void *t, int64_t ldt,
                          const void *B, int64_t r, int nseg, const int64_t *seg_end,
                          const int64_t *seg_tcol, void *y, int64_t ldy, void *stream);

/*
 * clef_w8a8_gateup_swiglu_lora -- the INT8 gate/up SwiGLU call with the gate
 * and up LoRA adds fused [LORA; USAGE: fuse_mlp]: with t_gu = [x A_gate^T |
 * x A_up^T] from one clef_lora_shrink over the stacked A factors (each padded
 * with zero rows to r_pad),
 *   g = bf16(bf16(gate epilogue value) + sum_j t_gu[m][j] * B_gate[n][j])
 *   u = bf16(bf16(up epilogue value) + sum_j t_gu[m][r_pad + j] * B_up[n][j])
 *   h[m][n] = bf16(silu(g) * u)    (silu as in clef_swiglu_bf16)
 * -- the same bytes as clef_w8a8_linear on the packed weight (bf16 [M][2N])
 * followed by clef_lora_gateup_swiglu, without g and u ever reaching memory.
 * t_gu: bf16 [M][>= 2 r_pad] at pitch ldt (t_gate in columns 0 .. r_pad - 1,
 * t_up in r_pad .. 2 r_pad - 1; columns past r in each must be finite);
 * B_gate, B_up: bf16 [N][r] dense.  Other arguments and requirements as
 * clef_w8a8_gateup_swiglu; 0 < r <= 1024, r % 8 == 0, ldt % 8 == 0.
 */
int clef_w8a8_gateup_swiglu_lora(const int8_t *qx, const float *sx, const int8_t *qw_gu, const float *sw_gu,
                                 const void *bias_gu, int64_t M, int64_t N, int64_t K, const void *t_gu,
                                 int64_t ldt, const void *B_gate, const void *B_up, int64_t r, void *h,
                                 int64_t ldh, void *stream);

/*
 * clef_lora_shrink / clef_lora_expand_add -- the two stages of clef_lora_add
 * as separate calls [LORA], for adapters that share an input: with their A
 * factors stacked (each zero-padded to a multiple of 64 rows) one shrink
 * call reads x once for all of them, and each adapter's expand call reads its
 * own column block of t (t + offset, the shared pitch ldt).  clef_lora_add is
 * exactly clef_lora_shrink into t_scratch (ldt = r_pad) followed by
 * clef_lora_expand_add from it.
 * clef_lora_shrink: t[m][j] = bf16(sum_k x[m][k] * A[j][k]) for j < r_pad
 *   (rows j >= r of A read as zeros, so those columns of t are 0).  The fp32
 *   sum runs in the tensor core's order; for K >= 6144 it is taken as four
 *   fixed parts of ceil(K / 256) x 64 elements (the last the rest), added in
 *   K order, whatever M is, so a row's bits never depend on the call's row
 *   count.  With a workspace bound to the stream (clef_bind_workspace), the
 *   parts of a partly empty last wave of tiles run on several SMs.
 *   x: bf16 [M][K], pitch ldx; A: bf16 [r][K] dense; t: bf16 [M][r_pad],
 *   pitch ldt (only columns 0 .. r_pad - 1 written).
 * clef_lora_expand_add: y[m][n] = bf16((float)y[m][n] + sum_{j<r} t[m][j] * B[n][j])
 *   in place.  t: bf16, columns 0 .. r_pad - 1 read (pitch ldt; columns
 *   r .. r_pad - 1 are multiplied by zeros); B: bf16 [N][r] dense; y: bf16
 *   [M][N], pitch ldy.
 * Requirements: K % 8 == 0, N % 8 == 0, r % 8 == 0, 0 < r <= 4096,
 *   ldx >= K, ldt >= r_pad, ldy >= N, all pitches multiples of 8, every
 *   pointer (t + offset included) 16-byte aligned.
 */
int clef_lora_shrink(const void *x, int64_t ldx, const void *A, int64_t M, int64_t K, int64_t r,
                     void *t, int64_t ldt, void *stream);
int clef_lora_expand_add(const void *t, int64_t ldt, const void *B, int64_t M, int64_t N, int64_t r,
                         void *y, int64_t ldy, void *stream);

/*
 * clef_lora_gateup_swiglu -- runtime LoRA on the gate and up projections
 * [LORA], followed by the MLP product [USAGE], in one pass over the base
 * gate/up values: with t_g = bf16(x A_gate^T) and t_u = bf16(x A_up^T) as in
 * clef_lora_add,
 *   g[m][n] = bf16((float)y_gu[m][n]     + sum_j t_g[m][j] * B_gate[n][j])
 *   u[m][n] = bf16((float)y_gu[m][N + n] + sum_j t_u[m][j] * B_up[n][j])
 *   h[m][n] = bf16(silu(g) * u)   (fp32, silu(g) = g / (1 + exp(-g)) as in
 *                                  clef_swiglu_bf16)
 * -- the same rounded operations as two clef_lora_add calls on the halves of
 * y_gu followed by clef_swiglu_bf16, without writing g and u back.
 * x: bf16 [M][K], row pitch ldx; A_gate, A_up: bf16 [r][K] dense; B_gate,
 * B_up: bf16 [N][r] dense; t_scratch: bf16 [M][2 r_pad] dense scratch
 * (r_pad = r rounded up to 64; receives t_g then t_u); y_gu: bf16 [M][2N]
 * base gate values then up values (the output of clef_w8a8_linear on the
 * packed weight), row pitch ld_gu, read only; h: bf16 [M][N], row pitch ldh.
 * Requirements: K % 8 == 0, r % 8 == 0, 0 < r <= 1024, N % 8 == 0,
 *   ldx >= K, ld_gu >= 2N, ldh >= N, all pitches multiples of 8.
 */
int clef_lora_gateup_swiglu(const void *x, int64_t ldx, const void *A_gate, const void *B_gate,
                            const void *A_up, const void *B_up, int64_t M, int64_t K, int64_t N,
                            int64_t r, void *t_scratch, const void *y_gu, int64_t ld_gu,
                            void *h, int64_t ldh, void *stream);

/*
 * clef_swiglu_bf16 -- the unfused MLP reading (fuse_mlp off in [USAGE]):
 * y_gu holds bf16 gate values in columns 0..N-1 and up values in N..2N-1
 * (row pitch ldg); h[m][n] = bf16(silu(float(g)) * float(u)), silu(g) =
 * g / (1 + exp(-g)) in fp32 with the hardware exp2 and reciprocal
 * approximations (within one bf16 ulp of the correctly rounded value).
 * Requirements: N % 8 == 0, ldg >= 2N, ldg % 8 == 0, ldh >= N, ldh % 8 == 0.
 */
int clef_swiglu_bf16(const void *y_gu, int64_t M, int64_t N, int64_t ldg,
                     void *h, int64_t ldh, void *stream);

/*
 * clef_w8a8_gemm_s32 -- the INT8 GEMM with its raw accumulator as output
 * (acc[m][n] = sum_k qx[m][k] * qw[n][k], exact int32, row pitch ldc),
 * through the same kernel and mainloop as clef_w8a8_linear.  It exists so
 * that the integer accumulators can be compared bit for bit.
 * Requirements: K % 16 == 0, N % 8 == 0, ldc >= N, ldc % 8 == 0.
 */
int clef_w8a8_gemm_s32(const int8_t *qx, const int8_t *qw, int64_t M, int64_t N, int64_t K,
                       int32_t *acc, int64_t ldc, void *stream);

/*
 * clef_lora_add_noalloc -- the same LoRA add as clef_lora_add, without the
 * t_scratch argument, for callers that cannot allocate device memory: a host
 * whose runtime owns a fixed device-memory budget and forbids allocations
 * outside it, a plugin living inside another framework's allocator, or code
 * that must not pay the device-wide synchronisation cudaMalloc/cudaFree can
 * imply.  The pages have no counterpart of this call; it is a library
 * convenience.
 * t lives in a library-owned static device array of 4,194,304 bf16 elements
 * (8 MiB, held by every GPU that loads the library until exit):
 * M * round_up(r, 64) beyond that returns CLEF_ERR_INVALID_ARG.  The call
 * allocates nothing.  Its first call on a device looks up the array's device
 * address (cudaGetSymbolAddress) with that device current; make that first
 * call before any stream capture.  All calls share the array and it keeps the
 * previous call's contents (nothing needs clearing: each call rewrites every
 * element it reads), so calls whose kernels may overlap on the GPU race and
 * must be serialised.  It runs the same launches as clef_lora_add (tile
 * widths, the clef_set_wait_limit_ns limit and the clef_test_force_timeout
 * knob included), so its output bytes equal clef_lora_add's.  Other
 * arguments and requirements as clef_lora_add.
 */
int clef_lora_add_noalloc(const void *x, int64_t ldx, const void *A, const void *B,
                          int64_t M, int64_t K, int64_t N, int64_t r,
                          void *y, int64_t ldy, void *stream);

/*
 * clef_gemm_workspace_bytes / clef_bind_workspace -- optional scratch that
 * lets the INT8 GEMMs (clef_w8a8_linear, clef_w8a8_gemm_s32; M > 128) split
 * tiles across SMs when the last wave of whole 256 x 256 tiles would leave
 * more than 8% of the CTA pairs idle ("stream-K": the whole waves run as
 * whole tiles, the remaining tiles' K is dealt to all pairs in even runs of
 * at least 16 k-blocks of 64 (1,024 K elements; 8 k-blocks, 512 elements,
 * for a launch of under one wave), and the pieces of a tile meet as exact
 * int32 partial sums,
 * so the bytes of every output equal those of an unsplit launch).  The GEMM
 * time follows the number of tile waves (1502 x 5120 x 17408 and 1502 x 6400
 * x 17408 take the same time unsplit), so a shape with a partly empty last
 * wave gains up to the idle fraction.  A launch of less than one wave is
 * split only when its tiles would keep under an eighth of the pairs busy
 * (small M, long K); the gate/up SwiGLU calls never split.  clef_fp8_linear
 * with K >= 8192 sums every tile's K as three fixed parts whatever M is (see
 * there); with a workspace bound, the tiles of a last wave that fits three
 * times in the pairs run as their parts on three pairs each, the same bytes
 * as unsplit.  Other FP8 calls never split.  The LoRA x A^T of
 * clef_lora_shrink, clef_lora_add and clef_lora_gateup_swiglu does the same
 * with four parts for K >= 6144 (see clef_lora_shrink).
 * clef_gemm_workspace_bytes: the size needed on the current device (about
 * 38 MB on a 152-SM GB300), written to *bytes.
 * clef_bind_workspace: binds a caller-owned device buffer of that size to
 * `stream` on the current device (ws = NULL unbinds); INT8 and FP8 linear
 * calls on that stream may then use it, calls on unbound streams never split.  The buffer
 * must be zero-filled when bound; every launch leaves its counter block
 * zeroed again (after a CLEF_ERR_TIMEOUT, refill the buffer with zeros before
 * further use).  Launches that use one buffer must not run concurrently: bind
 * a separate buffer to each stream whose work may overlap.  Binding is host
 * bookkeeping (no stream operation), so it may be done while the stream is
 * being captured into a graph; the graph then keeps the buffer's address.
 * Requirements: ws 16-byte aligned and bytes >= the counter block (the
 * workspace is used for splitting only when bytes >= the size returned);
 * at most 256 bindings.
 */
int clef_gemm_workspace_bytes(int64_t *bytes);
int clef_bind_workspace(void *stream, void *ws, int64_t bytes);

/*
 * ---- linears over 4-bit weights ----
 *
 * clef_quant_w4 -- packs bf16 weights w [N][K] (row pitch ldw elements) as
 * 4-bit codes with a bf16 scale for each run of `group` (32, 64 or 128)
 * weights of a row:
 *   s = bf16(amax / 7);  c = clamp(rne(w / s), -8, 7)   (0 where s is 0)
 * Packed row: K rounded up to K_pad, a multiple of 128; K_pad / 2 bytes.  Of
 * each block of 128 weights, byte 16 t + 4 j (t, j in 0..3) starts the
 * little-endian word of weights 32 j + 8 t .. + 7, whose nibble i < 4 holds
 * weight 2 i and nibble i + 4 weight 2 i + 1, each as c + 8.  Weights past K
 * are zeros.  qw: uint8 [N][K_pad / 2]; sw: bf16 [N][K_pad / group].
 * Requirements: K % 8 == 0, K <= 65536, ldw >= K, ldw % 8 == 0, N <= 2^24;
 *   w, qw and sw 16-byte aligned.  N = 0 is a valid empty call.
 *
 * clef_w4_linear -- y[m][n] = bf16(sum_g sw[n][g] * (sum_{k in g} c[n][k] x[m][k]) + bias[n])
 * with fp32 sums, for calls of few rows: weights are read once for every 16
 * rows (for every 8 where 16 do not fit on chip, from K = 29,704 on).  x counts to 2^-38 of the largest value of its row (in each eighth of
 * K), and the sums' rounding goes by (|c| + 8) |x|, so values a millionth of
 * another one in their group may be lost beside it.  Any finite x will do; an infinity
 * or a NaN makes its row of y NaN.  The order of a row's sum follows N and K alone, so its bits do not
 * depend on M.  x: bf16 [M][K], pitch ldx; bias: bf16 [N] or NULL; y: bf16
 * [M][N], pitch ldy (any: y and bias need 2-byte alignment only).
 * Requirements: as above, M <= 2^19, ldx >= K, ldx % 8 == 0, ldy >= N.
 */
int clef_quant_w4(const void *w, int64_t N, int64_t K, int64_t ldw, int group, void *qw, void *sw, void *stream);
int clef_w4_linear(const void *x, int64_t ldx, const void *qw, const void *sw, int group, const void *bias,
                   int64_t M, int64_t N, int64_t K, void *y, int64_t ldy, void *stream);

/*
 * ---- the paged 8-bit cache ----
 *
 * A pool is `planes` planes (a layer's keys, then its values, layer by layer)
 * of `pages` pages each; a page holds `page` tokens (16, 32, 64 or 128) of
 * every key/value head: codes [pages][heads][page][dim], one byte each (kind
 * 0: int8 in -127..127; 1: e4m3), dim 64, 128 or 256, and fp32 scales
 * [pages][heads] >= 0; value = code * scale.  plane_bytes and plane_scales are
 * the distances between planes in bytes and floats.  The calls of one layer
 * take its key plane's address, the value plane following it.  A sequence is a
 * row of table (int32 [seqs][width], pitch ldt) and a length in lens: its
 * token i is at page table[i / page], place i % page.  Entries of a row past
 * the sequence's pages are never read, but by clef_kv_gather, which is not told
 * the lengths.  refs: int32 [pages], how many
 * sequences hold a page (0: free).
 *
 * Indices and lengths live in device memory, so the host cannot check them:
 * the kernels do, leave out what is out of range and record
 * CLEF_ERR_BAD_PAGE (clef_poll_status); a token of an attention whose page is
 * out of range counts with a key and a value of zeros.  Limits: 4,096 sequences, 2^20 pages a
 * sequence, 2^24 pages.  Codes must be 16-byte aligned, integers 4-byte.
 *
 * clef_kv_append -- writes the newest tokens' keys and values.  lens holds
 * the lengths with the new tokens; the rows of a sequence are its last ones:
 * rows row_start[b] .. row_start[b + 1] - 1 of k and v (row_start: int32
 * [seqs + 1]), or rows / seqs each where row_start is NULL.  k, v: bf16,
 * token pitches ldk, ldv and head pitches ldk_head, ldv_head in elements.
 * A page's scale grows with what it holds (top = 127 or 448):
 *   s = max(s_old, fp32(amax / top)), s_old = 0 for a page without tokens;
 *   where s grew, earlier codes become encode(value(code) * fp32(s_old / s));
 *   new codes are encode(v * min(fp32(1 / s), FLT_MAX)), zeros where s = 0.
 * Each growth rounds the page's earlier codes once more.  With s_0 the scale
 * after a value's own append and s_1 .. s_g those that it grew to since (g = 0
 * for a page written by one call), the value that the cache stands for is off by
 *   int8: at most (s_0 + .. + s_g) / 2;
 *   e4m3: at most ((17/16)^(g + 1) - 1) |v| + (s_0 + .. + s_g) (17/16)^g 2^-10,
 * beside the fp32 roundings.  Normal values appended one by one in pages of 64
 * tokens see four growths a page: 1.3 (int8) and 1.4 (e4m3) times the error, in
 * the mean square, of a page written at once.
 * The pages written must belong to one sequence each.  clef_kv_reserve and
 * clef_kv_fork see to it where the reservation of the new tokens was made;
 * where it was not (CLEF_ERR_NO_PAGES), the lengths do not hold the new tokens
 * and an append would write over the last ones, in pages that may be shared.
 * So a call that may find the pool full takes row_start from
 * clef_kv_reserve_rows.  k and v must be finite: a page of a head has one
 * scale, so an infinity or a NaN is felt by the page's other tokens too.
 *
 * clef_kv_gather -- k_out[r], v_out[r] = bf16(code * scale) of token pos[r]
 * of sequence seq[r]; outputs bf16 [rows][heads * dim], pitches ldk, ldv;
 * zeros where a sequence is not one of the table, a position is past its width or the
 * page there is not one of the pool.  A position past the sequence's length reads
 * whatever the table's entry and the page last held, so the caller keeps pos[r]
 * below it.
 *
 * clef_kv_attention -- softmax attention of queries over the cache, for query
 * row i of sequence b (n rows) and head h reading key/value head h / (q_heads
 * / heads):  o = sum_j softmax_j(scale * q . k_j) v_j over its tokens j <
 * lens[b], with causal only j <= lens[b] - n + i (the queries are the last
 * tokens).  Rows that see nothing are zeros; a row of a head whose queries are
 * not all finite is NaN.  q: bf16, pitches ldq (token) and
 * ldq_head; rows and row_start as for append; out: bf16, pitches ldo,
 * ldo_head; lse: fp32 [rows][q_heads], log of the sum of exponentials
 * (-infinity for a row that sees nothing), or NULL.  Sums are fp32; the
 * weights that multiply values are rounded to fp16.  The pages' scales may be
 * any finite ones, however far apart.  A row's bits depend on its own sequence
 * alone.  workspace: clef_kv_attention_workspace bytes with
 * ragged = (row_start != NULL) and max_len = width * page, 16-byte aligned; its
 * contents need no preparation and are not kept.
 *
 * clef_kv_reserve -- lens[b] += grow[b] for every sequence, with the pages
 * that takes: the lowest free ones, in the order of the sequences.
 * clef_kv_reserve_rows also writes row_start (int32 [seqs + 1], or NULL): the
 * running sum of grow, row_start[seqs] the rows in all, or zeros where nothing
 * was reserved.  An append that takes it, or takes min(row_start[seqs], its own
 * row_start[i]), writes the rows that have a place, and nothing after a failure.
 * clef_kv_fork -- sequence dst[i], empty before, becomes a copy of src[i] as it
 * was before the call: whole pages are shared (refs + 1), a part-filled last
 * page is copied to the lowest free page.  scratch: int32 [2 n].
 * Either changes nothing and records CLEF_ERR_NO_PAGES if the free pages do
 * not suffice, CLEF_ERR_BAD_PAGE if an argument on the device is out of range.
 * clef_kv_free -- the sequences list[0 .. n - 1] become empty; their pages'
 * refs - 1.
 * clef_kv_compact -- moves pages so that the L held ones are 0 .. L - 1 (the
 * k-th lowest held page past L - 1 to the k-th lowest free page below), with
 * every sequence's row written to table_out, refs to refs_out and L to *live
 * (may be NULL).  A pool of no pages is an empty call, which writes nothing.  table_out and refs_out may be table and refs.  scratch: int32
 * [3 pages + 1].
 * clef_kv_copy_pages -- page dst[i] = page src[i] in every plane; no target
 * may also be a source or listed twice.
 */
int clef_kv_append(const void *k, int64_t ldk, int64_t ldk_head, const void *v, int64_t ldv, int64_t ldv_head,
                   int64_t rows, const int32_t *row_start, int kind, void *codes, int64_t plane_bytes,
                   float *scales, int64_t plane_scales, int64_t pages, int heads, int page, int dim,
                   const int32_t *table, int64_t ldt, int64_t seqs, int64_t width, const int32_t *lens,
                   void *stream);
int clef_kv_gather(int kind, const void *codes, int64_t plane_bytes, const float *scales, int64_t plane_scales,
                   int64_t pages, int heads, int page, int dim, const int32_t *table, int64_t ldt, int64_t seqs,
                   int64_t width, const int32_t *seq, const int32_t *pos, int64_t rows, void *k_out, int64_t ldk,
                   void *v_out, int64_t ldv, void *stream);
int clef_kv_attention_workspace(int64_t rows, int ragged, int64_t seqs, int q_heads, int heads, int dim,
                                int64_t max_len, int64_t *bytes);
int clef_kv_attention(const void *q, int64_t ldq, int64_t ldq_head, int64_t rows, const int32_t *row_start,
                      int q_heads, int kind, const void *codes, int64_t plane_bytes, const float *scales,
                      int64_t plane_scales, int64_t pages, int heads, int page, int dim, const int32_t *table,
                      int64_t ldt, int64_t seqs, int64_t width, const int32_t *lens, float scale, int causal,
                      void *out, int64_t ldo, int64_t ldo_head, float *lse, void *workspace,
                      int64_t workspace_bytes, void *stream);
int clef_kv_reserve(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
                    int64_t pages, int page, const int32_t *grow, void *stream);
int clef_kv_reserve_rows(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
                         int64_t pages, int page, const int32_t *grow, int32_t *row_start, void *stream);
int clef_kv_fork(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                 int64_t pages, int heads, int page, int dim, int32_t *table, int64_t ldt, int64_t seqs,
                 int64_t width, int32_t *lens, int32_t *refs, const int32_t *src, const int32_t *dst, int64_t n,
                 int32_t *scratch, void *stream);
int clef_kv_free(int32_t *table, int64_t ldt, int64_t seqs, int64_t width, int32_t *lens, int32_t *refs,
                 int64_t pages, int page, const int32_t *list, int64_t n, void *stream);
int clef_kv_compact(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                    int64_t pages, int heads, int page, int dim, const int32_t *table, int64_t ldt, int64_t seqs,
                    int64_t width, const int32_t *lens, const int32_t *refs, int32_t *table_out, int64_t ldt_out,
                    int32_t *refs_out, int32_t *live, int32_t *scratch, void *stream);
int clef_kv_copy_pages(void *codes, int64_t plane_bytes, float *scales, int64_t plane_scales, int64_t planes,
                       int64_t pages, int heads, int page, int dim, const int32_t *src, const int32_t *dst,
                       int64_t n, void *stream);

/*
 * ---- between the projections ----
 *
 * clef_rms_norm -- root-mean-square norm of the rows of x, with the residual's
 * addition:  h = x + residual (x alone where residual is NULL),
 *   residual_out = bf16(h),  y = bf16(h w / sqrt(mean(h^2) + eps)),
 * from the fp32 sum h, before its rounding.  x, residual, residual_out, y: bf16
 * [M][K] with pitches ldx, ldr, ldro, ldy; w: bf16 [K].  residual_out may be the
 * residual, and y may be x, with the same pitch; otherwise the outputs are disjoint from
 * the inputs and from each other.  A row's bits depend on the row and w alone.
 *
 * clef_rms_norm_quant -- the same with 8-bit codes of the unrounded result v = h w
 * / sqrt(mean(h^2) + eps) as the linears take them: modes CLEF_ACT_INT8_H128,
 * CLEF_ACT_FP8_E4M3 and CLEF_ACT_FP8_E4M3_H128 give a scale a row (clef_quant_act's
 * definition on v, which is never rounded to bf16), CLEF_ACT_FP8_E4M3_B128 the
 * scales [M][ceil(K / 128)] of clef_quant_fp8_block.  q: [M][K], dense; scale: fp32.
 * y also receives bf16(v) (unrotated: what a LoRA's shrink takes) where it is not
 * NULL.
 * Requirements of both: K % 16 == 0 (% 128 for the rotated modes), K <= 32768,
 * pitches >= K and multiples of 8, tensors 16-byte and scale 4-byte aligned, 1e-20
 * <= eps <= 1e20; h and h w are within fp32.
 *
 * clef_quant_fp8_block -- e4m3 codes of x (bf16 [M][K], pitch ldx) with a scale for
 * each block of `rows` (1: activations, 128: weights) rows by 128 columns (the last
 * ones of either may be smaller):
 *   s = amax / 448, q = e4m3_rn_satfinite(x * min(448 / amax, FLT_MAX)), zeros for zeros.
 * q: e4m3 [M][K], dense; scale: fp32 [ceil(M / rows)][ceil(K / 128)].
 * Requirements: K % 16 == 0, K <= 65536, ldx >= K, ldx % 8 == 0; x and q 16-byte
 * aligned, scale 4-byte.
 *
 * clef_fp8_block_linear -- the linear over such codes: with b the blocks of 128 of K,
 *   y[m][n] = bf16(sum_b sx[m][b] sw[n / 128][b] sum_{k in b} qx[m][k] qw[n][k] + bias[n])
 * with fp32 sums: a block's in the tensor core's order, the blocks' in one that follows
 * M, N and K of the call (so a row's bits may differ between calls of other M, never
 * between calls of one size).  A product sx sw is fp32 too.  sx: fp32 [M][ceil(K / 128)]; sw: fp32
 * [ceil(N / 128)][ceil(K / 128)]; both 4-byte aligned.  Other arguments and
 * requirements as clef_fp8_linear.
 *
 * clef_fp8_block_gateup_swiglu -- h = bf16(g / (1 + exp(-g)) * u) of the unrounded
 * values g, u of rows n and N + n of the packed weight [2N][K]; N % 128 == 0, so that
 * no block of scales holds rows of both.  silu as in clef_swiglu_bf16.
 *
 * clef_rotary -- rotation of heads by the positions of their tokens.  Pair i of
 * rot / 2 is the values (i, i + rot / 2) of a head, or (2 i, 2 i + 1) where
 * interleaved; with t_i the angle of pos[token] at pair i,
 *   (a, b) -> gain (a cos t_i - b sin t_i, b cos t_i + a sin t_i)   (fp32, rounded once);
 * values from rot on are copied.  turns: int64 [rot / 2], the turns (of 2 pi) a
 * position in units of 2^-64, modulo one turn; t_i = 2 pi (pos turns_i mod 2^64) / 2^64,
 * exact for every int32 position (a negative one turns back).
 * x, out: bf16 [tokens][heads][dim] with token pitches ldx, ldo and head pitches
 * ldx_head, ldo_head; out may be x with the same pitches, and is disjoint from it
 * otherwise.  pos: int32 [tokens].
 * Requirements: dim % 8 == 0, dim <= 1024, rot even, 2 <= rot <= dim, heads <= 1024,
 * pitches >= dim and multiples of 8; x and out 16-byte, turns 8-byte, pos 4-byte
 * aligned.  Accesses are of 16, 8, 4 or 2 bytes where rot is a multiple of 16, 8, 4 or
 * 2; where interleaved, of 16, 8 or 4 where it is one of 8, 4 or 2.
 */
int clef_rms_norm(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, int64_t M, int64_t K,
                  float eps, void *residual_out, int64_t ldro, void *y, int64_t ldy, void *stream);
int clef_rms_norm_quant(const void *x, int64_t ldx, const void *residual, int64_t ldr, const void *w, int64_t M,
                        int64_t K, float eps, int mode, void *residual_out, int64_t ldro, void *y, int64_t ldy,
                        void *q, float *scale, void *stream);
int clef_quant_fp8_block(const void *x, int64_t M, int64_t K, int64_t ldx, int rows, void *q, float *scale,
                         void *stream);
int clef_fp8_block_linear(const void *qx, const float *sx, const void *qw, const float *sw, const void *bias, int64_t M,
                          int64_t N, int64_t K, void *y, int64_t ldy, void *stream);
int clef_fp8_block_gateup_swiglu(const void *qx, const float *sx, const void *qw_gu, const float *sw_gu,
                                 const void *bias_gu, int64_t M, int64_t N, int64_t K, void *h, int64_t ldh,
                                 void *stream);
int clef_rotary(const void *x, int64_t ldx, int64_t ldx_head, int64_t tokens, int heads, int dim, int rot,
                int interleaved, const int32_t *pos, const int64_t *turns, float gain, void *out, int64_t ldo,
                int64_t ldo_head, void *stream);

/*
 * clef_mma_peak -- dense tensor-core rate of this device for one instruction
 * route, measured by the library's own microbenchmark (the denominators of
 * the GEMMs' roofline fractions; not part of the projection path):
 *   kind 0: tcgen05.mma kind::f16 with bf16 operands and an fp32 accumulator
 *           (the route of the INT8 GEMMs, whose int8 codes are multiplied
 *           exactly as fp16, and of the LoRA products);
 *   kind 1: tcgen05.mma kind::f8f6f4 with e4m3 operands (the FP8 GEMMs);
 *   kind 2: mma.sync m16n8k32 s8 x s8 -> s32 (the legacy integer route).
 * The tcgen05 kinds run one CTA pair per two SMs issuing 256 x 256 MMAs back
 * to back from shared memory into two TMEM accumulators (no copies); kind 2
 * runs register-operand MMA chains in every warp.  One warm-up launch, then
 * `iters` iterations (4 MMAs of 256 x 256 x 64 (bf16) or x 128 (e4m3) per
 * iteration; 8 m16n8k32 MMAs per warp for kind 2) timed with CUDA events on
 * a private stream; *tflops = 2 x multiply-adds / seconds / 1e12.
 * Synchronises; not for use during stream capture.
 * Requirements: kind in 0..2, 0 < iters <= 2^24.
 */
int clef_mma_peak(int kind, int64_t iters, double *tflops);

/*
 * clef_poll_status -- synchronises the device, then returns and clears the
 * device-side status word (CLEF_OK if no kernel recorded an error).
 */
int clef_poll_status(void);

/*
 * clef_set_wait_limit_ns -- time limit of every device-side wait in kernels
 * launched afterwards (default 1e9 ns).  A wait that exceeds it records
 * CLEF_ERR_TIMEOUT and its kernel winds down and returns.  Test knob.
 */
void clef_set_wait_limit_ns(uint64_t ns);

/*
 * clef_test_force_timeout -- test knob for the device-side failure path.
 * on = 1: the W8A8/FP8/LoRA GEMM kernels launched afterwards make their MMA
 * issuer wait on a barrier that nothing signals; the wait runs out after the
 * clef_set_wait_limit_ns limit, CLEF_ERR_TIMEOUT is recorded in the status
 * word and the kernel winds down (their outputs are then undefined).
 * on = n >= 2: only the CTA (or CTA pair) working through tile-loop slot
 * n - 2 does so, while the others finish their tiles (a stream-K launch then
 * leaves the counters of the tiles that slot shared nonzero: the case
 * clef_bind_workspace's refill rule is for).  0 (default) or negative: off.
 */
void clef_test_force_timeout(int on);

/*
 * clef_set_quant_staging -- which quantizer kernel clef_quant_act launches
 * afterwards.  Two kernels compute the same codes and scales bit for bit: a
 * persistent one that stages rows in shared memory through TMA (for row
 * lengths that are a multiple of 64 and at most 32768) and a one-CTA-per-row
 * one (every row length).  mode 1 (default): the staged kernel for calls of
 * at least 8 rows per SM, where it streams faster; mode 2: the staged kernel
 * wherever the row length allows; mode 0: always the per-row kernel.  Other
 * values are clamped to this range.  The switch exists so that each kernel
 * can be tested and timed.
 */
void clef_set_quant_staging(int mode);

/*
 * clef_set_pdl -- programmatic dependent launch for the kernels the library
 * launches afterwards.  on != 0 (default): each launch carries CUDA's
 * programmatic stream-serialization attribute, so that a kernel's CTAs may be
 * scheduled, and run their set-up (barriers, tensor-memory allocation,
 * descriptor prefetch), while the stream's previous kernel finishes; every
 * kernel waits for the kernels it follows to complete, with their writes
 * visible, before it reads or writes global memory, so results are the same
 * bytes either way.  on == 0: plain stream order.  The switch exists so that
 * both can be tested and timed.
 */
void clef_set_pdl(int on);

/*
 * clef_set_sm_budget -- how many SMs the library's compute launches issued
 * afterwards may fill (GEMMs, LoRA launches, quantizers, norms that keep rows
 * ahead; a block linear takes one cluster of up to eight CTAs at least): sms, rounded down
 * to an even count, or every SM of the device for sms == 0 or sms at least
 * the device's count.  Results are the same bytes under any budget (the
 * tile order and every split follow the shapes, not the SM count; only the
 * number of persistent CTAs changes).  A persistent GEMM CTA takes a whole
 * SM, so work on another stream (clef_copy_sm streaming the next step's
 * inputs) gets SMs only if the budget leaves some free.  Process-wide, like
 * clef_set_pdl; launches captured into a CUDA graph keep the budget that was
 * in force when they were captured.  Stream-K tails (clef_bind_workspace)
 * are dealt over the CTA pairs the budget allows.  Returns
 * CLEF_ERR_INVALID_ARG (budget unchanged) for a negative sms or sms == 1.
 */
int clef_set_sm_budget(int sms);

/*
 * clef_copy_sm -- copy bytes bytes from src to dst with loads and stores
 * issued by ctas CTAs (one per SM; clusters of two where ctas is even)
 * instead of a copy engine.  src and dst are any addresses the device can
 * access: device memory, or page-locked host memory (cudaHostAlloc or
 * cudaHostRegister), read and written through its device mapping.  Pageable
 * host memory returns CLEF_ERR_INVALID_ARG (nothing launched) unless the
 * device reads pageable memory directly (cudaDevAttrPageableMemoryAccess).
 * Copy-engine transfers from page-locked host memory were measured to stall
 * for 20-180 ms, on some GB300 machines about every half second and on others
 * rarely; SM loads over the same link ran at the same rate without stalls on
 * every box tried.  With a budget (clef_set_sm_budget) of the device's SMs
 * less ctas, the copy runs beside the compute launches of another stream.
 * Requirements: dst and src 16-byte aligned, bytes >= 0 and a multiple of
 * 16, 1 <= ctas <= 64, the two ranges disjoint.  Ordered on stream like any
 * kernel; bytes == 0 returns CLEF_OK without a launch.
 */
int clef_copy_sm(void *dst, const void *src, int64_t bytes, int ctas, void *stream);

/* Human-readable name of a status code (static string). */
const char *clef_status_string(int status);

/* Text of the most recent argument or CUDA error seen by this thread's calls
 * (empty if none); valid until the thread's next failing call. */
const char *clef_last_error(void);

/* ABI version of this library (major * 100 + minor). */
int clef_abi_version(void);

#ifdef __cplusplus
}
#endif

#endif /* CLEF_H */

/*
 * fp8q.h -- C ABI of libfp8q.so: amax-scaled FP8 quantization and the
 * block-scaled FP8 GEMM on AMD Instinct MI355X (gfx950).
 *
 * Sources cited below:
 *   [A] the PyTorch-native FP8 article, m.nxbn.cn/news/137885 (its own
 *       section numbers: 1.2 format table, 1.3 "FN" semantics, 3.1 FP8
 *       linear, 4.1 scale factors, 4.2 delayed scaling, 4.3 margin);
 *   [H] the handbook chapter "混合精度与 FP8 训练" (anrans.github.io,
 *       ai-infra-handbooks), section "FP8 训练": quant / per_tensor /
 *       per_block, the precision-per-op table, and the hardware notes on
 *       promoting partial sums every 128 elements.
 *
 * Conventions shared by every entry point
 *   - Pointers are device pointers (hipMalloc'd or torch CUDA tensors)
 *     unless stated otherwise.  The caller owns every buffer: the library
 *     never allocates, frees, synchronizes or copies to the host.
 *   - `stream` is a hipStream_t passed as void*; NULL is the default
 *     stream.  Every call is asynchronous on that stream.
 *   - Arguments are validated on the host before anything is enqueued.  A
 *     return other than FP8Q_OK means nothing was enqueued, except
 *     FP8Q_EHIP (a launch failed; fp8q_last_error() has the HIP text).
 *   - Formats: FP8Q_E4M3FN = OCP E4M3FN (bias 7, max 448, no Inf,
 *     0x7F/0xFF are NaN); FP8Q_E5M2 = OCP E5M2 (bias 15, max 57344) ([A]
 *     1.2, 1.3).  One code is one byte.
 *   - Scales are dequantization scales s (x ~= dec(q) * s), fp32:
 *     s = fl32(fl32(max(amax, eps) * margin) / MAX), MAX = 448 or 57344
 *     ([H] per_block: amax.clamp(min=1e-12) / MAX; margin from [A] 4.3).
 *   - Encoding: q = enc(fl32(x / s)) where fl32 is IEEE fp32 division and
 *     enc rounds to nearest, ties to even, saturates at +-MAX, keeps the
 *     sign of zero and maps NaN to 0x7F ([H] quant: (x / s).clamp(-MAX,
 *     MAX).to(FP8)).  Results are bit-identical to that definition.
 *   - Row-major 2-D operands with leading dimensions in elements.
 *   - Reentrant; the only global state is the thread-local error text.
 */
#ifndef FP8Q_H
#define FP8Q_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  FP8Q_OK = 0,
  FP8Q_EINVAL = 1,   /* null pointer, non-positive size, bad enum value  */
  FP8Q_ESHAPE = 2,   /* a size is not a multiple of 128 where required    */
  FP8Q_EALIGN = 3,   /* pointer or leading dimension breaks 16-B alignment */
  FP8Q_EHIP = 4,     /* the HIP runtime refused the launch                */
  FP8Q_ENOTIMPL = 5  /* combination not provided by this build            */
} fp8q_status;

typedef enum { FP8Q_F32 = 0, FP8Q_BF16 = 1 } fp8q_dtype;
typedef enum { FP8Q_E4M3FN = 0, FP8Q_E5M2 = 1 } fp8q_format;
typedef enum { FP8Q_GRAN_TENSOR = 0, FP8Q_GRAN_1x128 = 1, FP8Q_GRAN_128x128 = 2 } fp8q_gran;

/* Statistic of the amax history that sets the delayed scale ([A] 4.2: the
 * window maximum; the mean as a gentler choice; an exponential moving
 * average smoothing the amax, as Transformer Engine does; [A] 4.3). */
typedef enum { FP8Q_STAT_MAX = 0, FP8Q_STAT_MEAN = 1, FP8Q_STAT_EMA = 2 } fp8q_window_stat;

/* Activations: SiLU g / (1 + e^-g) and GELU in its tanh form
 * g (1 + tanh(sqrt(2/pi) (g + 0.044715 g^3))) / 2 (the gated projection and
 * the linear layer); none, ReLU and GELU itself, g (1 + erf(g / sqrt(2))) / 2
 * (the linear layer alone). */
typedef enum {
  FP8Q_ACT_SILU = 0,
  FP8Q_ACT_GELU = 1,
  FP8Q_ACT_NONE = 2,
  FP8Q_ACT_RELU = 3,
  FP8Q_ACT_GELU_ERF = 4
} fp8q_act;

/* Delayed-scaling state ([A] 4.2 DelayedScaler): a window of the last
 * `window` amax values and the scale derived from them.  Device-resident,
 * caller-allocated (8-byte aligned), plain data (copy it to the host to
 * checkpoint it).  `ring` holds the history (first `window` entries used),
 * `pos` the next slot, `count` the number of values seen (saturating at
 * window), `scale` the dequantization scale in force, 1.0 until the window
 * fills; `stat` the fp8q_window_stat, `alpha` the EMA coefficient and `ema`
 * the EMA of every amax seen (fp64; 0 unless stat is FP8Q_STAT_EMA).
 * `amax_acc` is the running amax of the current step: the tensors quantized
 * with fp8q_quantize_tensor_delayed fold their max|x| into it, and
 * fp8q_delayed_scaler_update consumes it and sets it back to 0. */
typedef struct {
  float ring[1024];
  int32_t window;
  int32_t count;
  int32_t pos;
  float max_val;
  float eps;
  float margin;
  float scale;
  int32_t stat;
  float alpha;
  float amax_acc;
  double ema;
} fp8q_scaler;

/* Library version (major*100 + minor). */
int fp8q_version(void);

/* Text for a status code; static storage. */
const char* fp8q_status_string(int status);

/* Text of the last FP8Q_EHIP or validation failure on this thread. */
const char* fp8q_last_error(void);

/* amax = max_i |x_i| over n elements ([A] 4.1; [H] per_tensor).
 * x: n elements of dtype dt, 16-B aligned.  amax: one fp32, overwritten
 * by the reduction's last workgroup (one launch; whatever *amax held
 * before is ignored).  A NaN anywhere gives the quiet NaN 0x7FC00000;
 * +-Inf gives +Inf.  Calls in flight at the same time must not share the
 * amax buffer (different buffers are independent). */
int fp8q_amax(const void* x, fp8q_dtype dt, int64_t n, float* amax, void* stream);

/* Per-tensor quantization with a scale held in device memory, the form
 * delayed scaling uses ([A] 4.2: the scale from earlier steps quantizes
 * the current tensor; [H] per_tensor).
 * x: n elements of dtype dt, 16-B aligned.  scale: one fp32 dequant scale
 * s, read on the device when the kernel runs (e.g. &state->scale).
 * q: n codes, 16-B aligned.
 * amax_out: nullable.  When given, *amax_out = max_i |x_i| of this call's
 *   x, overwritten in the same launch (the last workgroup of the quantizing
 *   pass writes it; whatever the buffer held before is ignored).  A NaN
 *   anywhere gives the quiet NaN 0x7FC00000.  This fuses the amax that
 *   delayed scaling records for the next step into the same pass over x
 *   ([A] 4.2); hand it to fp8q_delayed_scaler_update.  Calls in flight at
 *   the same time must not share an amax_out buffer. */
int fp8q_quantize_tensor(const void* x, fp8q_dtype dt, int64_t n, fp8q_format f, const float* scale,
                         uint8_t* q, float* amax_out, void* stream);

/* fp8q_quantize_tensor that also writes the round trip: y = fl32(dec(q) * s)
 * (fp32, or rounded to nearest-even bf16; NaN -> the quiet NaN), bit for bit
 * what fp8q_dequantize makes of the codes, in the same pass over x -- the
 * handbook's quant ([H]: (x / s).clamp().to(FP8).float() * s) and the
 * quantize-dequantize of a fake-quantized forward copy ([A] 4.2).
 * y: n elements of out_dt, 16-B aligned; other arguments and errors as
 * fp8q_quantize_tensor. */
int fp8q_quantize_tensor_dq(const void* x, fp8q_dtype dt, int64_t n, fp8q_format f, const float* scale,
                            uint8_t* q, float* amax_out, void* y, fp8q_dtype out_dt, void* stream);

/* The per-tensor quantization of one delayed-scaling step ([A] 4.2: the
 * scale derived from earlier steps quantizes this step's tensor, and this
 * step's amax is recorded for the next): q = enc(fl32(x / state->scale)),
 * and max|x| is folded into state->amax_acc as a running maximum (NaN
 * winning), so several tensors or micro-batches of one step feed one
 * window entry; fp8q_delayed_scaler_update(state, NULL) then pushes it into
 * the window and sets it back to 0.  No reset launch is needed: the state
 * owns the accumulator.  With y non-null the round trip y = fl32(dec(q) *
 * s) is written in the same pass, as fp8q_quantize_tensor_dq writes it.
 * x: n elements of dtype dt, 16-B aligned; q: n codes, 16-B aligned; y:
 * nullable, n elements of out_dt, 16-B aligned; state: initialized by
 * fp8q_delayed_scaler_init[_stat], 8-B aligned.  Calls that fold into one
 * state may overlap (the fold is atomic); the update must follow them all
 * on the stream. */
int fp8q_quantize_tensor_delayed(const void* x, fp8q_dtype dt, int64_t n, fp8q_format f, fp8q_scaler* state,
                                 uint8_t* q, void* y, fp8q_dtype out_dt, void* stream);

/* Fine-grained 1x128 quantization of activations ([H] per_block(x, 1,
 * 128); DeepSeek-V3 activation tiling).  For row r and column block kb:
 *   s = scale(amax(x[r, 128kb : 128kb+128]), eps), q = enc(fl32(x/s)).
 * x: rows x cols, element (r,c) at x[r*ldx + c]; cols % 128 == 0;
 *   ldx >= cols; x and ldx*sizeof(dt) 16-B aligned.
 * q: codes at q[r*ldq + c]; ldq >= cols, 16-B aligned.
 * scales: fp32 at scales[r*ld_s + kb], ld_s >= cols/128.
 * eps: lower clamp of amax (the pages use 1e-12); must be > 0. */
int fp8q_quantize_1x128(const void* x, fp8q_dtype dt, int64_t rows, int64_t cols, int64_t ldx,
                        fp8q_format f, float eps, uint8_t* q, int64_t ldq, float* scales,
                        int64_t ld_s, void* stream);

/* Fine-grained 1x128 quantization of the transpose: the operands of the
 * weight-gradient GEMM are reduced over tokens, so activations and output
 * gradients stored [tokens, features] are needed as [features, tokens]
 * codes with one scale per 128 tokens ([H] fine-grained scaling along the
 * reduced dimension; [A] 6.3 E5M2 gradients).  Equal to fp8q_quantize_1x128
 * of x^T, without materializing x^T:
 *   for column c of x and row block rb:
 *   s = scale(amax(x[128rb : 128rb+128, c]), eps), q[c, r] = enc(fl32(x[r, c]/s)).
 * x: rows x cols, element (r,c) at x[r*ldx + c]; rows % 128 == 0,
 *   cols % 64 == 0; ldx >= cols; x and ldx*sizeof(dt) 16-B aligned.
 * q: codes of x^T at q[c*ldq + r]; ldq >= rows, q and ldq 16-B aligned.
 * scales: fp32 at scales[c*ld_s + rb], ld_s >= rows/128.
 * eps: lower clamp of amax; must be > 0. */
int fp8q_quantize_1x128_t(const void* x, fp8q_dtype dt, int64_t rows, int64_t cols, int64_t ldx,
                          fp8q_format f, float eps, uint8_t* q, int64_t ldq, float* scales,
                          int64_t ld_s, void* stream);

/* MX (microscaling) FP8 quantization: every 32 consecutive elements of a
 * row share one power-of-two scale X = 2^e held as an E8M0 byte e + 127
 * (0xFF = NaN); [H] names this hardware-native block scaling as the next
 * step after 1x128 / 128x128.  The conversion follows the OCP Microscaling
 * Formats (MX) specification v1.0, 6.3: e = floor(log2 max|x|) - emax
 * (emax = 8 for E4M3FN, 15 for E5M2), clamped to [-127, 127];
 * q = enc(x / X), round to nearest even, clamped to +-MAX.  An all-zero
 * block has e = -127; a block holding a NaN or an Inf gets scale byte 0xFF
 * and codes 0x7F.
 * x: rows x cols at x[r*ldx + c]; cols % 32 == 0; x and ldx*sizeof(dt)
 *   16-B aligned.  q: codes at q[r*ldq + c], q and ldq 16-B aligned.
 * scales: bytes at scales[r*ld_s + c/32], ld_s >= cols/32. */
int fp8q_quantize_mx(const void* x, fp8q_dtype dt, int64_t rows, int64_t cols, int64_t ldx, fp8q_format f,
                     uint8_t* q, int64_t ldq, uint8_t* scales, int64_t ld_s, void* stream);

/* MX dequantization y = fl32(dec(q) * 2^(s - 127)) (scale byte 0xFF: NaN,
 * the quiet NaN 0x7FC00000), bf16 output as RNE of that fp32.  Layouts as
 * fp8q_quantize_mx; cols % 32 == 0; q 16-B aligned with ldq % 8 == 0; y and
 * its rows 16-B aligned. */
int fp8q_dequantize_mx(const uint8_t* q, fp8q_format f, int64_t rows, int64_t cols, int64_t ldq,
                       const uint8_t* scales, int64_t ld_s, void* y, fp8q_dtype out_dt, int64_t ldy, void* stream);

/* Fine-grained 128x128 quantization of weights ([H] per_block(x, 128,
 * 128)).  As fp8q_quantize_1x128 with one scale per 128x128 tile:
 * scales[rb*ld_s + kb] for rows 128rb.. and columns 128kb..;
 * rows % 128 == 0 and cols % 128 == 0. */
int fp8q_quantize_128x128(const void* x, fp8q_dtype dt, int64_t rows, int64_t cols, int64_t ldx,
                          fp8q_format f, float eps, uint8_t* q, int64_t ldq, float* scales,
                          int64_t ld_s, void* stream);

/* Set a device-resident scaler to its initial state ([A] 4.2 __init__):
 * empty history, scale = 1.0, statistic the window maximum.  window in
 * [1, 1024] (1 gives current scaling), max_val > 0 (448 or 57344),
 * eps > 0, margin > 0 ([A] 4.3; 1.0 means none). */
int fp8q_delayed_scaler_init(fp8q_scaler* state, int32_t window, float max_val, float eps,
                             float margin, void* stream);

/* As fp8q_delayed_scaler_init with the history statistic chosen ([A] 4.2,
 * 4.3).  FP8Q_STAT_MAX: max of the window.  FP8Q_STAT_MEAN: mean of the
 * window, its values summed in fp64 by pairwise (binary-tree) summation
 * over the 1024 slots (unused slots 0), divided by window in fp64,
 * rounded to fp32.  FP8Q_STAT_EMA: e = amax for the first value, then
 * e = alpha*amax + (1-alpha)*e with each product and the sum rounded to
 * fp64 (no fused multiply-add); alpha in (0, 1]; the statistic is fl32(e)
 * and the window only sets when the scale first moves.  The scale is then
 * fl32(fl32(max(stat, eps) * margin) / max_val).  A NaN amax makes max and
 * mean NaN while it is in the window and the EMA NaN until re-init.
 * Errors: FP8Q_EINVAL for a bad stat or alpha, as above otherwise. */
int fp8q_delayed_scaler_init_stat(fp8q_scaler* state, int32_t window, float max_val, float eps,
                                  float margin, fp8q_window_stat stat, float alpha, void* stream);

/* One delayed-scaling step ([A] 4.2 update): push *amax into the ring
 * (and into the EMA); amax may be NULL, meaning the state's own amax_acc
 * (filled by fp8q_quantize_tensor_delayed).  Once `window` values have
 * been seen, scale =
 * fl32(fl32(max(stat, eps) * margin) / max_val) with stat the state's
 * statistic (max(ring) by default), otherwise the scale stays at its
 * previous value.  *amax is then reset to 0 (the quantizers overwrite it
 * anyway).  A NaN amax propagates into the scale.
 * Runs as one wavefront; never syncs with the host. */
int fp8q_delayed_scaler_update(fp8q_scaler* state, float* amax, void* stream);

/* Dequantization x^ = fl32(dec(q) * s) ([H] quant: .float() * scale),
 * written as fp32 or rounded to nearest-even bf16 (NaN -> quiet NaN).
 * q: rows x cols codes at q[r*ldq + c].  scales by granularity g:
 *   TENSOR: scales[0]; 1x128: scales[r*ld_s + c/128];
 *   128x128: scales[(r/128)*ld_s + c/128].
 * y: y[r*ldy + c] of dtype out_dt.  cols % 128 == 0 for the block
 * granularities; q and y 16-B aligned; ldq, ldy multiples of 4 (ignored
 * when rows == 1, so a flat tensor of any length is rows=1, cols=n). */
int fp8q_dequantize(const uint8_t* q, fp8q_format f, int64_t rows, int64_t cols, int64_t ldq,
                    const float* scales, fp8q_gran g, int64_t ld_s, void* y, fp8q_dtype out_dt,
                    int64_t ldy, void* stream);

/* Block-scaled FP8 GEMM ([A] 3.1 F.linear(x, w) with w stored [out, in];
 * [H] FP8 inputs with fp32 accumulation, partial sums promoted to fp32
 * every 128 elements of K):
 *   C[m,n] = sum_kb (sA[m,kb] * sB(n,kb)) * P_kb[m,n],
 *   P_kb[m,n] = sum_{k in [128kb, 128kb+128)} dec(A[m,k]) * dec(B[n,k]),
 * each P_kb formed in fp32 and folded into an fp32 accumulator.
 * Every product and every in-block sum is carried out in full fp32 (the
 * codes are decoded exactly and multiplied on the bf16 matrix cores), so
 * |C - C_exact| stays within a few fp32 roundings of
 * D[m,n] = sum_kb |sA*sB| * sum_k |dec(a)*dec(b)|.
 * A: M x K codes of format fa at A[m*lda + k].
 * sA: 1x128 scales along K at sA[m*sA_sm + kb*sA_skb].
 * B: N x K codes of format fb at B[n*ldb + k] (the weight as nn.Linear
 *   stores it, or any K-contiguous operand).
 * sB: gb = FP8Q_GRAN_128x128: sB[(n/128)*sB_sn + kb*sB_skb] (ceil(N/128) rows);
 *     gb = FP8Q_GRAN_1x128:   sB[n*sB_sn + kb*sB_skb].
 * C: M x N at C[m*ldc + n], fp32 or bf16 (round to nearest even).
 * K % 128 == 0 (else FP8Q_ESHAPE); M, N >= 1 with ragged edges masked;
 * lda, ldb >= K and multiples of 16; A, B 16-B aligned; ldc >= N.
 * NaN or Inf codes make the affected outputs non-finite. */
int fp8q_gemm_blockscaled(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA,
                          int64_t sA_sm, int64_t sA_skb, const uint8_t* B, fp8q_format fb,
                          int64_t ldb, const float* sB, fp8q_gran gb, int64_t sB_sn,
                          int64_t sB_skb, void* C, fp8q_dtype out_dt, int64_t ldc, int64_t M,
                          int64_t N, int64_t K, void* stream);

/* The same GEMM with each 128-wide block product P_kb taken from the FP8
 * matrix cores directly (twice the MFMA rate).  Arguments and layout as
 * fp8q_gemm_blockscaled.  Inside a block the hardware aligns each group of
 * eight products to the largest one and drops what lies about 2^-14 below
 * it -- the limited FP8 accumulator that motivates promotion every 128 K
 * in [H] -- so the error bound is |C - C_exact| <= 2^-10 * D[m,n] rather
 * than a few fp32 roundings; the promotion across blocks is fp32. */
int fp8q_gemm_blockscaled_fast(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA,
                               int64_t sA_sm, int64_t sA_skb, const uint8_t* B, fp8q_format fb,
                               int64_t ldb, const float* sB, fp8q_gran gb, int64_t sB_sn,
                               int64_t sB_skb, void* C, fp8q_dtype out_dt, int64_t ldc, int64_t M,
                               int64_t N, int64_t K, void* stream);

/* fp8q_gemm_blockscaled with the output quantized in the epilogue, for
 * the next layer's input ([A] 5.1: casts to and from a wide type between
 * FP8 operations eat the gain; [H] fine-grained 1x128 scaling): the fp32
 * C of fp8q_gemm_blockscaled is never written; instead, per row and 128
 * consecutive columns, Cs[m*ld_cs + n/128] = fl32(max(amax, eps) / MAX_fc)
 * and Cq[m*ldcq + n] = enc_fc(fl32(C[m,n] / s)), bit for bit what
 * fp8q_quantize_1x128 makes of that fp32 C (saturating, RNE, NaN -> 0x7F).
 * Arguments as fp8q_gemm_blockscaled (exact path) plus: fc the output
 * format, eps > 0, Cq [M, N] codes with ldcq >= N, Cs [M, N/128] fp32 with
 * ld_cs >= N/128.  N % 128 == 0 and K % 128 == 0 (else FP8Q_ESHAPE). */
int fp8q_gemm_blockscaled_q(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                            int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                            fp8q_gran gb, int64_t sB_sn, int64_t sB_skb, fp8q_format fc, float eps, uint8_t* Cq,
                            int64_t ldcq, float* Cs, int64_t ld_cs, int64_t M, int64_t N, int64_t K,
                            void* stream);

/* fp8q_gemm_blockscaled with the output quantized along M in the epilogue,
 * for a gradient produced by this GEMM (a dgrad whose output is the
 * previous layer's output gradient): the previous layer's weight-gradient
 * GEMM reduces over tokens (M), so it takes C^T as codes with one scale per
 * 128 tokens ([H] fine-grained 1x128 scaling along the reduced dimension;
 * [A] 6.3 gradients in E5M2; [A] 5.1 casts to and from a wide type between
 * FP8 operations eat the gain).  The fp32 C of fp8q_gemm_blockscaled is
 * never written; instead, per column n and 128 consecutive rows,
 *   Cst[n*ld_cst + m/128] = fl32(max(amax(C[128(m/128) : +128, n]), eps) / MAX_fc),
 *   Cqt[n*ldcqt + m]     = enc_fc(fl32(C[m,n] / s)),
 * bit for bit what fp8q_quantize_1x128_t makes of that fp32 C.  With Cq and
 * Cs non-null the same epilogue also writes the row-wise output of
 * fp8q_gemm_blockscaled_q (what the previous layer's dgrad takes), from the
 * same accumulators.
 * Arguments as fp8q_gemm_blockscaled (exact path) plus: fc the output
 * format, eps > 0; Cqt [N, M] codes, ldcqt >= M, Cqt and ldcqt 16-B
 * aligned; Cst [N, M/128] fp32, ld_cst >= M/128; Cq, Cs nullable together
 * (ldcq >= N, ld_cs >= N/128).  M % 128 == 0 and K % 128 == 0, and
 * N % 128 == 0 when Cq is given (else FP8Q_ESHAPE); otherwise N >= 1. */
int fp8q_gemm_blockscaled_qt(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                             int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                             fp8q_gran gb, int64_t sB_sn, int64_t sB_skb, fp8q_format fc, float eps, uint8_t* Cqt,
                             int64_t ldcqt, float* Cst, int64_t ld_cst, uint8_t* Cq, int64_t ldcq, float* Cs,
                             int64_t ld_cs, int64_t M, int64_t N, int64_t K, void* stream);

/* MX GEMM ([H] FP8 training, hardware note: 32 elements share one scale
 * factor in hardware): C[m,n] = sum over 32-element K blocks kb of
 *   2^(sA[m,kb] - 127) * 2^(sB[n,kb] - 127) * sum_{k in kb} dec(A[m,k]) dec(B[n,k]),
 * the product of two fp8q_quantize_mx outputs (B as [N,K], K-contiguous).
 * The scaled FP8 MFMA of gfx950 applies both scales and accumulates the
 * whole K in fp32; like fp8q_gemm_blockscaled_fast it is bounded by
 * |C - C_exact| <= 2^-10 * D, D the same sum over |terms|, while the scaled
 * terms stay in fp32's normal range (products of two scales far from 1 can
 * underflow to zero or overflow to Inf in fp32).
 * A [M,K] codes, lda; B [N,K] codes, ldb (16-B aligned rows); sA [M, K/32]
 * and sB [N, K/32] E8M0 bytes with row strides ld_sa, ld_sb (multiples of
 * 4, >= K/32); K % 128 == 0; M, N free.  C [M,N] fp32 or bf16 (RNE), ldc.
 * A scale byte 0xFF makes the result unspecified (NaN blocks). */
int fp8q_gemm_mx(const uint8_t* A, fp8q_format fa, int64_t lda, const uint8_t* sA, int64_t ld_sa,
                 const uint8_t* B, fp8q_format fb, int64_t ldb, const uint8_t* sB, int64_t ld_sb, void* C,
                 fp8q_dtype out_dt, int64_t ldc, int64_t M, int64_t N, int64_t K, void* stream);

/* ---- Feed-forward operators: what stands between two block-scaled products
 * of a transformer layer, forward and backward, for prompts, training steps
 * and single tokens. */

/* Root-mean-square norm with the residual's addition and a 1x128 FP8 output,
 * the input of the next fp8q_gemm_blockscaled / fp8q_glu_blockscaled ([A]
 * 5.1: casts through a wide type between FP8 operations eat the gain):
 *   v = x + res (res NULL: v = x);  rstd = 1 / sqrt(mean_c(v^2) + norm_eps);
 *   y = (v * rstd) * w;  q, scales = fp8q_quantize_1x128(y).
 * v, the sum of squares and y are fp32; z and y are rounded once, to the
 * nearest even, when they are stored, and neither the norm nor the codes
 * read the rounded values.
 * x, res, z, y: rows x cols of dtype dt (row strides ldx, ldr, ldz, ldy).
 * res, z, y, rstd nullable; z is v (the residual stream), and may be x or
 * res itself.  w: cols weights of dtype wdt.  q nullable together with
 * scales (y is then required): codes of format f at q[r*ldq + c], fp32
 * scales at scales[r*ld_s + c/128], ld_s >= cols/128; eps is their amax
 * clamp.  rstd: rows fp32, what fp8q_rmsnorm_bwd takes.
 * cols % 128 == 0, cols <= 65536 (else FP8Q_ESHAPE); norm_eps > 0; every
 * pointer and row 16-B aligned (scales, rstd 4-B).  A row that holds a NaN
 * gives NaN scales and codes 0x7F; the fp32 sum of squares overflows to Inf
 * where its root passes 1.8e19, and such a row gives zeros (NaN at an Inf).
 * Rows beyond what one launch has threads for (67 million up to 2048
 * columns, 4 to 16 million beyond) take several launches; at most 2^31-1. */
int fp8q_rmsnorm_1x128(const void* x, fp8q_dtype dt, int64_t ldx, const void* res, int64_t ldr, const void* w,
                       fp8q_dtype wdt, int64_t rows, int64_t cols, float norm_eps, void* z, int64_t ldz, void* y,
                       int64_t ldy, fp8q_format f, float eps, uint8_t* q, int64_t ldq, float* scales, int64_t ld_s,
                       float* rstd, void* stream);

/* Bytes of workspace fp8q_rmsnorm_bwd needs for the weight's gradient (at
 * most 2048 bytes per column; 0 for sizes it refuses). */
int64_t fp8q_rmsnorm_bwd_workspace(int64_t rows, int64_t cols);

/* Gradients of fp8q_rmsnorm_1x128 (the quantization passed straight through):
 *   xh = z * rstd, t = dy * w,
 *   dx = rstd * (t - xh * mean_c(t * xh)) + dres,   dw[c] = sum_r dy * xh.
 * dx is the gradient of x and of res alike.  dy, z, dres, dx: rows x cols of
 * dtype dt; z is the forward's z (x itself without a residual), rstd its
 * rstd.  dres (nullable): the gradient that reaches v past the norm, on the
 * residual stream; dx may be dy or dres itself.  dw: cols fp32, overwritten; NULL
 * skips it (ws then unused).  ws: ws_bytes >= fp8q_rmsnorm_bwd_workspace,
 * 16-B aligned, overwritten; calls in flight must not share it.  Sums are
 * fp32, in an order fixed by rows and cols alone.  Sizes and alignment as
 * fp8q_rmsnorm_1x128. */
int fp8q_rmsnorm_bwd(const void* dy, fp8q_dtype dt, int64_t lddy, const void* z, int64_t ldz, const void* w,
                     fp8q_dtype wdt, const float* rstd, const void* dres, int64_t lddr, int64_t rows, int64_t cols,
                     void* dx, int64_t lddx, float* dw, void* ws, int64_t ws_bytes, void* stream);

/* Gated projection: both products, the activation and the product of the
 * two in one kernel,
 *   g = A Bg^T,  u = A Bu^T  (each as fp8q_gemm_blockscaled),
 *   H[m,n] = act(g[m,n]) * u[m,n].
 * A: M x K codes, 1x128 scales, as fp8q_gemm_blockscaled.  Bg, Bu: F x K
 * codes of format fb, both with row stride ldb; sBg, sBu: their 128x128
 * scales at [(n/128)*sB_sn + kb*sB_skb].  One [2F, K] matrix is passed as
 * its two halves.  H: M x F fp32 or bf16 at H[m*ldh + n].  gu (nullable):
 * g and u rounded to bf16 for the backward pass, M x 2F at gu[m*ldgu + n]
 * and gu[m*ldgu + F + n], ldgu >= 2F; H is made from the unrounded ones.
 * K % 128 == 0 (else FP8Q_ESHAPE); M, F >= 1; alignment as the GEMM.  A, Bg
 * and Bu each span less than 4 GiB (else FP8Q_ESHAPE), in the forms below too. */
int fp8q_glu_blockscaled(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                         int64_t sA_skb, const uint8_t* Bg, const uint8_t* Bu, fp8q_format fb, int64_t ldb,
                         const float* sBg, const float* sBu, int64_t sB_sn, int64_t sB_skb, fp8q_act act, void* H,
                         fp8q_dtype out_dt, int64_t ldh, uint16_t* gu, int64_t ldgu, int64_t M, int64_t F, int64_t K,
                         void* stream);

/* The same on the FP8 matrix cores (twice the rate), g and u within the
 * bound of fp8q_gemm_blockscaled_fast; a few rows, which the weight's bytes
 * bound, are computed exactly here too. */
int fp8q_glu_blockscaled_fast(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                              int64_t sA_skb, const uint8_t* Bg, const uint8_t* Bu, fp8q_format fb, int64_t ldb,
                              const float* sBg, const float* sBu, int64_t sB_sn, int64_t sB_skb, fp8q_act act,
                              void* H, fp8q_dtype out_dt, int64_t ldh, uint16_t* gu, int64_t ldgu, int64_t M,
                              int64_t F, int64_t K, void* stream);

/* fp8q_glu_blockscaled with H as 1x128 codes of format fc, the input of the
 * down projection: bit for bit what fp8q_quantize_1x128 makes of its fp32 H.
 * Hq: M x F codes (ldhq >= F), Hs: [M, F/128] fp32 (ld_hs >= F/128); eps the
 * amax clamp.  F % 128 == 0 as well (else FP8Q_ESHAPE); Hq and its rows 4-B
 * aligned.  ws: ws_bytes >= fp8q_glu_blockscaled_q_workspace, 16-B aligned,
 * overwritten; NULL where that is 0.  Calls in flight must not share it. */
int fp8q_glu_blockscaled_q(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                           int64_t sA_skb, const uint8_t* Bg, const uint8_t* Bu, fp8q_format fb, int64_t ldb,
                           const float* sBg, const float* sBu, int64_t sB_sn, int64_t sB_skb, fp8q_act act,
                           fp8q_format fc, float eps, uint8_t* Hq, int64_t ldhq, float* Hs, int64_t ld_hs,
                           uint16_t* gu, int64_t ldgu, int64_t M, int64_t F, int64_t K, void* ws, int64_t ws_bytes,
                           void* stream);

/* Bytes of workspace fp8q_glu_blockscaled_q needs: 4*M*F for a few rows, whose
 * output is quantized by a second launch, 0 for more (and for sizes it
 * refuses). */
int64_t fp8q_glu_blockscaled_q_workspace(int64_t M, int64_t F);

/* Gradient of the gated projection at its pre-activations, quantized for the
 * products that follow, with H recomputed:
 *   dg = dH * u * act'(g),  du = dH * act(g),  H = act(g) * u   (fp32),
 * D = [dg | du] (M x 2F).  From dH (M x F of dtype dt) and the forward's gu:
 *   Dq, Ds: D as 1x128 codes along features, codes at Dq[m*lddq + n], scales
 *     [M, 2F/128] (ld_ds): dX = D [Wg; Wu] is fp8q_gemm_blockscaled of Dq and
 *     the weight stored [K, 2F];
 *   Dt, Dst (nullable together): D^T as 1x128 codes along tokens, 2F x Mp at
 *     Dt[n*lddt + m], scales [2F, Mp/128] (ld_dst): d[Wg; Wu] = D^T X;
 *   Ht, Hst (nullable together): H^T likewise, F x Mp, of format fh, for the
 *     down projection's weight gradient.
 * Mp is M rounded up to a multiple of 128: the padding is written as zero
 * codes, so any M can be reduced over.  fc: format of D (E4M3FN or E5M2);
 * eps the amax clamp.  F % 128 == 0 and fewer than 2^23 blocks of 128 x 128
 * (else FP8Q_ESHAPE); lddt, ldht >= Mp;
 * dH, gu, Dq, Dt, Ht and their rows 16-B aligned. */
int fp8q_glu_bwd_q(const void* dH, fp8q_dtype dt, int64_t lddh, const uint16_t* gu, int64_t ldgu, fp8q_act act,
                   fp8q_format fc, float eps, uint8_t* Dq, int64_t lddq, float* Ds, int64_t ld_ds, uint8_t* Dt,
                   int64_t lddt, float* Dst, int64_t ld_dst, fp8q_format fh, uint8_t* Ht, int64_t ldht, float* Hst,
                   int64_t ld_hst, int64_t M, int64_t F, void* stream);

/* fp8q_gemm_blockscaled for a few rows (1 <= M <= 64: single tokens, decoding
 * batches), where the bytes of B are the work.  Arguments, layout and error
 * bound as fp8q_gemm_blockscaled; more rows are FP8Q_ESHAPE, and so is an
 * operand that spans 4 GiB or more. */
int fp8q_gemm_blockscaled_few(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                              int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                              fp8q_gran gb, int64_t sB_sn, int64_t sB_skb, void* C, fp8q_dtype out_dt, int64_t ldc,
                              int64_t M, int64_t N, int64_t K, void* stream);

/* Layer norm with the residual's addition and a 1x128 FP8 output, the input
 * of the next block-scaled product ([A] 5.1: casts through a wide type between
 * FP8 operations eat the gain; the statistics are fp32, [H] precision per op):
 *   v = x + res (res NULL: v = x);  mean = mean_c(v);
 *   rstd = 1 / sqrt(mean_c((v - mean)^2) + norm_eps);
 *   y = (v - mean) * rstd * w + b;  q, scales = fp8q_quantize_1x128(y).
 * v, both sums and y are fp32; z and y are rounded once, to the nearest even,
 * when they are stored, and neither the norm nor the codes read the rounded
 * values.
 * x, res, z, y: rows x cols of dtype dt (row strides ldx, ldr, ldz, ldy).
 * res, z, y, mean, rstd nullable; z is v (the residual stream), and may be x
 * or res itself.  w (nullable: ones), b (nullable: zeros): cols elements of
 * dtype wdt.  q nullable together with scales (y is then required): codes of
 * format f at q[r*ldq + c], fp32 scales at scales[r*ld_s + c/128], ld_s >=
 * cols/128; eps is their amax clamp.  mean, rstd: rows fp32, what
 * fp8q_layernorm_bwd takes.
 * cols % 8 == 0, with codes cols % 128 == 0, cols <= 65536 (else FP8Q_ESHAPE);
 * norm_eps > 0; every pointer and row 16-B aligned (scales, mean, rstd 4-B).
 * A row that holds an Inf or a NaN gives NaN throughout (codes 0x7F, NaN
 * scales); where the fp32 sum of squares overflows (distances from the mean
 * whose root sum of squares passes 1.8e19) rstd is 0 and y is b; where a sum of
 * the row's own values passes fp32's largest, its mean is not finite and y is
 * NaN throughout, as for an Inf.  At most 2^31-1 rows. */
int fp8q_layernorm_1x128(const void* x, fp8q_dtype dt, int64_t ldx, const void* res, int64_t ldr, const void* w,
                         const void* b, fp8q_dtype wdt, int64_t rows, int64_t cols, float norm_eps, void* z, int64_t ldz,
                         void* y, int64_t ldy, fp8q_format f, float eps, uint8_t* q, int64_t ldq, float* scales,
                         int64_t ld_s, float* mean, float* rstd, void* stream);

/* Bytes of workspace fp8q_layernorm_bwd needs for the gradients of weight and
 * bias (at most 2048 bytes per column; 0 for sizes it refuses). */
int64_t fp8q_layernorm_bwd_workspace(int64_t rows, int64_t cols);

/* Gradients of fp8q_layernorm_1x128 (the quantization passed straight
 * through):
 *   xh = (z - mean) * rstd, t = dy * w,
 *   dx = rstd * (t - mean_c(t) - xh * mean_c(t * xh)) + dres,
 *   dw[c] = sum_r dy * xh,  db[c] = sum_r dy.
 * dx is the gradient of x and of res alike.  dy, z, dres, dx: rows x cols of
 * dtype dt; z is the forward's z (x itself without a residual), mean and rstd
 * its statistics, w its weight (nullable: ones).  dres (nullable): the gradient
 * that reaches v past the norm, on the residual stream; dx may be dy or dres
 * itself.  dw, db: cols fp32, overwritten; each NULL skips it (both: ws is
 * unused).  ws: ws_bytes >= fp8q_layernorm_bwd_workspace, 16-B aligned,
 * overwritten; calls in flight must not share it.  Sums are fp32, in an order
 * fixed by rows and cols alone.  Sizes and alignment as fp8q_layernorm_1x128
 * without codes. */
int fp8q_layernorm_bwd(const void* dy, fp8q_dtype dt, int64_t lddy, const void* z, int64_t ldz, const void* w,
                       fp8q_dtype wdt, const float* mean, const float* rstd, const void* dres, int64_t lddr, int64_t rows,
                       int64_t cols, void* dx, int64_t lddx, float* dw, float* db, void* ws, int64_t ws_bytes,
                       void* stream);

/* Linear layer: the product of fp8q_gemm_blockscaled with what a layer does
 * to it in the same kernel,
 *   v[m,n] = (A B^T)[m,n] + bias[n],   C[m,n] = act(v[m,n]) + res[m,n].
 * A: M x K codes, 1x128 scales, B: N x K codes, 128x128 scales at
 * [(n/128)*sB_sn + kb*sB_skb], as fp8q_gemm_blockscaled.  bias (nullable): N
 * elements of dtype bias_dt (ignored without one), of any element alignment.
 * act: any fp8q_act.  res (nullable): M x N of C's dtype, row stride ldr; C
 * may be res itself (the residual stream updated in place).  C: M x N fp32 or
 * bf16 at C[m*ldc + n].  pre (nullable): v rounded to bf16 for
 * fp8q_linear_bwd_q, M x N, row stride ldpre >= N; C is made from the unrounded v.
 * Everything behind the product is fp32; C is rounded once.  ReLU keeps NaN;
 * SiLU and both GELUs give NaN at -Inf.
 * ws: ws_bytes >= fp8q_linear_blockscaled_workspace, 16-B aligned,
 * overwritten; NULL where that is 0.  Calls in flight must not share it.
 * The order of every sum is fixed by M, N, K, exact or _fast, and the device's
 * number of compute units: the same bits every call.
 * K % 128 == 0 (else FP8Q_ESHAPE); M, N >= 1; alignment as the GEMM; C, res
 * and pre aligned to their elements.  A and B each span less than 4 GiB (else
 * FP8Q_ESHAPE), in the forms below too. */
int fp8q_linear_blockscaled(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm, int64_t sA_skb,
                            const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB, int64_t sB_sn, int64_t sB_skb,
                            const void* bias, fp8q_dtype bias_dt, fp8q_act act, const void* res, int64_t ldr, void* C,
                            fp8q_dtype out_dt, int64_t ldc, uint16_t* pre, int64_t ldpre, int64_t M, int64_t N, int64_t K,
                            void* ws, int64_t ws_bytes, void* stream);

/* The same on the FP8 matrix cores (twice the rate), the product within the
 * bound of fp8q_gemm_blockscaled_fast; a few rows, which the weight's bytes
 * bound, may be computed exactly here too. */
int fp8q_linear_blockscaled_fast(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                                 int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                                 int64_t sB_sn, int64_t sB_skb, const void* bias, fp8q_dtype bias_dt, fp8q_act act,
                                 const void* res, int64_t ldr, void* C, fp8q_dtype out_dt, int64_t ldc, uint16_t* pre,
                                 int64_t ldpre, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes, void* stream);

/* fp8q_linear_blockscaled with act(v) as 1x128 codes of format fc, the input
 * of the next product: what fp8q_quantize_1x128 makes of the fp32 act(v).
 * Cq: M x N codes (ldcq >= N), Cs: [M, N/128] fp32 (ld_cs >= N/128); eps the
 * amax clamp.  N % 128 == 0 as well (else FP8Q_ESHAPE); Cq and its rows 16-B
 * aligned. */
int fp8q_linear_blockscaled_q(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                              int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                              int64_t sB_sn, int64_t sB_skb, const void* bias, fp8q_dtype bias_dt, fp8q_act act,
                              fp8q_format fc, float eps, uint8_t* Cq, int64_t ldcq, float* Cs, int64_t ld_cs,
                              uint16_t* pre, int64_t ldpre, int64_t M, int64_t N, int64_t K, void* ws, int64_t ws_bytes,
                              void* stream);

/* The same on the FP8 matrix cores, as fp8q_linear_blockscaled_fast. */
int fp8q_linear_blockscaled_q_fast(const uint8_t* A, fp8q_format fa, int64_t lda, const float* sA, int64_t sA_sm,
                                   int64_t sA_skb, const uint8_t* B, fp8q_format fb, int64_t ldb, const float* sB,
                                   int64_t sB_sn, int64_t sB_skb, const void* bias, fp8q_dtype bias_dt, fp8q_act act,
                                   fp8q_format fc, float eps, uint8_t* Cq, int64_t ldcq, float* Cs, int64_t ld_cs,
                                   uint16_t* pre, int64_t ldpre, int64_t M, int64_t N, int64_t K, void* ws,
                                   int64_t ws_bytes, void* stream);

/* Bytes of workspace the linear layer's forms need: `fast` (0 or 1) for the
 * _fast forms, `codes` for the _q forms.  Ask for any size: 4*M*N for the codes
 * of a few rows, and of few rows or many the tiles that do not fill a round of
 * the device's compute units may leave partial sums, less than 4 MiB for each
 * compute unit in all.  0 where neither happens, and for sizes they refuse.  The
 * answer holds on the device that is current when it is asked. */
int64_t fp8q_linear_blockscaled_workspace(int fast, int codes, int64_t M, int64_t N, int64_t K);

/* Bytes of workspace fp8q_linear_bwd_q needs for the bias's gradient: 4*N for
 * each 128 tokens, 0 up to 128 tokens (and for sizes it refuses). */
int64_t fp8q_linear_bwd_q_workspace(int64_t M, int64_t N);

/* Gradient of the linear layer at its pre-activations, quantized for the
 * products that follow, with the bias's gradient and the layer's output again:
 *   D = dC * act'(pre),  dbias[n] = sum_m D[m,n],  H = act(pre)   (fp32).
 * (The residual's gradient is dC itself.)  From dC (M x N of dtype dt) and the
 * forward's pre (may be NULL for FP8Q_ACT_NONE without Ht):
 *   Dq, Ds: D as 1x128 codes along features, codes at Dq[m*lddq + n], scales
 *     [M, N/128] (ld_ds): dA = D B is fp8q_gemm_blockscaled of Dq and the
 *     weight stored [K, N];
 *   Dt, Dst (nullable together): D^T as 1x128 codes along tokens, N x Mp at
 *     Dt[n*lddt + m], scales [N, Mp/128] (ld_dst): dB = D^T A;
 *   Ht, Hst (nullable together): H^T likewise, N x Mp, of format fh, for the
 *     next layer's weight gradient;
 *   dbias (nullable): N fp32, overwritten; sums in an order fixed by M and N.
 * Mp is M rounded up to a multiple of 128: the padding is written as zero
 * codes (0x7F in a block that holds a NaN, as its scale is one), so any M can
 * be reduced over.  fc: format of D; eps the amax clamp.
 * ReLU's gradient is 0 where pre <= 0, whatever dC holds there.  Where pre is
 * +Inf or -Inf, act' is its limit, 1 or 0 (none: 1), and H what the forward gives:
 * +Inf stays, -Inf is 0 for ReLU and NaN for SiLU and both GELUs.
 * ws: ws_bytes >= fp8q_linear_bwd_q_workspace where dbias is given, 16-B
 * aligned, overwritten; calls in flight must not share it.
 * N % 128 == 0 and fewer than 2^23 blocks of 128 x 128 (else FP8Q_ESHAPE);
 * lddt, ldht >= Mp; dC, pre, Dq, Dt, Ht and their rows 16-B aligned. */
int fp8q_linear_bwd_q(const void* dC, fp8q_dtype dt, int64_t lddc, const uint16_t* pre, int64_t ldpre, fp8q_act act,
                      fp8q_format fc, float eps, uint8_t* Dq, int64_t lddq, float* Ds, int64_t ld_ds, uint8_t* Dt,
                      int64_t lddt, float* Dst, int64_t ld_dst, fp8q_format fh, uint8_t* Ht, int64_t ldht, float* Hst,
                      int64_t ld_hst, float* dbias, int64_t M, int64_t N, void* ws, int64_t ws_bytes, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* FP8Q_H */

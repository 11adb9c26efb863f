// Declarations and device helpers shared by the feed-forward operators
// (fp8q_norm.hip, fp8q_layernorm.hip, fp8q_glu.hip, fp8q_linear.hip,
// fp8q_glu_bwd.hip, fp8q_linear_bwd.hip, fp8q_few.hip).
#pragma once

#include "fp8q_internal.h"

namespace fp8q {

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));
typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));
typedef float v4f __attribute__((ext_vector_type(4)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2bf __attribute__((ext_vector_type(2)));

// Two fp32 -> two bf16 in a dword, round to nearest even (off by at most
// half a bf16 step, 2^-8 of the value).
__device__ __forceinline__ uint32_t pk_bf16(float a, float b) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector(v2f{a, b}, v2bf));
}

// Four values -> four codes of a 1x128 block with the block's own scale s,
// the arithmetic of fp8q_quantize_1x128 on fp32 input: the correctly rounded
// quotient from r = 1/s while s lies in [2^-80, 2^80] (`fast`), IEEE division
// otherwise.  The first needs no saturation: no value passes the block's
// maximum, whose quotient is at most MAX and one fp32 rounding.  A block that
// holds a NaN has a NaN scale and takes the second form (0x7F); one that
// holds an Inf has an Inf scale, and its finite values become 0.
template <int FMT>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float s, float r, bool fast) {
  if (fast) return pack4<FMT>(div_rn(a, s, r), div_rn(b, s, r), div_rn(c, s, r), div_rn(d, s, r));
  return enc1<FMT>(a / s) | (enc1<FMT>(b / s) << 8) | (enc1<FMT>(c / s) << 16) | (enc1<FMT>(d / s) << 24);
}

// block_scale without the division's long form: MAX is 7 * 2^6 or 7 * 2^13,
// so fl32(m / MAX) is the quotient by 7, corrected as in div_rn, times a power
// of two, wherever neither leaves the normal range; NaN, Inf and extreme
// maxima take the division.
template <int FMT>
__device__ __forceinline__ float block_scale7(float amax, float eps) {
  const float m = (amax < eps) ? eps : amax;
  if (m >= 0x1p-80f && m <= 0x1p100f) return div_rn(m, 7.0f, 1.0f / 7.0f) * (7.0f / max_finite(FMT));
  return m / max_finite(FMT);
}

// fl32(1 / s) for s in [2^-80, 2^80] (scale_ok), in a third of the division's
// instructions: the hardware's reciprocal is within one step, and one Newton
// step whose residual is exact in an FMA rounds it correctly (equal to the IEEE
// quotient for each of the 2^23 mantissas; powers of two only scale it).  Other
// s take the division in encode4, which does not read it.
__device__ __forceinline__ float recip(float s) {
  const float r = __builtin_amdgcn_rcpf(s);
  return __builtin_fmaf(__builtin_fmaf(-s, r, 1.0f), r, r);
}

// The larger of m and |x|, or NaN if one is (v_maximum3_f32: the magnitude
// costs nothing, where an integer maximum takes an AND for each value).
__device__ __forceinline__ float max_abs(float m, float x) { return __builtin_elementwise_maximum(m, __builtin_fabsf(x)); }

__device__ __forceinline__ uint32_t abs_bits(float x) { return __float_as_uint(x) & 0x7FFFFFFFu; }

// Eight elements of a row as loaded, and as fp32.
template <int DT>
struct Raw8 {
  u32x4 v[DT == FP8Q_F32 ? 2 : 1];
  template <bool STREAM = true>
  __device__ __forceinline__ void load(const void* p, int64_t i) {
    const u32x4* q = (const u32x4*)((const char*)p + i * (DT == FP8Q_F32 ? 4 : 2));
#pragma unroll
    for (int k = 0; k < (DT == FP8Q_F32 ? 2 : 1); ++k) v[k] = STREAM ? __builtin_nontemporal_load(q + k) : q[k];
  }
  // the same value eight times (one that bf16 holds)
  __device__ __forceinline__ void fill(float x) {
    const uint32_t u = __float_as_uint(x);
#pragma unroll
    for (int k = 0; k < (DT == FP8Q_F32 ? 2 : 1); ++k)
#pragma unroll
      for (int e = 0; e < 4; ++e) v[k][e] = DT == FP8Q_F32 ? u : (u >> 16) * 0x10001u;
  }
  __device__ __forceinline__ float operator[](int e) const {
    if constexpr (DT == FP8Q_F32) return __uint_as_float(v[e >> 2][e & 3]);
    else return e & 1 ? bf_hi(v[0][e >> 1]) : bf_lo(v[0][e >> 1]);
  }
};

// Eight fp32 values into a row, rounded to its type.
template <int DT>
__device__ __forceinline__ void store8(void* p, int64_t i, const float (&v)[8]) {
  if constexpr (DT == FP8Q_F32) {
    u32x4* q = (u32x4*)((float*)p + i);
    u32x4 a, b;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = __float_as_uint(v[e]), b[e] = __float_as_uint(v[4 + e]);
    __builtin_nontemporal_store(a, q);
    __builtin_nontemporal_store(b, q + 1);
  } else {
    u32x4 a;
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] = pk_bf16(v[2 * e], v[2 * e + 1]);
    __builtin_nontemporal_store(a, (u32x4*)((uint16_t*)p + i));
  }
}

// Eight weights (fp32 or bf16), cached: every row reads the same ones.
__device__ __forceinline__ void load_w8(const void* w, int wdt, int64_t i, float (&v)[8]) {
  if (wdt == FP8Q_F32) {
    const float4 a = *(const float4*)((const float*)w + i), b = *(const float4*)((const float*)w + i + 4);
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    const u32x4 a = *(const u32x4*)((const uint16_t*)w + i);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[2 * e] = bf_lo(a[e]), v[2 * e + 1] = bf_hi(a[e]);
  }
}

// Sum over the 64 lanes, the same bits in every lane (each step adds the
// same two partial sums in both partners): quads, half rows and rows of 16
// lanes by DPP, then the rows.
__device__ __forceinline__ float wave_sum(float v) {
#define FP8Q_DPP_ADD(CTRL_) \
  v += __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL_, 0xF, 0xF, false))
  FP8Q_DPP_ADD(0xB1);   // lane ^ 1
  FP8Q_DPP_ADD(0x4E);   // lane ^ 2
  FP8Q_DPP_ADD(0x141);  // the other quad of the half row
  FP8Q_DPP_ADD(0x140);  // the other half of the row
#undef FP8Q_DPP_ADD
  v += __shfl_xor(v, 16);
  v += __shfl_xor(v, 32);
  return v;
}

struct NormFwd {
  const void *x, *res, *w;
  void *z, *y;
  uint8_t* q;
  float *scales, *rstd;
  int64_t ldx, ldr, ldz, ldy, ldq, ld_s, rows, cols;
  float neps, qeps;
  int dt, wdt, fmt;
};
struct NormBwd {
  const void *dy, *z, *w, *dres;
  const float* rstd;
  void* dx;
  float *dw, *ws;
  int64_t lddy, ldz, lddr, lddx, rows, cols;
  int dt, wdt;
};
static constexpr int64_t kNormMaxCols = 65536;
int launch_rmsnorm_1x128(const NormFwd& p, hipStream_t st);
int launch_rmsnorm_bwd(const NormBwd& p, hipStream_t st);
// Partial sums of the weight's gradient that a backward call of this many
// rows and columns writes (each a row of `cols` floats of the workspace).
int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols);

// w, b: nullable (ones, zeros), both of type wdt.
struct LayerNormFwd {
  const void *x, *res, *w, *b;
  void *z, *y;
  uint8_t* q;
  float *scales, *mean, *rstd;
  int64_t ldx, ldr, ldz, ldy, ldq, ld_s, rows, cols;
  float neps, qeps;
  int dt, wdt, fmt;
};
// pw, pb, ldp: where the kernel leaves each workgroup's column sums (set by
// the launch).
struct LayerNormBwd {
  const void *dy, *z, *w, *dres;
  const float *mean, *rstd;
  void* dx;
  float *dw, *db, *ws, *pw, *pb;
  int64_t lddy, ldz, lddr, lddx, rows, cols, ldp;
  int dt, wdt;
};
int launch_layernorm_1x128(const LayerNormFwd& p, hipStream_t st);
int launch_layernorm_bwd(const LayerNormBwd& p, hipStream_t st);
// Partial rows of both column sums (2 * cols floats each) that a backward
// call writes.
int64_t layernorm_bwd_parts(int64_t rows, int64_t cols);
// Column sums of a table of `parts` rows of `cols` floats (a multiple of
// four), 16-byte aligned: the first `split` columns to a, the rest to b.
void launch_column_sums(const float* ws, int64_t parts, int64_t cols, int64_t split, float* a, float* b, hipStream_t st);

// A gated projection (B1 the second matrix, act) or, with B1 null, a plain
// product; N output columns.  The output is out_dt elements, or codes of
// format fc with scales when `scales` is given (ws: see glu_q_workspace); gu
// (nullable) gets the pre-activations, [M, 2N] bf16.
struct Proj {
  const uint8_t *A, *B0, *B1;
  const float *sA, *s0, *s1;
  void* out;
  float *scales, *ws;
  uint16_t* gu;
  int64_t lda, sA_sm, sA_skb, ldb, sB_sn, sB_skb, ldo, ld_s, ldgu, M, N, K;
  float eps;
  int fa, fb, gb, act, out_dt, fc;
};
// What a linear layer adds to its product, each part optional: a bias (bdt) of
// any element alignment, an activation, the pre-activations kept as bf16 and a
// residual of the output's type.  vo, vp, vr: whether the rows of the output,
// of pre and of the residual are 16-byte aligned.
struct Epilogue {
  const void *bias, *res;
  uint16_t* pre;
  int64_t ldr, ldpre;
  int bdt, act;
  bool vo, vp, vr;
};
// Rows the product of a few rows takes at most.
static constexpr int64_t kFewRows = 64;
// e (nullable; plain products with 128x128 B scales only): a linear layer's epilogue.
int launch_few(const Proj& p, const Epilogue* e, const char* what, hipStream_t st);
// The linear layer: p.out as out_dt, or codes and p.scales; p.ws as the workspace.
int launch_linear(const Proj& p, const Epilogue& e, bool fast, const char* what, hipStream_t st);
int64_t linear_workspace(bool fast, bool codes, int64_t M, int64_t N, int64_t K);
int launch_glu(const Proj& p, bool fast, const char* what, hipStream_t st);
// Bytes of fp32 workspace the quantized gated projection takes: its output
// where the few-row kernel makes it, none otherwise.
int64_t glu_q_workspace(int64_t M, int64_t F);

// The block-scaled FP8-MFMA product with 128x128 B scales on tiles of two
// heights, and whether a product is better off so.
bool gemm_fast_cut(int64_t M, int64_t N, int64_t K);
int launch_gemm_fast_cut(Proj p, const char* what, hipStream_t st);

struct GluBwd {
  const void* dh;
  const uint16_t* gu;
  uint8_t *d, *dt_, *ht;
  float *ds, *dts, *hts;
  int64_t lddh, ldgu, ldd, ld_ds, lddt, ld_dts, ldht, ld_hts, M, F;
  float eps;
  int dh_dt, act, fc, fh;
};
int launch_glu_bwd(const GluBwd& p, hipStream_t st);

struct LinearBwd {
  const void* dc;
  const uint16_t* pre;
  uint8_t *d, *dt_, *ht;
  float *ds, *dts, *hts, *dbias, *ws;
  int64_t lddc, ldpre, ldd, ld_ds, lddt, ld_dts, ldht, ld_hts, M, N;
  float eps;
  int dc_dt, act, fc, fh;
};
int launch_linear_bwd(const LinearBwd& p, hipStream_t st);

}  // namespace fp8q

// Matrix-core helpers of the feed-forward kernels: FP8 codes decoded to the
// 16-bit operands of the exact path, and the activation with its gradient.
#pragma once

#include "fp8q_ffn.h"

#include <type_traits>

namespace fp8q {
namespace ffn {

typedef int v8i __attribute__((ext_vector_type(8)));
typedef __bf16 v8bf __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));

// Operand type of the exact path: bf16, or f16 when an operand is E5M2 (an
// E5M2 code is the upper byte of its f16, so its decode is a byte permute).
// Both hold every code exactly, and their products are exact in fp32.
template <bool H16>
struct Op {
  using v8 = v8bf;
  using v2 = v2bf;
};
template <>
struct Op<true> {
  using v8 = v8h;
  using v2 = v2h;
};

template <int FMT, bool H16, bool HI>
__device__ __forceinline__ typename Op<H16>::v2 dec2(uint32_t w) {
  if constexpr (!H16 && FMT == FP8Q_E4M3FN)
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8((int)w, 1.0f, HI);
  else if constexpr (!H16)
    return __builtin_amdgcn_cvt_scalef32_pk_bf16_bf8((int)w, 1.0f, HI);
  else if constexpr (FMT == FP8Q_E4M3FN)
    return __builtin_amdgcn_cvt_scalef32_pk_f16_fp8((int)w, 1.0f, HI);
  else
    return __builtin_bit_cast(v2h, __builtin_amdgcn_perm(0u, w, HI ? 0x030C020Cu : 0x010C000Cu));
}

// Eight codes -> one 16x16x32 operand.
template <int FMT, bool H16>
__device__ __forceinline__ typename Op<H16>::v8 dec8(uint32_t lo, uint32_t hi) {
  const auto a = dec2<FMT, H16, false>(lo), b = dec2<FMT, H16, true>(lo);
  const auto c = dec2<FMT, H16, false>(hi), d = dec2<FMT, H16, true>(hi);
  typename Op<H16>::v8 r;
  r[0] = a[0]; r[1] = a[1]; r[2] = b[0]; r[3] = b[1];
  r[4] = c[0]; r[5] = c[1]; r[6] = d[0]; r[7] = d[1];
  return r;
}

template <bool H16>
__device__ __forceinline__ v4f mfma32(typename Op<H16>::v8 a, typename Op<H16>::v8 b, v4f c) {
  if constexpr (H16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(a, b, c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// 1 / (1 + e^-x) by the hardware's base-2 exponential and reciprocal, each
// within an fp32 step, 2 * 2^-24 of its value.  The product x log2(e) and its
// rounded constant are off by 1.23 |x| 2^-24 in the exponent, the sum by
// 2^-24: together (1.25 |x| + 5) 2^-24 of the result where that is normal
// (x > -87).  Below, e^-x passes to Inf and the result to 0, its limit.
__device__ __forceinline__ float sigmoid(float x) {
  return __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(x * -1.4426950408889634f));
}

// act(g), and act'(g) where asked for.  SiLU: g * sigmoid(g).  GELU (tanh
// form): g * p with p = (1 + tanh(k))/2 = sigmoid(2k),
// k = sqrt(2/pi) (g + 0.044715 g^3).
template <int ACT, bool GRAD>
__device__ __forceinline__ float activation(float g, float& grad) {
  if constexpr (ACT == FP8Q_ACT_SILU) {
    const float sg = sigmoid(g);
    if (GRAD) grad = sg * (1.0f + g * (1.0f - sg));
    return g * sg;
  }
  const float c = 0.7978845608028654f, a = 0.044715f;
  const float p = sigmoid(2.0f * c * (g + a * g * g * g));
  if (GRAD) {
    // p' = 2 p (1 - p) k'; 0 where p is 0 or 1, though g^2 may be Inf there
    const float d = 2.0f * p * (1.0f - p);
    grad = d == 0.0f ? p : p + g * (d * c * (1.0f + 3.0f * a * g * g));
  }
  return g * p;
}
template <int ACT>
__device__ __forceinline__ float activation(float g) {
  float unused;
  return activation<ACT, false>(g, unused);
}

// The linear layer's activations: those two, none, ReLU, and GELU itself,
// g * P(g) with P the normal distribution function.  For a = |g| and
// Q(a) = 1 - P(a): Q = exp(-a^2/2) t poly(t), t = 1 / (1 + 0.3 a), where the
// polynomial is fitted to Q exp(a^2/2) / t for 0 <= a <= 14 (relative error
// 2^-22.4, constants rounded to fp32; Q is 0 in fp32 from 13.2 on), and P(g) = Q for g < 0, 1 - Q
// otherwise, so neither tail cancels.  With the hardware's exponential and
// reciprocal Q is off by (1.5 g^2 + 16) 2^-24 of its value: g^2 log2(e)/2 is
// rounded twice and its constant once, the rest are a dozen roundings.
//
// Where an activation passes nothing on (ReLU's negative side) its gradient is
// 0 whatever arrives, Inf and NaN included; NaN pre-activations stay NaN.
// linear_act gives act(g); linear_act_bwd dc * act'(g), and h = act(g).  The
// derivative's second term, g p', is 0 at both ends but Inf * 0 if formed from an
// infinite g, so it is formed from g clamped to where p has long been 0 or 1.
__device__ __forceinline__ float normal_cdf(float g, float& e) {
  const float a = __builtin_fabsf(g), t = __builtin_amdgcn_rcpf(__builtin_fmaf(0.3f, a, 1.0f));
  e = __builtin_amdgcn_exp2f(g * g * -0.72134752044448170f);
  float r = 0.03567475825548172f;
  r = __builtin_fmaf(r, t, -0.15720301866531372f);
  r = __builtin_fmaf(r, t, 0.20635339617729187f);
  r = __builtin_fmaf(r, t, -0.05368354171514511f);
  r = __builtin_fmaf(r, t, 0.1285615712404251f);
  r = __builtin_fmaf(r, t, 0.09991350769996643f);
  r = __builtin_fmaf(r, t, 0.1207539513707161f);
  r = __builtin_fmaf(r, t, 0.11962930113077164f);
  const float q = e * (r * t);
  return g < 0.0f ? q : 1.0f - q;
}
template <int ACT>
__device__ __forceinline__ float linear_act(float g) {
  if constexpr (ACT == FP8Q_ACT_NONE) return g;
  else if constexpr (ACT == FP8Q_ACT_RELU) return g <= 0.0f ? 0.0f : g;
  else if constexpr (ACT == FP8Q_ACT_GELU_ERF) {
    float e;
    return g * normal_cdf(g, e);
  } else return activation<ACT>(g);
}
template <int ACT>
__device__ __forceinline__ float linear_act_bwd(float dc, float g, float& h) {
  if constexpr (ACT == FP8Q_ACT_NONE) {
    h = g;
    return dc;
  } else if constexpr (ACT == FP8Q_ACT_RELU) {
    h = linear_act<ACT>(g);
    return g <= 0.0f ? 0.0f : dc;
  } else if constexpr (ACT == FP8Q_ACT_GELU_ERF) {
    float e;
    const float p = normal_cdf(g, e), d = e * 0.3989422804014327f;
    h = g * p;
    return dc * (d == 0.0f ? p : __builtin_fmaf(g, d, p));  // g may be Inf where the density is 0
  } else if constexpr (ACT == FP8Q_ACT_SILU) {
    const float p = sigmoid(g);  // NaN where g is, whatever the clamp gives there
    h = g * p;
    return dc * __builtin_fmaf(__builtin_amdgcn_fmed3f(g, -128.0f, 128.0f) * p, 1.0f - p, p);
  } else {
    // p = sigmoid(2 k), k = c (g + a g^3): p' = p (1 - p) 2 c (1 + 3 a g^2).  Beyond 16 p is 0 or 1.  The exponent
    // has g itself, which leaves p a NaN where the clamp does not
    constexpr float c2 = 2.0f * 0.7978845608028654f, a = 0.044715f, l = -1.4426950408889634f;
    const float x = __builtin_amdgcn_fmed3f(g, -16.0f, 16.0f), x2 = x * x;
    const float p = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(g * __builtin_fmaf(x2, l * c2 * a, l * c2)));
    const float q = x * p;
    h = g * p;
    return dc * __builtin_fmaf(__builtin_fmaf(-q, p, q), __builtin_fmaf(x2, 3.0f * a * c2, c2), p);
  }
}
// f with the activation as a constant: the choice is made once around a
// loop, so that the exponentials of its elements overlap.
template <typename F>
__device__ __forceinline__ void with_linear_act(int act, F f) {
  switch (act) {
    case FP8Q_ACT_SILU: f(std::integral_constant<int, FP8Q_ACT_SILU>{}); break;
    case FP8Q_ACT_GELU: f(std::integral_constant<int, FP8Q_ACT_GELU>{}); break;
    case FP8Q_ACT_RELU: f(std::integral_constant<int, FP8Q_ACT_RELU>{}); break;
    case FP8Q_ACT_GELU_ERF: f(std::integral_constant<int, FP8Q_ACT_GELU_ERF>{}); break;
    default: f(std::integral_constant<int, FP8Q_ACT_NONE>{}); break;
  }
}
// The same for the gated projection's two.
template <typename F>
__device__ __forceinline__ void with_activation(int act, F f) {
  if (act == FP8Q_ACT_SILU) f(std::integral_constant<int, FP8Q_ACT_SILU>{});
  else f(std::integral_constant<int, FP8Q_ACT_GELU>{});
}

// ---- tiles.  The layouts, the copies and the tile order are those of the
// block-scaled GEMM: a staged row is 128 bytes (one K block), its 16-byte
// chunk c in slot c ^ swz(row) so that the sixteen rows of a fragment read
// fall on different banks.
__device__ __forceinline__ int swz_chunk(int r, int c) { return c ^ ((r & 6) | ((r >> 3) & 1)); }

// Global-to-LDS copies as inline assembly: the compiler would wait for every
// one of them before the first LDS read.  The kernel orders them with its own
// vmcnt waits and barriers.  M0 holds the LDS address of lane 0; lane l
// writes `size` bytes at M0 + l * size.
__device__ __forceinline__ void lds_dma16(uint32_t lds_addr, const uint8_t* sbase, uint32_t voff) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2"
               :
               : "s"(lds_addr), "v"(voff), "s"(sbase)
               : "memory", "m0");
}
__device__ __forceinline__ void lds_dma4(uint32_t lds_addr, const float* gptr) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off"
               :
               : "s"(lds_addr), "v"(gptr)
               : "memory", "m0");
}
__device__ __forceinline__ uint32_t lds_addr_of(const void* p) {
  return (uint32_t)(uintptr_t)(const __attribute__((address_space(3))) void*)p;
}

// An empty asm that claims to rewrite v, which keeps the compiler from
// moving the arithmetic around it.
__device__ __forceinline__ void pin(v4f& v) { asm volatile("" : "+v"(v)); }

// Tile number -> (tile row, tile column): each XCD gets a contiguous range,
// walked in groups of eight tile rows.
__device__ __forceinline__ void tile_of(int64_t bid, int64_t nbid, int64_t ntm, int64_t ntn, int64_t& tm, int64_t& tn) {
  int64_t t = bid;
  if ((nbid & 7) == 0) t = (bid & 7) * (nbid >> 3) + (bid >> 3);
  const int64_t per_group = 8 * ntn, g = t / per_group, first = 8 * g;
  const int64_t gs = (ntm - first) < 8 ? (ntm - first) : 8, r = t - g * per_group;
  tm = first + r % gs;
  tn = r / gs;
}

// Four consecutive elements of an output row from one lane; `vec`: the row
// pieces are aligned for one store.
template <typename T>
__device__ __forceinline__ void store_row4(T* dst, v4f v, int64_t left, bool vec) {
  if constexpr (sizeof(T) == 4) {
    if (vec && left >= 4) {
      *(v4f*)dst = v;
      return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (e < left) dst[e] = v[e];
  } else {
    const uint32_t a = pk_bf16(v[0], v[1]), b = pk_bf16(v[2], v[3]);
    if (vec && left >= 4) {
      *(u32x2*)dst = u32x2{a, b};
      return;
    }
    if (left > 0) dst[0] = (T)a;
    if (left > 1) dst[1] = (T)(a >> 16);
    if (left > 2) dst[2] = (T)b;
    if (left > 3) dst[3] = (T)(b >> 16);
  }
}

}  // namespace ffn
}  // namespace fp8q

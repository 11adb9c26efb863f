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
// f with the activation as a constant: the choice is made once around a
// loop, so that the exponentials of its elements overlap.
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

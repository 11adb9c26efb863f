// Gradient of the linear layer at its pre-activations, quantized for the two
// products that follow, with the bias's gradient, for gfx950.
//
//   d = dC * act'(v),  dbias[n] = sum_m d[m,n],  h = act(v)
//
// from dC [M, N] and the forward's bf16 pre-activations v [M, N].  One pass
// leaves d as 1x128 codes along features (the operand of dA = d B), the codes
// of its transpose along tokens (the operand of dB = d^T A), the sums of each
// 128 tokens for the bias and, recomputed, the codes of h^T along tokens (the
// operand of the next layer's weight gradient).  Nothing wide is written: 4
// bytes are read and 3 written per element (bf16, h asked for).
//   8192 x 18432, GELU, h asked for: 1.07 GB in 213 to 221 us + 5 for the bias's
//   sum (4.9 TB/s; 173 us at an elementwise pass's 6.19): the vector ALU is busy
//   88 % of it, some 43 instructions an element for the activation with its
//   derivative and three quantized outputs.  1000 x 4096 ReLU fp32 without h:
//   9.7 + 1.6 us (33 MB, 5.4 us): one turn of latency and the second launch.
//
// A workgroup of 512 threads takes 128 tokens x 128 features, so both kinds
// of block lie inside it.  Thread (rg, cl) holds tokens 4rg .. 4rg + 3 and
// features 8cl .. 8cl + 7: 16 lanes make a row's maximum by DPP; a column's
// maximum and sum are made over the thread's tokens, the four row groups of
// the wavefront and the eight wavefronts (LDS), always in that order; and its
// four tokens' codes of a column are one dword of the transposed tile in LDS,
// which leaves in 128-byte pieces.  Rows past M count as zeros: the transposed
// outputs are whole 128-token blocks, their padding zero codes.
#include "fp8q_mfma.h"

namespace fp8q {

using namespace ffn;

// Dword of the transposed tile that holds tokens 4rg .. 4rg+3 of feature c.
// Four neighbouring dwords (one 16-byte read) stay together; the XOR spreads
// a write's sixteen features over the banks.
__device__ __forceinline__ int tr_slot(int c, int rg) { return c * 32 + (rg ^ (4 * ((c >> 3) & 7))); }

// NH: 2 with h, 1 without.
template <int DC, int FC, int FH, int NH>
__global__ __launch_bounds__(512, 4) void k_linear_bwd(const LinearBwd p) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[NH][128 * 32];
  __shared__ uint32_t cmax[NH][8][128];
  __shared__ float csum[8][128];
  __shared__ int slow;  // a column's scale needs the division
  __shared__ float2 cs[NH][128];  // a column's scale and its reciprocal, column 8 cl + e at 16 e + cl
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cl = tid & 15, rg = tid >> 4;
  // Order of tiles: each XCD a contiguous part (ids go to the eight in turn),
  // and in it sixteen token blocks of a feature block after one another, whose
  // transposed pieces adjoin.
  const uint32_t nf = (uint32_t)(p.N / 128), nm = (uint32_t)((p.M + 127) / 128);  // fewer than 2^23 tiles
  uint32_t id = blockIdx.x;
  if (nf * nm % 8 == 0) id = (id & 7) * (nf * nm / 8) + (id >> 3);
  const uint32_t grp = id / (16 * nf), r16 = id - grp * 16 * nf, gs = nm - grp * 16 < 16 ? nm - grp * 16 : 16;
  const uint32_t fb = r16 / gs, mb = grp * 16 + r16 % gs;
  const int64_t f0 = (int64_t)fb * 128, m0 = (int64_t)mb * 128;
  const int64_t col = f0 + 8 * cl;

  float v[NH][4][8];  // d, h
  with_linear_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
    constexpr bool PRE = ACT != FP8Q_ACT_NONE || NH == 2;
    Raw8<DC> dc[4];
    Raw8<FP8Q_BF16> g[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // rows past M read the last one; zeros for both make d and h zero
      const int64_t at = m0 + 4 * rg + q, row = at < p.M ? at : p.M - 1;
      dc[q].load(p.dc, row * p.lddc + col);
      if constexpr (PRE) g[q].load(p.pre, row * p.ldpre + col);
    }
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (m0 + 4 * rg + q >= p.M) {
        dc[q].fill(0.0f);
        if constexpr (PRE) g[q].fill(0.0f);
      }
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float h = 0.0f;
        if constexpr (PRE) v[0][q][e] = linear_act_bwd<ACT>(dc[q][e], g[q][e], h);
        else v[0][q][e] = dc[q][e];
        if constexpr (NH == 2) v[1][q][e] = h;
      }
    }
  });

  // along features: four rows' scales, then their codes, by the quick quotient
  // where every lane's scale allows it
  {
    float s[4], r[4];
    bool ok = true;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      float m = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max_abs(m, v[0][q][e]);
      s[q] = block_scale7<FC>(__uint_as_float(canon_abs_bits(row16_max(__float_as_uint(m)))), p.eps);
      r[q] = recip(s[q]);
      ok = ok && scale_ok(s[q]);
    }
    auto codes = [&](auto fast) {
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int64_t row = m0 + 4 * rg + q;
        const float(&x)[8] = v[0][q];
        const bool f = decltype(fast)::value || scale_ok(s[q]);
        const u32x2 w = {encode4<FC>(x[0], x[1], x[2], x[3], s[q], r[q], f),
                         encode4<FC>(x[4], x[5], x[6], x[7], s[q], r[q], f)};
        if (row < p.M) {  // 16 lanes share a row
          __builtin_nontemporal_store(w, (u32x2*)(p.d + row * p.ldd + col));
          if (cl == 0) p.ds[row * p.ld_ds + fb] = s[q];
        }
      }
    };
    if (__all(ok)) codes(std::true_type{});
    else codes(std::false_type{});
  }

  // along tokens.  The wavefront's four row groups meet in its registers: two
  // exchanges of halves and of rows of 16 lanes, each joining two columns at once,
  // leave lane group j with columns 2j and 2j + 1 of the eight.
  auto join = [&](auto op, uint32_t(&x)[8]) {
    uint32_t y[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const auto t = __builtin_amdgcn_permlane32_swap(x[e], x[e + 4], false, false);
      y[e] = op(t[0], t[1]);
    }
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const auto t = __builtin_amdgcn_permlane16_swap(y[e], y[e + 2], false, false);
      x[e] = op(t[0], t[1]);
    }
  };
  const int slot = 32 * (lane >> 4) + cl;  // column 8 cl + e at 16 e + cl
  auto larger = [](uint32_t a, uint32_t b) { return max(a, b); };
  auto added = [](uint32_t a, uint32_t b) { return __float_as_uint(__uint_as_float(a) + __uint_as_float(b)); };
#pragma unroll
  for (int k = 0; k < NH; ++k) {
    uint32_t m[8];
#pragma unroll
    for (int e = 0; e < 8; ++e)
      m[e] = __float_as_uint(max_abs(max_abs(max_abs(__builtin_fabsf(v[k][0][e]), v[k][1][e]), v[k][2][e]), v[k][3][e]));
    join(larger, m);
    cmax[k][wave][slot] = m[0];
    cmax[k][wave][slot + 16] = m[1];
  }
  if (p.ws) {
    uint32_t a[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) a[e] = __float_as_uint((v[0][0][e] + v[0][1][e]) + (v[0][2][e] + v[0][3][e]));
    join(added, a);
    csum[wave][slot] = __uint_as_float(a[0]);
    csum[wave][slot + 16] = __uint_as_float(a[1]);
  }
  if (tid == 0) slow = 0;
  __syncthreads();
  if (tid < 128 * NH) {
    const int k = tid >> 7, c = tid & 127, at = (c & 7) * 16 + (c >> 3);
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, cmax[k][w][at]);
    const float amax = __uint_as_float(canon_abs_bits(m));
    const float s = k == 0 ? block_scale7<FC>(amax, p.eps) : block_scale7<FH>(amax, p.eps);
    cs[k][at] = make_float2(s, recip(s));
    if (!scale_ok(s)) slow = 1;
    if (k == 0) {
      if (p.dt_) p.dts[(f0 + c) * p.ld_dts + mb] = s;
    } else {
      p.hts[(f0 + c) * p.ld_hts + mb] = s;
    }
  } else if (p.ws && tid >= 384) {
    const int c = tid & 127, at = (c & 7) * 16 + (c >> 3);
    float a = 0.0f;
#pragma unroll
    for (int w = 0; w < 8; ++w) a += csum[w][at];
    p.ws[mb * p.N + f0 + c] = a;
  }
  if (!p.dt_ && NH == 1) return;
  __syncthreads();
  auto codes_t = [&](auto fast) {
#pragma unroll
    for (int k = 0; k < NH; ++k)
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float s = cs[k][16 * e + cl].x, r = cs[k][16 * e + cl].y;
        const bool f = decltype(fast)::value || scale_ok(s);
        tile[k][tr_slot(8 * cl + e, rg)] = k == 0 ? encode4<FC>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, f)
                                                  : encode4<FH>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, f);
      }
  };
  if (slow == 0) codes_t(std::true_type{});
  else codes_t(std::false_type{});
  __syncthreads();
#pragma unroll
  for (int k = 0; k < NH; ++k) {
    if (k == 0 && !p.dt_) continue;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int c = it * 64 + (tid >> 3), ch = tid & 7;  // 16 tokens of a feature
      const u32x4 w = *(const u32x4*)&tile[k][tr_slot(c, 4 * ch)];
      uint8_t* dst = k == 0 ? p.dt_ + (f0 + c) * p.lddt : p.ht + (f0 + c) * p.ldht;
      __builtin_nontemporal_store(w, (u32x4*)(dst + m0 + 16 * ch));
    }
  }
}

template <int DC, int FC>
static void launch_f(const LinearBwd& p, hipStream_t st) {
  const dim3 grid((unsigned)(p.N / 128 * ((p.M + 127) / 128))), block(512);
  if (!p.ht) hipLaunchKernelGGL((k_linear_bwd<DC, FC, 0, 1>), grid, block, 0, st, p);
  else if (p.fh == FP8Q_E4M3FN) hipLaunchKernelGGL((k_linear_bwd<DC, FC, FP8Q_E4M3FN, 2>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((k_linear_bwd<DC, FC, FP8Q_E5M2, 2>), grid, block, 0, st, p);
}

int launch_linear_bwd(const LinearBwd& q, hipStream_t st) {
  const int64_t nm = (q.M + 127) / 128;
  // a launch holds fewer than 2^32 threads
  if (q.N / 128 * nm > 0xFFFFFFFFll / 512) return fail(FP8Q_ESHAPE, "linear_bwd_q: more than 2^23-1 tiles of 128 x 128");
  LinearBwd p = q;
  // the sums of 128 tokens: one row of the workspace a block, one alone is the result
  p.ws = !p.dbias ? nullptr : nm == 1 ? p.dbias : p.ws;
  if (p.dc_dt == FP8Q_F32) {
    if (p.fc == FP8Q_E4M3FN) launch_f<FP8Q_F32, FP8Q_E4M3FN>(p, st);
    else launch_f<FP8Q_F32, FP8Q_E5M2>(p, st);
  } else {
    if (p.fc == FP8Q_E4M3FN) launch_f<FP8Q_BF16, FP8Q_E4M3FN>(p, st);
    else launch_f<FP8Q_BF16, FP8Q_E5M2>(p, st);
  }
  if (p.dbias && nm > 1) launch_column_sums(p.ws, nm, p.N, p.N, p.dbias, nullptr, st);
  return check_launch("linear_bwd_q");
}

}  // namespace fp8q

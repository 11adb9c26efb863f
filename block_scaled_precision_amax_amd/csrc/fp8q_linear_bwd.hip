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
  __shared__ float2 cs[NH][128];  // a column's scale and its reciprocal, column 8 cl + e at 16 e + cl
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cl = tid & 15, rg = tid >> 4;
  const int64_t nf = p.N / 128, nm = (p.M + 127) / 128;
  // Order of tiles: each XCD a contiguous part (ids go to the eight in turn),
  // and in it sixteen token blocks of a feature block after one another, whose
  // transposed pieces adjoin.
  int64_t id = blockIdx.x;
  if (nf * nm % 8 == 0) id = (id & 7) * (nf * nm / 8) + (id >> 3);
  const int64_t grp = id / (16 * nf), r16 = id - grp * 16 * nf, gs = nm - grp * 16 < 16 ? nm - grp * 16 : 16;
  const int64_t fb = r16 / gs, mb = grp * 16 + r16 % gs;
  const int64_t f0 = fb * 128, m0 = mb * 128;
  const int64_t col = f0 + 8 * cl;

  float v[NH][4][8];  // d, h
  with_linear_act(p.act, [&](auto act) {
    constexpr int ACT = decltype(act)::value;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // rows past M read the last one, and their values count as zero
      const bool in = m0 + 4 * rg + q < p.M;
      const int64_t row = in ? m0 + 4 * rg + q : p.M - 1;
      Raw8<DC> dc;
      Raw8<FP8Q_BF16> g;
      dc.load(p.dc, row * p.lddc + col);
      if (ACT != FP8Q_ACT_NONE || NH == 2) g.load(p.pre, row * p.ldpre + col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float h = 0.0f;
        const float d = ACT == FP8Q_ACT_NONE && NH == 1 ? dc[e] : linear_act_bwd<ACT>(dc[e], g[e], h);
        v[0][q][e] = in ? d : 0.0f;
        if constexpr (NH == 2) v[1][q][e] = in ? h : 0.0f;
      }
    }
  });

  // along features
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = m0 + 4 * rg + q;
    if (row >= p.M) continue;  // 16 lanes share a row
    const float(&x)[8] = v[0][q];
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[e]));
    const float s = block_scale7<FC>(__uint_as_float(canon_abs_bits(row16_max(m))), p.eps);
    const float r = 1.0f / s;
    const bool fast = scale_ok(s);
    const u32x2 w = {encode4<FC>(x[0], x[1], x[2], x[3], s, r, fast), encode4<FC>(x[4], x[5], x[6], x[7], s, r, fast)};
    __builtin_nontemporal_store(w, (u32x2*)(p.d + row * p.ldd + col));
    if (cl == 0) p.ds[row * p.ld_ds + fb] = s;
  }

  // along tokens
#pragma unroll
  for (int k = 0; k < NH; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t m = max(max(abs_bits(v[k][0][e]), abs_bits(v[k][1][e])), max(abs_bits(v[k][2][e]), abs_bits(v[k][3][e])));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lane < 16) cmax[k][wave][16 * e + cl] = m;
    }
  if (p.ws) {
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      float a = (v[0][0][e] + v[0][1][e]) + (v[0][2][e] + v[0][3][e]);
      a += __shfl_xor(a, 16);
      a += __shfl_xor(a, 32);
      if (lane < 16) csum[wave][16 * e + cl] = a;
    }
  }
  __syncthreads();
  if (tid < 128 * NH) {
    const int k = tid >> 7, c = tid & 127, at = (c & 7) * 16 + (c >> 3);
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, cmax[k][w][at]);
    const float amax = __uint_as_float(canon_abs_bits(m));
    const float s = k == 0 ? block_scale7<FC>(amax, p.eps) : block_scale7<FH>(amax, p.eps);
    cs[k][at] = make_float2(s, 1.0f / s);
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
#pragma unroll
  for (int k = 0; k < NH; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = cs[k][16 * e + cl].x, r = cs[k][16 * e + cl].y;
      const bool fast = scale_ok(s);
      tile[k][tr_slot(8 * cl + e, rg)] = k == 0 ? encode4<FC>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, fast)
                                                : encode4<FH>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, fast);
    }
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

// Gradient of the gated projection at its pre-activations, quantized for the
// two products that follow, for gfx950.
//
//   h = act(g) * u,  dg = dh * u * act'(g),  du = dh * act(g)
//
// from dh [M, F] and the forward's bf16 pre-activations gu = [g | u] [M, 2F].
// One pass leaves [dg | du] as 1x128 codes along features (the operand of
// dX = [dg du] W), the codes of its transpose along tokens (the operand of
// dW = [dg du]^T X) and, recomputed, the codes of h^T along tokens (the
// operand of the down projection's weight gradient).  Nothing wide is
// written: 6 bytes are read and 5 written per element of dh (bf16).  8192 x
// 18432: 390 us, 4.3 TB/s; 65 vector instructions an element keep the ALUs
// busy for some 60% of that, and two workgroups a compute unit (their
// registers and LDS) overlap only so much of the rest.
//
// A workgroup of 512 threads takes 128 tokens x 128 features, so both kinds
// of block lie inside it.  Thread (rg, cl) holds tokens 4rg .. 4rg + 3 and
// features 8cl .. 8cl + 7: 16 lanes make a row's maximum by DPP, a column's
// is made over the thread's tokens, the four row groups of the wavefront and
// the eight wavefronts (LDS), and its four tokens' codes of a column are one
// dword of the transposed tile in LDS, which leaves in 128-byte pieces.
// Rows past M count as zeros: the transposed outputs are whole 128-token
// blocks, their padding zero codes.
#include "fp8q_mfma.h"

namespace fp8q {

using namespace ffn;

// Dword of the transposed tile that holds tokens 4rg .. 4rg+3 of feature c.
// Four neighbouring dwords (one 16-byte read) stay together; the XOR spreads
// a write's sixteen features over the banks.
__device__ __forceinline__ int tr_slot(int c, int rg) { return c * 32 + (rg ^ (4 * ((c >> 3) & 7))); }

template <int DH, int FC, int FH>
__global__ __launch_bounds__(512, 4) void k_glu_bwd(const GluBwd p) {
  __shared__ __attribute__((aligned(16))) uint32_t tile[3][128 * 32];
  __shared__ uint32_t cmax[3][8][128];
  __shared__ float2 cs[3][128];  // a column's scale and its reciprocal, column 8 cl + e at 16 e + cl
  const int tid = threadIdx.x, lane = tid & 63;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int cl = tid & 15, rg = tid >> 4;
  const int64_t nf = p.F / 128, nm = (p.M + 127) / 128;
  // Order of tiles: each XCD a contiguous part (ids go to the eight in turn),
  // and in it sixteen token blocks of a feature block after one another, whose
  // transposed pieces adjoin (8192 x 18432: 385 us against 404 along features).
  int64_t id = blockIdx.x;
  if (nf * nm % 8 == 0) id = (id & 7) * (nf * nm / 8) + (id >> 3);
  const int64_t grp = id / (16 * nf), r16 = id - grp * 16 * nf, gs = nm - grp * 16 < 16 ? nm - grp * 16 : 16;
  const int64_t fb = r16 / gs, mb = grp * 16 + r16 % gs;
  const int64_t f0 = fb * 128, m0 = mb * 128;
  const int64_t col = f0 + 8 * cl;

  float v[3][4][8];  // dg, du, h
  with_activation(p.act, [&](auto act) {
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      // rows past M read the last one, and their values count as zero
      const bool in = m0 + 4 * rg + q < p.M;
      const int64_t row = in ? m0 + 4 * rg + q : p.M - 1;
      Raw8<DH> dh;
      Raw8<FP8Q_BF16> g, u;
      dh.load(p.dh, row * p.lddh + col);
      g.load(p.gu, row * p.ldgu + col);
      u.load(p.gu, row * p.ldgu + p.F + col);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        float da;
        const float a = activation<decltype(act)::value, true>(g[e], da);
        v[0][q][e] = in ? dh[e] * u[e] * da : 0.0f;
        v[1][q][e] = in ? dh[e] * a : 0.0f;
        v[2][q][e] = in ? a * u[e] : 0.0f;
      }
    }
  });

  // along features
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const int64_t row = m0 + 4 * rg + q;
    if (row >= p.M) continue;  // 16 lanes share a row
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float(&x)[8] = v[k][q];
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e) m = max(m, abs_bits(x[e]));
      const float s = block_scale7<FC>(__uint_as_float(canon_abs_bits(row16_max(m))), p.eps);
      const float r = 1.0f / s;
      const bool fast = scale_ok(s);
      const u32x2 w = {encode4<FC>(x[0], x[1], x[2], x[3], s, r, fast), encode4<FC>(x[4], x[5], x[6], x[7], s, r, fast)};
      __builtin_nontemporal_store(w, (u32x2*)(p.d + row * p.ldd + k * p.F + col));
      if (cl == 0) p.ds[row * p.ld_ds + ((k * p.F + f0) >> 7)] = s;
    }
  }
  if (!p.dt_ && !p.ht) return;

  // along tokens
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      uint32_t m = max(max(abs_bits(v[k][0][e]), abs_bits(v[k][1][e])), max(abs_bits(v[k][2][e]), abs_bits(v[k][3][e])));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lane < 16) cmax[k][wave][16 * e + cl] = m;
    }
  __syncthreads();
  if (tid < 384) {
    const int k = tid >> 7, c = tid & 127;
    uint32_t m = 0;
#pragma unroll
    for (int w = 0; w < 8; ++w) m = max(m, cmax[k][w][(c & 7) * 16 + (c >> 3)]);
    const float amax = __uint_as_float(canon_abs_bits(m));
    const float s = k < 2 ? block_scale7<FC>(amax, p.eps) : block_scale7<FH>(amax, p.eps);
    cs[k][(c & 7) * 16 + (c >> 3)] = make_float2(s, 1.0f / s);
    if (k < 2) {
      if (p.dt_) p.dts[(k * p.F + f0 + c) * p.ld_dts + mb] = s;
    } else if (p.ht) {
      p.hts[(f0 + c) * p.ld_hts + mb] = s;
    }
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k)
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const float s = cs[k][16 * e + cl].x, r = cs[k][16 * e + cl].y;
      const bool fast = scale_ok(s);
      tile[k][tr_slot(8 * cl + e, rg)] =
          k < 2 ? encode4<FC>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, fast)
                : encode4<FH>(v[k][0][e], v[k][1][e], v[k][2][e], v[k][3][e], s, r, fast);
    }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    if (k < 2 ? !p.dt_ : !p.ht) continue;
#pragma unroll
    for (int it = 0; it < 2; ++it) {
      const int c = it * 64 + (tid >> 3), ch = tid & 7;  // 16 tokens of a feature
      const u32x4 w = *(const u32x4*)&tile[k][tr_slot(c, 4 * ch)];
      uint8_t* dst = k < 2 ? p.dt_ + (k * p.F + f0 + c) * p.lddt : p.ht + (f0 + c) * p.ldht;
      __builtin_nontemporal_store(w, (u32x4*)(dst + m0 + 16 * ch));
    }
  }
}

template <int DH, int FC, int FH>
static void launch_t(const GluBwd& p, hipStream_t st) {
  hipLaunchKernelGGL((k_glu_bwd<DH, FC, FH>), dim3((unsigned)(p.F / 128 * ((p.M + 127) / 128))), dim3(512), 0, st, p);
}

template <int DH>
static void launch_f(const GluBwd& p, hipStream_t st) {
  if (p.fc == FP8Q_E4M3FN) {
    if (p.fh == FP8Q_E4M3FN) launch_t<DH, 0, 0>(p, st);
    else launch_t<DH, 0, 1>(p, st);
  } else {
    if (p.fh == FP8Q_E4M3FN) launch_t<DH, 1, 0>(p, st);
    else launch_t<DH, 1, 1>(p, st);
  }
}

int launch_glu_bwd(const GluBwd& p, hipStream_t st) {
  // a launch holds fewer than 2^32 threads
  if (p.F / 128 * ((p.M + 127) / 128) > 0xFFFFFFFFll / 512)
    return fail(FP8Q_ESHAPE, "glu_bwd_q: more than 2^23-1 tiles of 128 x 128");
  if (p.dh_dt == FP8Q_F32) launch_f<FP8Q_F32>(p, st);
  else launch_f<FP8Q_BF16>(p, st);
  return check_launch("glu_bwd_q");
}

}  // namespace fp8q

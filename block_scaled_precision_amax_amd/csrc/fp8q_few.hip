// Block-scaled products of a few rows (single tokens, decoding batches) for
// gfx950: a plain product C = A B^T and the gated projection
// h = act(A Bg^T) * (A Bu^T).
//
//   C[m,n] = sum_kb sA[m,kb] sB(n,kb) P_kb[m,n],
//   P_kb[m,n] = sum_{k in block kb} dec(A[m,k]) dec(B[n,k])
//
// With M <= 64 rows the weight's bytes are the work: each is read once, at
// 2 M flop a byte, so the kernel is a stream of B through the matrix cores.
// A wavefront takes 16 rows of B (of Bg and of Bu) and every KS-th block of
// 128 K; its lanes load 32 consecutive bytes of their row straight into
// registers (four lanes cover a 128-byte line), decode them without loss and
// multiply against the same block of A, which stays in the caches.
// Everything after the decode is fp32: products of two codes are exact, each
// block sum is folded into an fp32 accumulator with its scales.
//
// The sum over K blocks is the same for every split: block kb belongs to
// class kb % 8, the blocks of a class are added in order, and the eight
// classes are joined as ((0+1)+(2+3))+((4+5)+(6+7)).  KS = 8 wavefronts take
// a class each; KS = 2 take four each and join them in registers.  So the
// quantized output holds the codes of exactly the fp32 values that the
// unquantized one stores.
#include "fp8q_mfma.h"

namespace fp8q {

using namespace ffn;

static constexpr int kClasses = 8;

__device__ __forceinline__ v4f add4(v4f a, v4f b) {
  return v4f{a[0] + b[0], a[1] + b[1], a[2] + b[2], a[3] + b[3]};
}

// KS wavefronts share the K blocks of NCG groups of 16 columns; RT tiles of
// 16 rows.  OUT: FP8Q_F32, FP8Q_BF16, or 2 + format for 1x128 codes (NCG = 8:
// a workgroup then holds the 128 columns of a block).
template <int FA, int FB, int GB, bool GLU, int OUT, int NCG, int KS, int RT>
__global__ __launch_bounds__(64 * NCG * KS) void k_few(const Proj p) {
  constexpr bool H16 = FA == FP8Q_E5M2 || FB == FP8Q_E5M2;
  constexpr int NJ = GLU ? 2 : 1;
  using V8 = typename Op<H16>::v8;
  __shared__ __attribute__((aligned(16))) v4f red[KS][NCG][RT][NJ][64];
  __shared__ uint32_t rmax[OUT >= 2 ? NCG : 1][RT * 16];
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = wave / KS, ks = wave % KS;
  const int64_t n0 = ((int64_t)blockIdx.x * NCG + cg) * 16;
  const int64_t m0 = (int64_t)blockIdx.y * (RT * 16);
  const int nkb = (int)(p.K / 128);

  // the lane's row of B and rows of A; past the edge the last row is read
  // (its results are never stored)
  const int64_t bn = n0 + lr < p.N ? n0 + lr : p.N - 1;
  const uint8_t* b[NJ];
  b[0] = p.B0 + bn * p.ldb + 32 * lq;
  if constexpr (GLU) b[1] = p.B1 + bn * p.ldb + 32 * lq;
  const uint8_t* a[RT];
  const float* sa[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    const int64_t m = m0 + 16 * i + lr < p.M ? m0 + 16 * i + lr : p.M - 1;
    a[i] = p.A + m * p.lda + 32 * lq;
    sa[i] = p.sA + m * p.sA_sm;
  }
  const int64_t nb = n0 < p.N ? n0 : p.N - 1;
  const float* sb[NJ];
  sb[0] = p.s0 + (nb >> 7) * p.sB_sn;
  if constexpr (GLU) sb[1] = p.s1 + (nb >> 7) * p.sB_sn;
  // 1x128 scales: the lane's four columns
  const float* sbn[4];
  if constexpr (GB == FP8Q_GRAN_1x128) {
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t n = n0 + 4 * lq + e;
      sbn[e] = p.s0 + (n < p.N ? n : p.N - 1) * p.sB_sn;
    }
  }

  constexpr int CL = kClasses / KS;  // classes of this wavefront: CL * ks ..
  static_assert(CL == 1 || CL == 4, "the join below");
  v4f acc[RT][NJ], sum[CL > 1 ? 2 : 1][RT][NJ];
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) f(i, j);
  };
#pragma unroll
  for (int t = 0; t < CL; ++t) {
  each([&](int i, int j) { acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f}; });
  for (int kb = CL * ks + t; kb < nkb; kb += kClasses) {
    u32x4 rb[NJ][2];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      const u32x4* q = (const u32x4*)(b[j] + (int64_t)kb * 128);
      rb[j][0] = __builtin_nontemporal_load(q);
      rb[j][1] = __builtin_nontemporal_load(q + 1);
    }
    V8 fb[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) fb[j][k] = dec8<FB, H16>(rb[j][k >> 1][2 * (k & 1)], rb[j][k >> 1][2 * (k & 1) + 1]);
    float sbv[NJ];
    v4f sb4;
    if constexpr (GB == FP8Q_GRAN_1x128) {
#pragma unroll
      for (int e = 0; e < 4; ++e) sb4[e] = sbn[e][kb * p.sB_skb];
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) sbv[j] = sb[j][kb * p.sB_skb];
    }
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      const u32x4* q = (const u32x4*)(a[i] + (int64_t)kb * 128);
      const u32x4 r0 = q[0], r1 = q[1];
      const float s = sa[i][kb * p.sA_skb];
      V8 fa[4];
      fa[0] = dec8<FA, H16>(r0.x, r0.y);
      fa[1] = dec8<FA, H16>(r0.z, r0.w);
      fa[2] = dec8<FA, H16>(r1.x, r1.y);
      fa[3] = dec8<FA, H16>(r1.z, r1.w);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        // B first: the lane gets row 16i + lr and columns 4lq .. 4lq + 3
        v4f t = v4f{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
        for (int k = 0; k < 4; ++k) t = mfma32<H16>(fb[j][k], fa[k], t);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(t[e], s * (GB == FP8Q_GRAN_1x128 ? sb4[e] : sbv[j]), acc[i][j][e]);
      }
    }
  }
  each([&](int i, int j) {
    if constexpr (CL == 1) {
      sum[0][i][j] = acc[i][j];
    } else {
      if (t & 1) sum[t >> 1][i][j] = add4(sum[t >> 1][i][j], acc[i][j]);
      else sum[t >> 1][i][j] = acc[i][j];
      if (t == 3) sum[0][i][j] = add4(sum[0][i][j], sum[1][i][j]);
    }
  });
  }
  each([&](int i, int j) { red[ks][cg][i][j][lane] = sum[0][i][j]; });
  __syncthreads();

  // wavefront ks of a column group finishes row tiles ks, ks + KS, ...
  constexpr int IT = (RT + KS - 1) / KS;
  v4f h[IT];
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    const int i = u * KS + ks;
    h[u] = v4f{0.0f, 0.0f, 0.0f, 0.0f};
    if (i >= RT) continue;
    v4f s[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v4f o[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) o[k] = red[k][cg][i][j][lane];
#pragma unroll
      for (int w = 1; w < KS; w *= 2)
#pragma unroll
        for (int k = 0; k + w < KS; k += 2 * w) o[k] = add4(o[k], o[k + w]);
      s[j] = o[0];
    }
    const int64_t row = m0 + 16 * i + lr, col = n0 + 4 * lq;
    const bool in = row < p.M && col < p.N;
    if constexpr (GLU) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[u][e] = activation(p.act, s[0][e]) * s[1][e];
      if (p.gu && in) {
        uint16_t* g = p.gu + row * p.ldgu + col;
        const bool vec = ((((uintptr_t)p.gu) | (uintptr_t)(2 * p.ldgu) | (uintptr_t)(2 * p.N)) & 7) == 0;
        store_row4(g, s[0], p.N - col, vec);
        store_row4(g + p.N, s[1], p.N - col, vec);
      }
    } else {
      h[u] = s[0];
    }
    if constexpr (OUT == FP8Q_F32) {
      const bool vec = ((((uintptr_t)p.out) | (uintptr_t)(4 * p.ldo)) & 15) == 0;
      if (in) store_row4((float*)p.out + row * p.ldo + col, h[u], p.N - col, vec);
    } else if constexpr (OUT == FP8Q_BF16) {
      const bool vec = ((((uintptr_t)p.out) | (uintptr_t)(2 * p.ldo)) & 7) == 0;
      if (in) store_row4((uint16_t*)p.out + row * p.ldo + col, h[u], p.N - col, vec);
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, abs_bits(h[u][e]));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lq == 0) rmax[cg][16 * i + lr] = m;
    }
  }
  if constexpr (OUT >= 2) {
    static_assert(NCG == 8, "a workgroup holds the 128 columns of a block");
    constexpr int QF = OUT - 2;
    __syncthreads();
#pragma unroll
    for (int u = 0; u < IT; ++u) {
      const int i = u * KS + ks;
      if (i >= RT) continue;
      uint32_t m = 0;
#pragma unroll
      for (int c = 0; c < NCG; ++c) m = max(m, rmax[c][16 * i + lr]);
      const float s = block_scale<QF>(__uint_as_float(canon_abs_bits(m)), p.eps);
      const float r = 1.0f / s;
      const int64_t row = m0 + 16 * i + lr;
      if (row >= p.M) continue;
      const uint32_t w = encode4<QF>(h[u][0], h[u][1], h[u][2], h[u][3], s, r, scale_ok(s));
      uint8_t* dst = (uint8_t*)p.out + row * p.ldo + n0 + 4 * lq;
      if ((((uintptr_t)p.out | (uintptr_t)p.ldo) & 3) == 0) {
        *(uint32_t*)dst = w;
      } else {
#pragma unroll
        for (int e = 0; e < 4; ++e) dst[e] = (uint8_t)(w >> (8 * e));
      }
      if (cg == 0 && lq == 0) p.scales[row * p.ld_s + (n0 >> 7)] = s;
    }
  }
}

template <int FA, int FB, int GB, bool GLU, int OUT, int RT>
static void launch_rt(const Proj& p, hipStream_t st) {
  constexpr int NCG = OUT >= 2 ? 8 : 1, KS = OUT >= 2 ? 2 : 8;
  const int64_t gx = (p.N + 16 * NCG - 1) / (16 * NCG), gy = (p.M + 16 * RT - 1) / (16 * RT);
  hipLaunchKernelGGL((k_few<FA, FB, GB, GLU, OUT, NCG, KS, RT>), dim3((unsigned)gx, (unsigned)gy),
                     dim3(64 * NCG * KS), 0, st, p);
}

template <int FA, int FB, int GB, bool GLU, int OUT>
static void launch_m(const Proj& p, hipStream_t st) {
  if (p.M <= 16) launch_rt<FA, FB, GB, GLU, OUT, 1>(p, st);
  else if (p.M <= 32) launch_rt<FA, FB, GB, GLU, OUT, 2>(p, st);
  else launch_rt<FA, FB, GB, GLU, OUT, 4>(p, st);
}

template <int FA, int FB>
static void launch_f(const Proj& p, hipStream_t st) {
  constexpr int BLK = FP8Q_GRAN_128x128;
  if (p.B1) {
    if (p.scales && p.fc == FP8Q_E4M3FN) launch_m<FA, FB, BLK, true, 2 + FP8Q_E4M3FN>(p, st);
    else if (p.scales) launch_m<FA, FB, BLK, true, 2 + FP8Q_E5M2>(p, st);
    else if (p.out_dt == FP8Q_F32) launch_m<FA, FB, BLK, true, FP8Q_F32>(p, st);
    else launch_m<FA, FB, BLK, true, FP8Q_BF16>(p, st);
  } else if (p.gb == FP8Q_GRAN_1x128) {
    if (p.out_dt == FP8Q_F32) launch_m<FA, FB, FP8Q_GRAN_1x128, false, FP8Q_F32>(p, st);
    else launch_m<FA, FB, FP8Q_GRAN_1x128, false, FP8Q_BF16>(p, st);
  } else {
    if (p.out_dt == FP8Q_F32) launch_m<FA, FB, BLK, false, FP8Q_F32>(p, st);
    else launch_m<FA, FB, BLK, false, FP8Q_BF16>(p, st);
  }
}

int launch_few(const Proj& p, const char* what, hipStream_t st) {
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_f<0, 0>(p, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_f<1, 0>(p, st);
  else if (p.fa == FP8Q_E4M3FN) launch_f<0, 1>(p, st);
  else launch_f<1, 1>(p, st);
  return check_launch(what);
}

}  // namespace fp8q

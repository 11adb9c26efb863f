// Block-scaled products of a few rows (single tokens, decoding batches) for
// gfx950: a plain product C = A B^T and the gated projection
// h = act(A Bg^T) * (A Bu^T).
//
//   C[m,n] = sum_kb sA[m,kb] sB(n,kb) P_kb[m,n],
//   P_kb[m,n] = sum_{k in block kb} dec(A[m,k]) dec(B[n,k])
//
// With M <= 64 rows the weight's bytes are the work: each is read once, at
// 2 M flop a byte, so the kernel is a stream of B through the matrix cores.
// A wavefront takes 16 rows of B (of Bg and of Bu) and a share of the blocks
// of 128 K.  A compute unit asks for one 128-byte line at a time, whole or in
// part, and a load that touches sixteen half lines costs sixteen requests
// (24 GB/s a compute unit measured, against 41 with whole lines), so a load
// takes eight rows, eight lanes a line; the rows then change lanes through a
// 2 KB tile of LDS that is the wavefront's own (no barrier), are decoded
// without loss and multiplied against the same block of A.  Loads run PD
// blocks ahead of the arithmetic: a wavefront's own stream has to cover the
// memory's latency.  Everything after the decode is fp32: products of two
// codes are exact, each block sum is folded into an fp32 accumulator with its
// scales.
//
// The sum over K blocks is the same for every split: block kb belongs to
// class kb % 8, the blocks of a class are added in order, and the classes are
// joined as (((0+1)+2)+3) + (((4+5)+6)+7).  KS wavefronts share the classes
// and join their own in registers, the rest in LDS, so the quantized output
// holds the codes of exactly the fp32 values that the unquantized one stores.
#include "fp8q_mfma.h"

#include <type_traits>

namespace fp8q {

using namespace ffn;

static constexpr int kClasses = 8;
// K blocks whose A scales a workgroup keeps in LDS.  Read where they are
// used, they cost a request per lane and block (sixteen rows, a line each),
// more than A itself; K beyond this (20480) reads them so.
static constexpr int kScaleBlocks = 160;

__device__ __forceinline__ v4f add4(v4f a, v4f b) {
  return v4f{a[0] + b[0], a[1] + b[1], a[2] + b[2], a[3] + b[3]};
}

// KS wavefronts share the K blocks of a group of 16 NJ columns (GLU: 16 of g
// and of u, NJ = 2); NCG such groups a workgroup; RT tiles of 16 rows.  OUT:
// FP8Q_F32, FP8Q_BF16, or 2 + format for 1x128 codes (NCG = 8: a workgroup
// then holds the 128 columns of a block).
template <int FA, int FB, int GB, bool GLU, int OUT, int NJ, int NCG, int KS, int RT, int PD>
__global__ __launch_bounds__(64 * NCG * KS) void k_few(const Proj p) {
  constexpr bool H16 = FA == FP8Q_E5M2 || FB == FP8Q_E5M2;
  constexpr int GC = GLU ? 16 : 16 * NJ;  // columns of a group
  using V8 = typename Op<H16>::v8;
  // the wavefronts' exchange tiles (NJ of B, RT of A), then their partial sums
  constexpr int XCH = NCG * KS * (NJ + RT) * 2048, RED = KS * NCG * RT * NJ * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[XCH > RED ? XCH : RED];
  __shared__ uint32_t rmax[OUT >= 2 ? NCG : 1][RT * 16];
  constexpr int SP = RT * 16 + 1;  // [block][row], padded for the writes
  __shared__ float sa_lds[kScaleBlocks * SP];
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int cg = wave / KS, ks = wave % KS;
  const int64_t n0 = ((int64_t)blockIdx.x * NCG + cg) * GC;
  const int nkb = (int)(p.K / 128);

  // the lane's rows of B and of A, l / 8 and 8 + l / 8 of a tile, and its
  // 16-byte chunk l % 8 of them; past the edge the last row is read (its
  // results are never stored)
  const int xr = lane >> 3, xc = lane & 7;
  auto clampn = [&](int64_t n) { return n < p.N ? n : p.N - 1; };
  const uint8_t* b[NJ][2];
  const float* sb[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t c0 = GLU ? n0 : n0 + 16 * j;
#pragma unroll
    for (int v = 0; v < 2; ++v) b[j][v] = (GLU && j ? p.B1 : p.B0) + clampn(c0 + 8 * v + xr) * p.ldb + 16 * xc;
    // 1x128 scales: the lane's four columns start at sb[j]
    sb[j] = (GLU && j ? p.s1 : p.s0) + (GB == FP8Q_GRAN_1x128 ? 0 : (clampn(c0) >> 7) * p.sB_sn);
  }
  const uint8_t* a[RT][2];
  const float* sa[RT];
  int srow[RT];
#pragma unroll
  for (int i = 0; i < RT; ++i) {
    auto clampm = [&](int64_t m) { return m < p.M ? m : p.M - 1; };
#pragma unroll
    for (int v = 0; v < 2; ++v) a[i][v] = p.A + clampm(16 * i + 8 * v + xr) * p.lda + 16 * xc;
    srow[i] = (int)clampm(16 * i + lr);
    sa[i] = p.sA + srow[i] * p.sA_sm;
  }
  // exchange: chunk c of row r in slot swz_chunk(r, c) of the row
  uint8_t* const xch = lds + wave * (NJ + RT) * 2048;
  const int w0 = xr * 128 + 16 * swz_chunk(xr, xc), w1 = (8 + xr) * 128 + 16 * swz_chunk(8 + xr, xc);
  const int r0 = lr * 128 + 16 * swz_chunk(lr, 2 * lq), r1 = lr * 128 + 16 * swz_chunk(lr, 2 * lq + 1);

  struct Stage {
    u32x4 rb[NJ][2], ra[RT][2];
    float sb[NJ][GB == FP8Q_GRAN_1x128 ? 4 : 1];
  };
  Stage ring[PD];
  auto load_b = [&](Stage& g, int kb) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int v = 0; v < 2; ++v) g.rb[j][v] = __builtin_nontemporal_load((const u32x4*)(b[j][v] + (int64_t)kb * 128));
      if constexpr (GB == FP8Q_GRAN_1x128) {
#pragma unroll
        for (int e = 0; e < 4; ++e) g.sb[j][e] = sb[j][clampn(n0 + 16 * j + 4 * lq + e) * p.sB_sn + kb * p.sB_skb];
      } else {
        g.sb[j][0] = sb[j][kb * p.sB_skb];
      }
    }
  };
  auto load_a = [&](Stage& g, int kb) {
#pragma unroll
    for (int i = 0; i < RT; ++i) {
#pragma unroll
      for (int v = 0; v < 2; ++v) g.ra[i][v] = *(const u32x4*)(a[i][v] + (int64_t)kb * 128);
    }
  };
  auto load = [&](Stage& g, int kb) {
    load_b(g, kb);
    load_a(g, kb);
  };

  constexpr int CL = kClasses / KS;  // classes CL * ks .. of this wavefront
  static_assert(CL == 1 || CL == 4 || CL == 8, "the joins below");
  // the next block of the wavefront: its class's next, or the first of its
  // next class (nkb: none is left)
  auto next = [&](int kb) {
    if (kb + kClasses < nkb) return kb + kClasses;
    const int c = (kb & (kClasses - 1)) + 1;
    return c < CL * (ks + 1) && c < nkb ? c : nkb;
  };
  v4f acc[RT][NJ], sum[CL == 8 ? 2 : 1][RT][NJ];
  auto each = [&](auto f) {
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int j = 0; j < NJ; ++j) f(i, j);
  };
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  each([&](int i, int j) {
    acc[i][j] = zero;
    sum[0][i][j] = zero;
    if (CL == 8) sum[CL == 8][i][j] = zero;
  });

  // One block: its rows go to the exchange tiles, which frees the registers
  // for the block PD ahead (`ahead` loads it), then the products.
  auto put = [&](const u32x4* raw, int slot) {
    *(u32x4*)(xch + slot * 2048 + w0) = raw[0];
    *(u32x4*)(xch + slot * 2048 + w1) = raw[1];
  };
  // lane (lr, lq) gets bytes 32 lq .. + 32 of row lr, 8 of them for each MFMA
  auto get = [&](int slot, auto fmt, V8* f) {
    constexpr int FM = decltype(fmt)::value;
    const u32x4 x0 = *(const u32x4*)(xch + slot * 2048 + r0), x1 = *(const u32x4*)(xch + slot * 2048 + r1);
    f[0] = dec8<FM, H16>(x0.x, x0.y);
    f[1] = dec8<FM, H16>(x0.z, x0.w);
    f[2] = dec8<FM, H16>(x1.x, x1.y);
    f[3] = dec8<FM, H16>(x1.z, x1.w);
  };
  const bool sa_in_lds = nkb <= kScaleBlocks;
  auto consume = [&](Stage& g, int kb, auto ahead) {
    float s[RT][NJ][GB == FP8Q_GRAN_1x128 ? 4 : 1];
#pragma unroll
    for (int j = 0; j < NJ; ++j) put(g.rb[j], j);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      put(g.ra[i], NJ + i);
      const float sai = sa_in_lds ? sa_lds[kb * SP + srow[i]] : sa[i][kb * p.sA_skb];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < (GB == FP8Q_GRAN_1x128 ? 4 : 1); ++e) s[i][j][e] = sai * g.sb[j][e];
    }
    // the lanes read each other's rows; the wavefront's LDS accesses run in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    ahead();
    V8 fb[NJ][4];
#pragma unroll
    for (int j = 0; j < NJ; ++j) get(j, std::integral_constant<int, FB>{}, fb[j]);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      V8 fa[4];
      get(NJ + i, std::integral_constant<int, FA>{}, fa);
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        // B first: the lane gets row 16i + lr and columns 4lq .. 4lq + 3
        v4f t = zero;
#pragma unroll
        for (int k = 0; k < 4; ++k) t = mfma32<H16>(fb[j][k], fa[k], t);
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc[i][j][e] = __builtin_fmaf(t[e], s[i][j][GB == FP8Q_GRAN_1x128 ? e : 0], acc[i][j][e]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");  // read before the next block's rows
  };

  int kp = CL * ks;  // the next block to load
  if (kp > nkb) kp = nkb;
#pragma unroll
  for (int u = 0; u < PD; ++u) {
    if (kp < nkb) {
      load(ring[u], kp);
      kp = next(kp);
    }
  }
  if (sa_in_lds) {
#pragma unroll 4
    for (int t = threadIdx.x; t < (int)p.M * nkb; t += 64 * NCG * KS) {
      const int r = t / nkb, kb = t - r * nkb;
      sa_lds[kb * SP + r] = p.sA[r * p.sA_sm + kb * p.sA_skb];
    }
  }
  __syncthreads();
  for (int kb = CL * ks; kb < nkb;) {
#pragma unroll
    for (int u = 0; u < PD; ++u) {
      if (kb >= nkb) break;
      consume(ring[u], kb, [&] {
        if (kp < nkb) {
          load(ring[u], kp);
          kp = next(kp);
        }
      });
      const int nx = next(kb);
      if constexpr (CL > 1) {
        if (kb + kClasses >= nkb) {  // the class ends
          const bool second = CL == 8 && (kb & 4);
          each([&](int i, int j) {
            if (second) sum[CL == 8][i][j] = add4(sum[CL == 8][i][j], acc[i][j]);
            else sum[0][i][j] = add4(sum[0][i][j], acc[i][j]);
            acc[i][j] = zero;
          });
        }
      }
      kb = nx;
    }
  }
  __syncthreads();  // the exchange tiles become the partial sums
  v4f(*red)[NCG][RT][NJ][64] = (v4f(*)[NCG][RT][NJ][64])lds;
  each([&](int i, int j) {
    red[ks][cg][i][j][lane] = CL == 1 ? acc[i][j] : CL == 4 ? sum[0][i][j] : add4(sum[0][i][j], sum[CL == 8][i][j]);
  });
  __syncthreads();

  // wavefront ks of a column group finishes row tiles ks, ks + KS, ...
  constexpr int IT = (RT + KS - 1) / KS;
  constexpr int NH = GLU ? 1 : NJ;  // column tiles of the output
  v4f h[IT][NH];
#pragma unroll
  for (int u = 0; u < IT; ++u) {
    const int i = u * KS + ks;
    h[u][0] = zero;
    if (i >= RT) continue;
    v4f s[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      v4f o[KS];
#pragma unroll
      for (int k = 0; k < KS; ++k) o[k] = red[k][cg][i][j][lane];
      if constexpr (KS == 8) {
#pragma unroll
        for (int k = 1; k < 4; ++k) o[0] = add4(o[0], o[k]), o[4] = add4(o[4], o[4 + k]);
        o[0] = add4(o[0], o[4]);
      } else if constexpr (KS == 2) {
        o[0] = add4(o[0], o[1]);
      }
      s[j] = o[0];
    }
    const int64_t row = 16 * i + lr, col = n0 + 4 * lq;
    const bool in = row < p.M && col < p.N;
    if constexpr (GLU) {
#pragma unroll
      for (int e = 0; e < 4; ++e) h[u][0][e] = activation(p.act, s[0][e]) * s[1][e];
      if (p.gu && in) {
        uint16_t* g = p.gu + row * p.ldgu + col;
        const bool vec = ((((uintptr_t)p.gu) | (uintptr_t)(2 * p.ldgu) | (uintptr_t)(2 * p.N)) & 7) == 0;
        store_row4(g, s[0], p.N - col, vec);
        store_row4(g + p.N, s[1], p.N - col, vec);
      }
    } else {
#pragma unroll
      for (int j = 0; j < NJ; ++j) h[u][j] = s[j];
    }
    if constexpr (OUT < 2) {
      using T = std::conditional_t<OUT == FP8Q_F32, float, uint16_t>;
      const bool vec = ((((uintptr_t)p.out) | (uintptr_t)(sizeof(T) * p.ldo)) & (4 * sizeof(T) - 1)) == 0;
      if (row < p.M) {
#pragma unroll
        for (int j = 0; j < NH; ++j)
          if (col + 16 * j < p.N) store_row4((T*)p.out + row * p.ldo + col + 16 * j, h[u][j], p.N - col - 16 * j, vec);
      }
    } else {
      uint32_t m = 0;
#pragma unroll
      for (int e = 0; e < 4; ++e) m = max(m, abs_bits(h[u][0][e]));
      m = max(m, (uint32_t)__shfl_xor((int)m, 16));
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      if (lq == 0) rmax[cg][16 * i + lr] = m;
    }
  }
  if constexpr (OUT >= 2) {
    static_assert(GLU && NCG == 8, "a workgroup holds the 128 columns of a block");
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
      const int64_t row = 16 * i + lr;
      if (row >= p.M) continue;
      const uint32_t w = encode4<QF>(h[u][0][0], h[u][0][1], h[u][0][2], h[u][0][3], s, r, scale_ok(s));
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

template <int FA, int FB, int GB, bool GLU, int OUT, int NJ, int RT>
static void launch_rt(const Proj& p, hipStream_t st) {
  // codes: 16 wavefronts where their registers suffice
  #ifndef V_KSQ
#define V_KSQ 2
#define V_PDQ 1
#define V_PD1 1
#define V_PDN 1
#endif
  #ifndef V_NJ
#define V_NJ 2
#endif
  constexpr int NCG = OUT >= 2 ? 8 : 1, KS = OUT < 2 ? 8 : RT == 1 ? V_KSQ : 1, PD = RT == 1 ? (OUT >= 2 ? V_PDQ : V_PD1) : V_PDN;
  constexpr int COLS = NCG * (GLU ? 16 : 16 * NJ);
  hipLaunchKernelGGL((k_few<FA, FB, GB, GLU, OUT, NJ, NCG, KS, RT, PD>), dim3((unsigned)((p.N + COLS - 1) / COLS)),
                     dim3(64 * NCG * KS), 0, st, p);
}

template <int FA, int FB, int GB, bool GLU, int OUT>
static void launch_m(const Proj& p, hipStream_t st) {
  // a plain product of more rows shares each tile of A among 32 columns
  if (p.M <= 16) launch_rt<FA, FB, GB, GLU, OUT, GLU ? 2 : 1, 1>(p, st);
  else if (p.M <= 32) launch_rt<FA, FB, GB, GLU, OUT, 2, 2>(p, st);
  else if (p.M <= 48) launch_rt<FA, FB, GB, GLU, OUT, 2, 3>(p, st);
  else launch_rt<FA, FB, GB, GLU, OUT, 2, 4>(p, st);
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

// Tiles of block-scaled FP8 products: their shape and the loop over K that
// fills a tile's accumulators.  Shared by the gated projection (fp8q_glu.hip)
// and the linear layer (fp8q_linear.h).
//
// fast: 256 rows (or 128), v_mfma_scale_f32_16x16x128_f8f6f4 on the codes;
// exact: 128 rows (or 64), codes decoded to bf16 / f16 without loss and
// multiplied exactly (fp32 sums) by v_mfma_f32_16x16x32.  256 columns of B in
// all.  Every P_kb is folded into fp32 accumulators with one FMA per element.
#pragma once

#include "fp8q_mfma.h"

namespace fp8q {

using namespace ffn;

static constexpr int BK = 128;
static constexpr int kThreads = 512;
static constexpr int TJ = 4;

template <bool FAST, int TI_>
struct Shape {
  static constexpr int TI = TI_, BM = 32 * TI, NST = TI == 8 ? 2 : 3;
  static constexpr int A_STAGE = BM * BK, B_STAGE = 256 * BK;
  static constexpr int LDS = NST * (A_STAGE + B_STAGE);
};

// The block sums of one tile, folded into acc: rows m0 .. m0 + BM of A against
// 128 rows n0 .. of B0 and the same rows of B1 (PAIR) or 256 rows of B0, K
// blocks kb0 .. nkb - 1 (one at least).  Eight wavefronts (2 x 4), each TI x 4
// tiles of 16 x 16: column tiles 0, 1 of the first 128 columns and 2, 3 of the
// others; lane (lr, lq) gets row 16 (wm TI + i) + lr and columns 32 wn + 16 (j & 1)
// + 4 lq .. + 3.  lds: the stages (1024-byte aligned), free to write on entry;
// after the last block other wavefronts may still read them.
template <int FA, int FB, bool FAST, int TI, bool PAIR>
__device__ __forceinline__ void tile_product(const Proj& p, const float* __restrict__ s0, const float* __restrict__ s1,
                                             uint8_t* lds, float (*lds_sa)[32 * TI], int tid, int64_t m0, int64_t n0,
                                             int64_t kb0, int64_t nkb, v4f (&acc)[TI][TJ]) {
  using S = Shape<FAST, TI>;
  constexpr int BM = S::BM, NST = S::NST;
  constexpr int B0 = NST * S::A_STAGE;  // the B stages follow the A stages
  const uint32_t lds_at = lds_addr_of(lds), sa_at = lds_addr_of(lds_sa);
  const int64_t M = p.M, N = p.N;
  const int lane = tid & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int wm = wave >> 2, wn = wave & 3;

  // Copies: a copy stalls the wavefront that issues it, so wavefronts 0-3
  // issue all of them and 4-7, on the same SIMDs, go on with MFMAs.
  // Wavefront w takes rows (w, w + 4) * BM/8 .. of A, rows 32w .. of each half
  // of B (of two matrices the same offsets) and the A scales of its rows.  Lane l of an
  // eight-row piece fills slot l % 8 of row l / 8.  Rows past an edge read
  // the last row (their results are never stored).
  constexpr int NA = BM / 64, SAL = BM / 8;
  uint32_t a_off[2][NA], b_off[4], b_off1[4];
  auto off = [&](int64_t r0, int r, int64_t rows, int64_t ld) {
    const int64_t g = r0 + r < rows ? r0 + r : rows - 1;
    return (uint32_t)(g * ld + 16 * swz_chunk(r, lane & 7));
  };
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int q = 0; q < NA; ++q)
      a_off[h][q] = off(m0, (((wave & 3) + 4 * h) * NA + q) * 8 + (lane >> 3), M, p.lda);
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    b_off[q] = off(n0, ((wave & 3) * 4 + q) * 8 + (lane >> 3), N, p.ldb);
    b_off1[q] = PAIR ? b_off[q] : off(n0 + 128, ((wave & 3) * 4 + q) * 8 + (lane >> 3), N, p.ldb);
  }
  // A scales in the order the lanes read them: slot h*16TI + lr*TI + i
  // holds row h*16TI + 16i + lr
  const float* sa_row[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const int s = ((wave & 3) + 4 * h) * SAL + (lane < SAL ? lane : 0);
    const int64_t r = m0 + (s / (16 * TI)) * 16 * TI + 16 * (s % TI) + (s % (16 * TI)) / TI;
    sa_row[h] = p.sA + (r < M ? r : M - 1) * p.sA_sm;
  }
  constexpr int NW = 2 * NA + 8 + 2;  // copies per copying wavefront and block
  auto stage_block = [&](int64_t kb, int st) {
    if (wm != 0) return;
    const uint8_t *a = p.A + kb * BK, *g = p.B0 + kb * BK, *u = p.B1 + kb * BK;
    const uint32_t la = lds_at + st * S::A_STAGE, lb = lds_at + B0 + st * S::B_STAGE;
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int q = 0; q < NA; ++q)
        lds_dma16(__builtin_amdgcn_readfirstlane(la + ((wave + 4 * h) * NA + q) * 1024), a, a_off[h][q]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      lds_dma16(__builtin_amdgcn_readfirstlane(lb + (wave * 4 + q) * 1024), g, b_off[q]);
      lds_dma16(__builtin_amdgcn_readfirstlane(lb + (16 + wave * 4 + q) * 1024), u, b_off1[q]);
    }
    if (lane < SAL) {
#pragma unroll
      for (int h = 0; h < 2; ++h)
        lds_dma4(__builtin_amdgcn_readfirstlane(sa_at + 4 * (st * BM + (wave + 4 * h) * SAL)), sa_row[h] + kb * p.sA_skb);
    }
  };

#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < TJ; ++j) acc[i][j] = v4f{0.0f, 0.0f, 0.0f, 0.0f};

  const int a_row0 = (wm * TI * 16 + lr) * BK;
  auto b_row = [&](int j) { return ((j >> 1) * 128 + 32 * wn + 16 * (j & 1) + lr) * BK; };
  const int o0 = 16 * swz_chunk(lr, 2 * lq), o1 = 16 * swz_chunk(lr, 2 * lq + 1);
  // every column of the tile lies in one 128-column block of scales; they
  // are read by scalar loads (restrict arguments): a vector load here would
  // wait for every copy in flight
  const float* sg = s0 + (n0 >> 7) * p.sB_sn;
  const int64_t nu = PAIR ? n0 : n0 + 128 < N ? n0 + 128 : N - 1;
  const float* su = s1 + (nu >> 7) * p.sB_sn;

  constexpr bool H16 = FA == FP8Q_E5M2 || FB == FP8Q_E5M2;
  using V8 = typename Op<H16>::v8;
  using V2 = typename Op<H16>::v2;
  V8 xfb[FAST ? 1 : TJ][4], xfa[4];  // exact path: decoded fragments carried to the next block

  // One block: its products folded into acc.  The MFMAs take B first, so a
  // lane gets row 16i + lr and columns 4lq .. 4lq + 3 of a tile.  The fold of
  // row tile i - 1 runs in the shadow of row tile i's MFMAs.  PF (exact
  // path): before the last row tile the next block is published and its
  // first fragments are decoded behind that tile's MFMAs.
  auto compute = [&](int64_t kb, int s, auto pf_tag, int nxt, bool wait_all) {
    constexpr bool PF = decltype(pf_tag)::value;
    const float fg = sg[kb * p.sB_skb], fu = su[kb * p.sB_skb];
    const uint8_t* la = lds + s * S::A_STAGE + a_row0;
    const uint8_t* lb = lds + B0 + s * S::B_STAGE;
    float cf[TI];
    const float* lc = lds_sa[s] + wm * TI * 16 + lr * TI;
#pragma unroll
    for (int q = 0; q < TI / 2; ++q) {
      const float2 c2 = *(const float2*)(lc + 2 * q);
      cf[2 * q] = c2.x, cf[2 * q + 1] = c2.y;
    }
    float cg[TI], cu[TI];
#pragma unroll
    for (int i = 0; i < TI; ++i) cg[i] = cf[i] * fg, cu[i] = cf[i] * fu;
    auto fold = [&](int i, int j, int e, float v) {
      acc[i][j][e] = __builtin_fmaf(v, j < 2 ? cg[i] : cu[i], acc[i][j][e]);
    };
    v4f pp[TJ], pn[TJ];
    if constexpr (FAST) {
      auto frag = [&](const uint8_t* base) {
        const u32x4 x0 = *(const u32x4*)(base + o0);
        const u32x4 x1 = *(const u32x4*)(base + o1);
        return v8i{(int)x0.x, (int)x0.y, (int)x0.z, (int)x0.w, (int)x1.x, (int)x1.y, (int)x1.z, (int)x1.w};
      };
      v8i fb[TJ];
#pragma unroll
      for (int j = 0; j < TJ; ++j) fb[j] = frag(lb + b_row(j));
      v8i fa = frag(la), fn = fa;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        if (i + 1 < TI) fn = frag(la + 16 * (i + 1) * BK);
#pragma unroll
        for (int j = 0; j < TJ; ++j) {
          pn[j] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(fb[j], fa, v4f{0.0f, 0.0f, 0.0f, 0.0f}, FB, FA, 0, 0,
                                                                  0, 0);
          pin(pn[j]);
          if (i > 0) {
#pragma unroll
            for (int e = 0; e < 4; ++e) fold(i - 1, j, e, pp[j][e]);
            pin(acc[i - 1][j]);
          }
          __builtin_amdgcn_sched_barrier(0);
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) pp[j] = pn[j];
        fa = fn;
      }
    } else {
      // lane group lq owns bytes 32lq .. +32 of the block for the four
      // MFMAs, bytes 8k .. +8 of them going to MFMA k; A and B alike
      auto raw32 = [&](const uint8_t* base, u32x2* r) {
        const u32x4 x0 = *(const u32x4*)(base + o0);
        const u32x4 x1 = *(const u32x4*)(base + o1);
        r[0] = u32x2{x0.x, x0.y};
        r[1] = u32x2{x0.z, x0.w};
        r[2] = u32x2{x1.x, x1.y};
        r[3] = u32x2{x1.z, x1.w};
      };
      V8 fa[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) fa[k] = xfa[k];
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        u32x2 raw[4], rb[TJ][4], ra[4];
        if (i + 1 < TI) raw32(la + 16 * (i + 1) * BK, raw);
        if constexpr (PF) {
          // every read of stage s precedes this barrier
          if (i + 1 == TI) {
            if (wait_all)
              asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
            else
              asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NW) : "memory");
            __syncthreads();
            const uint8_t* lbn = lds + B0 + nxt * S::B_STAGE;
#pragma unroll
            for (int j = 0; j < TJ; ++j) raw32(lbn + b_row(j), rb[j]);
            raw32(lds + nxt * S::A_STAGE + a_row0, ra);
          }
        }
        V2 part[4][4];
#pragma unroll
        for (int k = 0; k < 4; ++k)
#pragma unroll
          for (int j = 0; j < TJ; ++j) {
            pn[j] = mfma32<H16>(xfb[j][k], fa[k], k == 0 ? v4f{0.0f, 0.0f, 0.0f, 0.0f} : pn[j]);
            if (i > 0) fold(i - 1, j, k, pp[j][k]);
            if (i + 1 < TI) {
              const uint32_t w = (j & 2) ? raw[k].y : raw[k].x;
              part[k][j] = (j & 1) ? dec2<FA, H16, true>(w) : dec2<FA, H16, false>(w);
            } else if constexpr (PF) {
              xfb[j][k] = dec8<FB, H16>(rb[j][k].x, rb[j][k].y);
              if (j + 1 == TJ) xfa[k] = dec8<FA, H16>(ra[k].x, ra[k].y);
            }
          }
        if (i + 1 < TI) {
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            V8 f;
#pragma unroll
            for (int q = 0; q < 4; ++q) f[2 * q] = part[k][q][0], f[2 * q + 1] = part[k][q][1];
            fa[k] = f;
          }
        }
#pragma unroll
        for (int j = 0; j < TJ; ++j) pp[j] = pn[j];
      }
    }
#pragma unroll
    for (int j = 0; j < TJ; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) fold(TI - 1, j, e, pp[j][e]);
  };
  auto next_stage = [](int st) { return st + 1 == NST ? 0 : st + 1; };
  using PF1 = std::integral_constant<bool, true>;
  using PF0 = std::integral_constant<bool, false>;

  // Prologue: the first NST - 1 blocks in flight, wait for block 0.
  stage_block(kb0, 0);
  if (NST == 3 && kb0 + 1 < nkb) {
    stage_block(kb0 + 1, 1);
    asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NW) : "memory");
  } else {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  __syncthreads();
  int st = 0;
  int64_t kb = kb0;
  if constexpr (FAST && NST == 2) {
    for (; kb + 1 < nkb; ++kb) {
      stage_block(kb + 1, next_stage(st));
      compute(kb, st, PF0{}, 0, true);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      st = next_stage(st);
    }
  } else if constexpr (FAST) {
    // two blocks in flight: block kb + 2 goes into the stage that block
    // kb - 1 left at the last barrier
    for (; kb + 2 < nkb; ++kb) {
      const int s1 = next_stage(st);
      stage_block(kb + 2, next_stage(s1));
      compute(kb, st, PF0{}, 0, true);
      asm volatile("s_waitcnt vmcnt(%0)" ::"n"(NW) : "memory");
      __syncthreads();
      st = s1;
    }
    if (kb + 1 < nkb) {
      compute(kb, st, PF0{}, 0, true);
      asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
      __syncthreads();
      st = next_stage(st);
      ++kb;
    }
  } else {
    auto dec32 = [&](const uint8_t* base, auto fmt, V8* out) {
      constexpr int FM = decltype(fmt)::value;
      const u32x4 x0 = *(const u32x4*)(base + o0);
      const u32x4 x1 = *(const u32x4*)(base + o1);
      out[0] = dec8<FM, H16>(x0.x, x0.y);
      out[1] = dec8<FM, H16>(x0.z, x0.w);
      out[2] = dec8<FM, H16>(x1.x, x1.y);
      out[3] = dec8<FM, H16>(x1.z, x1.w);
    };
#pragma unroll
    for (int j = 0; j < TJ; ++j) dec32(lds + B0 + b_row(j), std::integral_constant<int, FB>{}, xfb[FAST ? 0 : j]);
    dec32(lds + a_row0, std::integral_constant<int, FA>{}, xfa);
    for (; kb + 2 < nkb; ++kb) {
      const int s1 = next_stage(st), s2 = next_stage(s1);
      stage_block(kb + 2, s2);
      compute(kb, st, PF1{}, s1, false);
      st = s1;
    }
    if (kb + 1 < nkb) {
      compute(kb, st, PF1{}, next_stage(st), true);
      st = next_stage(st);
      ++kb;
    }
  }
  compute(kb, st, PF0{}, 0, true);

}

// Workgroups of a launch: one per compute unit, a multiple of eight so that a
// workgroup's tiles stay on its XCD.
static int64_t grid_size() {
  const int64_t g = device_cu_count() / 8 * 8;
  return g < 8 ? 8 : g;
}

}  // namespace fp8q

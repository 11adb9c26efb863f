// Gated projection h = act(A Bg^T) * (A Bu^T) on block-scaled FP8 operands
// for gfx950, many rows (a few rows go to fp8q_few.hip).
//
//   g[m,f] = sum_kb sA[m,kb] sBg(f,kb) P_kb,  u likewise with Bu,
//   P_kb = sum over the 128 k of a block of dec(a) dec(b),
//   h = act(g) * u
//
// One kernel computes both products of a tile: its B tile holds 128 rows of
// Bg and the same 128 rows of Bu, and a wavefront owns matching columns of
// both, so g and u of an element end in one lane and neither is written
// (unless asked for, as bf16).  The A tile is read once for both.
//
// Paths and tiling are those of the block-scaled GEMM.  fast: 256 rows x 128
// h columns, v_mfma_scale_f32_16x16x128_f8f6f4 on the codes; exact: 128 x
// 128, codes decoded to bf16 / f16 without loss and multiplied exactly
// (fp32 sums) by v_mfma_f32_16x16x32.  Eight wavefronts (2 x 4), each TI x 4
// tiles of 16 x 16: column tiles 0, 1 of g and 2, 3 of u.  Every P_kb is
// folded into fp32 accumulators with one FMA per element.
//
// Measured at 16384 x 18432 x 7168: fast 3.58 ms (2420 TFLOP/s), 3.74 ms with g
// and u kept; the tiles' 56 blocks take 95 us of a tile's 103, bound by MFMA
// and LDS issue, the rest is the epilogue.  Exact 4096 x 18432 x 7168: 1.81 ms
// (1196 TFLOP/s), bound by the decodes beside the bf16 MFMAs.
#include "fp8q_tiles.h"

namespace fp8q {

// The tiles of one launch: `count` from number `first` of the ntm x ntn tile
// grid, or (halves) both halves of count / 2 tiles of twice this height.
struct Part {
  int64_t ntm, ntn, first, count;
  bool halves;
};

// A BM x 128 tile of T through LDS: `put` is called for the lane's 4-column
// pieces, then whole rows leave 16 bytes a lane.  Chunk c of row r sits in
// slot c ^ (r & 15), so the sixteen rows of a write fall on different banks.
template <typename T, int TI, typename F>
__device__ __forceinline__ void stage_tile(uint8_t* stg, int wm, int wn, int lr, int lq, F value) {
  constexpr int EPC = 16 / (int)sizeof(T);
#pragma unroll
  for (int i = 0; i < TI; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int r = (wm * TI + i) * 16 + lr, col = 32 * wn + 16 * j + 4 * lq;
      T* d = (T*)stg + r * 128 + EPC * ((col / EPC) ^ (r & 15)) + col % EPC;
      const v4f v = value(i, j);
      if constexpr (sizeof(T) == 2)
        *(u32x2*)d = u32x2{pk_bf16(v[0], v[1]), pk_bf16(v[2], v[3])};
      else
        *(v4f*)d = v;
    }
}
template <typename T, int BM>
__device__ __forceinline__ void drain_tile(const uint8_t* stg, int tid, T* out, int64_t ldo, int64_t m0, int64_t n0,
                                           int64_t M, int64_t N) {
  constexpr int EPC = 16 / (int)sizeof(T), CH = 128 / EPC, RPI = kThreads / CH;
  const bool vec = (((uintptr_t)out | (uintptr_t)(ldo * sizeof(T))) & 15) == 0;
  const int c = tid % CH;
  const int64_t col = n0 + EPC * c;
#pragma unroll 4
  for (int it = 0; it < BM / RPI; ++it) {
    const int r = it * RPI + tid / CH;
    const u32x4 v = *(const u32x4*)((const T*)stg + r * 128 + EPC * (c ^ (r & 15)));
    const int64_t row = m0 + r;
    if (row >= M || col >= N) continue;
    T* dst = out + row * ldo + col;
    if (vec && col + EPC <= N) {
      __builtin_nontemporal_store(v, (u32x4*)dst);
    } else {
#pragma unroll
      for (int q = 0; q < EPC; ++q) {
        if (col + q >= N) continue;
        if constexpr (sizeof(T) == 2)
          dst[q] = (T)(v[q >> 1] >> (16 * (q & 1)));
        else
          dst[q] = __uint_as_float(v[q]);
      }
    }
  }
}

// OUT: FP8Q_F32, FP8Q_BF16 or 2 + format (1x128 codes).  GLU false: a plain
// product, whose tiles are 256 columns of one matrix (B1 and its scales are
// B0's, 128 columns on).
template <int FA, int FB, int OUT, bool FAST, int TI_, bool GLU>
__global__ __launch_bounds__(kThreads, 1) void k_glu(const Proj p, const float* __restrict__ s0,
                                                     const float* __restrict__ s1, const Part t) {
  using S = Shape<FAST, TI_>;
  constexpr int TI = S::TI, BM = S::BM, NST = S::NST;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ __attribute__((aligned(16))) float lds_sa[NST][BM];
  __shared__ uint32_t lds_rmax[OUT >= 2 ? 4 : 1][OUT >= 2 ? BM : 1];
  const int64_t M = p.M, N = p.N, nkb = p.K / BK;

  for (int64_t tile = blockIdx.x; tile < t.count; tile += gridDim.x) {
    // derived again for every tile: hoisted, it all stays live and spills
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int64_t tm, tn;
    tile_of(t.first + (t.halves ? tile >> 1 : tile), t.ntm * t.ntn, t.ntm, t.ntn, tm, tn);
    const int64_t m0 = t.halves ? (2 * tm + (tile & 1)) * BM : tm * BM, n0 = tn * (GLU ? 128 : 256);
    if (m0 >= M) continue;  // the lower half of a ragged tile

    v4f acc[TI][TJ];
    tile_product<FA, FB, FAST, TI, GLU>(p, s0, s1, lds, lds_sa, tid, m0, n0, 0, nkb, acc);

    // ---- epilogue, through the LDS of the stages
    __syncthreads();
    auto gate = [&](int i, int j) { return acc[i][j]; };
    auto up = [&](int i, int j) { return acc[i][j + 2]; };
    if (GLU && p.gu) {
      stage_tile<uint16_t, TI>(lds, wm, wn, lr, lq, gate);
      stage_tile<uint16_t, TI>(lds + BM * 256, wm, wn, lr, lq, up);
      __syncthreads();
      drain_tile<uint16_t, BM>(lds, tid, p.gu, p.ldgu, m0, n0, M, N);
      drain_tile<uint16_t, BM>(lds + BM * 256, tid, p.gu + N, p.ldgu, m0, n0, M, N);
      __syncthreads();
    }
    if constexpr (GLU) {
      with_activation(p.act, [&](auto act) {
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int e = 0; e < 4; ++e)
              acc[i][j][e] = activation<decltype(act)::value>(acc[i][j][e]) * acc[i][j + 2][e];
      });
    }
    if constexpr (OUT < 2) {
      using T = std::conditional_t<OUT == FP8Q_F32, float, uint16_t>;
      stage_tile<T, TI>(lds, wm, wn, lr, lq, gate);
      __syncthreads();
      drain_tile<T, BM>(lds, tid, (T*)p.out, p.ldo, m0, n0, M, N);
      if constexpr (!GLU) {
        __syncthreads();
        stage_tile<T, TI>(lds, wm, wn, lr, lq, up);
        __syncthreads();
        drain_tile<T, BM>(lds, tid, (T*)p.out, p.ldo, m0, n0 + 128, M, N);
      }
    } else {
      // a row's 128 columns lie in four wavefronts: their maxima meet in LDS
      constexpr int QF = OUT - 2;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        uint32_t m = 0;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int e = 0; e < 4; ++e) m = max(m, abs_bits(acc[i][j][e]));
        m = max(m, (uint32_t)__shfl_xor((int)m, 16));
        m = max(m, (uint32_t)__shfl_xor((int)m, 32));
        if (lq == 0) lds_rmax[wn][(wm * TI + i) * 16 + lr] = m;
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        const int r = (wm * TI + i) * 16 + lr;
        const uint32_t m = max(max(lds_rmax[0][r], lds_rmax[1][r]), max(lds_rmax[2][r], lds_rmax[3][r]));
        const float s = block_scale7<QF>(__uint_as_float(canon_abs_bits(m)), p.eps);
        const float inv = 1.0f / s;
        if (wn == 0 && lq == 0 && m0 + r < M) p.scales[(m0 + r) * p.ld_s + (n0 >> 7)] = s;
#pragma unroll
        for (int j = 0; j < 2; ++j)
          // chunk c of a 128-byte row in slot c ^ ((r >> 1) & 7)
          *(uint32_t*)(lds + r * 128 + 16 * ((2 * wn + j) ^ ((r >> 1) & 7)) + 4 * lq) =
              encode4<QF>(acc[i][j][0], acc[i][j][1], acc[i][j][2], acc[i][j][3], s, inv, scale_ok(s));
      }
      __syncthreads();
      uint8_t* out = (uint8_t*)p.out;
      const bool vec = (((uintptr_t)out | (uintptr_t)p.ldo) & 15) == 0;
#pragma unroll
      for (int it = 0; it < BM / 64; ++it) {
        const int r = it * 64 + (tid >> 3), c = tid & 7;
        const u32x4 v = *(const u32x4*)(lds + r * 128 + 16 * (c ^ ((r >> 1) & 7)));
        if (m0 + r >= M) continue;
        uint8_t* dst = out + (m0 + r) * p.ldo + n0 + 16 * c;  // N is a multiple of 128
        if (vec) {
          __builtin_nontemporal_store(v, (u32x4*)dst);
        } else {
#pragma unroll
          for (int q = 0; q < 16; ++q) dst[q] = (uint8_t)(v[q >> 2] >> (8 * (q & 3)));
        }
      }
    }
    __syncthreads();  // the epilogue's LDS reads precede the next tile's copies
  }
}

// How a product of ntn tile columns is cut, and what it costs in thousandths
// of a microsecond per K block.  A round of up to a tile per compute unit takes
// 1.4 us a block with tall tiles (256 rows FP8-MFMA, 128 exact) and 0.85 with
// low ones (half the rows) while few units work, 1.7 and 1.05 when all do.
// So: whole rounds of tall tiles, and the rest, if it is at most half a
// round, as a second launch of its halves; or low tiles throughout.
//   exact 1023 x 9000 x 4096 (568 tall tiles): 163 us in three rounds, 146 in
//   two and a round of halves; fast 128 x 18432 x 7168: 94 us tall, 75 low.
struct Cut {
  bool low;       // low tiles throughout
  int64_t tall;   // tall tiles, then
  int64_t split;  // tall tiles taken as halves
  int64_t cost;
};
static Cut cut_tiles(int64_t M, int64_t rows, int64_t ntn, int64_t launch_cost) {
  const int64_t cu = grid_size(), tiles = (M + rows - 1) / rows * ntn;
  const int64_t low = 850 * ((((M + rows / 2 - 1) / (rows / 2)) * ntn + cu - 1) / cu);
  const int64_t full = tiles / cu, rest = tiles - full * cu;
  const bool split = full > 0 && rest > 0 && 2 * rest <= cu && 850 + launch_cost < 1360;
  const int64_t tall = 1360 * full + (rest == 0 ? 0 : split ? 850 + launch_cost : 1360);
  if (low < tall) return {true, 0, 0, low};
  return {false, split ? full * cu : tiles, split ? rest : 0, tall};
}
// A second launch costs about 3 us.
static int64_t second_launch(int64_t K) { return 3000 * 128 / K; }

template <int FA, int FB, int OUT, bool FAST, int TI, bool GLU>
static void launch_part(const Proj& p, const Part& t, hipStream_t st) {
  const int64_t g = grid_size();
  hipLaunchKernelGGL((k_glu<FA, FB, OUT, FAST, TI, GLU>), dim3((unsigned)(t.count < g ? t.count : g)), dim3(kThreads), 0, st,
                     p, p.s0, p.s1, t);
}

template <int FA, int FB, int OUT, bool FAST, bool GLU>
static void launch_cut(const Proj& p, const Cut& c, hipStream_t st) {
  constexpr int TALL = FAST ? 8 : 4, LOW = TALL / 2;
  const int64_t ntn = GLU ? (p.N + 127) / 128 : (p.N + 255) / 256;
  const int64_t ntm = (p.M + 32 * TALL - 1) / (32 * TALL), ltm = (p.M + 32 * LOW - 1) / (32 * LOW);
  if (c.low) {
    launch_part<FA, FB, OUT, FAST, LOW, GLU>(p, {ltm, ntn, 0, ltm * ntn, false}, st);
    return;
  }
  launch_part<FA, FB, OUT, FAST, TALL, GLU>(p, {ntm, ntn, 0, c.tall, false}, st);
  if (c.split) launch_part<FA, FB, OUT, FAST, LOW, GLU>(p, {ntm, ntn, c.tall, 2 * c.split, true}, st);
}

template <int FA, int FB>
static void launch_f(const Proj& p, bool fast, const Cut& c, hipStream_t st) {
  if (p.scales) {
    if (p.fc == FP8Q_E4M3FN) launch_cut<FA, FB, 2 + FP8Q_E4M3FN, false, true>(p, c, st);
    else launch_cut<FA, FB, 2 + FP8Q_E5M2, false, true>(p, c, st);
  } else if (fast) {
    if (p.out_dt == FP8Q_F32) launch_cut<FA, FB, FP8Q_F32, true, true>(p, c, st);
    else launch_cut<FA, FB, FP8Q_BF16, true, true>(p, c, st);
  } else {
    if (p.out_dt == FP8Q_F32) launch_cut<FA, FB, FP8Q_F32, false, true>(p, c, st);
    else launch_cut<FA, FB, FP8Q_BF16, false, true>(p, c, st);
  }
}

// Whether a call takes the few-row kernel, where a workgroup of 16 columns and
// up to 64 rows takes 0.12 us and 0.058 per 16 rows a K block; workgroups per
// compute unit (at least one) x that, against the tiles' cost.  The choice
// goes by M and F alone, so that the workspace does.
//   F = 4096, K = 4096: 10 us at 16 rows and 25 us at 128 against 30 on tiles,
//   48 against 31 us at 256; F = 18432, K = 7168: 45 us at 16 rows and 65 at 32
//   against 60 and 62.
static bool few_rows(int64_t M, int64_t F, bool fast) {
  const int64_t cu = grid_size();
  const int64_t groups = (M + 63) / 64, tiles = ((M + groups - 1) / groups + 15) / 16;
  if (groups > 65535) return false;  // the second dimension of a launch
  int64_t wgs = groups * ((F + 15) / 16);
  if (wgs < cu) wgs = cu;
  return wgs * (120 + 58 * tiles) < cut_tiles(M, fast ? 256 : 128, (F + 127) / 128, 0).cost * cu;
}

int64_t glu_q_workspace(int64_t M, int64_t F) { return few_rows(M, F, false) ? 4 * M * F : 0; }

int launch_glu(const Proj& p, bool fast, const char* what, hipStream_t st) {
  if (few_rows(p.M, p.N, fast)) {
    if (!p.scales) return launch_few(p, nullptr, what, st);
    Proj h = p;
    h.out = p.ws, h.ldo = p.N, h.out_dt = FP8Q_F32, h.scales = nullptr;
    if (int rc = launch_few(h, nullptr, what, st)) return rc;
    return launch_quantize_1x128(p.ws, FP8Q_F32, p.M, p.N, p.N, p.fc, p.eps, (uint8_t*)p.out, p.ldo, p.scales, p.ld_s, st);
  }
  const Cut c = cut_tiles(p.M, fast ? 256 : 128, (p.N + 127) / 128, second_launch(p.K));
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_f<0, 0>(p, fast, c, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_f<1, 0>(p, fast, c, st);
  else if (p.fa == FP8Q_E4M3FN) launch_f<0, 1>(p, fast, c, st);
  else launch_f<1, 1>(p, fast, c, st);
  return check_launch(what);
}

// The block-scaled FP8-MFMA product where whole rounds of 256-row tiles do
// not fit it (the gradients' products: 1000 x 4096 x 8192 has 64 of them).  The
// same instructions in the same order per element as its own kernel, so the
// same bits.
bool gemm_fast_cut(int64_t M, int64_t N, int64_t K) {
  const Cut c = cut_tiles(M, 256, (N + 255) / 256, second_launch(K));
  return c.low || c.split;
}

template <int FA, int FB>
static void launch_product(const Proj& p, const Cut& c, hipStream_t st) {
  if (p.out_dt == FP8Q_F32) launch_cut<FA, FB, FP8Q_F32, true, false>(p, c, st);
  else launch_cut<FA, FB, FP8Q_BF16, true, false>(p, c, st);
}

int launch_gemm_fast_cut(Proj p, const char* what, hipStream_t st) {
  p.B1 = p.B0, p.s1 = p.s0;
  const Cut c = cut_tiles(p.M, 256, (p.N + 255) / 256, second_launch(p.K));
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_product<0, 0>(p, c, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_product<1, 0>(p, c, st);
  else if (p.fa == FP8Q_E4M3FN) launch_product<0, 1>(p, c, st);
  else launch_product<1, 1>(p, c, st);
  return check_launch(what);
}

}  // namespace fp8q

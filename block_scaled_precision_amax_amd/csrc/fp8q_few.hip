// Block-scaled products of a few rows (single tokens, decoding batches) for
// gfx950: a plain product C = A B^T and the gated projection
// h = act(A Bg^T) * (A Bu^T).
//
//   C[m,n] = sum_kb sA[m,kb] sB(n,kb) P_kb[m,n],
//   P_kb[m,n] = sum_{k in block kb} dec(A[m,k]) dec(B[n,k])
//
// With M <= 64 rows the weight's bytes are the work: each is read once, at
// 2 M flop a byte, so the kernel is a stream of B through the matrix cores
// (beyond 64 rows each group of up to 64 reads it again).  7168 x 18432: 22 us at
// one row (6 TB/s), 37 at 48; the gated 18432 x 7168 at one row: 41 us.  Every
// workgroup reads all of A, from the L2, for its 16 or 32 columns: up to 32 rows
// that is at most what it reads of B, at 48 it is half as much again, and there
// 7168 columns also make 224 workgroups for 256 compute units.
// A wavefront takes 16 rows of B (of Bg and of Bu) and a share of the blocks
// of 128 K.  A compute unit asks for one 128-byte line at a time, whole or in
// part, and a load that touches sixteen half lines costs sixteen requests
// (24 GB/s a compute unit measured, against 41 with whole lines), so a load
// takes eight rows, eight lanes a line; the rows then change lanes through a
// 2 KB tile of LDS that is the wavefront's own (no barrier), are decoded
// without loss and multiplied against the same block of A.  The next
// block's loads are issued as soon as this one's rows are in LDS; a deeper
// pipeline cost registers and was slower (21.5 against 23.7 us for 7168 x
// 18432, one row).  Everything after the decode is fp32: products of two
// codes are exact, each block sum is folded into an fp32 accumulator with its
// scales.
//
// Wavefront w of a workgroup adds blocks w, w + 8, ... in order and the eight
// sums are joined in LDS in a fixed order.  The quantized output of the gated
// projection is the same kernel's fp32 output in a workspace and the 1x128
// quantizer: a workgroup that held the 128 columns of a block would leave
// most compute units without work (2048 columns: 16 workgroups, 42 us against
// 12).
#include "fp8q_mfma.h"

namespace fp8q {

using namespace ffn;

static constexpr int kWaves = 8;
// K blocks whose A scales a workgroup keeps in LDS.  Read where they are
// used, they cost a request per lane and block (sixteen rows, a line each),
// more than A itself; K beyond this (20480) reads them so.
static constexpr int kScaleBlocks = 160;

// Eight wavefronts share the K blocks of a group of columns: 16 of g and the
// same 16 of u (GLU, NJ = 2), or 16 NJ columns.  RT tiles of 16 rows.  OUT:
// FP8Q_F32 or FP8Q_BF16.  E: Epilogue for a linear layer, else Nothing (a plain
// product that asks at run time for the parts of an epilogue takes 22.13 us
// instead of 22.02 at one row of 7168 x 18432, 36.56 instead of 36.43 at 48).
struct Nothing {};
template <int FA, int FB, int GB, bool GLU, int OUT, int NJ, int RT, typename E>
__global__ __launch_bounds__(64 * kWaves) void k_few(const Proj p, const E ep) {
  constexpr bool H16 = FA == FP8Q_E5M2 || FB == FP8Q_E5M2;
  constexpr int NS = GB == FP8Q_GRAN_1x128 ? 4 : 1;  // B scales of a lane's four columns
  using V8 = typename Op<H16>::v8;
  // the wavefronts' exchange tiles (NJ of B, RT of A), then their partial sums
  constexpr int XCH = kWaves * (NJ + RT) * 2048, RED = kWaves * RT * NJ * 1024;
  __shared__ __attribute__((aligned(1024))) uint8_t lds[XCH > RED ? XCH : RED];
  constexpr int SP = RT * 16 + 1;  // [block][row], padded for the writes
  __shared__ float sa_lds[kScaleBlocks * SP];
  const int lane = threadIdx.x & 63, lr = lane & 15, lq = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int64_t n0 = (int64_t)blockIdx.x * (GLU ? 16 : 16 * NJ);
  const int64_t m0 = (int64_t)blockIdx.y * (16 * RT);
  const int rows = (int)(p.M - m0 < 16 * RT ? p.M - m0 : 16 * RT);
  const int nkb = (int)(p.K / 128);

  // the lane's rows of B and of A, l / 8 and 8 + l / 8 of a tile, and its
  // 16-byte chunk l % 8 of them; past the edge the last row is read (its
  // results are never stored)
  const int xr = lane >> 3, xc = lane & 7;
  auto clampn = [&](int64_t n) { return n < p.N ? n : p.N - 1; };
  auto clampm = [&](int m) { return m < rows ? m : rows - 1; };
  const uint8_t *b[NJ][2], *a[RT][2];
  const float *sb[NJ], *sa[RT];
  int srow[RT];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    const int64_t c0 = GLU ? n0 : n0 + 16 * j;
#pragma unroll
    for (int v = 0; v < 2; ++v) b[j][v] = (GLU && j ? p.B1 : p.B0) + clampn(c0 + 8 * v + xr) * p.ldb + 16 * xc;
    sb[j] = (GLU && j ? p.s1 : p.s0) + (NS == 4 ? 0 : (clampn(c0) >> 7) * p.sB_sn);
  }
#pragma unroll
  for (int i = 0; i < RT; ++i) {
#pragma unroll
    for (int v = 0; v < 2; ++v) a[i][v] = p.A + (m0 + clampm(16 * i + 8 * v + xr)) * p.lda + 16 * xc;
    srow[i] = clampm(16 * i + lr);
    sa[i] = p.sA + (m0 + srow[i]) * p.sA_sm;
  }
  // exchange: chunk c of row r in slot swz_chunk(r, c) of the row
  uint8_t* const xch = lds + wave * (NJ + RT) * 2048;
  const int w0 = xr * 128 + 16 * swz_chunk(xr, xc), w1 = (8 + xr) * 128 + 16 * swz_chunk(8 + xr, xc);
  const int r0 = lr * 128 + 16 * swz_chunk(lr, 2 * lq), r1 = lr * 128 + 16 * swz_chunk(lr, 2 * lq + 1);

  u32x4 rb[NJ][2], ra[RT][2];
  float sbv[NJ][NS];
  auto load = [&](int kb) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
#pragma unroll
      for (int v = 0; v < 2; ++v) rb[j][v] = __builtin_nontemporal_load((const u32x4*)(b[j][v] + (int64_t)kb * 128));
#pragma unroll
      for (int e = 0; e < NS; ++e)
        sbv[j][e] = sb[j][(NS == 4 ? clampn(n0 + 16 * j + 4 * lq + e) * p.sB_sn : 0) + kb * p.sB_skb];
    }
#pragma unroll
    for (int i = 0; i < RT; ++i)
#pragma unroll
      for (int v = 0; v < 2; ++v) ra[i][v] = *(const u32x4*)(a[i][v] + (int64_t)kb * 128);
  };
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

  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  v4f acc[RT][NJ];
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) acc[i][j] = zero;

  if (wave < nkb) load(wave);
  const bool sa_in_lds = nkb <= kScaleBlocks;
  if (sa_in_lds) {
#pragma unroll 4
    for (int t = threadIdx.x; t < rows * nkb; t += 64 * kWaves) {
      const int r = t / nkb, kb = t - r * nkb;
      sa_lds[kb * SP + r] = p.sA[(m0 + r) * p.sA_sm + kb * p.sA_skb];
    }
  }
  __syncthreads();
  for (int kb = wave; kb < nkb; kb += kWaves) {
    float s[RT][NJ][NS];
#pragma unroll
    for (int j = 0; j < NJ; ++j) put(rb[j], j);
#pragma unroll
    for (int i = 0; i < RT; ++i) {
      put(ra[i], NJ + i);
      const float sai = sa_in_lds ? sa_lds[kb * SP + srow[i]] : sa[i][kb * p.sA_skb];
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < NS; ++e) s[i][j][e] = sai * sbv[j][e];
    }
    // the lanes read each other's rows; the wavefront's LDS accesses run in order
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");
    if (kb + kWaves < nkb) load(kb + kWaves);
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
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(t[e], s[i][j][NS == 4 ? e : 0], acc[i][j][e]);
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront", "local");  // read before the next block's rows
  }

  __syncthreads();  // the exchange tiles become the partial sums
  v4f(*red)[RT][NJ][64] = (v4f(*)[RT][NJ][64])lds;
#pragma unroll
  for (int i = 0; i < RT; ++i)
#pragma unroll
    for (int j = 0; j < NJ; ++j) red[wave][i][j][lane] = acc[i][j];
  __syncthreads();

  // wavefront i finishes row tile i
  const int i = wave;
  const int64_t row = m0 + 16 * i + lr, col = n0 + 4 * lq;
  if (i >= RT || row >= p.M) return;
  v4f o[NJ];
#pragma unroll
  for (int j = 0; j < NJ; ++j) {
    o[j] = red[0][i][j][lane];
#pragma unroll
    for (int k = 1; k < kWaves; ++k) {
      const v4f v = red[k][i][j][lane];
#pragma unroll
      for (int e = 0; e < 4; ++e) o[j][e] += v[e];
    }
  }
  if constexpr (GLU) {
    if (p.gu && col < p.N) {
      uint16_t* g = p.gu + row * p.ldgu + col;
      const bool vec = ((((uintptr_t)p.gu) | (uintptr_t)(2 * p.ldgu) | (uintptr_t)(2 * p.N)) & 7) == 0;
      store_row4(g, o[0], p.N - col, vec);
      store_row4(g + p.N, o[1], p.N - col, vec);
    }
    with_activation(p.act, [&](auto act) {
#pragma unroll
      for (int e = 0; e < 4; ++e) o[0][e] = activation<decltype(act)::value>(o[0][e]) * o[1][e];
    });
  }
  using T = std::conditional_t<OUT == FP8Q_F32, float, uint16_t>;
  if constexpr (std::is_same_v<E, Epilogue>) {
    // four columns a lane, whatever their alignment
    if (ep.bias) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int64_t c = clampn(col + 16 * j + e);
          o[j][e] += ep.bdt == FP8Q_F32 ? ((const float*)ep.bias)[c] : bf_lo(((const uint16_t*)ep.bias)[c]);
        }
    }
    if (ep.pre) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
        if (col + 16 * j < p.N) store_row4(ep.pre + row * ep.ldpre + col + 16 * j, o[j], p.N - col - 16 * j, ep.vp);
    }
    with_linear_act(ep.act, [&](auto act) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[j][e] = linear_act<decltype(act)::value>(o[j][e]);
    });
    if (ep.res) {
#pragma unroll
      for (int j = 0; j < NJ; ++j)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const T r = ((const T*)ep.res)[row * ep.ldr + clampn(col + 16 * j + e)];
          if constexpr (OUT == FP8Q_F32) o[j][e] += r;
          else o[j][e] += bf_lo(r);
        }
    }
  }
  const bool vec = ((((uintptr_t)p.out) | (uintptr_t)(sizeof(T) * p.ldo)) & (4 * sizeof(T) - 1)) == 0;
#pragma unroll
  for (int j = 0; j < (GLU ? 1 : NJ); ++j)
    if (col + 16 * j < p.N) store_row4((T*)p.out + row * p.ldo + col + 16 * j, o[j], p.N - col - 16 * j, vec);
}

template <int FA, int FB, int GB, bool GLU, int OUT, int NJ, int RT, typename E>
static void launch_rt(const Proj& p, const E& e, hipStream_t st) {
  constexpr int COLS = GLU ? 16 : 16 * NJ, ROWS = 16 * RT;
  hipLaunchKernelGGL((k_few<FA, FB, GB, GLU, OUT, NJ, RT, E>),
                     dim3((unsigned)((p.N + COLS - 1) / COLS), (unsigned)((p.M + ROWS - 1) / ROWS)), dim3(64 * kWaves), 0,
                     st, p, e);
}

template <int FA, int FB, int GB, bool GLU, int OUT, typename E>
static void launch_m(const Proj& p, const E& e, hipStream_t st) {
  // a plain product of more than 16 rows shares each tile of A among 32
  // columns; beyond 64 rows, equal groups of up to 64 each read the weight
  const int64_t groups = (p.M + 63) / 64, rows = (p.M + groups - 1) / groups;
  if (p.M <= 16) launch_rt<FA, FB, GB, GLU, OUT, GLU ? 2 : 1, 1>(p, e, st);
  else if (rows <= 32) launch_rt<FA, FB, GB, GLU, OUT, 2, 2>(p, e, st);
  else if (rows <= 48) launch_rt<FA, FB, GB, GLU, OUT, 2, 3>(p, e, st);
  else launch_rt<FA, FB, GB, GLU, OUT, 2, 4>(p, e, st);
}

template <int FA, int FB, int GB, bool GLU, typename E>
static void launch_out(const Proj& p, const E& e, hipStream_t st) {
  if (p.out_dt == FP8Q_F32) launch_m<FA, FB, GB, GLU, FP8Q_F32>(p, e, st);
  else launch_m<FA, FB, GB, GLU, FP8Q_BF16>(p, e, st);
}

template <int FA, int FB>
static void launch_f(const Proj& p, const Epilogue* e, hipStream_t st) {
  constexpr int BLK = FP8Q_GRAN_128x128;
  if (e) launch_out<FA, FB, BLK, false>(p, *e, st);
  else if (p.B1) launch_out<FA, FB, BLK, true>(p, Nothing{}, st);
  else if (p.gb == FP8Q_GRAN_1x128) launch_out<FA, FB, FP8Q_GRAN_1x128, false>(p, Nothing{}, st);
  else launch_out<FA, FB, BLK, false>(p, Nothing{}, st);
}

int launch_few(const Proj& p, const Epilogue* e, const char* what, hipStream_t st) {
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_f<0, 0>(p, e, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_f<1, 0>(p, e, st);
  else if (p.fa == FP8Q_E4M3FN) launch_f<0, 1>(p, e, st);
  else launch_f<1, 1>(p, e, st);
  return check_launch(what);
}

}  // namespace fp8q

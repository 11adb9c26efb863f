// Linear layer C = act(A B^T + bias) + residual on block-scaled FP8 operands
// for gfx950, and its form that leaves act(A B^T + bias) as 1x128 codes.
//
//   v[m,n] = sum_kb sA[m,kb] sB(n,kb) P_kb + bias[n],
//   P_kb   = sum over the 128 k of a block of dec(a) dec(b),
//   C = act(v) + res  or  s, q = 1x128 codes of act(v);  pre = bf16(v) on request
//
// Two ways, by the cost of each: the few-row kernel (fp8q_few.hip), and tiles
// with the epilogue behind their last block, where the tiles that do not fill a
// round of the compute units may have K cut into parts: their sums go to a
// workspace and a second kernel joins them, with the same epilogue.
//
// What bounds it, measured:
//   1 x 18432 x 7168, GELU, codes: HBM, 132 MB of weight in 22.6 us of k_few, 4
//     for the epilogue's launch;
//   48 x 7168 x 18432 with residual, exact: 28 us in 9 parts of K (the weight at
//     4.7 TB/s and 12 MB of sums out), 7 to join them;
//   1023 x 9000 x 4096, GELU, exact fp32: 89 to 91 us + 7: 40 blocks of K (the round's 32,
//     and 8 for the 32 tiles left after it, in 4 parts) at 1.5 to 1.6 us; the rest is
//     two starts and a tile's epilogue with nothing beside them;
//   16384 x 18432 x 7168, erf GELU, codes and pre-activations, exact: 3950 to 4160
//     us, 1040 to 1100 TFLOP/s.  By the slope over K 3.9 ms are blocks of K, 1.92 us
//     each where a single round of tiles takes 1.67 (the decode takes the vector
//     ALU's slots, and a long run the clock) and the plain product with codes 1.80;
//     0.27 are the 36 rounds' epilogues with the matrix cores idle, 7.5 us a tile,
//     1.6 of them without bias, activation and pre-activations;
//   the same on FP8-MFMA: 2140 to 2230 us, 1.8 to 2.1 us a block of K and 21 a
//     tile's epilogue, 10 without those three; fp32 instead of codes 2235 to 2260;
//   8192 x 7168 x 18432 with residual, FP8-MFMA: 938 to 969 us + 28 to join the
//     last 128 tiles, 2180 to 2240 TFLOP/s, LDS and matrix issue, clock.
#include "fp8q_linear.h"

namespace fp8q {

// The parts' sum and the epilogue: 16 rows x 128 columns of a tile of 32 TI rows
// a workgroup, eight columns a lane, the parts added in their order.
template <int OUT, int TI>
__global__ __launch_bounds__(256) void k_linear_join(const Proj p, const Epilogue ep, const Split t) {
  constexpr int BM = 32 * TI, PER = 2 * (BM / 16);  // workgroups of a tile
  const int64_t at = blockIdx.x / PER;              // of the tiles in parts
  const int g = blockIdx.x % PER, i = g >> 1, h = g & 1, lr = threadIdx.x >> 4, c = 8 * (threadIdx.x & 15);
  int64_t tm, tn;
  tile_of(t.full + at, t.ntm * t.ntn, t.ntm, t.ntn, tm, tn);
  const int64_t row = tm * BM + 16 * i + lr, col = tn * 256 + 128 * h + c;
  if (row >= p.M || col >= p.N) return;
  float b[8];
  load_bias8(ep, col, p.N, b);
  // wavefront, register and lane that held columns c .. c + 3; the next four are 16 lanes on
  const int wave = 4 * (i / TI) + c / 32, reg = (i % TI) * TJ + 2 * h + (c / 16 & 1), lane = 16 * (c / 4 & 3) + lr;
  const float* w = p.ws + at * (BM * 256) + wave * (TI * TJ * 256) + reg * 256 + lane * 4;
  v4f x = *(const v4f*)w, y = *(const v4f*)(w + 64);
#pragma unroll 8
  for (int k = 1; k < t.parts; ++k) {
    w += t.rest * (BM * 256);
    const v4f u = *(const v4f*)w, z = *(const v4f*)(w + 64);
#pragma unroll
    for (int e = 0; e < 4; ++e) x[e] += u[e], y[e] += z[e];
  }
  // not before the parts, whose loads come from nearer and would wait for it
  const int64_t rows[1] = {row};
  const bool in[1] = {true};
  Res8<OUT> res[1];
  if constexpr (kEarly<OUT>) load_res8<OUT>(ep, rows, in, col, p.N, res);
  float v[1][8] = {{x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]}};
  finish8<OUT>(p, ep, row, col, v, b, res);
}

// The epilogue alone, on sums that lie as M x N in the workspace (the few-row
// kernel's, where codes are asked for).
template <int OUT>
__global__ __launch_bounds__(256) void k_linear_finish(const Proj p, const Epilogue ep) {
  const int64_t nb = p.N / 128, g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // a row's 128 columns
  const int64_t row = g / nb, col = (g - row * nb) * 128 + 8 * (threadIdx.x & 15);
  if (row >= p.M) return;
  float b[8], v[1][8];
  load_bias8(ep, col, p.N, b);
  Raw8<FP8Q_F32> x;
  x.load(p.ws, row * p.N + col);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[0][k] = x[k];
  Res8<OUT> none[1];
  finish8<OUT>(p, ep, row, col, v, b, none);
}

// How a call goes, and its cost in nanoseconds.  Measured, the codes of either
// operand in HBM:
//   a block of K of a tile, all compute units at work: exact 1050 (64 rows) and
//   1680 (128), FP8-MFMA 980 (128) and 1600 (256); its start and end 2500 and
//   5000, of outputs without activation (with one and the pre-activations kept
//   7500 exact and 21000 FP8-MFMA, which every way of tiles pays); a join 4000 and
//   its bytes, written and read, at 4 TB/s;
//   a workgroup of the few-row kernel, a block of K: 80 with 16 rows and columns,
//   85 + 44 for each 16 rows with 32 columns; its start and end 1500.
// A round is a workgroup per compute unit.
//   exact 48 x 7168 x 18432: few rows 37.5 us, 8 parts 36.1, whole tiles 139;
//   200 x 7168 x 18432: 4 parts 80, whole 143, few rows 159;
//   256 x 2048 x 7168: few rows 18.6, 8 parts 22.2, whole 54.
struct Plan {
  bool few, low;  // low: tiles of half the rows
  Split split;
  int64_t cost;
};
static constexpr int kMaxParts = 16;

static Plan plan_linear(bool fast, int64_t M, int64_t N, int64_t K) {
  const int64_t cu = grid_size(), nkb = K / BK, ntn = (N + 255) / 256;
  Plan best = {};
  best.cost = INT64_MAX;
  const int64_t groups = (M + 63) / 64, rt = ((M + groups - 1) / groups + 15) / 16;
  if (groups <= 65535) {  // the second dimension of a launch
    const int64_t cols = M <= 16 ? 16 : 32, wgs = groups * ((N + cols - 1) / cols);
    best.few = true;
    best.cost = (wgs + cu - 1) / cu * (nkb * (M <= 16 ? 80 : 85 + 44 * rt) + 1500);
  }
  for (int low = 0; low < 2; ++low) {
    const int64_t bm = (fast ? 256 : 128) >> low, ntm = (M + bm - 1) / bm, tiles = ntm * ntn;
    const int64_t block = fast ? (low ? 980 : 1600) : (low ? 1050 : 1680), ends = low ? 2500 : 5000;
    auto take = [&](int64_t full, int parts, int64_t cost) {
      if (cost < best.cost) best = {false, low == 1, {ntm, ntn, full, tiles - full, parts}, cost};
    };
    take(tiles, 1, (tiles + cu - 1) / cu * (nkb * block + ends));
    const int64_t full = tiles / cu * cu, rest = tiles - full;
    for (int parts = 2; rest > 0 && parts <= kMaxParts && parts <= nkb; ++parts)
      take(full, parts, full / cu * (nkb * block + ends) + (rest * parts + cu - 1) / cu * ((nkb + parts - 1) / parts * block + ends) +
                            4000 + 2 * rest * parts * bm * 256 * 4 / 4000);
  }
  return best;
}

int64_t linear_workspace(bool fast, bool codes, int64_t M, int64_t N, int64_t K) {
  const Plan c = plan_linear(fast, M, N, K);
  if (c.few) return codes ? 4 * M * N : 0;
  return c.split.rest * c.split.parts * (((fast ? 256 : 128) >> c.low) * 256 * 4);
}

template <int OUT>
static void launch_join(const Proj& p, const Epilogue& e, const Split& t, int ti, hipStream_t st) {
  const dim3 grid((unsigned)(t.rest * 4 * ti)), block(256);
  if (ti == 8) hipLaunchKernelGGL((k_linear_join<OUT, 8>), grid, block, 0, st, p, e, t);
  else if (ti == 4) hipLaunchKernelGGL((k_linear_join<OUT, 4>), grid, block, 0, st, p, e, t);
  else hipLaunchKernelGGL((k_linear_join<OUT, 2>), grid, block, 0, st, p, e, t);
}

void launch_linear_join(const Proj& p, const Epilogue& e, const Split& t, int ti, hipStream_t st) {
  if (p.scales) {
    if (p.fc == FP8Q_E4M3FN) launch_join<2 + FP8Q_E4M3FN>(p, e, t, ti, st);
    else launch_join<2 + FP8Q_E5M2>(p, e, t, ti, st);
  } else if (p.out_dt == FP8Q_F32) launch_join<FP8Q_F32>(p, e, t, ti, st);
  else launch_join<FP8Q_BF16>(p, e, t, ti, st);
}

int launch_linear(const Proj& q, const Epilogue& e, bool fast, const char* what, hipStream_t st) {
  const Plan c = plan_linear(fast, q.M, q.N, q.K);
  Proj p = q;
  if (c.few) {
    if (!p.scales) return launch_few(p, &e, what, st);
    p.out = p.ws, p.ldo = p.N, p.out_dt = FP8Q_F32, p.scales = nullptr;
    if (int rc = launch_few(p, nullptr, what, st)) return rc;
    const dim3 grid((unsigned)((q.M * (q.N / 128) + 15) / 16)), block(256);
    if (q.fc == FP8Q_E4M3FN) hipLaunchKernelGGL((k_linear_finish<2 + FP8Q_E4M3FN>), grid, block, 0, st, q, e);
    else hipLaunchKernelGGL((k_linear_finish<2 + FP8Q_E5M2>), grid, block, 0, st, q, e);
    return check_launch(what);
  }
  p.B1 = p.B0, p.s1 = p.s0;
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_linear_tiles<0, 0>(p, e, fast, c.low, c.split, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_linear_tiles<1, 0>(p, e, fast, c.low, c.split, st);
  else if (p.fa == FP8Q_E4M3FN) launch_linear_tiles<0, 1>(p, e, fast, c.low, c.split, st);
  else launch_linear_tiles<1, 1>(p, e, fast, c.low, c.split, st);
  return check_launch(what);
}

}  // namespace fp8q

// Root-mean-square norm with the residual's addition and a 1x128 FP8
// output, and its gradients, for gfx950.
//
//   v    = x + r                          (r optional; fp32)
//   rstd = 1 / sqrt(mean(v^2) + eps)      (fp32, over the row)
//   y    = (v * rstd) * w
//   s    = fl32(max(amax of 128 y, qeps) / MAX),  q = enc(fl32(y / s))
//
//   xh = z * rstd,  t = dy * w
//   dx = rstd * (t - xh * mean(t * xh)) + dres
//   dw = sum over rows of dy * xh
//
// Both directions are HBM streams: every element is read once and written
// once, a row stays in registers between its sum and its output, and the
// block maximum of eight elements a lane is four DPP steps.  16384 x 7168 bf16
// with residual: forward 137 us (6.0 TB/s), gradients 171 us (5.5 TB/s); a
// row alone is 3.8 us, most of it the launch.
#include "fp8q_ffn.h"

namespace fp8q {

// Sum of one value per thread over the threads of a row: TPR = 64 is one
// wavefront, otherwise the whole workgroup.  `part` has one slot per
// wavefront and is used by one call at a time (two alternate).
template <int TPR>
__device__ __forceinline__ float row_sum(float v, float* part) {
  v = wave_sum(v);
  if constexpr (TPR > 64) {
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.0f;
#pragma unroll
    for (int i = 0; i < TPR / 64; ++i) v += part[i];
  }
  return v;
}

// One row per TPR threads, V groups of eight consecutive elements a thread:
// group g of thread t is elements 8 * (g * TPR + t), so 16 neighbouring
// lanes hold one 128-element block.  A row's loads are issued together,
// without a branch (a thread past the last column reads the last group
// again), and the weight, which the caches hold, after the sum: kept from the
// start, its registers cost a workgroup in flight (143 against 137 us for
// 16384 x 7168 bf16 with residual).  Walking several rows per workgroup with
// the next row's loads ahead was no faster (148 us).
template <int DT, int WDT, int TPR, int V, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_1x128(const NormFwd p) {
  constexpr int TH = TPR < 256 ? 256 : TPR;
  __shared__ float part[TH / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (TH / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;  // whole wavefronts; no barrier with TPR == 64
  const int nv = (int)(p.cols / 8);
  Raw8<DT> x[V], r[V];
  Raw8<WDT> w[V];
  int cc[V];
  bool in[V];
#pragma unroll
  for (int g = 0; g < V; ++g) {
    in[g] = g * TPR + t < nv;
    cc[g] = in[g] ? g * TPR + t : nv - 1;
    x[g].load(p.x, row * p.ldx + 8 * cc[g]);
    if constexpr (RES) r[g].load(p.res, row * p.ldr + 8 * cc[g]);
  }
  float v[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[g][e] = RES ? x[g][e] + r[g][e] : x[g][e];
      s = __builtin_fmaf(v[g][e], v[g][e], s);
    }
    ss += in[g] ? s : 0.0f;
  }
  ss = row_sum<TPR>(ss, part);
#pragma unroll
  for (int g = 0; g < V; ++g) w[g].template load<false>(p.w, 8 * cc[g]);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.neps);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    if (!in[g]) continue;  // whole 16-lane rows: cols is a multiple of 128
    const int c = cc[g];
    // the sum is stored in x's type; the norm goes on from the unrounded sum
    if (p.z) store8<DT>(p.z, row * p.ldz + 8 * c, v[g]);
    float y[8];
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = v[g][e] * rstd * w[g][e];
      m = max(m, abs_bits(y[e]));
    }
    if (p.y) store8<DT>(p.y, row * p.ldy + 8 * c, y);
    if (p.q) {
      const float amax = __uint_as_float(canon_abs_bits(row16_max(m)));
      const bool e4 = p.fmt == FP8Q_E4M3FN;
      const float s = e4 ? block_scale7<FP8Q_E4M3FN>(amax, p.qeps) : block_scale7<FP8Q_E5M2>(amax, p.qeps);
      const bool fast = scale_ok(s);
      const float inv = 1.0f / s;
      u32x2 q;
      if (e4)
        q = u32x2{encode4<FP8Q_E4M3FN>(y[0], y[1], y[2], y[3], s, inv, fast),
                  encode4<FP8Q_E4M3FN>(y[4], y[5], y[6], y[7], s, inv, fast)};
      else
        q = u32x2{encode4<FP8Q_E5M2>(y[0], y[1], y[2], y[3], s, inv, fast),
                  encode4<FP8Q_E5M2>(y[4], y[5], y[6], y[7], s, inv, fast)};
      __builtin_nontemporal_store(q, (u32x2*)(p.q + row * p.ldq + 8 * c));
      if ((t & 15) == 0) p.scales[row * p.ld_s + (c >> 4)] = s;
    }
  }
}

// A launch holds fewer than 2^32 threads: more rows take several, one after
// another (four rows a workgroup of 256: from 67 million rows on).
template <int DT, int WDT, int TPR, int V>
static void launch_fwd(const NormFwd& p, hipStream_t st) {
  constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
  constexpr int64_t most = 0xFFFFFFFFll / TH * R;
  auto at = [](const void* v, int64_t bytes) { return v ? (char*)v + bytes : nullptr; };
  for (int64_t r = 0; r < p.rows; r += most) {
    NormFwd c = p;
    const int es = DT == FP8Q_F32 ? 4 : 2;
    c.rows = p.rows - r < most ? p.rows - r : most;
    c.x = at(p.x, r * p.ldx * es), c.res = at(p.res, r * p.ldr * es);
    c.z = at(p.z, r * p.ldz * es), c.y = at(p.y, r * p.ldy * es);
    c.q = (uint8_t*)at(p.q, r * p.ldq), c.scales = (float*)at(p.scales, r * p.ld_s * 4), c.rstd = (float*)at(p.rstd, r * 4);
    const dim3 grid((unsigned)((c.rows + R - 1) / R)), block(TH);
    if (p.res) hipLaunchKernelGGL((k_rmsnorm_1x128<DT, WDT, TPR, V, true>), grid, block, 0, st, c);
    else hipLaunchKernelGGL((k_rmsnorm_1x128<DT, WDT, TPR, V, false>), grid, block, 0, st, c);
  }
}

template <int DT, int WDT>
static void dispatch_fwd(const NormFwd& p, hipStream_t st) {
  const int64_t c = p.cols;
  if (c <= 64 * 8) launch_fwd<DT, WDT, 64, 1>(p, st);
  else if (c <= 64 * 8 * 2) launch_fwd<DT, WDT, 64, 2>(p, st);
  else if (c <= 64 * 8 * 4) launch_fwd<DT, WDT, 64, 4>(p, st);
  else if (c <= 256 * 8 * 2) launch_fwd<DT, WDT, 256, 2>(p, st);
  else if (c <= 256 * 8 * 4) launch_fwd<DT, WDT, 256, 4>(p, st);
  else if (c <= 512 * 8 * 4) launch_fwd<DT, WDT, 512, 4>(p, st);
  else if (c <= 1024 * 8 * 4) launch_fwd<DT, WDT, 1024, 4>(p, st);
  else launch_fwd<DT, WDT, 1024, 8>(p, st);
}

int launch_rmsnorm_1x128(const NormFwd& p, hipStream_t st) {
  if (p.dt == FP8Q_F32) {
    if (p.wdt == FP8Q_F32) dispatch_fwd<FP8Q_F32, FP8Q_F32>(p, st);
    else dispatch_fwd<FP8Q_F32, FP8Q_BF16>(p, st);
  } else {
    if (p.wdt == FP8Q_F32) dispatch_fwd<FP8Q_BF16, FP8Q_F32>(p, st);
    else dispatch_fwd<FP8Q_BF16, FP8Q_BF16>(p, st);
  }
  return check_launch("rmsnorm_1x128");
}

// ---------------------------------------------------------------- backward
// Each TPR threads walk rows part, part + parts, ... and keep the weight's
// gradient of their columns in registers; at the end every workgroup writes
// its sums as one row of the workspace, and k_norm_dw adds those rows in a
// fixed order, so the result does not depend on timing.  The next row's
// loads are issued before this row's sum is joined.  Parts: at most two
// workgroups a compute unit (512; what their registers allow); one per eight
// rows below that, but 256 as far as there are rows, so that every compute
// unit has one.  The partial rows, written and read once, are then 3% of the
// call's own bytes at 16384 rows of bf16 with residual, 13% to 17% at 2048
// to 4096 rows of bf16, and a third at 513 rows of fp32, where 13 us go to
// up to three rows after one another and the second launch.
static constexpr int64_t kNormParts = 512;

int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols) {
  const int64_t per = cols <= 2048 ? 4 : 1;  // rows a workgroup holds at once
  const int64_t all = (rows + per - 1) / per;
  int64_t g = rows / 8 < 256 ? 256 : rows / 8;
  if (g > kNormParts) g = kNormParts;
  return all < g ? all : g;
}

template <int DT, int TPR, int V, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_bwd(const NormBwd p) {
  constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
  // The weight waits in LDS (two planes of four, free of bank conflicts), as
  // far as it fits: a global read here would come back behind the next row's
  // loads.
  constexpr int NW = V * TPR;  // groups of eight columns
  constexpr bool WL = NW * 32 <= 128 * 1024;
  __shared__ float part[2][TH / 64];
  __shared__ float4 w_lds[2][WL ? NW : 1];
  const int t = threadIdx.x % TPR;
  const int nv = (int)(p.cols / 8);
  auto weights = [&](int c, float(&w)[8]) {
    if constexpr (WL) {
      const float4 a = w_lds[0][c], b = w_lds[1][c];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      load_w8(p.w, p.wdt, 8 * c, w);
    }
  };
  float dw[V][8];
#pragma unroll
  for (int g = 0; g < V; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[g][e] = 0.0f;
  const float rc = 1.0f / (float)p.cols;
  int flip = 0;
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / TPR;
  // The loop has no branch around a load, so that each wait counts exactly
  // what it needs: a thread past the last column reads the last group again
  // and its part of the sum is dropped, and the last row is read again for
  // want of a next one (cache hits).
  int cc[V];
  bool in[V];
#pragma unroll
  for (int g = 0; g < V; ++g) {
    in[g] = g * TPR + t < nv;
    cc[g] = in[g] ? g * TPR + t : nv - 1;
  }
  // rows are held as loaded and widened twice: in fp32 their registers would
  // leave room for fewer workgroups
  struct Row {
    Raw8<DT> dy[V], z[V];
    float rstd;
  } even, odd;  // taken in turn: copying one to the other would wait for its loads
  auto load = [&](Row& w, int64_t r) {
    if (r >= p.rows) r = p.rows - 1;
    w.rstd = p.rstd[r];
#pragma unroll
    for (int g = 0; g < V; ++g) {
      w.dy[g].load(p.dy, r * p.lddy + 8 * cc[g]);
      w.z[g].load(p.z, r * p.ldz + 8 * cc[g]);
    }
  };
  load(even, row);
  if constexpr (WL) {
    for (int c = threadIdx.x; c < nv; c += TH) {
      float w[8];
      load_w8(p.w, p.wdt, 8 * c, w);
      w_lds[0][c] = make_float4(w[0], w[1], w[2], w[3]);
      w_lds[1][c] = make_float4(w[4], w[5], w[6], w[7]);
    }
    __syncthreads();
  }
  auto one = [&](Row& cur, Row& nxt) {
    const float rs = cur.rstd;
    Raw8<DT> dr[V];
    if constexpr (RES) {
#pragma unroll
      for (int g = 0; g < V; ++g) dr[g].load(p.dres, row * p.lddr + 8 * cc[g]);
    }
    float dot = 0.0f;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float w[8], d = 0.0f;
      weights(cc[g], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = cur.z[g][e] * rs;
        dw[g][e] = __builtin_fmaf(cur.dy[g][e], xh, dw[g][e]);
        d = __builtin_fmaf(cur.dy[g][e] * w[e], xh, d);
      }
      dot += in[g] ? d : 0.0f;
    }
    load(nxt, row + step);
    dot = row_sum<TPR>(dot, part[flip]) * rc;
    flip ^= 1;  // the next row's sums go to the other slots: no wave still reads those
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float w[8], d[8];
      weights(cc[g], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        d[e] = rs * __builtin_fmaf(-(cur.z[g][e] * rs), dot, cur.dy[g][e] * w[e]);
        if constexpr (RES) d[e] += dr[g][e];
      }
      if (in[g]) store8<DT>(p.dx, row * p.lddx + 8 * cc[g], d);
    }
  };
  for (; row < p.rows; row += step) {
    one(even, odd);
    row += step;
    if (row >= p.rows) break;
    one(odd, even);
  }
  if (!p.dw) return;
  if constexpr (R > 1) {
    // the workgroup's R row groups into one row of partial sums
    __shared__ float sum[R][V * 512];
#pragma unroll
    for (int g = 0; g < V; ++g)
#pragma unroll
      for (int e = 0; e < 8; ++e) sum[threadIdx.x / TPR][8 * (g * TPR + t) + e] = dw[g][e];
    __syncthreads();
    for (int c = threadIdx.x; c < p.cols; c += TH) {
      float a = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) a += sum[r][c];
      p.ws[(int64_t)blockIdx.x * p.cols + c] = a;
    }
  } else {
#pragma unroll
    for (int g = 0; g < V; ++g) {
      const int c = g * TPR + t;
      if (c >= nv) continue;
      float4* o = (float4*)(p.ws + (int64_t)blockIdx.x * p.cols + 8 * c);
      o[0] = make_float4(dw[g][0], dw[g][1], dw[g][2], dw[g][3]);
      o[1] = make_float4(dw[g][4], dw[g][5], dw[g][6], dw[g][7]);
    }
  }
}

// dw[c] = sum of the partial rows: 64 columns per workgroup, sixteen groups
// of threads each adding every sixteenth row, joined in a fixed order.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ ws, int64_t parts, int64_t cols,
                                                 float* __restrict__ dw) {
  __shared__ float sum[16][64];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
  const float* p = ws + (int64_t)blockIdx.x * 64 + 4 * c;
  v4f a = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
  for (int64_t r = k; r < parts; r += 16) {
    const v4f b = *(const v4f*)(p + r * cols);
#pragma unroll
    for (int e = 0; e < 4; ++e) a[e] += b[e];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[k][4 * c + e] = a[e];
  __syncthreads();
  if (threadIdx.x < 64) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][threadIdx.x];
    dw[(int64_t)blockIdx.x * 64 + threadIdx.x] = t;
  }
}

template <int DT, int TPR, int V>
static void launch_bwd(const NormBwd& p, int64_t parts, hipStream_t st) {
  const dim3 grid((unsigned)parts), block(TPR < 256 ? 256 : TPR);
  if (p.dres) hipLaunchKernelGGL((k_rmsnorm_bwd<DT, TPR, V, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((k_rmsnorm_bwd<DT, TPR, V, false>), grid, block, 0, st, p);
}

template <int DT>
static void dispatch_bwd(const NormBwd& p, int64_t parts, hipStream_t st) {
  const int64_t c = p.cols;
  if (c <= 64 * 8) launch_bwd<DT, 64, 1>(p, parts, st);
  else if (c <= 64 * 8 * 2) launch_bwd<DT, 64, 2>(p, parts, st);
  else if (c <= 64 * 8 * 4) launch_bwd<DT, 64, 4>(p, parts, st);
  else if (c <= 256 * 8 * 2) launch_bwd<DT, 256, 2>(p, parts, st);
  else if (c <= 256 * 8 * 4) launch_bwd<DT, 256, 4>(p, parts, st);
  else if (c <= 512 * 8 * 4) launch_bwd<DT, 512, 4>(p, parts, st);
  else if (c <= 1024 * 8 * 4) launch_bwd<DT, 1024, 4>(p, parts, st);
  else launch_bwd<DT, 1024, 8>(p, parts, st);
}

int launch_rmsnorm_bwd(const NormBwd& q, hipStream_t st) {
  const int64_t parts = rmsnorm_bwd_parts(q.rows, q.cols);
  NormBwd p = q;
  const bool direct = parts == 1 && ((uintptr_t)p.dw & 15) == 0;
  if (direct && p.dw) p.ws = p.dw;  // the one row of partial sums is the result
  if (p.dt == FP8Q_F32) dispatch_bwd<FP8Q_F32>(p, parts, st);
  else dispatch_bwd<FP8Q_BF16>(p, parts, st);
  if (p.dw && !direct)
    hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)(p.cols / 64)), dim3(256), 0, st, p.ws, parts, p.cols, p.dw);
  return check_launch("rmsnorm_bwd");
}

}  // namespace fp8q

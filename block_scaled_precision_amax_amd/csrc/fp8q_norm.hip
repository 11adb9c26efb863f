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
// block maximum of eight elements a lane is four DPP steps.
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
// lanes hold one 128-element block.
template <int DT, int FMT, int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_1x128(const NormFwd p) {
  constexpr int TH = TPR < 256 ? 256 : TPR;
  __shared__ float part[TH / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (TH / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;  // whole wavefronts; no barrier with TPR == 64
  const int nv = (int)(p.cols / 8);
  float v[V][8];
  float ss = 0.0f;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    const int c = g * TPR + t;
    if (c < nv) {
      load8<DT>(p.x, row * p.ldx + 8 * c, v[g]);
      if (p.res) {
        float r[8];
        load8<DT>(p.res, row * p.ldr + 8 * c, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[g][e] += r[e];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) v[g][e] = 0.0f;
    }
#pragma unroll
    for (int e = 0; e < 8; ++e) ss = __builtin_fmaf(v[g][e], v[g][e], ss);
  }
  ss = row_sum<TPR>(ss, part);
  const float rstd = 1.0f / sqrtf(ss / (float)p.cols + p.neps);
  if (t == 0 && p.rstd) p.rstd[row] = rstd;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    const int c = g * TPR + t;
    if (c >= nv) continue;  // whole 16-lane rows: cols is a multiple of 128
    // the sum is stored in x's type; the norm goes on from the unrounded sum
    if (p.z) store8<DT>(p.z, row * p.ldz + 8 * c, v[g]);
    float w[8], y[8];
    load_w8(p.w, p.wdt, 8 * c, w);
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      y[e] = v[g][e] * rstd * w[e];
      m = max(m, abs_bits(y[e]));
    }
    if (p.y) store8<DT>(p.y, row * p.ldy + 8 * c, y);
    if (p.q) {
      const float s = block_scale<FMT>(__uint_as_float(canon_abs_bits(row16_max(m))), p.qeps);
      const bool fast = scale_ok(s);
      const float r = 1.0f / s;
      const u32x2 q = {encode4<FMT>(y[0], y[1], y[2], y[3], s, r, fast),
                       encode4<FMT>(y[4], y[5], y[6], y[7], s, r, fast)};
      __builtin_nontemporal_store(q, (u32x2*)(p.q + row * p.ldq + 8 * c));
      if ((t & 15) == 0) p.scales[row * p.ld_s + (c >> 4)] = s;
    }
  }
}

template <int DT, int FMT, int TPR, int V>
static void launch_fwd(const NormFwd& p, hipStream_t st) {
  constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
  hipLaunchKernelGGL((k_rmsnorm_1x128<DT, FMT, TPR, V>), dim3((unsigned)((p.rows + R - 1) / R)), dim3(TH), 0, st, p);
}

template <int DT, int FMT>
static void dispatch_fwd(const NormFwd& p, hipStream_t st) {
  const int64_t c = p.cols;
  if (c <= 64 * 8) launch_fwd<DT, FMT, 64, 1>(p, st);
  else if (c <= 64 * 8 * 2) launch_fwd<DT, FMT, 64, 2>(p, st);
  else if (c <= 64 * 8 * 4) launch_fwd<DT, FMT, 64, 4>(p, st);
  else if (c <= 256 * 8 * 2) launch_fwd<DT, FMT, 256, 2>(p, st);
  else if (c <= 256 * 8 * 4) launch_fwd<DT, FMT, 256, 4>(p, st);
  else if (c <= 256 * 8 * 8) launch_fwd<DT, FMT, 256, 8>(p, st);
  else launch_fwd<DT, FMT, 1024, 8>(p, st);
}

int launch_rmsnorm_1x128(const NormFwd& p, hipStream_t st) {
  if (p.dt == FP8Q_F32) {
    if (p.fmt == FP8Q_E4M3FN) dispatch_fwd<FP8Q_F32, FP8Q_E4M3FN>(p, st);
    else dispatch_fwd<FP8Q_F32, FP8Q_E5M2>(p, st);
  } else {
    if (p.fmt == FP8Q_E4M3FN) dispatch_fwd<FP8Q_BF16, FP8Q_E4M3FN>(p, st);
    else dispatch_fwd<FP8Q_BF16, FP8Q_E5M2>(p, st);
  }
  return check_launch("rmsnorm_1x128");
}

// ---------------------------------------------------------------- backward
// Each TPR threads walk rows part, part + parts, ... and keep the weight's
// gradient of their columns in registers; at the end every workgroup writes
// its sums as one row of the workspace, and k_norm_dw adds those rows in a
// fixed order, so the result does not depend on timing.
static constexpr int64_t kNormParts = 512;

static int norm_tpr(int64_t cols) { return cols <= 2048 ? 64 : cols <= 16384 ? 256 : 1024; }

int64_t rmsnorm_bwd_parts(int64_t rows, int64_t cols) {
  const int64_t per = norm_tpr(cols) == 64 ? 4 : 1;  // rows a workgroup holds at once
  const int64_t g = (rows + per - 1) / per;
  return g < kNormParts ? g : kNormParts;
}

template <int DT, int TPR, int V>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_rmsnorm_bwd(const NormBwd p) {
  constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
  __shared__ float part[2][TH / 64];
  const int t = threadIdx.x % TPR;
  const int nv = (int)(p.cols / 8);
  float dw[V][8];
#pragma unroll
  for (int g = 0; g < V; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[g][e] = 0.0f;
  const float rc = 1.0f / (float)p.cols;
  int flip = 0;
  for (int64_t row = (int64_t)blockIdx.x * R + threadIdx.x / TPR; row < p.rows; row += (int64_t)gridDim.x * R) {
    const float rstd = p.rstd[row];
    float tt[V][8], xh[V][8];
    float dot = 0.0f;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      const int c = g * TPR + t;
      if (c < nv) {
        float w[8];
        load8<DT>(p.dy, row * p.lddy + 8 * c, tt[g]);
        load8<DT>(p.z, row * p.ldz + 8 * c, xh[g]);
        load_w8(p.w, p.wdt, 8 * c, w);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          xh[g][e] *= rstd;
          dw[g][e] = __builtin_fmaf(tt[g][e], xh[g][e], dw[g][e]);
          tt[g][e] *= w[e];
          dot = __builtin_fmaf(tt[g][e], xh[g][e], dot);
        }
      }
    }
    dot = row_sum<TPR>(dot, part[flip]) * rc;
    flip ^= 1;  // the next row's sums go to the other slots: no wave still reads those
#pragma unroll
    for (int g = 0; g < V; ++g) {
      const int c = g * TPR + t;
      if (c >= nv) continue;
      float d[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) d[e] = rstd * __builtin_fmaf(-xh[g][e], dot, tt[g][e]);
      if (p.dres) {
        float r[8];
        load8<DT>(p.dres, row * p.lddr + 8 * c, r);
#pragma unroll
        for (int e = 0; e < 8; ++e) d[e] += r[e];
      }
      store8<DT>(p.dx, row * p.lddx + 8 * c, d);
    }
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

// dw[c] = sum of the partial rows: 32 columns per workgroup, eight threads
// per column each adding every eighth row, joined in a fixed order.
__global__ __launch_bounds__(256) void k_norm_dw(const float* __restrict__ ws, int64_t parts, int64_t cols,
                                                 float* __restrict__ dw) {
  __shared__ float sum[8][32];
  const int c = threadIdx.x & 31, k = threadIdx.x >> 5;
  const int64_t col = (int64_t)blockIdx.x * 32 + c;
  float a = 0.0f;
  for (int64_t r = k; r < parts; r += 8) a += ws[r * cols + col];
  sum[k][c] = a;
  __syncthreads();
  if (k == 0) {
    a = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) a += sum[i][c];
    dw[col] = a;
  }
}

template <int DT, int TPR, int V>
static void launch_bwd(const NormBwd& p, int64_t parts, hipStream_t st) {
  hipLaunchKernelGGL((k_rmsnorm_bwd<DT, TPR, V>), dim3((unsigned)parts), dim3(TPR < 256 ? 256 : TPR), 0, st, p);
}

template <int DT>
static void dispatch_bwd(const NormBwd& p, int64_t parts, hipStream_t st) {
  const int64_t c = p.cols;
  if (c <= 64 * 8) launch_bwd<DT, 64, 1>(p, parts, st);
  else if (c <= 64 * 8 * 2) launch_bwd<DT, 64, 2>(p, parts, st);
  else if (c <= 64 * 8 * 4) launch_bwd<DT, 64, 4>(p, parts, st);
  else if (c <= 256 * 8 * 2) launch_bwd<DT, 256, 2>(p, parts, st);
  else if (c <= 256 * 8 * 4) launch_bwd<DT, 256, 4>(p, parts, st);
  else if (c <= 256 * 8 * 8) launch_bwd<DT, 256, 8>(p, parts, st);
  else launch_bwd<DT, 1024, 8>(p, parts, st);
}

int launch_rmsnorm_bwd(const NormBwd& p, hipStream_t st) {
  const int64_t parts = rmsnorm_bwd_parts(p.rows, p.cols);
  if (p.dt == FP8Q_F32) dispatch_bwd<FP8Q_F32>(p, parts, st);
  else dispatch_bwd<FP8Q_BF16>(p, parts, st);
  if (p.dw)
    hipLaunchKernelGGL(k_norm_dw, dim3((unsigned)(p.cols / 32)), dim3(256), 0, st, p.ws, parts, p.cols, p.dw);
  return check_launch("rmsnorm_bwd");
}

}  // namespace fp8q

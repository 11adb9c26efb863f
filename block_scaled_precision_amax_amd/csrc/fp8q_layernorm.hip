// Layer norm with the residual's addition and a 1x128 FP8 output, and its
// gradients, for gfx950.
//
//   v    = x + r                          (r optional; fp32)
//   mean = sum(v) / n,  rstd = 1 / sqrt(sum((v - mean)^2) / n + eps)
//   y    = (v - mean) * rstd * w + b      (w, b optional)
//   s    = fl32(max(amax of 128 y, qeps) / MAX),  q = enc(fl32(y / s))
//
//   xh = (z - mean) * rstd,  t = dy * w
//   dx = rstd * (t - mean(t) - xh * mean(t * xh)) + dres
//   dw = sum over rows of dy * xh,  db = sum over rows of dy
//
// Both directions are HBM streams: every element is read once and written
// once, a row stays in registers between its sums and its output, and the
// block maximum of eight elements a lane is four DPP steps.  The variance is
// the mean of the squared distances from the mean, a second sum over the
// registers, and not mean(v^2) - mean^2, which loses it where a row lies far
// from zero.
//   16384 x 7168 bf16 with residual: forward to z, codes and statistics
//   (826 MB) 151 us, gradients (940 MB) 157 us, where an elementwise pass that
//   moves 6.19 TB/s takes 133 and 152.
//   One row of 7168: 4.5 us, the latency of two loads (the row, then weight and
//   bias), two sums across the workgroup and the stores.
//   Gradients of 513 x 4096: 13 + 4 us (25 MB, 4.1 us): two turns of loads, two
//   sums and a store one after the other, and the column sums' launch.
#include "fp8q_ffn.h"

namespace fp8q {

// Sum of one value per thread over the threads of a row: TPR = 64 is one
// wavefront, otherwise the whole workgroup.  `part` has one slot per
// wavefront and belongs to this call alone until the next barrier.
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

// Group c of the weight or bias, as loaded, or the constant that its absence
// stands for.
template <int WDT>
__device__ __forceinline__ void load_or(Raw8<WDT>& r, const void* p, int c, float constant) {
  if (p) r.template load<false>(p, 8 * c);
  else r.fill(constant);
}

// Eight sums as they are stored, kept from before the mean is taken off.
template <int DT>
struct Sum8 {
  float v[8];
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 8; ++e) v[e] = x[e];
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const { store8<DT>(p, i, v); }
};
template <>
struct Sum8<FP8Q_BF16> {
  u32x4 v;
  __device__ __forceinline__ void set(const float (&x)[8]) {
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = pk_bf16(x[2 * e], x[2 * e + 1]);
  }
  __device__ __forceinline__ void store(void* p, int64_t i) const {
    __builtin_nontemporal_store(v, (u32x4*)((uint16_t*)p + i));
  }
};

// The codes of group c of a row.
__device__ __forceinline__ void store_codes(const LayerNormFwd& p, int64_t row, int c, const float (&y)[8]) {
  float m = 0.0f;
#pragma unroll
  for (int e = 0; e < 8; ++e) m = max_abs(m, y[e]);
  const float amax = __uint_as_float(canon_abs_bits(row16_max(__float_as_uint(m))));
  const bool e4 = p.fmt == FP8Q_E4M3FN;
  const float s = e4 ? block_scale7<FP8Q_E4M3FN>(amax, p.qeps) : block_scale7<FP8Q_E5M2>(amax, p.qeps);
  const bool fast = scale_ok(s);
  const float inv = recip(s);
  u32x2 q;
  if (e4)
    q = u32x2{encode4<FP8Q_E4M3FN>(y[0], y[1], y[2], y[3], s, inv, fast),
              encode4<FP8Q_E4M3FN>(y[4], y[5], y[6], y[7], s, inv, fast)};
  else
    q = u32x2{encode4<FP8Q_E5M2>(y[0], y[1], y[2], y[3], s, inv, fast),
              encode4<FP8Q_E5M2>(y[4], y[5], y[6], y[7], s, inv, fast)};
  __builtin_nontemporal_store(q, (u32x2*)(p.q + row * p.ldq + 8 * c));
  if ((threadIdx.x & 15) == 0) p.scales[row * p.ld_s + (c >> 4)] = s;
}

// One row per TPR threads, V groups of eight consecutive elements a thread:
// group g of thread t is elements 8 * (g * TPR + t), so 16 neighbouring
// lanes hold one 128-element block.  Nothing branches around a load or a
// store, so that each wait counts exactly what it needs: sixteen lanes past the
// last column take the last block (without codes, a lane the last group) once
// more, leave it out of the sums and store what its own lanes store.  A row's
// loads are issued together; weight and bias, which the caches hold, after the
// sums, a group ahead of its use and before the stores of the group at hand: a
// load behind a store waits for it (all after the sums: 150 us and a third
// fewer rows in flight; each with its group: 154).
template <int DT, int WDT, int TPR, int V, bool RES>
__global__ __launch_bounds__(TPR < 256 ? 256 : TPR) void k_layernorm_1x128(const LayerNormFwd p) {
  constexpr int TH = TPR < 256 ? 256 : TPR;
  __shared__ float part[2][TH / 64];
  const int t = threadIdx.x % TPR;
  const int64_t row = (int64_t)blockIdx.x * (TH / TPR) + threadIdx.x / TPR;
  if (TPR == 64 && row >= p.rows) return;  // whole wavefronts; no barrier with TPR == 64
  const int nv = (int)(p.cols / 8);
  const float n = (float)p.cols;
  Raw8<DT> x[V], r[V];
  int cc[V];
  bool in[V];
#pragma unroll
  for (int g = 0; g < V; ++g) {
    in[g] = g * TPR + t < nv;
    cc[g] = in[g] ? g * TPR + t : p.q ? nv - 16 + (t & 15) : nv - 1;
    x[g].load(p.x, row * p.ldx + 8 * cc[g]);
    if constexpr (RES) r[g].load(p.res, row * p.ldr + 8 * cc[g]);
  }
  float v[V][8];
  float sum = 0.0f;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[g][e] = RES ? x[g][e] + r[g][e] : x[g][e];
      s += v[g][e];
    }
    sum += in[g] ? s : 0.0f;
  }
  Sum8<DT> z[V];
#pragma unroll
  for (int g = 0; g < V; ++g) z[g].set(v[g]);
  const float mean = row_sum<TPR>(sum, part[0]) / n;
  float ss = 0.0f;
#pragma unroll
  for (int g = 0; g < V; ++g) {
    float s = 0.0f;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      v[g][e] -= mean;
      s = __builtin_fmaf(v[g][e], v[g][e], s);
    }
    ss += in[g] ? s : 0.0f;
  }
  Raw8<WDT> w[2], b[2];
  auto load_affine = [&](int g) {
    load_or(w[g & 1], p.w, cc[g], 1.0f);
    load_or(b[g & 1], p.b, cc[g], 0.0f);
  };
  ss = row_sum<TPR>(ss, part[1]);
  load_affine(0);
  const float rstd = 1.0f / sqrtf(ss / n + p.neps);
#pragma unroll
  for (int g = 0; g < V; ++g) {
    if (g + 1 < V) load_affine(g + 1);
    __builtin_amdgcn_sched_barrier(0);
    const int c = cc[g];
    float y[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(v[g][e] * rstd, w[g & 1][e], b[g & 1][e]);
    // the sum is stored in x's type; the norm goes on from the unrounded sum
    if (p.z) z[g].store(p.z, row * p.ldz + 8 * c);
    if (p.y) store8<DT>(p.y, row * p.ldy + 8 * c, y);
    if (p.q) store_codes(p, row, c, y);
    __builtin_amdgcn_sched_barrier(0);
  }
  if (t == 0) {
    if (p.mean) p.mean[row] = mean;
    if (p.rstd) p.rstd[row] = rstd;
  }
}

// The same for many rows: a workgroup walks rows block, block + blocks, ...
// with its columns' weight and bias in registers and the next row's loads
// issued before this row's sums are joined.
template <int DT, int WDT, int TPR, int V, bool RES>
__global__ __launch_bounds__(TPR) void k_layernorm_walk(const LayerNormFwd p) {
  __shared__ float part[4][TPR / 64];
  const int t = threadIdx.x, nv = (int)(p.cols / 8);
  const float n = (float)p.cols;
  int cc[V];
  bool in[V];
  Raw8<WDT> w[V], b[V];
#pragma unroll
  for (int g = 0; g < V; ++g) {
    in[g] = g * TPR + t < nv;
    cc[g] = in[g] ? g * TPR + t : p.q ? nv - 16 + (t & 15) : nv - 1;
    load_or(w[g], p.w, cc[g], 1.0f);
    load_or(b[g], p.b, cc[g], 0.0f);
  }
  struct Row {
    Raw8<DT> x[V], r[V];
  } even, odd;
  auto load = [&](Row& a, int64_t row) {
    if (row >= p.rows) row = p.rows - 1;  // read again for want of a next one
#pragma unroll
    for (int g = 0; g < V; ++g) {
      a.x[g].load(p.x, row * p.ldx + 8 * cc[g]);
      if constexpr (RES) a.r[g].load(p.res, row * p.ldr + 8 * cc[g]);
    }
  };
  int64_t row = blockIdx.x;
  load(even, row);
  auto one = [&](const Row& cur, Row& nxt, int slot) {
    float v[V][8];
    float sum = 0.0f;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[g][e] = RES ? cur.x[g][e] + cur.r[g][e] : cur.x[g][e];
        s += v[g][e];
      }
      sum += in[g] ? s : 0.0f;
    }
    load(nxt, row + gridDim.x);
    Sum8<DT> z[V];
#pragma unroll
    for (int g = 0; g < V; ++g) z[g].set(v[g]);
    const float mean = row_sum<TPR>(sum, part[slot]) / n;
    float ss = 0.0f;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float s = 0.0f;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[g][e] -= mean;
        s = __builtin_fmaf(v[g][e], v[g][e], s);
      }
      ss += in[g] ? s : 0.0f;
    }
    ss = row_sum<TPR>(ss, part[slot + 1]);
    const float rstd = 1.0f / sqrtf(ss / n + p.neps);
#pragma unroll
    for (int g = 0; g < V; ++g) {
      const int c = cc[g];
      float y[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) y[e] = __builtin_fmaf(v[g][e] * rstd, w[g][e], b[g][e]);
      if (p.z) z[g].store(p.z, row * p.ldz + 8 * c);
      if (p.y) store8<DT>(p.y, row * p.ldy + 8 * c, y);
      if (p.q) store_codes(p, row, c, y);
    }
    if (t == 0) {
      if (p.mean) p.mean[row] = mean;
      if (p.rstd) p.rstd[row] = rstd;
    }
  };
  // two rows' sums alternate between the slots: no wavefront still reads those written
  for (; row < p.rows; row += gridDim.x) {
    one(even, odd, 0);
    row += gridDim.x;
    if (row >= p.rows) break;
    one(odd, even, 2);
  }
}

// A launch holds fewer than 2^32 threads: more rows take several, one after
// another (four rows a workgroup of 256: from 67 million rows on).
template <int DT, int WDT, int TPR, int V>
static void launch_fwd(const LayerNormFwd& p, hipStream_t st) {
  constexpr int TH = TPR < 256 ? 256 : TPR, R = TH / TPR;
  constexpr int64_t most = 0xFFFFFFFFll / TH * R;
  auto at = [](const void* v, int64_t bytes) { return v ? (char*)v + bytes : nullptr; };
  for (int64_t r = 0; r < p.rows; r += most) {
    LayerNormFwd c = p;
    const int es = DT == FP8Q_F32 ? 4 : 2;
    c.rows = p.rows - r < most ? p.rows - r : most;
    c.x = at(p.x, r * p.ldx * es), c.res = at(p.res, r * p.ldr * es);
    c.z = at(p.z, r * p.ldz * es), c.y = at(p.y, r * p.ldy * es);
    c.q = (uint8_t*)at(p.q, r * p.ldq), c.scales = (float*)at(p.scales, r * p.ld_s * 4);
    c.mean = (float*)at(p.mean, r * 4), c.rstd = (float*)at(p.rstd, r * 4);
    const dim3 grid((unsigned)((c.rows + R - 1) / R)), block(TH);
    if (p.res) hipLaunchKernelGGL((k_layernorm_1x128<DT, WDT, TPR, V, true>), grid, block, 0, st, c);
    else hipLaunchKernelGGL((k_layernorm_1x128<DT, WDT, TPR, V, false>), grid, block, 0, st, c);
  }
}

template <int DT, int WDT, int TPR, int V>
static void launch_walk(const LayerNormFwd& p, int64_t blocks, hipStream_t st) {
  if (p.res) hipLaunchKernelGGL((k_layernorm_walk<DT, WDT, TPR, V, true>), dim3((unsigned)blocks), dim3(TPR), 0, st, p);
  else hipLaunchKernelGGL((k_layernorm_walk<DT, WDT, TPR, V, false>), dim3((unsigned)blocks), dim3(TPR), 0, st, p);
}

template <int DT, int WDT>
static void dispatch_fwd(const LayerNormFwd& p, hipStream_t st) {
  const int64_t c = p.cols;
  const int64_t cu = device_cu_count();
  // Walking pays where a row of fp32 or a wide one leaves few rows in flight:
  // 8192 x 8192 fp32 with residual 158 us against 185, 2048 rows 44.5 against 49.0,
  // 1024 rows the same; 7168 x 16384 bf16 143 against 150, 2048 rows 48.4 against
  // 47.2.  16384 x 7168 bf16: 148 to 153 against 150.
  if (DT == FP8Q_F32 && c > 512 * 8 && c <= 1024 * 8 && p.rows >= 8 * cu) launch_walk<DT, WDT, 1024, 1>(p, cu, st);
  else if (c > 1024 * 8 && c <= 1024 * 8 * 2 && p.rows >= 16 * cu) launch_walk<DT, WDT, 1024, 2>(p, cu, st);
  else if (c <= 64 * 8) launch_fwd<DT, WDT, 64, 1>(p, st);
  else if (c <= 64 * 8 * 2) launch_fwd<DT, WDT, 64, 2>(p, st);
  else if (c <= 64 * 8 * 4) launch_fwd<DT, WDT, 64, 4>(p, st);
  else if (c <= 256 * 8 * 2) launch_fwd<DT, WDT, 256, 2>(p, st);
  else if (c <= 256 * 8 * 4) launch_fwd<DT, WDT, 256, 4>(p, st);
  else if (c <= 512 * 8 * 4) launch_fwd<DT, WDT, 512, 4>(p, st);
  else if (c <= 1024 * 8 * 4) launch_fwd<DT, WDT, 1024, 4>(p, st);
  else launch_fwd<DT, WDT, 1024, 8>(p, st);
}

int launch_layernorm_1x128(const LayerNormFwd& p, hipStream_t st) {
  if (p.dt == FP8Q_F32) {
    if (p.wdt == FP8Q_F32) dispatch_fwd<FP8Q_F32, FP8Q_F32>(p, st);
    else dispatch_fwd<FP8Q_F32, FP8Q_BF16>(p, st);
  } else {
    if (p.wdt == FP8Q_F32) dispatch_fwd<FP8Q_BF16, FP8Q_F32>(p, st);
    else dispatch_fwd<FP8Q_BF16, FP8Q_BF16>(p, st);
  }
  return check_launch("layernorm_1x128");
}

// ---------------------------------------------------------------- backward
// R groups of TPR threads walk rows, R rows at a time a workgroup, and keep both
// column sums of their columns in registers; at the end every workgroup adds
// its groups' and writes them as one row of the workspace ([dw | db]), and
// k_column_sums adds those rows in a fixed order, so the result does not depend
// on timing.  The next rows' loads are issued before these rows' sums are
// joined.
struct BwdShape {
  int tpr, v, r;
};
static constexpr BwdShape bwd_shape(int64_t cols) {
  return cols <= 64 * 8         ? BwdShape{64, 1, 4}
         : cols <= 64 * 8 * 2   ? BwdShape{64, 2, 4}
         : cols <= 64 * 8 * 4   ? BwdShape{64, 4, 4}
         : cols <= 256 * 8 * 2  ? BwdShape{256, 2, 2}
         : cols <= 512 * 8 * 2  ? BwdShape{512, 2, 1}
         : cols <= 512 * 8 * 4  ? BwdShape{512, 4, 1}
         : cols <= 1024 * 8 * 4 ? BwdShape{1024, 4, 1}
                                : BwdShape{1024, 8, 1};
}

// Workgroups: one a compute unit of 256, as few as take the same number of turns.
// (Two a unit, where their registers let one and a half run: 16384 x 7168 bf16
// with residual 169 us against 156; 2048 columns 62 against 57.)
static constexpr int64_t kParts = 256;
int64_t layernorm_bwd_parts(int64_t rows, int64_t cols) {
  const int64_t all = (rows + bwd_shape(cols).r - 1) / bwd_shape(cols).r;
  const int64_t turns = (all + kParts - 1) / kParts;
  return (all + turns - 1) / turns;
}

template <int DT, int TPR, int V, int R, bool RES>
__global__ __launch_bounds__(TPR* R) void k_layernorm_bwd(const LayerNormBwd p) {
  constexpr int TH = TPR * R;
  // The weight waits in LDS (two planes of four, free of bank conflicts), as
  // far as it fits: a global read here would come back behind the next row's
  // loads.
  constexpr int NW = V * TPR;  // groups of eight columns
  constexpr bool WL = NW * 32 <= 128 * 1024;
  __shared__ float part[2][2][TH / 64];
  __shared__ float4 w_lds[2][WL ? NW : 1];
  const int t = threadIdx.x % TPR, group = threadIdx.x / TPR;
  const int nv = (int)(p.cols / 8);
  auto ones_or_w = [&](int c, float(&w)[8]) {
    if (p.w) {
      load_w8(p.w, p.wdt, 8 * c, w);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) w[e] = 1.0f;
    }
  };
  auto weights = [&](int c, float(&w)[8]) {
    if constexpr (WL) {
      const float4 a = w_lds[0][c], b = w_lds[1][c];
      w[0] = a.x, w[1] = a.y, w[2] = a.z, w[3] = a.w, w[4] = b.x, w[5] = b.y, w[6] = b.z, w[7] = b.w;
    } else {
      ones_or_w(c, w);
    }
  };
  float dw[V][8], db[V][8];
#pragma unroll
  for (int g = 0; g < V; ++g)
#pragma unroll
    for (int e = 0; e < 8; ++e) dw[g][e] = 0.0f, db[g][e] = 0.0f;
  const float rc = 1.0f / (float)p.cols;
  int flip = 0;
  const int64_t step = (int64_t)gridDim.x * R;
  int64_t first = (int64_t)blockIdx.x * R;  // the workgroup's rows at hand: first .. first + R - 1
  // The loop has no branch around a load, so that each wait counts exactly
  // what it needs: a thread past the last column reads the last group again
  // and its part of the sums is dropped, and past the last row that row is
  // read again (cache hits) and counts as zeros.
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
    float mean, rstd;
  } even, odd;  // taken in turn: copying one to the other would wait for its loads
  auto load = [&](Row& w, int64_t r) {
    if (r >= p.rows) r = p.rows - 1;
    w.mean = p.mean[r];
    w.rstd = p.rstd[r];
#pragma unroll
    for (int g = 0; g < V; ++g) {
      w.dy[g].load(p.dy, r * p.lddy + 8 * cc[g]);
      w.z[g].load(p.z, r * p.ldz + 8 * cc[g]);
    }
  };
  load(even, first + group);
  if constexpr (WL) {
    for (int c = threadIdx.x; c < nv; c += TH) {
      float w[8];
      ones_or_w(c, w);
      w_lds[0][c] = make_float4(w[0], w[1], w[2], w[3]);
      w_lds[1][c] = make_float4(w[4], w[5], w[6], w[7]);
    }
    __syncthreads();
  }
  auto one = [&](Row& cur, Row& nxt) {
    int64_t row = first + group;
    const bool valid = row < p.rows;
    if (R > 1 && !valid) {  // whole wavefronts
      row = p.rows - 1;
      cur.mean = 0.0f;  // finite, whatever that row holds
      cur.rstd = 0.0f;
#pragma unroll
      for (int g = 0; g < V; ++g) cur.dy[g].fill(0.0f), cur.z[g].fill(0.0f);
    }
    const float rs = cur.rstd, mu = cur.mean;
    Raw8<DT> dr[V];
    if constexpr (RES) {
#pragma unroll
      for (int g = 0; g < V; ++g) dr[g].load(p.dres, row * p.lddr + 8 * cc[g]);
    }
    float dot = 0.0f, sum = 0.0f;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float w[8], d = 0.0f, s = 0.0f;
      weights(cc[g], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (cur.z[g][e] - mu) * rs, tt = cur.dy[g][e] * w[e];
        dw[g][e] = __builtin_fmaf(cur.dy[g][e], xh, dw[g][e]);
        db[g][e] += cur.dy[g][e];
        d = __builtin_fmaf(tt, xh, d);
        s += tt;
      }
      dot += in[g] ? d : 0.0f;
      sum += in[g] ? s : 0.0f;
    }
    load(nxt, first + step + group);
    dot = wave_sum(dot), sum = wave_sum(sum);
    if constexpr (TPR > 64) {
      float(&pt)[2][TH / 64] = part[flip];
      flip ^= 1;  // the next rows' sums go to the other slots: no wave still reads those
      if ((threadIdx.x & 63) == 0) pt[0][threadIdx.x >> 6] = dot, pt[1][threadIdx.x >> 6] = sum;
      __syncthreads();
      dot = 0.0f, sum = 0.0f;
#pragma unroll
      for (int i = 0; i < TPR / 64; ++i) {
        dot += pt[0][group * (TPR / 64) + i];
        sum += pt[1][group * (TPR / 64) + i];
      }
    }
    dot *= rc, sum *= rc;
#pragma unroll
    for (int g = 0; g < V; ++g) {
      float w[8], d[8];
      weights(cc[g], w);
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float xh = (cur.z[g][e] - mu) * rs;
        d[e] = rs * (__builtin_fmaf(-xh, dot, cur.dy[g][e] * w[e]) - sum);
        if constexpr (RES) d[e] += dr[g][e];
      }
      if (in[g] && valid) store8<DT>(p.dx, row * p.lddx + 8 * cc[g], d);
    }
  };
  // the same turns for every wavefront: the barriers are inside
  for (; first < p.rows; first += step) {
    one(even, odd);
    first += step;
    if (first >= p.rows) break;
    one(odd, even);
  }
  // one row of column sums per workgroup
  float* const out[2] = {p.pw ? p.pw + (int64_t)blockIdx.x * p.ldp : nullptr,
                         p.pb ? p.pb + (int64_t)blockIdx.x * p.ldp : nullptr};
  if constexpr (R > 1) {
    // the workgroup's R row groups meet in LDS, one sum after the other
    __shared__ float sum[R][V * TPR * 8];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!out[k]) continue;
      __syncthreads();
#pragma unroll
      for (int g = 0; g < V; ++g)
#pragma unroll
        for (int e = 0; e < 8; ++e) sum[group][8 * (g * TPR + t) + e] = k ? db[g][e] : dw[g][e];
      __syncthreads();
      for (int c = threadIdx.x; c < p.cols; c += TH) {
        float a = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) a += sum[r][c];
        out[k][c] = a;
      }
    }
  } else {
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      if (!out[k]) continue;
#pragma unroll
      for (int g = 0; g < V; ++g) {
        if (!in[g]) continue;
        const float(&s)[8] = k ? db[g] : dw[g];
        float* o = out[k] + 8 * cc[g];
        *(float4*)o = make_float4(s[0], s[1], s[2], s[3]);
        *(float4*)(o + 4) = make_float4(s[4], s[5], s[6], s[7]);
      }
    }
  }
}

// Sums of a table's columns, parts rows of `cols` floats: the first `split`
// columns go to a, the rest to b (either may be null).  64 columns per workgroup,
// sixteen groups of threads each adding every sixteenth row, joined in a
// fixed order.
__global__ __launch_bounds__(256) void k_column_sums(const float* __restrict__ ws, int64_t parts, int64_t cols,
                                                     int64_t split, float* __restrict__ a, float* __restrict__ b) {
  __shared__ float sum[16][64];
  const int c = threadIdx.x & 15, k = threadIdx.x >> 4;
  const int64_t c0 = (int64_t)blockIdx.x * 64;
  const bool in = c0 + 4 * c < cols;  // cols is a multiple of four
  const float* p = ws + c0 + 4 * c;
  v4f v = {0.0f, 0.0f, 0.0f, 0.0f};
  if (in) {
#pragma unroll 8
    for (int64_t r = k; r < parts; r += 16) {
      const v4f u = *(const v4f*)(p + r * cols);
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] += u[e];
    }
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) sum[k][4 * c + e] = v[e];
  __syncthreads();
  const int64_t col = c0 + threadIdx.x;
  if (threadIdx.x < 64 && col < cols) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) t += sum[i][threadIdx.x];
    float* out = col < split ? a : b;
    if (out) out[col < split ? col : col - split] = t;
  }
}

void launch_column_sums(const float* ws, int64_t parts, int64_t cols, int64_t split, float* a, float* b, hipStream_t st) {
  hipLaunchKernelGGL(k_column_sums, dim3((unsigned)((cols + 63) / 64)), dim3(256), 0, st, ws, parts, cols, split, a, b);
}

template <int DT, int64_t COLS>
static void launch_bwd(const LayerNormBwd& p, int64_t parts, hipStream_t st) {
  constexpr BwdShape s = bwd_shape(COLS);
  const dim3 grid((unsigned)parts), block(s.tpr * s.r);
  if (p.dres) hipLaunchKernelGGL((k_layernorm_bwd<DT, s.tpr, s.v, s.r, true>), grid, block, 0, st, p);
  else hipLaunchKernelGGL((k_layernorm_bwd<DT, s.tpr, s.v, s.r, false>), grid, block, 0, st, p);
}

// The shape of the smallest limit that holds the columns.
template <int DT>
static void dispatch_bwd(const LayerNormBwd& p, int64_t parts, hipStream_t st) {
  const int64_t c = p.cols;
  if (c <= 512) launch_bwd<DT, 512>(p, parts, st);
  else if (c <= 1024) launch_bwd<DT, 1024>(p, parts, st);
  else if (c <= 2048) launch_bwd<DT, 2048>(p, parts, st);
  else if (c <= 4096) launch_bwd<DT, 4096>(p, parts, st);
  else if (c <= 8192) launch_bwd<DT, 8192>(p, parts, st);
  else if (c <= 16384) launch_bwd<DT, 16384>(p, parts, st);
  else if (c <= 32768) launch_bwd<DT, 32768>(p, parts, st);
  else launch_bwd<DT, 65536>(p, parts, st);
}

int launch_layernorm_bwd(const LayerNormBwd& q, hipStream_t st) {
  const int64_t parts = layernorm_bwd_parts(q.rows, q.cols);
  LayerNormBwd p = q;
  const bool sums = p.dw || p.db;
  // the one row of a single part is the result, where its stores are aligned
  const bool direct = parts == 1 && (((uintptr_t)p.dw | (uintptr_t)p.db) & 15) == 0;
  p.ldp = 2 * p.cols;
  p.pw = !sums ? nullptr : direct ? p.dw : p.ws;
  p.pb = !sums ? nullptr : direct ? p.db : p.ws + p.cols;
  if (p.dt == FP8Q_F32) dispatch_bwd<FP8Q_F32>(p, parts, st);
  else dispatch_bwd<FP8Q_BF16>(p, parts, st);
  if (sums && !direct) launch_column_sums(p.ws, parts, 2 * p.cols, p.cols, p.dw, p.db, st);
  return check_launch("layernorm_bwd");
}

}  // namespace fp8q

// Linear layer C = act(A B^T + bias) + residual on block-scaled FP8 operands
// for gfx950, and its form that leaves act(A B^T + bias) as 1x128 codes.
//
//   v[m,n] = sum_kb sA[m,kb] sB(n,kb) P_kb + bias[n],
//   P_kb   = sum over the 128 k of a block of dec(a) dec(b),
//   C = act(v) + res  or  s, q = 1x128 codes of act(v);  pre = bf16(v) on request
//
// Three ways, by the cost of each: tiles with the epilogue behind their last
// block; the same tiles with K cut into parts whose sums go to a workspace,
// joined by a second kernel with the same epilogue, where there are too few
// tiles for the compute units; and the few-row kernel (fp8q_few.hip).
#include "fp8q_tiles.h"

namespace fp8q {

// OUT of the kernels below: FP8Q_F32, FP8Q_BF16, 2 + format (1x128 codes) or
// kPart, the bare sums as fp32 in the workspace.
static constexpr int kPart = 4;

// Row stride of a plane of the workspace.
__host__ __device__ constexpr int64_t plane_ld(int64_t N) { return (N + 7) / 8 * 8; }

// Bias of eight columns, zeros past the last one or without a bias.
__device__ __forceinline__ void load_bias8(const Epilogue& e, int64_t col, int64_t N, float (&b)[8]) {
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    b[k] = 0.0f;
    if (e.bias && col + k < N)
      b[k] = e.bdt == FP8Q_F32 ? ((const float*)e.bias)[col + k] : bf_lo(((const uint16_t*)e.bias)[col + k]);
  }
}

// Eight elements of an output row, of which `left` exist.
template <int DT>
__device__ __forceinline__ void store_edge8(void* p, int64_t i, const float (&v)[8], int64_t left, bool vec) {
  if (vec && left >= 8) {
    store8<DT>(p, i, v);
    return;
  }
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    if (k >= left) continue;
    if constexpr (DT == FP8Q_F32) ((float*)p)[i + k] = v[k];
    else ((uint16_t*)p)[i + k] = (uint16_t)pk_bf16(v[k], 0.0f);
  }
}

// Everything behind the sums of one row's columns col .. col + 7 (col a
// multiple of eight, col < N): v are the sums, b their bias.  Sixteen
// neighbouring lanes hold a block of 128 columns.
template <int OUT>
__device__ __forceinline__ void finish8(const Proj& p, const Epilogue& e, int64_t row, int64_t col, float (&v)[8],
                                        const float (&b)[8]) {
  const int64_t left = p.N - col;
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] += b[k];
  if (e.pre) store_edge8<FP8Q_BF16>(e.pre, row * e.ldpre + col, v, left, e.vp);
  with_linear_act(e.act, [&](auto act) {
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = linear_act<decltype(act)::value>(v[k]);
  });
  if constexpr (OUT < 2) {
    if (e.res) {
      const int64_t i = row * e.ldr + col;
      if (e.vr && left >= 8) {
        Raw8<OUT> r;
        r.load(e.res, i);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[k] += r[k];
      } else {
#pragma unroll
        for (int k = 0; k < 8; ++k)
          if (k < left) v[k] += OUT == FP8Q_F32 ? ((const float*)e.res)[i + k] : bf_lo(((const uint16_t*)e.res)[i + k]);
      }
    }
    store_edge8<OUT>(p.out, row * p.ldo + col, v, left, e.vo);
  } else {
    // N is a multiple of 128: the sixteen lanes of a block are all here
    constexpr int QF = OUT - 2;
    uint32_t m = 0;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = max(m, abs_bits(v[k]));
    const float s = block_scale7<QF>(__uint_as_float(canon_abs_bits(row16_max(m))), p.eps);
    const float inv = 1.0f / s;
    const bool fast = scale_ok(s);
    const u32x2 q = {encode4<QF>(v[0], v[1], v[2], v[3], s, inv, fast), encode4<QF>(v[4], v[5], v[6], v[7], s, inv, fast)};
    __builtin_nontemporal_store(q, (u32x2*)((uint8_t*)p.out + row * p.ldo + col));
    if ((threadIdx.x & 15) == 0) p.scales[row * p.ld_s + (col >> 7)] = s;
  }
}

// Tiles of BM rows x 256 columns; with kPart, of `splits` parts of K.  The
// sums pass through LDS as fp32, 128 columns at a time where both halves do
// not fit, so that a lane then holds eight consecutive columns: its loads
// and stores are 16 bytes and a block of codes lies in 16 lanes.  Chunk c
// (four floats) of row r sits in slot c ^ (r & 15), free of bank conflicts
// both ways.
template <int FA, int FB, int OUT, bool FAST, int TI_>
__global__ __launch_bounds__(kThreads, 1) void k_linear(const Proj p, const float* __restrict__ s0,
                                                        const float* __restrict__ s1, const Part t, const Epilogue ep,
                                                        const int splits) {
  using S = Shape<FAST, TI_>;
  constexpr int TI = S::TI, BM = S::BM, NST = S::NST;
  constexpr int HALF = BM * 128 * 4, AT_ONCE = 2 * HALF <= S::LDS ? 2 : 1;
  static_assert(HALF <= S::LDS, "a half of the tile's sums fits the stages");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ __attribute__((aligned(16))) float lds_sa[NST][BM];
  const int64_t M = p.M, N = p.N, nkb = p.K / BK;

  for (int64_t tile = blockIdx.x; tile < t.count; tile += gridDim.x) {
    // derived again for every tile: hoisted, it all stays live and spills
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    int64_t tm, tn, part = 0, kb0 = 0, kb1 = nkb, id = tile;
    if constexpr (OUT == kPart) {
      const int64_t tiles = t.ntm * t.ntn;
      part = id / tiles, id -= part * tiles;
      kb0 = part * nkb / splits, kb1 = (part + 1) * nkb / splits;
    }
    tile_of(t.first + (t.halves ? id >> 1 : id), t.ntm * t.ntn, t.ntm, t.ntn, tm, tn);
    const int64_t m0 = t.halves ? (2 * tm + (id & 1)) * BM : tm * BM, n0 = tn * 256;
    if (m0 >= M) continue;  // the lower half of a ragged tile

    v4f acc[TI][TJ];
    tile_product<FA, FB, FAST, TI, false>(p, s0, s1, lds, lds_sa, tid, m0, n0, kb0, kb1, acc);

    __syncthreads();  // every wavefront has read its last stage
#pragma unroll
    for (int h0 = 0; h0 < 2; h0 += AT_ONCE) {
#pragma unroll
      for (int h = h0; h < h0 + AT_ONCE; ++h)
#pragma unroll
        for (int i = 0; i < TI; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const int r = (wm * TI + i) * 16 + lr, c = 8 * wn + 4 * j + lq;
            *(v4f*)(lds + (h - h0) * HALF + r * 512 + 16 * (c ^ (r & 15))) = acc[i][2 * h + j];
          }
      __syncthreads();
#pragma unroll
      for (int h = h0; h < h0 + AT_ONCE; ++h) {
        const int c = 2 * (tid & 15);
        const int64_t col = n0 + 128 * h + 4 * c;
        float b[8];
        if constexpr (OUT != kPart) load_bias8(ep, col, N, b);
        if (col < N) {
#pragma unroll 2
          for (int it = 0; it < BM / 32; ++it) {
            const int r = it * 32 + (tid >> 4);
            const int64_t row = m0 + r;
            if (row >= M) break;
            const uint8_t* at = lds + (h - h0) * HALF + r * 512;
            const v4f x = *(const v4f*)(at + 16 * (c ^ (r & 15))), y = *(const v4f*)(at + 16 * ((c + 1) ^ (r & 15)));
            float v[8] = {x[0], x[1], x[2], x[3], y[0], y[1], y[2], y[3]};
            if constexpr (OUT == kPart) {
              // whole groups of eight: a plane's rows hold them; plain stores, the join reads them next
              float* w = p.ws + (part * M + row) * plane_ld(N) + col;
              *(v4f*)w = x;
              *(v4f*)(w + 4) = y;
            } else {
              finish8<OUT>(p, ep, row, col, v, b);
            }
          }
        }
      }
      __syncthreads();  // before the other half, or the next tile's copies
    }
  }
}

// The planes' sum and the epilogue: eight columns a lane, the planes added in
// their order.
template <int OUT>
__global__ __launch_bounds__(256) void k_linear_join(const Proj p, const Epilogue ep, const int planes) {
  const int64_t N = p.N, nb = (N + 127) / 128, ld = plane_ld(N);
  const int64_t g = (int64_t)blockIdx.x * 16 + (threadIdx.x >> 4);  // a row's 128 columns
  const int64_t row = g / nb, col = (g - row * nb) * 128 + 8 * (threadIdx.x & 15);
  if (row >= p.M || col >= N) return;
  float b[8], v[8];
  load_bias8(ep, col, N, b);
  const float* w = p.ws + row * ld + col;
  const int64_t plane = p.M * ld;
  Raw8<FP8Q_F32> x;
  x.load(w, 0);
#pragma unroll
  for (int k = 0; k < 8; ++k) v[k] = x[k];
#pragma unroll 4
  for (int s = 1; s < planes; ++s) {
    x.load(w, s * plane);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] += x[k];
  }
  finish8<OUT>(p, ep, row, col, v, b);
}

static int launch_join(const Proj& p, const Epilogue& e, int planes, const char* what, hipStream_t st) {
  const int64_t wgs = (p.M * ((p.N + 127) / 128) + 15) / 16;
  const dim3 grid((unsigned)wgs), block(256);
  if (p.scales) {
    if (p.fc == FP8Q_E4M3FN) hipLaunchKernelGGL((k_linear_join<2 + FP8Q_E4M3FN>), grid, block, 0, st, p, e, planes);
    else hipLaunchKernelGGL((k_linear_join<2 + FP8Q_E5M2>), grid, block, 0, st, p, e, planes);
  } else if (p.out_dt == FP8Q_F32) {
    hipLaunchKernelGGL((k_linear_join<FP8Q_F32>), grid, block, 0, st, p, e, planes);
  } else {
    hipLaunchKernelGGL((k_linear_join<FP8Q_BF16>), grid, block, 0, st, p, e, planes);
  }
  return check_launch(what);
}

// How a call goes.  few: the few-row kernel; parts > 1: tiles of so many parts
// of K and the join; otherwise tiles by `cut`.
struct Plan {
  bool few;
  int parts;
  Cut cut;
};
static Plan plan_linear(bool fast, int64_t M, int64_t N, int64_t K) {
  Plan r = {};
  r.few = M <= 64;
  r.parts = 1;
  r.cut = cut_tiles(M, fast ? 256 : 128, (N + 255) / 256, second_launch(K));
  return r;
}

int64_t linear_workspace(bool fast, bool codes, int64_t M, int64_t N, int64_t K) {
  const Plan c = plan_linear(fast, M, N, K);
  if (c.few) return codes ? 4 * M * plane_ld(N) : 0;
  return c.parts > 1 ? 4 * c.parts * M * plane_ld(N) : 0;
}

template <int FA, int FB, int OUT, bool FAST, int TI>
static void launch_tiles(const Proj& p, const Epilogue& e, const Part& t, int parts, hipStream_t st) {
  const int64_t g = grid_size();
  hipLaunchKernelGGL((k_linear<FA, FB, OUT, FAST, TI>), dim3((unsigned)(t.count < g ? t.count : g)), dim3(kThreads), 0, st, p,
                     p.s0, p.s1, t, e, parts);
}

template <int FA, int FB, int OUT, bool FAST>
static void launch_cut(const Proj& p, const Epilogue& e, const Plan& c, hipStream_t st) {
  constexpr int TALL = FAST ? 8 : 4, LOW = TALL / 2;
  const int64_t ntn = (p.N + 255) / 256;
  const int64_t ntm = (p.M + 32 * TALL - 1) / (32 * TALL), ltm = (p.M + 32 * LOW - 1) / (32 * LOW);
  if constexpr (OUT == kPart) {
    launch_tiles<FA, FB, OUT, FAST, LOW>(p, e, {ltm, ntn, 0, ltm * ntn * c.parts, false}, c.parts, st);
  } else if (c.cut.low) {
    launch_tiles<FA, FB, OUT, FAST, LOW>(p, e, {ltm, ntn, 0, ltm * ntn, false}, 1, st);
  } else {
    launch_tiles<FA, FB, OUT, FAST, TALL>(p, e, {ntm, ntn, 0, c.cut.tall, false}, 1, st);
    if (c.cut.split) launch_tiles<FA, FB, OUT, FAST, LOW>(p, e, {ntm, ntn, c.cut.tall, 2 * c.cut.split, true}, 1, st);
  }
}

template <int FA, int FB, bool FAST>
static void launch_out(const Proj& p, const Epilogue& e, const Plan& c, hipStream_t st) {
  if (c.parts > 1) launch_cut<FA, FB, kPart, FAST>(p, e, c, st);
  else if (p.scales) {
    if (p.fc == FP8Q_E4M3FN) launch_cut<FA, FB, 2 + FP8Q_E4M3FN, FAST>(p, e, c, st);
    else launch_cut<FA, FB, 2 + FP8Q_E5M2, FAST>(p, e, c, st);
  } else if (p.out_dt == FP8Q_F32) launch_cut<FA, FB, FP8Q_F32, FAST>(p, e, c, st);
  else launch_cut<FA, FB, FP8Q_BF16, FAST>(p, e, c, st);
}

template <int FA, int FB>
static void launch_f(const Proj& p, const Epilogue& e, bool fast, const Plan& c, hipStream_t st) {
  if (fast) launch_out<FA, FB, true>(p, e, c, st);
  else launch_out<FA, FB, false>(p, e, c, st);
}

int launch_linear(const Proj& q, const Epilogue& e, bool fast, const char* what, hipStream_t st) {
  const Plan c = plan_linear(fast, q.M, q.N, q.K);
  Proj p = q;
  if (c.few) {
    if (!p.scales) return launch_few(p, &e, what, st);
    p.out = p.ws, p.ldo = plane_ld(p.N), p.out_dt = FP8Q_F32, p.scales = nullptr;
    if (int rc = launch_few(p, nullptr, what, st)) return rc;
    return launch_join(q, e, 1, what, st);
  }
  p.B1 = p.B0, p.s1 = p.s0;
  if (p.fa == FP8Q_E4M3FN && p.fb == FP8Q_E4M3FN) launch_f<0, 0>(p, e, fast, c, st);
  else if (p.fa == FP8Q_E5M2 && p.fb == FP8Q_E4M3FN) launch_f<1, 0>(p, e, fast, c, st);
  else if (p.fa == FP8Q_E4M3FN) launch_f<0, 1>(p, e, fast, c, st);
  else launch_f<1, 1>(p, e, fast, c, st);
  if (int rc = check_launch(what)) return rc;
  return c.parts > 1 ? launch_join(q, e, c.parts, what, st) : FP8Q_OK;
}

}  // namespace fp8q

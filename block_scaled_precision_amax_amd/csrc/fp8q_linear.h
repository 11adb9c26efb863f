// The linear layer's tiles: the epilogue and the kernel that runs it behind a
// tile's last block.  Each pair of operand formats is compiled in a file of its
// own (fp8q_linear_<A>_<B>.hip), so that they build side by side; the mathematics,
// the choice of kernel and what bounds them are in fp8q_linear.hip.
#pragma once

#include "fp8q_tiles.h"

namespace fp8q {

// OUT of the kernels below: FP8Q_F32, FP8Q_BF16 or 2 + format (1x128 codes).

// The tiles of a call: the first `full` of the ntm x ntn grid go through all of
// K, the others (`rest`) in `parts` parts of it.
struct Split {
  int64_t ntm, ntn, full, rest;
  int parts;
};

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

// The residual of U rows' columns col .. col + 7, where whole pieces can be
// loaded.  A bf16 one is asked for before the sums are read back, so that it
// comes beside them (8192 x 8192 x 2048 FP8-MFMA with GELU and pre-activations:
// 198 us, loaded where it is added 204; 1024 x 8192 x 4096 exact 66.7 against 68).
// An fp32 one holds twice the registers and is loaded where it is added: early, a
// large product gains 2 % and one of a few rounds, with or without it, loses 1 to 2.
template <int OUT>
using Res8 = Raw8<OUT == FP8Q_F32 ? FP8Q_F32 : FP8Q_BF16>;
template <int OUT>
constexpr bool kEarly = OUT == FP8Q_BF16;
template <int OUT, int U>
__device__ __forceinline__ void load_res8(const Epilogue& e, const int64_t (&row)[U], const bool (&in)[U], int64_t col,
                                          int64_t N, Res8<OUT> (&r)[U]) {
  if (!e.res || !e.vr || N - col < 8) return;
#pragma unroll
  for (int u = 0; u < U; ++u)
    if (in[u]) r[u].load(e.res, row[u] * e.ldr + col);
}

// Everything behind the sums of U rows' columns col .. col + 7 (col a multiple
// of eight, col < N): v are the sums, b their bias, in[u] whether row u exists
// (the same for the sixteen lanes that hold a block of 128 columns).  The rows
// go side by side, so that one's long chain (exponential, reciprocal, block
// maximum, quotient) fills the other's waits.
template <int OUT, int ACT, int U>
__device__ __forceinline__ void finish8(const Proj& p, const Epilogue& e, const int64_t (&row)[U], const bool (&in)[U],
                                        int64_t col, float (&v)[U][8], const float (&b)[8], Res8<OUT> (&res)[U]) {
  const int64_t left = p.N - col;
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] += b[k];
  if (e.pre) {
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in[u]) store_edge8<FP8Q_BF16>(e.pre, row[u] * e.ldpre + col, v[u], left, e.vp);
  }
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[u][k] = linear_act<ACT>(v[u][k]);
  if constexpr (OUT < 2) {
    if (e.res) {
      if (e.vr && left >= 8) {
        if constexpr (!kEarly<OUT>) load_res8<OUT>(e, row, in, col, p.N, res);
#pragma unroll
        for (int u = 0; u < U; ++u)
#pragma unroll
          for (int k = 0; k < 8; ++k) v[u][k] += res[u][k];
      } else {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int64_t i = row[u] * e.ldr + col;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            if (in[u] && k < left)
              v[u][k] += OUT == FP8Q_F32 ? ((const float*)e.res)[i + k] : bf_lo(((const uint16_t*)e.res)[i + k]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u)
      if (in[u]) store_edge8<OUT>(p.out, row[u] * p.ldo + col, v[u], left, e.vo);
  } else {
    // N is a multiple of 128: the sixteen lanes of a block are all here
    constexpr int QF = OUT - 2;
    float s[U], r[U];
    bool ok = true;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float m = 0.0f;
#pragma unroll
      for (int k = 0; k < 8; ++k) m = max_abs(m, v[u][k]);
      s[u] = block_scale7<QF>(__uint_as_float(canon_abs_bits(row16_max(__float_as_uint(m)))), p.eps);
      r[u] = recip(s[u]);
      ok = ok && scale_ok(s[u]);
    }
    auto codes = [&](auto fast) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float(&x)[8] = v[u];
        const bool f = decltype(fast)::value || scale_ok(s[u]);
        const u32x2 q = {encode4<QF>(x[0], x[1], x[2], x[3], s[u], r[u], f), encode4<QF>(x[4], x[5], x[6], x[7], s[u], r[u], f)};
        if (!in[u]) continue;
        __builtin_nontemporal_store(q, (u32x2*)((uint8_t*)p.out + row[u] * p.ldo + col));
        if ((threadIdx.x & 15) == 0) p.scales[row[u] * p.ld_s + (col >> 7)] = s[u];
      }
    };
    if (__all(ok)) codes(std::true_type{});
    else codes(std::false_type{});
  }
}
// One row, any activation.
template <int OUT>
__device__ __forceinline__ void finish8(const Proj& p, const Epilogue& e, int64_t row, int64_t col, float (&v)[1][8],
                                        const float (&b)[8], Res8<OUT> (&res)[1]) {
  const int64_t rows[1] = {row};
  const bool in[1] = {true};
  with_linear_act(e.act, [&](auto act) { finish8<OUT, decltype(act)::value, 1>(p, e, rows, in, col, v, b, res); });
}

// Tiles of BM rows x 256 columns.  The sums of a whole tile pass through LDS as
// fp32, 128 columns at a time where both halves do not fit, so that a lane then
// holds eight consecutive columns: its loads and stores are 16 bytes and a
// block of codes lies in 16 lanes.  Chunk c (four floats) of row r sits in slot
// c ^ (r & 15), free of bank conflicts both ways.  The sums of a part leave as
// the lanes hold them, a register of a wavefront in 1 KB of its tile's plane.
template <int FA, int FB, int OUT, bool FAST, int TI_>
__global__ __launch_bounds__(kThreads, 1) void k_linear(const Proj p, const float* __restrict__ s0,
                                                        const float* __restrict__ s1, const Split t, const Epilogue ep) {
  using S = Shape<FAST, TI_>;
  constexpr int TI = S::TI, BM = S::BM, NST = S::NST;
  constexpr int HALF = BM * 128 * 4, AT_ONCE = 2 * HALF <= S::LDS ? 2 : 1;
  static_assert(HALF <= S::LDS, "a half of the tile's sums fits the stages");
  __shared__ __attribute__((aligned(1024))) uint8_t lds[S::LDS];
  __shared__ __attribute__((aligned(16))) float lds_sa[NST][BM];
  const int64_t M = p.M, N = p.N, nkb = p.K / BK, count = t.full + t.rest * t.parts;

  for (int64_t tile = blockIdx.x; tile < count; tile += gridDim.x) {
    // derived again for every tile: hoisted, it all stays live and spills
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int lane = tid & 63, lr = lane & 15, lq = lane >> 4;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int wm = wave >> 2, wn = wave & 3;
    const bool whole = tile < t.full;
    int64_t id = tile, kb0 = 0, kb1 = nkb;
    if (!whole) {
      const int64_t part = (tile - t.full) / t.rest;
      id = tile - part * t.rest;
      kb0 = part * nkb / t.parts, kb1 = (part + 1) * nkb / t.parts;
    }
    int64_t tm, tn;
    tile_of(id, t.ntm * t.ntn, t.ntm, t.ntn, tm, tn);
    const int64_t m0 = tm * BM, n0 = tn * 256;

    v4f acc[TI][TJ];
    tile_product<FA, FB, FAST, TI, false>(p, s0, s1, lds, lds_sa, tid, m0, n0, kb0, kb1, acc);

    __syncthreads();  // every wavefront has read its last stage
    if (!whole) {
      float* plane = p.ws + (tile - t.full) * (BM * 256) + wave * (TI * TJ * 256) + lane * 4;
#pragma unroll
      for (int i = 0; i < TI; ++i) {
        if (m0 + (wm * TI + i) * 16 >= M) break;  // the join reads no row past M
#pragma unroll
        for (int j = 0; j < TJ; ++j) *(v4f*)(plane + (i * TJ + j) * 256) = acc[i][j];
      }
      continue;
    }
    // the half is a constant: indexed by a variable, the sums would leave the registers
    auto drain = [&](auto first) {
      constexpr int h0 = decltype(first)::value;
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
      with_linear_act(ep.act, [&](auto act) {
        constexpr int U = BM < 128 ? BM / 32 : 4;  // 16384 x 18432 x 7168 FP8-MFMA with GELU: 2136 us, one row at a time 2258
        for (int h = h0; h < h0 + AT_ONCE; ++h) {
          const int c = 2 * (tid & 15);
          const int64_t col = n0 + 128 * h + 4 * c;
          if (col >= N) continue;
          float b[8];
          load_bias8(ep, col, N, b);
          for (int it = 0; it < BM / 32; it += U) {
            int64_t row[U];
            bool in[U];
            float v[U][8];
            Res8<OUT> res[U];
#pragma unroll
            for (int u = 0; u < U; ++u) row[u] = m0 + (it + u) * 32 + (tid >> 4), in[u] = row[u] < M;
            if constexpr (kEarly<OUT>) load_res8<OUT>(ep, row, in, col, N, res);
#pragma unroll
            for (int u = 0; u < U; ++u) {
              const int r = (it + u) * 32 + (tid >> 4);
              const uint8_t* at = lds + (h - h0) * HALF + r * 512;
              const v4f x = *(const v4f*)(at + 16 * (c ^ (r & 15))), y = *(const v4f*)(at + 16 * ((c + 1) ^ (r & 15)));
#pragma unroll
              for (int k = 0; k < 4; ++k) v[u][k] = x[k], v[u][4 + k] = y[k];
            }
            finish8<OUT, decltype(act)::value, U>(p, ep, row, in, col, v, b, res);
          }
        }
      });
      __syncthreads();  // before the other half, or the next tile's copies
    };
    drain(std::integral_constant<int, 0>{});
    if constexpr (AT_ONCE == 1) drain(std::integral_constant<int, 1>{});
  }
}

// The parts' sum and the epilogue, for tiles of 32 ti rows (fp8q_linear.hip).
void launch_linear_join(const Proj& p, const Epilogue& e, const Split& t, int ti, hipStream_t st);

// The tiles of operands of formats FA and FB (low: of half the rows), and the
// join where some have K in parts.
template <int FA, int FB>
void launch_linear_tiles(const Proj& p, const Epilogue& e, bool fast, bool low, const Split& t, hipStream_t st);
#define FP8Q_TILES(FA_, FB_) \
  template <>                \
  void launch_linear_tiles<FA_, FB_>(const Proj&, const Epilogue&, bool, bool, const Split&, hipStream_t)
FP8Q_TILES(FP8Q_E4M3FN, FP8Q_E4M3FN);
FP8Q_TILES(FP8Q_E4M3FN, FP8Q_E5M2);
FP8Q_TILES(FP8Q_E5M2, FP8Q_E4M3FN);
FP8Q_TILES(FP8Q_E5M2, FP8Q_E5M2);
#undef FP8Q_TILES

template <int FA, int FB, int OUT, bool FAST, int TI>
static void launch_tiles(const Proj& p, const Epilogue& e, const Split& t, hipStream_t st) {
  const int64_t g = grid_size(), count = t.full + t.rest * t.parts;
  hipLaunchKernelGGL((k_linear<FA, FB, OUT, FAST, TI>), dim3((unsigned)(count < g ? count : g)), dim3(kThreads), 0, st, p, p.s0,
                     p.s1, t, e);
  if (t.rest) launch_linear_join(p, e, t, TI, st);
}

template <int FA, int FB, int OUT>
static void launch_rows(const Proj& p, const Epilogue& e, bool fast, bool low, const Split& t, hipStream_t st) {
  if (fast) {
    if (low) launch_tiles<FA, FB, OUT, true, 4>(p, e, t, st);
    else launch_tiles<FA, FB, OUT, true, 8>(p, e, t, st);
  } else {
    if (low) launch_tiles<FA, FB, OUT, false, 2>(p, e, t, st);
    else launch_tiles<FA, FB, OUT, false, 4>(p, e, t, st);
  }
}

template <int FA, int FB>
static void launch_out(const Proj& p, const Epilogue& e, bool fast, bool low, const Split& t, hipStream_t st) {
  if (p.scales) {
    if (p.fc == FP8Q_E4M3FN) launch_rows<FA, FB, 2 + FP8Q_E4M3FN>(p, e, fast, low, t, st);
    else launch_rows<FA, FB, 2 + FP8Q_E5M2>(p, e, fast, low, t, st);
  } else if (p.out_dt == FP8Q_F32) launch_rows<FA, FB, FP8Q_F32>(p, e, fast, low, t, st);
  else launch_rows<FA, FB, FP8Q_BF16>(p, e, fast, low, t, st);
}

}  // namespace fp8q

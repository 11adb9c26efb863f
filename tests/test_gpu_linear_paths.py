"""GPU checks of what test_gpu_linear.py leaves out of the layer norm and the linear layer.  Tolerances as there."""
import pytest
import torch

from block_scaled_precision_amax_amd import workloads as W
from test_gpu_linear import (BF, E4, E5, EPS, ERF, GELU, LIPSCHITZ, NONE, RELU, SILU, U, act64, bwd_call, check_codes, operands,
                             product, run_norm)

pytestmark = pytest.mark.gpu

INF = float("inf")


# ------------------------------------------------------------------ the gradient at infinite pre-activations
@pytest.mark.parametrize("act", range(5))
def test_linear_bwd_at_infinite_pre_activations(fq, gpu, act):
    """The derivative is its limit, 1 or 0, and what lies beside an infinite pre-activation keeps its own gradient; the
    output again is what the forward gives."""
    N = 256
    top = torch.finfo(torch.bfloat16).max
    x = torch.tensor([INF, -INF, top, -top, 17.0, -17.0, 200.0, -200.0, 1.0, -1.0, 0.25, -0.0, 6.0, -6.0, 3.0, -0.5] * (N // 16))
    pre = x.to(gpu).bfloat16()[None].expand(3, N).contiguous()
    dC = torch.full((3, N), 1.5, device=gpu)
    D, Ds, Dt, Dts, Ht, Hts, db = bwd_call(fq, dC, pre, act, E4, E4, 3, N)
    p = pre[0].double()
    far = p.abs() > 100
    _, da, _, tda = act64(act, torch.where(far, torch.zeros_like(p), p))
    da = torch.where(far, torch.ones_like(da) if act == NONE else (p > 0).double(), da)
    tda = torch.where(far, torch.zeros_like(tda), tda)
    # three tokens: two additions, and the product's rounding
    assert ((db.double() - 4.5 * da).abs() <= 4.5 * tda + 4 * U * 4.5 * da.abs()).all()
    d, td = (1.5 * t[None].expand(3, N) for t in (da, tda + U * da.abs()))
    check_codes(D, Ds, d, td, E4)
    rows = lambda t: torch.cat([t, t.new_zeros(125, N)]).t().contiguous()  # noqa: E731
    check_codes(Dt, Dts, rows(d), rows(td), E4)
    # the output again, where it is infinite or nothing: +Inf stays, -Inf is NaN for SiLU and both GELUs, 0 for ReLU
    h = torch.where(p == INF, p, torch.zeros_like(p) if act == RELU else p if act == NONE else p * float("nan")).float()
    q, s = torch.empty(N, 128, dtype=torch.uint8, device=gpu), torch.empty(N, 1, device=gpu)
    fq.fp8q_quantize_1x128_t(rows(h[None].expand(3, N)).t().contiguous(), 128, N, N, E4, EPS, q, 128, s, 1)
    at = p.isinf()
    assert torch.equal(Ht[at], q[at]) and torch.equal(Hts[at].nan_to_num(7.0), s[at].nan_to_num(7.0))
    assert Hts[~at].isfinite().all()


@pytest.mark.parametrize("act", [SILU, GELU, ERF, RELU])
def test_an_infinite_pre_activation_spoils_nothing(fq, gpu, act):
    """Many tokens, one +Inf: the gradients are those of a large finite value, bit for bit, in both layouts and the sum."""
    M, N = 300, 384
    pre = W.normal((M, N), seed=2, device=gpu, std=1.7, dtype=torch.bfloat16)
    dC = W.gradient(M, N, seed=1, device=gpu, dtype=torch.bfloat16)
    pre[130, 200] = 1000.0
    want = bwd_call(fq, dC, pre, act, E5, E4, M, N, want_h=False)
    pre[130, 200] = INF
    got = bwd_call(fq, dC, pre, act, E5, E4, M, N, want_h=False)
    assert all(a is None or torch.equal(a, b) for a, b in zip(got, want))


# ------------------------------------------------------------------ layer norm
@pytest.mark.parametrize("rows,cols", [(4, 512), (4, 2304), (2052, 8192)])
def test_layernorm_of_rows_whose_sums_overflow(fq, gpu, rows, cols):
    """Finite rows near fp32's largest value: where only the squares overflow the bias is left, where the sum itself does
    the row is NaN as if it held an Inf, and the other rows know nothing of it."""
    x = torch.randn(rows, cols, device=gpu, generator=torch.Generator(gpu).manual_seed(3))
    b = torch.linspace(-1, 1, cols, device=gpu)
    want = run_norm(fq, x, None, None, b, E4)
    bad = x.clone()
    bad[0] = 1e38
    bad[1] = torch.tensor([1e38, -1e38], device=gpu).repeat(cols // 2)  # every partial sum of a pair is 0
    bad[3] = -3e38
    z, y, q, s, mean, rstd = run_norm(fq, bad, None, None, b, E4)
    assert torch.equal(z, bad)
    for i, sign in ((0, INF), (3, -INF)):
        assert mean[i] == sign and rstd[i] == 0
        assert y[i].isnan().all() and (q[i] == 0x7F).all() and s[i].isnan().all()
    assert mean[1] == 0 and rstd[1] == 0 and torch.equal(y[1], b)
    keep = torch.arange(rows, device=gpu) > 3
    keep[2] = True
    assert all(torch.equal(a[keep], c[keep]) for a, c in zip((z, y, q, s, mean, rstd), want))


@pytest.mark.parametrize("rows,cols,fmt", [(4096, 9088, E4), (4099, 9088, E5), (4101, 16384, E4)])
def test_layernorm_codes_of_walked_bf16_rows(fq, gpu, rows, cols, fmt):
    """Many wide bf16 rows: the codes are the quantizer's of the fp32 norm of the same values, bit for bit."""
    x = (W.activation(rows, cols, seed=2, factor=30.0, device=gpu, dtype=torch.float32) + 3).bfloat16()
    r = W.normal((rows, cols), seed=5, device=gpu, std=2.0, dtype=torch.bfloat16) if rows % 2 else None
    w = 1 + W.normal((cols,), seed=6, device=gpu, std=0.1, dtype=torch.float32)
    b = W.normal((cols,), seed=7, device=gpu, std=0.3, dtype=torch.float32)
    x[7, 5] = float("nan")
    z, y, q, s, mean, rstd = run_norm(fq, x, r, w, b, fmt, pad=64)
    y32 = run_norm(fq, x.float(), None if r is None else r.float(), w, b, fmt, codes=False)[1]
    wq, ws = torch.empty(rows, cols, dtype=torch.uint8, device=gpu), torch.empty(rows, cols // 128, device=gpu)
    fq.fp8q_quantize_1x128(y32, rows, cols, cols, fmt, EPS, wq, cols, ws, cols // 128)
    keep = torch.arange(rows, device=gpu) != 7
    assert torch.equal(q, wq) and torch.equal(s[keep], ws[keep]) and s[7].isnan().all() and (q[7] == 0x7F).all()
    assert torch.equal(y[keep], y32.bfloat16()[keep])


# ------------------------------------------------------------------ gradient of the linear layer: the order of its tiles
@pytest.mark.parametrize("M,N", [(2100, 640), (2305, 1024), (2049, 256), (4000, 384)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_linear_bwd_of_many_blocks_both_ways(fq, gpu, M, N, dt):
    """More than sixteen token blocks and several feature blocks, whose last group of token blocks is short: without an
    activation the quantizers' codes, bit for bit; with one against 64 bits; the bias's gradient in both."""
    padT = lambda t: torch.cat([t, t.new_zeros(-M % 128, N)]).t().contiguous()  # noqa: E731
    Mp = M + -M % 128
    dC = W.gradient(M, N, seed=1, device=gpu, dtype=dt)
    pre = W.normal((M, N), seed=2, device=gpu, std=1.7, dtype=torch.bfloat16)
    blocks = -(-M // 128)
    n = 2 + 2 + 8 + -(-blocks // 16) + 16

    D, Ds, Dt, Dts, Ht, Hts, db = bwd_call(fq, dC, pre, NONE, E5, E4, M, N)
    q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
    fq.fp8q_quantize_1x128(dC, M, N, N, E5, EPS, q, N, s, N // 128)
    assert torch.equal(D, q) and torch.equal(Ds, s)
    for t, fmt, codes, scales in ((dC, E5, Dt, Dts), (pre, E4, Ht, Hts)):
        q, s = torch.empty(N, Mp, dtype=torch.uint8, device=gpu), torch.empty(N, Mp // 128, device=gpu)
        fq.fp8q_quantize_1x128_t(padT(t).t().contiguous(), Mp, N, N, fmt, EPS, q, Mp, s, Mp // 128)
        assert torch.equal(codes, q) and torch.equal(scales, s)
    d = dC.double()
    assert ((db.double() - d.sum(0)).abs() <= n * U * d.abs().sum(0)).all()

    act = GELU if N % 256 else SILU
    D, Ds, Dt, Dts, Ht, Hts, db = bwd_call(fq, dC, pre, act, E4, E5, M, N)
    h, da, th, tda = act64(act, pre)
    d, td = d * da, d.abs() * tda + U * (d * da).abs()
    check_codes(D, Ds, d, td, E4)
    check_codes(Dt, Dts, padT(d), padT(td), E4)
    check_codes(Ht, Hts, padT(h), padT(th + U * h.abs()), E5)
    assert ((db.double() - d.sum(0)).abs() <= n * U * d.abs().sum(0) + td.sum(0)).all()


# ------------------------------------------------------------------ the linear layer's tiles
# Shapes that go as tiles on 256 compute units, and whether some of them have K in parts (exact | FP8-MFMA).
TILES = [((65, 256, 7168), (True, True)), ((65, 9088, 512), (False, False)), ((200, 18432, 4096), (True, False)),
         ((1000, 8960, 2048), (True, False)), ((3000, 4096, 512), (False, False)), ((1000, 18432, 4096), (True, True)),
         ((385, 18432, 7168), (False, True))]


def check_way(fq, fast, M, N, K, parts):
    """Tiles, not the few-row kernel, whose codes take 4 M N bytes; with parts of K or not."""
    need = [fq.fp8q_linear_blockscaled_workspace(int(fast), codes, M, N, K) for codes in (0, 1)]
    if torch.cuda.get_device_properties(0).multi_processor_count == 256:
        assert need[0] == need[1] and (need[0] > 0) == parts


@pytest.mark.parametrize("shape,parts", TILES)
@pytest.mark.parametrize("fast", [False, True])
def test_tiles_with_bf16_residual_and_bias_and_transposed_scales(fq, gpu, shape, parts, fast):
    """Against 64 bits on rows from every part of a tile, and every element against the fp32 output without the residual;
    rows aligned and not, widths of no whole eight, in place."""
    M, N, K = shape
    check_way(fq, fast, M, N, K, parts[fast])
    i = [s for s, _ in TILES].index(shape)
    fa, fb = i % 2, (i // 2) % 2
    A, sA, B, sB = operands(gpu, M, N, K, fa, fb, seed=i)
    sAt, sBt = sA.t().contiguous(), sB.t().contiguous()
    f = fq.fp8q_linear_blockscaled_fast if fast else fq.fp8q_linear_blockscaled
    rows = torch.tensor(sorted({r for e in range(0, M, 64) for r in (e + 1, e + 16, e + 47) if r < M} | {0, M - 1})[:40]
                        + [M - 2, M - 1], device=gpu)
    v, D = product(A[rows], fa, sA[rows], B, fb, sB, K)
    for n, act, extra in ((N, i % 5, 8), (N - 3, (i + 2) % 5, 8), (N - 3, (i + 3) % 5, 0), (N, (i + 1) % 5, 1)):
        # rows of whole sixteen bytes, or (extra 0 and 1) elements alone are aligned
        ld = (n + 7) // 8 * 8 + extra if extra != 1 else n + 1
        off = 0 if extra == 8 else 1
        ld += off
        bias = W.normal((n,), seed=3, device=gpu, dtype=torch.bfloat16 if (i + n) % 2 else torch.float32)
        buf = W.normal((M, ld), seed=5, device=gpu, std=2.0, dtype=torch.bfloat16)
        res = buf[:, off:off + n]

        def run(C, res, bias=bias, act=act, n=n):
            f(A, fa, K, sAt, 1, M, B, fb, K, sBt, 1, sBt.shape[1], bias, act, res, 0 if res is None else res.stride(0), C,
              C.stride(0), None, 0, M, n, K)

        C = torch.full((M, ld), 7.0, dtype=torch.bfloat16, device=gpu)
        run(C[:, off:], res)
        C0 = torch.empty(M, n, device=gpu)
        run(C0, None)
        w = v[:, :n] + bias.double()
        tv = (2.0 ** -10 if fast else 1e-5) * D[:, :n] + 2 * U * w.abs()
        want, _, ta, _ = act64(act, w)
        assert ((C0[rows].double() - want).abs() <= LIPSCHITZ * tv + 1.01 * ta + U * want.abs()).all()
        want = want + res[rows].double()
        tol = LIPSCHITZ * tv + 1.01 * ta + U * want.abs()
        assert ((C[rows, off:off + n].double() - want).abs() <= 1.01 * tol + BF * want.abs()).all()
        assert torch.equal(C[:, off:off + n], (C0 + res.float()).bfloat16())
        assert (C[:, :off] == 7).all() and (C[:, off + n:] == 7).all()
        beside = buf[:, off + n:].clone()
        run(res, res)  # the residual stream updated in place
        assert torch.equal(res, C[:, off:off + n]) and torch.equal(buf[:, off + n:], beside)


@pytest.mark.parametrize("fa", [E4, E5])
@pytest.mark.parametrize("fb", [E4, E5])
def test_tiles_of_every_pair_of_formats(fq, gpu, fa, fb):
    """Whole tiles and tiles in parts of K, exact and FP8-MFMA: every element against 64 bits."""
    for (M, N, K), parts in TILES[:2]:
        A, sA, B, sB = operands(gpu, M, N, K, fa, fb, seed=M + 2 * fa + fb)
        v, D = product(A, fa, sA, B, fb, sB, K)
        for fast in (False, True):
            check_way(fq, fast, M, N, K, parts[fast])
            C = torch.full((M, N), float("nan"), device=gpu)
            f = fq.fp8q_linear_blockscaled_fast if fast else fq.fp8q_linear_blockscaled
            f(A, fa, K, sA, K // 128, 1, B, fb, K, sB, K // 128, 1, None, NONE, None, 0, C, N, None, 0, M, N, K)
            assert ((C.double() - v).abs() <= (2.0 ** -10 if fast else 1e-5) * D).all()


def test_raw_pointers_without_a_workspace(fq, gpu):
    """A's address alone, and addresses throughout: the workspace comes from the device at hand; few rows and parts of K."""
    for M, N, K in ((3, 256, 512), (65, 256, 7168)):
        A, sA, B, sB = operands(gpu, M, N, K, seed=M)
        bias = W.normal((N,), seed=3, device=gpu)
        outs = []
        for p in (lambda t: t, lambda t: t.data_ptr() if t is A else t, lambda t: t.data_ptr() if t is not bias else t):
            q, s = torch.zeros(M, N, dtype=torch.uint8, device=gpu), torch.zeros(M, N // 128, device=gpu)
            fq.fp8q_linear_blockscaled_q(p(A), E4, K, p(sA), K // 128, 1, p(B), E4, K, p(sB), K // 128, 1, p(bias), GELU, E4, EPS,
                                         p(q), N, p(s), N // 128, None, 0, M, N, K)
            outs.append((q, s))
        q, s = torch.zeros(M, N, dtype=torch.uint8, device=gpu), torch.zeros(M, N // 128, device=gpu)
        a = [t.data_ptr() for t in (A, sA, B, sB, q, s)]
        fq.fp8q_linear_blockscaled_q(a[0], E4, K, a[1], K // 128, 1, a[2], E4, K, a[3], K // 128, 1, None, GELU, E4, EPS, a[4], N,
                                     a[5], N // 128, None, 0, M, N, K)
        q2, s2 = torch.zeros_like(q), torch.zeros_like(s)
        fq.fp8q_linear_blockscaled_q(A, E4, K, sA, K // 128, 1, B, E4, K, sB, K // 128, 1, None, GELU, E4, EPS, q2, N, s2, N // 128,
                                     None, 0, M, N, K)
        assert torch.equal(q, q2) and torch.equal(s, s2)
        assert all(torch.equal(o[0], outs[0][0]) and torch.equal(o[1], outs[0][1]) for o in outs)

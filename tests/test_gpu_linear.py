"""GPU checks of the layer norm and the linear layer (forward in four forms,
gradient at the pre-activations) against plain implementations in 64 bits.

Tolerances, with u = 2^-24 (half an fp32 step): a chain of n fp32 additions is
off by at most n*u of the sum of magnitudes, a rounding to bf16 by 2^-8 of the
value, to E4M3 by 2^-4 and to E5M2 by 2^-3 (or half the format's smallest
step times the scale).  Products keep the block-scaled GEMM's bounds: 1e-5 of
the sum of magnitudes D on the exact path, 2^-10 of it on the FP8 matrix
cores.
"""
import math

import numpy as np
import pytest
import torch

from block_scaled_precision_amax_amd import workloads as W

pytestmark = pytest.mark.gpu

E4, E5 = 0, 1
MAXF = {E4: 448.0, E5: 57344.0}
HALF = {E4: 2.0 ** -4, E5: 2.0 ** -3}        # half a step, relative
TINY = {E4: 2.0 ** -10, E5: 2.0 ** -17}      # half the smallest step
EPS, NEPS = 1e-12, 1e-5
U = 2.0 ** -24
BF = 2.0 ** -8
F8 = {E4: torch.float8_e4m3fn, E5: torch.float8_e5m2}
SILU, GELU, NONE, RELU, ERF = range(5)
C0, A0 = math.sqrt(2 / math.pi), 0.044715


def strided(t, extra, fill=-3.0):
    """The same values in rows `extra` elements further apart, as the whole buffer."""
    b = torch.full((t.shape[0], t.shape[1] + extra), fill, dtype=t.dtype, device=t.device)
    b[:, :t.shape[1]] = t
    return b


# ------------------------------------------------------------------ activations in 64 bits, and their errors in fp32
def act64(act, x):
    """act(x), act'(x), and bounds of the errors of both in fp32."""
    x = x.double()
    if act == NONE:
        return x, torch.ones_like(x), 0 * x, 0 * x
    if act == RELU:
        return x.clamp(min=0), (x > 0).double(), 0 * x, 0 * x
    if act == ERF:
        # P within (1.5 x^2 + 16) u of its smaller tail; a product or two more
        # (by erfc: ndtr on the GPU is 1 + erf, whose lower tail cancels)
        p, d = 0.5 * torch.erfc(x * -math.sqrt(0.5)), torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
        rel = (1.5 * x * x + 20) * U
        return x * p, p + x * d, (x * p).abs() * rel + 1e-36, (p + x.abs() * d) * rel + 1e-36
    if act == SILU:
        # the sigmoid is within (1.25 |x| + 5) u; its gradient p (1 + x (1 - p)) has it twice and four roundings
        p = torch.sigmoid(x)
        rel = (1.25 * x.abs() + 7) * U
        return x * p, p * (1 + x * (1 - p)), (x * p).abs() * rel + 1e-35, p * (1 + x.abs()) * 2 * rel + 1e-35
    # GELU (tanh): p = sigmoid(z), z = 2 c (x + a x^3) within 5 u of its value, and (1.25 |z| + 5) u of the sigmoid;
    # 1 - p is off by u and what p is off by
    z = 2 * C0 * (x + A0 * x ** 3)
    p = torch.sigmoid(z)
    rel = (6.5 * z.abs() + 8) * U
    g = C0 * (1 + 3 * A0 * x * x)
    grad = p + x * 2 * p * (1 - p) * g
    return x * p, grad, (x * p).abs() * rel + 1e-35, p * rel + x.abs() * g * 4 * p * (rel + U) + 1e-35


LIPSCHITZ = 1.13  # |act'| of all five


# ------------------------------------------------------------------ layer norm
def norm_ref(x, r, w, b):
    """v, mean, rstd, y in 64 bits and the bounds of the last three."""
    v = x.double() + (r.double() if r is not None else 0)
    m = v.mean(1, keepdim=True)
    d = v - m
    var = (d * d).mean(1, keepdim=True)
    rs = 1 / torch.sqrt(var + NEPS)
    wd = w.double() if w is not None else torch.ones(1, dtype=torch.float64, device=x.device)
    y = d * rs * wd + (b.double() if b is not None else 0)
    # v is rounded once; sums: 64 additions a lane, 6 across lanes, 16 across wavefronts, a division
    tm = 90 * U * v.abs().mean(1, keepdim=True)
    # the mean's error enters the variance squared; the differences and squares are rounded once each, v once
    tv = 96 * U * var + 2 * U * (v.abs() * d.abs()).mean(1, keepdim=True) * 2 + tm * tm
    trs = (0.5 * tv / (var + NEPS) + 5 * U) * rs
    ty = wd.abs() * ((tm + U * d.abs() + U * v.abs()) * rs + d.abs() * (trs + 4 * U * rs)) + 2 * U * y.abs()
    return v, m[:, 0], rs[:, 0], y, tm[:, 0], trs[:, 0], ty


def run_norm(fq, x, r, w, b, fmt, pad=0, want_y=True, want_z=True, codes=True, stream=None):
    rows, cols = x.shape
    ld, dev = cols + pad, x.device
    xb = strided(x, pad) if pad else x
    rb = strided(r, pad) if pad and r is not None else r
    z = torch.full((rows, ld), 7.0, dtype=x.dtype, device=dev) if want_z else None
    y = torch.full((rows, ld), 7.0, dtype=x.dtype, device=dev) if want_y else None
    q = torch.full((rows, ld), 0xAA, dtype=torch.uint8, device=dev) if codes else None
    s = torch.full((rows, cols // 128 + pad), -7.0, device=dev) if codes else None
    mean, rstd = torch.full((rows + 1,), 9.0, device=dev), torch.full((rows + 1,), 9.0, device=dev)
    fq.fp8q_layernorm_1x128(xb, ld, rb, ld, w, b, rows, cols, NEPS, z, ld, y, ld, fmt, EPS, q, ld, s,
                            s.shape[1] if codes else 0, mean, rstd, stream=stream)
    torch.cuda.synchronize()
    assert mean[rows] == 9 and rstd[rows] == 9
    if pad:
        assert all((t[:, cols:] == f).all() for t, f in ((q, 0xAA), (z, 7), (y, 7)) if t is not None)
        assert s is None or (s[:, cols // 128:] == -7).all()
    cut = lambda t: None if t is None else t[:, :cols]  # noqa: E731
    return cut(z), cut(y), cut(q), None if s is None else s[:, :cols // 128], mean[:rows], rstd[:rows]


@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 40), (1, 128), (1, 7168), (5, 256), (3, 640), (7, 1152), (5, 1608), (33, 2048),
                                       (2, 2176), (4, 2504), (6, 4096), (9, 7168), (3, 10368), (2, 16384), (2, 18432),
                                       (2, 20008), (1, 65536)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layernorm(fq, orc, gpu, rows, cols, dt):
    fmt = E4 if rows % 2 else E5
    codes = cols % 128 == 0
    x = (W.activation(rows, cols, seed=rows + cols, factor=30.0, device=gpu, dtype=torch.float32) + 3).to(dt)
    r = W.normal((rows, cols), seed=5, device=gpu, std=2.0, dtype=dt) if cols not in (640, 40) else None
    w = 1 + W.normal((cols,), seed=6, device=gpu, std=0.1, dtype=torch.float32) if cols != 2176 else None
    b = W.normal((cols,), seed=7, device=gpu, std=0.3, dtype=torch.float32) if cols not in (256, 2504) else None
    if cols in (1152, 1608, 20008):
        w, b = w.bfloat16(), b.bfloat16()
    z, y, q, s, mean, rstd = run_norm(fq, x, r, w, b, fmt, pad=64 if rows in (3, 5, 33) else 0, codes=codes)
    v, m, rs, yr, tm, trs, ty = norm_ref(x, r, w, b)
    assert ((mean.double() - m).abs() <= tm).all()
    assert ((rstd.double() - rs).abs() <= trs).all()
    assert ((y.double() - yr).abs() <= ty + (BF * (yr.abs() + ty) if dt == torch.bfloat16 else 0)).all()
    # the stored sum is the sum rounded once
    assert torch.equal(z, (x.float() + (r.float() if r is not None else 0)).to(dt))
    if codes:  # those the quantizer makes of the fp32 norm
        y32 = y if dt == torch.float32 else run_norm(fq, x.float(), None if r is None else r.float(), w, b, fmt)[1]
        wq, ws = orc.quantize_blocks(np.ascontiguousarray(y32.cpu().numpy()), 1, 128, fmt)
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("rows,cols,dt", [(2050, 4104, torch.float32), (2051, 8192, torch.float32), (4100, 8200, torch.bfloat16),
                                          (4099, 16384, torch.float32), (4096, 9088, torch.bfloat16)])
def test_layernorm_of_many_wide_rows(fq, gpu, rows, cols, dt):
    """Rows walked by one workgroup a compute unit: against 64 bits, in place, codes as the quantizer makes them."""
    codes = cols % 128 == 0
    x = (W.activation(rows, cols, seed=2, factor=30.0, device=gpu, dtype=torch.float32) + 3).to(dt)
    r = W.normal((rows, cols), seed=5, device=gpu, std=2.0, dtype=dt) if rows % 2 else None
    w = 1 + W.normal((cols,), seed=6, device=gpu, std=0.1, dtype=torch.float32)
    b = W.normal((cols,), seed=7, device=gpu, std=0.3, dtype=torch.float32) if rows != 2051 else None
    x[7, 5] = float("nan")
    z, y, q, s, mean, rstd = run_norm(fq, x, r, w, b, E4, pad=64, codes=codes)
    keep = torch.arange(rows, device=gpu) != 7
    assert y[7].isnan().all() and y[keep].isfinite().all()
    for a in range(0, rows, 1024):
        k = torch.arange(a, min(rows, a + 1024), device=gpu)
        k = k[k != 7]
        v, m, rs, yr, tm, trs, ty = norm_ref(x[k], None if r is None else r[k], w, b)
        assert ((mean[k].double() - m).abs() <= tm).all() and ((rstd[k].double() - rs).abs() <= trs).all()
        assert ((y[k].double() - yr).abs() <= ty + (BF * (yr.abs() + ty) if dt == torch.bfloat16 else 0)).all()
    zf = (x.float() + (r.float() if r is not None else 0)).to(dt)
    assert torch.equal(z[keep], zf[keep])
    if codes and dt == torch.float32:
        wq, wsc = torch.empty(rows, cols, dtype=torch.uint8, device=gpu), torch.empty(rows, cols // 128, device=gpu)
        y = y.contiguous()
        fq.fp8q_quantize_1x128(y, rows, cols, cols, E4, EPS, wq, cols, wsc, cols // 128)
        assert torch.equal(q, wq) and torch.equal(s[keep], wsc[keep]) and s[7].isnan().all()
    a = x.clone()
    y2 = torch.empty_like(x)
    fq.fp8q_layernorm_1x128(a, cols, r, cols, w, b, rows, cols, NEPS, a, cols, y2, cols, E4, EPS, None, 0, None, 0)
    assert torch.equal(a[keep], zf[keep]) and torch.equal(y2[keep], y[:, :cols][keep])


def test_layernorm_codes_of_extreme_blocks(fq, orc, gpu):
    """Blocks whose scale leaves the quick quotient's range."""
    cols = 640
    x = torch.randn(6, cols, device=gpu)
    w = torch.ones(cols, device=gpu)
    w[128:256], w[256:384], w[384:512] = 1e30, 1e-35, 0.0
    for eps in (1e-12, 1e-37):
        for fmt in (E4, E5):
            y, q, s = torch.empty_like(x), torch.empty(6, cols, dtype=torch.uint8, device=gpu), torch.empty(6, 5, device=gpu)
            fq.fp8q_layernorm_1x128(x, cols, None, 0, w, None, 6, cols, NEPS, None, 0, y, cols, fmt, eps, q, cols, s, 5)
            wq, wsc = torch.empty_like(q), torch.empty_like(s)
            fq.fp8q_quantize_1x128(y, 6, cols, cols, fmt, eps, wq, cols, wsc, 5)
            assert torch.equal(q, wq) and torch.equal(s, wsc)


def test_layernorm_far_from_zero(fq, gpu):
    """Rows whose mean is a thousand times their spread: the variance is not lost."""
    x = 1000 + torch.randn(6, 2048, device=gpu, generator=torch.Generator(gpu).manual_seed(1))
    _, y, _, _, mean, rstd = run_norm(fq, x, None, None, None, E4)
    v, m, rs, yr, tm, trs, ty = norm_ref(x, None, None, None)
    assert ((rstd.double() - rs).abs() <= trs).all() and (trs < 1e-2 * rs).all()
    assert ((y.double() - yr).abs() <= ty).all()


def test_layernorm_optional_outputs_and_in_place(fq, gpu):
    rows, cols = 10, 1024
    x = W.activation(rows, cols, seed=1, factor=5.0, device=gpu, dtype=torch.bfloat16)
    r = W.normal((rows, cols), seed=2, device=gpu, dtype=torch.bfloat16)
    w, b = torch.ones(cols, device=gpu), torch.zeros(cols, device=gpu)
    z, y, q, s, mean, rstd = run_norm(fq, x, r, w, b, E4)
    # ones and zeros are what an absent weight and bias stand for
    for ww, bb in ((None, None), (w, None), (None, b)):
        z2, y2, q2, s2, m2, r2 = run_norm(fq, x, r, ww, bb, E4)
        assert all(torch.equal(a, c) for a, c in ((z, z2), (y, y2), (q, q2), (s, s2), (mean, m2), (rstd, r2)))
    _, y2, q2, s2, _, _ = run_norm(fq, x, r, w, b, E4, want_y=False, want_z=False)
    assert torch.equal(q, q2) and torch.equal(s, s2) and y2 is None
    y3 = torch.empty_like(x)
    fq.fp8q_layernorm_1x128(x, cols, r, cols, w, b, rows, cols, NEPS, None, 0, y3, cols, E4, EPS, None, 0, None, 0)
    assert torch.equal(y, y3)
    for which in (0, 1):  # z over x, and over the residual
        a, c = x.clone(), r.clone()
        q4, s4 = torch.empty_like(q), torch.empty_like(s)
        fq.fp8q_layernorm_1x128(a, cols, c, cols, w, b, rows, cols, NEPS, (a, c)[which], cols, None, 0, E4, EPS, q4, cols, s4,
                                cols // 128)
        assert torch.equal((a, c)[which], z) and torch.equal(q4, q) and torch.equal(s4, s)
        assert torch.equal((c, a)[which], (r, x)[which])


@pytest.mark.parametrize("cols", [512, 2304])
def test_layernorm_special_rows(fq, gpu, cols):
    x = torch.randn(7, cols, device=gpu)
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 7] = float("inf")
    x[3] = 5.0
    x[4] = torch.linspace(-1e25, 1e25, cols, device=gpu)
    x[5, 9] = -float("inf")
    b = torch.linspace(-1, 1, cols, device=gpu)
    z, y, q, s, mean, rstd = run_norm(fq, x, None, None, b, E4)
    for i in (0, 3):  # constant rows: no spread, the bias alone
        assert torch.equal(y[i], b) and torch.allclose(rstd[i], torch.tensor(NEPS, device=gpu).rsqrt())
    assert mean[3] == 5
    for i in (1, 2, 5):
        assert y[i].isnan().all() and (q[i] == 0x7F).all() and s[i].isnan().all() and rstd[i].isnan()
    assert rstd[4] == 0 and torch.equal(y[4], b)  # the sum of squares overflows
    yr, ty = norm_ref(x[6:], None, None, b)[3::3]
    assert ((y[6:].double() - yr).abs() <= ty).all()


def bwd_ref(dy, z, w, mean, rstd, dres):
    dy, z = dy.double(), z.double()
    m, rs = mean.double()[:, None], rstd.double()[:, None]
    xh = (z - m) * rs
    t = dy * (w.double() if w is not None else 1)
    a, k = t.mean(1, keepdim=True), (t * xh).mean(1, keepdim=True)
    dx = rs * (t - a - xh * k)
    mag = rs * (t.abs() + t.abs().mean(1, keepdim=True) + xh.abs() * (t * xh).abs().mean(1, keepdim=True))
    if dres is not None:
        dx = dx + dres.double()
    return dx, (dy * xh).sum(0), dy.sum(0), mag, (dy * xh).abs().sum(0), dy.abs().sum(0)


@pytest.mark.parametrize("rows,cols", [(1, 8), (3, 40), (1, 128), (3, 384), (2500, 128), (41, 1024), (700, 1608), (2300, 1920),
                                       (700, 2304), (9, 7168), (1300, 4096), (701, 2504), (513, 4096), (5, 16384), (3, 18432), (2, 20008), (1, 65536)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_layernorm_bwd(fq, gpu, rows, cols, dt):
    pad = 64 if rows % 2 else 0
    z = (W.activation(rows, cols, seed=rows, factor=20.0, device=gpu, dtype=torch.float32) - 2).to(dt)
    dy = W.gradient(rows, cols, seed=3, device=gpu, dtype=dt)
    dres = W.normal((rows, cols), seed=4, device=gpu, std=1e-3, dtype=dt) if cols not in (1024, 40) else None
    w = 1 + W.normal((cols,), seed=6, device=gpu, std=0.1, dtype=torch.float32) if cols != 1920 else None
    if cols in (2304, 1608):
        w = w.bfloat16()
    zd = z.double()
    mean = zd.mean(1).float()
    rstd = ((zd - zd.mean(1, keepdim=True)).square().mean(1) + NEPS).rsqrt().float()
    ws_bytes = fq.fp8q_layernorm_bwd_workspace(rows, cols)
    guard = torch.full((ws_bytes // 4 + 64,), 5.0, device=gpu)
    dx = torch.full((rows, cols + pad), 7.0, dtype=dt, device=gpu)
    dw, db = torch.full((cols + 4,), 3.0, device=gpu), torch.full((cols + 4,), 3.0, device=gpu)
    sp = lambda t: None if t is None else strided(t, pad) if pad else t  # noqa: E731
    ld = cols + pad
    zb, dyb, drb = sp(z), sp(dy), sp(dres)

    def call(dw, db):
        fq.fp8q_layernorm_bwd(dyb, ld, zb, ld, w, mean, rstd, drb, ld, rows, cols, dx, ld, dw, db, guard, ws_bytes)
        torch.cuda.synchronize()
        return dx.clone()

    first = call(dw, db)
    assert (guard[ws_bytes // 4:] == 5).all(), "wrote past the workspace"
    assert (dw[cols:] == 3).all() and (db[cols:] == 3).all() and (first[:, cols:] == 7).all()
    want, want_w, want_b, mag, mag_w, mag_b = bwd_ref(dy, z, w, mean, rstd, dres)
    # 64 fused additions a lane, 22 across lanes and wavefronts, then a handful of products
    tol = 100 * U * mag + 4 * U * want.abs() + (BF * want.abs() if dt == torch.bfloat16 else 0)
    assert ((first[:, :cols].double() - want).abs() <= tol).all()
    # rows of one workgroup, its four row groups, the partial rows a sixteenth at a time, and four roundings of a term
    parts = ws_bytes // (8 * cols)
    n = -(-rows // parts) + 4 + -(-parts // 16) + 16 + 4
    assert ((dw[:cols].double() - want_w).abs() <= n * U * mag_w).all()
    assert ((db[:cols].double() - want_b).abs() <= n * U * mag_b).all()
    # the same bits again; each sum alone; neither; and sums whose stores are not 16-byte aligned
    for kw, kb in ((1, 1), (1, 0), (0, 1), (0, 0)):
        for off in (0, 1):
            dw2, db2 = torch.full((cols + 4,), 3.0, device=gpu), torch.full((cols + 4,), 3.0, device=gpu)
            assert torch.equal(call(dw2[off:] if kw else None, db2[off:] if kb else None), first)
            for k, a, c in ((kw, dw2, dw), (kb, db2, db)):
                assert torch.equal(a[off:off + cols], c[:cols]) if k else (a == 3).all()


def test_layernorm_bwd_in_place_and_differences(fq, gpu):
    rows, cols = 3, 256
    g = torch.Generator().manual_seed(0)
    x, dy = (torch.randn(rows, cols, dtype=torch.float64, generator=g) for _ in range(2))
    w, b = 1 + 0.1 * torch.randn(cols, dtype=torch.float64, generator=g), torch.zeros(cols, dtype=torch.float64)

    def loss(x, w, b):
        d = x - x.mean(1, keepdim=True)
        return float((d / torch.sqrt((d * d).mean(1, keepdim=True) + NEPS) * w + b).mul(dy).sum())

    xg, dyg, wg = x.float().to(gpu), dy.float().to(gpu), w.float().to(gpu)
    mean = xg.double().mean(1).float()
    rstd = (xg.double().var(1, correction=0) + NEPS).rsqrt().float()
    ws = torch.empty(fq.fp8q_layernorm_bwd_workspace(rows, cols), dtype=torch.uint8, device=gpu)
    dx, dw, db = torch.empty_like(xg), torch.empty(cols, device=gpu), torch.empty(cols, device=gpu)
    args = (cols, xg, cols, wg, mean, rstd)
    fq.fp8q_layernorm_bwd(dyg, *args, None, 0, rows, cols, dx, cols, dw, db, ws, ws.numel())
    h = 1e-5
    for i, j in ((0, 0), (1, 77), (2, 255)):
        for t, got in ((x, dx[i, j]), (w, dw[j]), (b, db[j])):
            at = (i, j) if t is x else (j,)
            t[at] += h
            up = loss(x, w, b)
            t[at] -= 2 * h
            dn = loss(x, w, b)
            t[at] += h
            # the difference is off by h^2 f'''/6 and its rounding, the gradient by some fp32 steps of sums of 256
            assert abs(float(got) - (up - dn) / (2 * h)) <= 2e-5 * max(1.0, abs(float(got)))
    # over dy, and over the residual's gradient
    a = dyg.clone()
    fq.fp8q_layernorm_bwd(a, *args, None, 0, rows, cols, a, cols)
    assert torch.equal(a, dx)
    r = torch.randn(rows, cols, device=gpu)
    want = torch.empty_like(r)
    fq.fp8q_layernorm_bwd(dyg, *args, r, cols, rows, cols, want, cols)
    fq.fp8q_layernorm_bwd(dyg, *args, r, cols, rows, cols, r, cols)
    assert torch.equal(r, want)


# ------------------------------------------------------------------ linear
def operands(gpu, M, N, K, fa=E4, fb=E4, pad=0, seed=0):
    """Codes and scales of A (1x128) and B (128x128) on the GPU, rows `pad` bytes further apart."""
    A = strided(W.fp8_codes((M, K), fa, seed=seed, device=gpu), pad, 0x55)
    B = strided(W.fp8_codes((N, K), fb, seed=seed + 1, device=gpu), pad, 0x55)
    g = torch.Generator(device=gpu).manual_seed(seed + 2)
    sA = torch.rand(M, K // 128, generator=g, device=gpu) * (2 / MAXF[fa]) + 0.1 / MAXF[fa]
    sB = torch.rand(-(-N // 128), K // 128, generator=g, device=gpu) * (0.4 / MAXF[fb]) + 0.1 / MAXF[fb]
    return A, sA, B, sB


def product(A, fa, sA, B, fb, sB, K):
    """The product and the sum of magnitudes in 64 bits."""
    a = A[:, :K].contiguous().view(F8[fa]).double() * sA.double().repeat_interleave(128, 1)
    b = B[:, :K].contiguous().view(F8[fb]).double() * sB.double().repeat_interleave(128, 0)[:B.shape[0]].repeat_interleave(128, 1)
    return torch.mm(a, b.t()), torch.mm(a.abs(), b.abs().t())


def call(fq, A, fa, sA, B, fb, sB, bias, act, out, M, N, K, fast=False, res=None, pre=None, q=None, **kw):
    Kb = K // 128
    a = (A, fa, A.stride(0), sA, Kb, 1, B, fb, B.stride(0), sB, Kb, 1, bias, act)
    p = (pre, pre.stride(0) if pre is not None else 0, M, N, K)
    if q is not None:
        fc, s = q
        f = fq.fp8q_linear_blockscaled_q_fast if fast else fq.fp8q_linear_blockscaled_q
        f(*a, fc, EPS, out, out.stride(0), s, s.stride(0), *p, **kw)
    else:
        f = fq.fp8q_linear_blockscaled_fast if fast else fq.fp8q_linear_blockscaled
        f(*a, res, 0 if res is None else res.stride(0), out, out.stride(0), *p, **kw)


SHAPES = [(1, 128, 128), (1, 1000, 1024), (2, 7, 256), (15, 130, 384), (16, 384, 640), (17, 1000, 256), (33, 256, 1152),
          (48, 72, 2176), (64, 129, 512), (65, 128, 128), (70, 260, 384), (128, 256, 256), (129, 384, 640), (200, 40, 4096),
          (257, 200, 512), (300, 1152, 1280)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fast", [False, True])
def test_linear(fq, gpu, M, N, K, fast):
    i = SHAPES.index((M, N, K))
    fa, fb, act, pad = (i // 2) % 2, (i // 4) % 2, i % 5, (16 if i % 3 == 0 else 0)
    A, sA, B, sB = operands(gpu, M, N, K, fa, fb, pad, seed=M + N)
    bias = [None, W.normal((N,), seed=3, device=gpu), W.normal((N,), seed=3, device=gpu).bfloat16()][i % 3]
    vec = (N + 7) // 8 * 8
    for dt, ld in ((torch.float32, N + 3), (torch.float32, vec), (torch.bfloat16, N + 1), (torch.bfloat16, vec)):
        res = torch.randn(M, ld + 8, device=gpu, generator=torch.Generator(gpu).manual_seed(2)).to(dt) if (i + ld) % 2 else None
        if res is not None and ld != vec:
            res = res[:, 1:]  # elements alone are aligned
        C = torch.full((M, ld), 7.0, dtype=dt, device=gpu)
        pre = torch.full((M, ld), 7.0, dtype=torch.bfloat16, device=gpu)
        call(fq, A, fa, sA, B, fb, sB, bias, act, C, M, N, K, fast, res, pre)
        torch.cuda.synchronize()
        assert (C[:, N:] == 7).all() and (pre[:, N:] == 7).all()
        v, D = product(A, fa, sA, B, fb, sB, K)
        if bias is not None:
            v = v + bias.double()
        tv = (2.0 ** -10 if fast else 1e-5) * D + 2 * U * v.abs()
        want, _, ta, _ = act64(act, v)
        tol = LIPSCHITZ * tv + 1.01 * ta
        if res is not None:
            want = want + res[:, :N].double()
        tol = tol + U * want.abs()
        if dt == torch.bfloat16:
            tol = tol * 1.01 + BF * want.abs()
        assert ((C[:, :N].double() - want).abs() <= tol).all()
        assert ((pre[:, :N].double() - v).abs() <= 1.01 * tv + BF * v.abs()).all()
        if res is not None:  # the residual stream updated in place
            call(fq, A, fa, sA, B, fb, sB, bias, act, res, M, N, K, fast, res)
            assert torch.equal(res[:, :N], C[:, :N])


@pytest.mark.parametrize("M,N,K", [(1, 128, 256), (3, 384, 128), (16, 256, 1024), (40, 128, 640), (64, 256, 256),
                                   (66, 128, 384), (130, 384, 256), (257, 256, 2048), (300, 640, 512)])
@pytest.mark.parametrize("fc", [E4, E5])
@pytest.mark.parametrize("fast", [False, True])
def test_linear_q_equals_quantized_output(fq, gpu, M, N, K, fc, fast):
    A, sA, B, sB = operands(gpu, M, N, K, seed=M)
    act = (M + N // 128 + fc) % 5
    bias = W.normal((N,), seed=3, device=gpu) if M % 2 else None
    h = torch.empty(M, N, device=gpu)
    pre, pre2 = (torch.empty(M, N, dtype=torch.bfloat16, device=gpu) for _ in range(2))
    call(fq, A, E4, sA, B, E4, sB, bias, act, h, M, N, K, fast, None, pre)
    want, ws = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
    fq.fp8q_quantize_1x128(h, M, N, N, fc, EPS, want, N, ws, N // 128)
    q = torch.full((M, N + 16), 0xAA, dtype=torch.uint8, device=gpu)
    s = torch.full((M, N // 128 + 1), -7.0, device=gpu)
    call(fq, A, E4, sA, B, E4, sB, bias, act, q, M, N, K, fast, None, pre2, q=(fc, s))
    torch.cuda.synchronize()
    assert torch.equal(q[:, :N], want) and torch.equal(s[:, :-1], ws) and torch.equal(pre, pre2)
    assert (q[:, N:] == 0xAA).all() and (s[:, -1] == -7).all()


def test_linear_formats(fq, gpu):
    """Every pair of operand formats, in each kernel."""
    for fa in (E4, E5):
        for fb in (E4, E5):
            for M in (3, 100, 300):
                N, K = 384, 1024
                A, sA, B, sB = operands(gpu, M, N, K, fa, fb, seed=M)
                v, D = product(A, fa, sA, B, fb, sB, K)
                for fast in (False, True):
                    C = torch.empty(M, N, device=gpu)
                    call(fq, A, fa, sA, B, fb, sB, None, NONE, C, M, N, K, fast)
                    assert ((C.double() - v).abs() <= (2.0 ** -10 if fast else 1e-5) * D).all()


def test_linear_without_anything_is_the_product(fq, gpu):
    """Without bias, activation and residual, a few rows and the FP8-MFMA tiles give the products' own bits."""
    for M, N, K in ((5, 300, 512), (2048, 2048, 256)):
        A, sA, B, sB = operands(gpu, M, N, K, seed=M)
        C, D = torch.empty(M, N, device=gpu), torch.empty(M, N, device=gpu)
        f = fq.fp8q_gemm_blockscaled_few if M <= 64 else fq.fp8q_gemm_blockscaled_fast
        f(A, E4, K, sA, K // 128, 1, B, E4, K, sB, fq.GRAN_128x128, K // 128, 1, D, N, M, N, K)
        call(fq, A, E4, sA, B, E4, sB, None, NONE, C, M, N, K, True)
        assert torch.equal(C, D)


@pytest.mark.parametrize("M", [1, 70])
@pytest.mark.parametrize("act", range(5))
def test_activations(fq, gpu, M, act):
    """Zero codes leave the bias alone as the pre-activation: the activation over its whole range, in fp32."""
    N, K = 65536, 128
    x = torch.cat([torch.linspace(-14, 14, 32768), torch.logspace(-30, 30, 16384), -torch.logspace(-30, 30, 16384)]).to(gpu)
    A, B = (torch.zeros(n, K, dtype=torch.uint8, device=gpu) for n in (M, N))
    sA, sB = torch.ones(M, 1, device=gpu), torch.ones(N // 128, 1, device=gpu)
    C = torch.empty(M, N, device=gpu)
    call(fq, A, E4, sA, B, E4, sB, x, act, C, M, N, K)
    want, _, tol, _ = act64(act, x)
    want = torch.where(x.abs() > 1e4, x.double().clamp(min=0) if act != NONE else x.double(), want)  # where cubes overflow
    tol = torch.where(x.abs() > 1e4, torch.zeros_like(tol) + 1e-30, tol)
    assert ((C.double() - want).abs() <= tol).all()
    assert torch.equal(C, C[:1].expand(M, N))
    special = torch.tensor([float("nan"), float("inf"), -0.0, 0.0] * 32, device=gpu)
    C = torch.empty(M, 128, device=gpu)
    call(fq, A, E4, sA, B[:128], E4, sB[:1], special, act, C, M, 128, K)
    assert C[:, 0::4].isnan().all() and (C[:, 1::4] == float("inf")).all() and (C[:, 2::4] == 0).all() and (C[:, 3::4] == 0).all()


@pytest.mark.parametrize("M,N,K", [(2305, 8000, 256), (1025, 12100, 384), (1281, 36800, 128), (2305, 8000, 2048), (200, 1000, 18432),
                                   (500, 520, 7168), (1000, 4096, 4096)])
def test_linear_many_tiles(fq, gpu, M, N, K):
    """Up to several tiles per compute unit, of either height, long reductions of few tiles, a ragged edge both ways."""
    A, sA, B, sB = operands(gpu, M, N, K, seed=4)
    bias = W.normal((N,), seed=3, device=gpu)
    res = W.normal((M, N), seed=5, device=gpu)
    rows = torch.tensor([r for r in (0, 1, 127, 128, 199, 255, 256, 499, 512, 999, 1000, 1024, 1279, 1280, 2047, 2048, 2303, 2304)
                         if r < M], device=gpu)
    v, D = product(A[rows], E4, sA[rows], B, E4, sB, K)
    v = v + bias.double()
    for fast in (False, True):
        C = torch.full((M, N), float("nan"), device=gpu)
        pre = torch.full((M, N), float("nan"), dtype=torch.bfloat16, device=gpu)
        call(fq, A, E4, sA, B, E4, sB, bias, SILU, C, M, N, K, fast, res, pre)
        tv = (2.0 ** -10 if fast else 1e-5) * D + 2 * U * v.abs()
        want, _, ta, _ = act64(SILU, v)
        want = want + res[rows].double()
        assert ((C[rows].double() - want).abs() <= LIPSCHITZ * tv + 1.01 * ta + U * want.abs()).all()
        assert ((pre[rows].double() - v).abs() <= 1.01 * tv + BF * v.abs()).all()
        assert C.isfinite().all() and pre.isfinite().all()
        # every row: the codes' form is the same kernel's other end
        if N % 128 == 0:
            call(fq, A, E4, sA, B, E4, sB, bias, SILU, C, M, N, K, fast)
            q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            wq, ws = torch.empty_like(q), torch.empty_like(s)
            fq.fp8q_quantize_1x128(C, M, N, N, E4, EPS, wq, N, ws, N // 128)
            call(fq, A, E4, sA, B, E4, sB, bias, SILU, q, M, N, K, fast, q=(E4, s))
            assert torch.equal(q, wq) and torch.equal(s, ws)


# Every way a call goes on 256 compute units (exact | FP8-MFMA): whole tiles of either height, one round and several, and
# tiles in parts of K, alone and behind whole rounds; a few rows elsewhere.
WAYS = [
    (65, 256, 7168),     # low tiles in parts | low tiles in parts
    (200, 18432, 4096),  # low tiles in parts behind a round | whole low tiles
    (65, 9088, 512),     # whole low tiles | whole low tiles
    (385, 18432, 512),   # two rounds of low tiles | whole tall tiles
    (65, 18432, 7168),   # tall tiles in parts | low tiles in parts
    (1000, 8960, 2048),  # tall tiles in parts behind a round | whole low tiles
    (200, 18432, 512),   # whole tall tiles | whole low tiles
    (3000, 4096, 512),   # two rounds of tall tiles | low tiles
    (385, 18432, 7168),  # tall | low tiles in parts behind a round
    (1000, 18432, 512),  # rounds of low or tall tiles, both
    (1000, 18432, 4096), # tall | tall tiles in parts behind a round
    (2049, 12928, 512),  # rounds | two rounds of tall tiles
]


@pytest.mark.parametrize("M,N,K", WAYS)
@pytest.mark.parametrize("fast", [False, True])
def test_linear_every_way(fq, gpu, M, N, K, fast):
    """Formats, activations, biases, residuals and ragged columns in each; outputs against sampled rows, the other forms
    against the fp32 one."""
    i = WAYS.index((M, N, K))
    fa, fb = (i // 2) % 2, i % 2
    A, sA, B, sB = operands(gpu, M, N, K, fa, fb, 16 if i % 4 == 0 else 0, seed=i)
    rows = torch.tensor(sorted({r for e in range(0, M, 64) for r in (e, e + 15, e + 63) if r < M} | {M - 1})[:40]
                        + [M - 2, M - 1], device=gpu)
    v, D = product(A[rows], fa, sA[rows], B, fb, sB, K)
    for n, act in ((N, i % 5), (N - 3, (i + 1) % 5)):
        bias = W.normal((n,), seed=3, device=gpu) if i % 3 else None
        w = v[:, :n] + (bias.double() if bias is not None else 0)
        res = W.normal((M, n), seed=5, device=gpu) if (i + n) % 2 else None
        pre = torch.full((M, n + 1), 7.0, dtype=torch.bfloat16, device=gpu)
        C = torch.full((M, n + 4), 7.0, device=gpu)
        call(fq, A, fa, sA, B, fb, sB, bias, act, C, M, n, K, fast, res, pre)
        tv = (2.0 ** -10 if fast else 1e-5) * D[:, :n] + 2 * U * w.abs()
        want, _, ta, _ = act64(act, w)
        if res is not None:
            want = want + res[rows].double()
        assert ((C[rows, :n].double() - want).abs() <= LIPSCHITZ * tv + 1.01 * ta + U * want.abs()).all()
        assert ((pre[rows, :n].double() - w).abs() <= 1.01 * tv + BF * w.abs()).all()
        assert C[:, :n].isfinite().all() and (C[:, n:] == 7).all() and (pre[:, n:] == 7).all()
        # bf16: the same sums rounded once; the workspace of exactly the size asked for
        Cb = torch.empty(M, n, dtype=torch.bfloat16, device=gpu)
        nb = fq.fp8q_linear_blockscaled_workspace(int(fast), 0, M, n, K)
        ws = torch.full((nb // 4 + 64,), 5.0, device=gpu)
        call(fq, A, fa, sA, B, fb, sB, bias, act, Cb, M, n, K, fast, None if res is None else torch.zeros_like(Cb), ws=ws,
             ws_bytes=nb)
        C0 = torch.empty(M, n, device=gpu)
        call(fq, A, fa, sA, B, fb, sB, bias, act, C0, M, n, K, fast)
        assert (ws[nb // 4:] == 5).all() and torch.equal(Cb, C0.bfloat16())
    # codes: what the quantizer makes of the fp32 output
    bias = W.normal((N,), seed=3, device=gpu)
    C = torch.empty(M, N, device=gpu)
    call(fq, A, fa, sA, B, fb, sB, bias, i % 5, C, M, N, K, fast)
    for fc in (E4, E5):
        q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
        wq, wsc = torch.empty_like(q), torch.empty_like(s)
        fq.fp8q_quantize_1x128(C, M, N, N, fc, EPS, wq, N, wsc, N // 128)
        call(fq, A, fa, sA, B, fb, sB, bias, i % 5, q, M, N, K, fast, q=(fc, s))
        assert torch.equal(q, wq) and torch.equal(s, wsc)
    # a NaN code spoils its row alone, blocks of zeros and NaN scales among it
    A[M // 2, K - 1] = 0x7F
    q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
    wq, wsc = torch.empty_like(q), torch.empty_like(s)
    C1 = torch.empty_like(C)
    call(fq, A, fa, sA, B, fb, sB, bias, i % 5, C1, M, N, K, fast)
    keep = torch.arange(M, device=gpu) != M // 2
    assert C1[M // 2].isnan().all() and torch.equal(C1[keep], C[keep])
    fq.fp8q_quantize_1x128(C1, M, N, N, E4, EPS, wq, N, wsc, N // 128)
    call(fq, A, fa, sA, B, fb, sB, bias, i % 5, q, M, N, K, fast, q=(E4, s))
    assert torch.equal(q, wq) and torch.equal(s[keep], wsc[keep]) and s[M // 2].isnan().all()


def test_linear_extreme_scales_in_tiles(fq, gpu):
    """Blocks whose scale leaves the quick quotient's range: all zeros, products near fp32's ends."""
    M, N, K = 200, 18432, 512
    A, sA, B, sB = operands(gpu, M, N, K, seed=3)
    sA[1], sA[2], sA[3] = 0.0, 1e-30, 1e30
    bias = torch.zeros(N, device=gpu)
    C = torch.empty(M, N, device=gpu)
    for fast in (False, True):
        call(fq, A, E4, sA, B, E4, sB, bias, NONE, C, M, N, K, fast)
        for fc in (E4, E5):
            q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            wq, wsc = torch.empty_like(q), torch.empty_like(s)
            fq.fp8q_quantize_1x128(C, M, N, N, fc, EPS, wq, N, wsc, N // 128)
            call(fq, A, E4, sA, B, E4, sB, bias, NONE, q, M, N, K, fast, q=(fc, s))
            assert torch.equal(q, wq) and torch.equal(s, wsc)


def test_linear_far_rows_in_tiles(fq, gpu):
    """Rows of the output, the residual and the pre-activations 2^27 bytes apart, past 2^32 in all, in the tiled kernel and
    the join."""
    for M, N, K in ((65, 9088, 512), (65, 256, 7168)):
        ld = 1 << 26
        buf, far = (torch.empty(M * ld, dtype=torch.bfloat16, device=gpu).view(M, ld)[:, :N] for _ in range(2))
        A, sA, B, sB = operands(gpu, M, N, K, seed=6)
        res = W.normal((M, N), seed=5, device=gpu, dtype=torch.bfloat16)
        buf.copy_(res)
        C, pre = torch.empty_like(res), torch.empty_like(res)
        call(fq, A, E4, sA, B, E4, sB, None, GELU, C, M, N, K, True, res, pre)
        call(fq, A, E4, sA, B, E4, sB, None, GELU, buf, M, N, K, True, buf, far)
        assert torch.equal(buf, C) and torch.equal(far, pre)
        del buf, far


def test_linear_rows_do_not_touch_each_other(fq, gpu):
    """A NaN code spoils its own row alone, in every kernel."""
    for M, K in ((20, 256), (150, 256), (150, 4096), (400, 1024)):
        N = 256
        A, sA, B, sB = operands(gpu, M, N, K, seed=1)
        for fast in (False, True):
            h0, h1 = torch.empty(M, N, device=gpu), torch.empty(M, N, device=gpu)
            call(fq, A, E4, sA, B, E4, sB, None, RELU, h0, M, N, K, fast)
            A2 = A.clone()
            A2[3, 200] = 0x7F
            call(fq, A2, E4, sA, B, E4, sB, None, RELU, h1, M, N, K, fast)
            keep = torch.arange(M, device=gpu) != 3
            assert h1[3].isnan().all() and torch.equal(h0[keep], h1[keep])
            q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            call(fq, A2, E4, sA, B, E4, sB, None, RELU, q, M, N, K, fast, q=(E4, s))
            assert (q[3] == 0x7F).all() and s[3].isnan().all() and s[keep].isfinite().all()


def test_linear_scale_strides_and_workspace(fq, gpu):
    """Transposed scale layouts; the caller's own workspace, of exactly the size asked for."""
    for M, K in ((5, 384), (200, 384), (200, 4096)):
        N = 256
        A, sA, B, sB = operands(gpu, M, N, K, seed=9)
        for fast in (0, 1):
            want = torch.empty(M, N, device=gpu)
            call(fq, A, E4, sA, B, E4, sB, None, ERF, want, M, N, K, bool(fast))
            C = torch.empty(M, N, device=gpu)
            n = fq.fp8q_linear_blockscaled_workspace(fast, 0, M, N, K)
            ws = torch.full((n // 4 + 64,), 5.0, device=gpu)
            f = fq.fp8q_linear_blockscaled_fast if fast else fq.fp8q_linear_blockscaled
            f(A, E4, K, sA.t().contiguous(), 1, M, B, E4, K, sB.t().contiguous(), 1, 2, None, ERF, None, 0, C, N, None, 0, M, N, K,
              ws, n)
            assert torch.equal(C, want) and (ws[n // 4:] == 5).all()
            n = fq.fp8q_linear_blockscaled_workspace(fast, 1, M, N, K)
            ws = torch.full((n // 4 + 64,), 5.0, device=gpu)
            q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            call(fq, A, E4, sA, B, E4, sB, None, ERF, q, M, N, K, bool(fast), q=(E4, s), ws=ws, ws_bytes=n)
            wq, wsc = torch.empty_like(q), torch.empty_like(s)
            fq.fp8q_quantize_1x128(want, M, N, N, E4, EPS, wq, N, wsc, 2)
            assert torch.equal(q, wq) and torch.equal(s, wsc) and (ws[n // 4:] == 5).all()


# ------------------------------------------------------------------ gradient of the linear layer
def bwd_call(fq, dC, pre, act, fc, fh, M, N, want_t=True, want_h=True, want_b=True, pad=0, stream=None):
    dev, Mp = dC.device, -(-M // 128) * 128
    u8 = lambda r, c: torch.full((r, c + pad), 0xAA, dtype=torch.uint8, device=dev)  # noqa: E731
    f4 = lambda r, c: torch.full((r, c + (1 if pad else 0)), -7.0, device=dev)  # noqa: E731
    D, Ds = u8(M, N), f4(M, N // 128)
    Dt, Dts = (u8(N, Mp), f4(N, Mp // 128)) if want_t else (None, None)
    Ht, Hts = (u8(N, Mp), f4(N, Mp // 128)) if want_h else (None, None)
    db = torch.full((N + 4,), 3.0, device=dev) if want_b else None
    n = fq.fp8q_linear_bwd_q_workspace(M, N)
    ws = torch.full((n // 4 + 64,), 5.0, device=dev)
    st = lambda t: 0 if t is None else t.stride(0)  # noqa: E731
    fq.fp8q_linear_bwd_q(dC, dC.stride(0), pre, st(pre), act, fc, EPS, D, st(D), Ds, st(Ds), Dt, st(Dt), Dts, st(Dts), fh, Ht,
                         st(Ht), Hts, st(Hts), db, M, N, ws, n, stream=stream)
    torch.cuda.synchronize()
    assert (ws[n // 4:] == 5).all() and (db is None or (db[N:] == 3).all())
    if pad:
        for t, c in ((D, N), (Dt, Mp), (Ht, Mp)):
            assert t is None or (t[:, c:] == 0xAA).all()
        for t, c in ((Ds, N // 128), (Dts, Mp // 128), (Hts, Mp // 128)):
            assert t is None or (t[:, c:] == -7).all()
    cut = lambda t, c: None if t is None else t[:, :c]  # noqa: E731
    return (cut(D, N), cut(Ds, N // 128), cut(Dt, Mp), cut(Dts, Mp // 128), cut(Ht, Mp), cut(Hts, Mp // 128),
            None if db is None else db[:N])


def check_codes(q, s, x, tol, fmt):
    """Codes and scales against 64-bit values x that the kernel holds within tol."""
    b, t = x.reshape(x.shape[0], -1, 128), tol.reshape(x.shape[0], -1, 128)
    want = b.abs().amax(2).clamp(min=EPS) / MAXF[fmt]
    assert ((s.double() - want).abs() <= t.amax(2) / MAXF[fmt] + 2 * U * want).all()
    got = q.contiguous().view(F8[fmt]).double().view(b.shape) * s.double()[:, :, None]
    assert ((got - b).abs() <= HALF[fmt] * (b.abs() + t) + TINY[fmt] * s.double()[:, :, None] + t + 4 * U * b.abs()).all()


@pytest.mark.parametrize("M,N", [(1, 128), (5, 256), (127, 128), (128, 384), (129, 640), (300, 1152), (1000, 256), (2100, 128)])
@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float32])
def test_linear_bwd(fq, gpu, M, N, dt):
    act, fc, fh, pad = (M + N // 128) % 5, M % 2, (M // 2) % 2, (16 if M in (5, 129) else 0)
    for act in (act, (act + 2) % 5):
        dC = W.gradient(M, N, seed=1, device=gpu, dtype=dt)
        pre = W.normal((M, N), seed=2, device=gpu, std=1.7, dtype=torch.bfloat16)
        D, Ds, Dt, Dts, Ht, Hts, db = bwd_call(fq, strided(dC, pad) if pad else dC, strided(pre, pad) if pad else pre, act, fc, fh,
                                               M, N, pad=pad)
        h, da, th, tda = act64(act, pre)
        d = dC.double() * da
        td = dC.double().abs() * tda + U * d.abs()
        padT = lambda t: torch.cat([t, t.new_zeros(-M % 128, N)]).t().contiguous()  # noqa: E731
        check_codes(D, Ds, d, td, fc)
        check_codes(Dt, Dts, padT(d), padT(td), fc)
        check_codes(Ht, Hts, padT(h), padT(th + U * h.abs()), fh)
        if M % 128:  # the padding holds zero codes
            assert (Dt[:, M:] == 0).all() and (Ht[:, M:] == 0).all()
        # 4 tokens of a thread, 4 row groups, 8 wavefronts, then the blocks a sixteenth at a time
        n = 2 + 2 + 8 + (0 if M <= 128 else -(-(-(-M // 128)) // 16) + 16)
        assert ((db.double() - d.sum(0)).abs() <= n * U * d.abs().sum(0) + td.sum(0)).all()
        # each output alone, the same bits
        for t, hh, b in ((True, False, True), (False, True, False), (False, False, True), (False, False, False)):
            o = bwd_call(fq, dC, pre, act, fc, fh, M, N, t, hh, b)
            for x, y in zip(o, (D, Ds, Dt, Dts, Ht, Hts, db)):
                assert x is None or torch.equal(x, y)


def test_linear_bwd_without_activation_is_the_quantizer(fq, gpu):
    """No activation: the codes are the quantizers' of dC, bit for bit, and no pre-activations are needed."""
    M, N = 256, 384
    for dt in (torch.bfloat16, torch.float32):
        for fc in (E4, E5):
            dC = W.gradient(M, N, seed=1, device=gpu, dtype=dt)
            D, Ds, Dt, Dts, _, _, db = bwd_call(fq, dC, None, NONE, fc, E4, M, N, want_h=False)
            q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            fq.fp8q_quantize_1x128(dC, M, N, N, fc, EPS, q, N, s, N // 128)
            qt, st = torch.empty(N, M, dtype=torch.uint8, device=gpu), torch.empty(N, M // 128, device=gpu)
            fq.fp8q_quantize_1x128_t(dC, M, N, N, fc, EPS, qt, M, st, M // 128)
            assert torch.equal(D, q) and torch.equal(Ds, s) and torch.equal(Dt, qt) and torch.equal(Dts, st)
            x = torch.randn(M, N, device=gpu).bfloat16()
            o = bwd_call(fq, dC, x, NONE, fc, E4, M, N)
            fq.fp8q_quantize_1x128_t(x, M, N, N, E4, EPS, qt, M, st, M // 128)
            assert torch.equal(o[0], q) and torch.equal(o[4], qt) and torch.equal(o[5], st)


@pytest.mark.parametrize("act", range(5))
def test_linear_bwd_every_pre_activation(fq, gpu, act):
    """One token: the bias's gradient is dC * act' in fp32, for every finite bf16 pre-activation; against the formula, and
    against differences of the activation."""
    N = 65536
    pre = torch.arange(N, dtype=torch.int32, device=gpu).to(torch.int16).view(torch.bfloat16)[None]
    dC = torch.full((1, N), 1.5, device=gpu)
    db = bwd_call(fq, dC, pre, act, E5, E4, 1, N)[6]
    x = pre[0].double()
    fine = x.isfinite() & (x.abs() < 1e4)
    _, da, _, tda = act64(act, x)
    assert ((db.double() - 1.5 * da).abs() <= 1.5 * tda + 2 * U * da.abs())[fine].all()
    big = x.isfinite() & (x.abs() >= 1e4)
    assert (db[big] == (1.5 if act == NONE else 1.5 * (x[big] > 0).float())).all()
    if act == RELU:
        assert (db[x == 0] == 0).all() and (db[x.isnan()] == 1.5).all()
    elif act != NONE:
        assert db[x.isnan()].isnan().all()
    mid = fine & (x.abs() < 20) & (x.abs() > 1e-3)
    h = 1e-4
    diff = (act64(act, x + h)[0] - act64(act, x - h)[0]) / (2 * h)
    # h^2 / 6 of a third derivative that stays under 4, and 2^-53 / h of the values
    assert ((db.double() - 1.5 * diff).abs() <= 1.5 * (4 * h * h + tda) + 1e-10 + 2 * U)[mid].all()


def test_relu_passes_nothing_of_what_it_masks(fq, gpu):
    """Inf and NaN gradients where ReLU cut the layer off: zeros, and finite scales."""
    M, N = 130, 256
    pre = torch.randn(M, N, device=gpu).bfloat16()
    dC = torch.randn(M, N, device=gpu)
    want = bwd_call(fq, torch.where(pre > 0, dC, torch.zeros_like(dC)), pre, RELU, E4, E4, M, N)
    bad = torch.where(torch.arange(N, device=gpu) % 2 == 0, float("inf"), float("nan"))
    got = bwd_call(fq, torch.where(pre > 0, dC, bad.expand(M, N)).contiguous(), pre, RELU, E4, E4, M, N)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_linear_bwd_codes_of_extreme_blocks(fq, gpu):
    """Blocks of zeros, Inf, NaN and magnitudes whose scale leaves the quick quotient's range, along both dimensions: the
    quantizers' codes, bit for bit; blocks without them too."""
    M, N = 256, 384
    for eps in (1e-12, 1e-37):
        dC = torch.randn(M, N, device=gpu)
        dC[:, 3], dC[:, 4], dC[:, 5], dC[9], dC[10], dC[11] = 1e30, 1e-34, 0.0, 1e-36, 0.0, 1e32
        dC[3, 7], dC[200, 140] = float("nan"), float("inf")
        for fc in (E4, E5):
            D, Ds = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
            Dt, Dts = torch.empty(N, M, dtype=torch.uint8, device=gpu), torch.empty(N, M // 128, device=gpu)
            fq.fp8q_linear_bwd_q(dC, N, None, 0, NONE, fc, eps, D, N, Ds, N // 128, Dt, M, Dts, M // 128, E4, None, 0, None, 0, None,
                                 M, N)
            q, s, qt, st = torch.empty_like(D), torch.empty_like(Ds), torch.empty_like(Dt), torch.empty_like(Dts)
            fq.fp8q_quantize_1x128(dC, M, N, N, fc, eps, q, N, s, N // 128)
            fq.fp8q_quantize_1x128_t(dC, M, N, N, fc, eps, qt, M, st, M // 128)
            for a, b in ((D, q), (Dt, qt), (Ds.nan_to_num(7.0), s.nan_to_num(7.0)), (Dts.nan_to_num(7.0), st.nan_to_num(7.0))):
                assert torch.equal(a, b)


def test_linear_bwd_special_gradients(fq, gpu):
    """A NaN gradient marks its blocks and its column's sum alone; an Inf its block's scale."""
    M, N = 256, 256
    dC = torch.randn(M, N, device=gpu)
    dC[3, 5], dC[200, 140] = float("nan"), float("inf")
    D, Ds, Dt, Dts, _, _, db = bwd_call(fq, dC, None, NONE, E4, E4, M, N, want_h=False)
    nan = torch.zeros(M, 2, dtype=torch.bool, device=gpu)
    nan[3, 0] = True
    assert torch.equal(Ds.isnan(), nan) and (D[3, :128] == 0x7F).all() and Ds[200, 1].isinf()
    assert Dts[5, 0].isnan() and Dts.isnan().sum() == 1 and (Dt[5, :128] == 0x7F).all() and Dts[140, 1].isinf()
    assert db[5].isnan() and db[140].isinf() and db.isfinite().sum() == N - 2


# ------------------------------------------------------------------ streams, graphs, far rows, the operators together
def test_explicit_streams(fq, gpu):
    """Two streams at once, each with its own workspace from torch's allocator, against one after the other."""
    M, N, K = 65, 256, 7168
    ops = [operands(gpu, M, N, K, seed=s) for s in (1, 2)]
    bias = W.normal((N,), seed=3, device=gpu)

    def run(o, stream):
        A, sA, B, sB = o
        outs = []
        for m in (5, M):  # a few rows; tiles in parts of K
            q, s = torch.empty(m, N, dtype=torch.uint8, device=gpu), torch.empty(m, N // 128, device=gpu)
            call(fq, A, E4, sA, B, E4, sB, bias, GELU, q, m, N, K, q=(E4, s), stream=stream)
            outs += [q, s]
        return outs

    want = [run(o, None) for o in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in ops]
    for _ in range(3):
        got = [run(o, s if i else s.cuda_stream) for i, (o, s) in enumerate(zip(ops, streams))]
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for g, w in zip(got, want) for a, b in zip(g, w))


def test_calls_from_several_threads(fq, gpu):
    """Calls release the interpreter's lock: four threads, each on a stream of its own, with refused calls in between,
    against one after the other; a refusal's text is its thread's."""
    from concurrent.futures import ThreadPoolExecutor

    M, N, K = 65, 256, 2048
    ops = [operands(gpu, M, N, K, seed=s) for s in range(4)]
    bias = W.normal((N,), seed=3, device=gpu)

    def run(i, stream):
        A, sA, B, sB = ops[i]
        q, s = torch.empty(M, N, dtype=torch.uint8, device=gpu), torch.empty(M, N // 128, device=gpu)
        call(fq, A, E4, sA, B, E4, sB, bias, GELU, q, M, N, K, q=(E4, s), stream=stream)
        return q, s

    want = [run(i, None) for i in range(4)]
    torch.cuda.synchronize()

    def work(i):
        stream = torch.cuda.Stream()
        got = []
        for k in range(20):
            got.append(run(i, stream))
            cols = 8 * (1000 + i) + 1
            with pytest.raises(fq.Fp8qError, match=str(cols)):
                fq.fp8q_layernorm_1x128(bias, N, None, 0, None, None, 1, cols, 1e-5, None, 0, bias, cols, 0, 1e-12, None, 0, None,
                                        0, stream=stream)
        stream.synchronize()
        return got

    with ThreadPoolExecutor(4) as ex:
        for got, w in zip(ex.map(work, range(4)), want):
            assert all(torch.equal(a, b) for g in got for a, b in zip(g, w))


def example():
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "mlp.py")
    spec = importlib.util.spec_from_file_location("mlp_example", path)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("tokens,K,F", [(150, 512, 1024), (1, 128, 256), (300, 1024, 2048)])
def test_mlp_against_64_bits(gpu, tokens, K, F):
    """The operators as a layer uses them: outputs and every gradient against the same layer in 64 bits.  Each operand's
    codes are off by up to 2^-4 (E4M3) or 2^-3 (E5M2) of a value, as independent errors of a third to a half of that root
    mean square; a product of two such operands, chained twice, stays within 15%."""
    res = example().main(tokens, K, F)
    assert len(res) == 9 and max(res.values()) <= 0.15, res


@pytest.mark.parametrize("M", [3, 150, 1100])
def test_mlp_captured_in_a_graph(gpu, M):
    """A step captured once and replayed on changing inputs, eager work in between, equals the eager step bit for bit."""
    ex = example()
    params, (x, r, dy) = ex.inputs(M, 512, 1024, gpu)
    layer = ex.Mlp(*params)

    def step():
        y, saved = layer.forward(x, r)
        return [y, *layer.backward(saved, dy), layer.token(x[:3], r[:3])]

    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for i in range(4):
        x.copy_(torch.randn(x.shape, generator=torch.Generator(gpu).manual_seed(i), device=gpu))
        dy.mul_(0.5)
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        want = step()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_far_rows(fq, gpu):
    """Rows more than 2^32 bytes apart in every strided tensor of the norm and the gradient."""
    cols, ld = 256, (1 << 31) + 64
    buf = torch.empty(ld + cols, dtype=torch.bfloat16, device=gpu)
    rows2 = lambda t: torch.as_strided(t, (2, cols), (ld, 1))  # noqa: E731
    x, out = rows2(buf), rows2(torch.empty_like(buf))
    x.copy_(torch.randn(2, cols, device=gpu))
    near = x.contiguous()
    want = run_norm(fq, near, None, None, None, E4, codes=False)[1]
    fq.fp8q_layernorm_1x128(x, ld, None, 0, None, None, 2, cols, NEPS, None, 0, out, ld, E4, EPS, None, 0, None, 0)
    assert torch.equal(out.contiguous(), want)
    mean, rstd = near.float().mean(1), near.float().var(1, correction=0).add(NEPS).rsqrt()
    dx = torch.empty_like(near)
    fq.fp8q_layernorm_bwd(near, cols, near, cols, None, mean, rstd, None, 0, 2, cols, dx, cols)
    fq.fp8q_layernorm_bwd(x, ld, x, ld, None, mean, rstd, None, 0, 2, cols, out, ld)
    assert torch.equal(out.contiguous(), dx)
    a = bwd_call(fq, near, near, SILU, E4, E4, 2, cols)
    b = bwd_call(fq, x, x, SILU, E4, E4, 2, cols)
    assert all(torch.equal(s, t) for s, t in zip(a, b))
    A, sA, B, sB = operands(gpu, 2, cols, 128)
    C, pre = torch.empty(2, cols, dtype=torch.bfloat16, device=gpu), torch.empty(2, cols, dtype=torch.bfloat16, device=gpu)
    call(fq, A, E4, sA, B, E4, sB, None, SILU, C, 2, cols, 128, False, near, pre)
    call(fq, A, E4, sA, B, E4, sB, None, SILU, out, 2, cols, 128, False, x)
    assert torch.equal(out.contiguous(), C)

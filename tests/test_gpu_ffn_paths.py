"""GPU checks of the feed-forward operators' paths that small shapes do not reach: explicit streams, the tiled kernels'
epilogues, long reductions, many token blocks, very many rows, far rows.  Tolerances as in test_gpu_ffn.py.
"""
import numpy as np
import pytest
import torch

from block_scaled_precision_amax_amd import workloads as W
from test_gpu_ffn import BF, E4, E5, EPS, NEPS, U, act64, bwd_call, glu_call, operands

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ streams
def test_glu_q_on_an_explicit_stream_without_workspace(fq, gpu):
    """The workspace of a few rows comes from the pool of the stream that uses it, however the stream is named."""
    M, F, K = 3, 512, 256
    A, sA, B, sB = operands(gpu, M, F, K, seed=2)
    assert fq.fp8q_glu_blockscaled_q_workspace(M, F) > 0
    want, ws = torch.empty(M, F, dtype=torch.uint8, device=gpu), torch.empty(M, F // 128, device=gpu)
    glu_call(fq, None, A, E4, sA, B, E4, sB, 0, want, None, M, F, K, q=(E4, ws))
    side = torch.cuda.Stream()
    for stream in (side, side.cuda_stream, torch.cuda.default_stream(), 0):
        q, s = torch.zeros_like(want), torch.zeros_like(ws)
        torch.cuda.synchronize()
        before = torch.cuda.current_stream()
        glu_call(fq, None, A, E4, sA, B, E4, sB, 0, q, None, M, F, K, q=(E4, s), stream=stream)
        assert torch.cuda.current_stream() == before
        torch.cuda.synchronize()
        assert torch.equal(q, want) and torch.equal(s, ws)
    with torch.cuda.stream(side):  # the block given back to the side stream's pool is the next one taken there
        p = torch.empty(4 * M * F, dtype=torch.uint8, device=gpu).data_ptr()
    torch.cuda.synchronize()
    glu_call(fq, None, A, E4, sA, B, E4, sB, 0, q, None, M, F, K, q=(E4, s), stream=side)
    with torch.cuda.stream(side):
        assert torch.empty(4 * M * F, dtype=torch.uint8, device=gpu).data_ptr() == p
    torch.cuda.synchronize()


# ------------------------------------------------------------------ very many rows
def test_glu_of_very_many_rows_and_few_columns(fq, gpu):
    """More groups of 64 rows than the 65535 a launch's second dimension holds: the rows repeat every 4096."""
    F, K, n = 16, 128, 4096
    M = 64 * 65535 + 65
    base, sbase, B, sB = operands(gpu, n, F, K, seed=6)
    A, sA = base.repeat(-(-M // n), 1)[:M], sbase.repeat(-(-M // n), 1)[:M]
    a = base.view(torch.float8_e4m3fn).double() * sbase.double()
    w = [b.view(torch.float8_e4m3fn).double() * s.double() for b, s in zip(B, sB)]
    (g, Dg), (u, Du) = [(a @ x.t(), a.abs() @ x.abs().t()) for x in w]
    want = g * torch.sigmoid(g) * u
    for fn, rel in (("fp8q_glu_blockscaled", 1e-5), ("fp8q_glu_blockscaled_fast", 2.0 ** -10)):
        h = torch.full((M, F), float("nan"), device=gpu)
        glu_call(fq, fn, A, E4, sA, B, E4, sB, 0, h, None, M, F, K)
        # as test_glu: |silu'| <= 1.13
        tol = 1.13 * rel * Dg * (u.abs() + rel * Du) + (g * torch.sigmoid(g)).abs() * rel * Du + want.abs() * 600 * 2.0 ** -24
        assert ((h[:n].double() - want).abs() <= tol + 1e-30).all()
        full = M // n * n
        assert (h[:full].view(-1, n, F) == h[:n]).all() and torch.equal(h[full:], h[:M - full])


def test_norm_of_very_many_rows(fq, gpu):
    """More rows than one launch has threads for (four rows and 256 threads a workgroup, 2^32 threads): the rows repeat
    every 4096, and so do their outputs."""
    cols, n = 128, 4096
    rows = (1 << 26) + 5
    base = W.activation(n, cols, seed=3, factor=5.0, device=gpu, dtype=torch.bfloat16)
    x = base.repeat(-(-rows // n), 1)[:rows]
    w = 1 + W.normal((cols,), seed=6, device=gpu, std=0.1, dtype=torch.float32)

    def run(x):
        r = x.shape[0]
        z, y = torch.zeros_like(x), torch.zeros_like(x)
        q, s, rstd = torch.zeros(r, cols, dtype=torch.uint8, device=gpu), torch.zeros(r, 1, device=gpu), torch.zeros(r, device=gpu)
        fq.fp8q_rmsnorm_1x128(x, cols, x, cols, w, r, cols, NEPS, z, cols, y, cols, E4, EPS, q, cols, s, 1, rstd)
        return z, y, q, s, rstd

    full = rows // n * n
    for got, want in zip(run(x), run(base)):
        assert (got[:full].view(-1, *want.shape) == want).all() and torch.equal(got[full:], want[:rows - full])


# ------------------------------------------------------------------ gated projection on tiles
# Low tiles throughout, whole rounds of tall ones, and tall ones with the halves of the rest, ragged both ways.
TILED = [(200, 4000, 512), (129, 4224, 384), (1025, 6144, 128), (2000, 4500, 1280), (300, 4097, 256), (513, 8191, 640)]


def on_tiles(fq, M, F):
    """The few-row kernel's output goes through a workspace, the tiles' does not."""
    return fq.fp8q_glu_blockscaled_q_workspace(M, -(-F // 128) * 128) == 0


@pytest.mark.parametrize("M,F,K", TILED)
@pytest.mark.parametrize("fa", [E4, E5])
@pytest.mark.parametrize("fb", [E4, E5])
def test_glu_on_tiles(fq, orc, gpu, M, F, K, fa, fb):
    assert on_tiles(fq, M, F)
    i = TILED.index((M, F, K))
    act, pad, Kb, Fb = (i + fa) % 2, 16 * ((i + fb) % 2), K // 128, -(-F // 128)
    A, sA, B, sB = operands(gpu, M, F, K, fa, fb, pad, seed=M + F)
    if i % 2:  # scales [K/128, rows]
        sc = (sA.t().contiguous(), 1, M), (sB[0].t().contiguous(), sB[1].t().contiguous(), 1, Fb)
    else:
        sc = (sA, Kb, 1), (sB[0], sB[1], Kb, 1)
    if pad:  # one matrix, passed as its halves
        both = torch.cat(B)
        W0, W1 = both, both[F:]
    else:
        W0, W1 = B
    rows = np.array([r for r in (0, 1, 15, 63, 64, 127, 128, 191, 199, 255, 256, 299, 512, 1023, 1024, 1791, 1792, 1999) if r < M])
    An, Bn = A[:, :K].cpu().numpy(), [b[:, :K].cpu().numpy() for b in B]
    (g, Dg), (u, Du) = [orc.gemm_blockscaled(An, fa, sA.cpu().numpy(), Bn[j], fb, sB[j].cpu().numpy(), orc.GRAN_128x128, rows=rows)
                        for j in (0, 1)]
    g, u, Dg, Du = map(torch.from_numpy, (g, u, Dg, Du))
    a64 = act64(act, g)
    outs = []
    for fn, rel in (("fp8q_glu_blockscaled", 1e-5), ("fp8q_glu_blockscaled_fast", 2.0 ** -10)):

        def call(dt, ld, ldgu):
            h = torch.full((M, ld), 7.0, dtype=dt, device=gpu)
            gu = torch.full((M, ldgu), 7.0, dtype=torch.bfloat16, device=gpu) if ldgu else None
            getattr(fq, fn)(A, fa, A.stride(0), *sc[0], W0, W1, fb, W0.stride(0), *sc[1], act, h, ld, gu, ldgu, M, F, K)
            assert (h[:, F:] == 7).all() and (gu is None or (gu[:, 2 * F:] == 7).all())
            return h[:, :F], None if gu is None else gu[:, :2 * F]

        up8 = -(-F // 8) * 8
        h, gu = call(torch.float32, F + 3 - F % 2, 2 * F + 5)  # rows of no alignment
        for dt, ld, ldgu in ((torch.float32, up8, 2 * up8 + 8), (torch.bfloat16, up8, 0), (torch.bfloat16, F + 3 - F % 2, 2 * F)):
            h2, gu2 = call(dt, ld, ldgu)
            assert torch.equal(h2, h.to(dt)) and (gu2 is None or torch.equal(gu2, gu))
        # as test_glu: |act'| <= 1.13, the exponential's argument is off by a few u of at most 176
        tol = 1.13 * rel * Dg * (u.abs() + rel * Du) + a64.abs() * rel * Du + (a64 * u).abs() * 600 * U + 1e-30
        assert ((h[rows].cpu().double() - a64 * u).abs() <= tol).all()
        for k, (x, D) in enumerate(((g, Dg), (u, Du))):
            assert ((gu[rows, k * F:(k + 1) * F].cpu().double() - x).abs() <= BF * x.abs() + 1.01 * rel * D).all()
        assert h.isfinite().all() and gu.isfinite().all()
        outs.append(h)
    assert not torch.equal(*outs)  # the few-row kernel would give both forms the same bits


@pytest.mark.parametrize("M,F,K", [(200, 4096, 256), (129, 4224, 384), (1025, 6144, 128), (2000, 4608, 1280)])
@pytest.mark.parametrize("fc", [E4, E5])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4), (E4, E5), (E5, E5)])
def test_glu_q_on_tiles(fq, gpu, M, F, K, fc, fa, fb):
    """The codes leave the tiles as the quantizer makes them of the fp32 output: zero blocks, blocks whose scale takes the
    IEEE division and infinite ones among them, rows aligned to 16 bytes and to 4."""
    assert on_tiles(fq, M, F)
    A, sA, B, sB = operands(gpu, M, F, K, fa, fb, seed=M + fc)
    A[7] = 0
    sA[9] *= 1e-12
    sA[M - 1] *= 1e15
    sA[40] *= 1e22
    act = (fa + fc) % 2
    h, gu = torch.empty(M, F, device=gpu), torch.empty(M, 2 * F, dtype=torch.bfloat16, device=gpu)
    glu_call(fq, "fp8q_glu_blockscaled", A, fa, sA, B, fb, sB, act, h, gu, M, F, K)
    want, ws = torch.empty(M, F, dtype=torch.uint8, device=gpu), torch.empty(M, F // 128, device=gpu)
    fq.fp8q_quantize_1x128(h, M, F, F, fc, EPS, want, F, ws, F // 128)
    assert (want[7] & 0x7F == 0).all() and (ws[M - 1] > 2.0 ** 80).any() and ws[40].isinf().any()
    for off, save in ((0, True), (4, False)):
        q = torch.full((M, F + 16 + off), 0xAA, dtype=torch.uint8, device=gpu)
        s = torch.full((M, F // 128 + 1), -7.0, device=gpu)
        gu2 = torch.empty_like(gu) if save else None
        glu_call(fq, None, A, fa, sA, B, fb, sB, act, q[:, off:], gu2, M, F, K, q=(fc, s))
        assert torch.equal(q[:, off:off + F], want) and torch.equal(s[:, :-1], ws)
        assert gu2 is None or torch.equal(gu2, gu)
        assert (q[:, :off] == 0xAA).all() and (q[:, off + F:] == 0xAA).all() and (s[:, -1] == -7).all()


@pytest.mark.parametrize("M,F,K", [(200, 4096, 256), (1025, 6144, 128)])
def test_a_nan_on_tiles_stays_in_its_row_and_column(fq, gpu, M, F, K):
    assert on_tiles(fq, M, F)
    A, sA, B, sB = operands(gpu, M, F, K, seed=1)
    A2, B2 = A.clone(), [b.clone() for b in B]
    A2[3, 100] = 0x7F
    B2[1][130, 5] = 0x7F  # up: column 130 alone
    rows, cols = torch.arange(M, device=gpu) != 3, torch.arange(F, device=gpu) != 130
    for fn in ("fp8q_glu_blockscaled", "fp8q_glu_blockscaled_fast"):
        h0, h1 = torch.empty(M, F, device=gpu), torch.empty(M, F, device=gpu)
        glu_call(fq, fn, A, E4, sA, B, E4, sB, 0, h0, None, M, F, K)
        glu_call(fq, fn, A2, E4, sA, B2, E4, sB, 0, h1, None, M, F, K)
        assert h1[3].isnan().all() and h1[:, 130].isnan().all() and torch.equal(h0[rows][:, cols], h1[rows][:, cols])
    q, s = torch.empty(M, F, dtype=torch.uint8, device=gpu), torch.empty(M, F // 128, device=gpu)
    glu_call(fq, None, A2, E4, sA, B2, E4, sB, 0, q, None, M, F, K, q=(E4, s))
    blocks = torch.arange(F // 128, device=gpu) != 1
    assert (q[3] == 0x7F).all() and s[3].isnan().all()
    assert (q[:, 128:256] == 0x7F).all() and s[:, 1].isnan().all() and s[rows][:, blocks].isfinite().all()


# ------------------------------------------------------------------ long reductions, many token blocks, the re-tiled product
@pytest.mark.parametrize("M", [1, 20, 50])
@pytest.mark.parametrize("fa,fb", [(E4, E4), (E5, E4), (E4, E5)])
def test_few_rows_with_a_long_reduction(fq, orc, gpu, M, fa, fb):
    """More K blocks than the few-row kernel keeps A scales for in LDS (160)."""
    N, K, Kb = 40, 20608, 161
    A, sA, B, sB = operands(gpu, M, N, K, fa, fb, pad=16, seed=M)
    sb = (sB[0].repeat_interleave(128, 0)[:N] * torch.linspace(0.5, 2.0, N, device=gpu)[:, None]).contiguous()
    An, Bn = A[:, :K].cpu().numpy(), [b[:, :K].cpu().numpy() for b in B]
    for gb, s in ((2, sB[0]), (1, sb)):
        C = torch.full((M, N), float("nan"), device=gpu)
        fq.fp8q_gemm_blockscaled_few(A, fa, A.stride(0), sA, Kb, 1, B[0], fb, B[0].stride(0), s, gb, Kb, 1, C, N, M, N, K)
        ref, D = orc.gemm_blockscaled(An, fa, sA.cpu().numpy(), Bn[0], fb, s.cpu().numpy(), gb)
        assert (np.abs(C.cpu().numpy().astype(np.float64) - ref) <= 1e-5 * D).all()
    h, gu = torch.full((M, N), float("nan"), device=gpu), torch.empty(M, 2 * N, dtype=torch.bfloat16, device=gpu)
    glu_call(fq, "fp8q_glu_blockscaled", A, fa, sA, B, fb, sB, 1, h, gu, M, N, K)
    (g, Dg), (u, Du) = [orc.gemm_blockscaled(An, fa, sA.cpu().numpy(), Bn[j], fb, sB[j].cpu().numpy(), orc.GRAN_128x128)
                        for j in (0, 1)]
    g, u, Dg, Du = map(torch.from_numpy, (g, u, Dg, Du))
    a64, rel = act64(1, g), 1e-5
    tol = 1.13 * rel * Dg * (u.abs() + rel * Du) + a64.abs() * rel * Du + (a64 * u).abs() * 600 * U + 1e-30
    assert ((h.cpu().double() - a64 * u).abs() <= tol).all()
    for k, (x, D) in enumerate(((g, Dg), (u, Du))):
        assert ((gu[:, k * N:(k + 1) * N].cpu().double() - x).abs() <= BF * x.abs() + 1.01 * rel * D).all()


@pytest.mark.parametrize("M,F", [(2177, 384), (2200, 512), (4100, 128)])
def test_glu_bwd_of_many_token_blocks(fq, orc, gpu, M, F):
    """More than the sixteen token blocks that are walked together, the last group ragged; exact values as in
    test_glu_bwd_exact_values."""
    g = torch.Generator().manual_seed(M)
    dh = torch.randn(M, F, generator=g).bfloat16()
    u = (torch.randn(M, F, generator=g) * 3).bfloat16()
    gu = torch.cat([torch.full((M, F), 40.0, dtype=torch.bfloat16), u], 1)
    D, Ds, Dt, Dts, Ht, Hts = bwd_call(fq, dh.to(gpu), gu.to(gpu), 0, E5, E4, M, F, pad=16)
    d = torch.cat([dh.float() * u.float(), dh.float() * 40], 1)
    padt = lambda t: np.ascontiguousarray(torch.nn.functional.pad(t.t(), (0, Dt.shape[1] - M)).numpy())  # noqa: E731
    for q, s, v, fmt in ((D, Ds, d.numpy(), E5), (Dt, Dts, padt(d), E5), (Ht, Hts, padt(40 * u.float()), E4)):
        wq, ws = orc.quantize_blocks(v, 1, 128, fmt)
        assert np.array_equal(q.cpu().numpy(), wq) and np.array_equal(s.cpu().numpy(), ws)


@pytest.mark.parametrize("M,N,K", [(1, 1, 128), (100, 300, 256), (129, 4096, 384), (1000, 2200, 640)])
@pytest.mark.parametrize("fa,fb", [(E4, E5), (E5, E5), (E5, E4)])
@pytest.mark.parametrize("any_code", [False, True])
def test_fast_product_is_the_same_on_either_tile_in_every_format(fq, gpu, M, N, K, fa, fb, any_code):
    """Rows on 128-row tiles equal, bit for bit, those of a product with so many rows that it runs on 256-row tiles; with
    every code among the operands, NaN and infinities are where they are there."""
    big = 256 * (256 // -(-N // 256))
    A, sA, B, sB = operands(gpu, max(M, big - 99), N, K, fa, fb, seed=N)
    if any_code:
        A, B = A.random_(0, 256), [b.random_(0, 256) for b in B]
        A[M // 2:M // 2 + 1] = A[M // 2:M // 2 + 1] & 0x3F  # a row without either
        B[0][N // 2:N // 2 + 1] = B[0][N // 2:N // 2 + 1] & 0x3F
    C, D = torch.full((M, N), 7.0, device=gpu), torch.full((A.shape[0], N), 7.0, device=gpu)
    for out, rows in ((C, M), (D, A.shape[0])):
        fq.fp8q_gemm_blockscaled_fast(A, fa, K, sA, K // 128, 1, B[0], fb, K, sB[0], 2, K // 128, 1, out, N, rows, N, K)
    assert torch.equal(C.isnan(), D[:M].isnan()) and torch.equal(C.nan_to_num(nan=0.5), D[:M].nan_to_num(nan=0.5))
    assert C[M // 2, N // 2].isfinite() and (any_code or C.isfinite().all())


# ------------------------------------------------------------------ offsets past 31 and 32 bits
def far(t, ld, buf, at=0):
    """t's rows `ld` elements apart in buf, from element `at` on."""
    v = buf.view(t.dtype)[at:].as_strided(t.shape, (ld, 1))
    v.copy_(t)
    return v


def test_products_of_operands_just_under_4_gib(fq, gpu):
    """Rows so far apart that the operands span almost 4 GiB, outputs more: the results are those of adjacent rows."""
    F, K, Kb = 4096, 256, 2
    ldb, ldo = (0xFFFFFFFF - K) // (F - 1) // 16 * 16, 1 << 23
    buf, out = torch.empty(1 << 32, dtype=torch.uint8, device=gpu), torch.empty(200 * ldo, dtype=torch.float32, device=gpu)
    for M in (3, 200):
        A, sA, B, sB = operands(gpu, M, F, K, seed=M)
        lda = (0xFFFFFFFF - K) // (M - 1) // 16 * 16
        assert (F - 1) * ldb > 0xF0000000 and (M - 1) * lda > 0xF0000000
        Bf = [far(b, ldb, buf, j * K) for j, b in enumerate(B)]  # side by side in one buffer
        Af = far(A, lda, torch.empty(1 << 32, dtype=torch.uint8, device=gpu))
        for fn in ("fp8q_glu_blockscaled", "fp8q_glu_blockscaled_fast"):
            h, hf = torch.empty(M, F, device=gpu), out.as_strided((M, F), (ldo, 1))
            glu_call(fq, fn, A, E4, sA, B, E4, sB, 0, h, None, M, F, K)
            glu_call(fq, fn, Af, E4, sA, Bf, E4, sB, 0, hf, None, M, F, K)
            assert torch.equal(h, hf)
        for name in ("fp8q_gemm_blockscaled_fast", "fp8q_gemm_blockscaled_few")[:1 if M > 64 else 2]:
            C, Cf = torch.empty(M, F, device=gpu), out.as_strided((M, F), (ldo, 1))
            for a, b, c in ((A, B[0], C), (Af, Bf[0], Cf)):
                getattr(fq, name)(a, E4, a.stride(0), sA, Kb, 1, b, E4, b.stride(0), sB[0], 2, Kb, 1, c, c.stride(0), M, F, K)
            assert torch.equal(C, Cf)
        del Af


def test_norm_and_gradients_of_rows_far_apart(fq, gpu):
    """Row offsets past 2^32 bytes in every operand: the results are those of adjacent rows."""
    rows, cols, ld = 300, 256, 1 << 23  # 5 GB of bf16
    bufs = [torch.empty(rows * ld, dtype=torch.bfloat16, device=gpu) for _ in range(4)]
    x, r, dy = (W.normal((rows, cols), seed=i, device=gpu, dtype=torch.bfloat16) for i in range(3))
    w = torch.ones(cols, device=gpu)
    xf, rf, zf, yf = (far(t, ld, b) for t, b in zip((x, r, x, x), bufs))

    def norm(x, r, z, y):
        q, s, rstd = torch.empty(rows, cols, dtype=torch.uint8, device=gpu), torch.empty(rows, 2, device=gpu), torch.empty(rows, device=gpu)
        n = [t.stride(0) for t in (x, r, z, y)]
        fq.fp8q_rmsnorm_1x128(x, n[0], r, n[1], w, rows, cols, NEPS, z, n[2], y, n[3], E4, EPS, q, cols, s, 2, rstd)
        return z, y, q, s, rstd

    got, want = norm(xf, rf, zf, yf), norm(x, r, torch.empty_like(x), torch.empty_like(x))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    rstd, dyf = want[4], far(dy, ld, bufs[0])
    ws = torch.empty(fq.fp8q_rmsnorm_bwd_workspace(rows, cols) // 4, device=gpu)

    def bwd(dy, z, dres, dx):
        dw = torch.empty(cols, device=gpu)
        n = [t.stride(0) for t in (dy, z, dres, dx)]
        fq.fp8q_rmsnorm_bwd(dy, n[0], z, n[1], w, rstd, dres, n[2], rows, cols, dx, n[3], dw, ws, ws.numel() * 4)
        return dx, dw

    assert all(torch.equal(a, b) for a, b in zip(bwd(dyf, zf, rf, yf), bwd(dy, want[0], r, torch.empty_like(x))))
    # the gated projection's gradient: dh and gu far apart, and its transposed codes
    M, F = rows, cols // 2
    dh, gu = dy[:, :F].contiguous(), r
    plain = bwd_call(fq, dh, gu, 0, E5, E4, M, F)
    ldt = 1 << 24
    T = torch.empty(2 * F * ldt, dtype=torch.uint8, device=gpu).as_strided((2 * F, 384), (ldt, 1))
    D, Ds, s = torch.empty(M, 2 * F, dtype=torch.uint8, device=gpu), torch.empty(M, 2, device=gpu), torch.empty(2 * F, 3, device=gpu)
    dhf, guf = far(dh, ld, bufs[2]), far(gu, ld, bufs[3])
    fq.fp8q_glu_bwd_q(dhf, ld, guf, ld, 0, E5, EPS, D, 2 * F, Ds, 2, T, ldt, s, 3, E4, None, 0, None, 0, M, F)
    assert all(torch.equal(a, b) for a, b in zip((D, Ds, T, s), plain))

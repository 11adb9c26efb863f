"""GPU checks of the feed-forward operators' paths that small shapes do not reach: explicit streams, the tiled kernels'
epilogues, long reductions, many token blocks, very many rows.  Tolerances as in test_gpu_ffn.py.
"""
import pytest
import torch

from block_scaled_precision_amax_amd import workloads as W
from test_gpu_ffn import E4, E5, EPS, NEPS, glu_call, operands

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

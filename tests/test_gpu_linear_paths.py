"""GPU checks of what test_gpu_linear.py leaves out of the layer norm and the linear layer.  Tolerances as there."""
import pytest
import torch

from block_scaled_precision_amax_amd import workloads as W
from test_gpu_linear import E4, E5, EPS, ERF, GELU, NONE, RELU, SILU, U, act64, bwd_call, check_codes, run_norm

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

"""Refusals of the layer norm and the linear layer, without a GPU: every bad
argument is answered with its status before anything would be enqueued, and
the binding's checks of types and devices raise."""
import pytest
import torch

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced


def _call(fq, name, ok, kw):
    assert not set(kw) - set(ok), kw
    rc = getattr(fq.lib(), name)(*{**ok, **kw}.values())
    return rc, fq.lib().fp8q_last_error().decode()


NORM = dict(x=FAKE, dt=1, ldx=256, res=FAKE, ldr=256, w=FAKE, b=FAKE, wdt=0, rows=4, cols=256, neps=1e-5, z=FAKE, ldz=256,
            y=FAKE, ldy=256, f=0, eps=1e-12, q=FAKE, ldq=256, s=FAKE, ld_s=2, mean=FAKE, rstd=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(s=None), "EINVAL"), (dict(q=None, s=None, y=None), "EINVAL"),
    (dict(dt=2), "EINVAL"), (dict(wdt=3), "EINVAL"), (dict(f=2), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(rows=-1), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(neps=0.0), "EINVAL"), (dict(neps=float("nan")), "EINVAL"),
    (dict(eps=0.0), "EINVAL"), (dict(eps=float("inf")), "EINVAL"), (dict(cols=200), "ESHAPE"), (dict(cols=12), "ESHAPE"),
    (dict(cols=65536 + 128), "ESHAPE"), (dict(rows=1 << 31), "ESHAPE"), (dict(ldx=128), "EINVAL"),
    (dict(ldr=128), "EINVAL"), (dict(ldz=128), "EINVAL"), (dict(ldy=128), "EINVAL"), (dict(ldq=128), "EINVAL"),
    (dict(ld_s=1), "EINVAL"), (dict(x=FAKE + 8), "EALIGN"), (dict(w=FAKE + 4), "EALIGN"), (dict(b=FAKE + 8), "EALIGN"),
    (dict(ldx=260), "EALIGN"), (dict(ldq=264), "EALIGN"), (dict(s=FAKE + 2), "EALIGN"), (dict(mean=FAKE + 1), "EALIGN"),
    (dict(rstd=FAKE + 1), "EALIGN"),
])
def test_layernorm_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_layernorm_1x128", NORM, kw)
    assert rc == getattr(fq, status) and msg.startswith("layernorm_1x128"), (rc, msg)


NORM_BWD = dict(dy=FAKE, dt=1, lddy=256, z=FAKE, ldz=256, w=FAKE, wdt=0, mean=FAKE, rstd=FAKE, dres=FAKE, lddr=256, rows=4,
                cols=256, dx=FAKE, lddx=256, dw=FAKE, db=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), "EINVAL"), (dict(z=None), "EINVAL"), (dict(mean=None), "EINVAL"), (dict(rstd=None), "EINVAL"),
    (dict(dx=None), "EINVAL"), (dict(ws=None), "EINVAL"), (dict(ws=None, db=None), "EINVAL"),
    (dict(ws=None, dw=None), "EINVAL"), (dict(ws_bytes=64), "EINVAL"), (dict(dt=5), "EINVAL"), (dict(wdt=-1), "EINVAL"),
    (dict(rows=0), "EINVAL"), (dict(rows=1 << 31), "ESHAPE"), (dict(cols=130), "ESHAPE"), (dict(lddx=128), "EINVAL"),
    (dict(lddy=260), "EALIGN"), (dict(ws=FAKE + 4), "EALIGN"), (dict(dw=FAKE + 2), "EALIGN"), (dict(db=FAKE + 2), "EALIGN"),
    (dict(dres=FAKE + 8), "EALIGN"), (dict(w=FAKE + 8), "EALIGN"), (dict(mean=FAKE + 2), "EALIGN"),
])
def test_layernorm_bwd_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_layernorm_bwd", NORM_BWD, kw)
    assert rc == getattr(fq, status) and msg.startswith("layernorm_bwd"), (rc, msg)


def test_layernorm_bwd_workspace(fq):
    for rows in (1, 3, 100, 5000, 1 << 20):
        for cols in (8, 128, 1608, 2048, 4096, 16384, 65536):
            b = fq.fp8q_layernorm_bwd_workspace(rows, cols)
            assert 8 * cols <= b <= 4096 * cols and b % (8 * cols) == 0
    for bad in ((0, 128), (1, 0), (1, 130), (1, 65664), (-1, 128), (1 << 31, 128)):
        assert fq.fp8q_layernorm_bwd_workspace(*bad) == 0


LINEAR = dict(A=FAKE, fa=0, lda=256, sA=FAKE, sm=2, skb=1, B=FAKE, fb=0, ldb=256, sB=FAKE, sn=2, sk=1, bias=FAKE, bdt=0, act=2,
              res=FAKE, ldr=128, C=FAKE, odt=1, ldc=128, pre=FAKE, ldpre=128, M=40, N=128, K=256, ws=FAKE,
              ws_bytes=1 << 30, stream=None)
BAD = [
    (dict(A=None), "EINVAL"), (dict(sA=None), "EINVAL"), (dict(B=None), "EINVAL"), (dict(sB=None), "EINVAL"),
    (dict(fa=2), "EINVAL"), (dict(fb=-1), "EINVAL"), (dict(M=0), "EINVAL"), (dict(N=0), "EINVAL"), (dict(K=0), "EINVAL"),
    (dict(K=192), "ESHAPE"), (dict(lda=128), "EINVAL"), (dict(ldb=128), "EINVAL"), (dict(sm=-1), "EINVAL"),
    (dict(sk=-1), "EINVAL"), (dict(A=FAKE + 8), "EALIGN"), (dict(ldb=264), "EALIGN"), (dict(sA=FAKE + 2), "EALIGN"),
    (dict(ldb=1 << 32), "ESHAPE"), (dict(act=5), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(bdt=2), "EINVAL"),
    (dict(bias=FAKE + 2), "EALIGN"), (dict(bias=FAKE + 1, bdt=1), "EALIGN"), (dict(ldpre=127), "EINVAL"),
    (dict(pre=FAKE + 1), "EALIGN"),
]


@pytest.mark.parametrize("name", ["fp8q_linear_blockscaled", "fp8q_linear_blockscaled_fast"])
@pytest.mark.parametrize("kw,status", BAD + [
    (dict(C=None), "EINVAL"), (dict(odt=2), "EINVAL"), (dict(ldc=127), "EINVAL"), (dict(C=FAKE + 1), "EALIGN"),
    (dict(ldr=127), "EINVAL"), (dict(res=FAKE + 1), "EALIGN"), (dict(res=FAKE + 2, odt=0), "EALIGN")])
def test_linear_refusals(fq, name, kw, status):
    rc, msg = _call(fq, name, LINEAR, kw)
    assert rc == getattr(fq, status) and msg.startswith(name[5:] + ":"), (rc, msg)


LINEAR_Q = {k: v for k, v in LINEAR.items() if k not in ("res", "ldr", "C", "odt", "ldc")}
LINEAR_Q = dict(list(LINEAR_Q.items())[:15] + [("fc", 0), ("eps", 1e-12), ("Cq", FAKE), ("ldcq", 128), ("Cs", FAKE), ("ld_cs", 1)]
                + list(LINEAR_Q.items())[15:])


@pytest.mark.parametrize("name", ["fp8q_linear_blockscaled_q", "fp8q_linear_blockscaled_q_fast"])
@pytest.mark.parametrize("kw,status", BAD + [
    (dict(Cq=None), "EINVAL"), (dict(Cs=None), "EINVAL"), (dict(fc=2), "EINVAL"), (dict(eps=-1.0), "EINVAL"),
    (dict(N=100), "ESHAPE"), (dict(ldcq=112), "EINVAL"), (dict(ld_cs=0), "EINVAL"), (dict(Cs=FAKE + 2), "EALIGN"),
    (dict(Cq=FAKE + 8), "EALIGN"), (dict(ldcq=136), "EALIGN"), (dict(ws=None), "EINVAL"), (dict(ws_bytes=0), "EINVAL"),
    (dict(ws=FAKE + 8), "EALIGN")])
def test_linear_q_refusals(fq, name, kw, status):
    rc, msg = _call(fq, name, LINEAR_Q, kw)
    assert rc == getattr(fq, status) and msg.startswith(name[5:] + ":"), (rc, msg)


def test_linear_workspace(fq):
    w = fq.fp8q_linear_blockscaled_workspace
    for fast in (0, 1):
        # a token's codes go through the workspace; many rows need none
        assert w(fast, 1, 1, 18432, 7168) >= 4 * 18432
        assert w(fast, 0, 16384, 18432, 7168) == w(fast, 1, 16384, 18432, 7168) == 0
        for bad in ((0, 128, 128), (1, 0, 128), (1, 128, 0), (1, 128, 192), (-1, 128, 128), (1 << 40, 128, 128)):
            assert w(fast, 1, *bad) == 0
        assert w(fast, 1, 1, 100, 128) == 0


BWD = dict(dC=FAKE, dt=1, lddc=128, pre=FAKE, ldpre=128, act=0, fc=1, eps=1e-12, Dq=FAKE, lddq=128, Ds=FAKE, ld_ds=1, Dt=FAKE,
           lddt=256, Dst=FAKE, ld_dst=2, fh=0, Ht=FAKE, ldht=256, Hst=FAKE, ld_hst=2, dbias=FAKE, M=200, N=128, ws=FAKE,
           ws_bytes=1024, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dC=None), "EINVAL"), (dict(Dq=None), "EINVAL"), (dict(Ds=None), "EINVAL"), (dict(Dst=None), "EINVAL"),
    (dict(Dt=None), "EINVAL"), (dict(Hst=None), "EINVAL"), (dict(Ht=None), "EINVAL"), (dict(pre=None), "EINVAL"),
    (dict(pre=None, act=2), "EINVAL"), (dict(dt=2), "EINVAL"), (dict(fc=2), "EINVAL"), (dict(fh=2), "EINVAL"),
    (dict(act=5), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(eps=0.0), "EINVAL"), (dict(M=0), "EINVAL"),
    (dict(N=0), "EINVAL"), (dict(N=96), "ESHAPE"), (dict(M=(1 << 31) + 1), "ESHAPE"), (dict(lddc=64), "EINVAL"),
    (dict(ldpre=120), "EINVAL"), (dict(lddq=112), "EINVAL"), (dict(ld_ds=0), "EINVAL"), (dict(lddt=208), "EINVAL"),
    (dict(ld_dst=1), "EINVAL"), (dict(ldht=208), "EINVAL"), (dict(ld_hst=1), "EINVAL"), (dict(dC=FAKE + 8), "EALIGN"),
    (dict(lddc=132), "EALIGN"), (dict(ldpre=132), "EALIGN"), (dict(lddt=264), "EALIGN"), (dict(Ht=FAKE + 4), "EALIGN"),
    (dict(Dst=FAKE + 2), "EALIGN"), (dict(dbias=FAKE + 2), "EALIGN"), (dict(ws=None), "EINVAL"),
    (dict(ws_bytes=1023), "EINVAL"), (dict(ws=FAKE + 8), "EALIGN"),
])
def test_linear_bwd_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_linear_bwd_q", BWD, kw)
    assert rc == getattr(fq, status) and msg.startswith("linear_bwd_q"), (rc, msg)


def test_linear_bwd_too_many_blocks(fq):
    M = 1 << 31
    big = dict(M=M, N=128, lddt=M, ld_dst=M // 128, ldht=M, ld_hst=M // 128, ws_bytes=1 << 40)
    rc, msg = _call(fq, "fp8q_linear_bwd_q", BWD, big)
    assert rc == fq.ESHAPE and "tiles" in msg


def test_linear_bwd_workspace(fq):
    w = fq.fp8q_linear_bwd_q_workspace
    assert w(1, 128) == w(128, 4096) == 0 and w(129, 4096) == 4 * 2 * 4096 and w(8192, 18432) == 4 * 64 * 18432
    for bad in ((0, 128), (300, 0), (300, 100), (-1, 128), (1 << 40, 128)):
        assert w(*bad) == 0


def test_the_binding_refuses_types_and_host_tensors(fq):
    bf, f32 = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 128)
    w = torch.ones(128)
    ln = lambda x, r, w, b: fq.fp8q_layernorm_1x128(x, 128, r, 128, w, b, 2, 128, 1e-5, None, 0, x, 128, 0, 1e-12, None, 0,  # noqa: E731
                                                    None, 0, stream=0)
    with pytest.raises(TypeError):
        ln(bf, f32, w, None)
    with pytest.raises(TypeError):
        ln(bf, bf, w, w.bfloat16())
    with pytest.raises(TypeError):
        ln(bf, bf, w.half(), None)
    with pytest.raises(ValueError, match="GPU"):
        ln(bf, bf, w, w)
    with pytest.raises(TypeError):
        fq.fp8q_layernorm_bwd(bf, 128, bf, 128, w, w.double(), w, None, 0, 2, 128, bf, 128, stream=0)
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_layernorm_bwd(bf, 128, bf, 128, w, w, w, None, 0, 2, 128, bf, 128, stream=0)
    q, s = torch.zeros(2, 128, dtype=torch.uint8), torch.zeros(2, 1)

    def lin(f=fq.fp8q_linear_blockscaled, A=q, sA=s, bias=w, res=bf, C=bf, pre=None):
        f(A, 0, 128, sA, 1, 1, q, 0, 128, s, 1, 1, bias, 0, res, 128, C, 128, pre, 128, 2, 2, 128, stream=0)

    for f in (fq.fp8q_linear_blockscaled, fq.fp8q_linear_blockscaled_fast):
        for bad in (dict(A=bf), dict(sA=bf), dict(bias=w.half()), dict(res=f32), dict(C=bf.half(), res=None), dict(pre=f32)):
            with pytest.raises(TypeError):
                lin(f, **bad)
        with pytest.raises(ValueError, match="GPU"):
            lin(f)
    for f in (fq.fp8q_linear_blockscaled_q, fq.fp8q_linear_blockscaled_q_fast):
        with pytest.raises(TypeError):
            f(q, 0, 128, s, 1, 1, q, 0, 128, s, 1, 1, w, 0, 0, 1e-12, bf, 128, s, 1, None, 0, 2, 128, 128, stream=0)
        with pytest.raises(ValueError, match="GPU"):
            f(q, 0, 128, s, 1, 1, q, 0, 128, s, 1, 1, w, 0, 0, 1e-12, q, 128, s, 1, None, 0, 2, 128, 128, stream=0)
    with pytest.raises(TypeError):
        fq.fp8q_linear_bwd_q(bf, 128, f32, 128, 0, 0, 1e-12, q, 128, s, 1, None, 0, None, 0, 0, None, 0, None, 0, None, 2, 128,
                             stream=0)
    with pytest.raises(ValueError, match="GPU"):
        fq.fp8q_linear_bwd_q(bf, 128, bf, 128, 0, 0, 1e-12, q, 128, s, 1, None, 0, None, 0, 0, None, 0, None, 0, None, 2, 128,
                             stream=0)

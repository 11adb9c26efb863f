"""Refusals of the feed-forward entry points, without a GPU: every bad
argument is answered with its status before anything would be enqueued, and
the binding's dtype checks raise."""
import pytest
import torch

FAKE = 0x10000  # a 16-byte aligned address that is never dereferenced


def _call(fq, name, ok, kw):
    assert not set(kw) - set(ok), kw
    rc = getattr(fq.lib(), name)(*{**ok, **kw}.values())
    return rc, fq.lib().fp8q_last_error().decode()


NORM = dict(x=FAKE, dt=1, ldx=256, res=FAKE, ldr=256, w=FAKE, wdt=0, rows=4, cols=256, neps=1e-6, z=FAKE, ldz=256, y=FAKE,
            ldy=256, f=0, eps=1e-12, q=FAKE, ldq=256, s=FAKE, ld_s=2, rstd=FAKE, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=None), "EINVAL"), (dict(w=None), "EINVAL"), (dict(q=None), "EINVAL"), (dict(s=None), "EINVAL"),
    (dict(q=None, s=None, y=None), "EINVAL"), (dict(dt=2), "EINVAL"), (dict(wdt=3), "EINVAL"), (dict(f=2), "EINVAL"),
    (dict(rows=0), "EINVAL"), (dict(rows=-1), "EINVAL"), (dict(cols=0), "EINVAL"), (dict(neps=0.0), "EINVAL"),
    (dict(neps=float("nan")), "EINVAL"), (dict(eps=0.0), "EINVAL"), (dict(eps=float("inf")), "EINVAL"),
    (dict(cols=200), "ESHAPE"), (dict(cols=65536 + 128), "ESHAPE"), (dict(rows=1 << 31), "ESHAPE"),
    (dict(ldx=128), "EINVAL"), (dict(ldr=128), "EINVAL"), (dict(ldz=128), "EINVAL"), (dict(ldy=128), "EINVAL"),
    (dict(ldq=128), "EINVAL"), (dict(ld_s=1), "EINVAL"), (dict(x=FAKE + 8), "EALIGN"), (dict(w=FAKE + 4), "EALIGN"),
    (dict(ldx=260), "EALIGN"), (dict(ldq=264), "EALIGN"), (dict(s=FAKE + 2), "EALIGN"), (dict(rstd=FAKE + 1), "EALIGN"),
])
def test_rmsnorm_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_rmsnorm_1x128", NORM, kw)
    assert rc == getattr(fq, status) and msg.startswith("rmsnorm_1x128"), (rc, msg)


NORM_BWD = dict(dy=FAKE, dt=1, lddy=256, z=FAKE, ldz=256, w=FAKE, wdt=0, rstd=FAKE, dres=FAKE, lddr=256, rows=4, cols=256,
                dx=FAKE, lddx=256, dw=FAKE, ws=FAKE, ws_bytes=1 << 20, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dy=None), "EINVAL"), (dict(z=None), "EINVAL"), (dict(rstd=None), "EINVAL"), (dict(dx=None), "EINVAL"),
    (dict(ws=None), "EINVAL"), (dict(ws_bytes=64), "EINVAL"), (dict(dt=5), "EINVAL"), (dict(rows=0), "EINVAL"),
    (dict(cols=130), "ESHAPE"), (dict(lddx=128), "EINVAL"), (dict(lddy=260), "EALIGN"), (dict(ws=FAKE + 4), "EALIGN"),
    (dict(dw=FAKE + 2), "EALIGN"), (dict(dres=FAKE + 8), "EALIGN"),
])
def test_rmsnorm_bwd_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_rmsnorm_bwd", NORM_BWD, kw)
    assert rc == getattr(fq, status) and msg.startswith("rmsnorm_bwd"), (rc, msg)


def test_rmsnorm_bwd_workspace(fq):
    for rows in (1, 3, 100, 5000, 1 << 20):
        for cols in (128, 2048, 4096, 16384, 65536):
            b = fq.fp8q_rmsnorm_bwd_workspace(rows, cols)
            assert 4 * cols <= b <= 4096 * cols and b % (4 * cols) == 0
    for bad in ((0, 128), (1, 0), (1, 130), (1, 65664), (-1, 128)):
        assert fq.fp8q_rmsnorm_bwd_workspace(*bad) == 0


GLU = dict(A=FAKE, fa=0, lda=256, sA=FAKE, sm=2, skb=1, Bg=FAKE, Bu=FAKE, fb=0, ldb=256, sBg=FAKE, sBu=FAKE, sn=2, sk=1,
           act=0, H=FAKE, odt=1, ldh=128, gu=FAKE, ldgu=256, M=40, F=128, K=256, stream=None)
PROJ_BAD = [
    (dict(A=None), "EINVAL"), (dict(sA=None), "EINVAL"), (dict(fa=2), "EINVAL"), (dict(fb=-1), "EINVAL"),
    (dict(M=0), "EINVAL"), (dict(K=0), "EINVAL"), (dict(K=192), "ESHAPE"), (dict(lda=128), "EINVAL"),
    (dict(ldb=128), "EINVAL"), (dict(sm=-1), "EINVAL"), (dict(sk=-1), "EINVAL"), (dict(A=FAKE + 8), "EALIGN"),
    (dict(ldb=264), "EALIGN"), (dict(sA=FAKE + 2), "EALIGN"), (dict(ldb=1 << 32), "ESHAPE"),
]
GLU_BAD = PROJ_BAD + [(dict(Bg=None), "EINVAL"), (dict(Bu=None), "EINVAL"), (dict(sBu=None), "EINVAL"), (dict(F=0), "EINVAL"),
                      (dict(act=2), "EINVAL"), (dict(act=-1), "EINVAL"), (dict(ldgu=255), "EINVAL"),
                      (dict(gu=FAKE + 1), "EALIGN"), (dict(Bu=FAKE + 4), "EALIGN")]


@pytest.mark.parametrize("name", ["fp8q_glu_blockscaled", "fp8q_glu_blockscaled_fast"])
@pytest.mark.parametrize("kw,status", GLU_BAD + [(dict(H=None), "EINVAL"), (dict(odt=2), "EINVAL"), (dict(ldh=127), "EINVAL"),
                                                 (dict(H=FAKE + 1), "EALIGN")])
def test_glu_refusals(fq, name, kw, status):
    rc, msg = _call(fq, name, GLU, kw)
    assert rc == getattr(fq, status) and msg.startswith(name[5:]), (rc, msg)


GLU_Q = dict(A=FAKE, fa=0, lda=256, sA=FAKE, sm=2, skb=1, Bg=FAKE, Bu=FAKE, fb=0, ldb=256, sBg=FAKE, sBu=FAKE, sn=2, sk=1,
             act=1, fc=0, eps=1e-12, Hq=FAKE, ldhq=128, Hs=FAKE, ld_hs=1, gu=None, ldgu=0, M=40, F=128, K=256, ws=FAKE,
             ws_bytes=4 * 40 * 128, stream=None)


@pytest.mark.parametrize("kw,status", [(k if "ldgu" not in k else dict(gu=FAKE, **k), s) for k, s in GLU_BAD] + [
    (dict(Hq=None), "EINVAL"), (dict(Hs=None), "EINVAL"), (dict(fc=2), "EINVAL"), (dict(eps=-1.0), "EINVAL"),
    (dict(F=100), "ESHAPE"), (dict(ldhq=100), "EINVAL"), (dict(ld_hs=0), "EINVAL"), (dict(Hs=FAKE + 2), "EALIGN"),
    (dict(ws=None), "EINVAL"), (dict(ws_bytes=4 * 40 * 128 - 1), "EINVAL"), (dict(ws=FAKE + 8), "EALIGN"),
    (dict(Hq=FAKE + 2), "EALIGN"), (dict(ldhq=130), "EALIGN")])
def test_glu_q_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_glu_blockscaled_q", GLU_Q, {**dict(gu=None), **kw} if "gu" not in kw else {"ldgu": 256, **kw})
    assert rc == getattr(fq, status) and msg.startswith("glu_blockscaled_q"), (rc, msg)


def test_glu_q_workspace(fq):
    assert fq.fp8q_glu_blockscaled_q_workspace(1, 18432) == 4 * 18432
    assert fq.fp8q_glu_blockscaled_q_workspace(16384, 18432) == 0
    for bad in ((0, 128), (1, 0), (1, 130)):
        assert fq.fp8q_glu_blockscaled_q_workspace(*bad) == 0


GLU_BWD = dict(dH=FAKE, dt=1, lddh=128, gu=FAKE, ldgu=256, act=0, fc=1, eps=1e-12, Dq=FAKE, lddq=256, Ds=FAKE, ld_ds=2,
               Dt=FAKE, lddt=256, Dst=FAKE, ld_dst=2, fh=0, Ht=FAKE, ldht=256, Hst=FAKE, ld_hst=2, M=200, F=128, stream=None)


@pytest.mark.parametrize("kw,status", [
    (dict(dH=None), "EINVAL"), (dict(gu=None), "EINVAL"), (dict(Dq=None), "EINVAL"), (dict(Ds=None), "EINVAL"),
    (dict(Dst=None), "EINVAL"), (dict(Dt=None), "EINVAL"), (dict(Hst=None), "EINVAL"), (dict(dt=2), "EINVAL"),
    (dict(fc=2), "EINVAL"), (dict(fh=2), "EINVAL"), (dict(act=7), "EINVAL"), (dict(eps=0.0), "EINVAL"),
    (dict(M=0), "EINVAL"), (dict(F=0), "EINVAL"), (dict(F=96), "ESHAPE"), (dict(lddh=64), "EINVAL"),
    (dict(ldgu=248), "EINVAL"), (dict(lddq=128), "EINVAL"), (dict(ld_ds=1), "EINVAL"), (dict(lddt=208), "EINVAL"),
    (dict(ld_dst=1), "EINVAL"), (dict(ldht=208), "EINVAL"), (dict(ld_hst=1), "EINVAL"), (dict(dH=FAKE + 8), "EALIGN"),
    (dict(lddh=132), "EALIGN"), (dict(ldgu=260), "EALIGN"), (dict(lddt=264), "EALIGN"), (dict(Ht=FAKE + 4), "EALIGN"),
    (dict(Dst=FAKE + 2), "EALIGN"),
])
def test_glu_bwd_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_glu_bwd_q", GLU_BWD, kw)
    assert rc == getattr(fq, status) and msg.startswith("glu_bwd_q"), (rc, msg)


FEW = dict(A=FAKE, fa=0, lda=256, sA=FAKE, sm=2, skb=1, B=FAKE, fb=0, ldb=256, sB=FAKE, gb=2, sn=2, sk=1, C=FAKE, odt=0,
           ldc=128, M=4, N=128, K=256, stream=None)


@pytest.mark.parametrize("kw,status", PROJ_BAD + [
    (dict(B=None), "EINVAL"), (dict(C=None), "EINVAL"), (dict(gb=0), "EINVAL"), (dict(odt=2), "EINVAL"),
    (dict(N=0), "EINVAL"), (dict(M=65), "ESHAPE"), (dict(ldc=127), "EINVAL"), (dict(C=FAKE + 2), "EALIGN")])
def test_few_refusals(fq, kw, status):
    rc, msg = _call(fq, "fp8q_gemm_blockscaled_few", FEW, kw)
    assert rc == getattr(fq, status) and msg.startswith("gemm_blockscaled_few"), (rc, msg)


def test_mixed_dtypes_are_refused_by_the_binding(fq):
    x, r = torch.zeros(2, 128, dtype=torch.bfloat16), torch.zeros(2, 128)
    w = torch.ones(128)
    with pytest.raises(TypeError):
        fq.fp8q_rmsnorm_1x128(x, 128, r, 128, w, 2, 128, 1e-6, None, 0, None, 0, 0, 1e-12, 1, 128, 1, 1, None, stream=0)
    with pytest.raises(TypeError):
        fq.fp8q_rmsnorm_bwd(x, 128, r, 128, w, w, None, 0, 2, 128, x, 128, stream=0)
    with pytest.raises(TypeError):
        fq.fp8q_glu_bwd_q(x.half(), 128, 1, 256, 0, 0, 1e-12, 1, 256, 1, 2, None, 0, None, 0, 0, None, 0, None, 0, 2, 128,
                          stream=0)


class _Recorder:
    """Stands in for the library and for torch's stream calls: which stream was current when memory was taken."""

    def __init__(self, fq, monkeypatch):
        self.taken, self.current, self.call = [], ["current"], None
        rec = self

        class Lib:
            def fp8q_glu_blockscaled_q_workspace(self, M, F):
                return 512

            def fp8q_glu_blockscaled_q(self, *args):
                rec.call = args
                return fq.OK

        class On:
            def __init__(self, stream):
                self.stream = stream

            def __enter__(self):
                rec.current.append(self.stream)

            def __exit__(self, *e):
                rec.current.pop()

        class Block:
            def data_ptr(self):
                return FAKE

            def record_stream(self, stream):
                pass

        def empty(n, dtype, device):
            rec.taken.append((n, str(device), rec.current[-1]))
            return Block()

        monkeypatch.setattr(fq, "lib", lambda: Lib())
        monkeypatch.setattr(torch, "empty", empty)
        monkeypatch.setattr(torch.cuda, "stream", On)
        monkeypatch.setattr(torch.cuda, "ExternalStream", lambda h, device=None: ("external", h, str(device)))
        monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: ("default", str(device)))
        monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)


def _glu_q(fq, A, out, stream):
    s = torch.zeros(2, 1)
    fq.fp8q_glu_blockscaled_q(A, 0, 128, s, 1, 1, FAKE, FAKE, 0, 128, s, s, 1, 1, 0, 0, 1e-12, out, 128, s, 1, None, 0, 2, 128,
                              128, stream=stream)


@pytest.mark.parametrize("handle,want", [(0x7700, ("external", 0x7700, "cpu")), (0, ("default", "cpu"))])
def test_workspace_is_taken_on_the_stream_that_uses_it(fq, monkeypatch, handle, want):
    """A block from another stream's pool may still be read or written by that stream's pending work."""
    rec = _Recorder(fq, monkeypatch)
    A = torch.zeros(2, 128, dtype=torch.uint8)
    _glu_q(fq, A, A, handle)
    assert rec.taken == [(512, "cpu", want)]
    assert rec.call[-1] == handle and rec.call[-2] == 512


def test_workspace_on_a_stream_object(fq, monkeypatch):
    class Stream:
        cuda_stream, device = 0x7700, torch.device("cpu")

    rec = _Recorder(fq, monkeypatch)
    A = torch.zeros(2, 128, dtype=torch.uint8)
    _glu_q(fq, A, A, Stream)
    assert [t[2] for t in rec.taken] == [Stream] and rec.call[-1] == 0x7700


def test_workspace_with_raw_pointers(fq, monkeypatch):
    """Outputs given as addresses: the device is the first operand's, or the current one."""
    rec = _Recorder(fq, monkeypatch)
    A = torch.zeros(2, 128, dtype=torch.uint8)
    _glu_q(fq, A, FAKE, 0x7700)
    _glu_q(fq, FAKE, FAKE, 0x7700)
    assert [t[1] for t in rec.taken] == ["cpu", "cuda:3"]
    assert rec.taken[1][2] == ("external", 0x7700, "cuda:3") and rec.call[0] == FAKE


F32, B16, U8 = (torch.zeros(4, 256, dtype=d) for d in (torch.float32, torch.bfloat16, torch.uint8))


def _norm(fq, x=B16, w=F32, q=U8, s=F32, rstd=F32):
    fq.fp8q_rmsnorm_1x128(x, 256, None, 0, w, 0, 256, 1e-6, None, 0, None, 0, 0, 1e-12, q, 256, s, 2, rstd, stream=0)


def _norm_bwd(fq, x=B16, rstd=F32, dw=F32):
    fq.fp8q_rmsnorm_bwd(x, 256, x, 256, F32, rstd, None, 0, 0, 256, x, 256, dw, F32, 4096, stream=0)


def _glu(fq, name="fp8q_glu_blockscaled", A=U8, sA=F32, Bg=U8, Bu=U8, sBg=F32, sBu=F32, gu=B16):
    getattr(fq, name)(A, 0, 256, sA, 2, 1, Bg, Bu, 0, 256, sBg, sBu, 2, 1, 0, F32, 128, gu, 256, 0, 128, 256, stream=0)


def _glu_fast(fq, **kw):
    _glu(fq, "fp8q_glu_blockscaled_fast", **kw)


def _glu_codes(fq, A=U8, sA=F32, Bg=U8, Bu=U8, sBg=F32, sBu=F32, H=U8, Hs=F32, gu=B16):
    fq.fp8q_glu_blockscaled_q(A, 0, 256, sA, 2, 1, Bg, Bu, 0, 256, sBg, sBu, 2, 1, 0, 0, 1e-12, H, 128, Hs, 1, gu, 256, 0, 128,
                              256, F32, 4096, stream=0)


def _glu_bwd(fq, gu=B16, D=U8, Ds=F32, Dt=U8, Dst=F32, Ht=U8, Hst=F32):
    fq.fp8q_glu_bwd_q(B16, 128, gu, 256, 0, 0, 1e-12, D, 256, Ds, 2, Dt, 128, Dst, 1, 0, Ht, 128, Hst, 1, 0, 128, stream=0)


def _few(fq, A=U8, sA=F32, B=U8, sB=F32):
    fq.fp8q_gemm_blockscaled_few(A, 0, 256, sA, 2, 1, B, 0, 256, sB, 2, 2, 1, F32, 128, 0, 128, 256, stream=0)


TYPED = [(_norm, dict(f4=("s", "rstd"), u8=("q",))), (_norm_bwd, dict(f4=("rstd", "dw"))),
         (_glu, dict(f4=("sA", "sBg", "sBu"), u8=("A", "Bg", "Bu"), b2=("gu",))),
         (_glu_fast, dict(f4=("sA", "sBg", "sBu"), u8=("A", "Bg", "Bu"), b2=("gu",))),
         (_glu_codes, dict(f4=("sA", "sBg", "sBu", "Hs"), u8=("A", "Bg", "Bu", "H"), b2=("gu",))),
         (_glu_bwd, dict(f4=("Ds", "Dst", "Hst"), u8=("D", "Dt", "Ht"), b2=("gu",))),
         (_few, dict(f4=("sA", "sB"), u8=("A", "B")))]
WRONG = dict(f4=(B16, F32.double(), F32.half()), u8=(B16, F32), b2=(F32, F32.half(), U8))


@pytest.mark.parametrize("call,arg,kind", [(c, a, k) for c, kinds in TYPED for k, args in kinds.items() for a in args])
def test_operands_of_a_fixed_type(fq, call, arg, kind):
    """An fp32 output given as a narrower tensor would be written past its end, another type misread: the binding refuses
    it.  Every call here has no rows, which the library answers (EINVAL) once the types pass."""
    for wrong in WRONG[kind]:
        with pytest.raises(TypeError):
            call(fq, **{arg: wrong})
    right = dict(f4=(F32, FAKE), u8=(U8, U8.view(torch.int8), U8.view(torch.float8_e4m3fn), U8.view(torch.float8_e5m2), FAKE),
                 b2=(B16, B16.view(torch.int16), FAKE))
    for ok in right[kind]:
        with pytest.raises(fq.Fp8qError):
            call(fq, **{arg: ok})


def test_glu_bwd_tiles_of_one_launch(fq):
    """A launch holds fewer than 2^32 threads; at 512 a tile that is 2^23 - 1 tiles."""
    F, M = 128 * 4096, 128 * 2048
    kw = dict(lddh=F, ldgu=2 * F, lddq=2 * F, ld_ds=F // 64, Dt=None, Dst=None, Ht=None, Hst=None, F=F, M=M)
    rc, msg = _call(fq, "fp8q_glu_bwd_q", GLU_BWD, kw)
    assert rc == fq.ESHAPE and "tiles" in msg, (rc, msg)

"""The layer norm and the linear layer without a GPU: what the binding asks of the library and of torch, on which device and
stream (with both replaced by recorders), workspaces, and refusals of sizes that overflow."""
import contextlib
import types

import pytest
import torch


class Operand:
    """A tensor of the second device, as far as the binding looks."""

    dtype, device = torch.bfloat16, torch.device("cuda", 1)

    def get_device(self):
        return 1


@pytest.fixture
def two_devices(fq, monkeypatch):
    """Device 0 current, operands on device 1; the library answers 256 bytes of workspace on device 0 and 512 on device 1."""
    r = types.SimpleNamespace(current=0, asked=[], given=[], called=[])

    @contextlib.contextmanager
    def device(d):
        before, r.current = r.current, d
        try:
            yield
        finally:
            r.current = before

    def ask(fast, codes, M, N, K):
        r.asked.append((r.current, fast, codes, M, N, K))
        return 256 << r.current

    def entry(name):
        def f(dev, *args):
            r.called.append((r.current, name, dev, args))
            return 0
        return f

    def workspace(n, handle, stream, t):
        r.given.append((n, handle, r.current if isinstance(t, int) else t.get_device()))
        return "workspace of %d" % n

    names = ("fp8q_linear_blockscaled", "fp8q_linear_blockscaled_fast", "fp8q_linear_blockscaled_q",
             "fp8q_linear_blockscaled_q_fast")
    fq.lib()
    monkeypatch.setattr(fq, "_lib", types.SimpleNamespace(fp8q_linear_blockscaled_workspace=ask))
    monkeypatch.setattr(fq, "_native", types.SimpleNamespace(**{n: entry(n) for n in names}))
    monkeypatch.setattr(fq, "_get_device", lambda: r.current)
    monkeypatch.setattr(fq, "_raw_stream", lambda d: 1000 + d)
    monkeypatch.setattr(fq, "_workspace", workspace)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(cuda_stream=1000 + r.current))
    return r


def forms(fq, A, t, **kw):
    """Every form of the linear layer: its name, whether it is the FP8-MFMA one and leaves codes, and a call of it."""
    a = (A, 0, 128, t, 1, 1, t, 0, 128, t, 1, 1, None, fq.ACT_NONE)
    for name in ("fp8q_linear_blockscaled", "fp8q_linear_blockscaled_fast"):
        yield name, int(name.endswith("fast")), 0, lambda f=getattr(fq, name): f(*a, None, 0, t, 8, None, 0, 3, 8, 128, **kw)
    for name in ("fp8q_linear_blockscaled_q", "fp8q_linear_blockscaled_q_fast"):
        yield name, int(name.endswith("fast")), 1, lambda f=getattr(fq, name): f(*a, 0, 1e-12, t, 128, t, 1, None, 0, 3, 128, 128,
                                                                                **kw)


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("stream", [None, 77])
def test_the_workspace_is_asked_for_and_taken_where_the_operands_lie(fq, two_devices, raw, stream):
    """A's own device, or with a raw pointer for A that of the first operand that is a tensor."""
    t = Operand()
    for name, fast, codes, call in forms(fq, 0x10000 if raw else t, t, stream=stream):
        call()
        N = 128 if codes else 8
        handle = stream or 1001
        assert two_devices.asked.pop() == (1, fast, codes, 3, N, 128)
        assert two_devices.given.pop() == (512, handle, 1)
        current, called, dev, args = two_devices.called.pop()
        assert (current, called, dev) == (1, name, 1) and args[-3:] == ("workspace of 512", 512, handle)
        assert not (two_devices.asked or two_devices.given or two_devices.called) and two_devices.current == 0


def test_a_workspace_that_is_given_is_not_asked_for(fq, two_devices):
    t = Operand()
    for name, _, _, call in forms(fq, t, t, ws=t, ws_bytes=99):
        call()
        current, called, dev, args = two_devices.called.pop()
        assert (current, called, dev) == (1, name, 1) and args[-3:] == (t, 99, 1001)
        assert not (two_devices.asked or two_devices.given)


def test_linear_workspace_of_any_size(fq):
    """Many rows may need one too, and a call without it is refused; bounded as the header says."""
    import random

    w = fq.fp8q_linear_blockscaled_workspace
    M, N, K = 8192, 7168, 18432
    need = w(1, 0, M, N, K)
    assert need > 0 and w(1, 1, M, N, K) == need
    p = 0x10000  # never dereferenced
    args = lambda ws, n: (p, 0, K, p, K // 128, 1, p, 0, K, p, K // 128, 1, None, 0, fq.ACT_NONE, None, 0, p, fq.BF16, N, None, 0,  # noqa: E731
                          M, N, K, ws, n, None)
    for ws, n in ((None, 0), (None, need), (p, need - 1)):
        assert fq.lib().fp8q_linear_blockscaled_fast(*args(ws, n)) == fq.EINVAL
        assert str(need) in fq.lib().fp8q_last_error().decode()
    assert fq.lib().fp8q_linear_blockscaled_fast(*args(p + 8, need)) == fq.EALIGN
    rng = random.Random(1)
    units = torch.cuda.get_device_properties(0).multi_processor_count if torch.cuda.is_available() else 256
    for _ in range(4000):
        M, N, K = (max(1, round(2 ** rng.uniform(0, 15))) for _ in range(3))
        N, K = -(-N // 128) * 128, -(-K // 128) * 128
        for fast in (0, 1):
            for codes in (0, 1):
                n = w(fast, codes, M, N, K)
                assert n == codes * 4 * M * N or 0 <= n < units << 22, (fast, codes, M, N, K, n)


def test_layernorm_bwd_workspace_is_at_most_2048_bytes_a_column(fq):
    for cols in (8, 128, 1608, 4096, 16384, 65536):
        assert max(fq.fp8q_layernorm_bwd_workspace(r, cols) for r in (1, 255, 256, 257, 513, 1025, 70000, (1 << 31) - 1)) \
            == 2048 * cols


SPANS = [dict(M=(1 << 57) + 128), dict(N=(1 << 57) + 128), dict(M=(1 << 62) + 128), dict(M=(1 << 33) + 128, lda=1 << 31),
         dict(N=(1 << 29) + 128, ldb=1 << 35), dict(K=(1 << 63) - 128, lda=(1 << 63) - 16, ldb=(1 << 63) - 16)]


@pytest.mark.parametrize("kw", SPANS)
@pytest.mark.parametrize("form", ["linear", "linear_fast", "linear_q", "linear_q_fast", "gemm", "gemm_fast", "gemm_q", "gemm_qt",
                                  "gemm_mx", "gemm_few", "glu", "glu_fast", "glu_q"])
def test_spans_that_pass_64_bits_are_refused(fq, form, kw):
    """The 4 GiB limit holds where the span itself overflows 64 bits and comes out small."""
    p, far, L = 0x10000, 1 << 60, fq.lib()  # p is never dereferenced
    c = dict(dict(M=128, N=128, K=128, lda=128, ldb=128), **kw)
    M, N, K = c["M"], c["N"], c["K"]
    if form == "gemm_few":
        M = min(M, 64)
    a, b, d, ld = (p, 0, c["lda"], p, 1, 1), (p, 0, c["ldb"], p), (M, N, K), max(N, M, 128)
    g, ep = (fq.GRAN_128x128, 1, 1), (None, 0, fq.ACT_NONE)
    glu = (*a, p, p, 0, c["ldb"], p, p, 1, 1, fq.ACT_SILU)
    rc = {
        "linear": lambda: L.fp8q_linear_blockscaled(*a, *b, 1, 1, *ep, None, 0, p, 0, ld, None, 0, *d, p, far, None),
        "linear_fast": lambda: L.fp8q_linear_blockscaled_fast(*a, *b, 1, 1, *ep, None, 0, p, 0, ld, None, 0, *d, p, far, None),
        "linear_q": lambda: L.fp8q_linear_blockscaled_q(*a, *b, 1, 1, *ep, 0, 1e-12, p, ld, p, ld, None, 0, *d, p, far, None),
        "linear_q_fast": lambda: L.fp8q_linear_blockscaled_q_fast(*a, *b, 1, 1, *ep, 0, 1e-12, p, ld, p, ld, None, 0, *d, p, far,
                                                                  None),
        "gemm": lambda: L.fp8q_gemm_blockscaled(*a, *b, *g, p, 0, ld, *d, None),
        "gemm_fast": lambda: L.fp8q_gemm_blockscaled_fast(*a, *b, *g, p, 0, ld, *d, None),
        "gemm_q": lambda: L.fp8q_gemm_blockscaled_q(*a, *b, *g, 0, 1e-12, p, ld, p, ld, *d, None),
        "gemm_qt": lambda: L.fp8q_gemm_blockscaled_qt(*a, *b, *g, 0, 1e-12, p, ld, p, ld, None, 0, None, 0, *d, None),
        "gemm_mx": lambda: L.fp8q_gemm_mx(*a[:4], far, *b, far, p, 0, ld, *d, None),
        "gemm_few": lambda: L.fp8q_gemm_blockscaled_few(*a, *b, *g, p, 0, ld, *d, None),
        "glu": lambda: L.fp8q_glu_blockscaled(*glu, p, 0, ld, None, 0, *d, None),
        "glu_fast": lambda: L.fp8q_glu_blockscaled_fast(*glu, p, 0, ld, None, 0, *d, None),
        "glu_q": lambda: L.fp8q_glu_blockscaled_q(*glu, 0, 1e-12, p, ld, p, ld, None, 0, *d, p, far, None),
    }[form]()
    if form == "gemm_few" and "M" in kw and "lda" not in kw:
        return  # at most 64 rows: nothing overflows
    assert rc == fq.ESHAPE, fq.lib().fp8q_last_error().decode()
    assert "4 GiB" in fq.lib().fp8q_last_error().decode()


def test_no_workspace_for_sizes_whose_span_passes_64_bits(fq):
    w = fq.fp8q_linear_blockscaled_workspace
    for fast in (0, 1):
        for codes in (0, 1):
            for M, N, K in (((1 << 57) + 1, 128, 128), (16, 1 << 57, 128), (16, 128, 1 << 62), (16, (1 << 62) + 128, 128),
                            (16, 128, (1 << 63) - 128), ((1 << 63) - 1, 128, 128), (17, 1 << 59, 128)):
                assert w(fast, codes, M, N, K) == 0, (M, N, K)

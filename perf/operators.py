"""The feed-forward operators of the library as measurable cases: plain forms
in elementary torch operations, the calls a user makes of the library, and the
values the definitions give in 64 bits.

Operators (`op` of a case):
  norm      residual addition, root-mean-square norm, 1x128 FP8 output
  norm_bwd  its gradients: of the input (and residual) and of the weight
  glu       gated projection h = silu(A Wg^T) * (A Wu^T) on block-scaled FP8
            operands; form "q" leaves h as 1x128 FP8 codes, "exact" as fp32
            and "fast" (FP8 matrix instructions) as bf16
  glu_bwd   its gradients of the input and of both weights, from dh, through
            1x128 FP8 codes along features and along tokens
  few       block-scaled product of a few rows (the down projection of single
            tokens)

FP8 outputs are returned as float8 tensors beside their fp32 scales.
"""
import math

import torch

own = False

QEPS = 1e-12    # lower clamp of a block's amax
NEPS = 1e-6     # added to the mean square of a row
MAXF = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
LIMIT_NORM = 16384 * 7168           # elements of the largest norm
LIMIT_GLU = 16384 * 18432 * 7168    # M*F*K of the largest gated projection
LIMIT_BWD = 8192 * 18432 * 7168


def listed():
    return [
        # one token of a decode step: latency
        {"name": "norm token", "op": "norm", "rows": 1, "cols": 7168, "dtype": "bf16", "res": True, "y": False, "fmt": "e4m3"},
        # the norm in front of a layer's projections, a training step's tokens
        {"name": "norm train", "op": "norm", "rows": 16384, "cols": 7168, "dtype": "bf16", "res": True, "y": False, "fmt": "e4m3"},
        # a ragged prompt in fp32 without a residual (the first layer), the normed values kept beside the codes
        {"name": "norm prompt fp32", "op": "norm", "rows": 777, "cols": 4096, "dtype": "f32", "res": False, "y": True, "fmt": "e5m2"},
        # the training step's backward
        {"name": "norm bwd train", "op": "norm_bwd", "rows": 16384, "cols": 7168, "dtype": "bf16", "res": True},
        # a small micro-batch in fp32
        {"name": "norm bwd micro", "op": "norm_bwd", "rows": 513, "cols": 4096, "dtype": "f32", "res": False},
        # one token of a decode step, codes for the down projection
        {"name": "glu token", "op": "glu", "form": "q", "M": 1, "F": 18432, "K": 7168, "save": False},
        # a ragged prompt, an output width that is no multiple of a tile
        {"name": "glu prompt", "op": "glu", "form": "exact", "M": 1023, "F": 9000, "K": 4096, "save": False},
        # the training step's forward, pre-activations kept for the backward
        {"name": "glu train", "op": "glu", "form": "fast", "M": 16384, "F": 18432, "K": 7168, "save": True},
        # the backward of a micro-batch with a ragged number of tokens
        {"name": "glu bwd micro", "op": "glu_bwd", "M": 1000, "F": 4096, "K": 4096, "fmt": "e5m2"},
        # the backward of a training step
        {"name": "glu bwd train", "op": "glu_bwd", "M": 8192, "F": 18432, "K": 7168, "fmt": "e4m3"},
        # the down projection of one token, and of a batch of decoding requests
        {"name": "down token", "op": "few", "M": 1, "N": 7168, "K": 18432, "dtype": "bf16"},
        {"name": "down batch", "op": "few", "M": 48, "N": 7168, "K": 18432, "dtype": "bf16"},
    ]


def _lu(rng, lo, hi, step=1):
    """A multiple of `step`, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    v = min(hi, max(lo, int(round(v / step)) * step))
    return v + step if v == 3072 else v


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "glu", "glu", "glu_bwd", "few"])
    if op in ("norm", "norm_bwd"):
        cols = _lu(rng, 128, 16384, 128)
        c = {"op": op, "rows": _lu(rng, 1, LIMIT_NORM // cols if cols > 7168 else 16384), "cols": cols,
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "res": rng.random() < 0.6}
        if c["dtype"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
        if op == "norm":
            c["y"] = rng.random() < 0.3
            c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"])
        return c
    if op == "few":
        return {"op": op, "M": _lu(rng, 1, 64), "N": _lu(rng, 512, 7168), "K": _lu(rng, 512, 18432, 128),
                "dtype": rng.choice(["bf16", "f32"])}
    K = _lu(rng, 512, 7168, 128)
    F = _lu(rng, 512, 18432, 128)
    if op == "glu_bwd":
        return {"op": op, "M": _lu(rng, 64, 8192), "F": F, "K": K, "fmt": rng.choice(["e4m3", "e4m3", "e5m2"])}
    form = rng.choice(["q", "exact", "fast"])
    if form != "q" and rng.random() < 0.5:
        F -= rng.randrange(1, 16) * 8 + rng.randrange(8)
    return {"op": op, "form": form, "M": _lu(rng, 1, 16384), "F": F, "K": K, "save": rng.random() < 0.5}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(std) if std != 1.0 else x


def _act(g, rows, cols, outlier=4, factor=30.0):
    """N(0,1) activations with a few outlier channels."""
    x = _normal(g, rows, cols)
    x[:, :outlier] *= factor
    return x


def _grad(g, rows, cols, lo=1e-6, hi=1e-2):
    """Random-sign gradients, log-uniform magnitudes."""
    x = torch.rand(rows, cols, generator=g, device="cuda")
    x = x.mul_(math.log(hi / lo)).add_(math.log(lo)).exp_()
    return torch.where(torch.rand(rows, cols, generator=g, device="cuda") < 0.5, -x, x)


def _blocks(x, br, fmt="e4m3"):
    """Codes (uint8) and fp32 scales of br x 128 blocks, ragged rows allowed for br = 128."""
    rows, cols = x.shape
    pad = -rows % br
    v = torch.nn.functional.pad(x, (0, 0, 0, pad)) if pad else x
    v = v.reshape((rows + pad) // br, br, cols // 128, 128)
    s = v.abs().amax(dim=(1, 3)).clamp_(min=QEPS) / MAXF[fmt]
    q = (v / s[:, None, :, None]).clamp_(-MAXF[fmt], MAXF[fmt]).to(F8[fmt]).view(torch.uint8)
    return q.reshape(rows + pad, cols)[:rows].contiguous(), s.contiguous()


def _ld(n, step):
    return -(-n // step) * step


def _weight(g, rows, cols):
    """A 0.02*N(0,1) weight as codes with 128x128 scales, made in row chunks."""
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-rows // 128), cols // 128, device="cuda")
    for r in range(0, rows, 4096):
        e = min(rows, r + 4096)
        q[r:e], s[r // 128:-(-e // 128)] = _blocks(_normal(g, e - r, cols, std=0.02), 128)
    return q, s


def _out(rows, cols, dtype, step=1):
    """An output buffer whose rows start 16-byte aligned, and its rows x cols view."""
    b = torch.empty(rows, _ld(cols, step), dtype=dtype, device="cuda")
    return b[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    st = {"case": c}
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols, dt = c["rows"], c["cols"], DT[c["dtype"]]
        st["w"] = 1.0 + _normal(g, cols, std=0.1)
        st["x"] = _act(g, rows, cols).to(dt)
        st["res"] = _normal(g, rows, cols, std=2.0 if op == "norm" else 1e-3).to(dt) if c["res"] else None
        if op == "norm":
            st["z"] = torch.empty_like(st["x"]) if c["res"] else None
            st["yout"] = torch.empty_like(st["x"]) if c["y"] else None
            st["q"] = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
            st["s"] = torch.empty(rows, cols // 128, device="cuda")
            st["rstd"] = torch.empty(rows, device="cuda")
        else:
            st["dy"] = _grad(g, rows, cols).to(dt)
            st["rstd"] = (st["x"].float().square().mean(1) + NEPS).rsqrt()
            st["dx"] = torch.empty_like(st["x"])
            st["dw"] = torch.empty(cols, device="cuda")
            # the library's workspace for the weight's gradient: 4 bytes a column for each of up to 1024 partial sums
            st["ws"] = torch.empty(1024 * cols, device="cuda")
        return st
    if op == "few":
        M, N, K = c["M"], c["N"], c["K"]
        st["A"], st["sA"] = _blocks(_act(g, M, K), 1)
        st["B"], st["sB"] = _weight(g, N, K)
        st["C"] = _out(M, N, DT[c["dtype"]], 8)
        return st
    M, F, K = c["M"], c["F"], c["K"]
    if op == "glu":
        st["A"], st["sA"] = _blocks(_act(g, M, K), 1)
        st["Wg"], st["sg"] = _weight(g, F, K)
        st["Wu"], st["su"] = _weight(g, F, K)
        st["gu"] = _out(M, 2 * F, torch.bfloat16, 8) if c["save"] else None
        if c["form"] == "q":
            st["h"] = torch.empty(M, F, dtype=torch.uint8, device="cuda")
            st["hs"] = torch.empty(M, F // 128, device="cuda")
        else:
            st["h"] = _out(M, F, torch.float32 if c["form"] == "exact" else torch.bfloat16, 8)
        return st
    # glu_bwd: what the forward left (pre-activations, the input's codes along tokens) and both weights, gate above up, stored [K, 2F]
    Mp = _ld(M, 128)
    x = torch.zeros(Mp, K, device="cuda")
    x[:M] = _act(g, M, K)
    st["Xt"], st["sXt"] = _blocks(x.t().contiguous(), 1)
    del x
    st["Wt"], st["sWt"] = _weight(g, K, 2 * F)
    st["gu"] = torch.empty(M, 2 * F, dtype=torch.bfloat16, device="cuda")
    st["dh"] = torch.empty(M, F, dtype=torch.bfloat16, device="cuda")
    for r in range(0, M, 4096):
        e = min(M, r + 4096)
        st["gu"][r:e] = _normal(g, e - r, 2 * F, std=1.7)
        st["dh"][r:e] = _grad(g, e - r, F)
    u8 = dict(dtype=torch.uint8, device="cuda")
    st["D"], st["Ds"] = torch.empty(M, 2 * F, **u8), torch.empty(M, 2 * F // 128, device="cuda")
    st["Dt"], st["Dts"] = torch.empty(2 * F, Mp, **u8), torch.empty(2 * F, Mp // 128, device="cuda")
    st["Ht"], st["Hts"] = torch.empty(F, Mp, **u8), torch.empty(F, Mp // 128, device="cuda")
    st["dX"] = torch.empty(M, K, dtype=torch.bfloat16, device="cuda")
    st["dW"] = torch.empty(2 * F, K, dtype=torch.bfloat16, device="cuda")
    return st


# ------------------------------------------------------------------ the library's calls
def _run_own(st):
    import block_scaled_precision_amax_amd as fq

    c = st["case"]
    op = c["op"]
    if op == "norm":
        rows, cols = c["rows"], c["cols"]
        f = fq.E4M3FN if c["fmt"] == "e4m3" else fq.E5M2
        fq.fp8q_rmsnorm_1x128(st["x"], cols, st["res"], cols, st["w"], rows, cols, NEPS, st["z"], cols, st["yout"], cols,
                              f, QEPS, st["q"], cols, st["s"], cols // 128, st["rstd"])
        r = {"q": st["q"].view(F8[c["fmt"]]), "s": st["s"], "rstd": st["rstd"]}
        if c["res"]:
            r["z"] = st["z"]
        if c["y"]:
            r["y"] = st["yout"]
        return r
    if op == "norm_bwd":
        rows, cols = c["rows"], c["cols"]
        fq.fp8q_rmsnorm_bwd(st["dy"], cols, st["x"], cols, st["w"], st["rstd"], st["res"], cols, rows, cols, st["dx"],
                            cols, st["dw"], st["ws"], st["ws"].numel() * 4)
        return {"dx": st["dx"], "dw": st["dw"]}
    if op == "few":
        M, N, K = c["M"], c["N"], c["K"]
        fq.fp8q_gemm_blockscaled_few(st["A"], fq.E4M3FN, K, st["sA"], K // 128, 1, st["B"], fq.E4M3FN, K, st["sB"],
                                     fq.GRAN_128x128, K // 128, 1, st["C"], st["C"].stride(0), M, N, K)
        return st["C"]
    M, F, K = c["M"], c["F"], c["K"]
    if op == "glu":
        a = (st["A"], fq.E4M3FN, K, st["sA"], K // 128, 1, st["Wg"], st["Wu"], fq.E4M3FN, K, st["sg"], st["su"], K // 128,
             1, fq.ACT_SILU)
        gu = (st["gu"], st["gu"].stride(0) if c["save"] else 0)
        if c["form"] == "q":
            fq.fp8q_glu_blockscaled_q(*a, fq.E4M3FN, QEPS, st["h"], F, st["hs"], F // 128, *gu, M, F, K)
            r = {"h": st["h"].view(torch.float8_e4m3fn), "s": st["hs"]}
        else:
            f = fq.fp8q_glu_blockscaled if c["form"] == "exact" else fq.fp8q_glu_blockscaled_fast
            f(*a, st["h"], st["h"].stride(0), *gu, M, F, K)
            r = {"h": st["h"]}
        if c["save"]:
            r["gu"] = st["gu"]
        return r
    f = fq.E4M3FN if c["fmt"] == "e4m3" else fq.E5M2
    Mp = _ld(M, 128)
    fq.fp8q_glu_bwd_q(st["dh"], F, st["gu"], 2 * F, fq.ACT_SILU, f, QEPS, st["D"], 2 * F, st["Ds"], 2 * F // 128,
                      st["Dt"], Mp, st["Dts"], Mp // 128, fq.E4M3FN, st["Ht"], Mp, st["Hts"], Mp // 128, M, F)
    fq.fp8q_gemm_blockscaled_fast(st["D"], f, 2 * F, st["Ds"], 2 * F // 128, 1, st["Wt"], fq.E4M3FN, 2 * F, st["sWt"],
                                  fq.GRAN_128x128, 2 * F // 128, 1, st["dX"], K, M, K, 2 * F)
    fq.fp8q_gemm_blockscaled_fast(st["Dt"], f, Mp, st["Dts"], Mp // 128, 1, st["Xt"], fq.E4M3FN, Mp, st["sXt"],
                                  fq.GRAN_1x128, Mp // 128, 1, st["dW"], K, 2 * F, K, Mp)
    return {"dX": st["dX"], "dW": st["dW"], "ht": st["Ht"].view(torch.float8_e4m3fn), "hts": st["Hts"]}


# ------------------------------------------------------------------ the plain forms
def _deq(q, s, br, fmt="e4m3"):
    """Codes with br x 128 block scales as fp32 values."""
    v = q.view(F8[fmt]).float()
    full = s.repeat_interleave(128, dim=1)
    if br > 1:
        full = full.repeat_interleave(br, dim=0)[:q.shape[0]]
    return v * full


def _silu(x):
    return x / (1.0 + torch.exp(-x))


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op = c["op"]
    if op == "norm":
        dt = st["x"].dtype
        v = st["x"].float()
        if c["res"]:
            v = v + st["res"].float()
        rstd = torch.rsqrt(v.square().mean(dim=1) + NEPS)
        y = v * rstd[:, None] * st["w"]
        q, s = _blocks(y, 1, c["fmt"])
        r = {"q": q.view(F8[c["fmt"]]), "s": s, "rstd": rstd}
        if c["res"]:
            r["z"] = v.to(dt)
        if c["y"]:
            r["y"] = y.to(dt)
        return r
    if op == "norm_bwd":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = st["x"].float() * rstd
        t = dy * st["w"]
        dx = rstd * (t - xh * (t * xh).mean(dim=1, keepdim=True))
        if c["res"]:
            dx = dx + st["res"].float()
        return {"dx": dx.to(st["x"].dtype), "dw": (dy * xh).sum(dim=0)}
    if op == "few":
        return (_deq(st["A"], st["sA"], 1) @ _deq(st["B"], st["sB"], 128).t()).to(st["C"].dtype)
    if op == "glu":
        a = _deq(st["A"], st["sA"], 1)
        g = a @ _deq(st["Wg"], st["sg"], 128).t()
        u = a @ _deq(st["Wu"], st["su"], 128).t()
        h = _silu(g) * u
        if c["form"] == "q":
            q, s = _blocks(h, 1)
            r = {"h": q.view(torch.float8_e4m3fn), "s": s}
        else:
            r = {"h": h.to(st["h"].dtype)}
        if c["save"]:
            r["gu"] = torch.cat([g, u], dim=1).to(torch.bfloat16)
        return r
    M, F = c["M"], c["F"]
    g, u = st["gu"][:, :F].float(), st["gu"][:, F:].float()
    dh = st["dh"].float()
    sg = 1.0 / (1.0 + torch.exp(-g))
    d = torch.cat([dh * u * sg * (1.0 + g * (1.0 - sg)), dh * g * sg], dim=1)
    h = torch.nn.functional.pad((g * sg * u).t(), (0, -M % 128))
    del g, u, dh, sg
    hq, hs = _blocks(h.contiguous(), 1)
    del h
    dq = _deq(*_blocks(d, 1, c["fmt"]), 1, c["fmt"])
    dX = (dq @ _deq(st["Wt"], st["sWt"], 128).t()).to(torch.bfloat16)
    del dq
    dt = torch.nn.functional.pad(d.t(), (0, -M % 128))
    del d
    dtq = _deq(*_blocks(dt.contiguous(), 1, c["fmt"]), 1, c["fmt"])
    del dt
    dW = (dtq @ _deq(st["Xt"], st["sXt"], 1).t()).to(torch.bfloat16)
    return {"dX": dX, "dW": dW, "ht": hq.view(torch.float8_e4m3fn), "hts": hs}


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    op = c["op"]
    if op in ("norm", "norm_bwd"):
        rows, cols = c["rows"], c["cols"]
        n, es = rows * cols, 2 if c["dtype"] == "bf16" else 4
        if op == "norm":
            b = n * es * (1 + 2 * c["res"] + c["y"]) + n + 4 * n // 128 + 4 * rows + 4 * cols
            return {"bytes": b, "flops": 8 * n}
        return {"bytes": n * es * (3 + c["res"]) + 4 * rows + 8 * cols, "flops": 12 * n}
    if op == "few":
        M, N, K = c["M"], c["N"], c["K"]
        nb = -(-N // 128) * (K // 128)
        return {"bytes": (M + N) * K + 4 * (M * (K // 128) + nb) + M * N * (2 if c["dtype"] == "bf16" else 4),
                "flops": 2 * M * N * K}
    M, F, K = c["M"], c["F"], c["K"]
    if op == "glu":
        out = {"q": M * F + 4 * M * (F // 128), "exact": 4 * M * F, "fast": 2 * M * F}[c["form"]]
        b = M * K + 2 * F * K + 4 * (M + 2 * -(-F // 128)) * (K // 128) + out + (4 * M * F if c["save"] else 0)
        return {"bytes": b, "flops": 4 * M * F * K}
    Mp = _ld(M, 128)
    b = 6 * M * F + 2 * F * K + K * Mp + 4 * (2 * F // 128 * -(-K // 128) + K * Mp // 128)
    b += 2 * M * K + 4 * F * K + F * Mp + 4 * F * Mp // 128
    return {"bytes": b, "flops": 8 * M * F * K}


# ------------------------------------------------------------------ the definitions in 64 bits
def _table(fmt):
    """Value of each code, from its sign, exponent and mantissa fields."""
    eb, mb, bias = (4, 3, 7) if fmt == "e4m3" else (5, 2, 15)
    v = []
    for b in range(256):
        e, m = (b >> mb) & ((1 << eb) - 1), b & ((1 << mb) - 1)
        x = math.ldexp(m, 1 - bias - mb) if e == 0 else math.ldexp((1 << mb) + m, e - bias - mb)
        v.append(-x if b >> 7 else x)
    return torch.tensor(v, dtype=torch.float64, device="cuda")


def _values(q, s, br, fmt="e4m3"):
    """Codes and scales as float64 values, by table."""
    t = _table(fmt)[q.int()]
    for b in range(0, q.shape[0], br):
        t[b:b + br].view(-1, q.shape[1] // 128, 128).mul_(s[b // br].double()[None, :, None]) if br > 1 else None
    return t if br > 1 else t.view(q.shape[0], -1, 128).mul_(s.double()[:, :, None]).view(q.shape[0], -1)


def _quotient(v, fmt):
    """v / s and s of 1x128 blocks: the value a code stands for before its rounding."""
    b = v.view(v.shape[0], -1, 128)
    s = torch.clamp(b.abs().amax(2), min=QEPS) / MAXF[fmt]
    return (b / s[:, :, None]).view_as(v), s


def _on_grid(q, fmt):
    """Rounds to the nearest value of the format, ties to even."""
    mb, emin = (3, -6) if fmt == "e4m3" else (2, -14)
    _, e = torch.frexp(q)
    step = torch.ldexp(torch.ones_like(q), torch.clamp(e - 1, min=emin) - mb)
    return torch.round(q / step) * step


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "norm":
        rows = range(0, c["rows"], 2048)
        parts = []
        for r in rows:
            v = st["x"][r:r + 2048].double()
            if c["res"]:
                v = v + st["res"][r:r + 2048].double()
            rs = 1.0 / torch.sqrt((v * v).sum(1) / c["cols"] + NEPS)
            y = v * (rs[:, None] * st["w"].double())
            # an e5m2 code is up to an eighth of its value off: nothing to hold a code to
            q, s = _quotient(y, c["fmt"])
            parts.append((q if c["fmt"] == "e4m3" else None, s, rs, v, y))
        cat = lambda k: torch.cat([p[k] for p in parts])  # noqa: E731
        r = {"q": cat(0) if c["fmt"] == "e4m3" else None, "s": cat(1), "rstd": cat(2)}
        if c["res"]:
            r["z"] = cat(3)
        if c["y"]:
            r["y"] = cat(4)
        return r
    if op == "norm_bwd":
        dx, dw = [], torch.zeros(c["cols"], dtype=torch.float64, device="cuda")
        w = st["w"].double()
        for r in range(0, c["rows"], 2048):
            e = slice(r, r + 2048)
            x, dy, rs = st["x"][e].double(), st["dy"][e].double(), st["rstd"][e].double()[:, None]
            dot = ((dy * w) * x).sum(1, keepdim=True) / c["cols"]
            d = rs * (dy * w) - x * (rs ** 3 * dot)
            dx.append(d + st["res"][e].double() if c["res"] else d)
            dw += (dy * (x * rs)).sum(0)
        return {"dx": torch.cat(dx), "dw": dw}
    if op == "few":
        return torch.matmul(_values(st["A"], st["sA"], 1), _values(st["B"], st["sB"], 128).t())
    if op == "glu":
        wg, wu = _values(st["Wg"], st["sg"], 128).t(), _values(st["Wu"], st["su"], 128).t()
        hs, gus = [], []
        for r in range(0, c["M"], 2048):
            a = _values(st["A"][r:r + 2048], st["sA"][r:r + 2048], 1)
            g, u = torch.matmul(a, wg), torch.matmul(a, wu)
            if c["save"]:
                gus.append(torch.cat([g, u], 1).float())
            hs.append(g * torch.sigmoid(g) * u)
        h = torch.cat(hs)
        r = dict(zip("hs", _quotient(h, "e4m3"))) if c["form"] == "q" else {"h": h}
        if c["save"]:
            r["gu"] = torch.cat(gus)
        return r
    M, F, fmt = c["M"], c["F"], c["fmt"]
    Mp = _ld(M, 128)
    wt = _values(st["Wt"], st["sWt"], 128).t()
    dt = torch.zeros(2 * F, Mp, dtype=torch.float64, device="cuda")
    ht = torch.zeros(F, Mp, dtype=torch.float64, device="cuda")
    dX = []
    for r in range(0, M, 2048):
        e = slice(r, min(M, r + 2048))
        g, u, dh = st["gu"][e, :F].double(), st["gu"][e, F:].double(), st["dh"][e].double()
        p = torch.sigmoid(g)
        d = torch.cat([dh * u * (p + g * p * (1 - p)), dh * (g * p)], 1)
        ht[:, e] = (g * p * u).t()
        dt[:, e] = d.t()
        q, s = _quotient(d, fmt)
        dX.append(torch.matmul(_on_grid(q, fmt).view(q.shape[0], -1, 128).mul(s[:, :, None]).view_as(q), wt))
    del wt, q, s, d
    hq, hs = _quotient(ht, "e4m3")
    del ht
    xt = _values(st["Xt"], st["sXt"], 1).t()
    dW = []
    for r in range(0, 2 * F, 4096):
        q, s = _quotient(dt[r:r + 4096], fmt)
        dW.append(torch.matmul(_on_grid(q, fmt).view(q.shape[0], -1, 128).mul(s[:, :, None]).view_as(q), xt))
    return {"dX": torch.cat(dX), "dW": torch.cat(dW), "ht": hq, "hts": hs}

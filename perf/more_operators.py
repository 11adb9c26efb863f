"""Layer norm and the linear layer with its epilogue, forward and backward, as
measurable cases: plain forms in elementary torch operations, the calls a user
makes of the library, and the values the definitions give in 64 bits.

Operators (`op` of a case):
  lnorm       residual addition, layer norm, 1x128 FP8 output
  lnorm_bwd   its gradients: of the input (and residual), the weight and the bias
  linear      act(A W^T + bias) + residual on block-scaled FP8 operands; form
              "exact" and "fast" (FP8 matrix instructions) leave fp32 or bf16,
              "q" and "q_fast" 1x128 FP8 codes for the next product
  linear_bwd  the gradient at the linear layer's pre-activations as FP8 codes
              along features and along tokens, the bias's gradient, and the
              activation's output again as codes along tokens

FP8 outputs are returned as float8 tensors beside their fp32 scales.
"""
import math

import torch

own = False

QEPS = 1e-12    # lower clamp of a block's amax
NEPS = 1e-5     # added to a row's variance
MAXF = {"e4m3": 448.0, "e5m2": 57344.0}
F8 = {"e4m3": torch.float8_e4m3fn, "e5m2": torch.float8_e5m2}
DT = {"bf16": torch.bfloat16, "f32": torch.float32}
ACTS = ["none", "relu", "silu", "gelu", "gelu_erf"]
LIMIT_NORM = 16384 * 7168               # elements of the largest norm
LIMIT_LINEAR = 16384 * 18432 * 7168     # M*N*K of the largest linear layer
LIMIT_BWD = 8192 * 18432                # elements of the largest gradient


def listed():
    return [
        # one token of a decode step: latency
        {"name": "lnorm token", "op": "lnorm", "rows": 1, "cols": 7168, "dtype": "bf16", "wdt": "f32", "res": True, "y": False,
         "fmt": "e4m3"},
        # the norm in front of a layer's projections, a training step's tokens
        {"name": "lnorm train", "op": "lnorm", "rows": 16384, "cols": 7168, "dtype": "bf16", "wdt": "f32", "res": True,
         "y": False, "fmt": "e4m3"},
        # the last norm of a stack: a ragged prompt in fp32, no residual, normed values alone, a width of no whole block
        {"name": "lnorm last fp32", "op": "lnorm", "rows": 1023, "cols": 1608, "dtype": "f32", "wdt": "bf16", "res": False,
         "y": True, "fmt": None},
        # the training step's backward
        {"name": "lnorm bwd train", "op": "lnorm_bwd", "rows": 16384, "cols": 7168, "dtype": "bf16", "wdt": "f32", "res": True},
        # a small ragged micro-batch in fp32
        {"name": "lnorm bwd micro", "op": "lnorm_bwd", "rows": 513, "cols": 4096, "dtype": "f32", "wdt": "f32", "res": False},
        # the up projection of one token, codes for the down projection
        {"name": "up token", "op": "linear", "form": "q", "M": 1, "N": 18432, "K": 7168, "act": "gelu", "bdt": "f32",
         "res": False, "save": False, "dtype": None},
        # the down projection of a batch of decoding requests, added to the residual stream
        {"name": "down batch", "op": "linear", "form": "exact", "M": 48, "N": 7168, "K": 18432, "act": "none", "bdt": "bf16",
         "res": True, "save": False, "dtype": "bf16"},
        # a ragged prompt, an output width that is no multiple of a tile, fp32 for what follows
        {"name": "prompt", "op": "linear", "form": "exact", "M": 1023, "N": 9000, "K": 4096, "act": "gelu_erf", "bdt": "f32",
         "res": False, "save": False, "dtype": "f32"},
        # the training step's up projection: codes for the down projection, pre-activations kept for the backward
        {"name": "up train", "op": "linear", "form": "q_fast", "M": 16384, "N": 18432, "K": 7168, "act": "gelu_erf",
         "bdt": "f32", "res": False, "save": True, "dtype": None},
        # the training step's down projection, added to the residual stream
        {"name": "down train", "op": "linear", "form": "fast", "M": 8192, "N": 7168, "K": 18432, "act": "none", "bdt": "f32",
         "res": True, "save": False, "dtype": "bf16"},
        # the backward of a micro-batch with a ragged number of tokens, fp32 gradients
        {"name": "linear bwd micro", "op": "linear_bwd", "M": 1000, "N": 4096, "act": "relu", "dtype": "f32", "fmt": "e5m2",
         "ht": False},
        # the backward of a training step
        {"name": "linear bwd train", "op": "linear_bwd", "M": 8192, "N": 18432, "act": "gelu", "dtype": "bf16", "fmt": "e4m3",
         "ht": True},
    ]


def _lu(rng, lo, hi, step=1):
    """A multiple of `step`, spread over the logarithm of [lo, hi]."""
    v = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return min(hi // step * step, max(lo, int(round(v / step)) * step))


def draw(rng):
    op = rng.choice(["lnorm", "lnorm", "lnorm_bwd", "linear", "linear", "linear", "linear_bwd"])
    if op in ("lnorm", "lnorm_bwd"):
        codes = op == "lnorm" and rng.random() < 0.7
        cols = _lu(rng, 128, 16384, 128 if codes else 8)
        c = {"op": op, "rows": _lu(rng, 1, min(16384, LIMIT_NORM // cols)), "cols": cols,
             "dtype": rng.choice(["bf16", "bf16", "f32"]), "wdt": rng.choice(["f32", "bf16"]), "res": rng.random() < 0.6}
        if c["dtype"] == "f32":
            c["rows"] = max(1, c["rows"] // 2)
        if op == "lnorm":
            c["fmt"] = rng.choice(["e4m3", "e4m3", "e5m2"]) if codes else None
            c["y"] = not codes or rng.random() < 0.3
        return c
    act = rng.choice(ACTS)
    if op == "linear_bwd":
        N = _lu(rng, 128, 18432, 128)
        return {"op": op, "M": _lu(rng, 1, min(16384, LIMIT_BWD // N)), "N": N, "act": act,
                "dtype": rng.choice(["bf16", "bf16", "f32"]), "fmt": rng.choice(["e4m3", "e5m2"]),
                "ht": act != "none" and rng.random() < 0.6}
    form = rng.choice(["exact", "fast", "q", "q_fast"])
    K, N = _lu(rng, 512, 18432, 128), _lu(rng, 512, 18432, 128)
    codes = form.startswith("q")
    if not codes and rng.random() < 0.5:
        N -= rng.randrange(1, 128)
    # the exact products take twice as long
    limit = (LIMIT_LINEAR if form.endswith("fast") else LIMIT_LINEAR // 2) // (N * K)
    return {"op": op, "form": form, "M": _lu(rng, 1, min(16384, limit)), "N": N, "K": K, "act": act,
            "bdt": rng.choice(["f32", "bf16", None]), "res": not codes and rng.random() < 0.5, "save": rng.random() < 0.4,
            "dtype": None if codes else rng.choice(["bf16", "f32"])}


# ------------------------------------------------------------------ inputs
def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _normal(g, *shape, std=1.0):
    x = torch.randn(*shape, generator=g, device="cuda")
    return x.mul_(std) if std != 1.0 else x


def _acts(g, rows, cols, outlier=4, factor=30.0):
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
    """A weight of std cols^-1/2 as codes with 128x128 scales, made in row chunks."""
    q = torch.empty(rows, cols, dtype=torch.uint8, device="cuda")
    s = torch.empty(-(-rows // 128), cols // 128, device="cuda")
    for r in range(0, rows, 4096):
        e = min(rows, r + 4096)
        q[r:e], s[r // 128:-(-e // 128)] = _blocks(_normal(g, e - r, cols, std=cols ** -0.5), 128)
    return q, s


def _out(rows, cols, dtype, step=8):
    """An output buffer whose rows start 16-byte aligned, and its rows x cols view."""
    return torch.empty(rows, _ld(cols, step), dtype=dtype, device="cuda")[:, :cols]


def prepare(case, seed):
    g = _gen(seed)
    c = dict(case)
    st = {"case": c}
    op = c["op"]
    u8 = dict(dtype=torch.uint8, device="cuda")
    if op in ("lnorm", "lnorm_bwd"):
        rows, cols, dt = c["rows"], c["cols"], DT[c["dtype"]]
        st["w"] = (1.0 + _normal(g, cols, std=0.1)).to(DT[c["wdt"]])
        st["b"] = _normal(g, cols, std=0.1).to(DT[c["wdt"]])
        # rows away from zero: the mean is what the norm takes off
        st["x"] = (_acts(g, rows, cols) + _normal(g, rows, 1)).to(dt)
        st["res"] = _normal(g, rows, cols, std=2.0 if op == "lnorm" else 1e-3).to(dt) if c["res"] else None
        if op == "lnorm":
            st["z"] = torch.empty_like(st["x"]) if c["res"] else None
            st["yout"] = torch.empty_like(st["x"]) if c["y"] else None
            st["q"] = torch.empty(rows, cols, **u8) if c["fmt"] else None
            st["s"] = torch.empty(rows, cols // 128, device="cuda") if c["fmt"] else None
            st["mean"], st["rstd"] = torch.empty(rows, device="cuda"), torch.empty(rows, device="cuda")
        else:
            st["dy"] = _grad(g, rows, cols).to(dt)
            v = st["x"].float()
            st["mean"] = v.mean(1)
            st["rstd"] = ((v - st["mean"][:, None]).square().mean(1) + NEPS).rsqrt()
            st["dx"] = torch.empty_like(st["x"])
            st["dw"], st["db"] = torch.empty(cols, device="cuda"), torch.empty(cols, device="cuda")
            # the library's workspace for the two sums over rows: at most 4096 bytes a column
            st["ws"] = torch.empty(1024 * cols, device="cuda")
        return st
    M, N = c["M"], c["N"]
    if op == "linear":
        K = c["K"]
        st["A"], st["sA"] = _blocks(_acts(g, M, K), 1)
        st["W"], st["sW"] = _weight(g, N, K)
        st["bias"] = _normal(g, N, std=0.5).to(DT[c["bdt"]]) if c["bdt"] else None
        st["pre"] = _out(M, N, torch.bfloat16) if c["save"] else None
        st["res"] = None
        if c["form"].startswith("q"):
            st["h"], st["hs"] = torch.empty(M, N, **u8), torch.empty(M, N // 128, device="cuda")
        else:
            st["h"] = _out(M, N, DT[c["dtype"]])
            if c["res"]:
                st["res"] = _out(M, N, DT[c["dtype"]])
                st["res"].copy_(_normal(g, M, N, std=2.0))
        return st
    Mp = _ld(M, 128)
    st["dh"] = torch.empty(M, N, dtype=DT[c["dtype"]], device="cuda")
    st["pre"] = torch.empty(M, N, dtype=torch.bfloat16, device="cuda") if c["act"] != "none" else None
    for r in range(0, M, 4096):
        e = min(M, r + 4096)
        st["dh"][r:e] = _grad(g, e - r, N)
        if st["pre"] is not None:
            st["pre"][r:e] = _normal(g, e - r, N, std=1.7)
    st["D"], st["Ds"] = torch.empty(M, N, **u8), torch.empty(M, N // 128, device="cuda")
    st["Dt"], st["Dts"] = torch.empty(N, Mp, **u8), torch.empty(N, Mp // 128, device="cuda")
    st["Ht"] = torch.empty(N, Mp, **u8) if c["ht"] else None
    st["Hts"] = torch.empty(N, Mp // 128, device="cuda") if c["ht"] else None
    st["db"] = torch.empty(N, device="cuda")
    # the library's workspace for the bias's gradient: a row of sums for each 128 tokens
    st["ws"] = torch.empty(Mp // 128 * N, device="cuda")
    return st


# ------------------------------------------------------------------ the library's calls
def _run_own(st):
    import block_scaled_precision_amax_amd as fq

    c = st["case"]
    op = c["op"]
    fmt = {"e4m3": fq.E4M3FN, "e5m2": fq.E5M2, None: fq.E4M3FN}
    if op == "lnorm":
        rows, cols = c["rows"], c["cols"]
        fq.fp8q_layernorm_1x128(st["x"], cols, st["res"], cols, st["w"], st["b"], rows, cols, NEPS, st["z"], cols,
                                st["yout"], cols, fmt[c["fmt"]], QEPS, st["q"], cols, st["s"], cols // 128, st["mean"],
                                st["rstd"])
        r = {"mean": st["mean"], "rstd": st["rstd"]}
        if c["fmt"]:
            r["q"], r["s"] = st["q"].view(F8[c["fmt"]]), st["s"]
        if c["res"]:
            r["z"] = st["z"]
        if c["y"]:
            r["y"] = st["yout"]
        return r
    if op == "lnorm_bwd":
        rows, cols = c["rows"], c["cols"]
        fq.fp8q_layernorm_bwd(st["dy"], cols, st["x"], cols, st["w"], st["mean"], st["rstd"], st["res"], cols, rows, cols,
                              st["dx"], cols, st["dw"], st["db"], st["ws"], st["ws"].numel() * 4)
        return {"dx": st["dx"], "dw": st["dw"], "db": st["db"]}
    act = {"none": fq.ACT_NONE, "relu": fq.ACT_RELU, "silu": fq.ACT_SILU, "gelu": fq.ACT_GELU,
           "gelu_erf": fq.ACT_GELU_ERF}[c["act"]]
    M, N = c["M"], c["N"]
    if op == "linear":
        # FP8 matrix instructions serve bf16 outputs: their sums drop products 2^-14 below their neighbours, which a value
        # held in fp32 (a block's scale too) shows, so those come from the exact product
        K, fast = c["K"], c["form"] == "fast" and c["dtype"] == "bf16"
        a = (st["A"], fq.E4M3FN, K, st["sA"], K // 128, 1, st["W"], fq.E4M3FN, K, st["sW"], K // 128, 1, st["bias"], act)
        pre = (st["pre"], st["pre"].stride(0) if c["save"] else 0)
        if c["form"].startswith("q"):
            fq.fp8q_linear_blockscaled_q(*a, fq.E4M3FN, QEPS, st["h"], N, st["hs"], N // 128, *pre, M, N, K)
            r = {"h": st["h"].view(F8["e4m3"]), "s": st["hs"]}
        else:
            f = fq.fp8q_linear_blockscaled_fast if fast else fq.fp8q_linear_blockscaled
            ld = st["h"].stride(0)
            f(*a, st["res"], ld, st["h"], ld, *pre, M, N, K)
            r = {"h": st["h"]}
        if c["save"]:
            r["pre"] = st["pre"]
        return r
    Mp = _ld(M, 128)
    fq.fp8q_linear_bwd_q(st["dh"], N, st["pre"], N, act, fmt[c["fmt"]], QEPS, st["D"], N, st["Ds"], N // 128, st["Dt"], Mp,
                         st["Dts"], Mp // 128, fq.E4M3FN, st["Ht"], Mp, st["Hts"], Mp // 128, st["db"], M, N, st["ws"],
                         st["ws"].numel() * 4)
    r = {"d": st["D"].view(F8[c["fmt"]]), "ds": st["Ds"], "dt": st["Dt"].view(F8[c["fmt"]]), "dts": st["Dts"],
         "db": st["db"]}
    if c["ht"]:
        r["ht"], r["hts"] = st["Ht"].view(F8["e4m3"]), st["Hts"]
    return r


# ------------------------------------------------------------------ the plain forms
def _deq(q, s, br):
    """E4M3 codes with br x 128 block scales as fp32 values."""
    v = q.view(F8["e4m3"]).float()
    full = s.repeat_interleave(128, dim=1)
    if br > 1:
        full = full.repeat_interleave(br, dim=0)[:q.shape[0]]
    return v * full


C_TANH, A_TANH = math.sqrt(2 / math.pi), 0.044715


def _act(x, act):
    if act == "none":
        return x
    if act == "relu":
        return torch.where(x > 0, x, torch.zeros_like(x))
    if act == "silu":
        return x / (1.0 + torch.exp(-x))
    if act == "gelu":
        return x / (1.0 + torch.exp(-2.0 * C_TANH * (x + A_TANH * x * x * x)))
    return 0.5 * x * torch.erfc(x * -math.sqrt(0.5))


def _act_grad(x, act):
    if act == "none":
        return torch.ones_like(x)
    if act == "relu":
        return (x > 0).to(x.dtype)
    if act == "silu":
        p = 1.0 / (1.0 + torch.exp(-x))
        return p * (1.0 + x * (1.0 - p))
    if act == "gelu":
        p = 1.0 / (1.0 + torch.exp(-2.0 * C_TANH * (x + A_TANH * x * x * x)))
        return p + x * 2.0 * p * (1.0 - p) * C_TANH * (1.0 + 3.0 * A_TANH * x * x)
    return 0.5 * torch.erfc(x * -math.sqrt(0.5)) + x * torch.exp(-0.5 * x * x) * math.sqrt(0.5 / math.pi)


def run(st):
    if own:
        return _run_own(st)
    c = st["case"]
    op = c["op"]
    if op == "lnorm":
        dt = st["x"].dtype
        v = st["x"].float()
        if c["res"]:
            v = v + st["res"].float()
        mean = v.mean(dim=1)
        d = v - mean[:, None]
        rstd = torch.rsqrt(d.square().mean(dim=1) + NEPS)
        y = d * rstd[:, None] * st["w"].float() + st["b"].float()
        r = {"mean": mean, "rstd": rstd}
        if c["fmt"]:
            q, r["s"] = _blocks(y, 1, c["fmt"])
            r["q"] = q.view(F8[c["fmt"]])
        if c["res"]:
            r["z"] = v.to(dt)
        if c["y"]:
            r["y"] = y.to(dt)
        return r
    if op == "lnorm_bwd":
        dy, rstd = st["dy"].float(), st["rstd"][:, None]
        xh = (st["x"].float() - st["mean"][:, None]) * rstd
        t = dy * st["w"].float()
        dx = rstd * (t - t.mean(dim=1, keepdim=True) - xh * (t * xh).mean(dim=1, keepdim=True))
        if c["res"]:
            dx = dx + st["res"].float()
        return {"dx": dx.to(st["x"].dtype), "dw": (dy * xh).sum(dim=0), "db": dy.sum(dim=0)}
    if op == "linear":
        v = _deq(st["A"], st["sA"], 1) @ _deq(st["W"], st["sW"], 128).t()
        if c["bdt"]:
            v = v + st["bias"].float()
        h = _act(v, c["act"])
        if c["form"].startswith("q"):
            q, s = _blocks(h, 1)
            r = {"h": q.view(F8["e4m3"]), "s": s}
        else:
            if c["res"]:
                h = h + st["res"].float()
            r = {"h": h.to(DT[c["dtype"]])}
        if c["save"]:
            r["pre"] = v.to(torch.bfloat16)
        return r
    M = c["M"]
    d = st["dh"].float()
    if c["act"] != "none":
        d = d * _act_grad(st["pre"].float(), c["act"])
    q, s = _blocks(d, 1, c["fmt"])
    r = {"d": q.view(F8[c["fmt"]]), "ds": s}
    tq, ts = _blocks(torch.nn.functional.pad(d.t(), (0, -M % 128)).contiguous(), 1, c["fmt"])
    r["dt"], r["dts"], r["db"] = tq.view(F8[c["fmt"]]), ts, d.sum(dim=0)
    if c["ht"]:
        h = _act(st["pre"].float(), c["act"])
        hq, r["hts"] = _blocks(torch.nn.functional.pad(h.t(), (0, -M % 128)).contiguous(), 1)
        r["ht"] = hq.view(F8["e4m3"])
    return r


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    c = case
    op = c["op"]
    if op in ("lnorm", "lnorm_bwd"):
        rows, cols = c["rows"], c["cols"]
        n, es, ws = rows * cols, 2 if c["dtype"] == "bf16" else 4, 2 if c["wdt"] == "bf16" else 4
        if op == "lnorm":
            b = n * es * (1 + 2 * c["res"] + c["y"]) + (n + 4 * n // 128 if c["fmt"] else 0) + 8 * rows + 2 * ws * cols
            return {"bytes": b, "flops": 10 * n}
        return {"bytes": n * es * (3 + c["res"]) + 8 * rows + (8 + ws) * cols, "flops": 15 * n}
    M, N = c["M"], c["N"]
    if op == "linear":
        K = c["K"]
        es = {"bf16": 2, "f32": 4}.get(c["dtype"], 1)
        b = (M + N) * K + 4 * (M + -(-N // 128)) * (K // 128) + N * {"bf16": 2, "f32": 4, None: 0}[c["bdt"]]
        b += M * N * (es * (1 + c["res"]) + 2 * c["save"]) + (0 if c["dtype"] else 4 * M * (N // 128))
        return {"bytes": b, "flops": 2 * M * N * K}
    Mp, n = _ld(M, 128), M * N
    b = n * ((2 if c["dtype"] == "bf16" else 4) + 2 * (c["act"] != "none")) + n + 4 * n // 128 + 4 * N
    b += (1 + c["ht"]) * (N * Mp + 4 * N * Mp // 128)
    return {"bytes": b, "flops": 20 * n}


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


def _values(q, s, br):
    """E4M3 codes and scales as float64 values, by table."""
    t = _table("e4m3")[q.int()].view(q.shape[0], -1, 128)
    for b in range(0, q.shape[0], br) if br > 1 else ():
        t[b:b + br].mul_(s[b // br].double()[None, :, None])
    return (t if br > 1 else t.mul_(s.double()[:, :, None])).view(q.shape)


def _quotient(v, fmt):
    """v / s and s of 1x128 blocks: the value a code stands for before its rounding.  An e5m2 code is up to an eighth of
    its value off: nothing to hold a code to."""
    b = v.reshape(v.shape[0], -1, 128)
    s = torch.clamp(b.abs().amax(2), min=QEPS) / MAXF[fmt]
    return ((b / s[:, :, None]).view(v.shape) if fmt == "e4m3" else None), s


def _exact_act(x, act):
    """The activation and its derivative."""
    if act == "none":
        return x, torch.ones_like(x)
    if act == "relu":
        return torch.clamp(x, min=0), torch.sign(torch.clamp(x, min=0))
    if act == "gelu_erf":
        # the normal distribution function (by erfc: 1 + erf cancels in the lower tail) and its density
        p = torch.erfc(-x / math.sqrt(2)) / 2
        return x * p, p + x * torch.exp(-x * x / 2) / math.sqrt(2 * math.pi)
    if act == "silu":
        p, dk = torch.sigmoid(x), 1.0
    else:
        p, dk = torch.sigmoid(2 * C_TANH * (x + A_TANH * x ** 3)), 2 * C_TANH * (1 + 3 * A_TANH * x ** 2)
    return x * p, p + x * (p * (1 - p)) * dk


def _cat(parts):
    return None if parts[0] is None else torch.cat(parts)


def exact(case, seed):
    c, st = case, prepare(case, seed)
    op = c["op"]
    if op == "lnorm":
        parts = []
        for r in range(0, c["rows"], 2048):
            v = st["x"][r:r + 2048].double()
            if c["res"]:
                v = v + st["res"][r:r + 2048].double()
            m = v.sum(1) / c["cols"]
            var = torch.var(v, 1, correction=0)
            rs = 1.0 / torch.sqrt(var + NEPS)
            y = torch.addcmul(st["b"].double(), v - m[:, None], rs[:, None] * st["w"].double())
            parts.append((m, rs, v, y, *(_quotient(y, c["fmt"]) if c["fmt"] else (None, None))))
        m, rs, v, y, q, s = (_cat(list(p)) for p in zip(*parts))
        r = {"mean": m, "rstd": rs}
        if c["fmt"]:
            r["q"], r["s"] = q, s
        if c["res"]:
            r["z"] = v
        if c["y"]:
            r["y"] = y
        return r
    if op == "lnorm_bwd":
        dx = []
        dw, db = (torch.zeros(c["cols"], dtype=torch.float64, device="cuda") for _ in range(2))
        w = st["w"].double()
        for r in range(0, c["rows"], 2048):
            e = slice(r, r + 2048)
            rs = st["rstd"][e].double()[:, None]
            x, dy = st["x"][e].double() - st["mean"][e].double()[:, None], st["dy"][e].double()
            a = (dy * w).sum(1, keepdim=True) / c["cols"]
            k = ((dy * w) * x).sum(1, keepdim=True) / c["cols"]
            d = rs * (dy * w - a) - x * (rs ** 3 * k)
            dx.append(d + st["res"][e].double() if c["res"] else d)
            dw += (dy * (x * rs)).sum(0)
            db += dy.sum(0)
        return {"dx": torch.cat(dx), "dw": dw, "db": db}
    if op == "linear":
        w = _values(st["W"], st["sW"], 128).t()
        out = []
        for r in range(0, c["M"], 2048):
            v = torch.matmul(_values(st["A"][r:r + 2048], st["sA"][r:r + 2048], 1), w)
            if c["bdt"]:
                v += st["bias"].double()
            h = _exact_act(v, c["act"])[0]
            if c["form"].startswith("q"):
                part = list(_quotient(h, "e4m3"))
            else:
                part = [h + st["res"][r:r + 2048].double() if c["res"] else h]
            out.append(part + [v.float()] if c["save"] else part)
        names = (["h", "s"] if c["form"].startswith("q") else ["h"]) + (["pre"] if c["save"] else [])
        return {n: torch.cat(p) for n, p in zip(names, map(list, zip(*out)))}
    M, N, fmt = c["M"], c["N"], c["fmt"]
    cols = {k: [] for k in ("d", "ds", "dt", "dts", "ht", "hts", "db")}
    for f in range(0, N, 2048):  # by features: both kinds of block lie inside
        d = st["dh"][:, f:f + 2048].double()
        h, da = _exact_act(st["pre"][:, f:f + 2048].double(), c["act"]) if st["pre"] is not None else (None, 1.0)
        d = d * da
        for k, v in zip(("d", "ds"), _quotient(d, fmt)):
            cols[k].append(v)
        cols["db"].append(d.sum(0))
        for names, t, form in ((("dt", "dts"), d, fmt), (("ht", "hts"), h if c["ht"] else None, "e4m3")):
            if t is not None:
                t = torch.cat([t, t.new_zeros(-M % 128, t.shape[1])]).t().contiguous()
                for k, v in zip(names, _quotient(t, form)):
                    cols[k].append(v)
    r = {k: None if v[0] is None else torch.cat(v, 1 if k in ("d", "ds") else 0) for k, v in cols.items() if v}
    return r

"""The FP8 feed-forward half of an ungated transformer layer: a training step
and single tokens, on the library's entry points alone.

    z = x + r                        residual stream
    n = layernorm(z) * w + b         fp8q_layernorm_1x128 -> codes
    h = gelu(n W1^T + b1)            fp8q_linear_blockscaled_q_fast -> codes (a token: fp8q_linear_blockscaled_q)
    y = z + h W2^T + b2              fp8q_linear_blockscaled_fast, the residual stream

and back from dy: the gradients of x (and r), of w and b, of both matrices and
of both biases, each product on 1x128 codes along the dimension it reduces.

    python examples/mlp.py [tokens [features [hidden]]]

prints how far each result is from the same layer in 64 bits.
"""
import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_amax_amd as fq  # noqa: E402

E4, E5, EPS, NEPS = fq.E4M3FN, fq.E5M2, 1e-12, 1e-5


def codes(rows, cols, device):
    return (torch.empty(rows, cols, dtype=torch.uint8, device=device),
            torch.empty(rows, cols // 128, dtype=torch.float32, device=device))


class Mlp:
    """Weights as 128x128 E4M3FN codes in both layouts: [out, in] for the
    forward products, [in, out] for the input's gradients."""

    def __init__(self, w, b, w1, b1, w2, b2):
        self.w, self.b, self.b1, self.b2 = w, b, b1, b2
        self.F, self.K = w1.shape
        self.W1, self.W1t, self.W2, self.W2t = (self._weight(m) for m in (w1, w1.t(), w2, w2.t()))

    @staticmethod
    def _weight(m):
        m = m.contiguous()
        n, k = m.shape
        q, s = torch.empty(n, k, dtype=torch.uint8, device=m.device), torch.empty(n // 128, k // 128, device=m.device)
        fq.fp8q_quantize_128x128(m, n, k, k, E4, EPS, q, k, s, k // 128)
        return q, s

    def _norm(self, x, r, keep):
        M, K, dev = *x.shape, x.device
        z, n = torch.empty_like(x), torch.empty_like(x) if keep else None
        mean, rstd = torch.empty(M, device=dev), torch.empty(M, device=dev)
        q, s = codes(M, K, dev)
        fq.fp8q_layernorm_1x128(x, K, r, K, self.w, self.b, M, K, NEPS, z, K, n, K, E4, EPS, q, K, s, K // 128, mean, rstd)
        return z, n, q, s, mean, rstd

    def _args(self, q, s, weight, bias, act):
        (W, sW), k = weight, weight[0].shape[1]
        return q, E4, k, s, k // 128, 1, W, E4, k, sW, k // 128, 1, bias, act

    def token(self, x, r):
        """A decode step: the residual stream behind the layer."""
        M, F, K = x.shape[0], self.F, self.K
        z, _, q, s, _, _ = self._norm(x, r, False)
        hq, hs = codes(M, F, x.device)
        fq.fp8q_linear_blockscaled_q(*self._args(q, s, self.W1, self.b1, fq.ACT_GELU_ERF), E4, EPS, hq, F, hs, F // 128, None, 0,
                                     M, F, K)
        # the stream is updated in place
        fq.fp8q_linear_blockscaled(*self._args(hq, hs, self.W2, self.b2, fq.ACT_NONE), z, K, z, K, None, 0, M, K, F)
        return z

    def forward(self, x, r):
        M, F, K = x.shape[0], self.F, self.K
        z, n, q, s, mean, rstd = self._norm(x, r, True)
        pre = torch.empty(M, F, dtype=torch.bfloat16, device=x.device)
        hq, hs = codes(M, F, x.device)
        fq.fp8q_linear_blockscaled_q_fast(*self._args(q, s, self.W1, self.b1, fq.ACT_GELU_ERF), E4, EPS, hq, F, hs, F // 128, pre,
                                          F, M, F, K)
        y = torch.empty_like(x)
        fq.fp8q_linear_blockscaled_fast(*self._args(hq, hs, self.W2, self.b2, fq.ACT_NONE), z, K, y, K, None, 0, M, K, F)
        return y, (z, n, mean, rstd, pre)

    def backward(self, saved, dy):
        """The gradients of x (r's is the same), w, b, W1, b1, W2 and b2 from that of y."""
        z, n, mean, rstd, pre = saved
        M, F, K, dev = z.shape[0], self.F, self.K, z.device
        Mp = -(-M // 128) * 128

        def through(dC, act, pre, keep):
            """dC past an activation: codes along features and along tokens, the bias's gradient, the activation's output
            along tokens."""
            N = dC.shape[1]
            D, Dt, db = codes(M, N, dev), codes(N, Mp, dev), torch.empty(N, device=dev)
            Ht = codes(N, Mp, dev) if keep else (None, None)
            ws = torch.empty(fq.fp8q_linear_bwd_q_workspace(M, N), dtype=torch.uint8, device=dev)
            fq.fp8q_linear_bwd_q(dC, N, pre, N, act, E5, EPS, D[0], N, D[1], N // 128, Dt[0], Mp, Dt[1], Mp // 128, E4, Ht[0], Mp,
                                 Ht[1], Mp // 128, db, M, N, ws, ws.numel())
            return D, Dt, db, Ht

        def input_gradient(D, weight):
            (W, sW), (n, k) = weight, weight[0].shape
            out = torch.empty(M, n, dtype=torch.bfloat16, device=dev)
            fq.fp8q_gemm_blockscaled_fast(D[0], E5, k, D[1], k // 128, 1, W, E4, k, sW, fq.GRAN_128x128, k // 128, 1, out, n, M,
                                          n, k)
            return out

        def weight_gradient(a, b):  # a [n, Mp], b [k, Mp]: a b^T
            out = torch.empty(a[0].shape[0], b[0].shape[0], device=dev)
            fq.fp8q_gemm_blockscaled_fast(a[0], E5, Mp, a[1], Mp // 128, 1, b[0], E4, Mp, b[1], fq.GRAN_1x128, Mp // 128, 1, out,
                                          out.shape[1], *out.shape, Mp)
            return out

        D2, D2t, db2, _ = through(dy, fq.ACT_NONE, None, False)
        D1, D1t, db1, Ht = through(input_gradient(D2, self.W2t), fq.ACT_GELU_ERF, pre, True)
        npad = n if M == Mp else torch.cat([n, n.new_zeros(Mp - M, K)])
        nt = codes(K, Mp, dev)
        fq.fp8q_quantize_1x128_t(npad, Mp, K, K, E4, EPS, nt[0], Mp, nt[1], Mp // 128)
        dn = input_gradient(D1, self.W1t)
        dx, dw, db = torch.empty_like(z), torch.empty(K, device=dev), torch.empty(K, device=dev)
        ws = torch.empty(fq.fp8q_layernorm_bwd_workspace(M, K), dtype=torch.uint8, device=dev)
        fq.fp8q_layernorm_bwd(dn, K, z, K, self.w, mean, rstd, dy, K, M, K, dx, K, dw, db, ws, ws.numel())
        return dx, dw, db, weight_gradient(D1t, nt), db1, weight_gradient(D2t, Ht), db2


def reference(x, r, w, b, w1, b1, w2, b2):
    z = x + r
    c = z - z.mean(1, keepdim=True)
    n = c * torch.rsqrt((c * c).mean(1, keepdim=True) + NEPS) * w + b
    v = n @ w1.t() + b1
    return v * 0.5 * torch.erfc(v * -math.sqrt(0.5)) @ w2.t() + b2 + z


def off(got, want):
    want = want.detach()
    return float((got.double() - want).norm() / want.norm())


def inputs(tokens, K, F, device, seed=0):
    """Parameters (w, b, W1, b1, W2, b2) and bf16 activations (x, r, dy)."""
    g = torch.Generator(device=device).manual_seed(seed)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
    params = (1 + rand(K, std=0.1), rand(K, std=0.1), rand(F, K, std=K ** -0.5), rand(F, std=0.3), rand(K, F, std=F ** -0.5),
              rand(K, std=0.3))
    return params, [rand(tokens, K).bfloat16() for _ in range(3)]


def main(tokens=300, K=1024, F=2048, device="cuda"):
    params, (x, r, dy) = inputs(tokens, K, F, device)
    layer = Mlp(*params)
    y, saved = layer.forward(x, r)
    grads = layer.backward(saved, dy)
    yt = layer.token(x[:5], r[:5])

    leaves = [t.double().requires_grad_() for t in (x, *params)]
    ry = reference(leaves[0], r.double(), *leaves[1:])
    want = torch.autograd.grad(ry, leaves, dy.double())
    res = {"y": off(y, ry), "token": off(yt, ry[:5])}
    res.update({n: off(a, t) for n, a, t in zip(("dx", "dw", "db", "dW1", "db1", "dW2", "db2"), grads, want)})
    return res


if __name__ == "__main__":
    for name, v in main(*map(int, sys.argv[1:])).items():
        print(f"{name:6s} {v:.4f} off 64 bits")

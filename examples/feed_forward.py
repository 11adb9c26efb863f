"""The FP8 feed-forward half of a transformer layer: a training step and
single tokens, on the library's entry points alone.

    z = x + r                        residual stream
    n = rmsnorm(z) * w               fp8q_rmsnorm_1x128 -> codes
    h = silu(n Wg^T) * (n Wu^T)      fp8q_glu_blockscaled_fast, then fp8q_quantize_1x128
                                     (a token: fp8q_glu_blockscaled_q -> codes)
    y = h Wd^T                       fp8q_gemm_blockscaled_fast (a token: fp8q_gemm_blockscaled_few)

and back from dy: the gradients of x (and r), of w and of the three
matrices, each product on 1x128 codes along the dimension it reduces.

    python examples/feed_forward.py [tokens [features [hidden]]]

prints how far each result is from the same layer in fp32.
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import block_scaled_precision_amax_amd as fq  # noqa: E402

E4, E5, EPS, NEPS = fq.E4M3FN, fq.E5M2, 1e-12, 1e-6


def codes(rows, cols, device):
    return (torch.empty(rows, cols, dtype=torch.uint8, device=device),
            torch.empty(rows, cols // 128, dtype=torch.float32, device=device))


class FeedForward:
    """Weights as 128x128 E4M3FN codes in both layouts: [out, in] for the
    forward products, [in, out] for the input's gradients.  Gate and up are
    one matrix, gate above up."""

    def __init__(self, w, wgu, wd):
        self.w, dev = w.contiguous(), w.device
        self.F, self.K = wgu.shape[0] // 2, wgu.shape[1]
        self.gu, self.gu_t, self.d, self.d_t = (self._weight(m, dev) for m in (wgu, wgu.t(), wd, wd.t()))

    @staticmethod
    def _weight(m, dev):
        m = m.contiguous()
        n, k = m.shape
        q, s = torch.empty(n, k, dtype=torch.uint8, device=dev), torch.empty(n // 128, k // 128, device=dev)
        fq.fp8q_quantize_128x128(m, n, k, k, E4, EPS, q, k, s, k // 128)
        return q, s

    def _norm(self, x, r, want_n):
        M, K = x.shape
        z, n = torch.empty_like(x), torch.empty_like(x) if want_n else None
        q, s = codes(M, K, x.device)
        rstd = torch.empty(M, device=x.device)
        fq.fp8q_rmsnorm_1x128(x, K, r, K, self.w, M, K, NEPS, z, K, n, K, E4, EPS, q, K, s, K // 128, rstd)
        return z, n, q, s, rstd

    def _glu_args(self, q, s):
        (W, sW), F, K = self.gu, self.F, self.K
        return (q, E4, K, s, K // 128, 1, W, W[F:], E4, K, sW, sW[F // 128:], K // 128, 1, fq.ACT_SILU)

    def _product(self, q, f, s, weight, rows, out_dtype=torch.bfloat16):
        """rows x n: codes along the reduced dimension times a weight's codes."""
        W, sW = weight
        n, k = W.shape
        y = torch.empty(rows, n, dtype=out_dtype, device=q.device)
        fq.fp8q_gemm_blockscaled_fast(q, f, k, s, k // 128, 1, W, E4, k, sW, fq.GRAN_128x128, k // 128, 1, y, n, rows, n, k)
        return y

    def token(self, x, r):
        """A decode step of at most 64 rows: y and the residual stream."""
        M, F, K = x.shape[0], self.F, self.K
        z, _, q, s, _ = self._norm(x, r, False)
        hq, hs = codes(M, F, x.device)
        fq.fp8q_glu_blockscaled_q(*self._glu_args(q, s), E4, EPS, hq, F, hs, F // 128, None, 0, M, F, K)
        y = torch.empty_like(x)
        W, sW = self.d
        fq.fp8q_gemm_blockscaled_few(hq, E4, F, hs, F // 128, 1, W, E4, F, sW, fq.GRAN_128x128, F // 128, 1, y, K, M, K, F)
        return y, z

    def forward(self, x, r):
        M, F, K = x.shape[0], self.F, self.K
        z, n, q, s, rstd = self._norm(x, r, True)
        h = torch.empty(M, F, dtype=torch.bfloat16, device=x.device)
        gu = torch.empty(M, 2 * F, dtype=torch.bfloat16, device=x.device)
        fq.fp8q_glu_blockscaled_fast(*self._glu_args(q, s), h, F, gu, 2 * F, M, F, K)
        hq, hs = codes(M, F, x.device)
        fq.fp8q_quantize_1x128(h, M, F, F, E4, EPS, hq, F, hs, F // 128)
        y = self._product(hq, E4, hs, self.d, M, x.dtype)
        return y, z, (z, n, rstd, gu)

    def backward(self, saved, dy, dz):
        """dy: gradient of y; dz: gradient of the residual stream past this
        layer.  Returns the gradients of x (r's is the same), w, gate-up and
        down."""
        z, n, rstd, gu = saved
        M, F, K, dev = z.shape[0], self.F, self.K, z.device
        Mp = -(-M // 128) * 128

        def along_tokens(t, f):  # codes of t^T; ragged batches are padded with zero rows
            if Mp != M:
                t = torch.cat([t, t.new_zeros(Mp - M, t.shape[1])])
            q, s = codes(t.shape[1], Mp, dev)
            fq.fp8q_quantize_1x128_t(t, Mp, t.shape[1], t.shape[1], f, EPS, q, Mp, s, Mp // 128)
            return q, s

        def weight_gradient(a, fa, b, fb):  # a [n, Mp], b [k, Mp]: a b^T, bf16
            out = torch.empty(a[0].shape[0], b[0].shape[0], dtype=torch.bfloat16, device=dev)
            fq.fp8q_gemm_blockscaled_fast(a[0], fa, Mp, a[1], Mp // 128, 1, b[0], fb, Mp, b[1], fq.GRAN_1x128, Mp // 128, 1,
                                          out, out.shape[1], out.shape[0], out.shape[1], Mp)
            return out

        q, s = codes(M, K, dev)
        fq.fp8q_quantize_1x128(dy, M, K, K, E5, EPS, q, K, s, K // 128)
        dh = self._product(q, E5, s, self.d_t, M)
        D, Ds = codes(M, 2 * F, dev)
        Dt, Ht = codes(2 * F, Mp, dev), codes(F, Mp, dev)
        fq.fp8q_glu_bwd_q(dh, F, gu, 2 * F, fq.ACT_SILU, E5, EPS, D, 2 * F, Ds, 2 * F // 128, Dt[0], Mp, Dt[1], Mp // 128, E4,
                          Ht[0], Mp, Ht[1], Mp // 128, M, F)
        dwd = weight_gradient(along_tokens(dy, E5), E5, Ht, E4)
        dwgu = weight_gradient(Dt, E5, along_tokens(n, E4), E4)
        dn = self._product(D, E5, Ds, self.gu_t, M)
        dx, dw = torch.empty_like(z), torch.empty(K, device=dev)
        ws = torch.empty(fq.fp8q_rmsnorm_bwd_workspace(M, K), dtype=torch.uint8, device=dev)
        fq.fp8q_rmsnorm_bwd(dn, K, z, K, self.w, rstd, dz, K, M, K, dx, K, dw, ws, ws.numel())
        return dx, dw, dwgu, dwd


def reference(x, r, w, wgu, wd):
    z = x + r
    n = z * torch.rsqrt(z.square().mean(1, keepdim=True) + NEPS) * w
    g, u = (n @ wgu.t()).chunk(2, dim=1)
    return (g * torch.sigmoid(g) * u) @ wd.t(), z


def off(got, want):
    want = want.detach()
    return float((got.float() - want).norm() / want.norm())


def main(tokens=300, K=1024, F=2048, device="cuda"):
    g = torch.Generator(device=device).manual_seed(0)
    rand = lambda *s, std=1.0: torch.randn(*s, generator=g, device=device) * std  # noqa: E731
    w, wgu, wd = 1 + rand(K, std=0.1), rand(2 * F, K, std=K ** -0.5), rand(K, F, std=F ** -0.5)
    x, r, dy, dz = (rand(tokens, K).bfloat16() for _ in range(4))
    layer = FeedForward(w, wgu, wd)
    y, z, saved = layer.forward(x, r)
    grads = layer.backward(saved, dy, dz)
    yt, _ = layer.token(x[:5], r[:5])

    leaves = [t.float().requires_grad_() for t in (x, w, wgu, wd)]
    ry, rz = reference(leaves[0], r.float(), *leaves[1:])
    want = torch.autograd.grad([ry, rz], leaves, [dy.float(), dz.float()])
    res = {"y": off(y, ry), "z": off(z, rz), "token": off(yt, ry[:5])}
    res.update({n: off(a, b) for n, a, b in zip(("dx", "dw", "dWgu", "dWd"), grads, want)})
    return res


if __name__ == "__main__":
    for name, v in main(*map(int, sys.argv[1:])).items():
        print(f"{name:6s} {v:.4f} off fp32")

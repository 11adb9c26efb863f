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

"""Edges of the gradient norm and of clipping: whose memory the results are, and the precision of
long lists."""
import pytest
import torch

from helpers import cuda_ok

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F


def _pool(t):
    """The stream whose pool a tensor's memory belongs to."""
    return next(s["stream"] for s in torch.cuda.memory_snapshot()
                if s["address"] <= t.data_ptr() < s["address"] + s["total_size"])


def test_results_come_from_the_given_streams_pool():
    g = torch.ones(1000, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    norm, coef = F.grad_norm([g], stream=side)
    kept = F.GradList([g], stream=side)
    side.synchronize()
    for t in (norm, coef, kept.norm, kept.coef):
        assert _pool(t) == side.cuda_stream
    assert _pool(F.GradList([g]).norm) == torch.cuda.current_stream().cuda_stream

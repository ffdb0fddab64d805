"""Edges of the gradient norm and of clipping: whose memory the results are, and the precision of
long lists."""
import math

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


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("numel", [1 << 28, (1 << 19) - 3])
def test_the_norm_of_long_lists_has_no_bias(dtype, numel):
    """The error's mean over eight lists of normal values: what is left of the results' own
    roundings (each up to 2^-24, independent) and of a sum whose errors lean to one side. Held
    to the largest rounding of a single result."""
    errors = []
    for seed in range(8):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        g = (torch.randn(numel, generator=gen, device="cuda") * 1e-3).to(dtype)
        ref = math.sqrt(sum(float(p.double().square().sum()) for p in g.split(1 << 26)))
        errors.append(F.grad_norm([g])[0].item() / ref - 1)
    assert abs(sum(errors) / len(errors)) <= 2.0 ** -24


@pytest.mark.parametrize("bad", [math.inf, math.nan])
@pytest.mark.parametrize("numel", [100, 700001])
def test_coefficient_of_a_norm_that_is_not_finite(bad, numel):
    """0 or NaN, or the scale where nothing is to be clipped."""
    g = torch.full((numel,), 1e-3, device="cuda")
    g[-1] = bad
    norm, coef = F.grad_norm([g], scale=0.5)
    assert norm.isnan().item() == math.isnan(bad) and not torch.isfinite(norm).item()
    assert coef.item() == 0.5
    _, coef = F.grad_norm([g], max_norm=1.0, scale=0.5)
    assert coef.isnan().item() if math.isnan(bad) else coef.item() == 0

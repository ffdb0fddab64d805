"""A branch without gates, scale and a norm after it is a residual: branch_rmsnorm_quantize then
gives every byte that rmsnorm_quantize gives. The values are multiples of 1/8 below 1, so that the
sum of the two is exact in bf16 and a row's squares (multiples of 1/64, at most 3.1 each, 32768 of
them below 2^24 / 64) add up exactly in any order: rstd is the same, and nothing may differ."""
import pytest
import torch

from helpers import cuda_ok
from test_gpu_norm import _dev_gamma, _gamma

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F


@pytest.mark.parametrize("kind,pow2", [("mxfp8", False), ("blockwise", False), ("blockwise", True),
                                       ("tensorwise", False), ("delayed", False)])
@pytest.mark.parametrize("rows,cols", [(1, 128), (300, 256), (300, 1024), (700, 4096), (130, 5120),
                                       (40, 16384), (20, 32768), (77, 2064)])
def test_every_byte_is_the_norms(kind, pow2, rows, cols):
    if kind in ("mxfp8", "blockwise"):
        cols = cols // 128 * 128
    rec = F.Recipe(kind=kind, power_2_scales=pow2)
    gen = torch.Generator(device="cuda").manual_seed(rows)
    x, res = (torch.randint(-7, 8, (rows, cols), generator=gen, device="cuda").div(8)
              .to(torch.bfloat16) for _ in range(2))
    g = _dev_gamma(_gamma(cols), False)
    for col in (True, False):
        a, ha, ra, none, ya = F.branch_rmsnorm_quantize(rec, x, res, g, want_col=col, want_y=True)
        b, hb, rb, yb = F.rmsnorm_quantize(rec, x, g, residual=res, want_col=col, want_y=True)
        torch.cuda.synchronize()
        assert none is None and torch.equal(ha, x + res)
        assert all(torch.equal(u.view(torch.uint8), v.view(torch.uint8))
                   for u, v in ((ha, hb), (ra, rb), (ya, yb)))
        for f in ("row", "col", "row_scale", "col_scale", "amax", "scale", "scale_inv"):
            u, v = getattr(a, f), getattr(b, f)
            assert (u is None) == (v is None)
            assert u is None or torch.equal(u, v), f

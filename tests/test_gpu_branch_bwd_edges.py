"""The gated branch's backward pass on rows whose squares leave float32's range: the forward pass
leaves rstd 0 there, so xh and xo are zeros whatever the row holds, and no product of a gradient
with the row's own values may overflow on the way. Tolerances as in test_gpu_branch_bwd."""
import numpy as np
import pytest
import torch

from helpers import cuda_ok, from_dev_bf16, to_dev_bf16
from test_gpu_branch_bwd import _cuda, _kept, case, check
from workloads import bf16_bits_from_f32, bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

HUGE = 1e38                                             # its square and a sum of them: infinite


def _huge(bits, rows):
    """The rows set to +-HUGE, which bf16 holds."""
    sign = np.where(np.arange(bits.shape[1]) % 3 == 0, -1, 1).astype(np.float32)
    bits = bits.copy()
    bits[rows] = bf16_bits_from_f32(np.float32(HUGE) * sign)[None]
    return bits


@pytest.mark.parametrize("cols", [48, 1024, 4096, 5120, 16400, 32768])
@pytest.mark.parametrize("ckpt", [(False, False), (True, True), (True, False), (False, True)])
def test_rows_whose_squares_overflow(cols, ckpt):
    rows = 40
    c = case(rows, cols, token=True, ckpt=ckpt)
    # gradients whose product with such a row's elements leaves float32's range
    c["dy"] = bf16_bits_normal(rows, cols, seed=1, sigma=8.0)
    c["dres"] = bf16_bits_normal(rows, cols, seed=2, sigma=8.0)
    h, o = (_huge(bf16_bits_normal(rows, cols, seed=s), at) for s, at in ((3, [4, 39]), (5, [7, 39])))
    c["h"], c["hv"] = _kept(h, ckpt[0])
    c["o"], c["ov"] = _kept(o, ckpt[1])
    c["rstd"][[4, 39]] = 0
    c["ro"][[7, 39]] = 0
    c["t"][[4, 7, 39]] = 0.5
    d = check(c)
    assert all(bool(torch.isfinite(t.float()).all()) for t in d)
    dres = to_dev_bf16(c["dres"])
    assert torch.equal(d.dh[[4, 39]], dres[[4, 39]]) and not d.dbranch[[7, 39]].any()
    assert not d.dtoken_gate[[7, 39]].any()


def test_forward_and_backward_of_such_rows():
    """What the forward pass leaves of them is what the backward pass takes: no NaN on the way."""
    rows, cols = 20, 512
    o = to_dev_bf16(_huge(bf16_bits_normal(rows, cols, seed=1), [3]))
    res = to_dev_bf16(_huge(bf16_bits_normal(rows, cols, seed=2), [6]))
    dy, dres = (to_dev_bf16(bf16_bits_normal(rows, cols, seed=s, sigma=8.0)) for s in (3, 4))
    g = torch.ones(cols, device="cuda")
    _, h, rstd, ro, _ = F.branch_rmsnorm_quantize(None, o, res, g, gamma_post=g, gate=g,
                                                  want_row=False, want_col=False, want_y=True)
    torch.cuda.synchronize()
    assert float(ro[3]) == 0 and float(rstd[6]) == 0
    assert np.array_equal(from_dev_bf16(h)[3], from_dev_bf16(res)[3])
    c = dict(rstd=rstd.cpu().numpy(), ro=ro.cpu().numpy())
    d = F.branch_rmsnorm_bwd(dy, h, _cuda(c["rstd"]), g, o, rstd_branch=_cuda(c["ro"]),
                             gamma_post=g, gate=g, dres=dres)
    torch.cuda.synchronize()
    for t in d[:5]:
        assert bool(torch.isfinite(t.float()).all())
    assert torch.equal(d.dh[6], dres[6]) and not d.dbranch[3].any()


def test_no_columns():
    """A gradient per token is a sum over no columns: zeros, not what the buffer held."""
    x, t = torch.empty((5, 0), dtype=torch.bfloat16, device="cuda"), torch.ones(5, device="cuda")
    none, held = torch.empty(0, device="cuda"), torch.full((5,), 7.0, device="cuda")
    for stream in (None, torch.cuda.Stream()):
        mine = held.clone()
        torch.cuda.synchronize()
        d = F.branch_rmsnorm_bwd(x, x, t, none, x, token_gate=t, dtoken_gate=mine, stream=stream)
        torch.cuda.synchronize()
        assert not d.dtoken_gate.any() and d.dh.shape == (5, 0) and d.dgamma.numel() == 0

"""The pre-norm MLP block of the examples: its step against a float32 model of the same block,
clipping, and a single token when serving."""
import importlib.util
import pathlib

import pytest
import torch

from helpers import cuda_ok

pytestmark = pytest.mark.gpu

if cuda_ok():
    PATH = pathlib.Path(__file__).resolve().parent.parent / "examples" / "prenorm_mlp_step.py"
    SPEC = importlib.util.spec_from_file_location("prenorm_mlp_step", PATH)
    EX = importlib.util.module_from_spec(SPEC)
    SPEC.loader.exec_module(EX)


def _rel(a, b):
    return float((a.float() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens", [200, 256])
def test_step_against_float32(tokens):
    """FP8 operands (4 significant bits: 2^-4 relative rounding, about 3% in the mean of a
    product of two) leave the outputs within 10% in the 2-norm, the residual path exactly."""
    torch.manual_seed(0)
    hidden, ffn = 256, 512
    m = EX.PreNormMlp(hidden, ffn)
    x, res = (torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16) for _ in range(2))
    dy, dres = (torch.randn(tokens, hidden, device="cuda").to(torch.bfloat16) for _ in range(2))
    y, h = m.forward(x, res)
    dh = m.backward(dy, dres)

    hr = (x.float() + res.float()).to(torch.bfloat16).float().requires_grad_()
    g, w1, w2 = (t.float().requires_grad_() for t in (m.gamma, m.w1, m.w2))
    n = hr * (hr.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g
    yr = torch.nn.functional.gelu(n @ w1.t()) @ w2.t()
    ((yr * dy.float()).sum() + (hr * dres.float()).sum()).backward()
    assert torch.equal(h.float(), hr.detach())
    assert _rel(y, yr.detach()) < 0.1
    assert _rel(dh.float() - dres.float(), hr.grad - dres.float()) < 0.1
    for got, ref in ((m.dw1, w1), (m.dw2, w2), (m.dgamma, g)):
        assert _rel(got, ref.grad) < 0.1

    before = [t.clone() for t in (m.dw1, m.dw2, m.dgamma)]
    want = torch.stack([t.double().square().sum() for t in before]).sum().sqrt().item()
    norm, coef = m.clip(want / 4)
    assert abs(norm.item() - want) <= 1e-5 * want
    for t, b in zip((m.dw1, m.dw2, m.dgamma), before):
        assert torch.equal(t, (b.float() * coef).to(t.dtype))


def test_single_token_equals_the_batch():
    m = EX.PreNormMlp(512, 1024)
    x, res = (torch.randn(130, 512, device="cuda").to(torch.bfloat16) for _ in range(2))
    y, h = m.forward(x, res, train=False)
    for i in (0, 129):
        one, hi = m.forward(x[i:i + 1], res[i:i + 1], train=False)
        assert torch.equal(one[0], y[i]) and torch.equal(hi[0], h[i])

"""The stack of MLP blocks with norms on both sides of the examples: its step against a float32 model
of the same stack, a single token when serving, and the step captured into a graph."""
import importlib.util
import pathlib

import pytest
import torch

from helpers import cuda_ok

pytestmark = pytest.mark.gpu

if cuda_ok():
    PATH = pathlib.Path(__file__).resolve().parent.parent / "examples" / "sandwich_mlp_step.py"
    SPEC = importlib.util.spec_from_file_location("sandwich_mlp_step", PATH)
    EX = importlib.util.module_from_spec(SPEC)
    SPEC.loader.exec_module(EX)


def _rel(a, b):
    return float((a.float() - b).norm() / b.norm())


@pytest.mark.parametrize("tokens", [200, 256])
def test_step_against_float32(tokens):
    """A product of two FP8 operands (2^-4 relative rounding at most, 2.6% in the mean) is off by
    3.7%; the deepest gradients have six of them behind them, and a checkpoint: within 15%."""
    hidden, ffn = 256, 512
    m = EX.SandwichMlp(hidden, ffn)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    dy = torch.randn(tokens, hidden, generator=gen, device="cuda").to(torch.bfloat16)
    y = m.forward(x)
    dx = m.backward(dy)

    def norm(h, g):
        return h * (h.square().mean(1, keepdim=True) + 1e-5).rsqrt() * g

    leaves = {}

    def leaf(name, t):
        leaves[name] = t.float().requires_grad_()
        return leaves[name]

    h = xr = leaf("x", x)
    for i, b in enumerate(m.blocks):
        n = norm(h, leaf(f"gamma{i}", b.gamma))
        o = torch.nn.functional.gelu(n @ leaf(f"w1{i}", b.w1).t()) @ leaf(f"w2{i}", b.w2).t()
        h = h + m.scale * leaf(f"gate{i}", b.gate) * norm(o, leaf(f"post{i}", b.gamma_post))
    yr = norm(h, leaf("last", m.gamma))
    (yr * dy.float()).sum().backward()
    assert _rel(y, yr.detach()) < 0.15 and _rel(dx, xr.grad) < 0.15
    got = {"last": m.dgamma}
    for i, b in enumerate(m.blocks):
        got.update({f"gamma{i}": b.dgamma, f"post{i}": b.dgamma_post, f"gate{i}": b.dgate,
                    f"w1{i}": b.dw1, f"w2{i}": b.dw2})
    for name, g in got.items():
        assert _rel(g, leaves[name].grad) < 0.15, name


def test_single_token_equals_the_batch():
    m = EX.SandwichMlp(512, 1024)
    x = torch.randn(130, 512, device="cuda").to(torch.bfloat16)
    y = m.forward(x, train=False)
    for i in (0, 129):
        assert torch.equal(m.forward(x[i:i + 1], train=False)[0], y[i])


def test_step_in_a_graph():
    m = EX.SandwichMlp(256, 512)
    x = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    dy = torch.randn(200, 256, device="cuda").to(torch.bfloat16)
    y, dx = m.forward(x), m.backward(dy)
    ref = [t.clone() for b in m.blocks for t in (b.dw1, b.dw2, b.dgamma, b.dgamma_post, b.dgate)]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gy, gdx = m.forward(x), m.backward(dy)
    for b in m.blocks:
        for t in (b.dw1, b.dw2, b.dgamma, b.dgamma_post, b.dgate):
            t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    got = [t for b in m.blocks for t in (b.dw1, b.dw2, b.dgamma, b.dgamma_post, b.dgate)]
    assert torch.equal(gy, y) and torch.equal(gdx, dx)
    assert all(torch.equal(a, b) for a, b in zip(got, ref))

"""Pins of the oracle's RMSNorm, its backward pass and the gradient norm, each against something
that is not the oracle: torch's float64 autograd, finite differences, closed forms."""
import math

import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from workloads import bf16_bits_from_f32, bf16_bits_normal


def test_closed_forms():
    # a row of one value v: rstd = 1 / sqrt(v^2 + eps), so y is gamma for eps 0
    h = np.full((2, 8), 3.0)
    g = np.arange(8.0)
    assert np.allclose(O.rmsnorm_f64(h, g, 0.0), np.tile(g, (2, 1)), rtol=1e-15)
    assert np.allclose(O.rmsnorm_rstd_f64(np.zeros((1, 4)), 0.25), [2.0], rtol=1e-15)
    # one element a row: y does not depend on h, so dh is the residual's gradient alone
    dh, dg = O.rmsnorm_bwd_f64([[5.0]], [[2.0]], [0.5], [3.0], [[7.0]])
    assert np.allclose(dh, [[7.0]]) and np.allclose(dg, [5.0])


def test_residual_add_rounds_once():
    x = bf16_bits_normal(64, 64, seed=1)
    r = bf16_bits_normal(64, 64, seed=2, sigma=30.0)
    t = torch.from_numpy(O.bf16_to_f32(x) + O.bf16_to_f32(r)).to(torch.bfloat16)
    assert np.array_equal(O.residual_add_bf16(x, r), t.view(torch.int16).numpy().view(np.uint16))


@pytest.mark.parametrize("rows,cols", [(1, 16), (5, 48), (3, 256)])
def test_against_autograd(rows, cols):
    g = torch.Generator().manual_seed(rows * cols)
    h = torch.randn(rows, cols, generator=g, dtype=torch.float64, requires_grad=True)
    gamma = torch.randn(cols, generator=g, dtype=torch.float64, requires_grad=True)
    dy = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    dres = torch.randn(rows, cols, generator=g, dtype=torch.float64)
    rstd = (h.square().mean(1, keepdim=True) + 1e-5).rsqrt()
    y = h * rstd * gamma
    ((y * dy).sum() + (h * dres).sum()).backward()
    assert np.allclose(O.rmsnorm_f64(h.detach().numpy(), gamma.detach().numpy(), 1e-5),
                       y.detach().numpy(), rtol=1e-13, atol=0)
    dh, dg = O.rmsnorm_bwd_f64(dy.numpy(), h.detach().numpy(), rstd.detach().numpy()[:, 0],
                               gamma.detach().numpy(), dres.numpy())
    assert np.allclose(dh, h.grad.numpy(), rtol=1e-12, atol=1e-13)
    assert np.allclose(dg, gamma.grad.numpy(), rtol=1e-12, atol=1e-13)


def test_against_differences():
    rng = np.random.default_rng(3)
    h, gamma = rng.standard_normal((4, 32)), rng.standard_normal(32)
    dy, v = rng.standard_normal((4, 32)), rng.standard_normal((4, 32))
    dh, _ = O.rmsnorm_bwd_f64(dy, h, O.rmsnorm_rstd_f64(h, 1e-5), gamma)
    e = 1e-5                                   # error e^2 f''' ~ 1e-10 and 1e-16 / e = 1e-11
    diff = (np.sum(dy * O.rmsnorm_f64(h + e * v, gamma, 1e-5))
            - np.sum(dy * O.rmsnorm_f64(h - e * v, gamma, 1e-5))) / (2 * e)
    assert abs(np.sum(dh * v) - diff) < 1e-8


def test_quantised_value_is_near_the_norm():
    x = bf16_bits_normal(8, 128, seed=5)
    gamma = O.bf16_to_f32(bf16_bits_from_f32(np.linspace(0.5, 2, 128, dtype=np.float32)))
    f = O.bf16_to_f32(x)
    y = O.rmsnorm_f64(f, gamma, 1e-5)
    y32 = O.rmsnorm_y_f32(x, O.rmsnorm_rstd_f64(f, 1e-5).astype(np.float32), gamma)
    assert np.max(np.abs(y32 - y) / np.abs(y)) < 3 * 2.0 ** -24      # rstd and two products


def test_grad_norm_and_coef():
    assert O.grad_norm_f64([[3.0], [[4.0, 0.0]]]) == 5.0
    assert O.grad_norm_f64([[3.0], [4.0]], scale=0.5) == 2.5
    assert O.grad_norm_f64([]) == 0.0
    assert O.clip_coef_f64(0.5, 1.0) == 1.0
    assert math.isclose(O.clip_coef_f64(4.0, 1.0, 0.5), 0.125, rel_tol=1e-6)
    assert O.clip_coef_f64(math.inf, 1.0) == 0.0
    assert math.isnan(O.clip_coef_f64(math.nan, 1.0))
    assert O.clip_coef_f64(math.inf, math.inf, 2.0) == 2.0

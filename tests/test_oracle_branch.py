"""Pins of the oracle's gated branch, its backward pass and the 8-bit checkpoints, each against
something that is not the oracle: torch's float64 autograd, differences, hand-made blocks."""
import numpy as np
import pytest
import torch

from oracle import fp8_oracle as O
from workloads import bf16_bits_from_f32, bf16_bits_normal


@pytest.mark.parametrize("post", [True, False])
@pytest.mark.parametrize("gate", [True, False])
@pytest.mark.parametrize("token", [True, False])
def test_branch_against_autograd(post, gate, token):
    rows, cols, scale, eps = 5, 48, 0.3, 1e-3
    gen = torch.Generator().manual_seed(7)

    def leaf(*shape):
        return torch.randn(*shape, generator=gen, dtype=torch.float64).requires_grad_()

    o, res, dh = leaf(rows, cols), leaf(rows, cols), leaf(rows, cols).detach()
    a = leaf(cols) if post else None
    g = leaf(cols) if gate else None
    t = leaf(rows) if token else None
    rstd = (o.square().mean(1) + eps).rsqrt() if post else None
    n = o if not post else o * rstd[:, None] * a
    for f in (g, None if t is None else t[:, None]):
        n = n if f is None else n * f
    h = res + scale * n
    (h * dh).sum().backward()

    def arr(v):
        return None if v is None else v.detach().numpy()

    args = (arr(rstd), arr(a), arr(g), arr(t), scale)
    assert np.allclose(O.branch_sum_f64(arr(o), arr(res), *args), arr(h), rtol=1e-13, atol=1e-13)
    d = O.branch_bwd_f64(dh.numpy(), arr(o), *args)
    assert np.allclose(d["dbranch"], o.grad.numpy(), rtol=1e-11, atol=1e-13)
    for name, leaf_ in (("dgamma_post", a), ("dgate", g), ("dtoken_gate", t)):
        if leaf_ is not None:
            assert np.allclose(d[name], leaf_.grad.numpy(), rtol=1e-11, atol=1e-13)


def test_branch_backward_against_differences():
    rng = np.random.default_rng(5)
    o, res, dh, v = (rng.standard_normal((4, 32)) for _ in range(4))
    a, g, t, eps, e = rng.standard_normal(32), rng.standard_normal(32), rng.random(4), 1e-5, 1e-5

    def loss(x):
        return np.sum(dh * O.branch_sum_f64(x, res, O.rmsnorm_rstd_f64(x, eps), a, g, t, 0.7))

    d = O.branch_bwd_f64(dh, o, O.rmsnorm_rstd_f64(o, eps), a, g, t, 0.7)["dbranch"]
    diff = (loss(o + e * v) - loss(o - e * v)) / (2 * e)
    assert abs(np.sum(d * v) - diff) < 1e-8            # e^2 f''' and 1e-16 / e


def test_checkpoint_blocks_by_hand():
    x = np.zeros((2, 48), dtype=np.float32)
    x[0, 0], x[0, 1] = 448.0, 1.0                      # e = 0
    x[0, 32:] = 450.0                                  # the next bf16: e = 1; a block of 16 columns
    x[1, 5] = 2.0 ** -20                               # 256 2^-28 = 2^-20, and 448 2^-29 < 2^-20
    codes, scale = O.checkpoint_pack(bf16_bits_from_f32(x))
    assert codes.shape == (2, 48) and scale.shape == (2, 4)
    assert scale.tolist() == [[127, 128, 0, 0], [127 - 28, 0, 0, 0]]
    v = O.checkpoint_values(codes, scale)
    assert v[0, 0] == 448 and v[0, 1] == 1 and (v[0, 32:] == 448).all() and v[1, 5] == 2.0 ** -20
    assert not v[1, :5].any() and not v[1, 6:].any()


@pytest.mark.parametrize("cols", [16, 128, 176])
def test_checkpoint_error_is_half_a_step(cols):
    x = bf16_bits_normal(40, cols, seed=3, outlier_p=1e-2)
    codes, scale = O.checkpoint_pack(x)
    v, f = O.checkpoint_values(codes, scale), O.bf16_to_f32(x).astype(np.float64)
    step = np.repeat(2.0 ** (scale.astype(float) - 127), 32, axis=1)[:, :cols]
    assert np.all(np.abs(v - f) <= np.maximum(2.0 ** -4 * np.abs(f), 2.0 ** -10 * step))

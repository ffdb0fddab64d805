"""What the differences of branch_differences let through and what they do not: the oracle's
gradients, rounded as a kernel's outputs are, against wrong ones."""
import numpy as np
import pytest

from branch_differences import gradients, problem, wrong
from oracle import fp8_oracle as O

FORMS = [dict(), dict(post=False), dict(gate=False, dres=False), dict(token=False),
         dict(ckpt=(True, True), dres=False), dict(post=False, gate=False, token=False)]


def _outputs(p):
    d = gradients(p)
    for name in ("dh", "dbranch"):
        d[name] = O.bf16_to_f32(O.f64_to_bf16(d[name])).astype(np.float64)
    return {k: v if k in ("dh", "dbranch") else np.asarray(v, dtype=np.float32)
            for k, v in d.items()}


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,cols", [(24, 512), (3, 16), (7, 1040)])
def test_rounded_gradients_pass(rows, cols, form):
    p = problem(rows, cols, **form)
    assert wrong(p, _outputs(p)) == set()


@pytest.mark.parametrize("form", FORMS)
def test_wrong_gradients_do_not(form):
    p = problem(24, 512, **form)
    right = _outputs(p)
    names = {"dh", "dbranch", "dgamma"}
    names |= {n for n, at in (("dgamma_post", "a"), ("dgate", "g"), ("dtoken_gate", "t"))
              if p[at] is not None}
    for name in names:
        for change in (0.0, -1.0, 1.02, 0.98):
            assert wrong(p, {**right, name: right[name] * change}) == {name}, (name, change)


@pytest.mark.parametrize("form", FORMS)
def test_a_missing_term_is_found(form):
    p = problem(24, 512, **form)
    right = _outputs(p)
    r, xh = p["rstd"][:, None], p["h"] * p["rstd"][:, None]
    a = p["dy"] * p["gamma"]
    flat = p["dres"] + r * a                             # without the norm's projection
    assert wrong(p, {**right, "dh": flat}) == {"dh"}
    assert wrong(p, {**right, "dh": flat - r * xh * np.mean(a * xh)}) == {"dh"}    # of all rows
    one = np.ones((1, 1))
    t, ro = (one if v is None else v[:, None] for v in (p["t"], p["ro"]))
    w = p["scale"] * (one if p["a"] is None else p["a"]) * (one if p["g"] is None else p["g"])
    u = gradients(p)["dh"] * w
    if p["a"] is not None:
        assert wrong(p, {**right, "dbranch": ro * t * u}) == {"dbranch"}
        assert wrong(p, {**right, "dbranch": right["dbranch"] / ro}) == {"dbranch"}
    if p["g"] is not None:
        assert wrong(p, {**right, "dbranch": right["dbranch"] / p["g"]}) == {"dbranch"}
    if p["t"] is not None:
        assert wrong(p, {**right, "dbranch": right["dbranch"] * t}) == {"dbranch"}
        assert wrong(p, {**right, "dtoken_gate": right["dtoken_gate"] * p["t"]}) == {"dtoken_gate"}
    shifted = np.roll(right["dbranch"], 1, axis=1)       # a neighbour's column
    assert wrong(p, {**right, "dbranch": shifted}) == {"dbranch"}

"""Gradients of the gated branch and the norm behind it, held against central differences of the
formulas in float64, row by row: no use is made of the formulas of the gradients.

The loss is a sum over rows, and a row's loss depends on that row alone, so one pair of evaluations
gives every row's derivative along that row's part of a direction. Directions: the gradient itself
(the bound is then 2^-8 of the derivative, where a random one would let a wrong gradient through),
the row's own values (along which the norm's projection takes the derivative away), and a random
one. Bounds, for an output `got` and a direction v:

  2^-8 sum |v got|       the output's rounding to bf16 (dh, dbranch)
  sum |v| err            float32: K = 100 roundings (test_gpu_branch_bwd), and three times the
                         rounding of the saved rstd, of the terms' sizes
  1e-6 size              the difference itself: with steps of E = 1e-4 along v of root mean square 1
                         E^2 f''' / 6, f''' some ten times the size of the loss' terms (the rows' own
                         root mean squares are 1 and more), and 2^-52 / E
"""
import numpy as np

from oracle import fp8_oracle as O
from workloads import bf16_bits_from_f32, bf16_bits_normal

EPS, E = 1e-5, 1e-4
K = 104 * 2.0 ** -24


def _bf16(a):
    return O.bf16_to_f32(bf16_bits_from_f32(np.asarray(a, dtype=np.float32))).astype(np.float64)


def problem(rows, cols, post=True, gate=True, token=True, ckpt=(False, False), dres=True, seed=0):
    rng = np.random.default_rng(seed)
    p = dict(rows=rows, cols=cols, scale=0.5, ckpt=ckpt)
    for name, at, sigma in (("h", 0, 1.0), ("o", 1, 3.0)):
        bits = bf16_bits_normal(rows, cols, seed=seed + 1 + at, sigma=sigma)
        p[name + "_kept"] = O.checkpoint_pack(bits) if ckpt[at] else bits
        p[name] = O.checkpoint_values(*p[name + "_kept"]) if ckpt[at] \
            else O.bf16_to_f32(bits).astype(np.float64)
    p["dy_bits"] = bf16_bits_normal(rows, cols, seed=seed + 3, sigma=1e-2)
    p["dres_bits"] = bf16_bits_normal(rows, cols, seed=seed + 4, sigma=1e-2) if dres else None
    p["dy"] = O.bf16_to_f32(p["dy_bits"]).astype(np.float64)
    p["dres"] = O.bf16_to_f32(p["dres_bits"]).astype(np.float64) if dres else 0.0
    p["gamma"] = _bf16(1 + 0.2 * rng.standard_normal(cols))
    p["a"] = _bf16(1 + 0.2 * rng.standard_normal(cols)) if post else None
    p["g"] = _bf16(0.3 * rng.standard_normal(cols)) if gate else None
    p["t"] = (0.25 + rng.random(rows)).astype(np.float32).astype(np.float64) if token else None
    if token:
        p["t"][1::5] = 0
    p["rstd"] = O.rmsnorm_rstd_f64(p["h"], EPS)
    p["ro"] = O.rmsnorm_rstd_f64(p["o"], EPS) if post else None
    p["res"] = p["h"] - _stream(p, p["o"], 0.0)          # so that the stream is what is kept of it
    return p


def _stream(p, o, res, **changed):
    a, g, t = (changed.get(k, p[k]) for k in "agt")
    ro = O.rmsnorm_rstd_f64(o, EPS) if p["a"] is not None else None
    return O.branch_sum_f64(o, res, ro, a, g, t, p["scale"])


def _loss(p, o=None, res=None, gamma=None, **changed):
    """Every row's loss: sum_c dy y + dres h."""
    s = _stream(p, p["o"] if o is None else o, p["res"] if res is None else res, **changed)
    y = O.rmsnorm_f64(s, p["gamma"] if gamma is None else gamma, EPS)
    return np.sum(p["dy"] * y + p["dres"] * s, axis=1)


def gradients(p):
    """The oracle's."""
    dh, dgamma = O.rmsnorm_bwd_f64(p["dy"], p["h"], p["rstd"], p["gamma"], p["dres"])
    return dict(O.branch_bwd_f64(dh, p["o"], p["ro"], p["a"], p["g"], p["t"], p["scale"]), dh=dh,
                dgamma=dgamma)


def _errors(p):
    """What float32 may add to each element (test_gpu_branch_bwd has the reasons)."""
    one = np.ones((1, 1))
    a, g = (one if v is None else v[None] for v in (p["a"], p["g"]))
    t, ro = (one if v is None else v[:, None] for v in (p["t"], p["ro"]))
    r = p["rstd"][:, None]
    xh, b = p["h"] * r, np.abs(p["dy"] * p["gamma"])
    dh = K * (r * (b + np.abs(xh) * np.mean(b * np.abs(xh), 1, keepdims=True)) + np.abs(p["dres"]))
    w, xo, size = np.abs(p["scale"] * a * g), np.abs(p["o"] * ro), np.abs(gradients(p)["dh"])
    u = w * (dh + K * size)
    err = dict(dh=dh, dtoken_gate=np.sum(u * xo, 1))
    proj = xo * np.mean(u * xo, 1, keepdims=True) if p["a"] is not None else 0.0
    err["dbranch"] = ro * t * (u + proj)
    order = (p["rows"] + 70) * 2.0 ** -24 + K
    err["dgamma"] = order * np.sum(np.abs(p["dy"] * xh), 0)
    sums = p["scale"] * np.sum(t * xo * (order * size + dh), 0)
    err["dgamma_post"], err["dgate"] = sums * np.abs(g[0]), sums * np.abs(a[0])
    return err


def _along(v):
    rms = np.sqrt(np.mean(v * v, 1, keepdims=True))
    return np.divide(v, rms, out=np.zeros_like(v), where=rms > 0)


def wrong(p, got):
    """Names of the gradients (dh, dbranch, dgamma, ...) in `got` that a difference contradicts."""
    rng, ref, err, bad = np.random.default_rng(9), gradients(p), _errors(p), set()
    s = _stream(p, p["o"], p["res"])
    size = np.sum(np.abs(p["dy"] * O.rmsnorm_f64(s, p["gamma"], EPS)) + np.abs(p["dres"] * s), 1)
    for name, at in (("dh", "res"), ("dbranch", "o")):
        x, d = p[at], np.asarray(got[name], dtype=np.float64)
        for v in (ref[name], p["h"] if name == "dh" else p["o"], rng.standard_normal(x.shape)):
            v = _along(v)
            q = (_loss(p, **{at: x + E * v}) - _loss(p, **{at: x - E * v})) / (2 * E)
            tol = np.sum(np.abs(v) * (2.0 ** -8 * np.abs(d) + err[name]), 1) + 1e-6 * size
            if not np.all(np.abs(np.sum(d * v, 1) - q) <= tol):
                bad.add(name)
    if p["t"] is not None:
        q = (_loss(p, t=p["t"] + E) - _loss(p, t=p["t"] - E)) / (2 * E)
        if not np.all(np.abs(got["dtoken_gate"] - q) <= err["dtoken_gate"] + 1e-6 * size):
            bad.add("dtoken_gate")
    for name, at in (("dgamma", "gamma"), ("dgamma_post", "a"), ("dgate", "g")):
        if p[at] is None:
            continue
        for c in rng.integers(0, p["cols"], 12):
            v = np.zeros(p["cols"])
            v[c] = E
            q = np.sum(_loss(p, **{at: p[at] + v}) - _loss(p, **{at: p[at] - v})) / (2 * E)
            if not abs(got[name][c] - q) <= err[name][c] + 1e-6 * np.sum(size):
                bad.add(name)
    return bad

"""GPU parity of the gated branch's backward pass, of the norm's backward pass from an 8-bit
checkpoint, and of the FP8 copies made from one. Tolerances, against float64 with the same rstd:

  dh       as for the norm alone (test_gpu_norm): before its rounding to bf16 within E = BWD_K
           (100 float32 roundings) of the sizes of its terms.
  dbranch  u = dh w inherits |w| E; s adds fewer than 100 roundings of sum |u xo|, and the rest of
           the formula fewer than 10: before its rounding within rstd_branch t times
           (|w| E + |xo| mean(|w| E |xo|)) + BWD_K (|u| + |xo| mean |u xo|).
  S        at most rows + 70 additions a column of |t dh xo|, and E's share of each.
Codes and scales made from a checkpoint are compared exactly.
"""
import numpy as np
import pytest
import torch

from helpers import cuda_ok, from_dev_bf16, to_dev_bf16
from oracle import fp8_oracle as O
from test_gpu_norm import BWD_K, ROW_Q, _dev_gamma, _gamma, _rounds_from, check_copies
from workloads import bf16_bits_from_f32, bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

EPS = 1e-5
KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]


def _np(t):
    return t.cpu().numpy()


def _cuda(a):
    return None if a is None else torch.from_numpy(np.ascontiguousarray(a)).cuda()


def _kept(bits, ckpt):
    """What the backward pass is given of an activation, and its values."""
    if not ckpt:
        return to_dev_bf16(bits), O.bf16_to_f32(bits).astype(np.float64)
    codes, scale = O.checkpoint_pack(bits)
    return F.Checkpoint(_cuda(codes), _cuda(scale)), O.checkpoint_values(codes, scale)


def case(rows, cols, post=True, gate=True, token=False, ckpt=(True, True), dres=True, fp32=False,
         scale=0.3, seed=0):
    c = dict(rows=rows, cols=cols, scale=scale, fp32=fp32)
    c["dy"] = bf16_bits_normal(rows, cols, seed=seed, sigma=1e-2)
    c["dres"] = bf16_bits_normal(rows, cols, seed=seed + 1, sigma=1e-2) if dres else None
    h = bf16_bits_normal(rows, cols, seed=seed + 2, outlier_p=1e-3)
    o = bf16_bits_normal(rows, cols, seed=seed + 3, sigma=3.0, outlier_p=1e-3)
    c["h"], c["hv"] = _kept(h, ckpt[0])
    c["o"], c["ov"] = _kept(o, ckpt[1])
    c["rstd"] = O.rmsnorm_rstd_f64(O.bf16_to_f32(h), EPS).astype(np.float32)
    c["ro"] = O.rmsnorm_rstd_f64(O.bf16_to_f32(o), EPS).astype(np.float32) if post else None
    c["gamma"] = _gamma(cols, fp32)
    c["a"] = _gamma(cols, fp32, seed=10) if post else None
    c["g"] = O.bf16_to_f32(bf16_bits_from_f32(_gamma(cols, seed=11) - np.float32(1))) if gate \
        else None
    t = np.random.default_rng(12).random(rows, dtype=np.float32) if token else None
    if token:
        t[1::5] = 0
    c["t"] = t
    return c


def run(c, **kw):
    return F.branch_rmsnorm_bwd(
        to_dev_bf16(c["dy"]), c["h"], _cuda(c["rstd"]), _dev_gamma(c["gamma"], c["fp32"]), c["o"],
        rstd_branch=_cuda(c["ro"]), gamma_post=None if c["a"] is None else _dev_gamma(c["a"],
                                                                                     c["fp32"]),
        gate=None if c["g"] is None else _dev_gamma(c["g"], False), token_gate=_cuda(c["t"]),
        scale=c["scale"], dres=None if c["dres"] is None else to_dev_bf16(c["dres"]), **kw)


def check(c, d=None):
    d = run(c) if d is None else d
    torch.cuda.synchronize()
    rows = c["rows"]
    dy = O.bf16_to_f32(c["dy"]).astype(np.float64)
    dres = None if c["dres"] is None else O.bf16_to_f32(c["dres"])
    s32 = float(np.float32(c["scale"]))
    dh, dgamma = O.rmsnorm_bwd_f64(dy, c["hv"], c["rstd"], c["gamma"], dres)
    ref = O.branch_bwd_f64(dh, c["ov"], c["ro"], c["a"], c["g"], c["t"], s32)

    r = c["rstd"][:, None].astype(np.float64)
    xh, a = c["hv"] * r, dy * c["gamma"]
    e = r * (np.abs(a) + np.abs(xh) * np.mean(np.abs(a * xh), 1, keepdims=True))
    e = BWD_K * (e if dres is None else e + np.abs(dres))
    assert _rounds_from(d.dh, dh, e)
    order = (rows + 70) * 2.0 ** -24
    assert np.all(np.abs(_np(d.dgamma) - dgamma) <= order * np.sum(np.abs(dy * xh), 0))

    one = np.ones((1, 1))
    post, gate = (one if v is None else v[None, :].astype(np.float64) for v in (c["a"], c["g"]))
    t, ro = (one if v is None else v[:, None].astype(np.float64) for v in (c["t"], c["ro"]))
    w, xo = s32 * post * gate, np.abs(c["ov"] * ro)
    u, eu = np.abs(dh * w), np.abs(w) * e
    tol = eu + BWD_K * u
    if c["a"] is not None:
        tol = tol + xo * np.mean(eu * xo + BWD_K * u * xo, 1, keepdims=True)
    assert _rounds_from(d.dbranch, ref["dbranch"], ro * np.abs(t) * tol)
    sums = order * np.sum(t * np.abs(dh) * xo, 0) + np.sum(t * xo * e, 0)
    for name, there, factor in (("dgamma_post", c["a"], gate), ("dgate", c["g"], post)):
        got = getattr(d, name)
        assert (got is None) == (there is None)
        if got is not None:
            assert np.all(np.abs(_np(got) - ref[name]) <= np.abs(s32 * factor[0]) * sums)
    assert (d.dtoken_gate is None) == (c["t"] is None)
    if c["t"] is not None:
        tol = np.sum(eu * xo + BWD_K * u * xo, 1)
        assert np.all(np.abs(_np(d.dtoken_gate) - ref["dtoken_gate"]) <= tol)
        assert not d.dbranch[1::5].any()
    return d


SIZES = [(1, 16), (1, 4096), (2, 48), (37, 128), (333, 1552), (700, 4096), (64, 5120), (100, 8192),
         (50, 8208), (65, 16384), (9, 32768), (5, 16400)]


@pytest.mark.parametrize("rows,cols", SIZES)
@pytest.mark.parametrize("ckpt", [(True, True), (False, False), (True, False), (False, True)])
def test_backward(rows, cols, ckpt):
    check(case(rows, cols, ckpt=ckpt))
    check(case(rows, cols, ckpt=ckpt, dres=False, token=True, fp32=True))


@pytest.mark.parametrize("post,gate,token", [(True, False, False), (True, True, True),
                                             (False, True, False), (False, True, True),
                                             (False, False, False), (False, False, True)])
@pytest.mark.parametrize("rows,cols", [(3, 128), (620, 1040), (77, 4096), (20, 16384),
                                       (6, 32768)])
def test_forms(rows, cols, post, gate, token):
    for ckpt in ((True, True), (False, False)):
        check(case(rows, cols, post, gate, token, ckpt))


@pytest.mark.parametrize("rows,cols", [(5000, 256), (1300, 96), (5000, 2064), (6000, 1024),
                                       (1500, 4096), (800, 8192), (330, 16384), (350, 32768),
                                       (160, 16400)])
@pytest.mark.parametrize("ckpt", [(True, True), (False, False)])
def test_many_rows(rows, cols, ckpt):
    """A group of threads walks several rows."""
    check(case(rows, cols, ckpt=ckpt, token=True))


@pytest.mark.parametrize("rows,cols", [(1, 4624), (170, 4864), (700, 5104), (2, 5120), (400, 5120),
                                       (200, 5136)])
@pytest.mark.parametrize("ckpt", [(True, True), (False, False), (True, False), (False, True)])
def test_widths_around_5120(rows, cols, ckpt):
    """Groups of more than 512 threads (4624 to 5120 columns), whole and ragged, and the next width."""
    check(case(rows, cols, ckpt=ckpt, token=True))
    check(case(rows, cols, post=False, ckpt=ckpt, dres=False))


def test_against_differences():
    """dbranch, dh and dtoken_gate along directions against central differences of the formulas."""
    rows, cols = 24, 512
    c = case(rows, cols, ckpt=(False, False), token=True, dres=False)
    rng = np.random.default_rng(3)
    res = rng.standard_normal((rows, cols))
    dy, o, t = O.bf16_to_f32(c["dy"]).astype(np.float64), c["ov"], c["t"].astype(np.float64)

    def stream(b, t, res):
        return O.branch_sum_f64(b, res, O.rmsnorm_rstd_f64(b, EPS), c["a"], c["g"], t, c["scale"])

    def loss(b, t, res):
        return np.sum(dy * O.rmsnorm_f64(stream(b, t, res), c["gamma"], EPS))

    hb = O.f64_to_bf16(stream(o, t, res))              # the stream as it is stored
    res = res + (O.bf16_to_f32(hb) - stream(o, t, res))
    c["h"], c["hv"] = _kept(hb, False)
    c["rstd"] = O.rmsnorm_rstd_f64(c["hv"], EPS).astype(np.float32)
    d = run(c)
    torch.cuda.synchronize()
    e = 1e-5
    for got, at in ((d.dbranch, 0), (d.dtoken_gate, 1), (d.dh, 2)):
        got = got.double().cpu().numpy()
        v = rng.standard_normal(got.shape)
        lo, hi = [o, t, res], [o, t, res]
        lo[at], hi[at] = lo[at] - e * v, hi[at] + e * v
        diff = (loss(*hi) - loss(*lo)) / (2 * e)
        # the outputs' roundings to bf16 (half a step: 2^-8), float32's of their terms
        assert abs(np.sum(got * v) - diff) <= np.sum(np.abs(v) * (2.0 ** -8 * np.abs(got) + 1e-5))


def test_outputs_in_place_strides_and_padding():
    rows, cols = 75, 640
    wide = to_dev_bf16(bf16_bits_normal(rows, 4 * cols + 24, seed=3))
    dy, dres, h, o = (wide[:, i * (cols + 8):i * (cols + 8) + cols] for i in range(4))
    c = case(rows, cols, token=True)
    args = dict(rstd_branch=_cuda(c["ro"]), gamma_post=_dev_gamma(c["a"], False),
                gate=_dev_gamma(c["g"], False), token_gate=_cuda(c["t"]))
    rstd, gamma = _cuda(c["rstd"]), _dev_gamma(c["gamma"], False)

    def call(dy, dres, h, o, **kw):
        return F.branch_rmsnorm_bwd(dy, h, rstd, gamma, o, dres=dres, **args, **kw)

    ref = call(dy, dres, h, o)
    tight = [t.contiguous() for t in (dy, dres, h, o)]
    padded = torch.full((128, cols), float("nan"), dtype=torch.bfloat16, device="cuda")
    padded[:rows] = dy
    got = [call(*tight), call(padded, *tight[1:])]
    for i, j in ((0, 1), (1, 0), (2, 3), (3, 2), (1, 3)):
        t = [x.clone() for x in tight]
        got.append(call(*t, dh=t[i], dbranch=t[j]))
    torch.cuda.synchronize()
    for g in got:
        assert all(torch.equal(a, b) for a, b in zip(ref, g))
    same = tight[0].clone()
    with pytest.raises(F._lib.Fp8Error):
        call(*tight, dh=same, dbranch=same)


@pytest.mark.parametrize("cols", [48, 1024, 4096, 16384, 32768])
def test_tokens_that_pass_by(cols):
    """A token gate of 0: NaN and infinities in its row of branch reach its own dtoken_gate alone."""
    rows = 23
    c = case(rows, cols, ckpt=(False, False), token=True)
    o = from_dev_bf16(c["o"]).copy()
    o[1], o[6, 3], o[11] = 0x7FC0, 0x7F80, 0
    c["ro"][11] = np.inf
    ref = run(c)
    c["o"] = to_dev_bf16(o)
    c["ro"][1] = np.nan
    d = run(c)
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(ref[:5], d[:5]))
    assert bool(torch.isfinite(d.dbranch.float()).all()) and bool(torch.isfinite(d.dgate).all())
    keep = torch.ones(rows, dtype=torch.bool, device="cuda")
    keep[[1, 6, 11]] = False
    assert torch.equal(ref.dtoken_gate[keep], d.dtoken_gate[keep])
    assert bool(torch.isnan(d.dtoken_gate[1]))


def test_empty_and_partial_outputs():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    one, none = torch.ones(256, device="cuda"), torch.empty(0, device="cuda")
    d = F.branch_rmsnorm_bwd(e, e, none, one, e, rstd_branch=none, gamma_post=one, gate=one,
                             token_gate=none, dgamma=one * 3, dgamma_post=one * 3, dgate=one * 3)
    assert not (d.dgamma.any() or d.dgamma_post.any() or d.dgate.any())
    c = case(130, 384, token=True)
    full, part = run(c), run(c, want_dgamma=False)
    torch.cuda.synchronize()
    assert part.dgamma is None and part.dgamma_post is None and part.dgate is None
    assert torch.equal(full.dh, part.dh) and torch.equal(full.dbranch, part.dbranch)
    assert torch.equal(full.dtoken_gate, part.dtoken_gate)


def test_equal_calls_give_equal_bits_on_any_stream_and_in_graphs():
    c = case(200, 512, token=True)
    a = run(c)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = run(c, stream=side)
    side.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(a, b))
    ws = torch.empty(F.branch_rmsnorm_bwd_workspace_bytes(200, 512), dtype=torch.uint8,
                     device="cuda")
    dev = dict(dy=to_dev_bf16(c["dy"]), rstd=_cuda(c["rstd"]),
               gamma=_dev_gamma(c["gamma"], False), rstd_branch=_cuda(c["ro"]),
               gamma_post=_dev_gamma(c["a"], False), gate=_dev_gamma(c["g"], False),
               token_gate=_cuda(c["t"]), dres=to_dev_bf16(c["dres"]))
    outs = [torch.empty_like(t) for t in a]
    graphs = []
    for _ in range(2):                                  # two graphs share the workspace, in turn
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            F.branch_rmsnorm_bwd(h=c["h"], branch=c["o"], scale=c["scale"], workspace=ws,
                                 dh=outs[0], dbranch=outs[1], dgamma=outs[2],
                                 dgamma_post=outs[3], dgate=outs[4], dtoken_gate=outs[5], **dev)
        graphs.append(graph)
    for graph in graphs:
        for t in outs:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a, outs))


@pytest.mark.parametrize("cols", [2064, 16400, 32768])
def test_graph_of_ragged_and_wide_rows(cols):
    """Groups with whole and ragged warps, and clusters, captured and replayed."""
    c = case(37, cols, token=True)
    ref = check(c)
    dev = dict(dy=to_dev_bf16(c["dy"]), rstd=_cuda(c["rstd"]),
               gamma=_dev_gamma(c["gamma"], False), rstd_branch=_cuda(c["ro"]),
               gamma_post=_dev_gamma(c["a"], False), gate=_dev_gamma(c["g"], False),
               token_gate=_cuda(c["t"]), dres=to_dev_bf16(c["dres"]))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        d = F.branch_rmsnorm_bwd(h=c["h"], branch=c["o"], scale=c["scale"], **dev)
    for _ in range(2):
        for t in d:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(ref, d))


def test_offsets_past_32_bits():
    cols, rows = 32768, (1 << 31) // 32768 + 3
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = bf16_bits_normal(3, cols, seed=3)
    x[-3:] = to_dev_bf16(tail)
    ck = F.checkpoint(x)
    f = O.bf16_to_f32(tail).astype(np.float64)
    v = O.checkpoint_values(*O.checkpoint_pack(tail))
    one = torch.ones(cols, device="cuda")
    rstd = torch.ones(rows, device="cuda")
    d = F.branch_rmsnorm_bwd(x, ck, rstd, one, ck, rstd_branch=rstd, gamma_post=one, dres=x)
    torch.cuda.synchronize()
    ones, r = np.ones(cols), np.ones(3)
    dh, dgamma = O.rmsnorm_bwd_f64(f, v, r, ones, f)
    ref = O.branch_bwd_f64(dh, v, r, ones)
    big = np.max(np.abs(dh))
    size = BWD_K * 8 * (1 + big) ** 3                   # generous: terms are products of three
    assert _rounds_from(d.dh[-3:], dh, size) and _rounds_from(d.dbranch[-3:], ref["dbranch"], size)
    assert not d.dh[:-3].any() and not d.dbranch[:-3].any()
    assert np.all(np.abs(_np(d.dgamma) - dgamma) <= (rows + 70) * 2.0 ** -24
                  * np.sum(np.abs(f * v), 0))


@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 384), (45, 4096), (3, 16400)])
def test_nothing_written_outside(rows, cols):
    guard, held = 4096, []

    def between(t):
        n = t.numel() * t.element_size()
        big = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        held.append((big, n))
        view = big[guard:guard + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view

    c = case(rows, cols, token=True)
    d = run(c)
    outs = {k: between(torch.zeros_like(getattr(d, k))) for k in d._fields}
    ws = between(torch.zeros(F.branch_rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8,
                             device="cuda"))
    check(c, run(c, workspace=ws, **outs))
    for big, n in held:
        assert bool((big[:guard] == 0x5A).all()) and bool((big[guard + n:] == 0x5A).all())


# ---------------------------------------------------------------------------- the norm alone

@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (2, 48), (37, 128), (333, 1552),
                                       (700, 4096), (5000, 4096), (64, 5120), (100, 8192),
                                       (330, 16384), (9, 32768), (350, 32768), (5000, 256),
                                       (5000, 528)])
@pytest.mark.parametrize("dres", [True, False])
def test_norm_backward_from_a_checkpoint(rows, cols, dres):
    c = case(rows, cols, dres=dres)
    dr = None if c["dres"] is None else to_dev_bf16(c["dres"])
    dy, rstd, gamma = to_dev_bf16(c["dy"]), _cuda(c["rstd"]), _dev_gamma(c["gamma"], False)
    dh, dgamma = F.rmsnorm_bwd(dy, c["h"], rstd, gamma, dres=dr)
    torch.cuda.synchronize()
    f = O.bf16_to_f32(c["dy"]).astype(np.float64)
    res = None if dr is None else O.bf16_to_f32(c["dres"])
    ref, ref_g = O.rmsnorm_bwd_f64(f, c["hv"], c["rstd"], c["gamma"], res)
    r = c["rstd"][:, None].astype(np.float64)
    xh, t = c["hv"] * r, f * c["gamma"]
    size = r * (np.abs(t) + np.abs(xh) * np.mean(np.abs(t * xh), 1, keepdims=True))
    assert _rounds_from(dh, ref, BWD_K * (size if res is None else size + np.abs(res)))
    assert np.all(np.abs(_np(dgamma) - ref_g)
                  <= (rows + 70) * 2.0 ** -24 * np.sum(np.abs(f * xh), 0))
    # the checkpoint's values in bf16, which are exact, give the same bits
    same = F.rmsnorm_bwd(dy, F.checkpoint_read(c["h"]), rstd, gamma, dres=dr)
    torch.cuda.synchronize()
    assert torch.equal(dh, same[0]) and torch.equal(dgamma, same[1])


# ---------------------------------------------------------------------------- copies

def check_requantize(kind, rows, cols, norm, row, col, margin=0, pow2=False, fp32=False, seed=0):
    x = bf16_bits_normal(rows, cols, seed=seed, outlier_p=1e-3)
    ck, v = _kept(x, True)
    rstd = O.rmsnorm_rstd_f64(O.bf16_to_f32(x), EPS).astype(np.float32) if norm else None
    gamma = _gamma(cols, fp32) if norm else None
    rec = F.Recipe(kind=kind, margin=margin, power_2_scales=pow2)
    q = F.empty_qtensor(rec, -(-rows // ROW_Q[kind]) * ROW_Q[kind], cols, "activation", row, col)
    for t in (q.row, q.col):
        if t is not None:
            t.fill_(0xA5)
    scale = None
    if kind == "delayed":
        scale = np.float32(7.3)
        q.scale.fill_(float(scale))
        q.scale_inv.fill_(float(np.float32(1) / scale))
    out = F.checkpoint_quantize(rec, ck, _cuda(rstd),
                                None if gamma is None else _dev_gamma(gamma, fp32), want_row=row,
                                want_col=col, out=q)
    torch.cuda.synchronize()
    y = v.astype(np.float32)
    if norm:
        y = (y * rstd[:, None]) * gamma
    check_copies(out, y, kind, scale, margin, pow2, row, col)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 4096), (129, 1280), (257, 640), (1000, 2048),
                                       (33, 8192), (40, 16384), (2048, 4096), (160, 32768)])
@pytest.mark.parametrize("norm", [True, False])
def test_requantize(kind, rows, cols, norm):
    check_requantize(kind, rows, cols, norm, True, True)
    check_requantize(kind, rows, cols, norm, False, True)
    check_requantize(kind, rows, cols, norm, True, False)


@pytest.mark.parametrize("kind", ["tensorwise", "delayed"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (17, 48), (77, 2064), (250, 144), (15, 8208),
                                       (9000, 16)])
def test_requantize_ragged(kind, rows, cols):
    for norm in (True, False):
        check_requantize(kind, rows, cols, norm, True, True)
        check_requantize(kind, rows, cols, norm, False, True)
        check_requantize(kind, rows, cols, norm, True, False)


def test_requantize_options():
    check_requantize("blockwise", 200, 512, True, True, True, pow2=True)
    check_requantize("blockwise", 200, 512, False, True, True, margin=3)
    check_requantize("tensorwise", 200, 512, True, True, True, margin=-2, fp32=True)
    for kind in KINDS:                                  # --fp8-wgrad off: bf16(y) transposed
        x = bf16_bits_normal(130, 384, seed=4)
        ck, v = _kept(x, True)
        q = F.checkpoint_quantize(F.Recipe(kind=kind, fp8_wgrad=False), ck)
        torch.cuda.synchronize()
        y = np.zeros((q.rows, 384), dtype=np.float32)
        y[:130] = v
        assert np.array_equal(from_dev_bf16(q.col),
                              bf16_bits_from_f32(np.ascontiguousarray(y.T)))
        check_copies(q, y[:130], kind, scale=1.0, col=False)


def test_requantize_is_the_norms_of_the_values():
    """The copies of rmsnorm_quantize of the checkpoint's own values, byte for byte."""
    rec, rows, cols = F.Recipe(kind="mxfp8"), 700, 2048
    ck = F.checkpoint(to_dev_bf16(bf16_bits_normal(rows, cols, seed=1)))
    gamma = _dev_gamma(_gamma(cols), False)
    a, _, rstd, _ = F.rmsnorm_quantize(rec, F.checkpoint_read(ck), gamma)
    b = F.checkpoint_quantize(rec, ck, rstd, gamma)
    torch.cuda.synchronize()
    for f in ("row", "col", "row_scale", "col_scale"):
        assert torch.equal(getattr(a, f), getattr(b, f))


def test_requantize_special_values_and_negative_gamma():
    x = bf16_bits_normal(131, 256, seed=6)
    x[2, 40], x[5] = 0x7FC0, 0
    ck = F.checkpoint(to_dev_bf16(x))
    gamma = torch.randn(256, generator=torch.Generator().manual_seed(1)).cuda()
    q = F.checkpoint_quantize(F.Recipe(kind="mxfp8"), ck, torch.ones(131, device="cuda"), gamma)
    torch.cuda.synchronize()
    row, col = _np(q.row), _np(q.col)
    assert (row[2, 32:64] == 0x7F).all() and not (row[2, :32] == 0x7F).any()
    assert (col[32:64, 2] == 0x7F).all()
    assert not (row[5] & 0x7F).any()
    assert not row[131:].any() and not col[:, 131:].any()       # padding: +0
    e = F.Checkpoint(ck.codes[:0], ck.scale[:0])
    q = F.checkpoint_quantize(F.Recipe(kind="tensorwise"), e)
    torch.cuda.synchronize()
    assert q.rows == 0 and (q.amax.item(), q.scale.item(), q.scale_inv.item()) == (0.0, 1.0, 1.0)

"""GPU parity of the residual add + RMSNorm + quantize kernels and of the norm's backward.

Codes and scales are compared exactly: the oracle's quantiser is applied to the value that the
library defines, (h rstd) gamma in float32, with the GPU's own h and rstd, which are themselves
compared with the oracle (h exactly). Tolerances follow from the number of float32 additions:

  rstd  a row's squares are added in chains of at most 64 per thread, then 5 shuffles and 16
        warps; half of that relative error reaches rstd, plus the division, eps and root:
        (64 + 21) / 2 + 3 = 46 roundings of 2^-24 each, below RSTD_RTOL.
  dh    before its rounding to bf16 within BWD_K (100 float32 roundings) of the terms' sizes;
        rounding is monotonic, so the result lies between the roundings of those two ends.
  dgamma at most rows + 70 additions a column, of |dy xh| each.
"""
import numpy as np
import pytest
import torch

from helpers import bw_untile, cuda_ok, from_dev_bf16, mx_untile, same_f32, to_dev_bf16
from oracle import fp8_oracle as O
from workloads import bf16_bits_from_f32, bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

EPS = 1e-5
RSTD_RTOL = 3e-6
BWD_K = 100 * 2.0 ** -24
ROW_Q = {"mxfp8": 128, "blockwise": 128, "tensorwise": 16, "delayed": 16}


def _np(t):
    return t.cpu().numpy()


def _gamma(cols, fp32=False, seed=9):
    g = 1 + 0.2 * np.random.default_rng(seed).standard_normal(cols).astype(np.float32)
    return g if fp32 else O.bf16_to_f32(bf16_bits_from_f32(g))


def _dev_gamma(g, fp32):
    t = torch.from_numpy(g).cuda()
    return t if fp32 else t.to(torch.bfloat16)


def _check_scales(q, name, ref, rows, cols, kind, pow2):
    got = _np(getattr(q, name))
    if kind == "mxfp8":
        assert np.array_equal(mx_untile(got, rows, cols), ref[name])
    elif pow2:
        assert np.array_equal(mx_untile(got, rows, cols),
                              O.pow2_scales_as_e8m0(ref[name + "_inv"], 1, rows, cols))
    else:
        assert np.array_equal(bw_untile(got, rows, cols), ref[name + "_inv"])


def check_copies(q, y, kind, scale=None, margin=0, pow2=False, row=True, col=True):
    """The copies of q against the oracle's quantisation of y (float32, padded here)."""
    rows = -(-y.shape[0] // ROW_Q[kind]) * ROW_Q[kind]
    yp = np.zeros((rows, y.shape[1]), dtype=np.float32)
    yp[:y.shape[0]] = y
    assert (q.rows, q.cols) == yp.shape
    if kind == "mxfp8":
        ref = O.quantize_mxfp8(yp)
    elif kind == "blockwise":
        ref = O.quantize_blockwise_1x128(yp, margin, pow2=pow2)
    elif kind == "tensorwise":
        ref = O.quantize_tensorwise(yp, margin)
    else:
        d = O.DelayedScaling(4)
        d.scale = np.float32(scale)
        ref = d.quantize(yp)
    if row:
        assert np.array_equal(_np(q.row), ref["row"])
        if kind in ("mxfp8", "blockwise"):
            _check_scales(q, "row_scale", ref, rows, y.shape[1], kind, pow2)
    if col:
        assert np.array_equal(_np(q.col), ref["col"])
        if kind in ("mxfp8", "blockwise"):
            _check_scales(q, "col_scale", ref, y.shape[1], rows, kind, pow2)
    if kind in ("tensorwise", "delayed"):
        assert same_f32(_np(q.amax)[0], ref["amax"])
    if kind == "tensorwise":
        assert same_f32(_np(q.scale)[0], ref["scale"])
        assert same_f32(_np(q.scale_inv)[0], ref["scale_inv"])


def check_norm(kind, rows, cols, residual=True, row=True, col=True, gamma_fp32=False, margin=0,
               pow2=False, x_bits=None, eps=EPS, seed=0, want_y=False):
    x = bf16_bits_normal(rows, cols, seed=seed, outlier_p=1e-3) if x_bits is None else x_bits
    res = bf16_bits_normal(rows, cols, seed=seed + 1, sigma=2.0) if residual else None
    g = _gamma(cols, gamma_fp32)
    rec = F.Recipe(kind=kind, margin=margin, power_2_scales=pow2)
    q = F.empty_qtensor(rec, -(-rows // ROW_Q[kind]) * ROW_Q[kind], cols, "activation", row, col)
    for t in (q.row, q.col):                    # whatever was there before is overwritten
        if t is not None:
            t.fill_(0xA5)
    scale = None
    if kind == "delayed":
        scale = np.float32(7.3)
        q.scale.fill_(float(scale))
        q.scale_inv.fill_(float(np.float32(1) / scale))
    out, h, rstd, y = F.rmsnorm_quantize(
        rec, to_dev_bf16(x), _dev_gamma(g, gamma_fp32),
        residual=None if res is None else to_dev_bf16(res), eps=eps, want_row=row, want_col=col,
        want_y=want_y, out=q)
    torch.cuda.synchronize()
    hb = from_dev_bf16(h)
    assert np.array_equal(hb, x if res is None else O.residual_add_bf16(x, res))
    ref = O.rmsnorm_rstd_f64(O.bf16_to_f32(hb), eps)
    r = _np(rstd)
    assert np.max(np.abs(r - ref) / ref) <= RSTD_RTOL
    y32 = O.rmsnorm_y_f32(hb, r, g)
    check_copies(out, y32, kind, scale, margin, pow2, row, col)
    if want_y:
        assert np.array_equal(from_dev_bf16(y), bf16_bits_from_f32(y32))
    return out


KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 4096), (128, 256), (129, 1280), (257, 640),
                                       (1000, 2048), (640, 4096), (33, 8192), (40, 16384),
                                       (160, 32768)])
def test_both_copies(kind, rows, cols):
    check_norm(kind, rows, cols)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 4096), (2, 128), (31, 8192), (200, 1024), (5, 16384),
                                       (7, 32768), (700, 4096)])
def test_row_copy_alone(kind, rows, cols):
    check_norm(kind, rows, cols, col=False)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,residual", [(1500, 4096, False), (1500, 512, True),
                                                (2500, 128, True), (300, 32768, False)])
def test_many_rows(kind, rows, cols, residual):
    """More rows than run at once, so that a group of threads walks several."""
    check_norm(kind, rows, cols, residual=residual)


@pytest.mark.parametrize("kind", KINDS)
def test_column_copy_alone_without_residual(kind):
    check_norm(kind, 300, 1152, residual=False, row=False)


@pytest.mark.parametrize("kind", ["tensorwise", "delayed"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (17, 48), (77, 2064), (250, 144), (15, 8208)])
def test_per_tensor_ragged(kind, rows, cols):
    check_norm(kind, rows, cols, residual=False)
    check_norm(kind, rows, cols, col=False)


@pytest.mark.parametrize("col", [False, True])
def test_options(col):
    check_norm("blockwise", 200, 512, pow2=True, col=col)
    check_norm("blockwise", 200, 512, margin=3, col=col)
    check_norm("tensorwise", 200, 512, margin=-2, col=col)
    check_norm("mxfp8", 200, 512, gamma_fp32=True, want_y=True, col=col)
    check_norm("mxfp8", 200, 512, eps=0.5, col=col)


def test_bf16_column_copy():
    """--fp8-wgrad off: the column copy is bf16(y) transposed."""
    for kind in KINDS:
        rec = F.Recipe(kind=kind, fp8_wgrad=False)
        x = bf16_bits_normal(130, 384, seed=4)
        g = _gamma(384)
        rows = -(-130 // ROW_Q[kind]) * ROW_Q[kind]
        q = F.empty_qtensor(rec, rows, 384, "activation")
        q, h, rstd, _ = F.rmsnorm_quantize(rec, to_dev_bf16(x), _dev_gamma(g, False), out=q)
        torch.cuda.synchronize()
        y = np.zeros((rows, 384), dtype=np.float32)
        y[:130] = O.rmsnorm_y_f32(x, _np(rstd), g)
        assert q.col_bf16 == 1
        assert np.array_equal(from_dev_bf16(q.col), bf16_bits_from_f32(np.ascontiguousarray(y.T)))
        check_copies(q, y[:130], kind, scale=1.0, col=False)


def test_special_values():
    """Zero rows, a NaN, an infinity, subnormals and the largest magnitudes a square holds."""
    x = bf16_bits_normal(256, 512, seed=6)
    x[0] = 0
    x[1, 7] = 0x7FC0
    x[2, 300] = 0x7F80
    x[3] = 0x0001
    x[4, ::3] = bf16_bits_from_f32(np.float32([1e18]))[0]
    x[5] = 0x8000
    g = _gamma(512)
    for kind in KINDS:
        rec = F.Recipe(kind=kind)
        q = F.empty_qtensor(rec, 256, 512, "activation")
        q, _, rstd, y = F.rmsnorm_quantize(rec, to_dev_bf16(x), _dev_gamma(g, False), want_y=True,
                                           out=q)
        torch.cuda.synchronize()
        r, yb = _np(rstd), y.float().cpu().numpy()
        assert np.isnan(yb[1]).all()                     # NaN reaches its whole row
        assert np.isnan(yb[2, 300]) and not np.delete(yb[2], 300).any()     # inf * 0, v * 0
        assert not yb[0].any() and not yb[5].any()
        assert np.isfinite(np.delete(yb, (1, 2), axis=0)).all()
        assert np.array_equal(np.isnan(r), np.arange(256) == 1)
        row = _np(q.row)
        assert (row[1] == 0x7F).all() and row[2, 300] == 0x7F
        if kind in ("mxfp8", "blockwise"):               # clean rows are quantised as ever
            y32 = O.rmsnorm_y_f32(x, r, g)
            keep = np.setdiff1d(np.arange(256), (1, 2))
            ref = (O.quantize_mxfp8(y32[keep], want_col=False)["row"] if kind == "mxfp8"
                   else O.quantize_blockwise_1x128(y32)["row"][keep])
            assert np.array_equal(row[keep], ref)
        if kind == "mxfp8":
            e = mx_untile(_np(q.row_scale), 256, 512)
            assert (e[1] == 0xFF).all() and e[2, 300 // 32] == 0xFF and (e[0] == 0).all()


def test_bf16_output_alone():
    for rows, cols in [(1, 16), (5, 128), (333, 2064), (2, 32768)]:
        x = bf16_bits_normal(rows, cols, seed=rows)
        res = bf16_bits_normal(rows, cols, seed=rows + 1)
        g = _gamma(cols)
        y, h, rstd = F.rmsnorm(to_dev_bf16(x), _dev_gamma(g, False), to_dev_bf16(res))
        torch.cuda.synchronize()
        hb = from_dev_bf16(h)
        assert np.array_equal(hb, O.residual_add_bf16(x, res))
        assert np.array_equal(from_dev_bf16(y),
                              bf16_bits_from_f32(O.rmsnorm_y_f32(hb, _np(rstd), g)))


def test_strided_inputs_and_in_place():
    rows, cols = 75, 640
    wide = to_dev_bf16(bf16_bits_normal(rows, 2 * cols + 8, seed=3))
    x, res = wide[:, :cols], wide[:, cols + 8:]
    g = _dev_gamma(_gamma(cols), False)
    for kind in ("mxfp8", "delayed"):
        rec = F.Recipe(kind=kind)
        a = F.rmsnorm_quantize(rec, x, g, residual=res)
        b = F.rmsnorm_quantize(rec, x.contiguous(), g, residual=res.contiguous())
        stream = res.contiguous()                       # h written over the residual
        c = F.rmsnorm_quantize(rec, x, g, residual=stream, h=stream)
        d = F.rmsnorm_quantize(rec, a[1], g)            # the stream already added, no residual
        e = F.rmsnorm_quantize(rec, torch.cat([a[1], a[1]], 1)[:, :cols], g)
        torch.cuda.synchronize()
        for other in (b, c, d, e):
            assert torch.equal(a[0].row, other[0].row) and torch.equal(a[0].col, other[0].col)
            assert torch.equal(a[1], other[1]) and torch.equal(a[2], other[2])
    dy, dres = wide[:, 8:cols + 8], res
    a = F.rmsnorm_bwd(dy, x, b[2], g, dres=dres)
    b2 = F.rmsnorm_bwd(dy.contiguous(), x.contiguous(), b[2], g, dres=dres.contiguous())
    over = dres.contiguous()
    c = F.rmsnorm_bwd(dy, x, b[2], g, dres=over, dh=over)
    over2 = dy.contiguous()
    d = F.rmsnorm_bwd(over2, x, b[2], g, dres=dres, dh=over2)
    torch.cuda.synchronize()
    for other in (b2, c, d):
        assert torch.equal(a[0], other[0]) and torch.equal(a[1], other[1])


def test_empty():
    for kind in KINDS:
        rec = F.Recipe(kind=kind)
        q = F.empty_qtensor(rec, 0, 256, "activation")
        x = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
        q, _, rstd, _ = F.rmsnorm_quantize(rec, x, torch.ones(256, device="cuda"), out=q)
        torch.cuda.synchronize()
        assert q.rows == 0 and rstd.numel() == 0
        if kind == "tensorwise":
            assert (q.amax.item(), q.scale.item(), q.scale_inv.item()) == (0.0, 1.0, 1.0)
    dgamma = torch.full((256,), 3.0, device="cuda")
    F.rmsnorm_bwd(x, x, torch.empty(0, device="cuda"), torch.ones(256, device="cuda"),
                  dgamma=dgamma)
    assert not dgamma.any()


def test_feeds_the_linear_layer():
    """A single token and a ragged batch: the GEMM of the padded copies equals the GEMM of the
    oracle's dequantised operands on the rows that exist, and is zero on the padding."""
    for rows in (1, 37):
        x, w = bf16_bits_normal(rows, 512, seed=8), bf16_bits_normal(256, 512, seed=9, sigma=0.02)
        rec = F.Recipe(kind="mxfp8")
        q, _, rstd, _ = F.rmsnorm_quantize(rec, to_dev_bf16(x), _dev_gamma(_gamma(512), False),
                                           want_col=False)
        wq = F.quantize(rec, to_dev_bf16(w), "weight")
        out = F.linear_fwd(rec, q, wq, fp32=True)
        torch.cuda.synchronize()
        y = O.rmsnorm_y_f32(x, _np(rstd), _gamma(512))
        qy, qw = O.quantize_mxfp8(y, want_col=False), O.quantize_mxfp8(w)
        ref = O.gemm_tn_f64(O.dequant_mx(qy["row"], qy["row_scale"]),
                            O.dequant_mx(qw["row"], qw["row_scale"]))
        got = _np(out)
        assert np.max(np.abs(got[:rows] - ref)) <= 1e-5 * np.max(np.abs(ref))
        assert not got[rows:].any()


# ---------------------------------------------------------------------------- backward

def _rounds_from(t, ref, tol):
    """Whether every element of the bf16 tensor is the rounding of a value within tol of ref."""
    got = O.bf16_to_f32(from_dev_bf16(t))
    return bool(np.all((O.bf16_to_f32(O.f64_to_bf16(ref - tol)) <= got)
                       & (got <= O.bf16_to_f32(O.f64_to_bf16(ref + tol)))))


def check_bwd(rows, cols, dres=True, gamma_fp32=False, seed=0, want_dgamma=True):
    dy = bf16_bits_normal(rows, cols, seed=seed, sigma=1e-2)
    h = bf16_bits_normal(rows, cols, seed=seed + 1, outlier_p=1e-3)
    dr = bf16_bits_normal(rows, cols, seed=seed + 2, sigma=1e-2) if dres else None
    g = _gamma(cols, gamma_fp32)
    hf = O.bf16_to_f32(h)
    rstd = O.rmsnorm_rstd_f64(hf, EPS).astype(np.float32)
    dh, dg = F.rmsnorm_bwd(to_dev_bf16(dy), to_dev_bf16(h), torch.from_numpy(rstd).cuda(),
                           _dev_gamma(g, gamma_fp32), None if dr is None else to_dev_bf16(dr),
                           want_dgamma=want_dgamma)
    torch.cuda.synchronize()
    dyf = O.bf16_to_f32(dy).astype(np.float64)
    drf = None if dr is None else O.bf16_to_f32(dr)
    ref, ref_g = O.rmsnorm_bwd_f64(dyf, hf, rstd, g, drf)
    xh, t = hf * rstd[:, None].astype(np.float64), dyf * g
    size = rstd[:, None] * (np.abs(t) + np.abs(xh) * np.mean(np.abs(t * xh), 1, keepdims=True))
    if drf is not None:
        size = size + np.abs(drf)
    assert _rounds_from(dh, ref, BWD_K * size)
    if want_dgamma:
        tol = (rows + 70) * 2.0 ** -24 * np.sum(np.abs(dyf * xh), 0)
        assert np.all(np.abs(_np(dg) - ref_g) <= tol)
    else:
        assert dg is None


@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (2, 48), (37, 128), (333, 1552),
                                       (700, 4096), (64, 5120), (100, 8192), (50, 8208),
                                       (65, 16384), (9, 32768), (5000, 256)])
def test_backward(rows, cols):
    check_bwd(rows, cols)
    check_bwd(rows, cols, dres=False, gamma_fp32=True)


def test_backward_without_dgamma():
    check_bwd(200, 768, want_dgamma=False)


def test_backward_against_differences():
    """The GPU's dh along a direction against central differences of the oracle's forward."""
    rows, cols = 24, 512
    dy, h = bf16_bits_normal(rows, cols, seed=1), bf16_bits_normal(rows, cols, seed=2)
    g, hf = _gamma(cols), O.bf16_to_f32(h).astype(np.float64)
    rstd = O.rmsnorm_rstd_f64(hf, EPS).astype(np.float32)
    dh, dg = F.rmsnorm_bwd(to_dev_bf16(dy), to_dev_bf16(h), torch.from_numpy(rstd).cuda(),
                           _dev_gamma(g, False))
    torch.cuda.synchronize()
    got, dyf = O.bf16_to_f32(from_dev_bf16(dh)).astype(np.float64), O.bf16_to_f32(dy)
    v = np.random.default_rng(5).standard_normal((rows, cols))
    e = 1e-5

    def loss(a, b):
        return np.sum(dyf * O.rmsnorm_f64(a, b, EPS))

    diff = (loss(hf + e * v, g) - loss(hf - e * v, g)) / (2 * e)
    # dh's roundings to bf16, 2^-9 of an element in the mean (and float32 roundings of its terms)
    assert abs(np.sum(got * v) - diff) <= np.sum(np.abs(v) * (2.0 ** -9 * np.abs(got) + 1e-4))
    w = np.random.default_rng(6).standard_normal(cols)
    diff = (loss(hf, g + e * w) - loss(hf, g - e * w)) / (2 * e)
    tol = np.sum(np.abs(w) * (rows + 70) * 2.0 ** -24 * np.sum(np.abs(dyf * hf), 0)) + 1e-6
    assert abs(np.sum(_np(dg) * w) - diff) <= tol


def test_backward_is_deterministic_and_reads_no_padding():
    """dy with more rows than rstd (the padded tensor's gradient): the rest is not read."""
    rows, cols = 131, 1024
    dy = to_dev_bf16(bf16_bits_normal(256, cols, seed=1))
    dy[rows:] = float("nan")
    h = to_dev_bf16(bf16_bits_normal(rows, cols, seed=2))
    rstd = torch.rand(rows, device="cuda") + 0.5
    g = torch.ones(cols, device="cuda")
    a = F.rmsnorm_bwd(dy, h, rstd, g)
    b = F.rmsnorm_bwd(dy, h, rstd, g)
    torch.cuda.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert bool(torch.isfinite(a[0].float()).all()) and bool(torch.isfinite(a[1]).all())


def test_offsets_past_32_bits():
    """A bf16 norm and its backward of more than 2^31 elements: the last rows."""
    cols, rows = 32768, (1 << 31) // 32768 + 3
    x = torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda")
    x.fill_(1.0)
    tail = bf16_bits_normal(3, cols, seed=3)
    x[-3:] = to_dev_bf16(tail)
    g = _gamma(cols)
    y, _, rstd = F.rmsnorm(x, _dev_gamma(g, False))
    torch.cuda.synchronize()
    assert np.array_equal(from_dev_bf16(y[-3:]),
                          bf16_bits_from_f32(O.rmsnorm_y_f32(tail, _np(rstd[-3:]), g)))
    dh, dgamma = F.rmsnorm_bwd(x, x, rstd, _dev_gamma(g, False), dh=y)
    torch.cuda.synchronize()
    f = O.bf16_to_f32(tail)
    ref, _ = O.rmsnorm_bwd_f64(f, f, _np(rstd[-3:]), g)
    assert _rounds_from(dh[-3:], ref, BWD_K * 4 * (np.abs(f) + np.abs(ref) + 1))
    assert abs(float(dgamma[0]) - rows) < 64               # ones: dy xh = 1 in each row but three


# ---------------------------------------------------------------------------- surroundings

def test_other_stream_and_graph():
    """The calls run on the caller's stream and can be captured; replays give the same bytes."""
    rec = F.Recipe(kind="delayed")
    x, res = (to_dev_bf16(bf16_bits_normal(200, 512, seed=s)) for s in (1, 2))
    dy = to_dev_bf16(bf16_bits_normal(200, 512, seed=3))
    g = _dev_gamma(_gamma(512), False)
    q = F.empty_qtensor(rec, 208, 512, "activation")
    h, dh = torch.empty_like(x), torch.empty_like(x)
    rstd, dgamma = torch.empty(200, device="cuda"), torch.empty(512, device="cuda")
    ws = torch.empty(F.rmsnorm_workspace_bytes(rec, 200, 512), dtype=torch.uint8, device="cuda")
    wb = torch.empty(F.rmsnorm_bwd_workspace_bytes(200, 512), dtype=torch.uint8, device="cuda")
    outs = [q.row, q.col, q.amax, h, rstd, dh, dgamma]

    def step(stream=None):
        F.rmsnorm_quantize(rec, x, g, residual=res, out=q, h=h, rstd=rstd, workspace=ws,
                           stream=stream)
        F.rmsnorm_bwd(dy, h, rstd, g, dh=dh, dgamma=dgamma, workspace=wb, stream=stream)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs]
    side = torch.cuda.Stream()
    for t in outs:
        t.zero_()
    torch.cuda.synchronize()
    step(stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))
    # buffers that the calls make themselves come from the given stream's pool
    mx = F.Recipe(kind="mxfp8")
    a = F.rmsnorm_quantize(mx, x, g, residual=res, want_y=True, stream=side)
    da = F.rmsnorm_bwd(dy, a[1], a[2], g, stream=side)
    side.synchronize()
    b = F.rmsnorm_quantize(mx, x, g, residual=res, want_y=True)
    db = F.rmsnorm_bwd(dy, b[1], b[2], g)
    torch.cuda.synchronize()
    assert all(torch.equal(u, v) for u, v in zip(
        (a[0].row, a[0].col, a[0].row_scale, a[0].col_scale, *a[1:], *da),
        (b[0].row, b[0].col, b[0].row_scale, b[0].col_scale, *b[1:], *db)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in outs:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs, ref))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 384), (45, 4096)])
def test_nothing_written_outside(kind, rows, cols):
    """Every output between canaries: the buffers around it keep their bytes."""
    rec = F.Recipe(kind=kind)
    padded = -(-rows // ROW_Q[kind]) * ROW_Q[kind]
    guard, held = 4096, []

    def between(t):
        n = t.numel() * t.element_size()
        big = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        held.append((big, n))
        view = big[guard:guard + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view

    for want_col in (True, False):
        q = F.empty_qtensor(rec, padded, cols, "activation", True, want_col)
        for f in ("row", "col", "row_scale", "col_scale", "amax", "scale", "scale_inv"):
            if getattr(q, f) is not None:
                setattr(q, f, between(getattr(q, f)))
        x = to_dev_bf16(bf16_bits_normal(rows, cols, seed=1))
        h, y, dh = (between(torch.zeros_like(x)) for _ in range(3))
        rstd = between(torch.zeros(rows, device="cuda"))
        dgamma = between(torch.zeros(cols, device="cuda"))
        ws = between(torch.zeros(F.rmsnorm_workspace_bytes(rec, rows, cols), dtype=torch.uint8,
                                 device="cuda"))
        wb = between(torch.zeros(F.rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8,
                                 device="cuda"))
        g = torch.ones(cols, device="cuda")
        F.rmsnorm_quantize(rec, x, g, residual=x, want_col=want_col, out=q, h=h, rstd=rstd, y=y,
                           workspace=ws)
        F.rmsnorm_bwd(x, h, rstd, g, dres=x, dh=dh, dgamma=dgamma, workspace=wb)
        torch.cuda.synchronize()
        for big, n in held:
            assert bool((big[:guard] == 0x5A).all()) and bool((big[guard + n:] == 0x5A).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,residual", [(300, 8192, True), (300, 5120, True),
                                                (300, 2048, False), (160, 256, True)])
def test_more_rows_than_sms(kind, rows, cols, residual):
    check_norm(kind, rows, cols, residual=residual)


@pytest.mark.parametrize("rows,cols", [(160, 1024), (610, 1040), (1300, 96), (5000, 2064),
                                       (6000, 1024), (5000, 528)])
def test_backward_of_many_rows(rows, cols):
    check_bwd(rows, cols)
    check_bwd(rows, cols, dres=False, gamma_fp32=True)


@pytest.mark.parametrize("cols", [128, 512, 640, 1024, 2176, 2560, 4096, 5120, 16384])
@pytest.mark.parametrize("residual", [False, True])
def test_rows_do_not_depend_on_their_number(cols, residual):
    """A row alone, in a small and in a large batch, and with the residual added before: the same
    bits."""
    rec = F.Recipe(kind="mxfp8")
    x = to_dev_bf16(bf16_bits_normal(700, cols, seed=1))
    res = to_dev_bf16(bf16_bits_normal(700, cols, seed=2)) if residual else None
    g = _dev_gamma(_gamma(cols), False)

    def run(a, b):
        r = None if res is None else res[a:b]
        q, h, rstd, _ = F.rmsnorm_quantize(rec, x[a:b], g, residual=r, want_col=False)
        return q.row[:b - a], h, rstd

    ref = run(0, 700)
    for a, b in ((0, 1), (5, 6), (699, 700), (100, 140), (300, 600)):
        for got, want in zip(run(a, b), ref):
            assert torch.equal(got, want[a:b])
    q, _, rstd, _ = F.rmsnorm_quantize(rec, ref[1], g, want_col=False)
    assert torch.equal(q.row[:700], ref[0]) and torch.equal(rstd, ref[2])

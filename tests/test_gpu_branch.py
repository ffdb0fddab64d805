"""GPU parity of the gated branch with norms before and after it, and of its 8-bit checkpoints.

Codes, scales and checkpoints are compared exactly, given the GPU's own h and rstd; those:

  rstd  as for the norm alone (test_gpu_norm): RSTD_RTOL.
  h     before its rounding to bf16: w = gamma_post gate scale takes two float32 roundings, rstd
        times the token's gate one, the product with branch one and the fused sum one: within
        H_K = 6 roundings of 2^-24 of the term and of the sum. Rounding to bf16 is monotonic, so h
        lies between the roundings of the two ends.
"""
import numpy as np
import pytest
import torch

from helpers import cuda_ok, from_dev_bf16, to_dev_bf16
from oracle import fp8_oracle as O
from test_gpu_norm import ROW_Q, RSTD_RTOL, _dev_gamma, _gamma, _rounds_from, check_copies
from workloads import bf16_bits_from_f32, bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

EPS, EPS_POST = 1e-5, 1e-3
H_K = 6 * 2.0 ** -24
KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]
FORMS = [dict(post=True, gate=True, token=False), dict(post=True, gate=False, token=True),
         dict(post=False, gate=True, token=True), dict(post=False, gate=False, token=False)]


def _np(t):
    return t.cpu().numpy()


def same_checkpoint(ck, bits):
    codes, scale = O.checkpoint_pack(bits)
    return np.array_equal(_np(ck.codes), codes) and np.array_equal(_np(ck.scale), scale)


def filled(rows, cols):
    """A checkpoint's buffers with bytes that the call has to overwrite."""
    ck = F.empty_checkpoint(rows, cols)
    ck.codes.fill_(0xA5)
    ck.scale.fill_(0xA5)
    return ck


def check_branch(kind, rows, cols, post=True, gate=True, token=False, ckpt=True, col=True,
                 scale=0.3, fp32=False, margin=0, pow2=False, want_y=False, seed=0):
    o = bf16_bits_normal(rows, cols, seed=seed, sigma=3.0, outlier_p=1e-3)
    res = bf16_bits_normal(rows, cols, seed=seed + 1, outlier_p=1e-3)
    gamma = _gamma(cols, fp32)
    a = _gamma(cols, fp32, seed=10) if post else None
    g = _gamma(cols, not fp32, seed=11) - np.float32(1) if gate else None
    if g is not None and fp32:                                  # the gate's type is the other one
        g = O.bf16_to_f32(bf16_bits_from_f32(g))
    t = np.random.default_rng(12).random(rows, dtype=np.float32) if token else None
    if token:
        t[::5] = 0
    rec = F.Recipe(kind=kind, margin=margin, power_2_scales=pow2)
    q = F.empty_qtensor(rec, -(-rows // ROW_Q[kind]) * ROW_Q[kind], cols, "activation", True, col)
    for c in (q.row, q.col):
        if c is not None:
            c.fill_(0xA5)
    qscale = None
    if kind == "delayed":
        qscale = np.float32(7.3)
        q.scale.fill_(float(qscale))
        q.scale_inv.fill_(float(np.float32(1) / qscale))
    o_ck, h_ck = (filled(rows, cols), filled(rows, cols)) if ckpt else (None, None)
    out, h, rstd, rstd_o, y = F.branch_rmsnorm_quantize(
        rec, to_dev_bf16(o), to_dev_bf16(res), _dev_gamma(gamma, fp32),
        gamma_post=None if a is None else _dev_gamma(a, fp32),
        gate=None if g is None else _dev_gamma(g, not fp32),
        token_gate=None if t is None else torch.from_numpy(t).cuda(), scale=scale, eps=EPS,
        eps_post=EPS_POST, want_col=col, want_y=want_y, out=q, branch_ckpt=o_ck, h_ckpt=h_ck)
    torch.cuda.synchronize()
    of, rf = O.bf16_to_f32(o), O.bf16_to_f32(res).astype(np.float64)
    ro = None
    if post:
        ref = O.rmsnorm_rstd_f64(of, EPS_POST)
        ro = _np(rstd_o)
        assert np.max(np.abs(ro - ref) / ref) <= RSTD_RTOL
    else:
        assert rstd_o is None
    s32 = np.float32(scale)
    want = O.branch_sum_f64(of, rf, ro, a, g, t, s32)
    assert _rounds_from(h, want, H_K * (np.abs(want - rf) + np.abs(want)))
    hb = from_dev_bf16(h)
    if token:
        assert np.array_equal(hb[::5], res[::5])
    r, ref = _np(rstd), O.rmsnorm_rstd_f64(O.bf16_to_f32(hb), EPS)
    assert np.max(np.abs(r - ref) / ref) <= RSTD_RTOL
    y32 = O.rmsnorm_y_f32(hb, r, gamma)
    check_copies(out, y32, kind, qscale, margin, pow2, True, col)
    if want_y:
        assert np.array_equal(from_dev_bf16(y), bf16_bits_from_f32(y32))
    if ckpt:
        assert same_checkpoint(o_ck, o) and same_checkpoint(h_ck, hb)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (3, 4096), (129, 1280), (257, 640), (700, 2048),
                                       (33, 8192), (40, 16384), (20, 32768)])
def test_both_copies(kind, rows, cols):
    check_branch(kind, rows, cols)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,cols", [(1, 4096), (131, 256), (70, 5120)])
def test_forms(kind, form, rows, cols):
    check_branch(kind, rows, cols, **form)
    check_branch(kind, rows, cols, col=False, ckpt=False, fp32=True, **form)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1500, 4096), (2500, 128), (6000, 256), (1300, 1024),
                                       (500, 8192), (330, 16384), (320, 32768)])
def test_many_rows(kind, rows, cols):
    """More rows than run at once: a group of threads walks several, its ring of buffers round."""
    check_branch(kind, rows, cols, token=True, col=rows < 1000)


@pytest.mark.parametrize("kind", ["tensorwise", "delayed"])
@pytest.mark.parametrize("rows,cols", [(1, 16), (17, 48), (77, 2064), (250, 144), (15, 8208),
                                       (9000, 16)])
def test_per_tensor_ragged(kind, rows, cols):
    check_branch(kind, rows, cols)
    check_branch(kind, rows, cols, post=False, gate=False, col=False)


def test_options():
    check_branch("blockwise", 200, 512, pow2=True)
    check_branch("blockwise", 200, 512, margin=3, col=False)
    check_branch("tensorwise", 200, 512, margin=-2)
    check_branch("mxfp8", 200, 512, want_y=True, scale=-1.5)
    check_branch("mxfp8", 200, 512, scale=0.0)


def test_bf16_output_and_column_copy():
    """No recipe: y alone. --fp8-wgrad off: the column copy is bf16(y) transposed."""
    rows, cols = 131, 384
    o, res = (to_dev_bf16(bf16_bits_normal(rows, cols, seed=s)) for s in (1, 2))
    g = _gamma(cols)
    none, h, rstd, ro, y = F.branch_rmsnorm_quantize(None, o, res, _dev_gamma(g, False),
                                                     want_row=False, want_col=False, want_y=True)
    torch.cuda.synchronize()
    assert none is None and ro is None
    y32 = O.rmsnorm_y_f32(from_dev_bf16(h), _np(rstd), g)
    assert np.array_equal(from_dev_bf16(y), bf16_bits_from_f32(y32))
    for kind in KINDS:
        q = F.branch_rmsnorm_quantize(F.Recipe(kind=kind, fp8_wgrad=False), o, res,
                                      _dev_gamma(g, False))[0]
        torch.cuda.synchronize()
        yp = np.zeros((q.rows, cols), dtype=np.float32)
        yp[:rows] = y32
        assert q.col_bf16 == 1
        assert np.array_equal(from_dev_bf16(q.col), bf16_bits_from_f32(np.ascontiguousarray(yp.T)))


def test_a_plain_residual_is_the_norms():
    """Without gates, scale and a norm after the block, and where a float32 sum is exact (multiples of
    2^-8), every byte is rmsnorm_quantize's but for the last bits of rstd."""
    rec, rows, cols = F.Recipe(kind="mxfp8"), 300, 1024
    gen = torch.Generator(device="cuda").manual_seed(1)
    x, res = (torch.randint(-255, 256, (rows, cols), generator=gen, device="cuda")
              .div(256).to(torch.bfloat16) for _ in range(2))
    g = _dev_gamma(_gamma(cols), False)
    a = F.branch_rmsnorm_quantize(rec, x, res, g)
    b = F.rmsnorm_quantize(rec, x, g, residual=res)
    torch.cuda.synchronize()
    assert torch.equal(a[1], b[1])
    assert float(((a[2] - b[2]) / b[2]).abs().max()) <= 2 * RSTD_RTOL


@pytest.mark.parametrize("cols", [128, 512, 1024, 2176, 4096, 5120, 16384])
def test_rows_do_not_depend_on_their_number(cols):
    rec = F.Recipe(kind="mxfp8")
    o, res = (to_dev_bf16(bf16_bits_normal(700, cols, seed=s)) for s in (1, 2))
    g, w = _dev_gamma(_gamma(cols), False), _dev_gamma(_gamma(cols, seed=4), False)
    t = torch.rand(700, device="cuda")

    def run(a, b):
        ck = F.empty_checkpoint(b - a, cols)
        q, h, rstd, ro, _ = F.branch_rmsnorm_quantize(rec, o[a:b], res[a:b], g, gamma_post=w,
                                                      token_gate=t[a:b], want_col=False,
                                                      h_ckpt=ck)
        return q.row[:b - a], h, rstd, ro, ck.codes, ck.scale

    ref = run(0, 700)
    for a, b in ((0, 1), (5, 6), (699, 700), (100, 140), (300, 600)):
        for got, want in zip(run(a, b), ref):
            assert torch.equal(got, want[a:b])


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("cols", [48, 256, 4096])
def test_tokens_that_pass_by(kind, cols):
    """A token gate of 0: NaN, infinities and whatever lies in the row of branch reach nothing but
    that row's own rstd_branch and checkpoint; a zero row with eps 0 neither."""
    if kind in ("mxfp8", "blockwise") and cols % 128:
        cols = 384
    rows = 37
    o = bf16_bits_normal(rows, cols, seed=1)
    res = to_dev_bf16(bf16_bits_normal(rows, cols, seed=2))
    o[3], o[7, 5], o[8, 1], o[9] = 0x7FC0, 0x7F80, 0x7FC0, 0
    t = np.ones(rows, dtype=np.float32)
    t[[3, 7, 8, 9]] = 0.0
    t[8] = -0.0
    g = _gamma(cols)
    rec = F.Recipe(kind=kind)
    clean = o.copy()
    clean[[3, 7, 8, 9]] = bf16_bits_normal(4, cols, seed=3)
    got = [F.branch_rmsnorm_quantize(rec, to_dev_bf16(b), res, _dev_gamma(g, False),
                                     gamma_post=_dev_gamma(g, False), eps_post=0.0,
                                     token_gate=torch.from_numpy(t).cuda()) for b in (o, clean)]
    torch.cuda.synchronize()
    a, b = got
    assert torch.equal(a[1], b[1]) and torch.equal(a[2], b[2])
    assert torch.equal(a[0].row, b[0].row) and torch.equal(a[0].col, b[0].col)
    assert torch.equal(a[1][[3, 7, 8, 9]], res[[3, 7, 8, 9]])
    if a[0].amax is not None:
        assert torch.equal(a[0].amax, b[0].amax) and bool(torch.isfinite(a[0].amax).all())


def test_special_values():
    """NaN and infinities of a token that takes part, in either input."""
    rows, cols = 256, 512
    o, res = bf16_bits_normal(rows, cols, seed=6), bf16_bits_normal(rows, cols, seed=7)
    o[1, 7], o[2, 300], res[3, 9], res[4, 11] = 0x7FC0, 0x7F80, 0x7FC0, 0x7F80
    g = _gamma(cols)
    ck_o, ck_h = filled(rows, cols), filled(rows, cols)
    q, h, rstd, ro, y = F.branch_rmsnorm_quantize(
        F.Recipe(kind="mxfp8"), to_dev_bf16(o), to_dev_bf16(res), _dev_gamma(g, False),
        gamma_post=_dev_gamma(g, False), want_y=True, branch_ckpt=ck_o, h_ckpt=ck_h)
    torch.cuda.synchronize()
    hf, yf = h.float().cpu().numpy(), y.float().cpu().numpy()
    assert np.isnan(hf[1]).all() and np.isnan(yf[1]).all()       # NaN reaches its whole row
    assert np.isnan(hf[2, 300]) and np.array_equal(np.delete(hf[2], 300),
                                                   np.delete(O.bf16_to_f32(res)[2], 300))
    assert np.isnan(yf[3]).all() and np.isinf(hf[4, 11]) and np.isnan(yf[4, 11])
    assert np.isfinite(np.delete(yf, (1, 2, 3, 4), axis=0)).all()
    keep = np.setdiff1d(np.arange(rows), (1, 2, 3, 4))
    codes, scale = O.checkpoint_pack(o)
    assert np.array_equal(_np(ck_o.codes), codes & 0x7F | (codes & np.where(
        (codes & 0x7F) == 0x7F, 0, 0x80)).astype(np.uint8)) and np.array_equal(
            _np(ck_o.scale), scale)
    codes, scale = O.checkpoint_pack(from_dev_bf16(h))
    assert np.array_equal(_np(ck_h.codes)[keep], codes[keep])
    assert np.array_equal(_np(ck_h.scale), scale)


def test_strided_inputs_and_in_place():
    rows, cols = 75, 640
    wide = to_dev_bf16(bf16_bits_normal(rows, 2 * cols + 8, seed=3))
    o, res = wide[:, :cols], wide[:, cols + 8:]
    g = _dev_gamma(_gamma(cols), False)
    rec = F.Recipe(kind="mxfp8")
    a = F.branch_rmsnorm_quantize(rec, o, res, g, gamma_post=g)
    b = F.branch_rmsnorm_quantize(rec, o.contiguous(), res.contiguous(), g, gamma_post=g)
    over = res.contiguous()
    c = F.branch_rmsnorm_quantize(rec, o, over, g, gamma_post=g, h=over)
    over = o.contiguous()
    d = F.branch_rmsnorm_quantize(rec, over, res, g, gamma_post=g, h=over)
    torch.cuda.synchronize()
    for other in (b, c, d):
        assert torch.equal(a[0].row, other[0].row) and torch.equal(a[0].col, other[0].col)
        assert all(torch.equal(u, v) for u, v in zip(a[1:4], other[1:4]))


def test_empty():
    e = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    one = torch.ones(256, device="cuda")
    for kind in KINDS:
        q, h, rstd, ro, _ = F.branch_rmsnorm_quantize(F.Recipe(kind=kind), e, e, one,
                                                      gamma_post=one,
                                                      h_ckpt=F.empty_checkpoint(0, 256))
        torch.cuda.synchronize()
        assert q.rows == 0 and rstd.numel() == 0 and ro.numel() == 0
    ck = F.checkpoint(e)
    assert F.checkpoint_read(ck).shape == (0, 256)


# ---------------------------------------------------------------------------- checkpoints

@pytest.mark.parametrize("rows,cols", [(1, 16), (1, 4096), (3, 48), (37, 128), (333, 1552),
                                       (5, 32768), (1000, 2064), (4097, 272), (2, 70000),
                                       (257, 4096)])
def test_checkpoint(rows, cols):
    x = bf16_bits_normal(rows, cols, seed=rows, outlier_p=1e-3)
    ck = F.checkpoint(to_dev_bf16(x), out=filled(rows, cols))
    back = F.checkpoint_read(ck)
    torch.cuda.synchronize()
    assert same_checkpoint(ck, x)
    v = O.checkpoint_values(*O.checkpoint_pack(x))
    assert np.array_equal(O.bf16_to_f32(from_dev_bf16(back)).astype(np.float64), v)


def test_checkpoint_special_values():
    x = bf16_bits_normal(6, 96, seed=1)
    x[0] = 0
    x[1, 40], x[2, 3], x[3, 95] = 0x7FC0, 0x7F80, 0xFF80
    x[4] = 0x0001                                      # the smallest subnormal
    x[5, ::2] = 0x7F00                                 # 2^127
    ck = F.checkpoint(to_dev_bf16(x))
    back = F.checkpoint_read(ck)
    torch.cuda.synchronize()
    codes, scale = O.checkpoint_pack(x)
    assert np.array_equal(_np(ck.scale), scale) and np.array_equal(_np(ck.codes), codes)
    v = O.checkpoint_values(codes, scale)
    b = O.bf16_to_f32(from_dev_bf16(back)).astype(np.float64)
    assert np.array_equal(b, v, equal_nan=True)
    nan = np.isnan(b)
    assert nan[1, 32:64].all() and nan[2, :32].all() and nan[3, 64:].all() and nan.sum() == 96


def test_checkpoint_strided_and_past_32_bits():
    wide = to_dev_bf16(bf16_bits_normal(50, 400, seed=2))
    a, b = F.checkpoint(wide[:, 8:248]), F.checkpoint(wide[:, 8:248].contiguous())
    torch.cuda.synchronize()
    assert torch.equal(a.codes, b.codes) and torch.equal(a.scale, b.scale)
    cols, rows = 16384, (1 << 32) // 16384 + 3         # more than 2^32 elements: the last rows
    x = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = bf16_bits_normal(3, cols, seed=3)
    x[-3:] = to_dev_bf16(tail)
    ck = F.checkpoint(x)
    F.checkpoint_read(ck, out=x)
    torch.cuda.synchronize()
    assert not ck.codes[-4].any() and not x[-4].any()
    codes, scale = O.checkpoint_pack(tail)
    assert np.array_equal(_np(ck.codes[-3:]), codes) and np.array_equal(_np(ck.scale[-3:]), scale)
    assert np.array_equal(O.bf16_to_f32(from_dev_bf16(x[-3:])).astype(np.float64),
                          O.checkpoint_values(codes, scale))


def test_branch_offsets_past_32_bits():
    cols, rows = 32768, (1 << 31) // 32768 + 3
    o = torch.zeros((rows, cols), dtype=torch.bfloat16, device="cuda")
    tail = bf16_bits_normal(3, cols, seed=3)
    o[-3:] = to_dev_bf16(tail)
    ck = F.empty_checkpoint(rows, cols)
    g = torch.ones(cols, device="cuda")
    _, h, rstd, ro, y = F.branch_rmsnorm_quantize(None, o, o, g, gamma_post=g, want_row=False,
                                                  want_col=False, want_y=True, h=o, h_ckpt=ck)
    torch.cuda.synchronize()
    f = O.bf16_to_f32(tail).astype(np.float64)
    want = O.branch_sum_f64(f, f, _np(ro[-3:]), np.ones(cols))
    assert _rounds_from(h[-3:], want, H_K * 2 * (np.abs(want) + np.abs(f)))
    hb = from_dev_bf16(h[-3:])
    codes, scale = O.checkpoint_pack(hb)
    assert np.array_equal(_np(ck.codes[-3:]), codes) and np.array_equal(_np(ck.scale[-3:]), scale)
    assert np.array_equal(from_dev_bf16(y[-3:]), bf16_bits_from_f32(
        O.rmsnorm_y_f32(hb, _np(rstd[-3:]), np.ones(cols, dtype=np.float32))))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(1, 128), (130, 384), (45, 4096)])
def test_nothing_written_outside(kind, rows, cols):
    """Every output between canaries: the bytes around it keep their values."""
    guard, held = 4096, []

    def between(t):
        n = t.numel() * t.element_size()
        big = torch.full((n + 2 * guard,), 0x5A, dtype=torch.uint8, device="cuda")
        held.append((big, n))
        view = big[guard:guard + n].view(t.dtype).view(t.shape)
        view.copy_(t)
        return view

    rec = F.Recipe(kind=kind)
    q = F.empty_qtensor(rec, -(-rows // ROW_Q[kind]) * ROW_Q[kind], cols, "activation")
    for f in ("row", "col", "row_scale", "col_scale", "amax", "scale", "scale_inv"):
        if getattr(q, f) is not None:
            setattr(q, f, between(getattr(q, f)))
    x = to_dev_bf16(bf16_bits_normal(rows, cols, seed=1))
    h, y, back = (between(torch.zeros_like(x)) for _ in range(3))
    rstd, ro = (between(torch.zeros(rows, device="cuda")) for _ in range(2))
    cks = [F.Checkpoint(between(c.codes), between(c.scale))
           for c in (filled(rows, cols) for _ in range(3))]
    ws = between(torch.zeros(F.rmsnorm_workspace_bytes(rec, rows, cols), dtype=torch.uint8,
                             device="cuda"))
    g = torch.ones(cols, device="cuda")
    F.branch_rmsnorm_quantize(rec, x, x, g, gamma_post=g, out=q, h=h, rstd=rstd, rstd_branch=ro,
                              y=y, branch_ckpt=cks[0], h_ckpt=cks[1], workspace=ws)
    F.checkpoint_read(F.checkpoint(x, out=cks[2]), out=back)
    torch.cuda.synchronize()
    for big, n in held:
        assert bool((big[:guard] == 0x5A).all()) and bool((big[guard + n:] == 0x5A).all())


# ---------------------------------------------------------------------------- surroundings

def _fields(q):
    return [t for t in (q.row, q.col, q.row_scale, q.col_scale, q.amax, q.scale) if t is not None]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(3, 256), (200, 1152)])
def test_one_copy_alone(kind, rows, cols):
    """The column copy without the row copy, and the other way round: the same bytes as with both."""
    rec = F.Recipe(kind=kind)
    o, res = (to_dev_bf16(bf16_bits_normal(rows, cols, seed=s)) for s in (1, 2))
    g = _dev_gamma(_gamma(cols), False)

    def run(**kw):
        return F.branch_rmsnorm_quantize(rec, o, res, g, gamma_post=g, **kw)[0]

    both, row, col = run(), run(want_col=False), run(want_row=False)
    torch.cuda.synchronize()
    assert row.col is None and col.row is None
    assert torch.equal(both.row, row.row) and torch.equal(both.col, col.col)
    if both.amax is not None:
        assert torch.equal(both.amax, row.amax) and torch.equal(both.amax, col.amax)


def test_streams_graphs_and_calls_side_by_side():
    """The calls run on the given stream with buffers from its pool, two of them at once, and can be
    captured; the bytes are those of calls in turn."""
    rec, rows, cols = F.Recipe(kind="delayed"), 700, 2064
    o, res = (to_dev_bf16(bf16_bits_normal(rows, cols, seed=s)) for s in (1, 2))
    g, t = _dev_gamma(_gamma(cols), False), torch.rand(rows, device="cuda")

    def step(stream=None):
        cks = [F.empty_checkpoint(rows, cols) for _ in range(2)]
        q, h, rstd, ro, _ = F.branch_rmsnorm_quantize(
            rec, o, res, g, gamma_post=g, token_gate=t, branch_ckpt=cks[0], h_ckpt=cks[1],
            stream=stream)
        back = F.checkpoint_read(F.checkpoint(h, stream=stream), stream=stream)
        again = F.checkpoint_quantize(rec, cks[1], rstd, g, stream=stream)
        return [*_fields(q), h, rstd, ro, back, *_fields(again), cks[0].codes, cks[0].scale,
                cks[1].codes, cks[1].scale]

    ref = step()
    torch.cuda.synchronize()
    sides = [torch.cuda.Stream() for _ in range(2)]
    got = [step(s) for s in sides]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step()
    for _ in range(2):
        for x in captured:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
    for other in (*got, captured):
        assert all(torch.equal(a, b) for a, b in zip(ref, other))


def test_refused_calls_leave_no_error_behind():
    """What the library refuses is not launched, and the next call runs."""
    x = to_dev_bf16(bf16_bits_normal(4, 256, seed=1))
    g, rec = torch.ones(256, device="cuda"), F.Recipe(kind="mxfp8")
    ck = F.empty_checkpoint(4, 256)
    for bad in (dict(scale=float("nan")), dict(eps_post=-1.0), dict(branch_ckpt=ck, h_ckpt=ck)):
        with pytest.raises(F._lib.Fp8Error):
            F.branch_rmsnorm_quantize(rec, x, x, g, **bad)
    with pytest.raises(ValueError):
        F.branch_rmsnorm_quantize(rec, x, x, g, gate=g[:128])
    with pytest.raises(TypeError):
        F.branch_rmsnorm_quantize(rec, x, x.cpu(), g)
    with pytest.raises(TypeError):
        F.checkpoint(x, out=F.empty_checkpoint(4, 256, device="cpu"))
    with pytest.raises(F._lib.Fp8Error):
        F.checkpoint(x[:, :200].contiguous())
    F.branch_rmsnorm_quantize(rec, x, x, g, h_ckpt=ck)
    torch.cuda.synchronize()
    assert bool(torch.isfinite(F.checkpoint_read(ck).float()).all())


class _Elsewhere(torch.Tensor):
    """A tensor that says it lies on another device."""

    def get_device(self):
        return 1


def test_tensors_of_another_device_are_refused():
    """Kernels run on the current device: inputs and outputs that lie on another are refused, the
    copies' buffers among them."""
    x = to_dev_bf16(bf16_bits_normal(128, 256, seed=2))
    g, rstd = torch.ones(256, device="cuda"), torch.ones(128, device="cuda")
    rec, ck = F.Recipe(kind="mxfp8"), F.checkpoint(x)
    away = lambda t: t.as_subclass(_Elsewhere)          # noqa: E731
    outs = []
    for name in ("row", "col", "row_scale", "col_scale"):
        out = F.empty_qtensor(rec, 128, 256, "activation")
        setattr(out, name, away(getattr(out, name)))
        outs.append(out)
    delayed = F.empty_qtensor(F.Recipe(kind="delayed"), 128, 256, "activation")
    delayed.amax = away(delayed.amax)
    calls = [lambda o=o: F.branch_rmsnorm_quantize(rec, x, x, g, out=o) for o in outs]
    calls += [lambda o=o: F.checkpoint_quantize(rec, ck, out=o) for o in outs]
    calls += [lambda: F.branch_rmsnorm_quantize(F.Recipe(kind="delayed"), x, x, g, out=delayed),
              lambda: F.branch_rmsnorm_quantize(rec, x, x, away(g)),
              lambda: F.branch_rmsnorm_bwd(x, x, rstd, g, x, dh=away(torch.empty_like(x))),
              lambda: F.branch_rmsnorm_bwd(x, F.Checkpoint(ck.codes, away(ck.scale)), rstd, g, x),
              lambda: F.rmsnorm_bwd(x, F.Checkpoint(away(ck.codes), ck.scale), rstd, g),
              lambda: F.checkpoint(away(x)), lambda: F.checkpoint_read(ck, out=away(x))]
    for call in calls:
        with pytest.raises(ValueError, match="current device"):
            call()

"""The gated branch and the copies from a checkpoint at the edges of what is documented: the largest
copies, special values under every recipe, the bf16 column copy alone, captured graphs that share a
workspace."""
import pytest
import torch

from helpers import cuda_ok, to_dev_bf16
from test_gpu_norm import _dev_gamma, _gamma
from workloads import bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]
FIELDS = ("row", "col", "row_scale", "col_scale", "amax", "scale", "scale_inv")


def _bytes(t):
    return t.contiguous().view(torch.uint8)


def _same(a, b):
    for f in FIELDS:
        u, v = getattr(a, f), getattr(b, f)
        assert (u is None) == (v is None), f
        if u is not None and u.dtype == torch.float32:
            assert torch.equal(u.nan_to_num(-1.0), v.nan_to_num(-1.0)), f      # NaN: any payload
        elif u is not None:
            assert torch.equal(_bytes(u), _bytes(v)), f


@pytest.mark.parametrize("kind", ["mxfp8", "delayed"])
def test_largest_copies(kind):
    """Just below 2^31 elements, where offsets are 32 bits wide: all bytes are those of the norm
    (values whose sums are exact, as in test_gpu_branch_plain), and, made again from a checkpoint,
    those of the checkpoint's values."""
    cols = 8192
    rows = (1 << 31) // cols - 128
    rec = F.Recipe(kind=kind)
    x = torch.randint(-7, 8, (rows, cols), dtype=torch.int8, device="cuda")
    x = x.to(torch.bfloat16).div_(8)
    res = x.flip(0)
    g = _dev_gamma(_gamma(cols), False)
    ck = F.empty_checkpoint(rows, cols)
    a, h, rstd, _, _ = F.branch_rmsnorm_quantize(rec, x, res, g, h_ckpt=ck)
    b = F.rmsnorm_quantize(rec, x, g, residual=res, h=res)[0]
    torch.cuda.synchronize()
    _same(a, b)
    again = F.checkpoint_quantize(rec, ck, rstd, g, out=a)
    h = F.checkpoint_read(ck, out=h)
    b, _, ref, _ = F.rmsnorm_quantize(rec, h, g, out=b)
    torch.cuda.synchronize()
    rows_alike = rstd == ref                             # E4M3 holds these sums but for a few
    assert bool(rows_alike.any())
    assert torch.equal(again.row[:rows][rows_alike], b.row[:rows][rows_alike])
    b = F.checkpoint_quantize(rec, ck, ref, g, out=b)
    c = F.rmsnorm_quantize(rec, h, g, out=again)[0]
    torch.cuda.synchronize()
    _same(b, c)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("pow2", [False, True])
def test_copies_of_special_values(kind, pow2):
    """NaN, infinities, zeros, and large and small blocks: the bytes of the norm of the values that
    the checkpoint reads back as."""
    rows, cols = 300, 640
    x = bf16_bits_normal(rows, cols, seed=1)
    x[3, 40], x[17, 9], x[290, 639] = 0x7FC0, 0x7F80, 0xFF80
    x[20], x[21, :64], x[22], x[23, 32:64] = 0, 0, 0x0D80, 0x1F00      # 2^-100, 2^-65
    x[24], x[25, 5] = 0x5D80, 0xDD80                                   # 2^60, -2^60
    ck = F.checkpoint(to_dev_bf16(x))
    g = _dev_gamma(_gamma(cols), False)
    g[7], g[600] = -1.5, 0.0
    values = F.checkpoint_read(ck)
    for wgrad in (True, False):
        if pow2 and kind != "blockwise":
            continue
        rec = F.Recipe(kind=kind, power_2_scales=pow2, fp8_wgrad=wgrad)
        for row, col in ((True, True), (False, True), (True, False)):
            want, _, rstd, _ = F.rmsnorm_quantize(rec, values, g, want_row=row, want_col=col)
            got = F.checkpoint_quantize(rec, ck, rstd, g, want_row=row, want_col=col)
            torch.cuda.synchronize()
            assert got.col_bf16 == (0 if wgrad else 1)
            _same(want, got)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wgrad", [True, False])
def test_graphs_that_share_a_workspace(kind, wgrad):
    """Two forward passes and the copies made again, captured apart over one workspace and replayed
    in turn, on new values in the same buffers."""
    rows, cols = 333, 1152
    rec = F.Recipe(kind=kind, fp8_wgrad=wgrad)
    g, t = _dev_gamma(_gamma(cols), False), torch.rand(rows, device="cuda")
    ws = torch.empty(F.rmsnorm_workspace_bytes(rec, rows, cols), dtype=torch.uint8, device="cuda")
    ins = [[torch.empty((rows, cols), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
           for _ in range(2)]
    cks = [F.empty_checkpoint(rows, cols) for _ in range(2)]

    def forward(i):
        return F.branch_rmsnorm_quantize(rec, *ins[i], g, gamma_post=g, token_gate=t,
                                         h_ckpt=cks[i], workspace=ws, want_row=i == 0)

    def again(i, rstd):
        return F.checkpoint_quantize(rec, cks[i], rstd, g, workspace=ws, want_row=i == 1)

    def fill(seed):
        gen = torch.Generator(device="cuda").manual_seed(seed)
        for t in (t for pair in ins for t in pair):
            t.copy_(torch.randn((rows, cols), generator=gen, device="cuda"))

    fill(0)
    again(1, forward(1)[2])                              # whatever is set up once
    torch.cuda.synchronize()
    graphs, outs = [], []
    for i in (0, 1):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            a = forward(i)
            outs.append((a[0], a[1], a[2], again(i, a[2])))
    for seed in (1, 2):
        fill(seed)
        torch.cuda.synchronize()
        for graph in graphs:
            graph.replay()
        torch.cuda.synchronize()
        for i in (0, 1):
            a = forward(i)
            b = again(i, a[2])
            torch.cuda.synchronize()
            _same(outs[i][0], a[0])
            _same(outs[i][3], b)
            assert torch.equal(outs[i][1], a[1]) and torch.equal(outs[i][2], a[2])


def test_in_place_with_checkpoints_and_copies():
    """The stream written over the branch or over the residual, with both checkpoints, for a row
    count that ends inside a tile: the bytes of the call into a buffer of its own."""
    rows, cols = 451, 2176
    rec = F.Recipe(kind="mxfp8")
    o, res = (to_dev_bf16(bf16_bits_normal(rows, cols, seed=s)) for s in (1, 2))
    g = _dev_gamma(_gamma(cols), False)

    def call(o, res, h=None):
        cks = [F.empty_checkpoint(rows, cols) for _ in range(2)]
        q, h, rstd, ro, _ = F.branch_rmsnorm_quantize(rec, o, res, g, gamma_post=g, gate=g, h=h,
                                                      scale=0.3, branch_ckpt=cks[0], h_ckpt=cks[1])
        torch.cuda.synchronize()
        return [q.row, q.col, q.row_scale, q.col_scale, h, rstd, ro,
                *(t for c in cks for t in (c.codes, c.scale))]

    ref = call(o, res)
    a, b = o.clone(), res.clone()
    for got in (call(a, res, h=a), call(o, b, h=b)):
        assert all(torch.equal(u, v) for u, v in zip(ref, got))

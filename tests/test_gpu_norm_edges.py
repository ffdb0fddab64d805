"""Edges of the norm around the FP8 linear layer: buffers that a caller keeps, padding rows, ranges
of values, and shapes whose groups of threads walk several rows."""
import numpy as np
import pytest
import torch

from helpers import cuda_ok, from_dev_bf16, to_dev_bf16
from oracle import fp8_oracle as O
from test_gpu_norm import RSTD_RTOL, check_bwd, check_copies, check_norm
from workloads import bf16_bits_from_f32, bf16_bits_normal

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]
ROW_Q = {"mxfp8": 128, "blockwise": 128, "tensorwise": 16, "delayed": 16}


@pytest.mark.parametrize("kind", KINDS)
def test_refuses_an_output_that_is_not_on_the_gpu(kind):
    rec = F.Recipe(kind=kind)
    x = torch.zeros(3, 256, dtype=torch.bfloat16, device="cuda")
    for name in ("row", "col", "row_scale", "col_scale", "amax", "scale", "scale_inv"):
        out = F.empty_qtensor(rec, ROW_Q[kind], 256, "activation")
        if getattr(out, name) is not None:
            setattr(out, name, getattr(out, name).cpu())
            with pytest.raises(TypeError):
                F.rmsnorm_quantize(rec, x, torch.ones(256, device="cuda"), out=out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wgrad", [True, False])
@pytest.mark.parametrize("rows,cols,residual", [(1, 256, True), (5, 128, False),
                                                (125, 4096, False), (131, 640, True),
                                                (1003, 2048, False), (300, 16384, True)])
def test_padding_is_what_quantising_zero_rows_gives(kind, wgrad, rows, cols, residual):
    """A gamma with negative and zero entries: products with a padding row's zeros have gamma's
    sign, its codes (and bf16 columns) are +0 all the same. Rows that exist keep their -0."""
    g = np.random.default_rng(3).standard_normal(cols).astype(np.float32)
    g[::7], g[3::11] = 0.0, -0.0
    rec = F.Recipe(kind=kind, fp8_wgrad=wgrad)
    padded = -(-rows // ROW_Q[kind]) * ROW_Q[kind]
    q = F.empty_qtensor(rec, padded, cols, "activation")
    for t in (q.row, q.col):
        t.fill_(0xA5)
    x = bf16_bits_normal(rows, cols, seed=4)
    x[:, ::5] = 0x8000
    res = to_dev_bf16(np.full_like(x, 0x8000)) if residual else None
    q, h, rstd, _ = F.rmsnorm_quantize(rec, to_dev_bf16(x), torch.from_numpy(g).cuda(),
                                       residual=res, out=q)
    torch.cuda.synchronize()
    y = O.rmsnorm_y_f32(from_dev_bf16(h), rstd.cpu().numpy(), g)
    check_copies(q, y, kind, scale=1.0, col=wgrad)
    if not wgrad:
        yp = np.zeros((padded, cols), dtype=np.float32)
        yp[:rows] = y
        assert np.array_equal(from_dev_bf16(q.col), bf16_bits_from_f32(np.ascontiguousarray(yp.T)))


@pytest.mark.parametrize("kind", ["tensorwise", "delayed"])
@pytest.mark.parametrize("cols", [16, 48, 2064, 4096, 8208])
@pytest.mark.parametrize("col", [True, False])
def test_amax_of_infinities(kind, cols, col):
    """eps 0 and rows so small that their squares vanish in fp32: rstd is infinite and the
    outputs infinities. The lanes that have no column in a row of such a width add no NaN."""
    rec = F.Recipe(kind=kind)
    x = torch.full((16, cols), 1e-25, dtype=torch.bfloat16, device="cuda")
    q, _, rstd, y = F.rmsnorm_quantize(rec, x, torch.ones(cols, device="cuda"), eps=0.0,
                                       want_col=col, want_y=True)
    torch.cuda.synchronize()
    assert bool(torch.isinf(rstd).all()) and bool(torch.isinf(y).all())
    assert q.amax.item() == float("inf")
    x[3, 5] = 0.0                                   # 0 inf: a NaN of the row's own
    q = F.rmsnorm_quantize(rec, x, torch.ones(cols, device="cuda"), eps=0.0, want_col=col)[0]
    assert q.amax.isnan().item()


@pytest.mark.parametrize("cols,below,above", [(128, 181 / 128 * 2.0 ** 60, 182 / 128 * 2.0 ** 60),
                                              (4096, 255 / 128 * 2.0 ** 57, 2.0 ** 58),
                                              (32768, 181 / 128 * 2.0 ** 56,
                                               182 / 128 * 2.0 ** 56)])
def test_range_of_a_rows_squares(cols, below, above):
    """The last bf16 value before cols squares add up to 2^128, and the next one (in bf16, 181/128
    lies just below the root of 2): the formula's value, then rstd 0 and zeros. One element may be
    larger, as long as its square is in range."""
    assert cols * below ** 2 < 2.0 ** 128 <= cols * above ** 2
    x = torch.zeros(3, cols, dtype=torch.bfloat16, device="cuda")
    x[0], x[1], x[2, 7] = below, above, 2.0 ** 63
    assert float(x[0, 0]) == below and float(x[1, 0]) == above
    y, _, rstd = F.rmsnorm(x, torch.ones(cols, device="cuda"))
    torch.cuda.synchronize()
    r = rstd.cpu().numpy().astype(np.float64)
    for i, ref in ((0, 1 / below), (2, cols ** 0.5 * 2.0 ** -63)):
        assert abs(r[i] - ref) <= RSTD_RTOL * ref
    assert bool((y[0] == 1).all()) and y[2, 7].item() == torch.tensor(cols ** 0.5).bfloat16().item()
    assert r[1] == 0 and not y[1].any()


def _steps(rows, cols, threads_per_row, per_sm):
    """Rows that each group of threads of the row kernel walks, from its launch: CTAs of 256
    threads, as many per SM as run at once."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    return rows / (256 // threads_per_row * per_sm * sms)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols,residual,ahead",
                         [(66001, 128, False, 4), (40003, 128, True, 2), (33005, 256, False, 4),
                          (20007, 256, True, 2), (16009, 512, False, 2), (17001, 512, True, 1)])
def test_groups_that_walk_many_rows(kind, rows, cols, residual, ahead):
    """Several rows are on their way to a group of threads at once; its ring of buffers comes
    round twice at least, and ends on a ragged row."""
    assert _steps(rows, cols, 16 if cols == 128 else 32, 3) > 2 * ahead
    check_norm(kind, rows, cols, residual=residual, col=kind != "mxfp8")


@pytest.mark.parametrize("rows,residual", [(66001, False), (40003, True)])
def test_narrow_groups_that_walk_many_rows(rows, residual):
    """Two of a row's sixteen threads have columns."""
    assert _steps(rows, 16, 16, 3) > (8 if not residual else 4)
    for kind in ("tensorwise", "delayed"):
        check_norm(kind, rows, 16, residual=residual)
    x = to_dev_bf16(bf16_bits_normal(rows, 16, seed=2))
    res = to_dev_bf16(bf16_bits_normal(rows, 16, seed=3)) if residual else None
    g = torch.rand(16, device="cuda") + 0.5
    y, h, rstd = F.rmsnorm(x, g, res)
    torch.cuda.synchronize()
    want = O.rmsnorm_y_f32(from_dev_bf16(h), rstd.cpu().numpy(), g.cpu().numpy())
    assert np.array_equal(from_dev_bf16(y), bf16_bits_from_f32(want))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,cols", [(256, 32768), (2048, 4096), (1000, 8192)])
def test_column_blocks_that_walk_whole_tiles(kind, rows, cols):
    """More tiles of rows than CTAs for a column block, in the kernel that tests nothing per row:
    whole tiles, and a last one of which some rows are padding (per-tensor recipes pad to 16 rows
    only: their ragged case runs the general kernel)."""
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert (rows + 127) // 128 > max(1, 6 * sms // (cols // 64))
    check_norm(kind, rows, cols, residual=rows != 2048)


@pytest.mark.parametrize("rows,cols", [(330, 8192), (400, 16384), (350, 32768)])
def test_backward_of_wide_rows_that_follow_each_other(rows, cols):
    """One CTA per SM holds a row of these widths; each walks two or three."""
    assert rows > 2 * torch.cuda.get_device_properties(0).multi_processor_count
    check_bwd(rows, cols)
    check_bwd(rows, cols, dres=False, gamma_fp32=True)

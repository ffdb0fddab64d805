"""What the Python binding checks before the library sees an address, on CPU tensors: a call that
passes every check of shapes and types ends in the TypeError for tensors that are not on the GPU."""
import pytest
import torch

from scaled_quantize_fp8_gb300 import binding
from scaled_quantize_fp8_gb300 import build as B


@pytest.fixture(scope="module", autouse=True)
def lib():
    B.build()


KINDS = ["mxfp8", "blockwise", "tensorwise", "delayed"]


def _call(rec, out, rows=5, cols=256, **kw):
    x = torch.zeros(rows, cols, dtype=torch.bfloat16)
    return binding.rmsnorm_quantize(rec, x, torch.zeros(cols), out=out, **kw)


def _out(rec, cols=256, role="activation"):
    rows = 128 if rec.kind in ("mxfp8", "blockwise") else 16
    return binding.empty_qtensor(rec, rows, cols, role, device="cpu")


@pytest.mark.parametrize("kind", KINDS)
def test_norm_refuses_a_column_copy_of_the_other_type(kind):
    """Without FP8 wgrad the column copy takes two bytes an element, else one: buffers kept from
    before the recipe's flag changed have the right shape and the wrong size."""
    rec = binding.Recipe(kind=kind)
    out = _out(rec)
    rec.fp8_wgrad = False
    with pytest.raises(ValueError):
        _call(rec, out)
    out = _out(rec)
    rec.fp8_wgrad = True
    with pytest.raises(ValueError):
        _call(rec, out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("name", ["row", "col"])
def test_norm_refuses_copies_that_do_not_lie_row_by_row(kind, name):
    rec = binding.Recipe(kind=kind)
    out = _out(rec)
    t = getattr(out, name)
    setattr(out, name, t.t().contiguous().t())
    with pytest.raises(ValueError):
        _call(rec, out)
    setattr(out, name, t[:1].expand(t.shape))
    with pytest.raises(ValueError):
        _call(rec, out)


@pytest.mark.parametrize("kind", ["mxfp8", "blockwise"])
@pytest.mark.parametrize("name", ["row_scale", "col_scale"])
def test_norm_refuses_scales_that_are_too_few(kind, name):
    rec = binding.Recipe(kind=kind)
    out = _out(rec)
    t = getattr(out, name)
    setattr(out, name, t.reshape(-1)[:-1])
    with pytest.raises(ValueError):
        _call(rec, out)
    setattr(out, name, t.reshape(-1)[:1].expand(t.numel()))
    with pytest.raises(ValueError):
        _call(rec, out)
    if kind == "blockwise":                         # one scale for 128 x 128, as weights have
        with pytest.raises(ValueError):
            _call(rec, _out(rec, role="weight"))


@pytest.mark.parametrize("kind", ["tensorwise", "delayed"])
@pytest.mark.parametrize("name", ["amax", "scale", "scale_inv"])
def test_norm_refuses_malformed_scalars(kind, name):
    rec = binding.Recipe(kind=kind)
    for bad in (torch.zeros(0), torch.zeros(1, dtype=torch.bfloat16)):
        out = _out(rec)
        setattr(out, name, bad)
        with pytest.raises(ValueError):
            _call(rec, out)


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("wgrad", [True, False])
def test_norm_takes_what_empty_qtensor_makes(kind, wgrad):
    rec = binding.Recipe(kind=kind, fp8_wgrad=wgrad)
    with pytest.raises(TypeError, match="CUDA"):    # nothing else is wrong with the call
        _call(rec, _out(rec))
    with pytest.raises(TypeError, match="CUDA"):
        _call(rec, _out(rec), want_col=False)


def test_results_of_a_plain_list_come_from_the_calls_stream(monkeypatch):
    """grad_norm makes its own two results for a plain list of tensors. Taken from the current
    stream's pool, they could be memory that work queued there still uses, or uses again, while
    the kernels write them on the stream that was given."""
    seen = []

    def empty(shape, dtype, device, stream):
        seen.append(stream)
        return torch.empty(shape, dtype=dtype, device=device)

    monkeypatch.setattr(binding, "_empty", empty)
    with pytest.raises(TypeError, match="CUDA"):
        binding.grad_norm([torch.ones(3)], stream="side")
    assert seen == ["side"]
    binding.GradList([torch.ones(3)], stream="other")
    assert seen == ["side", "other"]


def test_gradients_on_more_than_one_device_are_refused():
    """The kernels run on one GPU: an address of another device's memory is not theirs to read."""
    here, there = torch.ones(3), torch.ones(3, device="meta")
    for grads, outs in (([here, there], None), ([here], [there]), ([there, here], None)):
        with pytest.raises(ValueError, match="device"):
            binding.GradList(grads, outs)


def test_a_recipe_holds_its_fields_and_nothing_else():
    """Calls leave no trace in a Recipe: it can be rebuilt from vars(), a field set through the
    dictionary counts, and a C form belongs to its caller."""
    rec = binding.Recipe(kind="mxfp8", margin=1)
    before = dict(vars(rec))
    c = rec.c()
    assert vars(rec) == before and binding.Recipe(**vars(rec)) == rec
    rec.__dict__.update(margin=5)
    assert rec.c().margin == 5
    c.margin = 7
    assert rec.c().margin == 5


def test_the_packed_recipe_is_the_structure():
    rec = binding.Recipe(kind="blockwise", format="hybrid", margin=-3, amax_history_len=17,
                         amax_compute_algo="most_recent", fp8_wgrad=False, power_2_scales=True)
    assert binding.L.pack_recipe(*rec._fields()) == bytes(rec.c())


def test_a_workspace_counts_for_the_memory_it_has():
    """An expanded tensor's bytes are not there: as small as none, so the call makes its own."""
    whole = torch.zeros(64, dtype=torch.uint8)
    assert binding._buffer(whole) == (whole.data_ptr(), 64)
    assert binding._buffer(torch.zeros(8, 4))[1] == 128
    for t in (None, whole[:1].expand(1 << 20), whole.view(8, 8)[:, :4]):
        assert binding._buffer(t) == (None, 0)


def test_outs_need_the_gradients_order_not_their_strides():
    """The stride of a dimension of one element says nothing about where elements lie."""
    column = torch.zeros(5, 1)
    for g, o in ((column.t(), torch.zeros(1, 5)), (torch.zeros(1, 5), column.t()),
                 (torch.zeros(3, 0).t(), torch.zeros(0, 3))):
        assert g.stride() != o.stride()
        binding.GradList([g], [o])
    with pytest.raises(ValueError):
        binding.GradList([torch.zeros(2, 5)], [torch.zeros(5, 2).t()])

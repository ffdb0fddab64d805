"""GPU tests of the global gradient norm and of clipping.

Tolerance of the norm: a thread adds at most 16 chunks of 16384 / 256 squares over four float32
sums before they go to float64, 256 additions of 2^-24 relative each; half of that reaches the
root: below NORM_RTOL. The clipped gradients are compared exactly, with the GPU's coefficient:
one float32 product, rounded once to the output's type."""
import math

import numpy as np
import pytest
import torch

from helpers import cuda_ok
from oracle import fp8_oracle as O

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F

NORM_RTOL = 8e-6
BF16, FP32 = torch.bfloat16, torch.float32


def _grads(sizes, dtype, seed=0, sigma=1e-3, packed=False):
    g = torch.Generator().manual_seed(seed)
    flat = (torch.randn(sum(sizes) + len(sizes) * 8, generator=g) * sigma).to(dtype).cuda()
    out, at = [], 0
    for s in sizes:
        out.append(flat[at:at + s])
        at += s if packed else -(-s // 8) * 8
    return out


def _f64(grads):
    return [g.double().cpu().numpy() for g in grads]


def check(grads, outs=None, max_norm=math.inf, scale=1.0):
    before = [g.clone() for g in grads]
    ref = O.grad_norm_f64(_f64(grads), scale)
    gl = F.GradList(grads, outs)
    norm, coef = F.grad_norm(gl, max_norm=max_norm, scale=scale)
    n, c = norm.item(), coef.item()
    assert abs(n - ref) <= NORM_RTOL * ref
    assert math.isclose(c, O.clip_coef_f64(n, max_norm, scale), rel_tol=4 * 2.0 ** -24)
    got = F.grad_clip(gl, coef)
    torch.cuda.synchronize()
    for g, b, o in zip(grads, before, got):
        assert torch.equal(o, (b.float() * coef).to(o.dtype))
        if o is not g:
            assert torch.equal(g, b)
    return n, c


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("packed", [False, True])
@pytest.mark.parametrize("sizes", [[1], [7], [8192], [8193], [1, 2, 3, 5, 8, 13, 21], [0, 5, 0],
                                   [3, 100003, 1, 65536, 8191], [1 << 20, 31]])
def test_norm_and_clip(sizes, dtype, packed):
    n, c = check(_grads(sizes, dtype, packed=packed), max_norm=1e9)
    assert c == 1.0
    for out in (BF16, FP32):
        grads = _grads(sizes, dtype, packed=packed)
        outs = [torch.zeros_like(g, dtype=out) for g in grads]
        check(grads, outs, max_norm=n / 3)
    _, c = check(_grads(sizes, dtype, packed=packed), max_norm=n / 3)        # in place
    assert 0.3 < c < 0.34


def test_outputs_at_other_offsets():
    """Outputs whose alignment differs from their gradient's, both types."""
    for dtype in (BF16, FP32):
        for out in (BF16, FP32):
            for a, b in ((0, 1), (1, 0), (3, 6), (5, 5)):
                src = _grads([5000], dtype)[0][a:a + 4000]
                dst = torch.zeros(4100, dtype=out, device="cuda")
                check([src], [dst[b:b + 4000]], max_norm=1e-3)
                assert not dst[:b].any() and not dst[b + 4000:].any()


@pytest.mark.parametrize("count", [63, 64, 65, 1024, 1025, 3000])
def test_many_tensors(count):
    """Lists around the sizes at which they are split over launches, both types mixed."""
    rng = np.random.default_rng(count)
    sizes = [int(v) for v in rng.integers(0, 300, count)]
    bf, fp = _grads(sizes, BF16, seed=1, packed=True), _grads(sizes, FP32, seed=2, packed=True)
    grads = [b if i % 3 else f for i, (b, f) in enumerate(zip(bf, fp))]
    check(grads, max_norm=1e-2)


def test_scale():
    grads = _grads([1000, 77], BF16)
    n, c = check(grads, max_norm=1e9, scale=0.125)
    assert c == 0.125
    check(_grads([1000, 77], BF16), max_norm=n / 2, scale=0.125)


def test_range_of_squares():
    """Gradients whose squares are below or above float32's range, alone and mixed."""
    for sigma in (1e-30, 1e-22, 1e-16, 1e15, 1e17, 1e25):
        for dtype in (BF16, FP32):
            check(_grads([9000, 5], dtype, sigma=sigma), max_norm=1.0)
    mixed = _grads([4096], FP32, sigma=1e-25) + _grads([4096], FP32, sigma=1.0)
    check(mixed, max_norm=1.0)


def test_not_finite():
    for dtype in (BF16, FP32):
        for bad, norm in ((math.inf, math.inf), (-math.inf, math.inf), (math.nan, math.nan)):
            for at in (0, 4321, 8999):
                grads = _grads([9000, 100], dtype)
                grads[0][at] = bad
                n, c = F.grad_norm(grads, max_norm=1.0)
                n, c = n.item(), c.item()
                assert (math.isnan(n) and math.isnan(c)) if math.isnan(norm) else \
                    (n == math.inf and c == 0.0)


def test_empty():
    norm, coef = F.grad_norm([], max_norm=2.0)
    assert norm.item() == 0.0 and coef.item() == 1.0
    F.grad_clip([], coef)
    zeros = [torch.zeros(100, device="cuda"), torch.zeros(0, device="cuda")]
    norm, coef = F.grad_norm(zeros, max_norm=2.0)
    assert norm.item() == 0.0 and coef.item() == 1.0


def test_dense_orders_and_strides():
    """A transposed weight gradient is dense: the norm does not depend on the order, and clipping
    in place scales every element."""
    w = _grads([96 * 40], BF16)[0].view(96, 40)
    v = _grads([2 * 3 * 16], FP32, seed=3)[0].view(2, 3, 16).permute(2, 0, 1)
    check([w.t(), v], max_norm=1e-3)


def test_deterministic_on_any_stream():
    grads = _grads([100000, 33, 70001], BF16, packed=True)
    a = F.grad_norm(grads, max_norm=1.0)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    b = F.grad_norm(grads, max_norm=1.0, stream=side)
    side.synchronize()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_graph_capture():
    grads = _grads([40000, 123], FP32)
    outs = [torch.zeros_like(g) for g in grads]
    gl = F.GradList(grads, outs)
    ws = torch.empty(F.grad_workspace_bytes(2), dtype=torch.uint8, device="cuda")
    norm, coef = torch.zeros(1, device="cuda"), torch.zeros(1, device="cuda")

    def step():
        F.grad_norm(gl, max_norm=1e-3, norm=norm, coef=coef, workspace=ws)
        F.grad_clip(gl, coef)

    step()
    torch.cuda.synchronize()
    ref = [t.clone() for t in outs + [norm, coef]]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for t in outs + [norm, coef]:
        t.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(outs + [norm, coef], ref))


def test_nothing_written_outside():
    guard = 512
    big = torch.full((guard * 2 + 10001,), 7.0, device="cuda")
    big[guard:guard + 10001] = 1e-3
    check([big[guard:guard + 10001]], max_norm=1e-3)
    assert bool((big[:guard] == 7).all()) and bool((big[guard + 10001:] == 7).all())


def test_offsets_past_32_bits():
    n = (1 << 31) + 12345
    g = torch.full((n,), 2.0 ** -10, dtype=BF16, device="cuda")
    norm, coef = F.grad_norm([g], max_norm=1.0)
    ref = 2.0 ** -10 * math.sqrt(n)
    assert abs(norm.item() - ref) <= NORM_RTOL * ref
    F.grad_clip([g], coef)
    torch.cuda.synchronize()
    want = (torch.tensor(2.0 ** -10) * coef.cpu()).to(BF16)
    assert torch.equal(g[-2:].cpu(), want.expand(2)) and torch.equal(g[:2].cpu(), want.expand(2))
    assert bool((g == want.cuda()).all())


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("bytes_", [(1 << 20) - 4, 1 << 20, (1 << 20) + 4])
@pytest.mark.parametrize("tensors", [1, 3])
def test_short_and_long_lists(dtype, bytes_, tensors):
    """Lists just below, at and above 1 MB, where one launch becomes two; split unevenly and at
    odd offsets."""
    n = bytes_ // (2 if dtype == BF16 else 4)
    sizes = [n] if tensors == 1 else [n - 5001, 1, 5000]
    c, _ = check(_grads(sizes, dtype, packed=True), max_norm=1e9)
    check(_grads(sizes, dtype, packed=True), max_norm=c / 2)


@pytest.mark.parametrize("count", [255, 256, 257])
def test_tiny_tensors_of_both_types(count):
    """As many tensors as a short list has room for, one less and one more."""
    grads = _grads([1 + i % 3 for i in range(count)], BF16, packed=True)
    grads[::2] = [g.float() for g in grads[::2]]
    check(grads, max_norm=1e-3)


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_range_and_not_finite_in_long_lists(dtype):
    for sigma in (1e-25, 1e17):
        check(_grads([700001, 3], dtype, sigma=sigma), max_norm=1.0)
    mixed = _grads([700001], dtype, sigma=1e-25) + _grads([600000], dtype, sigma=1.0)
    check(mixed, max_norm=1.0)
    for bad in (math.inf, math.nan):
        grads = _grads([700001, 3], dtype)
        grads[0][654321] = bad
        n, c = F.grad_norm(grads, max_norm=1.0)
        assert math.isnan(n.item()) if math.isnan(bad) else (n.item() == bad and c.item() == 0)


def test_norm_of_one_element():
    """The root over float32's whole range: the square's rounding and the mantissa's count half
    in the root, which is rounded itself, and so is its product with the scale: 3 * 2^-24."""
    values = [3.4e38, 1.5, 1.0, 2.0, math.sqrt(2), 3.0, 0.1, 7e-4, 1e-14, 9e-16, 2.0 ** -63, 1e-30,
              2.0 ** -126]
    for v in values:
        for scale in (1.0, 0.25):
            g = torch.full((1,), v, device="cuda")
            norm, _ = F.grad_norm([g], max_norm=1.0, scale=scale)
            ref = g.double().item() * scale
            assert abs(norm.item() - ref) <= 3 * 2.0 ** -24 * ref + 2.0 ** -149

"""Edges of the norm around the FP8 linear layer: buffers that a caller keeps, padding rows, ranges
of values, and shapes whose groups of threads walk several rows."""
import pytest
import torch

from helpers import cuda_ok

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

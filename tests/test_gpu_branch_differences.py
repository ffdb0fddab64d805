"""The gated branch's backward pass against central differences of the formulas (branch_differences
has the bounds; test_branch_differences shows which wrong gradients they find)."""
import numpy as np
import pytest
import torch

from branch_differences import problem, wrong
from helpers import cuda_ok, to_dev_bf16
from test_branch_differences import FORMS

pytestmark = pytest.mark.gpu

if cuda_ok():
    import scaled_quantize_fp8_gb300 as F


def _f32(v):
    return None if v is None else torch.from_numpy(np.asarray(v, dtype=np.float32)).cuda()


def _kept(p, name, ckpt):
    if not ckpt:
        return to_dev_bf16(p[name + "_kept"])
    return F.Checkpoint(*(torch.from_numpy(np.ascontiguousarray(v)).cuda()
                          for v in p[name + "_kept"]))


@pytest.mark.parametrize("form", FORMS)
@pytest.mark.parametrize("rows,cols", [(24, 512), (3, 16), (7, 1040), (40, 4096), (3, 5120),
                                       (4, 8208), (3, 16400)])
def test_backward(rows, cols, form):
    for ckpt in [form["ckpt"]] if "ckpt" in form else [(False, False), (True, False),
                                                       (False, True)]:
        p = problem(rows, cols, **{**form, "ckpt": ckpt})
        d = F.branch_rmsnorm_bwd(
            to_dev_bf16(p["dy_bits"]), _kept(p, "h", ckpt[0]), _f32(p["rstd"]), _f32(p["gamma"]),
            _kept(p, "o", ckpt[1]), rstd_branch=_f32(p["ro"]), gamma_post=_f32(p["a"]),
            gate=_f32(p["g"]), token_gate=_f32(p["t"]), scale=p["scale"],
            dres=None if p["dres_bits"] is None else to_dev_bf16(p["dres_bits"]))
        torch.cuda.synchronize()
        got = {k: v.double().cpu().numpy() for k, v in d._asdict().items() if v is not None}
        assert wrong(p, got) == set()

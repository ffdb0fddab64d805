"""C ABI checks, without a GPU, of the norm, its backward pass, the gradient norm and clipping:
struct layouts, and what is refused on the host before anything is launched."""
import ctypes
import math
import os
import shutil
import subprocess

import pytest
import torch

from scaled_quantize_fp8_gb300 import _lib as L
from scaled_quantize_fp8_gb300 import binding
from scaled_quantize_fp8_gb300 import build as B

# Made-up addresses that validation must reject: never where a kernel could reach them.
pytestmark = pytest.mark.skipif(torch.cuda.is_available(),
                                reason="fake-pointer validation tests run on CPU-only hosts")

NULL, ALIGN, SHAPE, UNSUPPORTED, WORKSPACE = 1, 2, 3, 4, 7


@pytest.fixture(scope="module")
def lib():
    B.build()
    return L.load()


STRUCTS = {"fp8_norm_input": L.NormInput, "fp8_norm_grad": L.NormGrad,
           "fp8_grad_item": L.GradItem, "fp8_clip_rule": L.ClipRule}


def test_struct_layouts(tmp_path):
    cc = shutil.which("gcc") or shutil.which("cc")
    inc = "/usr/local/cuda/include"
    if cc is None or not os.path.exists(os.path.join(inc, "cuda_runtime_api.h")):
        pytest.skip("needs a C compiler and the CUDA runtime headers")
    body = []
    for name, cls in STRUCTS.items():
        body.append(f'printf("%zu\\n", sizeof({name}));')
        body += [f'printf("%zu\\n", offsetof({name}, {f}));' for f, _ in cls._fields_]
    src = tmp_path / "l.c"
    src.write_text('#include <stdio.h>\n#include <stddef.h>\n#include "fp8lin.h"\n'
                   "int main(void) {" + "\n".join(body) + " return 0; }\n")
    subprocess.run([cc, "-std=c99", "-I", L.HEADER_DIR, "-I", inc, str(src), "-o",
                    str(tmp_path / "l")], check=True)
    got = [int(v) for v in subprocess.run([str(tmp_path / "l")], capture_output=True, text=True,
                                          check=True).stdout.split()]
    want = []
    for cls in STRUCTS.values():
        want += [ctypes.sizeof(cls)] + [getattr(cls, f).offset for f, _ in cls._fields_]
    assert got == want


def _rec(kind=L.RECIPE_MXFP8, **kw):
    r = L.Recipe(kind, 0, 0, 16, 0, 1, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _in(**kw):
    d = dict(x=0x8000, residual=0x9000, gamma=0xA000, ldx=256, ldr=256, rows=100, cols=256,
             gamma_fp32=0, eps=1e-5)
    d.update(kw)
    return L.NormInput(*[d[f] for f, _ in L.NormInput._fields_])


def _tensor(**kw):
    d = dict(row=0x1000, col=0x2000, row_scale=0x3000, col_scale=0x4000, amax=0x5000,
             scale=0x6000, scale_inv=0x7000)
    d.update(kw)
    return L.Tensor(*[d[f] for f in ("row", "col", "row_scale", "col_scale", "amax", "scale",
                                     "scale_inv")], 0, 0, 0, 0, 0)


def _norm(lib, rec=None, inp=None, wr=1, wc=1, h=0xB000, rstd=0xC000, y=None, out=None,
          ws=0xD000, ws_bytes=1 << 20):
    rec = _rec() if rec is None else rec
    out = _tensor() if out is None else out
    return lib.fp8_rmsnorm_quantize(ctypes.byref(rec) if rec else None,
                                    ctypes.byref(inp if inp is not None else _in()), wr, wc, h,
                                    rstd, y, ctypes.byref(out) if out else None, ws, ws_bytes,
                                    None, None)


def test_norm_refusals(lib):
    tw = _rec(L.RECIPE_TENSORWISE)
    assert lib.fp8_rmsnorm_quantize(ctypes.byref(_rec()), None, 1, 1, None, None, None,
                                    ctypes.byref(_tensor()), None, 0, None, None) == NULL
    assert _norm(lib, rec=False) == NULL                       # copies need a recipe
    assert _norm(lib, out=False) == NULL
    assert _norm(lib, wr=0, wc=0) == SHAPE                     # nothing to compute
    assert _norm(lib, rec=_rec(9)) == UNSUPPORTED
    assert _norm(lib, rec=_rec(format=1)) == UNSUPPORTED       # mxfp8 is E4M3 only
    assert _norm(lib, inp=_in(cols=192, ldx=256)) == SHAPE     # MXFP8: a multiple of 128
    assert _norm(lib, tw, _in(cols=200)) == SHAPE              # tensorwise: of 16
    assert _norm(lib, inp=_in(cols=32768 + 128, ldx=1 << 20, ldr=1 << 20)) == SHAPE
    assert _norm(lib, inp=_in(rows=-1)) == SHAPE
    assert _norm(lib, inp=_in(rows=(1 << 31) // 256)) == SHAPE  # 2^31 padded elements
    assert _norm(lib, inp=_in(ldx=248)) == SHAPE
    assert _norm(lib, inp=_in(ldx=260)) == SHAPE               # not a multiple of 8
    assert _norm(lib, inp=_in(ldr=128)) == SHAPE
    assert _norm(lib, inp=_in(eps=-1e-5)) == UNSUPPORTED
    assert _norm(lib, inp=_in(eps=math.nan)) == UNSUPPORTED
    assert _norm(lib, inp=_in(eps=math.inf)) == UNSUPPORTED
    assert _norm(lib, inp=_in(gamma_fp32=2)) == UNSUPPORTED
    assert _norm(lib, inp=_in(x=0)) == NULL
    assert _norm(lib, inp=_in(x=0x8008)) == ALIGN
    assert _norm(lib, inp=_in(gamma=0)) == NULL
    assert _norm(lib, inp=_in(residual=0x9004)) == ALIGN
    assert _norm(lib, h=None) == NULL                          # a residual needs h
    assert _norm(lib, h=0xB002) == ALIGN
    assert _norm(lib, inp=_in(ldr=512), h=0x9000) == SHAPE     # in place over strided rows
    assert _norm(lib, inp=_in(ldx=512), h=0x8000) == SHAPE
    assert _norm(lib, rstd=0xC002) == ALIGN
    assert _norm(lib, y=0xE008) == ALIGN
    assert _norm(lib, out=_tensor(row=0)) == NULL
    assert _norm(lib, out=_tensor(col_scale=0)) == NULL
    assert _norm(lib, out=_tensor(row_scale=0x3004)) == ALIGN
    assert _norm(lib, tw, out=_tensor(amax=0)) == NULL
    assert _norm(lib, ws=None) == WORKSPACE
    need = lib.fp8_rmsnorm_workspace_bytes(ctypes.byref(_rec()), 100, 256)
    assert need > 0 and _norm(lib, ws_bytes=need - 1) == WORKSPACE
    assert _norm(lib, ws=0xD004) == ALIGN
    t = _tensor()
    assert _norm(lib, inp=_in(x=0), out=t) == NULL and t.rows == 0     # untouched on refusal


def test_norm_bwd_refusals(lib):
    def bwd(dh=0xB000, dgamma=0xE000, ws=0xD000, ws_bytes=1 << 24, **kw):
        d = dict(dy=0x8000, h=0x9000, dres=0xA000, gamma=0xC000, rstd=0xF000, ld_dy=256,
                 ld_h=256, ld_dres=256, rows=100, cols=256, gamma_fp32=0)
        d.update(kw)
        inp = L.NormGrad(*[d[f] for f, _ in L.NormGrad._fields_])
        return lib.fp8_rmsnorm_bwd(ctypes.byref(inp), dh, dgamma, ws, ws_bytes, None, None)

    assert lib.fp8_rmsnorm_bwd(None, 0xB000, None, None, 0, None, None) == NULL
    for f in ("dy", "h", "gamma", "rstd"):
        assert bwd(**{f: 0}) == NULL
    for f in ("dy", "h", "dres", "gamma"):
        assert bwd(**{f: 0x8008}) == ALIGN
    assert bwd(rstd=0xF002) == ALIGN
    assert bwd(dh=None) == NULL and bwd(dh=0xB008) == ALIGN and bwd(dgamma=0xE004) == ALIGN
    for f in ("ld_dy", "ld_h", "ld_dres"):
        assert bwd(**{f: 248}) == SHAPE and bwd(**{f: 260}) == SHAPE
    assert bwd(cols=200) == SHAPE and bwd(cols=32784) == SHAPE and bwd(rows=-1) == SHAPE
    assert bwd(dh=0x8000, ld_dy=512) == SHAPE and bwd(dh=0xA000, ld_dres=512) == SHAPE
    assert bwd(gamma_fp32=3) == UNSUPPORTED
    need = lib.fp8_rmsnorm_bwd_workspace_bytes(100, 256)
    assert need > 0
    assert bwd(ws=None) == WORKSPACE and bwd(ws_bytes=need - 1) == WORKSPACE
    assert bwd(ws=0xD008) == ALIGN
    assert bwd(rows=0, dgamma=None) == 0                        # nothing to do


def test_grad_refusals(lib):
    def items(*its):
        return (L.GradItem * max(1, len(its)))(*[L.GradItem(*i) for i in its])

    ok = (0x8000, 0x9000, 100, 0, 1)

    def norm(its=(ok,), n=None, max_norm=1.0, scale=1.0, norm=0xA000, coef=0xB000, ws=0xC000,
             ws_bytes=1 << 20):
        return lib.fp8_grad_norm(len(its) if n is None else n, items(*its),
                                 ctypes.byref(L.ClipRule(max_norm, scale)), norm, coef, ws,
                                 ws_bytes, None)

    assert lib.fp8_grad_norm(1, items(ok), None, 0xA000, None, 0xC000, 1 << 20, None) == NULL
    assert lib.fp8_grad_norm(1, None, ctypes.byref(L.ClipRule(1.0, 1.0)), 0xA000, None, 0xC000,
                             1 << 20, None) == NULL
    assert norm(n=-1) == SHAPE
    for m in (0.0, -1.0, math.nan):
        assert norm(max_norm=m) == UNSUPPORTED
    for s in (0.0, -1.0, math.nan, math.inf):
        assert norm(scale=s) == UNSUPPORTED
    assert norm(norm=None) == NULL and norm(norm=0xA002) == ALIGN and norm(coef=0xB001) == ALIGN
    assert norm(its=(ok, (0, 0, 4, 0, 0))) == NULL
    assert norm(its=((0x8001, 0, 4, 0, 0),)) == ALIGN
    assert norm(its=((0x8002, 0, 4, 1, 0),)) == ALIGN
    assert norm(its=((0x8000, 0, -4, 0, 0),)) == SHAPE
    assert norm(its=((0x8000, 0, 1 << 43, 0, 0),)) == SHAPE
    assert norm(its=((0x8000, 0, 1 << 42, 0, 0),) * 2) == SHAPE
    assert norm(its=((0x8000, 0, 4, 2, 0),)) == UNSUPPORTED
    assert norm(ws=None) == WORKSPACE and norm(ws_bytes=8) == WORKSPACE
    assert norm(ws=0xC008) == ALIGN
    assert lib.fp8_grad_workspace_bytes(-1) == 0
    assert lib.fp8_grad_workspace_bytes(5000) > lib.fp8_grad_workspace_bytes(10) > 0

    def clip(*its, coef=0xA000):
        return lib.fp8_grad_clip(len(its), items(*its), coef, None)

    assert clip(ok, coef=None) == NULL and clip(ok, coef=0xA002) == ALIGN
    assert clip((0x8000, 0, 4, 0, 0)) == NULL
    assert clip((0x8000, 0x9002, 4, 0, 1)) == ALIGN
    assert clip((0x8000, 0x9000, 4, 0, 7)) == UNSUPPORTED
    assert clip((0x8000, 0x8000, 4, 0, 1)) == UNSUPPORTED       # in place needs one type


def test_binding_refusals():
    """What the Python binding refuses before it looks at an address (CPU tensors)."""
    bf, rec = torch.bfloat16, binding.Recipe(kind="mxfp8")
    x, g = torch.zeros(4, 256, dtype=bf), torch.zeros(256, dtype=bf)
    with pytest.raises(TypeError):
        binding.rmsnorm_quantize(rec, x.float(), g)
    with pytest.raises(ValueError):
        binding.rmsnorm_quantize(rec, torch.zeros(256, 4, dtype=bf).t(), g)
    with pytest.raises(ValueError):
        binding.rmsnorm_quantize(rec, x, g[:128])
    with pytest.raises(TypeError):
        binding.rmsnorm_quantize(rec, x, g.double())
    with pytest.raises(ValueError):
        binding.rmsnorm_quantize(rec, x, g, residual=x[:2])
    with pytest.raises(ValueError):
        binding.rmsnorm_quantize(rec, x, g, rstd=torch.zeros(5))
    with pytest.raises(ValueError):                            # not padded to 128 rows
        binding.rmsnorm_quantize(rec, x, g, out=binding.empty_qtensor(rec, 4, 256, device="cpu"))
    with pytest.raises(ValueError):
        binding.rmsnorm_bwd(x, x[:3], torch.zeros(4), g)
    with pytest.raises(ValueError):
        binding.rmsnorm_bwd(x, x, torch.zeros(4), g, dres=x[:3])
    with pytest.raises(TypeError):
        binding.GradList([x.double()])
    with pytest.raises(ValueError):
        binding.GradList([x[:, ::2]])
    with pytest.raises(ValueError):
        binding.GradList([x], [x, x])
    with pytest.raises(ValueError):
        binding.GradList([x], [torch.zeros(256, 4, dtype=bf).t()])
    with pytest.raises(TypeError):
        binding.grad_clip([x], torch.zeros(1, dtype=torch.float64))
    assert len(binding.GradList([x, x.t(), torch.zeros(3, 5, 7).permute(2, 0, 1)])) == 3


def test_binding_refuses_cpu_tensors():
    """Well-formed calls on CPU tensors: the library would take their addresses for the GPU's."""
    x, g = torch.zeros(4, 256, dtype=torch.bfloat16), torch.ones(256)
    out = torch.empty_like(x)
    with pytest.raises(TypeError):
        binding.rmsnorm(x, g, y=out)
    with pytest.raises(TypeError):
        binding.rmsnorm_bwd(x, x, torch.ones(4), g)
    with pytest.raises(TypeError):
        binding.grad_norm([x])
    with pytest.raises(TypeError):
        binding.grad_clip([x], torch.ones(1))
    with pytest.raises(TypeError):
        binding.grad_norm([x], norm=torch.zeros(2))

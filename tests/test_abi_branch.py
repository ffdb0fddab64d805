"""C ABI and binding checks, without a GPU, of the gated branch, its backward pass and the 8-bit
checkpoints: struct layouts, and what is refused on the host before anything is launched."""
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


STRUCTS = {"fp8_checkpoint": L.Checkpoint, "fp8_branch_input": L.BranchInput,
           "fp8_branch_grad": L.BranchGrad, "fp8_branch_grad_out": L.BranchGradOut}


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


def test_packed_forms_are_the_structures():
    """The bytes that the binding builds for each call."""
    assert L.pack_checkpoint(1, 2) == bytes(L.Checkpoint(1, 2))
    v = list(range(1, 14)) + [0.5, 0.25, 0.125]
    assert L.pack_branch_input(*v) == bytes(L.BranchInput(*v))
    p, q = list(range(1, 5)), list(range(9, 24))
    assert L.pack_branch_grad(*p, 5, 6, 7, 8, *q, 0.5) == bytes(
        L.BranchGrad(*p, L.Checkpoint(5, 6), L.Checkpoint(7, 8), *q, 0.5))
    assert L.pack_branch_grad_out(*range(1, 7)) == bytes(L.BranchGradOut(*range(1, 7)))


def _rec(kind=L.RECIPE_MXFP8, **kw):
    r = L.Recipe(kind, 0, 0, 16, 0, 1, 0)
    for k, v in kw.items():
        setattr(r, k, v)
    return r


def _tensor(**kw):
    d = dict(row=0x1000, col=0x2000, row_scale=0x3000, col_scale=0x4000, amax=0x5000,
             scale=0x6000, scale_inv=0x7000)
    d.update(kw)
    return L.Tensor(*[d[f] for f in ("row", "col", "row_scale", "col_scale", "amax", "scale",
                                     "scale_inv")], 0, 0, 0, 0, 0)


def _branch(lib, rec=None, wr=1, wc=1, h=0xB000, rstd_o=0xC100, rstd=0xC000, y=None, o_ck=None,
            h_ck=None, out=None, ws=0xD000, ws_bytes=1 << 20, none=False, **kw):
    d = dict(branch=0x8000, residual=0x9000, gamma_post=0xA000, gate=0xA100, token_gate=0xA204,
             gamma=0xA300, ld_branch=256, ld_residual=256, rows=100, cols=256, gamma_post_fp32=0,
             gate_fp32=1, gamma_fp32=0, scale=0.5, eps_post=1e-5, eps=1e-5)
    d.update(kw)
    inp = None if none else ctypes.byref(
        L.BranchInput(*[d[f] for f, _ in L.BranchInput._fields_]))
    rec = _rec() if rec is None else rec
    out = _tensor() if out is None else out
    ref = [None if c is None else ctypes.byref(L.Checkpoint(*c)) for c in (o_ck, h_ck)]
    return lib.fp8_branch_rmsnorm_quantize(ctypes.byref(rec) if rec else None, inp, wr, wc, h,
                                           rstd_o, rstd, y, *ref,
                                           ctypes.byref(out) if out else None, ws, ws_bytes, None,
                                           None)


def test_branch_refusals(lib):
    tw = _rec(L.RECIPE_TENSORWISE)
    assert _branch(lib, none=True) == NULL
    assert _branch(lib, rec=False) == NULL and _branch(lib, out=False) == NULL
    assert _branch(lib, wr=0, wc=0) == SHAPE                   # nothing to compute
    assert _branch(lib, rec=_rec(9)) == UNSUPPORTED
    assert _branch(lib, cols=192) == SHAPE                     # MXFP8: a multiple of 128
    assert _branch(lib, tw, cols=200) == SHAPE                 # tensorwise: of 16
    assert _branch(lib, cols=32768 + 128, ld_branch=1 << 20, ld_residual=1 << 20) == SHAPE
    assert _branch(lib, rows=-1) == SHAPE
    assert _branch(lib, rows=(1 << 31) // 256) == SHAPE        # 2^31 padded elements
    assert _branch(lib, tw, wr=0, wc=0, y=0xE000, cols=16, rows=(1 << 30) + 1) == SHAPE
    for f in ("ld_branch", "ld_residual"):
        assert _branch(lib, **{f: 248}) == SHAPE and _branch(lib, **{f: 260}) == SHAPE
        assert _branch(lib, **{f: (1 << 30) + 8}) == SHAPE
    for f in ("eps", "eps_post"):
        for v in (-1e-5, math.nan, math.inf):
            assert _branch(lib, **{f: v}) == UNSUPPORTED
    for v in (math.nan, math.inf, -math.inf):
        assert _branch(lib, scale=v) == UNSUPPORTED
    for f in ("gamma_post_fp32", "gate_fp32", "gamma_fp32"):
        assert _branch(lib, **{f: 2}) == UNSUPPORTED
    for f in ("branch", "residual", "gamma"):
        assert _branch(lib, **{f: 0}) == NULL and _branch(lib, **{f: 0x8008}) == ALIGN
    for f in ("gamma_post", "gate"):
        assert _branch(lib, **{f: 0x8008}) == ALIGN
    assert _branch(lib, token_gate=0xA202) == ALIGN
    assert _branch(lib, h=None) == NULL and _branch(lib, h=0xB002) == ALIGN
    assert _branch(lib, ld_residual=512, h=0x9000) == SHAPE    # in place over strided rows
    assert _branch(lib, ld_branch=512, h=0x8000) == SHAPE
    assert _branch(lib, rstd=0xC002) == ALIGN and _branch(lib, rstd_o=0xC102) == ALIGN
    assert _branch(lib, y=0xE008) == ALIGN
    assert _branch(lib, o_ck=(0, 0x1000)) == NULL and _branch(lib, h_ck=(0x1000, 0)) == NULL
    assert _branch(lib, o_ck=(0x1008, 0x2000)) == ALIGN
    assert _branch(lib, h_ck=(0x1000, 0x2004)) == ALIGN
    # one buffer for two outputs
    assert _branch(lib, rstd=0xC000, rstd_o=0xC000) == SHAPE
    assert _branch(lib, h=0xB000, y=0xB000) == SHAPE
    assert _branch(lib, o_ck=(0x1000, 0x2000), h_ck=(0x1000, 0x3000)) == SHAPE
    assert _branch(lib, o_ck=(0x1000, 0x2000), h_ck=(0x4000, 0x2000)) == SHAPE
    assert _branch(lib, out=_tensor(row=0)) == NULL
    assert _branch(lib, out=_tensor(col_scale=0)) == NULL
    assert _branch(lib, tw, out=_tensor(amax=0)) == NULL
    need = lib.fp8_rmsnorm_workspace_bytes(ctypes.byref(_rec()), 100, 256)
    assert _branch(lib, ws=None) == WORKSPACE and _branch(lib, ws_bytes=need - 1) == WORKSPACE
    assert _branch(lib, ws=0xD004) == ALIGN
    t = _tensor()
    assert _branch(lib, branch=0, out=t) == NULL and t.rows == 0       # untouched on refusal


def _bwd(lib, ws=0xD000, ws_bytes=1 << 24, out=None, none=False, **kw):
    d = dict(dy=0x8000, dres=0x8100, h=0x9000, branch=0x9100, h_ckpt=(0, 0), branch_ckpt=(0, 0),
             gamma_post=0xA000, gate=0xA100, token_gate=0xA204, gamma=0xA300, rstd_branch=0xF000,
             rstd=0xF100, ld_dy=256, ld_dres=256, ld_h=256, ld_branch=256, rows=100, cols=256,
             gamma_post_fp32=0, gate_fp32=0, gamma_fp32=0, scale=1.0)
    o = dict(dh=0xB000, dbranch=0xB100, dgamma=0xE000, dgamma_post=0xE100, dgate=0xE200,
             dtoken_gate=0xE304)
    o.update({k: v for k, v in kw.items() if k in o})
    d.update({k: v for k, v in kw.items() if k in d})
    d["h_ckpt"], d["branch_ckpt"] = L.Checkpoint(*d["h_ckpt"]), L.Checkpoint(*d["branch_ckpt"])
    inp = L.BranchGrad(*[d[f] for f, _ in L.BranchGrad._fields_])
    res = L.BranchGradOut(*[o[f] for f, _ in L.BranchGradOut._fields_])
    return lib.fp8_branch_rmsnorm_bwd(None if none else ctypes.byref(inp), ctypes.byref(res), ws,
                                      ws_bytes, None, None)


def test_branch_bwd_refusals(lib):
    assert _bwd(lib, none=True) == NULL
    assert lib.fp8_branch_rmsnorm_bwd(ctypes.byref(L.BranchGrad()), None, None, 0, None,
                                      None) == NULL
    for f in ("dy", "h", "branch", "gamma", "rstd", "rstd_branch", "dh", "dbranch"):
        assert _bwd(lib, **{f: 0}) == NULL, f
    for f in ("dy", "dres", "h", "branch", "gamma", "gamma_post", "gate", "dh", "dbranch",
              "dgamma", "dgamma_post", "dgate"):
        assert _bwd(lib, **{f: 0x8008}) == ALIGN, f
    for f in ("rstd", "rstd_branch", "token_gate", "dtoken_gate"):
        assert _bwd(lib, **{f: 0xF002}) == ALIGN, f
    for f in ("ld_dy", "ld_dres", "ld_h", "ld_branch"):
        for v in (248, 260, (1 << 30) + 8):
            assert _bwd(lib, **{f: v}) == SHAPE, f
    # a checkpoint stands in for the tensor, and is checked instead
    assert _bwd(lib, h=0, ld_h=0, h_ckpt=(0x9008, 0x9100)) == ALIGN
    assert _bwd(lib, branch=0, ld_branch=0, branch_ckpt=(0x9000, 0)) == NULL
    assert _bwd(lib, h=0, ld_h=0, h_ckpt=(0x9000, 0x9100), ws=None) == WORKSPACE
    # gradients of what is not there
    assert _bwd(lib, gamma_post=0) == NULL and _bwd(lib, gate=0) == NULL
    assert _bwd(lib, token_gate=0) == NULL
    for f in ("gamma_post_fp32", "gate_fp32", "gamma_fp32"):
        assert _bwd(lib, **{f: 3}) == UNSUPPORTED
    assert _bwd(lib, scale=math.nan) == UNSUPPORTED
    assert _bwd(lib, cols=200) == SHAPE and _bwd(lib, cols=32784) == SHAPE
    assert _bwd(lib, rows=-1) == SHAPE and _bwd(lib, rows=(1 << 30) + 1) == SHAPE
    # one buffer for two outputs; in place over strided rows
    assert _bwd(lib, dh=0xB100) == SHAPE
    for a, b in (("dgamma", "dgamma_post"), ("dgamma", "dgate"), ("dgamma_post", "dgate")):
        assert _bwd(lib, **{a: 0xE400, b: 0xE400}) == SHAPE
    for f, ld in (("dy", "ld_dy"), ("dres", "ld_dres"), ("h", "ld_h"), ("branch", "ld_branch")):
        for o in ("dh", "dbranch"):
            assert _bwd(lib, **{f: 0x4000, ld: 512, o: 0x4000}) == SHAPE
    need = lib.fp8_branch_rmsnorm_bwd_workspace_bytes(100, 256)
    assert need > 0 and lib.fp8_branch_rmsnorm_bwd_workspace_bytes(0, 256) == 0
    assert _bwd(lib, ws=None) == WORKSPACE and _bwd(lib, ws_bytes=need - 1) == WORKSPACE
    assert _bwd(lib, ws=0xD008) == ALIGN
    assert _bwd(lib, rows=0, dgamma=0, dgamma_post=0, dgate=0) == 0    # nothing to do
    assert _bwd(lib, cols=0) == 0


def test_checkpoint_refusals(lib):
    assert lib.fp8_checkpoint_scale_bytes(3, 16) == 12
    assert lib.fp8_checkpoint_scale_bytes(3, 144) == 24
    assert lib.fp8_checkpoint_scale_bytes(0, 16) == 0

    def write(x=0x8000, ldx=256, rows=10, cols=256, ck=(0x1000, 0x2000)):
        c = None if ck is None else ctypes.byref(L.Checkpoint(*ck))
        return lib.fp8_checkpoint_write(x, ldx, rows, cols, c, None)

    def read(x=0x8000, rows=10, cols=256, ck=(0x1000, 0x2000)):
        c = None if ck is None else ctypes.byref(L.Checkpoint(*ck))
        return lib.fp8_checkpoint_read(c, rows, cols, x, None)

    for call in (write, read):
        assert call(ck=None) == NULL and call(x=None) == NULL and call(x=0x8008) == ALIGN
        assert call(ck=(0, 0x2000)) == NULL and call(ck=(0x1000, 0)) == NULL
        assert call(ck=(0x1004, 0x2000)) == ALIGN and call(ck=(0x1000, 0x2002)) == ALIGN
        assert call(cols=200) == SHAPE and call(rows=-1) == SHAPE and call(cols=-16) == SHAPE
        assert call(rows=1 << 40) == SHAPE
        assert call(rows=0, x=None, ck=(0, 0)) == 0 and call(cols=0, x=None) == 0
    assert write(ldx=248) == SHAPE and write(ldx=260) == SHAPE

    def norm_bwd(ck=(0x9000, 0x9100), ws=0xD000, **kw):
        d = dict(dy=0x8000, h=0, dres=0, gamma=0xC000, rstd=0xF000, ld_dy=256, ld_h=0, ld_dres=0,
                 rows=100, cols=256, gamma_fp32=0)
        d.update(kw)
        inp = L.NormGrad(*[d[f] for f, _ in L.NormGrad._fields_])
        c = None if ck is None else ctypes.byref(L.Checkpoint(*ck))
        return lib.fp8_rmsnorm_bwd_checkpoint(ctypes.byref(inp), c, 0xB000, 0xE000, ws, 1 << 24,
                                              None, None)

    assert norm_bwd(ck=None) == NULL and norm_bwd(ck=(0, 0x9100)) == NULL
    assert norm_bwd(ck=(0x9000, 0x9104)) == ALIGN and norm_bwd(dy=0) == NULL
    assert norm_bwd(ws=None) == WORKSPACE and norm_bwd(cols=200) == SHAPE

    def quant(rec=None, ck=(0x9000, 0x9100), rows=100, cols=256, rstd=0xF000, gamma=0xC000,
              fp32=0, wr=1, wc=1, out=None, ws=0xD000, ws_bytes=1 << 20):
        rec = _rec() if rec is None else rec
        c = None if ck is None else ctypes.byref(L.Checkpoint(*ck))
        t = _tensor() if out is None else out
        return lib.fp8_checkpoint_quantize(ctypes.byref(rec), c, rows, cols, rstd, gamma, fp32, wr,
                                           wc, ctypes.byref(t), ws, ws_bytes, None, None)

    assert quant(ck=None) == NULL and quant(ck=(0x9000, 0)) == NULL
    assert quant(ck=(0x9008, 0x9100)) == ALIGN
    assert quant(rstd=None) == NULL and quant(gamma=None) == NULL      # both or neither
    assert quant(rstd=0xF002) == ALIGN and quant(gamma=0xC008) == ALIGN
    assert quant(fp32=2) == UNSUPPORTED and quant(rec=_rec(format=1)) == UNSUPPORTED
    assert quant(wr=0, wc=0) == SHAPE and quant(cols=192) == SHAPE and quant(rows=-1) == SHAPE
    assert quant(rows=(1 << 31) // 256) == SHAPE
    assert quant(out=_tensor(row=0)) == NULL and quant(out=_tensor(col_scale=0x4004)) == ALIGN
    assert quant(rec=_rec(L.RECIPE_DELAYED), out=_tensor(scale=0)) == NULL
    assert quant(ws=None) == WORKSPACE


def _bf(*shape):
    return torch.zeros(*shape, dtype=torch.bfloat16)


def test_binding_refusals():
    """What the Python binding refuses before it looks at an address (CPU tensors)."""
    rec, x, g = binding.Recipe(kind="mxfp8"), _bf(4, 256), _bf(256)
    call = binding.branch_rmsnorm_quantize
    for bad in (dict(branch=x.float()), dict(residual=x.float()), dict(gamma=g.double()),
                dict(gamma_post=g.double()), dict(gate=g.half()), dict(branch=g)):
        with pytest.raises(TypeError):
            call(**{**dict(recipe=rec, branch=x, residual=x, gamma=g), **bad})
    ck = binding.empty_checkpoint(4, 256, device="cpu")
    for bad in (dict(residual=x[:2]), dict(branch=_bf(256, 4).t()), dict(gamma=g[:128]),
                dict(gamma_post=g[:128]), dict(gate=g[:1].expand(256)), dict(gate=x),
                dict(token_gate=torch.zeros(5)), dict(token_gate=_bf(4)),
                dict(rstd=torch.zeros(5)), dict(gamma_post=g, rstd_branch=torch.zeros(5)),
                dict(h=_bf(4, 128)), dict(y=x.float()),
                dict(out=binding.empty_qtensor(rec, 4, 256, device="cpu")),
                dict(h_ckpt=binding.empty_checkpoint(4, 128, device="cpu")),
                dict(branch_ckpt=binding.Checkpoint(ck.codes, ck.scale[:2])),
                dict(h_ckpt=binding.Checkpoint(ck.codes.to(torch.int32), ck.scale)),
                dict(h_ckpt=binding.Checkpoint(ck.codes[:1].expand(4, 256), ck.scale))):
        with pytest.raises((ValueError, TypeError)):
            call(**{**dict(recipe=rec, branch=x, residual=x, gamma=g), **bad})
    back = binding.branch_rmsnorm_bwd
    one = torch.zeros(4)
    for bad in (dict(dy=x[:3]), dict(dy=g), dict(branch=_bf(4, 128)), dict(rstd=torch.zeros(5)),
                dict(gamma_post=g), dict(gamma_post=g, rstd_branch=torch.zeros(3)),
                dict(dres=x[:2]), dict(token_gate=torch.zeros(4, 1)), dict(dh=x.float()),
                dict(dgamma=_bf(256)), dict(gate=g, dgate=torch.zeros(255)),
                dict(token_gate=one, dtoken_gate=torch.zeros(5)),
                dict(h=binding.Checkpoint(ck.codes, ck.scale[:2]))):
        with pytest.raises((ValueError, TypeError)):
            back(**{**dict(dy=x, h=x, rstd=one, gamma=g, branch=x), **bad})
    with pytest.raises(TypeError):
        binding.checkpoint(x.float())
    with pytest.raises(TypeError):
        binding.checkpoint(g)
    with pytest.raises(ValueError):
        binding.checkpoint(x, out=binding.empty_checkpoint(4, 128, device="cpu"))
    with pytest.raises(ValueError):
        binding.checkpoint_read(ck, out=_bf(4, 128))
    with pytest.raises(ValueError):
        binding.checkpoint_quantize(rec, ck, rstd=one)
    with pytest.raises(ValueError):
        binding.checkpoint_quantize(rec, ck, out=binding.empty_qtensor(rec, 4, 256, device="cpu"))
    with pytest.raises(ValueError):
        binding.rmsnorm_bwd(x, binding.Checkpoint(ck.codes, ck.scale[:2]), one, g)


def test_binding_refuses_cpu_tensors():
    """Well-formed calls on CPU tensors: the library would take their addresses for the GPU's."""
    rec, x, g, one = binding.Recipe(kind="mxfp8"), _bf(4, 256), _bf(256), torch.zeros(4)
    ck = binding.empty_checkpoint(4, 256, device="cpu")
    for call in (lambda: binding.branch_rmsnorm_quantize(rec, x, x, g),
                 lambda: binding.branch_rmsnorm_bwd(x, x, one, g, x),
                 lambda: binding.branch_rmsnorm_bwd(x, ck, one, g, ck),
                 lambda: binding.rmsnorm_bwd(x, ck, one, g),
                 lambda: binding.checkpoint(x), lambda: binding.checkpoint(x, out=ck),
                 lambda: binding.checkpoint_read(ck),
                 lambda: binding.checkpoint_quantize(rec, ck)):
        with pytest.raises(TypeError, match="CUDA"):
            call()


def test_a_checkpoint_has_the_shape_of_its_tensor():
    ck = binding.empty_checkpoint(3, 144, device="cpu")
    assert ck.shape == (3, 144) and ck.scale.shape == (3, 8) and ck.device.type == "cpu"


def test_one_buffer_for_a_gate_gradient_and_a_sum(lib):
    for name in ("dgamma", "dgamma_post", "dgate"):
        assert _bwd(lib, dtoken_gate=0xE800, **{name: 0xE800}) == SHAPE

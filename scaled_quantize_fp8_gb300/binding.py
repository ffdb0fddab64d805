"""Python binding of the FP8 linear-layer C ABI: torch allocates device buffers and supplies
the stream; every step of the computation runs in the library's CUDA kernels.

Names follow the C ABI: quantize, amax_update, linear_fwd, linear_bwd, gelu_quantize,
dgelu_quantize. A quantised tensor is a QTensor holding its torch buffers; its C view is
built on demand.
"""
import ctypes
from dataclasses import dataclass, field
from typing import Optional

import torch

from . import _lib as L

KINDS = {"delayed": L.RECIPE_DELAYED, "tensorwise": L.RECIPE_TENSORWISE,
         "mxfp8": L.RECIPE_MXFP8, "blockwise": L.RECIPE_BLOCKWISE}
ROLES = {"activation": L.ROLE_ACTIVATION, "weight": L.ROLE_WEIGHT, "grad": L.ROLE_GRAD}


@dataclass
class Recipe:
    """The recipe statement (--fp8-recipe, --fp8-format, --fp8-margin,
    --fp8-amax-history-len, --fp8-amax-compute-algo, --fp8-wgrad)."""
    kind: str = "delayed"
    format: str = "e4m3"
    margin: int = 0
    amax_history_len: int = 1024
    amax_compute_algo: str = "max"
    fp8_wgrad: bool = True
    power_2_scales: bool = False

    def _fields(self):
        """The fields of the library's form, in order."""
        return (KINDS[self.kind], 0 if self.format == "e4m3" else 1, int(self.margin),
                int(self.amax_history_len), 0 if self.amax_compute_algo == "max" else 1,
                1 if self.fp8_wgrad else 0, 1 if self.power_2_scales else 0)

    def c(self):
        return L.Recipe(*self._fields())


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(stream=None):
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


@dataclass
class QTensor:
    """Codes and scales of one quantised tensor of source shape [rows, cols]."""
    rows: int
    cols: int
    kind: int
    role: int
    row: Optional[torch.Tensor] = None        # uint8 [rows, cols]
    col: Optional[torch.Tensor] = None        # uint8 [cols, rows]
    row_scale: Optional[torch.Tensor] = None
    col_scale: Optional[torch.Tensor] = None
    amax: Optional[torch.Tensor] = None       # float32 [1]
    scale: Optional[torch.Tensor] = None
    scale_inv: Optional[torch.Tensor] = None
    col_bf16: int = 0                         # 1: `col` is the bf16 transpose (wgrad in bf16)
    _c: object = field(default=None, repr=False)

    def c(self):
        row, col, rs, cs = self.row, self.col, self.row_scale, self.col_scale
        amax, scale, inv = self.amax, self.scale, self.scale_inv
        self._c = t = L.Tensor()
        L.pack_tensor(                               # half the time of the fields as arguments
            t, 0, 0 if row is None else row.data_ptr(), 0 if col is None else col.data_ptr(),
            0 if rs is None else rs.data_ptr(), 0 if cs is None else cs.data_ptr(),
            0 if amax is None else amax.data_ptr(), 0 if scale is None else scale.data_ptr(),
            0 if inv is None else inv.data_ptr(), self.rows, self.cols, self.kind, self.role,
            self.col_bf16)
        return t


def scale_shape(kind, role, rows, cols, pow2=False):
    """Storage of the scales of one copy whose codes are [rows, cols] (blocks along cols).
    Blockwise with power-of-two scales stores E8M0 bytes in the MXFP8 layout."""
    if kind == L.RECIPE_MXFP8 or (kind == L.RECIPE_BLOCKWISE and pow2):
        return (rows * cols // 32,), torch.uint8
    if kind == L.RECIPE_BLOCKWISE:
        if role == L.ROLE_WEIGHT:
            return (rows // 128, cols // 128), torch.float32
        return (cols // 128, rows), torch.float32
    return None, None


def empty_qtensor(recipe: Recipe, rows, cols, role="activation", want_row=True, want_col=True,
                  device="cuda"):
    kind, r = KINDS[recipe.kind], ROLES[role]
    q = QTensor(rows, cols, kind, r)
    if want_row:
        q.row = torch.empty((rows, cols), dtype=torch.uint8, device=device)
        shp, dt = scale_shape(kind, r, rows, cols, recipe.power_2_scales)
        if shp is not None:
            q.row_scale = torch.empty(shp, dtype=dt, device=device)
    if want_col:
        if not recipe.fp8_wgrad and r != L.ROLE_WEIGHT:
            # --fp8-wgrad off: the column copy is the bf16 transpose, read by the bf16 wgrad
            q.col = torch.empty((cols, rows), dtype=torch.bfloat16, device=device)
            q.col_bf16 = 1
        else:
            q.col = torch.empty((cols, rows), dtype=torch.uint8, device=device)
            shp, dt = scale_shape(kind, r, cols, rows, recipe.power_2_scales)
            if shp is not None:
                q.col_scale = torch.empty(shp, dtype=dt, device=device)
    if kind in (L.RECIPE_DELAYED, L.RECIPE_TENSORWISE):
        q.amax = torch.zeros(1, dtype=torch.float32, device=device)
        q.scale = torch.ones(1, dtype=torch.float32, device=device)
        q.scale_inv = torch.ones(1, dtype=torch.float32, device=device)
    return q


def workspace_bytes(recipe: Recipe, rows, cols):
    rc = recipe.c()
    return int(L.load().fp8_workspace_bytes(ctypes.byref(rc), rows, cols))


def quantize(recipe: Recipe, x: torch.Tensor, role="activation", want_row=True, want_col=True,
             out: Optional[QTensor] = None, workspace: Optional[torch.Tensor] = None,
             status: Optional[torch.Tensor] = None, stream=None):
    """fp8_quantize on a bf16 [rows, cols] tensor. For delayed scaling pass `out` whose
    scale / scale_inv hold the scale from the history (DelayedState.bind)."""
    lib = L.load()
    rows, cols = x.shape
    if out is None:
        out = empty_qtensor(recipe, rows, cols, role, want_row, want_col, device=x.device)
    rc = recipe.c()
    need = int(lib.fp8_workspace_bytes(ctypes.byref(rc), rows, cols))
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=x.device)
    ct = out.c()
    st = lib.fp8_quantize(ctypes.byref(rc), _ptr(x), rows, cols, ROLES[role], int(want_row),
                          int(want_col), ctypes.byref(ct), _ptr(workspace),
                          0 if workspace is None else workspace.numel(), _ptr(status),
                          _stream(stream))
    L.check(st, "fp8_quantize")
    out.rows, out.cols, out.kind, out.role = ct.rows, ct.cols, ct.kind, ct.role
    out.col_bf16 = ct.col_bf16
    return out


def quantize_group(recipe: Recipe, xs, roles, outs=None, want_row=True, want_col=True,
                   status: Optional[torch.Tensor] = None, stream=None, _stalled=False):
    """fp8_quantize_group: up to four bf16 [rows, cols] tensors quantised by one MXFP8 launch.
    `roles` and `outs` (QTensors, or None to allocate) run parallel to `xs`. `_stalled` calls
    the test hook fp8_test_quantize_group_stalled instead (the group's first tile never
    arrives, so CTA 0's bounded wait runs out and records FP8_ERR_TIMEOUT in `status`)."""
    lib = L.load()
    n = len(xs)
    if outs is None:
        outs = [None] * n
    outs = [o if o is not None else
            empty_qtensor(recipe, x.shape[0], x.shape[1], r, want_row, want_col, device=x.device)
            for x, r, o in zip(xs, roles, outs)]
    rc = recipe.c()
    cts = [o.c() for o in outs]
    items = (L.QuantizeItem * max(1, n))()
    for i, (x, r) in enumerate(zip(xs, roles)):
        items[i] = L.QuantizeItem(_ptr(x), x.shape[0], x.shape[1], ROLES[r], int(want_row),
                                  int(want_col), ctypes.pointer(cts[i]))
    fn = lib.fp8_test_quantize_group_stalled if _stalled else lib.fp8_quantize_group
    st = fn(ctypes.byref(rc), n, items, _ptr(status), _stream(stream))
    L.check(st, "fp8_quantize_group")
    for o, ct in zip(outs, cts):
        o.rows, o.cols, o.kind, o.role, o.col_bf16 = ct.rows, ct.cols, ct.kind, ct.role, ct.col_bf16
    return outs


def quantize_master(recipe: Recipe, w: torch.Tensor, want_row=True, want_col=True,
                    out: Optional[QTensor] = None, workspace: Optional[torch.Tensor] = None,
                    status: Optional[torch.Tensor] = None, stream=None):
    """fp8_quantize_master on an fp32 [rows, cols] master weight (role weight, no bf16
    rounding). For delayed scaling pass `out` bound to the weight's DelayedState."""
    if w.dtype != torch.float32:
        raise TypeError("quantize_master takes fp32 master weights")
    lib = L.load()
    rows, cols = w.shape
    if out is None:
        out = empty_qtensor(recipe, rows, cols, "weight", want_row, want_col, device=w.device)
    rc = recipe.c()
    need = int(lib.fp8_workspace_bytes(ctypes.byref(rc), rows, cols))
    if need and (workspace is None or workspace.numel() < need):
        workspace = torch.empty(need, dtype=torch.uint8, device=w.device)
    ct = out.c()
    st = lib.fp8_quantize_master(ctypes.byref(rc), _ptr(w), rows, cols, int(want_row),
                                 int(want_col), ctypes.byref(ct), _ptr(workspace),
                                 0 if workspace is None else workspace.numel(), _ptr(status),
                                 _stream(stream))
    L.check(st, "fp8_quantize_master")
    out.rows, out.cols, out.kind, out.role = ct.rows, ct.cols, ct.kind, ct.role
    out.col_bf16 = ct.col_bf16
    return out


def quantize_static_scratch(recipe: Recipe, x: torch.Tensor, role="activation", want_row=True,
                            want_col=True, out: Optional[QTensor] = None, status=None,
                            stream=None):
    """fp8_quantize_static_scratch: like quantize(), but the library supplies the amax scratch
    from a fixed array in its device image, so the call allocates nothing (for callers that
    cannot allocate device memory). Calls that overlap on the GPU share that array and race."""
    lib = L.load()
    rows, cols = x.shape
    if out is None:
        out = empty_qtensor(recipe, rows, cols, role, want_row, want_col, device=x.device)
    rc = recipe.c()
    ct = out.c()
    st = lib.fp8_quantize_static_scratch(ctypes.byref(rc), _ptr(x), rows, cols, ROLES[role],
                                         int(want_row), int(want_col), ctypes.byref(ct),
                                         _ptr(status), _stream(stream))
    L.check(st, "fp8_quantize_static_scratch")
    out.rows, out.cols, out.kind, out.role = ct.rows, ct.cols, ct.kind, ct.role
    out.col_bf16 = ct.col_bf16
    return out


class DelayedState:
    """Device-resident delayed-scaling state: amax history, head, scale, scale_inv."""

    def __init__(self, recipe: Recipe, device="cuda", role="activation"):
        self.recipe = recipe
        self.role = role
        self.history = torch.zeros(recipe.amax_history_len, dtype=torch.float32, device=device)
        self.head = torch.zeros(1, dtype=torch.int32, device=device)
        self.scale = torch.ones(1, dtype=torch.float32, device=device)
        self.scale_inv = torch.ones(1, dtype=torch.float32, device=device)

    def bind(self, q: QTensor):
        """Point a QTensor's scale / scale_inv at this state (the cast reads them)."""
        q.scale, q.scale_inv = self.scale, self.scale_inv
        return q


def amax_update(recipe: Recipe, state: DelayedState, amax_new: torch.Tensor, stream=None):
    lib = L.load()
    rc = recipe.c()
    h = L.AmaxHistory(state.history.data_ptr(), state.head.data_ptr(), state.history.numel())
    st = lib.fp8_amax_update(ctypes.byref(rc), ctypes.byref(h), ROLES[state.role], _ptr(amax_new),
                             _ptr(state.scale), _ptr(state.scale_inv), _stream(stream))
    L.check(st, "fp8_amax_update")


def linear_fwd(recipe: Recipe, x: QTensor, w: QTensor, y: Optional[torch.Tensor] = None,
               fp32=False, status=None, stream=None):
    lib = L.load()
    if y is None:
        y = torch.empty((x.rows, w.rows), dtype=torch.float32 if fp32 else torch.bfloat16,
                        device=x.row.device)
    rc = recipe.c()
    st = lib.fp8_linear_fwd(ctypes.byref(rc), ctypes.byref(x.c()), ctypes.byref(w.c()), _ptr(y),
                            int(fp32), _ptr(status), _stream(stream))
    L.check(st, "fp8_linear_fwd")
    return y


def quantize_stalled(recipe: Recipe, x: torch.Tensor, role: str, out: QTensor,
                     status: torch.Tensor, stream=None):
    """Test hook (fp8_test_quantize_stalled): fp8_quantize with CTA 0's first tile never
    arriving, so its bounded wait runs out (about two seconds) and it records
    FP8_ERR_TIMEOUT in `status` (an int32 device word, zeroed by the caller)."""
    lib = L.load()
    rows, cols = x.shape
    rc = recipe.c()
    need = int(lib.fp8_workspace_bytes(ctypes.byref(rc), rows, cols))
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=x.device)
    ct = out.c()
    st = lib.fp8_test_quantize_stalled(ctypes.byref(rc), _ptr(x), rows, cols, ROLES[role], 1, 1,
                                       ctypes.byref(ct), _ptr(ws), ws.numel(), _ptr(status),
                                       _stream(stream))
    L.check(st, "fp8_test_quantize_stalled")
    return out


def linear_fwd_stalled(recipe: Recipe, x: QTensor, w: QTensor, y: torch.Tensor,
                       status: torch.Tensor, stream=None):
    """Test hook (fp8_test_linear_fwd_stalled): fp8_linear_fwd with a pipeline stage that
    never becomes ready, so the kernel's bounded wait runs out (about two seconds) and it
    records FP8_ERR_TIMEOUT in `status` (an int32 device word, zeroed by the caller)."""
    lib = L.load()
    rc = recipe.c()
    st = lib.fp8_test_linear_fwd_stalled(ctypes.byref(rc), ctypes.byref(x.c()),
                                         ctypes.byref(w.c()), _ptr(y), _ptr(status),
                                         _stream(stream))
    L.check(st, "fp8_test_linear_fwd_stalled")
    return y


def linear_bwd(recipe: Recipe, dy: QTensor, x: Optional[QTensor], w: Optional[QTensor],
               want_dx=True, want_dw=True, dx=None, dw=None, fp32=False, status=None,
               stream=None):
    """dgrad (dy row copy x w column copy) and wgrad (dy and x column copies; bf16 when the
    recipe has fp8_wgrad off)."""
    lib = L.load()
    dt = torch.float32 if fp32 else torch.bfloat16
    dev = (dy.row if dy.row is not None else dy.col).device
    if want_dx and dx is None:
        dx = torch.empty((dy.rows, w.cols), dtype=dt, device=dev)
    if want_dw and dw is None:
        dw = torch.empty((dy.cols, x.cols), dtype=dt, device=dev)
    rc = recipe.c()
    cx = ctypes.byref(x.c()) if x is not None else None
    cw = ctypes.byref(w.c()) if w is not None else None
    st = lib.fp8_linear_bwd(ctypes.byref(rc), ctypes.byref(dy.c()), cx, cw,
                            _ptr(dx) if want_dx else None, _ptr(dw) if want_dw else None,
                            int(fp32), _ptr(status), _stream(stream))
    L.check(st, "fp8_linear_bwd")
    return dx, dw


def gelu_quantize(recipe: Recipe, h: torch.Tensor, want_a_bf16=False, a_q=None, h_q=None,
                  status=None, stream=None):
    """a = gelu(h) quantised (row + column copies) and h kept as an FP8 row copy."""
    lib = L.load()
    rows, cols = h.shape
    a_q = a_q or empty_qtensor(recipe, rows, cols, "activation", True, True, device=h.device)
    h_q = h_q or empty_qtensor(recipe, rows, cols, "activation", True, False, device=h.device)
    a_bf16 = torch.empty_like(h) if want_a_bf16 else None
    rc = recipe.c()
    ca, ch = a_q.c(), h_q.c()
    st = lib.fp8_gelu_quantize(ctypes.byref(rc), _ptr(h), rows, cols, _ptr(a_bf16),
                               ctypes.byref(ca), ctypes.byref(ch), _ptr(status), _stream(stream))
    L.check(st, "fp8_gelu_quantize")
    return a_q, h_q, a_bf16


def dgelu_quantize(recipe: Recipe, da: torch.Tensor, h_q: QTensor, want_dh_bf16=False,
                   dh_q=None, status=None, stream=None):
    """dh = da * gelu'(h) with h read from its FP8 copy, quantised (row + column copies)."""
    lib = L.load()
    rows, cols = da.shape
    dh_q = dh_q or empty_qtensor(recipe, rows, cols, "grad", True, True, device=da.device)
    dh_bf16 = torch.empty_like(da) if want_dh_bf16 else None
    rc = recipe.c()
    cd = dh_q.c()
    st = lib.fp8_dgelu_quantize(ctypes.byref(rc), _ptr(da), ctypes.byref(h_q.c()), _ptr(dh_bf16),
                                ctypes.byref(cd), _ptr(status), _stream(stream))
    L.check(st, "fp8_dgelu_quantize")
    return dh_q, dh_bf16


def linear_fwd_gelu(recipe: Recipe, x: QTensor, w: QTensor, a_q=None, h_q=None, status=None,
                    stream=None):
    """fc1 with GeLU fused into the GEMM epilogue: returns (a_q, h_q), the MXFP8 row and column
    copies of a = gelu(h) and the FP8 row copy of h = x . w^T; h is never stored in bf16."""
    lib = L.load()
    dev = x.row.device
    a_q = a_q or empty_qtensor(recipe, x.rows, w.rows, "activation", True, True, device=dev)
    h_q = h_q or empty_qtensor(recipe, x.rows, w.rows, "activation", True, False, device=dev)
    rc = recipe.c()
    st = lib.fp8_linear_fwd_gelu(ctypes.byref(rc), ctypes.byref(x.c()), ctypes.byref(w.c()),
                                 ctypes.byref(a_q.c()), ctypes.byref(h_q.c()), _ptr(status),
                                 _stream(stream))
    L.check(st, "fp8_linear_fwd_gelu")
    return a_q, h_q


def linear_dgrad_dgelu(recipe: Recipe, dy: QTensor, w: QTensor, h_q: QTensor, dh_q=None,
                       status=None, stream=None):
    """dgrad of fc2 with the GeLU backward fused: dh = (dy . w) * gelu'(h), h from its FP8 row
    copy, returned as MXFP8 row and column copies."""
    lib = L.load()
    dh_q = dh_q or empty_qtensor(recipe, dy.rows, w.cols, "grad", True, True,
                                 device=dy.row.device)
    rc = recipe.c()
    st = lib.fp8_linear_dgrad_dgelu(ctypes.byref(rc), ctypes.byref(dy.c()), ctypes.byref(w.c()),
                                    ctypes.byref(h_q.c()), ctypes.byref(dh_q.c()), _ptr(status),
                                    _stream(stream))
    L.check(st, "fp8_linear_dgrad_dgelu")
    return dh_q


# The calls below run at decode rates, where Python's share counts: pointers and the stream go to
# the library as plain integers, and structures are filled by position.

_BF16, _FP32 = torch.bfloat16, torch.float32


def _raw_stream(stream):
    if stream is not None:
        return stream.cuda_stream
    return torch._C._cuda_getCurrentRawStream(torch._C._cuda_getDevice())


def _empty(shape, dtype, device, stream):
    """A buffer that the call makes itself, from the pool of the stream that it runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=device)


def _buffer(t: Optional[torch.Tensor]):
    """A workspace as the library takes it: address and bytes (none where they do not lie in one
    piece, as in an expanded tensor)."""
    return (None, 0) if t is None or not t.is_contiguous() else (t.data_ptr(), t.nbytes)


def _rows_2d(t: torch.Tensor, cols, name: str):
    """Row pitch of a bf16 [rows, cols] tensor whose rows are contiguous."""
    if t.dtype is not _BF16 or t.dim() != 2:
        raise TypeError(f"{name}: a bf16 [rows, cols] tensor")
    if t.is_contiguous():
        return cols
    pitch, step = t.stride()
    if step != 1 and cols > 1:
        raise ValueError(f"{name}: the elements of a row must be contiguous")
    return pitch


def _like(t: torch.Tensor, shape, dtype, name: str):
    if t.dtype is not dtype or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name}: a contiguous {dtype} tensor of shape {tuple(shape)}")


def _not_on_gpu():
    """The library sees addresses only, so every tensor of a call must lie on the GPU."""
    raise TypeError("CUDA tensors wanted")


def _gamma(gamma: torch.Tensor, cols: int):
    dtype = gamma.dtype
    if dtype is not _BF16 and dtype is not _FP32:
        raise TypeError("gamma: bf16 or fp32")
    if gamma.shape != (cols,) or not gamma.is_contiguous():
        raise ValueError(f"gamma: a contiguous tensor of {cols} elements")
    return 1 if dtype is _FP32 else 0


def _bad_copy(shape, size):
    raise ValueError(f"out: contiguous copies of shape {shape} with {size} bytes an element, and "
                     "their scales")


def _packed_out(out: QTensor, recipe: Recipe, rows, cols, want_row, want_col, block):
    """The wanted buffers of `out` in the library's form, checked before the kernels write them:
    as empty_qtensor makes them for an activation of `rows` padded rows under this recipe. Codes
    take one byte, the column copy without FP8 wgrad two (and no scales); block scales one byte
    for 32 codes (four for 128 come to the same). What is missing the library refuses. Returns
    the structure and whether all of it lies on the GPU."""
    row = col = row_scale = col_scale = amax = scale = scale_inv = 0
    on_gpu = True
    if want_row:
        t = out.row
        if t is None or t.shape != (rows, cols) or t.itemsize != 1 or not t.is_contiguous():
            _bad_copy((rows, cols), 1)
        row, on_gpu = t.data_ptr(), t.is_cuda
        t = out.row_scale
        if block and t is not None:
            if t.nbytes * 32 < rows * cols or not t.is_contiguous():
                _bad_copy((rows, cols), 1)
            row_scale, on_gpu = t.data_ptr(), on_gpu and t.is_cuda
    if want_col:
        t, size = out.col, 1 if recipe.fp8_wgrad else 2
        if t is None or t.shape != (cols, rows) or t.itemsize != size or not t.is_contiguous():
            _bad_copy((cols, rows), size)
        col, on_gpu = t.data_ptr(), on_gpu and t.is_cuda
        t = out.col_scale
        if block and size == 1 and t is not None:
            if t.nbytes * 32 < rows * cols or not t.is_contiguous():
                _bad_copy((cols, rows), 1)
            col_scale, on_gpu = t.data_ptr(), on_gpu and t.is_cuda
    if not block:
        a, s, i = out.amax, out.scale, out.scale_inv
        for t in (a, s, i):
            if t is not None:
                if t.nbytes < 4:
                    raise ValueError("out: fp32 amax, scale and scale_inv")
                on_gpu = on_gpu and t.is_cuda
        amax = 0 if a is None else a.data_ptr()
        scale = 0 if s is None else s.data_ptr()
        scale_inv = 0 if i is None else i.data_ptr()
    ct = L.Tensor()
    L.pack_tensor(ct, 0, row, col, row_scale, col_scale, amax, scale, scale_inv, 0, 0, 0, 0, 0)
    return ct, on_gpu


def rmsnorm_workspace_bytes(recipe: Recipe, rows, cols):
    rc = recipe.c()
    return int(L.load().fp8_rmsnorm_workspace_bytes(ctypes.byref(rc), rows, cols))


def rmsnorm_quantize(recipe: Optional[Recipe], x: torch.Tensor, gamma: torch.Tensor,
                     residual: Optional[torch.Tensor] = None, eps=1e-5, want_row=True,
                     want_col=True, want_y=False, out: Optional[QTensor] = None,
                     h: Optional[torch.Tensor] = None, rstd: Optional[torch.Tensor] = None,
                     y: Optional[torch.Tensor] = None,
                     workspace: Optional[torch.Tensor] = None, status=None, stream=None):
    """fp8_rmsnorm_quantize: h = x + residual, RMSNorm of h and the FP8 copies of its output.

    x and residual are bf16 [rows, cols], their rows may be strided; any number of rows. Returns
    (out, h, rstd, y): `out` holds the copies of the output padded with rows of zeros to the
    recipe's row quantum (out.rows), h the new residual stream (x itself without a residual),
    rstd fp32 [rows] for rmsnorm_bwd, y the bf16 output (with want_y). Buffers that are not
    given are allocated; an `out` that is given has buffers as empty_qtensor makes them for this
    recipe, and for delayed scaling is bound to its DelayedState."""
    lib = L.load()
    shape = x.shape
    if len(shape) != 2:
        raise TypeError("x: a bf16 [rows, cols] tensor")
    rows, cols = shape
    ldx = _rows_2d(x, cols, "x")
    ldr, res_ptr, h_ptr = 0, 0, None
    if residual is not None:
        if residual.shape != shape:
            raise ValueError("residual: the shape of x")
        ldr, res_ptr = _rows_2d(residual, cols, "residual"), residual.data_ptr()
        if h is None:
            h = _empty(shape, _BF16, x.device, stream)
        else:
            _like(h, shape, _BF16, "h")
        h_ptr = h.data_ptr()
    else:
        h = x
    if rstd is None:
        rstd = _empty(rows, _FP32, x.device, stream)
    else:
        _like(rstd, (rows,), _FP32, "rstd")
    if y is not None:
        _like(y, shape, _BF16, "y")
    elif want_y:
        y = _empty(shape, _BF16, x.device, stream)
    inp = L.pack_norm_input(x.data_ptr(), res_ptr, gamma.data_ptr(), ldx, ldr, rows, cols,
                            _gamma(gamma, cols), eps)
    rc = out_ref = None
    on_gpu = True
    if want_row or want_col:
        block = recipe.kind in ("mxfp8", "blockwise")
        q = 128 if block else 16
        padded = -(-rows // q) * q
        if out is None:
            with torch.cuda.stream(stream):
                out = empty_qtensor(recipe, padded, cols, "activation", want_row, want_col,
                                    device=x.device)
        ct, on_gpu = _packed_out(out, recipe, padded, cols, want_row, want_col, block)
        fields = recipe._fields()
        out_ref, rc = ctypes.byref(ct), L.pack_recipe(*fields)
    if not (on_gpu and x.is_cuda and gamma.is_cuda and h.is_cuda and rstd.is_cuda
            and (residual is None or residual.is_cuda) and (y is None or y.is_cuda)
            and (workspace is None or workspace.is_cuda)):
        _not_on_gpu()
    args = (rc, inp, want_row, want_col, h_ptr, rstd.data_ptr(),
            None if y is None else y.data_ptr(), out_ref)
    rest = (None if status is None else status.data_ptr(), _raw_stream(stream))
    st = lib.fp8_rmsnorm_quantize(*args, *_buffer(workspace), *rest)
    if st == L.FP8_ERR_WORKSPACE:            # none given, or too small: one of the call's own
        workspace = _empty(lib.fp8_rmsnorm_workspace_bytes(rc, rows, cols), torch.uint8, x.device,
                           stream)
        st = lib.fp8_rmsnorm_quantize(*args, *_buffer(workspace), *rest)
    if st:
        L.check(st, "fp8_rmsnorm_quantize")
    if out_ref is not None:
        out.rows, out.cols, out.kind, out.role = padded, cols, fields[0], L.ROLE_ACTIVATION
        out.col_bf16 = 1 - fields[5]                       # as the library sets them
    return out, h, rstd, y


def rmsnorm(x: torch.Tensor, gamma: torch.Tensor, residual: Optional[torch.Tensor] = None,
            eps=1e-5, h=None, rstd=None, y=None, stream=None):
    """The norm alone, with a bf16 output (fp8_rmsnorm_quantize without a recipe). Returns
    (y, h, rstd)."""
    _, h, rstd, y = rmsnorm_quantize(None, x, gamma, residual, eps, False, False, True, h=h,
                                     rstd=rstd, y=y, stream=stream)
    return y, h, rstd


def rmsnorm_bwd_workspace_bytes(rows, cols):
    return int(L.load().fp8_rmsnorm_bwd_workspace_bytes(rows, cols))


def rmsnorm_bwd(dy: torch.Tensor, h: torch.Tensor, rstd: torch.Tensor, gamma: torch.Tensor,
                dres: Optional[torch.Tensor] = None, want_dgamma=True,
                dh: Optional[torch.Tensor] = None, dgamma: Optional[torch.Tensor] = None,
                workspace: Optional[torch.Tensor] = None, status=None, stream=None):
    """fp8_rmsnorm_bwd: the gradient of the residual stream (of x and residual alike, `dres` the
    gradient that reaches it past the norm) and of gamma. rstd's length is the number of rows;
    dy may have more (linear_bwd's dx of the padded tensor): the rest is not read. Returns
    (dh, dgamma)."""
    lib = L.load()
    shape = h.shape
    if len(shape) != 2 or dy.dim() != 2:
        raise TypeError("dy, h: bf16 [rows, cols] tensors")
    rows, cols = shape
    _like(rstd, (rows,), _FP32, "rstd")
    if dy.shape[0] < rows or dy.shape[1] != cols:
        raise ValueError("dy, h: [rows, cols] with one row per entry of rstd")
    ld_dres, dres_ptr = 0, 0
    if dres is not None:
        if dres.shape != shape:
            raise ValueError("dres: the shape of h")
        ld_dres, dres_ptr = _rows_2d(dres, cols, "dres"), dres.data_ptr()
    inp = L.pack_norm_grad(dy.data_ptr(), h.data_ptr(), dres_ptr, gamma.data_ptr(),
                           rstd.data_ptr(), _rows_2d(dy, cols, "dy"), _rows_2d(h, cols, "h"),
                           ld_dres, rows, cols, _gamma(gamma, cols))
    if dh is None:
        dh = _empty(shape, _BF16, h.device, stream)
    else:
        _like(dh, shape, _BF16, "dh")
    if not want_dgamma:
        dgamma = None
    else:
        if dgamma is None:
            dgamma = _empty(cols, _FP32, h.device, stream)
        else:
            _like(dgamma, (cols,), _FP32, "dgamma")
    if not (dy.is_cuda and h.is_cuda and rstd.is_cuda and gamma.is_cuda and dh.is_cuda
            and (dres is None or dres.is_cuda) and (dgamma is None or dgamma.is_cuda)
            and (workspace is None or workspace.is_cuda)):
        _not_on_gpu()
    args = (inp, dh.data_ptr(), None if dgamma is None else dgamma.data_ptr())
    rest = (None if status is None else status.data_ptr(), _raw_stream(stream))
    st = lib.fp8_rmsnorm_bwd(*args, *_buffer(workspace), *rest)
    if st == L.FP8_ERR_WORKSPACE:
        workspace = _empty(lib.fp8_rmsnorm_bwd_workspace_bytes(rows, cols), torch.uint8, h.device,
                           stream)
        st = lib.fp8_rmsnorm_bwd(*args, *_buffer(workspace), *rest)
    if st:
        L.check(st, "fp8_rmsnorm_bwd")
    return dh, dgamma


_GRAD_DTYPES = {torch.bfloat16: L.GRAD_BF16, torch.float32: L.GRAD_FP32}


def _dense(t: torch.Tensor):
    """Whether the tensor's elements fill one piece of memory, in whatever order."""
    if t.is_contiguous():
        return True
    n = 1
    for stride, size in sorted((t.stride(i), t.shape[i]) for i in range(t.dim())):
        if size != 1 and stride != n:
            return False
        n *= size
    return True


def _same_order(a: torch.Tensor, b: torch.Tensor):
    """Whether two tensors of one shape hold their elements in the same order in memory."""
    return a.stride() == b.stride() or a.numel() == 0 or all(
        size == 1 or s == t for size, s, t in zip(a.shape, a.stride(), b.stride()))


class GradList:
    """The gradients of a step as fp8_grad_norm and fp8_grad_clip take them: bf16 or fp32 CUDA
    tensors of any shape, dense in memory, on one device. `outs` are the tensors that
    grad_clip writes (the gradients themselves when not given), with the gradients' shapes and
    order in memory. The list holds the tensors' addresses: it is made once for gradients that
    stay in place, and anew for new tensors. It also holds the results of grad_norm, `norm` and
    `coef`, which come from the pool of `stream` (the current one if not given): a list whose
    calls run on another stream is made for that one, or its making is waited for there."""

    def __init__(self, grads, outs=None, stream=None):
        self.grads = list(grads)
        self.outs = self.grads if outs is None else list(outs)
        if len(self.outs) != len(self.grads):
            raise ValueError("outs: one tensor per gradient")
        self.device = self.grads[0].device if self.grads else torch.device("cuda")
        self.items = (L.GradItem * max(1, len(self.grads)))()
        for i, (g, o) in enumerate(zip(self.grads, self.outs)):
            if g.device != self.device or o.device != self.device:
                raise ValueError("gradients and outs must lie on one device")
            if g.dtype not in _GRAD_DTYPES or o.dtype not in _GRAD_DTYPES:
                raise TypeError("gradients: bf16 or fp32")
            if not _dense(g) or o.shape != g.shape or (o is not g and not _same_order(o, g)):
                raise ValueError("gradients must be dense, and outs have their shapes and orders")
            self.items[i] = L.GradItem(g.data_ptr(), o.data_ptr(), g.numel(),
                                       _GRAD_DTYPES[g.dtype], _GRAD_DTYPES[o.dtype])
        self.pointer = ctypes.pointer(self.items[0])
        self.on_gpu = not self.grads or self.device.type == "cuda"
        self.norm, self.coef = _empty((2, 1), _FP32, self.device, stream).unbind(0)

    def __len__(self):
        return len(self.grads)


def grad_workspace_bytes(n):
    return int(L.load().fp8_grad_workspace_bytes(n))


def _scalar(t: torch.Tensor, name: str):
    if t.dtype is not _FP32 or t.numel() != 1:
        raise TypeError(f"{name}: one fp32 element")
    return t


def grad_norm(grads, max_norm=float("inf"), scale=1.0, norm: Optional[torch.Tensor] = None,
              coef: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None,
              stream=None):
    """fp8_grad_norm of a GradList (or a list of tensors): returns (norm, coef), fp32 tensors of
    one element on the device. They are the list's own, written anew by its next grad_norm,
    unless others are given (an allocation per call would take as long as the kernels of a
    small list)."""
    lib = L.load()
    if not isinstance(grads, GradList):
        grads = GradList(grads, stream=stream)
    n = len(grads.grads)
    norm = grads.norm if norm is None else _scalar(norm, "norm")
    coef = grads.coef if coef is None else _scalar(coef, "coef")
    if not (grads.on_gpu and norm.is_cuda and coef.is_cuda
            and (workspace is None or workspace.is_cuda)):
        _not_on_gpu()
    args = (n, grads.pointer, L.pack_clip_rule(max_norm, scale), norm.data_ptr(),
            coef.data_ptr())
    st = lib.fp8_grad_norm(*args, *_buffer(workspace), _raw_stream(stream))
    if st == L.FP8_ERR_WORKSPACE:
        workspace = _empty(lib.fp8_grad_workspace_bytes(n), torch.uint8, grads.device, stream)
        st = lib.fp8_grad_norm(*args, *_buffer(workspace), _raw_stream(stream))
    if st:
        L.check(st, "fp8_grad_norm")
    return norm, coef


def grad_clip(grads, coef: torch.Tensor, stream=None):
    """fp8_grad_clip: outs = grads * coef (coef as grad_norm returns it). Returns the outs."""
    if not isinstance(grads, GradList):
        grads = GradList(grads, stream=stream)
    _scalar(coef, "coef")
    if not (grads.on_gpu and coef.is_cuda):
        _not_on_gpu()
    st = L.load().fp8_grad_clip(len(grads.grads), grads.pointer, coef.data_ptr(),
                                _raw_stream(stream))
    if st:
        L.check(st, "fp8_grad_clip")
    return grads.outs

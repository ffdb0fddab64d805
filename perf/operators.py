"""The operators around the FP8 linear layer, as cases to measure: RMSNorm with the residual's
addition and an FP8 output, its backward pass, the global gradient norm, and clipping.

Each case is one call as a training or serving step makes it. `run` computes it either with the
framework's kernels (`own` true) or in plain torch operations in 32 bits (`own` false).

Sizes are those of a hidden-4096, ffn-16384 MLP block with 8192 tokens and their neighbours: a
single token when serving, ragged token counts, narrow and wide hidden sizes.
"""
import itertools
import math
import random

import torch

own = False

EPS = 1e-5
MAX_NORM = 1.0
BLOCK_RECIPES = ("mxfp8", "blockwise")      # 1x32 E8M0 and 1x128 fp32 block scales


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token of a serving step: the norm in front of fc1, row copy only. Latency.
        dict(name="norm decode 1 token mxfp8", op="norm", recipe="mxfp8", rows=1, cols=4096,
             residual=True, col=False),
        # The MLP block of the training benchmark: residual add, norm, both MXFP8 copies.
        dict(name="norm train mxfp8", op="norm", recipe="mxfp8", rows=8192, cols=4096,
             residual=True, col=True),
        # The same under blockwise scales at the 4096^3 linear layer's size.
        dict(name="norm train blockwise", op="norm", recipe="blockwise", rows=4096, cols=4096,
             residual=True, col=True),
        # Delayed scaling: the scale is known, the tensor's amax is written for the history.
        dict(name="norm train delayed", op="norm", recipe="delayed", rows=8192, cols=4096,
             residual=False, col=True),
        # Current per-tensor scaling of a ragged batch of tokens at an odd hidden size.
        dict(name="norm ragged tensorwise", op="norm", recipe="tensorwise", rows=1003, cols=2064,
             residual=True, col=True),
        # Backward of the training block's norm; the residual branch's gradient is added.
        dict(name="norm backward train", op="norm_bwd", rows=8192, cols=4096, dres=True),
        # A short ragged micro batch, first norm of a stack (no residual branch).
        dict(name="norm backward ragged", op="norm_bwd", rows=333, cols=1552, dres=False),
        # A wide hidden size.
        dict(name="norm backward wide", op="norm_bwd", rows=2048, cols=16384, dres=True),
        # The vectors of a small model (norm weights, biases): packed, odd sizes, fp32.
        dict(name="grad norm vectors", op="grad_norm", tensors=64, lo=33, hi=8192, sizes=1,
             dtype="fp32", packed=True),
        # The weight gradients of two MLP blocks in bf16.
        dict(name="grad norm mlp", op="grad_norm", blocks=2, hidden=4096, ffn=16384,
             dtype="bf16", packed=False),
        # Norm and clipping of a small model's gradients, bf16 in, fp32 out for the optimizer.
        dict(name="grad clip small", op="grad_clip", blocks=4, hidden=256, ffn=1024,
             dtype="bf16", out="fp32", packed=False),
        # Norm and clipping of one MLP block's fp32 main gradients.
        dict(name="grad clip mlp", op="grad_clip", blocks=1, hidden=4096, ffn=16384,
             dtype="fp32", out="fp32", packed=False),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "norm", "norm_bwd", "grad_norm", "grad_clip"])
    if op in ("norm", "norm_bwd"):
        quantum = 128 if op == "norm" else 16
        recipe = rng.choice(["mxfp8", "blockwise", "delayed", "tensorwise"])
        if op == "norm" and recipe not in BLOCK_RECIPES:
            quantum = 16
        cols = quantum * max(1, _log_int(rng, 256, 16384) // quantum)
        rows = _log_int(rng, 1, min(16384, 8192 * 4096 // cols))
        if op == "norm":
            return dict(op=op, recipe=recipe, rows=rows, cols=cols,
                        residual=rng.random() < 0.7, col=rows >= 16 and rng.random() < 0.8)
        return dict(op=op, rows=rows, cols=cols, dres=rng.random() < 0.7)
    dtype = rng.choice(["bf16", "fp32"])
    if rng.random() < 0.5:
        case = dict(op=op, tensors=_log_int(rng, 1, 60), lo=1, hi=_log_int(rng, 100, 2000000),
                    sizes=rng.randrange(1 << 20), dtype=dtype, packed=rng.random() < 0.5)
    else:
        hidden = 16 * _log_int(rng, 4, 256)
        case = dict(op=op, blocks=rng.randint(1, 2), hidden=hidden,
                    ffn=min(16384, 4 * hidden), dtype=dtype, packed=False)
        if hidden > 2048:
            case["blocks"] = 1
    if op == "grad_clip":
        case["out"] = rng.choice([dtype, "fp32"])
    return case


def _padded(case):
    q = 128 if case["recipe"] in BLOCK_RECIPES else 16
    return -(-case["rows"] // q) * q


def _sizes(case):
    """Element counts of a gradient case's tensors: each block's two weights and its norm weight, or
    vectors of log-uniform lengths."""
    if "blocks" in case:
        one = [case["ffn"] * case["hidden"], case["hidden"] * case["ffn"], case["hidden"]]
        return one * case["blocks"]
    r = random.Random(case["sizes"])
    return [_log_int(r, case["lo"], case["hi"]) for _ in range(case["tensors"])]


def work(case):
    if case["op"] == "norm":
        n, padded = case["rows"] * case["cols"], _padded(case) * case["cols"]
        copies = 2 if case["col"] else 1
        scale = {"mxfp8": 1 / 32, "blockwise": 4 / 128}.get(case["recipe"], 0)
        b = 2 * n + (4 * n if case["residual"] else 0) + copies * (1 + scale) * padded
        return {"bytes": b + 4 * case["rows"] + 2 * case["cols"], "flops": (12 + 4 * copies) * n}
    if case["op"] == "norm_bwd":
        n = case["rows"] * case["cols"]
        return {"bytes": (8 if case["dres"] else 6) * n + 4 * case["rows"] + 6 * case["cols"],
                "flops": 12 * n}
    n, size = sum(_sizes(case)), {"bf16": 2, "fp32": 4}
    b = n * size[case["dtype"]]
    if case["op"] == "grad_clip":
        b += n * size[case["out"]]
    return {"bytes": b, "flops": (3 if case["op"] == "grad_clip" else 2) * n}


# ---------------------------------------------------------------- inputs

_TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}


def _normal(gen, shape, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(torch.bfloat16)


def _activations(gen, rows, cols):
    """N(0, 1) with a few large entries, as the residual stream of a trained model has."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    big = torch.rand((rows, cols), generator=gen, device="cuda") < 1e-3
    return torch.where(big, 50 * x, x).to(torch.bfloat16)


def _views(flat, sizes, packed):
    """The tensors as views of one gradient buffer: back to back, or each on a 256-byte boundary."""
    room = [s if packed else -(-s // 128) * 128 for s in sizes]
    return [flat[e - r:e - r + s] for s, r, e in zip(sizes, room, itertools.accumulate(room))]


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s = dict(case)
    if case["op"] in ("norm", "norm_bwd"):
        rows, cols = case["rows"], case["cols"]
        s["gamma"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
        s["x"] = _activations(gen, rows, cols)
    if case["op"] == "norm":
        if case["residual"]:
            s["res"] = _activations(gen, rows, cols)
        if case["recipe"] == "delayed":             # a scale as earlier steps' amaxes leave it
            s["scale"] = torch.rand(1, generator=gen, device="cuda") * 4 + 6
            s["scale_inv"] = 1 / s["scale"]
        if own:                                     # the buffers that a step keeps
            import scaled_quantize_fp8_gb300 as F
            s["rec"] = F.Recipe(kind=case["recipe"])
            q = F.empty_qtensor(s["rec"], _padded(case), cols, "activation", True, case["col"])
            if case["recipe"] == "delayed":
                q.scale, q.scale_inv = s["scale"], s["scale_inv"]
            s["q"] = q
            s["ws"] = torch.empty(F.rmsnorm_workspace_bytes(s["rec"], rows, cols),
                                  dtype=torch.uint8, device="cuda")
            s["h"] = torch.empty_like(s["x"]) if case["residual"] else None
            s["rstd"] = torch.empty(rows, dtype=torch.float32, device="cuda")
    elif case["op"] == "norm_bwd":
        s["dy"] = _normal(gen, (rows, cols), 1e-3)
        s["rstd"] = (s["x"].float().square().mean(1) + EPS).rsqrt()
        if case["dres"]:                            # the gradient on the residual stream
            s["stream"] = _normal(gen, (rows, cols), 1e-3)
        if own:
            import scaled_quantize_fp8_gb300 as F
            s["ws"] = torch.empty(F.rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8,
                                  device="cuda")
            s["dh"] = torch.empty_like(s["x"])
            s["dgamma"] = torch.empty(cols, dtype=torch.float32, device="cuda")
    else:
        sizes, dt = _sizes(case), _TYPES[case["dtype"]]
        total = sum(sizes) if case["packed"] else sum(-(-n // 128) * 128 for n in sizes)
        s["flat"] = torch.empty(total, dtype=dt, device="cuda")
        for part in s["flat"].split(1 << 26):
            part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * 1e-3)
        s["grads"] = _views(s["flat"], sizes, case["packed"])
        s["max_norm"] = MAX_NORM * 1e-3 * math.sqrt(sum(sizes)) / 2      # about half the norm
        if case["op"] == "grad_clip":
            s["out_flat"] = torch.zeros(total, dtype=_TYPES[case["out"]], device="cuda")
            s["outs"] = _views(s["out_flat"], sizes, case["packed"])
        if own:
            import scaled_quantize_fp8_gb300 as F
            s["list"] = F.GradList(s["grads"], s.get("outs"))
            s["ws"] = torch.empty(F.grad_workspace_bytes(len(sizes)), dtype=torch.uint8,
                                  device="cuda")
    return s


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _run_own(s):
    import scaled_quantize_fp8_gb300 as F
    if s["op"] == "norm":
        q, h, rstd, _ = F.rmsnorm_quantize(s["rec"], s["x"], s["gamma"], residual=s.get("res"),
                                           eps=EPS, want_col=s["col"], out=s["q"], h=s["h"],
                                           rstd=s["rstd"], workspace=s["ws"])
        block = s["recipe"] in BLOCK_RECIPES
        e8m0 = s["recipe"] == "mxfp8"
        r = {"row": q.row.view(torch.float8_e4m3fn), "rstd": rstd}
        if s["residual"]:
            r["h"] = h
        if s["col"]:
            r["col"] = q.col.view(torch.float8_e4m3fn)
        if block:
            r["row_scale"] = q.row_scale.view(torch.float8_e8m0fnu) if e8m0 else q.row_scale
            if s["col"]:
                r["col_scale"] = q.col_scale.view(torch.float8_e8m0fnu) if e8m0 else q.col_scale
        else:
            r["amax"] = q.amax
            if s["recipe"] == "tensorwise":
                r["scale"], r["scale_inv"] = q.scale, q.scale_inv
        return r
    if s["op"] == "norm_bwd":
        dh, dgamma = F.rmsnorm_bwd(s["dy"], s["x"], s["rstd"], s["gamma"], dres=s.get("stream"),
                                   dh=s["dh"], dgamma=s["dgamma"], workspace=s["ws"])
        return {"dh": dh, "dgamma": dgamma}
    norm, coef = F.grad_norm(s["list"], max_norm=s["max_norm"], workspace=s["ws"])
    if s["op"] == "grad_norm":
        return {"norm": norm, "coef": coef}
    F.grad_clip(s["list"], coef)
    return {"norm": norm, "coef": coef, "grads": s["out_flat"]}


def _tile_scales(e):
    """[rows, blocks] -> the tensor core's order: atoms of 128 rows x 4 blocks, row r % 32 outermost."""
    rows, blocks = e.shape
    e = e.view(rows // 128, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4)
    return e.contiguous().view(-1)


def _plain_copy(recipe, y, scale):
    """Codes (and block scales) of one copy of y, blocks along its last axis."""
    rows, cols = y.shape
    if recipe == "mxfp8":
        b = y.view(rows, cols // 32, 32)
        m, e = torch.frexp(b.abs().amax(2))          # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
        e = (e - 9 + (m > 0.875).int()).clamp(-127, 127)
        e = torch.where(m == 0, -127, e)
        codes = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes.view(rows, cols), _tile_scales((e + 127).to(torch.uint8)).view(
            torch.float8_e8m0fnu)
    if recipe == "blockwise":
        b = y.view(rows, cols // 128, 128)
        amax = b.abs().amax(2)
        sc = torch.where(amax > 0, 448 / amax, torch.ones_like(amax))
        codes = (b * sc.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes.view(rows, cols), (1 / sc).t().contiguous()
    return (y * scale).clamp(-448, 448).to(torch.float8_e4m3fn), None


def _run_plain(s):
    if s["op"] == "norm":
        r = {}
        h = s["x"]
        if s["residual"]:
            h = r["h"] = (s["x"].float() + s["res"].float()).to(torch.bfloat16)
        hf = h.float()
        r["rstd"] = rstd = (hf.square().mean(1) + EPS).rsqrt()
        y = hf * rstd.unsqueeze(1) * s["gamma"].float()
        y = torch.nn.functional.pad(y, (0, 0, 0, _padded(s) - s["rows"]))
        scale = s.get("scale")
        if s["recipe"] in ("delayed", "tensorwise"):
            r["amax"] = y.abs().amax().view(1)
        if s["recipe"] == "tensorwise":
            r["scale"] = scale = torch.where(r["amax"] > 0, 448 / r["amax"],
                                             torch.ones_like(r["amax"]))
            r["scale_inv"] = 1 / scale
        r["row"], r["row_scale"] = _plain_copy(s["recipe"], y, scale)
        if s["col"]:
            r["col"], r["col_scale"] = _plain_copy(s["recipe"], y.t().contiguous(), scale)
        return {k: v for k, v in r.items() if v is not None}
    if s["op"] == "norm_bwd":
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xh = s["x"].float() * rstd
        t = dy * s["gamma"].float()
        dh = rstd * (t - xh * (t * xh).mean(1, keepdim=True))
        if s["dres"]:
            dh = dh + s["stream"].float()
        return {"dh": dh.to(torch.bfloat16), "dgamma": (dy * xh).sum(0)}
    sq = [g.float().square().sum() for g in s["grads"]]
    norm = torch.stack(sq).sum().sqrt().view(1)
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    if s["op"] == "grad_norm":
        return {"norm": norm, "coef": coef}
    [o.copy_(g.float() * coef) for o, g in zip(s["outs"], s["grads"])]
    return {"norm": norm, "coef": coef, "grads": s["out_flat"]}


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """float64 -> the nearest E4M3 value (ties to even), saturating at 448."""
    mag = v.abs().clamp(max=448.0)
    k = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))).clamp(max=8)
    step = torch.exp2(k - 3)
    return torch.copysign((torch.round(mag / step) * step).clamp(max=448.0), v)


def _exact_copy(recipe, y, scale):
    rows, cols = y.shape
    if recipe not in BLOCK_RECIPES:
        return _e4m3(y * scale), None
    n = 32 if recipe == "mxfp8" else 128
    b = y.reshape(rows, -1, n)
    top = b.abs().max(dim=2).values
    if recipe == "blockwise":
        sc = torch.where(top > 0, 448.0 / top.clamp(min=1e-300), torch.ones_like(top))
        return _e4m3(b * sc[..., None]).reshape(rows, cols), (1 / sc).t()
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -140)))
    e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)       # the smallest that holds the
    e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e)            # block, whatever log2 rounds to
    e = e.clamp(-127, 127)
    codes = _e4m3(b * torch.exp2(-e)[..., None]).reshape(rows, cols)
    r = torch.arange(rows, device=y.device)[:, None]
    k = torch.arange(cols // n, device=y.device)[None, :]
    at = ((r // 128) * (cols // 128) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    tiled = torch.empty(rows * cols // n, dtype=torch.float64, device=y.device)
    tiled[at.reshape(-1)] = torch.exp2(e).reshape(-1)
    return codes, tiled


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        r = {}
        h = s["x"].double()
        if case["residual"]:
            r["h"] = (h + s["res"].double()).to(torch.bfloat16).double()   # the stream is bf16
            h = r["h"]
        rstd = 1 / torch.sqrt((h * h).sum(1) / case["cols"] + EPS)
        y = torch.zeros((_padded(case), case["cols"]), dtype=torch.float64, device="cuda")
        y[:case["rows"]] = h * rstd[:, None] * s["gamma"].double()[None, :]
        r["rstd"], scale = rstd, None
        if case["recipe"] not in BLOCK_RECIPES:
            r["amax"] = torch.max(y.abs()).reshape(1)
            scale = s["scale"].double() if case["recipe"] == "delayed" else 448.0 / r["amax"]
            if case["recipe"] == "tensorwise":
                r["scale"], r["scale_inv"] = scale, 1 / scale
        r["row"], r["row_scale"] = _exact_copy(case["recipe"], y, scale)
        if case["col"]:
            r["col"], r["col_scale"] = _exact_copy(case["recipe"], y.t(), scale)
        return {k: v for k, v in r.items() if v is not None}
    if case["op"] == "norm_bwd":
        h, dy, g = s["x"].double(), s["dy"].double(), s["gamma"].double()
        rstd = s["rstd"].double()[:, None]
        dot = (dy * g * h).sum(1, keepdim=True)
        dh = rstd * dy * g - h * rstd ** 3 * dot / case["cols"]
        if case["dres"]:
            dh = dh + s["stream"].double()
        return {"dh": dh, "dgamma": torch.einsum("rc,rc->c", dy, h * rstd)}
    total = sum(float((p.double() ** 2).sum()) for g in s["grads"] for p in g.split(1 << 26))
    norm = math.sqrt(total)
    c = min(1.0, s["max_norm"] / (norm + 1e-6))
    r = {"norm": torch.tensor([norm], dtype=torch.float64),
         "coef": torch.tensor([c], dtype=torch.float64)}
    if case["op"] == "grad_clip":
        r["grads"] = torch.zeros(s["flat"].numel(), dtype=torch.float64, device="cuda")
        for o, g in zip(_views(r["grads"], _sizes(case), case["packed"]), s["grads"]):
            o.copy_(g.double() * c)
    return r

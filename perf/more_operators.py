"""The operators between two blocks of a model whose linear layers run in FP8, as cases to measure:
a block's output normalised, gated, scaled and added to the residual stream, whose norm is written
as the next block's FP8 copies; its backward pass; activations checkpointed in 8 bits; and the
backward pass from such checkpoints.

Each case is one call as a training or serving step makes it. `run` computes it either with the
framework's kernels (`own` true) or in plain torch operations (`own` false).

    xo = o rstd_o,  h = bf16(res + scale gate t gamma_post xo),  y = (h rstd) gamma

The stream h is held in bf16 and the norm is taken of it as stored: where the sum lies next to a
border between two bf16 values, its last bits decide, so the plain form adds it up in 64 bits.

Sizes are those of a hidden-4096, ffn-16384 MLP block with 8192 tokens and their neighbours: a
single token when serving, ragged token counts, narrow and wide hidden sizes.
"""
import math

import torch

own = False

EPS = 1e-5
BLOCK_RECIPES = ("mxfp8", "blockwise")      # scales by blocks of 32 and 128


# ---------------------------------------------------------------- cases

def listed():
    return [
        # One token of a serving step: the end of one block and the norm of the next, row copy
        # only. Latency.
        dict(name="branch decode 1 token mxfp8", op="branch", recipe="mxfp8", rows=1, cols=4096,
             post=True, gate="channel", ckpt=False, col=False),
        # The training benchmark's block: norms before and after it, a gate per channel, both
        # MXFP8 copies, and what the backward pass needs kept in 8 bits.
        dict(name="branch train mxfp8", op="branch", recipe="mxfp8", rows=8192, cols=4096,
             post=True, gate="channel", ckpt=True, col=True),
        # Blockwise (power-of-two scales) at the 4096^3 linear layer's size, no gate.
        dict(name="branch train blockwise", op="branch", recipe="blockwise", rows=4096, cols=4096,
             post=True, gate="none", ckpt=False, col=True),
        # A ragged batch at an odd hidden size with a gate per token and no norm after the block.
        dict(name="branch ragged tensorwise", op="branch", recipe="tensorwise", rows=1003,
             cols=2064, post=False, gate="token", ckpt=True, col=True),
        # Backward of the training block from its 8-bit checkpoints.
        dict(name="branch backward train", op="branch_bwd", rows=8192, cols=4096, post=True,
             gate="channel", ckpt=True, dres=True),
        # A short ragged micro batch, activations kept in bf16, a gate per token.
        dict(name="branch backward ragged", op="branch_bwd", rows=333, cols=1552, post=True,
             gate="token", ckpt=False, dres=False),
        # Backward of a norm alone whose input was checkpointed: a training micro batch of short
        # ragged sequences, and the full block.
        dict(name="norm backward ckpt ragged", op="norm_bwd", rows=1003, cols=2064, dres=True),
        dict(name="norm backward ckpt train", op="norm_bwd", rows=8192, cols=4096, dres=True),
        # The input of the block's second linear layer, left in 8 bits by the forward pass.
        dict(name="checkpoint write ffn", op="ckpt", rows=8192, cols=16384, way="write"),
        # A small activation read back.
        dict(name="checkpoint read ragged", op="ckpt", rows=333, cols=1552, way="read"),
        # The column copy that wgrad reads, made again from the checkpoint of the stream.
        dict(name="requantize train mxfp8", op="requantize", recipe="mxfp8", rows=8192, cols=4096,
             norm=True, row=False),
        # Both copies of a checkpointed linear input, per-tensor scale, ragged.
        dict(name="requantize ragged tensorwise", op="requantize", recipe="tensorwise", rows=1003,
             cols=2064, norm=False, row=True),
    ]


def _log_int(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["branch", "branch", "branch_bwd", "branch_bwd", "norm_bwd", "ckpt",
                     "requantize"])
    case = dict(op=op)
    quantum = 16
    if op in ("branch", "requantize"):
        case["recipe"] = rng.choice(["mxfp8", "blockwise", "delayed", "tensorwise"])
        quantum = 128 if case["recipe"] in BLOCK_RECIPES else 16
    case["cols"] = quantum * max(1, _log_int(rng, 256, 16384) // quantum)
    case["rows"] = _log_int(rng, 1, min(16384, 8192 * 4096 // case["cols"]))
    if op in ("branch", "branch_bwd"):
        case["post"] = rng.random() < 0.7
        case["gate"] = rng.choice(["none", "channel", "token", "both"])
        case["ckpt"] = rng.random() < 0.5
    if op == "branch":
        case["col"] = case["rows"] >= 16 and rng.random() < 0.8
    if op in ("branch_bwd", "norm_bwd"):
        case["dres"] = rng.random() < 0.7
    if op == "ckpt":
        case["way"] = rng.choice(["write", "read"])
    if op == "requantize":
        case["norm"], case["row"] = rng.random() < 0.6, rng.random() < 0.5
    return case


def _padded(case):
    q = 128 if case["recipe"] in BLOCK_RECIPES else 16
    return -(-case["rows"] // q) * q


def _scale_pitch(cols):
    return -(-cols // 128) * 4


def work(case):
    rows, cols, op = case["rows"], case["cols"], case["op"]
    n, ck = rows * cols, rows * (cols + _scale_pitch(cols))
    if op == "ckpt":
        return {"bytes": 2 * n + ck, "flops": 3 * n}
    copies, block = 0, 0
    if "recipe" in case:
        block = 1 / 32 if case["recipe"] in BLOCK_RECIPES else 0
        copies = 1 + (case["col"] if op == "branch" else case["row"])
        copies *= _padded(case) * cols * (1 + block)
    if op == "requantize":
        return {"bytes": ck + copies + (4 * rows + 2 * cols if case["norm"] else 0),
                "flops": 6 * n}
    if op == "norm_bwd":
        return {"bytes": (6 if case["dres"] else 4) * n + ck + 4 * rows + 6 * cols,
                "flops": 12 * n}
    vectors = 2 * cols * (1 + case["post"] + (case["gate"] in ("channel", "both")))
    if op == "branch":
        b = 6 * n + copies + (2 * ck if case["ckpt"] else 0) + 8 * rows
        return {"bytes": b + vectors, "flops": 30 * n}
    b = (8 if case["dres"] else 6) * n + (2 * ck if case["ckpt"] else 4 * n) + 12 * rows
    return {"bytes": b + 3 * vectors, "flops": 30 * n}


# ---------------------------------------------------------------- inputs

def _normal(gen, shape, sigma=1.0):
    return (torch.randn(shape, generator=gen, device="cuda") * sigma).to(torch.bfloat16)


def _activations(gen, rows, cols):
    """N(0, 1) with a few large entries, as the residual stream of a trained model has."""
    x = torch.randn((rows, cols), generator=gen, device="cuda")
    big = torch.rand((rows, cols), generator=gen, device="cuda") < 1e-3
    return torch.where(big, 50 * x, x).to(torch.bfloat16)


def _near_one(gen, n):
    return (1 + 0.1 * torch.randn(n, generator=gen, device="cuda")).to(torch.bfloat16)


def _rstd(x):
    return (x.double().square().mean(1) + EPS).rsqrt().float()


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed))
    s, rows, cols = dict(case), case["rows"], case["cols"]
    s["x"] = _activations(gen, rows, cols)            # the stream, or what is checkpointed
    s["gamma"] = _near_one(gen, cols)
    if case["op"] in ("branch", "branch_bwd"):
        s["branch"] = _activations(gen, rows, cols)
        s["scale"] = 0.22                             # residual scale of a deep model
        s["gamma_post"] = _near_one(gen, cols) if case["post"] else None
        s["gate_c"] = (0.5 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16) \
            if case["gate"] in ("channel", "both") else None
        s["gate_t"] = torch.rand(rows, generator=gen, device="cuda") \
            if case["gate"] in ("token", "both") else None
        s["rstd_branch"] = _rstd(s["branch"]) if case["post"] else None
    if case["op"] in ("branch_bwd", "norm_bwd"):
        s["rstd"] = _rstd(s["x"])
        s["dy"] = _normal(gen, (rows, cols), 1e-3)
        s["dres"] = _normal(gen, (rows, cols), 1e-3) if case["dres"] else None
    if case["op"] == "requantize":
        s["rstd"] = _rstd(s["x"]) if case["norm"] else None
    if case.get("recipe") == "delayed":               # a scale as earlier steps' amaxes leave it
        s["q_scale"] = torch.rand(1, generator=gen, device="cuda") * 4 + 6
        s["q_scale_inv"] = 1 / s["q_scale"]
    # what a forward pass left in 8 bits
    if case["op"] in ("norm_bwd", "requantize") or case.get("way") == "read" or \
            (case["op"] == "branch_bwd" and case["ckpt"]):
        s["x_codes"], s["x_bytes"] = _pack(s.pop("x"))
        if case["op"] == "branch_bwd":
            s["branch_codes"], s["branch_bytes"] = _pack(s.pop("branch"))
    if own:
        _buffers(s, case)
    return s


def _buffers(s, case):
    """The buffers that a step keeps for its calls."""
    import scaled_quantize_fp8_gb300 as F
    rows, cols, op = case["rows"], case["cols"], case["op"]

    def new(*shape, dtype=torch.bfloat16):
        return torch.empty(shape, dtype=dtype, device="cuda")

    def kept(name):
        if name + "_codes" in s:
            return F.Checkpoint(s[name + "_codes"].view(torch.uint8), s[name + "_bytes"])
        return s[name]

    f32 = torch.float32
    if "recipe" in case:
        s["rec"] = F.Recipe(kind=case["recipe"],
                            power_2_scales=op == "branch" and case["recipe"] == "blockwise")
        row, col = (True, case["col"]) if op == "branch" else (case["row"], True)
        s["q"] = F.empty_qtensor(s["rec"], _padded(case), cols, "activation", row, col)
        if case["recipe"] == "delayed":
            s["q"].scale, s["q"].scale_inv = s["q_scale"], s["q_scale_inv"]
        s["ws"] = new(F.rmsnorm_workspace_bytes(s["rec"], rows, cols), dtype=torch.uint8)
    if op == "branch":
        s["h"], s["rstd"] = new(rows, cols), new(rows, dtype=f32)
        s["rstd_out"] = new(rows, dtype=f32) if case["post"] else None
        s["branch_ck"] = F.empty_checkpoint(rows, cols) if case["ckpt"] else None
        s["h_ck"] = F.empty_checkpoint(rows, cols) if case["ckpt"] else None
    elif op == "branch_bwd":
        s["h"], s["o"] = kept("x"), kept("branch")
        s["dh"], s["do"], s["dgamma"] = new(rows, cols), new(rows, cols), new(cols, dtype=f32)
        s["dgamma_post"] = new(cols, dtype=f32) if case["post"] else None
        s["dgate"] = new(cols, dtype=f32) if s["gate_c"] is not None else None
        s["dtoken"] = new(rows, dtype=f32) if s["gate_t"] is not None else None
        s["ws"] = new(F.branch_rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8)
    elif op == "norm_bwd":
        s["h"], s["dh"], s["dgamma"] = kept("x"), new(rows, cols), new(cols, dtype=f32)
        s["ws"] = new(F.rmsnorm_bwd_workspace_bytes(rows, cols), dtype=torch.uint8)
    elif op == "requantize":
        s["ck"] = kept("x")
    elif case["way"] == "write":
        s["ck"] = F.empty_checkpoint(rows, cols)
    else:
        s["ck"], s["out"] = kept("x"), new(rows, cols)


# ---------------------------------------------------------------- one pass

def run(s):
    return (_run_own if own else _run_plain)(s)


def _copies_own(s, q, r):
    """The copies of a QTensor as the values that their bytes stand for."""
    e8m0 = s["recipe"] == "mxfp8" or (s["recipe"] == "blockwise" and s["op"] == "branch")
    for name in ("row", "col"):
        codes, scale = getattr(q, name), getattr(q, name + "_scale")
        if codes is not None:
            r[name] = codes.view(torch.float8_e4m3fn)
            if scale is not None:
                r[name + "_scale"] = scale.view(torch.float8_e8m0fnu) if e8m0 else scale
    if s["recipe"] not in BLOCK_RECIPES:
        r["amax"] = q.amax
        if s["recipe"] == "tensorwise":
            r["scale"], r["scale_inv"] = q.scale, q.scale_inv
    return r


def _ckpt_own(name, ck, r):
    r[name + "_codes"] = ck.codes.view(torch.float8_e4m3fn)
    r[name + "_scale"] = ck.scale.view(torch.float8_e8m0fnu)
    return r


def _run_own(s):
    import scaled_quantize_fp8_gb300 as F
    op = s["op"]
    if op == "branch":
        q, h, rstd, rstd_branch, _ = F.branch_rmsnorm_quantize(
            s["rec"], s["branch"], s["x"], s["gamma"], gamma_post=s["gamma_post"],
            gate=s["gate_c"], token_gate=s["gate_t"], scale=s["scale"], eps=EPS, want_col=s["col"],
            out=s["q"], h=s["h"], rstd=s["rstd"], rstd_branch=s["rstd_out"],
            branch_ckpt=s["branch_ck"], h_ckpt=s["h_ck"], workspace=s["ws"])
        r = _copies_own(s, q, {"h": h, "rstd": rstd})
        if s["post"]:
            r["rstd_branch"] = rstd_branch
        if s["ckpt"]:
            _ckpt_own("branch", s["branch_ck"], r)
            _ckpt_own("h", s["h_ck"], r)
        return r
    if op == "branch_bwd":
        d = F.branch_rmsnorm_bwd(
            s["dy"], s["h"], s["rstd"], s["gamma"], s["o"], rstd_branch=s["rstd_branch"],
            gamma_post=s["gamma_post"], gate=s["gate_c"], token_gate=s["gate_t"],
            scale=s["scale"], dres=s["dres"], dh=s["dh"], dbranch=s["do"], dgamma=s["dgamma"],
            dgamma_post=s["dgamma_post"], dgate=s["dgate"], dtoken_gate=s["dtoken"],
            workspace=s["ws"])
        r = {"dh": d.dh, "dbranch": d.dbranch, "dgamma": d.dgamma}
        if s["post"]:
            r["dgamma_post"] = d.dgamma_post
        if s["gate_c"] is not None:
            r["dgate"] = d.dgate
        if s["gate_t"] is not None:
            r["dtoken_gate"] = d.dtoken_gate
        return r
    if op == "norm_bwd":
        dh, dgamma = F.rmsnorm_bwd(s["dy"], s["h"], s["rstd"], s["gamma"], dres=s["dres"],
                                   dh=s["dh"], dgamma=s["dgamma"], workspace=s["ws"])
        return {"dh": dh, "dgamma": dgamma}
    if op == "requantize":
        gamma = s["gamma"] if s["norm"] else None
        q = F.checkpoint_quantize(s["rec"], s["ck"], rstd=s["rstd"], gamma=gamma,
                                  want_row=s["row"], out=s["q"], workspace=s["ws"])
        return _copies_own(s, q, {})
    if s["way"] == "write":
        return _ckpt_own("x", F.checkpoint(s["x"], out=s["ck"]), {})
    return {"x": F.checkpoint_read(s["ck"], out=s["out"])}


def _exponent(amax):
    """The smallest e with amax <= 448 2^e, at least -127."""
    m, e = torch.frexp(amax)                          # amax = m 2^e, m in [0.5, 1); 448 = 0.875 2^9
    e = (e - 9 + (m > 0.875).int()).clamp(-127, 127)
    return torch.where(m == 0, -127, e)


def _pack(x):
    """Codes and E8M0 bytes, 4 for every 128 columns of a row, of a checkpoint of x."""
    rows, cols = x.shape
    f = torch.nn.functional.pad(x.float(), (0, -cols % 128)).view(rows, -1, 32)
    e = _exponent(f.abs().amax(2))
    codes = torch.ldexp(f, -e.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return codes.view(rows, -1)[:, :cols].contiguous(), (e + 127).to(torch.uint8)


def _unpack(codes, scale):
    """The values of a checkpoint, in 32 bits (exact)."""
    rows, cols = codes.shape
    e = (scale.int() - 127).repeat_interleave(32, 1)[:, :cols]
    return torch.ldexp(codes.float(), e)


def _tile_scales(e):
    """[rows, blocks] -> the tensor core's order: atoms of 128 rows x 4 blocks, row r % 32 outermost."""
    rows, blocks = e.shape
    e = e.view(rows // 128, 4, 32, blocks // 4, 4).permute(0, 3, 2, 1, 4)
    return e.contiguous().view(-1)


def _scale_of(amax):
    """448 / amax, a rounded quotient (of two tensors: 448 / amax alone is a rounded reciprocal times
    448, which decides other ties where the values have few bits); 1 for zeros."""
    return torch.where(amax > 0, torch.full_like(amax, 448.0) / amax, torch.ones_like(amax))


def _plain_copy(s, y, scale):
    """Codes (and block scales) of one copy of y, blocks along its last axis."""
    rows, cols = y.shape
    recipe = s["recipe"]
    if recipe not in BLOCK_RECIPES:
        return (y * scale).clamp(-448, 448).to(torch.float8_e4m3fn), None
    n = 32 if recipe == "mxfp8" else 128
    b = y.view(rows, cols // n, n)
    amax = b.abs().amax(2)
    if recipe == "blockwise" and s["op"] != "branch":
        sc = _scale_of(amax)
        codes = (b * sc.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
        return codes.view(rows, cols), (1 / sc).t().contiguous()
    e = _exponent(amax)
    if recipe == "blockwise":                         # a power of two; 1 for a block of zeros
        e = torch.where(amax > 0, e, 0)
    codes = torch.ldexp(b, -e.unsqueeze(2)).clamp(-448, 448).to(torch.float8_e4m3fn)
    tiled = _tile_scales((e + 127).to(torch.uint8).repeat_interleave(n // 32, 1))
    return codes.view(rows, cols), tiled.view(torch.float8_e8m0fnu)


def _plain_copies(s, y, row, col, r):
    y = torch.nn.functional.pad(y, (0, 0, 0, _padded(s) - s["rows"]))
    scale = s.get("q_scale")
    if s["recipe"] not in BLOCK_RECIPES:
        r["amax"] = y.abs().amax().view(1)
    if s["recipe"] == "tensorwise":
        r["scale"] = scale = _scale_of(r["amax"])
        r["scale_inv"] = 1 / scale
    if row:
        r["row"], r["row_scale"] = _plain_copy(s, y, scale)
    if col:
        r["col"], r["col_scale"] = _plain_copy(s, y.t().contiguous(), scale)
    return {k: v for k, v in r.items() if v is not None}


def _factor(s, dtype):
    """scale gate gamma_post: one for every column, times the token's gate."""
    w = torch.full((1, 1), s["scale"], dtype=dtype, device="cuda")
    if s["gamma_post"] is not None:
        w = w * s["gamma_post"].to(dtype)
    if s["gate_c"] is not None:
        w = w * s["gate_c"].to(dtype)
    t = s["gate_t"].to(dtype).unsqueeze(1) if s["gate_t"] is not None else 1.0
    return w, t


def _run_plain(s):
    op = s["op"]
    if op == "branch":
        r = {}
        o = s["branch"].double()                      # next to a border of bf16, see above
        w, t = _factor(s, torch.float64)
        if s["post"]:
            rstd_o = (o.square().mean(1) + EPS).rsqrt()
            r["rstd_branch"] = rstd_o.float()
            o = o * rstd_o.unsqueeze(1)
        r["h"] = h = (s["x"].double() + w * t * o).to(torch.bfloat16)
        hf = h.float()
        r["rstd"] = rstd = (hf.square().mean(1) + EPS).rsqrt()
        if s["ckpt"]:
            for name, v in (("branch", s["branch"]), ("h", h)):
                r[name + "_codes"], e = _pack(v)
                r[name + "_scale"] = e.view(torch.float8_e8m0fnu)
        y = hf * rstd.unsqueeze(1) * s["gamma"].float()
        return _plain_copies(s, y, True, s["col"], r)
    if op in ("branch_bwd", "norm_bwd"):
        h = _unpack(s["x_codes"], s["x_bytes"]) if "x_codes" in s else s["x"].float()
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xh = h * rstd
        a = dy * s["gamma"].float()
        dh = rstd * (a - xh * (a * xh).mean(1, keepdim=True))
        if s["dres"] is not None:
            dh = dh + s["dres"].float()
        r = {"dh": dh.to(torch.bfloat16), "dgamma": (dy * xh).sum(0)}
        if op == "norm_bwd":
            return r
        o = _unpack(s["branch_codes"], s["branch_bytes"]) if "branch_codes" in s \
            else s["branch"].float()
        w, t = _factor(s, torch.float32)
        u = dh * w
        if s["post"]:
            ro = s["rstd_branch"].unsqueeze(1)
            xo = o * ro
            do = ro * t * (u - xo * (u * xo).mean(1, keepdim=True))
        else:
            xo, do = o, u * t
        r["dbranch"] = do.to(torch.bfloat16)
        sums = (dh * t * xo).sum(0) * s["scale"]
        if s["post"]:
            r["dgamma_post"] = sums if s["gate_c"] is None else sums * s["gate_c"].float()
        if s["gate_c"] is not None:
            r["dgate"] = sums * s["gamma_post"].float() if s["post"] else sums
        if s["gate_t"] is not None:
            r["dtoken_gate"] = (u * xo).sum(1)
        return r
    if op == "requantize":
        y = _unpack(s["x_codes"], s["x_bytes"])
        if s["norm"]:
            y = y * s["rstd"].unsqueeze(1) * s["gamma"].float()
        return _plain_copies(s, y, s["row"], True, {})
    if s["way"] == "write":
        codes, e = _pack(s["x"])
        return {"x_codes": codes, "x_scale": e.view(torch.float8_e8m0fnu)}
    return {"x": _unpack(s["x_codes"], s["x_bytes"]).to(torch.bfloat16)}


# ---------------------------------------------------------------- 64 bits

def _e4m3(v):
    """float64 -> the nearest E4M3 value (ties to even), saturating at 448."""
    mag = v.abs().clamp(max=448.0)
    k = torch.floor(torch.log2(mag.clamp(min=2.0 ** -6))).clamp(max=8)
    step = torch.exp2(k - 3)
    return torch.copysign((torch.round(mag / step) * step).clamp(max=448.0), v)


def _pow2(top):
    """The least power of two p (2^-127 at least) with top <= 448 p."""
    e = torch.ceil(torch.log2((top / 448.0).clamp(min=2.0 ** -140)))
    e = torch.where(torch.exp2(e - 1) * 448.0 >= top, e - 1, e)       # the smallest that holds the
    e = torch.where(torch.exp2(e) * 448.0 < top, e + 1, e)            # block, whatever log2 rounds to
    return torch.exp2(e.clamp(-127, 127))


def _exact_ckpt(v):
    """Codes and scales [rows, 4 for every 128 columns] of a checkpoint."""
    rows, cols = v.shape
    wide = torch.zeros((rows, _scale_pitch(cols) * 32), dtype=torch.float64, device=v.device)
    wide[:, :cols] = v
    b = wide.reshape(rows, -1, 32)
    p = _pow2(b.abs().max(dim=2).values)
    return _e4m3(b / p[..., None]).reshape(rows, -1)[:, :cols], p


def _exact_read(codes, scale):
    p = torch.exp2(scale.double() - 127)
    columns = torch.arange(codes.shape[1], device=codes.device) // 32
    return codes.double() * p[:, columns]


def _exact_copy(case, y, scale):
    rows, cols = y.shape
    if case["recipe"] not in BLOCK_RECIPES:
        return _e4m3(y * scale), None
    n = 32 if case["recipe"] == "mxfp8" else 128
    b = y.reshape(rows, -1, n)
    top = b.abs().max(dim=2).values
    if case["recipe"] == "blockwise" and case["op"] != "branch":
        sc = torch.where(top > 0, 448.0 / top.clamp(min=1e-300), torch.ones_like(top))
        return _e4m3(b * sc[..., None]).reshape(rows, cols), (1 / sc).t()
    p = _pow2(top)
    if case["recipe"] == "blockwise":
        p = torch.where(top > 0, p, torch.ones_like(p))
    codes = _e4m3(b / p[..., None]).reshape(rows, cols)
    r = torch.arange(rows, device=y.device)[:, None]
    k = torch.arange(cols // 32, device=y.device)[None, :]
    at = ((r // 128) * (cols // 128) + k // 4) * 512 + (r % 32) * 16 + (r % 128) // 32 * 4 + k % 4
    tiled = torch.empty(rows * cols // 32, dtype=torch.float64, device=y.device)
    tiled[at.reshape(-1)] = p[:, :, None].expand(-1, -1, n // 32).reshape(-1)
    return codes, tiled


def _exact_copies(case, s, y, row, col, r):
    full = torch.zeros((_padded(case), case["cols"]), dtype=torch.float64, device="cuda")
    full[:case["rows"]] = y
    scale = None
    if case["recipe"] not in BLOCK_RECIPES:
        r["amax"] = torch.max(full.abs()).reshape(1)
        scale = s["q_scale"].double() if case["recipe"] == "delayed" else 448.0 / r["amax"]
        if case["recipe"] == "tensorwise":
            r["scale"], r["scale_inv"] = scale, 1 / scale
    if row:
        r["row"], r["row_scale"] = _exact_copy(case, full, scale)
    if col:
        r["col"], r["col_scale"] = _exact_copy(case, full.t(), scale)
    return {k: v for k, v in r.items() if v is not None}


def exact(case, seed):
    s, op = prepare(case, seed), case["op"]
    if op == "ckpt":
        if case["way"] == "read":
            return {"x": _exact_read(s["x_codes"], s["x_bytes"])}
        codes, p = _exact_ckpt(s["x"].double())
        return {"x_codes": codes, "x_scale": p}
    gamma = s["gamma"].double()[None, :]
    if op == "requantize":
        y = _exact_read(s["x_codes"], s["x_bytes"])
        if case["norm"]:
            y = y * s["rstd"].double()[:, None] * gamma
        return _exact_copies(case, s, y, case["row"], True, {})
    cols = case["cols"]
    if op == "norm_bwd":
        h = _exact_read(s["x_codes"], s["x_bytes"])
    else:
        one = torch.ones((), dtype=torch.float64, device="cuda")
        after = s["gamma_post"].double()[None, :] if case["post"] else one
        gate = s["gate_c"].double()[None, :] if s["gate_c"] is not None else one
        token = s["gate_t"].double()[:, None] if s["gate_t"] is not None else one
    if op == "branch":
        r = {}
        n = o = s["branch"].double()
        if case["post"]:
            r["rstd_branch"] = 1 / torch.sqrt((o * o).sum(1) / cols + EPS)
            n = o * r["rstd_branch"][:, None] * after
        stream = s["x"].double() + s["scale"] * (token * (gate * n))
        r["h"] = h = stream.to(torch.bfloat16).double()                # the stream is bf16
        r["rstd"] = 1 / torch.sqrt((h * h).sum(1) / cols + EPS)
        if case["ckpt"]:
            r["branch_codes"], r["branch_scale"] = _exact_ckpt(o)
            r["h_codes"], r["h_scale"] = _exact_ckpt(h)
        return _exact_copies(case, s, h * r["rstd"][:, None] * gamma, True, case["col"], r)
    if op == "branch_bwd":
        h = _exact_read(s["x_codes"], s["x_bytes"]) if case["ckpt"] else s["x"].double()
    dy, rstd = s["dy"].double(), s["rstd"].double()[:, None]
    dot = (dy * gamma * h).sum(1, keepdim=True)
    dh = rstd * dy * gamma - h * rstd ** 3 * dot / cols
    if case["dres"]:
        dh = dh + s["dres"].double()
    r = {"dh": dh, "dgamma": torch.einsum("rc,rc->c", dy, h * rstd)}
    if op == "norm_bwd":
        return r
    o = _exact_read(s["branch_codes"], s["branch_bytes"]) if case["ckpt"] else s["branch"].double()
    dn = s["scale"] * dh * gate * token               # the gradient of the normalised branch
    if case["post"]:
        ro = s["rstd_branch"].double()[:, None]
        dot = (dn * after * o).sum(1, keepdim=True)
        r["dbranch"] = ro * dn * after - o * ro ** 3 * dot / cols
        n = o * ro * after
        r["dgamma_post"] = torch.einsum("rc,rc->c", dn, o * ro)
    else:
        r["dbranch"], n = dn, o
    if s["gate_c"] is not None:
        r["dgate"] = s["scale"] * (dh * token * n).sum(0)
    if s["gate_t"] is not None:
        r["dtoken_gate"] = s["scale"] * (dh * gate * n).sum(1)
    return r

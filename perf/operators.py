"""Cases of the norm and 8-bit checkpoint operators, in plain form and as the library's calls.

The operators are those a rank's backward pass runs to produce the gradients that the reduction takes:

* layer norm, forward and backward, with the reduction of the weight's and the bias's gradient;
* 8-bit activation checkpoints: packing and unpacking, the norm recomputed from one, the norm's backward
  pass from one, and a linear layer's weight and bias gradient from one.

A checkpoint holds a row in blocks of 32 columns. A block has one exponent byte (127 + e) and 32 codes of
one byte; the value of a code is its e4m3 or integer value times 2^e, where e is the smallest integer (not
below -124) with the block's largest magnitude at most 448 * 2^e (e4m3) or 127 * 2^e (int8). Codes are
rounded to nearest, ties to even. The buffer is the codes, rows of P = 32 * ceil(cols / 32) bytes, then the
exponents, rows of P / 32 bytes.

A case has a "kind": "norm" (forward), "recompute" (forward that saves the checkpoint of its input, and the
forward again from that checkpoint, as the backward pass does it), "norm_bwd" (backward pass, from the input
or from its checkpoint), "ckpt" (packed and unpacked), "wgrad" (a linear layer's gradients from a
checkpoint) and "block" (norm forward with its output's checkpoint, then the weight gradient of the linear
layer behind it).
"""
import math

import torch

own = False

EPS = 1e-5


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one token through one norm: what a call costs when there is nothing to stream
        {"name": "norm 1x4096 bf16", "kind": "norm", "rows": 1, "cols": 4096, "x": "bf16", "y": "bf16",
         "params": "bf16", "pad": 0},
        # an odd width, rows of a wider buffer, a residual stream in fp32 with bf16 activations
        {"name": "norm 4097x1023 fp32-bf16", "kind": "norm", "rows": 4097, "cols": 1023, "x": "fp32", "y": "bf16",
         "params": "fp32", "pad": 9},
        # a micro-batch of 16k tokens at the transformer's width: saved in the forward pass, recomputed in
        # the backward pass
        {"name": "recompute 16384x4096 e4m3", "kind": "recompute", "rows": 16384, "cols": 4096, "x": "bf16",
         "y": "bf16", "params": "bf16", "format": "e4m3"},
        # the backward pass of a few rows: latency again, two launches
        {"name": "norm_bwd 16x768 fp32", "kind": "norm_bwd", "rows": 16, "cols": 768, "x": "fp32", "dy": "fp32",
         "params": "fp32", "grads": "fp32", "accumulate": False, "add_dx": False},
        # an ordinary one on the residual stream: dx added to the gradient that passed by, a later micro-step
        # whose weight gradients add into the flat gradient
        {"name": "norm_bwd 16384x4096 bf16", "kind": "norm_bwd", "rows": 16384, "cols": 4096, "x": "bf16",
         "dy": "bf16", "params": "bf16", "grads": "bf16", "accumulate": True, "add_dx": True},
        # the FFN's width, from the checkpoint in 8 bits
        {"name": "norm_bwd 24576x11008 int8", "kind": "norm_bwd", "rows": 24576, "cols": 11008, "x": "int8",
         "dy": "bf16", "params": "bf16", "grads": "fp32", "accumulate": False, "add_dx": False},
        # a small tensor whose last block is short
        {"name": "ckpt 333x1000 fp32 int8", "kind": "ckpt", "rows": 333, "cols": 1000, "x": "fp32", "format": "int8"},
        # a micro-batch of 64k tokens
        {"name": "ckpt 65536x4096 bf16 e4m3", "kind": "ckpt", "rows": 65536, "cols": 4096, "x": "bf16",
         "format": "e4m3"},
        # odd sizes everywhere, output gradients in fp32, with the bias's gradient
        {"name": "wgrad 1001x777x1000 fp32", "kind": "wgrad", "rows": 1001, "out": 777, "in": 1000, "dy": "fp32",
         "format": "int8", "grads": "fp32", "bias": True, "accumulate": False},
        # few tokens for a square projection: the sum over tokens is short
        {"name": "wgrad 2048x4096x4096 int8", "kind": "wgrad", "rows": 2048, "out": 4096, "in": 4096, "dy": "bf16",
         "format": "int8", "grads": "bf16", "bias": False, "accumulate": False},
        # the FFN's up projection over 16k tokens, a later micro-step: the largest
        {"name": "wgrad 16384x11008x4096 e4m3", "kind": "wgrad", "rows": 16384, "out": 11008, "in": 4096,
         "dy": "bf16", "format": "e4m3", "grads": "fp32", "bias": True, "accumulate": True},
        # a norm and the projection behind it, as a layer's step has them; few outputs, many tokens
        {"name": "block 8192x4096x1024 e4m3", "kind": "block", "rows": 8192, "cols": 4096, "out": 1024, "x": "bf16",
         "y": "bf16", "params": "bf16", "format": "e4m3", "dy": "bf16", "grads": "bf16"},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
        v = max(lo, min(hi, v))
        return v if rng.random() < 0.4 else max(lo, v // 16 * 16)  # odd sizes among them

    real, eight = ("bf16", "fp32"), ("e4m3", "int8")
    kind = rng.choice(("norm", "recompute", "norm_bwd", "norm_bwd", "ckpt", "wgrad", "wgrad", "block"))
    case = {"kind": kind}
    if kind == "wgrad":
        out, inn = size(16, 11008), size(16, 11008)
        rows = size(1, min(32768, max(1, (1 << 39) // (out * inn))))
        return case | {"rows": rows, "out": out, "in": inn, "dy": rng.choice(("bf16", "bf16", "fp32")),
                       "format": rng.choice(eight), "grads": rng.choice(real), "bias": rng.random() < 0.5,
                       "accumulate": rng.random() < 0.5}
    cols = size(64, 16384)
    rows = size(1, max(1, min(65536, (1 << 27) // cols)))
    case |= {"rows": rows, "cols": cols}
    if kind == "norm":
        return case | {"x": rng.choice(real), "y": rng.choice(real), "params": rng.choice(real),
                       "pad": rng.choice((0, 0, 8, 5))}
    if kind == "recompute":
        return case | {"x": rng.choice(real), "y": rng.choice(real), "params": rng.choice(real),
                       "format": rng.choice(eight)}
    if kind == "norm_bwd":
        return case | {"x": rng.choice(real + eight), "dy": rng.choice(real), "params": rng.choice(real),
                       "grads": rng.choice(real), "accumulate": rng.random() < 0.5, "add_dx": rng.random() < 0.5}
    if kind == "ckpt":
        return case | {"x": rng.choice(real), "format": rng.choice(eight)}
    return case | {"out": size(16, 4096), "x": rng.choice(real), "y": "bf16", "params": rng.choice(real),
                   "format": rng.choice(eight), "dy": "bf16", "grads": "bf16"}


# ----------------------------------------------------------------- inputs
REAL = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2.0, "fp32": 4.0, "e4m3": 33 / 32, "int8": 33 / 32}


def _activations(g, rows, cols):
    """A residual stream's values: channels of unequal size, a few of them far larger, an offset."""
    dev = "cuda"
    chan = torch.exp(0.4 * torch.randn(cols, generator=g, device=dev))
    chan = torch.where(torch.rand(cols, generator=g, device=dev) < 0.01, chan * 12, chan)
    off = 0.2 + 0.3 * torch.randn(cols, generator=g, device=dev)
    return torch.randn(rows, cols, generator=g, device=dev).mul_(chan).add_(off)


def _gradients(g, rows, cols):
    """Gradients of activations: small, rows of unequal size."""
    row = 1e-3 * torch.exp(0.7 * torch.randn(rows, 1, generator=g, device="cuda"))
    return torch.randn(rows, cols, generator=g, device="cuda").mul_(row)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind, rows = case["kind"], case["rows"]
    s = {"case": case}

    def empty(shape, kind_):
        return torch.empty(shape, dtype=REAL[kind_], device="cuda")

    if kind == "wgrad":
        s["dy"] = _gradients(g, rows, case["out"]).to(REAL[case["dy"]])
        s["ckpt"] = _to_buffer(*_encode(_activations(g, rows, case["in"]).bfloat16().float(), case["format"]), case["format"])
        s["dw"] = (1e-3 * torch.randn(case["out"], case["in"], generator=g, device="cuda")).to(REAL[case["grads"]])
        s["db"] = (1e-3 * torch.randn(case["out"], generator=g, device="cuda")).to(REAL[case["grads"]])
        return s
    cols = case["cols"]
    x = _activations(g, rows, cols)
    if case["x"] in REAL:
        x = x.to(REAL[case["x"]])
        if case.get("pad"):  # rows of a wider buffer
            wide = torch.zeros(rows, cols + case["pad"], dtype=x.dtype, device="cuda")
            wide[:, :cols] = x
            x = wide[:, :cols]
        s["x"] = x
    if kind == "ckpt":
        s["back"] = torch.empty(rows, cols, dtype=x.dtype, device="cuda")
        s["ckpt"] = torch.empty(_bytes(rows, cols), dtype=torch.uint8, device="cuda")
        return s
    s["w"] = (1 + 0.2 * torch.randn(cols, generator=g, device="cuda")).to(REAL[case["params"]])
    s["b"] = (0.1 * torch.randn(cols, generator=g, device="cuda")).to(REAL[case["params"]])
    if kind == "norm_bwd":
        # the statistics that the forward pass kept
        x32 = x.float()
        s["mean"] = x32.double().mean(1).float()
        s["rstd"] = (x32.double().var(1, unbiased=False) + EPS).rsqrt().float()
        if case["x"] not in REAL:
            s["ckpt"] = _to_buffer(*_encode(x.bfloat16().float(), case["x"]), case["x"])
        s["dy"] = _gradients(g, rows, cols).to(REAL[case["dy"]])
        s["dx"] = _gradients(g, rows, cols).to(REAL[case["dy"]])
        s["dw"] = (1e-3 * torch.randn(cols, generator=g, device="cuda")).to(REAL[case["grads"]])
        s["db"] = (1e-3 * torch.randn(cols, generator=g, device="cuda")).to(REAL[case["grads"]])
        return s
    s["y"] = empty((rows, cols), case["y"])
    s["mean"], s["rstd"] = empty((rows,), "fp32"), empty((rows,), "fp32")
    if kind in ("recompute", "block"):
        s["ckpt"] = torch.empty(_bytes(rows, cols), dtype=torch.uint8, device="cuda")
    if kind == "recompute":
        s["again"] = empty((rows, cols), case["y"])
        s["mean2"], s["rstd2"] = empty((rows,), "fp32"), empty((rows,), "fp32")
    if kind == "block":
        s["dy"] = _gradients(g, rows, case["out"]).to(REAL[case["dy"]])
        s["dw"] = empty((case["out"], cols), case["grads"])
    return s


# ------------------------------------------------------------- plain forms
def _pitch(cols):
    return 32 * -(-cols // 32)


def _bytes(rows, cols):
    return rows * (_pitch(cols) + _pitch(cols) // 32)


def _two_to(e):
    return torch.ldexp(torch.ones((), dtype=torch.float32, device=e.device), e)


def _encode(x, fmt):
    """(scaled and rounded values [rows, P/32, 32] in fp32, exponents [rows, P/32]) of fp32 x."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, _pitch(cols) - cols)).view(rows, -1, 32)
    amax = x.abs().amax(-1)
    m, k = torch.frexp(amax)
    e = k - 9 + (m > 0.875).int() if fmt == "e4m3" else k - 7 + (m > 127 / 128).int()
    e = torch.where(amax > 0, e, -124).clamp_min(-124)
    v = x * _two_to(-e).unsqueeze(-1)
    if fmt == "int8":
        return torch.round(v), e
    _, k = torch.frexp(v)
    step = _two_to(k.sub_(1).clamp_(min=-6).sub_(3))  # e4m3: three bits behind the leading one, down to 2^-9
    return torch.round(v / step) * step, e


def _decode(q, e, cols):
    return (q * _two_to(e).unsqueeze(-1)).view(q.shape[0], -1)[:, :cols]


def _to_buffer(q, e, fmt):
    rows = q.shape[0]
    codes = (q.to(torch.float8_e4m3fn) if fmt == "e4m3" else q.to(torch.int8)).view(torch.uint8)
    return torch.cat([codes.reshape(-1), (e + 127).to(torch.uint8).reshape(-1)])


def _from_buffer(buf, rows, cols, fmt):
    """fp32 values of a checkpoint."""
    p = _pitch(cols)
    q = buf[: rows * p].view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).view(rows, p // 32, 32).float()
    return _decode(q, buf[rows * p:].view(rows, p // 32).int() - 127, cols)


def _norm(x, w, b):
    mean = x.mean(1)
    d = x - mean.unsqueeze(1)
    rstd = 1 / torch.sqrt((d * d).mean(1) + EPS)
    return d * rstd.unsqueeze(1) * w.float() + b.float(), mean, rstd


def _norm_bwd(dy, x, mean, rstd, w):
    xh = (x - mean.unsqueeze(1)) * rstd.unsqueeze(1)
    dw, db = (dy * xh).sum(0), dy.sum(0)
    g = dy * w.float()
    c1, c2 = (g * xh).mean(1, keepdim=True), g.mean(1, keepdim=True)
    return (g - c2 - xh * c1) * rstd.unsqueeze(1), dw, db


def _plain(s):
    case = s["case"]
    kind, rows = case["kind"], case["rows"]
    if kind == "norm":
        y, mean, rstd = _norm(s["x"].float(), s["w"], s["b"])
        return {"y": y.to(REAL[case["y"]]), "mean": mean, "rstd": rstd}
    if kind == "recompute":
        x = s["x"].float()
        y, mean, rstd = _norm(x, s["w"], s["b"])
        again, mean2, rstd2 = _norm(_decode(*_encode(x, case["format"]), case["cols"]), s["w"], s["b"])
        dt = REAL[case["y"]]
        return {"y": y.to(dt), "mean": mean, "rstd": rstd, "again": again.to(dt), "mean2": mean2, "rstd2": rstd2}
    if kind == "norm_bwd":
        x = s["x"].float() if case["x"] in REAL else _from_buffer(s["ckpt"], rows, case["cols"], case["x"])
        dx, dw, db = _norm_bwd(s["dy"].float(), x, s["mean"], s["rstd"], s["w"])
        if case["add_dx"]:
            dx = dx + s["dx"].float()
        if case["accumulate"]:
            dw, db = dw + s["dw"].float(), db + s["db"].float()
        for n, v in (("dx", dx), ("dw", dw), ("db", db)):
            s[n].copy_(v)
        return {n: s[n] for n in ("dx", "dw", "db")}
    if kind == "ckpt":
        return _decode(*_encode(s["x"].float(), case["format"]), case["cols"]).to(s["x"].dtype)
    if kind == "wgrad":
        x = _from_buffer(s["ckpt"], rows, case["in"], case["format"])
        dy = s["dy"].float()
        dw, db = dy.t() @ x, dy.sum(0)
        if case["accumulate"]:
            dw, db = dw + s["dw"].float(), db + s["db"].float()
        s["dw"].copy_(dw)
        if not case["bias"]:
            return {"dw": s["dw"]}
        s["db"].copy_(db)
        return {"dw": s["dw"], "db": s["db"]}
    y, mean, rstd = _norm(s["x"].float(), s["w"], s["b"])
    y = y.to(REAL[case["y"]])
    dw = s["dy"].float().t() @ _decode(*_encode(y.float(), case["format"]), case["cols"])
    return {"y": y, "mean": mean, "rstd": rstd, "dw": dw.to(REAL[case["grads"]])}


# ------------------------------------------------------ the library's calls
def _workspace(s, nbytes):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in s or s["ws"].numel() < nbytes:
        s["ws"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _calls(s):
    import gradient_sync_zr_amd as zr

    case = s["case"]
    kind, rows = case["kind"], case["rows"]
    fmt = {"e4m3": zr.ZR_CKPT_E4M3, "int8": zr.ZR_CKPT_INT8}
    if kind == "wgrad":
        out, inn = case["out"], case["in"]
        ws = _workspace(s, zr.zr_ckpt_wgrad_workspace_bytes(rows, out, inn))
        zr.zr_ckpt_wgrad(s["dy"], s["ckpt"], rows, out, inn, s["dw"], dbias=s["db"] if case["bias"] else None,
                         format=fmt[case["format"]], accumulate=case["accumulate"], workspace=ws)
        return {"dw": s["dw"], "db": s["db"]} if case["bias"] else {"dw": s["dw"]}
    cols = case["cols"]
    if kind == "norm":
        zr.zr_layernorm_fwd(s["x"], rows, cols, s["y"], s["w"], s["b"], eps=EPS, mean=s["mean"], rstd=s["rstd"])
        return {n: s[n] for n in ("y", "mean", "rstd")}
    if kind == "recompute":
        f = fmt[case["format"]]
        zr.zr_layernorm_fwd(s["x"], rows, cols, s["y"], s["w"], s["b"], eps=EPS, mean=s["mean"], rstd=s["rstd"],
                            ckpt_x=s["ckpt"], ckpt_format=f)
        zr.zr_layernorm_fwd(s["ckpt"], rows, cols, s["again"], s["w"], s["b"], eps=EPS, mean=s["mean2"],
                            rstd=s["rstd2"], x_dtype=f)
        return {n: s[n] for n in ("y", "mean", "rstd", "again", "mean2", "rstd2")}
    if kind == "norm_bwd":
        ws = _workspace(s, zr.zr_layernorm_workspace_bytes(rows, cols))
        real = case["x"] in REAL
        zr.zr_layernorm_bwd(s["dy"], s["x"] if real else s["ckpt"], rows, cols, s["mean"], s["rstd"], s["w"],
                            dx=s["dx"], dweight=s["dw"], dbias=s["db"], x_dtype=None if real else fmt[case["x"]],
                            accumulate=case["accumulate"], add_dx=case["add_dx"], workspace=ws)
        return {n: s[n] for n in ("dx", "dw", "db")}
    if kind == "ckpt":
        zr.zr_ckpt_pack(s["x"], rows, cols, s["ckpt"], format=fmt[case["format"]])
        zr.zr_ckpt_unpack(s["ckpt"], rows, cols, s["back"], format=fmt[case["format"]])
        return s["back"]
    f = fmt[case["format"]]
    zr.zr_layernorm_fwd(s["x"], rows, cols, s["y"], s["w"], s["b"], eps=EPS, mean=s["mean"], rstd=s["rstd"],
                        ckpt_y=s["ckpt"], ckpt_format=f)
    ws = _workspace(s, zr.zr_ckpt_wgrad_workspace_bytes(rows, case["out"], cols))
    zr.zr_ckpt_wgrad(s["dy"], s["ckpt"], rows, case["out"], cols, s["dw"], format=f, workspace=ws)
    return {n: s[n] for n in ("y", "mean", "rstd", "dw")}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    kind, rows = case["kind"], case["rows"]
    if kind == "wgrad":
        out, inn = case["out"], case["in"]
        grads = SIZE[case["grads"]] * (out * inn + (out if case["bias"] else 0)) * (2 if case["accumulate"] else 1)
        return {"bytes": rows * out * SIZE[case["dy"]] + rows * _pitch(inn) * SIZE[case["format"]] + grads,
                "flops": 2.0 * rows * out * inn + (rows * out if case["bias"] else 0)}
    cols = case["cols"]
    n = rows * cols
    if kind == "ckpt":
        return {"bytes": 2 * (n * SIZE[case["x"]] + rows * _pitch(cols) * SIZE[case["format"]]), "flops": 4.0 * n}
    params = 2 * cols * SIZE[case["params"]]
    stats = 8 * rows
    if kind == "norm_bwd":
        x = (n if case["x"] in REAL else rows * _pitch(cols)) * SIZE[case["x"]]
        dx = n * SIZE[case["dy"]] * (2 if case["add_dx"] else 1)
        grads = 2 * cols * SIZE[case["grads"]] * (2 if case["accumulate"] else 1)
        return {"bytes": x + n * SIZE[case["dy"]] + dx + params / 2 + stats + grads, "flops": 14.0 * n}
    fwd = n * (SIZE[case["x"]] + SIZE[case["y"]]) + params + stats
    if kind == "norm":
        return {"bytes": fwd, "flops": 8.0 * n}
    saved = rows * _pitch(cols) * SIZE[case["format"]]
    if kind == "recompute":
        return {"bytes": fwd + 2 * saved + n * SIZE[case["y"]] + params + stats, "flops": 20.0 * n}
    out = case["out"]
    return {"bytes": fwd + 2 * saved + rows * out * SIZE[case["dy"]] + out * cols * SIZE[case["grads"]],
            "flops": 12.0 * n + 2.0 * rows * out * cols}


# ---------------------------------------------------------------- 64 bits
def _held(x, fmt):
    """What a checkpoint keeps of fp64 x, from the format's definition: the nearest value of its table."""
    rows, cols = x.shape
    p = _pitch(cols)
    blocks = torch.zeros(rows, p, dtype=torch.float64, device=x.device)
    blocks[:, :cols] = x
    blocks = blocks.view(-1, 32)
    top = 448.0 if fmt == "e4m3" else 127.0
    amax = blocks.abs().max(1, keepdim=True).values
    scale = torch.exp2(torch.ceil(torch.log2(amax / top)).clamp(min=-124.0))
    if fmt == "int8":
        table = torch.arange(128, dtype=torch.float64, device=x.device)
    else:  # code c: exponent c >> 3, fraction c & 7; 0x7F is not a number
        c = torch.arange(127, dtype=torch.float64, device=x.device)
        ex, fr = torch.floor(c / 8), c % 8
        table = torch.where(ex > 0, (1 + fr / 8) * torch.exp2(ex - 7), fr * 2.0 ** -9)
    middle = (table[1:] + table[:-1]) / 2
    for lo in range(0, blocks.shape[0], 1 << 20):
        part = blocks[lo: lo + (1 << 20)]
        a = part.abs() / scale[lo: lo + (1 << 20)]
        at = torch.searchsorted(middle, a)
        tie = a == middle[at.clamp(max=middle.numel() - 1)]
        at = at + (tie & (at % 2 == 1)).long()  # a tie goes to the even code
        part.copy_(torch.sign(part) * table[at] * scale[lo: lo + (1 << 20)])
    return blocks.view(rows, p)[:, :cols]


def _kept(buf, rows, cols, fmt):
    """The fp64 values of a checkpoint buffer, code by code."""
    p = _pitch(cols)
    code = torch.arange(256, device=buf.device)
    if fmt == "int8":
        value = torch.where(code < 128, code, code - 256).double()
    else:
        ex, fr = (code >> 3) & 15, (code & 7).double()
        value = torch.where(ex > 0, (1 + fr / 8) * torch.exp2(ex.double() - 7), fr * 2.0 ** -9)
        value = torch.where(code >= 128, -value, value)
    v = value[buf[: rows * p].long()].view(rows, p // 32, 32)
    return (v * torch.exp2(buf[rows * p:].double() - 127).view(rows, -1, 1)).view(rows, p)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    kind, rows = case["kind"], case["rows"]
    d = {n: v.double() for n, v in s.items() if isinstance(v, torch.Tensor) and v.dtype != torch.uint8}

    def forward(x):
        var, mean = torch.var_mean(x, 1, unbiased=False, keepdim=True)
        rstd = (var + EPS) ** -0.5
        return torch.addcmul(d["b"], (x - mean) * rstd, d["w"]), mean.squeeze(1), rstd.squeeze(1)

    if kind == "norm":
        return dict(zip(("y", "mean", "rstd"), forward(d["x"])))
    if kind == "recompute":
        first = dict(zip(("y", "mean", "rstd"), forward(d["x"])))
        return first | dict(zip(("again", "mean2", "rstd2"), forward(_held(d["x"], case["format"]))))
    if kind == "ckpt":
        return _held(d["x"], case["format"])
    if kind == "wgrad":
        x = _kept(s["ckpt"], rows, case["in"], case["format"])
        dw = torch.matmul(d["dy"].t().contiguous(), x)
        db = torch.matmul(torch.ones(1, rows, dtype=torch.float64, device="cuda"), d["dy"]).squeeze(0)
        if case["accumulate"]:
            dw, db = d["dw"] + dw, d["db"] + db
        return {"dw": dw, "db": db} if case["bias"] else {"dw": dw}
    if kind == "block":
        y, mean, rstd = forward(d["x"])
        held = _held(y.to(REAL[case["y"]]).double(), case["format"])
        return {"y": y, "mean": mean, "rstd": rstd, "dw": torch.matmul(d["dy"].t().contiguous(), held)}
    x = d["x"] if case["x"] in REAL else _kept(s["ckpt"], rows, case["cols"], case["x"])
    # the vector-Jacobian product of each row: J = rstd * (I - 1 1^T / n - xh xh^T / n), applied to w * dy
    xh = (x - d["mean"][:, None]) * d["rstd"][:, None]
    g = d["dy"] * d["w"]
    n = case["cols"]
    dx = d["rstd"][:, None] * (g - g.sum(1, keepdim=True) / n - xh * ((g * xh).sum(1, keepdim=True) / n))
    dw, db = torch.sum(d["dy"] * xh, 0), torch.sum(d["dy"], 0)
    if case["add_dx"]:
        dx = dx + d["dx"]
    if case["accumulate"]:
        dw, db = dw + d["dw"], db + d["db"]
    return {"dx": dx, "dw": dw, "db": db}

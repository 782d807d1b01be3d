"""Cases of the gradient clipping, AdamW, RMS norm and packed product operators, in plain form and as the
library's calls.

The operators are what a rank runs around the reduction, beside those of ``perf/operators.py``:

* the global gradient norm over many tensors, and the gradients scaled by the clipping coefficient;
* AdamW on the fp32 partitions, with that coefficient, writing the bf16 shards that the all-gather takes;
* RMS norm with the residual's addition, forward (its output also packed in 8 bits) and backward;
* linear layers on packed operands: packing in 8 and 4 bits, of a matrix and of its transpose, and the
  product of two packed operands.

A packed matrix holds a row in blocks of 32 columns. A block has one exponent byte (127 + e) and 32 codes, of one
byte (e4m3) or of four bits (e2m1, the even column in the low half); the value of a code is its e4m3 or e2m1 value
times 2^e, where e is the smallest integer (not below -124) with the block's largest magnitude at most M * 2^e, M =
448 or 6. Codes are rounded to nearest, ties to even. The buffer is the codes, rows of P = 32 * ceil(cols / 32) bytes
(P / 2 for e2m1), then the exponents, rows of P / 32 bytes.

A case has a "kind": "clip" (norm and scaled gradients), "step" (norm, then AdamW with the coefficient), "rms"
(forward), "rms_bwd", "linear" (product of a packed input, or of one that the pass packs, with a packed weight),
"dgrad" (input gradient: the output's gradient and the weight's transpose are packed, then multiplied) and "block" (RMS
norm with its output packed, then the linear layer that reads it).
"""
import math

import torch

own = False

EPS = 1e-5
LR, BETA1, BETA2, ADAM_EPS, DECAY, STEP = 3e-4, 0.9, 0.95, 1e-8, 0.1, 7


# ------------------------------------------------------------------ cases
def listed():
    return [
        # one small parameter: what the two calls cost when there is nothing to stream
        {"name": "clip 1x1000 fp32", "kind": "clip", "tensors": 1, "numel": 1000, "ragged": False, "dt": "fp32",
         "out": "fp32", "scale": 1.0},
        # eight ranks' partitions of half a billion parameters, sums of 4 micro-steps
        {"name": "clip 8x67108864 fp32-bf16", "kind": "clip", "tensors": 8, "numel": 67108864, "ragged": False,
         "dt": "fp32", "out": "bf16", "scale": 0.25},
        # a model's tensors as the backward pass leaves them, unequal and odd, most of them small
        {"name": "step 290 ragged bf16", "kind": "step", "tensors": 290, "numel": 400009, "ragged": True, "dt": "bf16",
         "shard": False, "max_norm": 1.0},
        # the partitions of eight ranks, a quarter of a billion parameters: the ZeRO step, with the shards to gather
        {"name": "step 8x33554432 fp32", "kind": "step", "tensors": 8, "numel": 33554432, "ragged": False, "dt": "fp32",
         "shard": True, "max_norm": 1.0},
        # one token through one norm: latency
        {"name": "rms 1x4096 bf16", "kind": "rms", "rows": 1, "cols": 4096, "x": "bf16", "y": "bf16", "params": "bf16",
         "residual": True, "pad": 0},
        # a micro-batch of 16k tokens on the residual stream
        {"name": "rms 16384x4096 bf16", "kind": "rms", "rows": 16384, "cols": 4096, "x": "bf16", "y": "bf16",
         "params": "bf16", "residual": True, "pad": 0},
        # an odd width, rows of a wider buffer, fp32 throughout
        {"name": "rms_bwd 4097x1023 fp32", "kind": "rms_bwd", "rows": 4097, "cols": 1023, "x": "fp32", "dy": "fp32",
         "params": "fp32", "grads": "fp32", "accumulate": False, "add_dx": False, "pad": 9},
        # the backward pass of 16k tokens from the 8-bit checkpoint, added to the gradient that passed by
        {"name": "rms_bwd 16384x4096 e4m3", "kind": "rms_bwd", "rows": 16384, "cols": 4096, "x": "e4m3", "dy": "bf16",
         "params": "bf16", "grads": "bf16", "accumulate": True, "add_dx": True, "pad": 0},
        # one token through a projection whose weight is held in 4 bits: the weight's bytes
        {"name": "linear 1x4096x4096 e4m3-e2m1", "kind": "linear", "rows": 1, "out": 4096, "in": 4096, "x": "e4m3",
         "w": "e2m1", "z": "bf16", "bias": False, "packed": True},
        # odd sizes everywhere: the gradient of a linear layer's input
        {"name": "dgrad 1001x777x1000 e4m3", "kind": "dgrad", "rows": 1001, "out": 777, "in": 1000, "x": "e4m3",
         "w": "e4m3", "z": "fp32", "bias": False, "packed": False},
        # the FFN's up projection over 16k tokens in 4 bits, its input packed on the way: the largest product
        {"name": "linear 16384x11008x4096 e2m1", "kind": "linear", "rows": 16384, "out": 11008, "in": 4096, "x": "e2m1",
         "w": "e2m1", "z": "bf16", "bias": True, "packed": False},
        # a norm and the projection behind it, as a layer's forward pass has them
        {"name": "block 8192x4096x4096 e4m3", "kind": "block", "rows": 8192, "out": 4096, "in": 4096, "x": "e4m3",
         "w": "e4m3", "z": "bf16", "bias": False, "packed": False},
    ]


def draw(rng):
    def size(lo, hi):
        v = int(math.exp(rng.uniform(math.log(lo), math.log(hi + 1))))
        v = max(lo, min(hi, v))
        return v if rng.random() < 0.4 else max(lo, v // 16 * 16)  # odd sizes among them

    real = ("bf16", "fp32")
    kind = rng.choice(("clip", "step", "step", "rms", "rms_bwd", "linear", "linear", "dgrad", "block"))
    case = {"kind": kind}
    if kind in ("clip", "step"):
        n = size(1, 24 if kind == "clip" else 400)
        case |= {"tensors": n, "numel": size(1, (1 << 27) // n), "ragged": rng.random() < 0.5, "dt": rng.choice(real)}
        if kind == "clip":
            return case | {"out": rng.choice(real), "scale": rng.choice((1.0, 0.25, 1 / 3))}
        return case | {"shard": rng.random() < 0.7, "max_norm": rng.choice((1.0, 0.1, 1e9))}
    if kind in ("rms", "rms_bwd"):
        cols = size(64, 16384)
        rows = size(1, max(1, min(65536, (1 << 26) // cols)))
        case |= {"rows": rows, "cols": cols, "params": rng.choice(real), "pad": rng.choice((0, 0, 8, 5))}
        if kind == "rms":
            return case | {"x": rng.choice(real), "y": rng.choice(real), "residual": rng.random() < 0.7}
        return case | {"x": rng.choice(real + ("e4m3", "int8")), "dy": rng.choice(real), "grads": rng.choice(real),
                       "accumulate": rng.random() < 0.5, "add_dx": rng.random() < 0.5}
    out, inn = size(16, 11008), size(16, 11008)
    rows = size(1, min(32768, max(1, (1 << 38) // (out * inn))))
    packed = ("e4m3", "e2m1")
    x = "e4m3" if kind == "block" else rng.choice(packed)
    return case | {"rows": rows, "out": out, "in": inn, "x": x, "w": rng.choice(packed), "z": rng.choice(real),
                   "bias": kind != "dgrad" and rng.random() < 0.5, "packed": kind == "linear" and rng.random() < 0.5}


# ----------------------------------------------------------------- inputs
REAL = {"bf16": torch.bfloat16, "fp32": torch.float32}
SIZE = {"bf16": 2.0, "fp32": 4.0, "e4m3": 33 / 32, "int8": 33 / 32, "e2m1": 17 / 32}


def _activations(g, rows, cols):
    """A residual stream's values: channels of unequal size, a few of them far larger."""
    dev = "cuda"
    chan = torch.exp(0.4 * torch.randn(cols, generator=g, device=dev))
    chan = torch.where(torch.rand(cols, generator=g, device=dev) < 0.01, chan * 12, chan)
    return torch.randn(rows, cols, generator=g, device=dev).mul_(chan)


def _gradients(g, rows, cols):
    """Gradients of activations: small, rows of unequal size."""
    row = 1e-3 * torch.exp(0.7 * torch.randn(rows, 1, generator=g, device="cuda"))
    return torch.randn(rows, cols, generator=g, device="cuda").mul_(row)


def _numels(case):
    """Sizes of the tensors: equal, or from a 64th of `numel` to all of it in turn, and odd."""
    n, most = case["tensors"], case["numel"]
    return [max(1, most >> (k * 5 % 7)) - (k % 3 if most > 500 else 0) for k in range(n)] if case["ragged"] else [most] * n


def _views(flat, numels):
    return list(flat.split(numels))


def _in_padded(x, pad):
    """x as the left columns of a buffer with `pad` more."""
    if not pad:
        return x
    wide = torch.zeros(x.shape[0], x.shape[1] + pad, dtype=x.dtype, device=x.device)
    wide[:, :x.shape[1]] = x
    return wide[:, :x.shape[1]]


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    kind = case["kind"]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if kind in ("clip", "step"):
        numels = s["numels"] = _numels(case)
        total = sum(numels)
        # tensors whose gradients are of unequal size
        s["grads"] = [randn(n).mul_(1e-3 * 2.0 ** (k % 4)).to(REAL[case["dt"]]) for k, n in enumerate(numels)]
        s["norm"], s["coef"] = torch.empty((), device="cuda"), torch.empty((), device="cuda")
        if kind == "clip":
            s["outs"] = [torch.empty(n, dtype=REAL[case["out"]], device="cuda") for n in numels]
            return s
        # the optimizer's state: flat, a view for each tensor
        s["p"] = randn(total).mul_(0.02)
        s["m"] = randn(total).mul_(1e-4)
        s["v"] = randn(total).mul_(1e-3).square_()
        s["views"] = {k: _views(s[k], numels) for k in ("p", "m", "v")}
        if case["shard"]:
            s["shard"] = torch.empty(total, dtype=torch.bfloat16, device="cuda")
            s["views"]["shard"] = _views(s["shard"], numels)
        return s
    rows = case["rows"]
    if kind in ("rms", "rms_bwd"):
        cols = case["cols"]
        s["w"] = (1 + 0.2 * randn(cols)).to(REAL[case["params"]])
        x = _activations(g, rows, cols)
        if kind == "rms":
            s["x"] = _in_padded(x.to(REAL[case["x"]]), case["pad"])
            s["y"] = torch.empty(rows, cols, dtype=REAL[case["y"]], device="cuda")
            s["rstd"] = torch.empty(rows, device="cuda")
            if case["residual"]:
                s["residual"] = _activations(g, rows, cols).to(REAL[case["x"]])
                s["h"] = torch.empty(rows, cols, dtype=REAL[case["x"]], device="cuda")
            return s
        if case["x"] in REAL:
            s["x"] = _in_padded(x.to(REAL[case["x"]]), case["pad"])
            x = s["x"].float()
        else:
            x = x.bfloat16().float()
            s["ckpt"] = _to_buffer(*_encode(x, case["x"]), case["x"])
        # the statistics that the forward pass kept
        s["rstd"] = (x.double().square().mean(1) + EPS).rsqrt().float()
        s["dy"] = _in_padded(_gradients(g, rows, cols).to(REAL[case["dy"]]), case["pad"])
        s["dx"] = _gradients(g, rows, cols).to(REAL[case["dy"]])
        s["dw"] = (1e-3 * randn(cols)).to(REAL[case["grads"]])
        return s
    out, inn = case["out"], case["in"]
    w = randn(out, inn).mul_(inn ** -0.5)
    if kind == "dgrad":
        s["dz"] = _gradients(g, rows, out).bfloat16()
        s["w"] = w.bfloat16()
        s["z"] = torch.empty(rows, inn, dtype=REAL[case["z"]], device="cuda")
        s["x8"], s["w8"] = _buffer(rows, out, case["x"]), _buffer(inn, out, case["w"])
        return s
    s["w8"] = _to_buffer(*_encode(w.bfloat16().float(), case["w"]), case["w"])
    s["z"] = torch.empty(rows, out, dtype=REAL[case["z"]], device="cuda")
    if case["bias"]:
        s["bias"] = (0.1 * randn(out)).to(REAL[case["z"]])
    x = _activations(g, rows, inn)
    if kind == "block":
        s["x"], s["residual"] = x.bfloat16(), _activations(g, rows, inn).bfloat16()
        s["h"], s["rstd"] = torch.empty_like(s["x"]), torch.empty(rows, device="cuda")
        s["weight"] = (1 + 0.2 * randn(inn)).bfloat16()
        s["x8"] = _buffer(rows, inn, case["x"])
    elif case["packed"]:
        s["x8"] = _to_buffer(*_encode(x.bfloat16().float(), case["x"]), case["x"])
    else:
        s["x"], s["x8"] = x.bfloat16(), _buffer(rows, inn, case["x"])
    return s


# ------------------------------------------------------------- plain forms
def _pitch(cols):
    return 32 * -(-cols // 32)


def _bytes(rows, cols, fmt):
    p = _pitch(cols)
    return rows * ((p // 2 if fmt == "e2m1" else p) + p // 32)


def _buffer(rows, cols, fmt):
    return torch.empty(_bytes(rows, cols, fmt), dtype=torch.uint8, device="cuda")


def _two_to(e):
    """2^e of whole e, exactly (from the bits: a power function may be off)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _encode(x, fmt):
    """(scaled and rounded values [rows, P/32, 32] in fp32, exponents [rows, P/32]) of fp32 x."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, _pitch(cols) - cols)).view(rows, -1, 32)
    amax = x.abs().amax(-1)
    m, k = torch.frexp(amax)
    if fmt == "e4m3":
        e = k - 9 + (m > 0.875).int()
    elif fmt == "int8":
        e = k - 7 + (m > 127 / 128).int()
    else:
        e = k - 3 + (m > 0.75).int()
    e = torch.where(amax > 0, e, -124).clamp_min(-124)
    v = x * _two_to(-e).unsqueeze(-1)
    if fmt == "int8":
        return torch.round(v), e
    _, k = torch.frexp(v)
    # the step: bits behind the leading one, down to the subnormals'
    step = _two_to(k.sub_(1).clamp_(min=-6 if fmt == "e4m3" else 0).sub_(3 if fmt == "e4m3" else 1))
    return torch.round(v / step) * step, e


def _decode(q, e, cols):
    return (q * _two_to(e).unsqueeze(-1)).view(q.shape[0], -1)[:, :cols]


def _held(x, fmt):
    return _decode(*_encode(x, fmt), x.shape[1])


def _e2m1(device):
    return torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], device=device)


def _to_buffer(q, e, fmt):
    if fmt == "e2m1":
        c = torch.bucketize(q.abs(), _e2m1(q.device)) + 8 * (q < 0)
        codes = (c[..., ::2] + 16 * c[..., 1::2]).to(torch.uint8)
    else:
        codes = (q.to(torch.float8_e4m3fn) if fmt == "e4m3" else q.to(torch.int8)).view(torch.uint8)
    return torch.cat([codes.reshape(-1), (e + 127).to(torch.uint8).reshape(-1)])


def _from_buffer(buf, rows, cols, fmt):
    """fp32 values of a packed matrix."""
    p = _pitch(cols)
    n = rows * (p // 2 if fmt == "e2m1" else p)
    codes = buf[:n]
    if fmt == "e2m1":
        table = torch.cat([_e2m1(buf.device), -_e2m1(buf.device)])
        q = table[torch.stack([codes & 15, codes >> 4], -1).int()]
    else:
        q = codes.view(torch.float8_e4m3fn if fmt == "e4m3" else torch.int8).float()
    return _decode(q.view(rows, p // 32, 32), buf[n:].view(rows, p // 32).int() - 127, cols)


def _norm_coef(s, scale, max_norm):
    """Norm and clipping coefficient of the gradients that stand for scale * grads."""
    grads = s["grads"] if len(s["grads"]) <= 32 else [torch.cat(s["grads"])]
    sums = torch.stack([g.double().square_().sum() for g in grads])
    norm = sums.sum().sqrt() * scale
    return norm.float(), (torch.clamp(max_norm / norm, max=1.0) * scale).float()


def _product(x, w, s, dt):
    z = x @ w.t()
    if "bias" in s:
        z = z + s["bias"].float()
    return z.to(dt)


def _rms(x, w):
    rstd = 1 / torch.sqrt((x * x).mean(1) + EPS)
    return x * rstd.unsqueeze(1) * w.float(), rstd


def _plain(s):
    case = s["case"]
    kind = case["kind"]
    if kind == "clip":
        norm, coef = _norm_coef(s, case["scale"], 1.0)
        return {"norm": norm, "coef": coef, "outs": [(g.float() * coef).to(REAL[case["out"]]) for g in s["grads"]]}
    if kind == "step":
        norm, coef = _norm_coef(s, 1.0, case["max_norm"])
        p, m, v = s["p"], s["m"], s["v"]
        g = torch.cat(s["grads"]).float() * coef
        m.mul_(BETA1).add_(g * (1 - BETA1))
        v.mul_(BETA2).add_(g * g * (1 - BETA2))
        root = (v / (1 - BETA2 ** STEP)).sqrt_().add_(ADAM_EPS)
        p.mul_(1 - LR * DECAY).sub_((m / root).mul_(LR / (1 - BETA1 ** STEP)))
        r = {"norm": norm, "coef": coef, "p": p, "m": m, "v": v}
        return r | {"shard": p.bfloat16()} if case["shard"] else r
    rows = case["rows"]
    if kind == "rms":
        h = s["x"]
        if case["residual"]:
            h = (h.float() + s["residual"].float()).to(REAL[case["x"]])
        y, rstd = _rms(h.float(), s["w"])
        r = {"y": y.to(REAL[case["y"]]), "rstd": rstd}
        return r | {"h": h} if case["residual"] else r
    if kind == "rms_bwd":
        x = s["x"].float() if case["x"] in REAL else _from_buffer(s["ckpt"], rows, case["cols"], case["x"])
        dy, rstd = s["dy"].float(), s["rstd"].unsqueeze(1)
        xh = x * rstd
        dw = (dy * xh).sum(0)
        g = dy * s["w"].float()
        dx = (g - xh * (g * xh).mean(1, keepdim=True)) * rstd
        if case["add_dx"]:
            dx = dx + s["dx"].float()
        if case["accumulate"]:
            dw = dw + s["dw"].float()
        s["dx"].copy_(dx)
        s["dw"].copy_(dw)
        return {"dx": s["dx"], "dw": s["dw"]}
    out, inn, dt = case["out"], case["in"], REAL[case["z"]]
    if kind == "dgrad":
        return _product(_held(s["dz"].float(), case["x"]), _held(s["w"].float().t(), case["w"]), s, dt)
    w = _from_buffer(s["w8"], out, inn, case["w"])
    if kind == "linear":
        x = _from_buffer(s["x8"], rows, inn, case["x"]) if case["packed"] else _held(s["x"].float(), case["x"])
        return _product(x, w, s, dt)
    h = (s["x"].float() + s["residual"].float()).bfloat16()
    y, rstd = _rms(h.float(), s["weight"])
    return {"h": h, "rstd": rstd, "z": _product(_held(y.bfloat16().float(), case["x"]), w, s, dt)}


# ------------------------------------------------------ the library's calls
def _workspace(s, nbytes):
    """The workspace that a program keeps beside its buffers."""
    if "ws" not in s or s["ws"].numel() < nbytes:
        s["ws"] = torch.empty(max(nbytes, 1), dtype=torch.uint8, device="cuda")
    return s["ws"]


def _calls(s):
    import gradient_sync_zr_amd as zr

    case = s["case"]
    kind = case["kind"]
    fmt = {"e4m3": zr.ZR_CKPT_E4M3, "int8": zr.ZR_CKPT_INT8, "e2m1": zr.ZR_CKPT_E2M1}
    if kind in ("clip", "step"):
        numels = s["numels"]
        ws = _workspace(s, zr.zr_grad_norm_workspace_bytes(len(numels)))
        if kind == "step" and "tables" not in s:  # what an optimizer keeps of its state: a table of each list
            s["tables"] = {k: zr.tensor_table(x, numels) for k, x in (s["views"] | {"grads": s["grads"]}).items()}
        t = s["tables"] if kind == "step" else s
        zr.zr_grad_norm(t["grads"], numels, s["norm"], s["coef"], max_norm=1.0 if kind == "clip" else case["max_norm"],
                        scale=case["scale"] if kind == "clip" else 1.0, workspace=ws)
        r = {"norm": s["norm"], "coef": s["coef"]}
        if kind == "clip":
            zr.zr_grad_scale(s["grads"], numels, s["coef"], s["outs"])
            return r | {"outs": s["outs"]}
        zr.zr_adamw(t["grads"], numels, t["p"], t["m"], t["v"], step=STEP, lr=LR, beta1=BETA1, beta2=BETA2,
                    eps=ADAM_EPS, weight_decay=DECAY, shards=t.get("shard"), coef=s["coef"])
        return r | {k: s[k] for k in s["views"]}
    rows = case["rows"]
    if kind == "rms":
        zr.zr_rmsnorm_fwd(s["x"], rows, case["cols"], s["y"], s["w"], eps=EPS, residual=s.get("residual"),
                          h=s.get("h"), rstd=s["rstd"])
        return {k: s[k] for k in ("y", "rstd", "h") if k in s}
    if kind == "rms_bwd":
        cols = case["cols"]
        ws = _workspace(s, zr.zr_rmsnorm_workspace_bytes(rows, cols))
        real = case["x"] in REAL
        zr.zr_rmsnorm_bwd(s["dy"], s["x"] if real else s["ckpt"], rows, cols, s["rstd"], s["w"], dx=s["dx"],
                          dweight=s["dw"], h_dtype=None if real else fmt[case["x"]], accumulate=case["accumulate"],
                          add_dx=case["add_dx"], workspace=ws)
        return {"dx": s["dx"], "dw": s["dw"]}
    out, inn = case["out"], case["in"]
    x, w = fmt[case["x"]], fmt[case["w"]]
    if kind == "dgrad":
        zr.zr_ckpt_pack(s["dz"], rows, out, s["x8"], format=x)
        zr.zr_ckpt_pack_t(s["w"], out, inn, s["w8"], format=w)
        out, inn = inn, out
    elif kind == "block":
        zr.zr_rmsnorm_fwd(s["x"], rows, inn, None, s["weight"], eps=EPS, residual=s["residual"], h=s["h"],
                          rstd=s["rstd"], ckpt_y=s["x8"], ckpt_format=x, y_dtype=zr.ZR_BF16)
    elif not case["packed"]:
        zr.zr_ckpt_pack(s["x"], rows, inn, s["x8"], format=x)
    ws = _workspace(s, zr.zr_ckpt_linear_workspace_bytes(rows, inn, out))
    zr.zr_ckpt_linear(s["x8"], s["w8"], rows, inn, out, s["z"], bias=s.get("bias"), x_format=x, w_format=w, workspace=ws)
    return {k: s[k] for k in ("h", "rstd", "z")} if kind == "block" else s["z"]


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------------------- work
def work(case):
    kind = case["kind"]
    if kind in ("clip", "step"):
        n, g = float(sum(_numels(case))), SIZE[case["dt"]]
        if kind == "clip":
            return {"bytes": n * (2 * g + SIZE[case["out"]]) + 8, "flops": 3.0 * n}
        return {"bytes": n * (2 * g + 24 + (2 if case["shard"] else 0)) + 8, "flops": 18.0 * n}
    rows = case["rows"]
    if kind in ("rms", "rms_bwd"):
        cols = case["cols"]
        n = float(rows * cols)
        if kind == "rms":
            x = SIZE[case["x"]]
            return {"bytes": n * (x * (3 if case["residual"] else 1) + SIZE[case["y"]]) + cols * SIZE[case["params"]] +
                    4 * rows, "flops": (5.0 if case["residual"] else 4.0) * n}
        x = (n if case["x"] in REAL else rows * _pitch(cols)) * SIZE[case["x"]]
        dx = n * SIZE[case["dy"]] * (2 if case["add_dx"] else 1)
        return {"bytes": x + n * SIZE[case["dy"]] + dx + cols * SIZE[case["params"]] + 4 * rows +
                cols * SIZE[case["grads"]] * (2 if case["accumulate"] else 1), "flops": 10.0 * n}
    out, inn = case["out"], case["in"]
    z = 2.0 * rows * out * inn
    if kind == "dgrad":  # read in 16 bits, written and read in the packed formats
        px, pw = rows * _pitch(out) * SIZE[case["x"]], inn * _pitch(out) * SIZE[case["w"]]
        return {"bytes": 2.0 * rows * out + 2.0 * out * inn + 2 * px + 2 * pw + rows * inn * SIZE[case["z"]],
                "flops": z + 3.0 * (rows * out + out * inn)}
    px, pw = rows * _pitch(inn) * SIZE[case["x"]], out * _pitch(inn) * SIZE[case["w"]]
    bytes_ = px + pw + rows * out * SIZE[case["z"]] + (out * SIZE[case["z"]] if case["bias"] else 0)
    if kind == "block":
        return {"bytes": bytes_ + px + 6.0 * rows * inn + 2 * inn + 4 * rows, "flops": z + 8.0 * rows * inn}
    if not case["packed"]:
        return {"bytes": bytes_ + px + 2.0 * rows * inn, "flops": z + 3.0 * rows * inn}
    return {"bytes": bytes_, "flops": z}


# ---------------------------------------------------------------- 64 bits
def _power(e):
    """2^e of whole e in fp64, exactly."""
    return ((e.long() + 1023) << 52).view(torch.float64)


def _values(fmt, device):
    """The non-negative values that a code stands for, by code."""
    if fmt == "int8":
        return torch.arange(128, dtype=torch.float64, device=device)
    bits, bias, n = (3, 7, 127) if fmt == "e4m3" else (1, 1, 8)
    c = torch.arange(n, dtype=torch.float64, device=device)
    ex, fr = torch.floor(c / 2 ** bits), c % 2 ** bits
    return torch.where(ex > 0, (1 + fr / 2 ** bits) * _power(ex - bias), fr * 2.0 ** (1 - bias - bits))


def _nearest(x, fmt):
    """What a packed matrix keeps of fp64 x, from the format's definition: the nearest value of its table."""
    rows, cols = x.shape
    p = _pitch(cols)
    blocks = torch.zeros(rows, p, dtype=torch.float64, device=x.device)
    blocks[:, :cols] = x
    blocks = blocks.view(-1, 32)
    table = _values(fmt, x.device)
    amax = blocks.abs().max(1, keepdim=True).values
    scale = _power(torch.ceil(torch.log2(amax / table[-1])).clamp(min=-124.0))
    # the logarithm of a power of two may come out next to it
    scale = torch.where((amax <= table[-1] * scale / 2) & (scale > 2.0 ** -124), scale / 2, scale)
    scale = torch.where(amax > table[-1] * scale, scale * 2, scale)
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
    """The fp64 values of a packed buffer, code by code."""
    p = _pitch(cols)
    t = _values(fmt, buf.device)
    if fmt == "int8":
        value = torch.cat([t, torch.arange(-128, 0, dtype=torch.float64, device=buf.device)])
    elif fmt == "e4m3":
        nan = torch.full((1,), float("nan"), dtype=torch.float64, device=buf.device)
        value = torch.cat([t, nan, -t, nan])
    else:
        value = torch.cat([t, -t])
    n = rows * (p // 2 if fmt == "e2m1" else p)
    codes = buf[:n].long()
    if fmt == "e2m1":
        codes = torch.stack([codes % 16, codes // 16], 1).view(-1)
    return (value[codes].view(rows, -1, 32) * _power(buf[n:].long() - 127).view(rows, -1, 1)).view(rows, p)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    kind = case["kind"]
    if kind in ("clip", "step"):
        grads = [g.double() for g in s["grads"]]
        scale, limit = (case["scale"], 1.0) if kind == "clip" else (1.0, case["max_norm"])
        norm = scale * math.sqrt(math.fsum(float(torch.dot(g, g)) for g in grads))
        coef = scale * min(1.0, limit / norm)
        r = {"norm": torch.tensor(norm, dtype=torch.float64), "coef": torch.tensor(coef, dtype=torch.float64)}
        if kind == "clip":
            return r | {"outs": [coef * g for g in grads]}
        g = coef * torch.cat(grads)
        m = torch.lerp(g, s["m"].double(), BETA1)
        v = torch.lerp(g.pow(2), s["v"].double(), BETA2)
        move = m / (1 - BETA1 ** STEP) / (torch.pow(v / (1 - BETA2 ** STEP), 0.5) + ADAM_EPS)
        p = s["p"].double()
        p = p - LR * (move + DECAY * p)
        r |= {"p": p, "m": m, "v": v}
        return r | {"shard": p} if case["shard"] else r
    rows = case["rows"]

    def forward(h, w):
        rstd = (h.pow(2).sum(1) / h.shape[1] + EPS).pow(-0.5)
        return torch.einsum("rc,r,c->rc", h, rstd, w.double()), rstd

    if kind == "rms":
        h = s["x"].double()
        if case["residual"]:
            total = h + s["residual"].double()
            h = total.to(REAL[case["x"]]).double()
        y, rstd = forward(h, s["w"])
        r = {"y": y, "rstd": rstd}
        return r | {"h": total} if case["residual"] else r
    if kind == "rms_bwd":
        h = s["x"].double() if case["x"] in REAL else _kept(s["ckpt"], rows, case["cols"], case["x"])
        dy, rstd = s["dy"].double(), s["rstd"].double()
        # y_j = h_j rstd w_j with rstd a function of h: d rstd / d h_i = -rstd^3 h_i / n
        g = dy * s["w"].double()
        along = (g * h).sum(1)
        dx = g * rstd[:, None] - h * (along * rstd.pow(3) / case["cols"])[:, None]
        dw = torch.matmul(rstd, dy * h)
        if case["add_dx"]:
            dx = dx + s["dx"].double()
        if case["accumulate"]:
            dw = dw + s["dw"].double()
        return {"dx": dx, "dw": dw}
    out, inn = case["out"], case["in"]
    if kind == "dgrad":
        w = _nearest(s["w"].double().t().contiguous(), case["w"])
        return torch.matmul(_nearest(s["dz"].double(), case["x"]), w.t().contiguous())
    w = _kept(s["w8"], out, inn, case["w"]).t().contiguous()
    bias = s["bias"].double() if case["bias"] else 0.0
    if kind == "linear":
        x = _kept(s["x8"], rows, inn, case["x"]) if case["packed"] else _nearest(s["x"].double(), case["x"])
        return torch.matmul(x, w) + bias
    total = s["x"].double() + s["residual"].double()
    y, rstd = forward(total.bfloat16().double(), s["weight"])
    return {"h": total, "rstd": rstd, "z": torch.matmul(_nearest(y.to(torch.bfloat16).double(), case["x"]), w) + bias}

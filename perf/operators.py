"""The 8-bit activation checkpoints and the operators that write and read them:
what a training step asks of them, case by case.

Operators
  checkpoint   a [rows, cols] 16-bit activation saved in 8 bits (one fp32 scale
               per 256 elements of a row) and restored
  glu          the gated (or plain) activation of an MLP: forward with the
               checkpoints of its inputs, backward from the checkpoints
  norm         residual add + RMS or layer norm: forward with the checkpoint
               of the residual stream, backward from it, parameter gradients
  weight_grad  a linear layer's weight and bias gradient from the checkpoint of
               its input, written into the 16-bit local gradient
"""

import math

import torch

own = False

BLOCK = 256
QMAX = {"int8": 127.0, "e4m3": 448.0}
FORMAT = {"int8": 1, "e4m3": 2}          # ZERO_ACT_INT8, ZERO_ACT_E4M3
FN = {"silu": 1, "gelu": 2, "gelu_tanh": 3}   # ZERO_GLU_*
KIND = {"rms": 1, "layer": 2}            # ZERO_NORM_*
DTYPE = {"f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5
DEVICE = "cuda"


def listed():
    return [
        # One token's hidden state (h = 1600): the launches are all there is.
        dict(name="checkpoint_one_token", op="checkpoint", rows=1, cols=1600, pad=0, dtype="f16", format="int8"),
        # A ragged batch with odd rows and an odd row stride: nothing is aligned.
        dict(name="checkpoint_ragged", op="checkpoint", rows=4095, cols=4801, pad=6, dtype="f16", format="e4m3"),
        # An MLP-wide activation of a long batch: pure streaming.
        dict(name="checkpoint_large", op="checkpoint", rows=16384, cols=16384, pad=0, dtype="bf16", format="int8"),
        # GPT-2's MLP (h = 1600, 4h) over one 1024-token context: GELU without a gate, forward and backward.
        dict(name="glu_gpt2", op="glu", mode="train", rows=1024, cols=6400, dtype="f16", fn="gelu_tanh", gated=False,
             format="int8", recompute=False),
        # Backward alone over a ragged batch, rows of odd length.
        dict(name="glu_ragged_backward", op="glu", mode="backward", rows=2047, cols=5461, dtype="bf16", fn="gelu",
             gated=True, format="e4m3", recompute=False),
        # A gated MLP (h = 4096, 4h) over 8192 tokens; gate and up are the halves of one product's output, and the
        # backward pass recomputes the activation for the next weight gradient.
        dict(name="glu_large", op="glu", mode="train", rows=8192, cols=16384, dtype="bf16", fn="silu", gated=True,
             format="int8", recompute=True),
        # GPT-2's layer norm over one context, with bias.
        dict(name="norm_gpt2", op="norm", mode="train", rows=1024, cols=1600, dtype="f16", kind="layer", bias=True,
             branch=True, alpha=1.0, format="int8"),
        # Few rows of odd length, backward alone: the parameter gradients' sum over rows is the work.
        dict(name="norm_ragged_backward", op="norm", mode="backward", rows=333, cols=5001, dtype="bf16", kind="rms",
             bias=False, branch=False, alpha=1.0, format="e4m3"),
        # A residual stream of h = 4096 with a residual scale, over 16384 tokens.
        dict(name="norm_large", op="norm", mode="train", rows=16384, cols=4096, dtype="bf16", kind="rms", bias=False,
             branch=True, alpha=0.5, format="int8"),
        # GPT-2's attention input product for a few dozen tokens.
        dict(name="weight_grad_few_tokens", op="weight_grad", rows=48, inner=1600, outer=4800, dtype="f16",
             format="e4m3", bias=True, accumulate=False),
        # GPT-2's MLP input product for four contexts less one token.
        dict(name="weight_grad_gpt2", op="weight_grad", rows=4095, inner=1600, outer=6400, dtype="f16", format="int8",
             bias=True, accumulate=False),
        # A wide MLP product (h = 4096, 4h) over 16384 tokens: bound by the matrix cores.
        dict(name="weight_grad_large", op="weight_grad", rows=16384, inner=4096, outer=16384, dtype="bf16",
             format="int8", bias=False, accumulate=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["checkpoint", "glu", "norm", "weight_grad"])
    c = dict(op=op, dtype=rng.choice(["f16", "bf16"]), format=rng.choice(["int8", "e4m3"]))
    c["rows"] = _log_uniform(rng, 1, 16384)
    if op == "checkpoint":
        c["cols"] = _log_uniform(rng, 1, 16384)
        c["pad"] = rng.choice([0, 0, rng.randrange(1, 64)])
    elif op == "glu":
        c["rows"] = min(c["rows"], 8192)
        c["cols"] = _log_uniform(rng, 8, 16384)
        c.update(mode=rng.choice(["train", "backward"]), fn=rng.choice(sorted(FN)), gated=rng.random() < 0.6,
                 recompute=rng.random() < 0.5)
    elif op == "norm":
        c["cols"] = _log_uniform(rng, 16, 4096)
        c.update(mode=rng.choice(["train", "backward"]), kind=rng.choice(["rms", "layer"]), bias=rng.random() < 0.5,
                 branch=rng.random() < 0.6, alpha=rng.choice([1.0, 0.5, 0.7071]))
    else:
        c["inner"] = _log_uniform(rng, 8, 4096)
        c["outer"] = _log_uniform(rng, 8, 16384)
        c.update(bias=rng.random() < 0.5, accumulate=rng.random() < 0.5)
    return c


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _activation(gen, rows, cols, dtype, std=1.0, stride=None):
    """N(0, std) with one column in 128 five times larger, as activations' channels are; rows `stride` apart."""
    stride = cols if stride is None else stride
    x = torch.randn(rows, stride, generator=gen, device=DEVICE)
    gain = torch.where(torch.rand(stride, generator=gen, device=DEVICE) < 1 / 128, 5.0 * std, std)
    return (x * gain).to(DTYPE[dtype])[:, :cols]


def _noise(gen, rows, cols, dtype, std):
    return (torch.randn(rows, cols, generator=gen, device=DEVICE) * std).to(DTYPE[dtype])


def _pitch(cols):
    return (cols + 15) // 16 * 16


def _checkpoint_buffers(rows, cols):
    return (torch.empty(rows, _pitch(cols), dtype=torch.uint8, device=DEVICE),
            torch.empty(rows, -(-cols // BLOCK), dtype=torch.float32, device=DEVICE))


def _encoded(x, fmt):
    """The checkpoint of x (code bytes padded to the pitch, scales), as an earlier forward pass left it."""
    rows, cols = x.shape
    codes, scales = _quantise(x, fmt)
    buf, _ = _checkpoint_buffers(rows, cols)
    buf.zero_()
    buf[:, :cols] = codes.view(torch.uint8)
    return buf, scales


def _stored_codes(buf, cols, fmt):
    return buf[:, :cols].view(torch.int8 if fmt == "int8" else torch.float8_e4m3fn)


def prepare(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    c = dict(case)
    op, rows, dt, fmt = c["op"], c["rows"], c["dtype"], c["format"]
    s = {"case": c}
    if op == "checkpoint":
        cols = c["cols"]
        s["x"] = _activation(gen, rows, cols, dt, stride=cols + c["pad"])
        s["codes"], s["scales"] = _checkpoint_buffers(rows, cols)
        s["y"] = torch.empty(rows, cols, dtype=DTYPE[dt], device=DEVICE)
    elif op == "glu":
        cols, parts = c["cols"], 2 if c["gated"] else 1
        x = _activation(gen, rows, parts * cols, dt)
        s["gate"] = x[:, :cols]
        s["up"] = x[:, cols:] if c["gated"] else None
        s["dh"] = _noise(gen, rows, cols, dt, 0.01)
        s["dx"] = torch.empty(rows, parts * cols, dtype=DTYPE[dt], device=DEVICE)
        s["h"] = torch.empty(rows, cols, dtype=DTYPE[dt], device=DEVICE)
        s["h2"] = torch.empty(rows, cols, dtype=DTYPE[dt], device=DEVICE) if c["recompute"] else None
        if c["mode"] == "train":
            s["ckpt"] = [_checkpoint_buffers(rows, cols) for _ in range(parts)]
        else:
            s["ckpt"] = [_encoded(v, fmt) for v in ((s["gate"], s["up"]) if c["gated"] else (s["gate"],))]
            s["gate"] = s["up"] = None           # the checkpoints are all that is left of them
    elif op == "norm":
        cols = c["cols"]
        s["x"] = _activation(gen, rows, cols, dt)
        s["branch"] = _noise(gen, rows, cols, dt, 0.5) if c["branch"] else None
        s["weight"] = (1.0 + 0.1 * torch.randn(cols, generator=gen, device=DEVICE)).to(DTYPE[dt])
        s["bias"] = _noise(gen, 1, cols, dt, 0.1)[0] if c["bias"] else None
        s["dy"] = _noise(gen, rows, cols, dt, 0.01)
        s["dres"] = _noise(gen, rows, cols, dt, 0.01)
        for k in ("res", "y", "dx", "dbranch"):
            s[k] = torch.empty(rows, cols, dtype=DTYPE[dt], device=DEVICE)
        s["dweight"] = torch.empty(cols, dtype=DTYPE[dt], device=DEVICE)
        s["dbias"] = torch.empty(cols, dtype=DTYPE[dt], device=DEVICE)
        s["mean"] = torch.empty(rows, device=DEVICE) if c["kind"] == "layer" else None
        s["rstd"] = torch.empty(rows, device=DEVICE)
        if c["mode"] == "train":
            s["ckpt"] = _checkpoint_buffers(rows, cols)
        else:
            s["ckpt"] = _encoded(s["x"], fmt)
            mean, s["rstd"] = _norm_stats(s["x"].float(), c["kind"])
            if c["kind"] == "layer":
                s["mean"] = mean
            s["x"] = s["branch"] = None
        if own:
            from zero_sharded_mixed_flat_amd import abi
            s["ws"] = torch.empty(abi.zero_act_norm_workspace_bytes(rows, cols), dtype=torch.uint8, device=DEVICE)
    else:
        inner, outer = c["inner"], c["outer"]
        s["ckpt"] = _encoded(_activation(gen, rows, inner, dt), fmt)
        s["dy"] = _noise(gen, rows, outer, dt, 0.01)
        # earlier micro-batches' gradient (accumulated into a copy, so that every pass does the same work)
        s["dweight0"] = _noise(gen, outer, inner, dt, 0.1) if c["accumulate"] else None
        s["dbias0"] = _noise(gen, 1, outer, dt, 0.1)[0] if c["accumulate"] and c["bias"] else None
        s["dweight"] = torch.empty(outer, inner, dtype=DTYPE[dt], device=DEVICE)
        s["dbias"] = torch.empty(outer, dtype=DTYPE[dt], device=DEVICE) if c["bias"] else None
        if own:
            from zero_sharded_mixed_flat_amd import abi
            s["ws"] = torch.empty(abi.zero_act_weight_grad_workspace_bytes(rows, inner, outer), dtype=torch.uint8,
                                  device=DEVICE)
    return s


# ---------------------------------------------------------------------------
# The plain forms
# ---------------------------------------------------------------------------

def _quantise(x, fmt):
    rows, cols = x.shape
    nb = -(-cols // BLOCK)
    v = torch.zeros(rows, nb * BLOCK, device=x.device)
    v[:, :cols] = x.float()
    v = v.view(rows, nb, BLOCK)
    scale = v.abs().amax(dim=2) / torch.tensor(QMAX[fmt], device=x.device)
    q = torch.where(scale.unsqueeze(2) > 0, v / scale.unsqueeze(2), torch.zeros_like(v))
    q = q.clamp(-QMAX[fmt], QMAX[fmt]).view(rows, nb * BLOCK)[:, :cols]
    return (q.round().to(torch.int8) if fmt == "int8" else q.to(torch.float8_e4m3fn)), scale


def _restore(codes, scales, dt):
    """code * scale, rounded to the activation's 16-bit type: what a backward pass reads."""
    cols = codes.shape[1]
    s = scales.repeat_interleave(BLOCK, dim=1)[:, :cols]
    return (codes.float() * s).to(DTYPE[dt])


def _act(g, fn):
    """f(g) and f'(g)."""
    if fn == "silu":
        sg = 1.0 / (1.0 + torch.exp(-g))
        return g * sg, sg * (1.0 + g * (1.0 - sg))
    if fn == "gelu":
        cdf = 0.5 * (1.0 + torch.erf(g * math.sqrt(0.5)))
        return g * cdf, cdf + g * torch.exp(-0.5 * g * g) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = torch.tanh(k * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * k * (1.0 + 3 * 0.044715 * g * g)


def _norm_stats(r, kind):
    mean = r.mean(dim=1) if kind == "layer" else torch.zeros(r.shape[0], device=r.device)
    var = (r - mean[:, None]).square().mean(dim=1)
    return mean, 1.0 / torch.sqrt(var + EPS)


def _plain_checkpoint(s):
    c = s["case"]
    return _restore(*_quantise(s["x"], c["format"]), c["dtype"])


def _plain_glu(s):
    c = s["case"]
    dt, fmt = c["dtype"], c["format"]
    out = []
    if c["mode"] == "train":
        h = _act(s["gate"].float(), c["fn"])[0]
        if c["gated"]:
            h = h * s["up"].float()
        out.append(h.to(DTYPE[dt]))
        pairs = [_quantise(v, fmt) for v in ((s["gate"], s["up"]) if c["gated"] else (s["gate"],))]
    else:
        pairs = [(_stored_codes(b, c["cols"], fmt), sc) for b, sc in s["ckpt"]]
    f, df = _act(_restore(*pairs[0], dt).float(), c["fn"])
    dh = s["dh"].float()
    if c["gated"]:
        u = _restore(*pairs[1], dt).float()
        out += [(dh * u * df).to(DTYPE[dt]), (dh * f).to(DTYPE[dt])]
        h = f * u
    else:
        out.append((dh * df).to(DTYPE[dt]))
        h = f
    if c["recompute"]:
        out.append(h.to(DTYPE[dt]))
    return out


def _plain_norm(s):
    c = s["case"]
    dt, fmt, kind = c["dtype"], c["format"], c["kind"]
    out = []
    w = s["weight"].float()
    if c["mode"] == "train":
        r16 = s["x"]
        if c["branch"]:
            r16 = (s["x"].float() + c["alpha"] * s["branch"].float()).to(DTYPE[dt])
            out.append(r16)
        r = r16.float()
        mean, rstd = _norm_stats(r, kind)
        y = (r - mean[:, None]) * rstd[:, None] * w
        if c["bias"]:
            y = y + s["bias"].float()
        out += [y.to(DTYPE[dt]), rstd] + ([mean] if kind == "layer" else [])
        codes, scales = _quantise(r16, fmt)
    else:
        codes, scales = _stored_codes(s["ckpt"][0], c["cols"], fmt), s["ckpt"][1]
        rstd = s["rstd"]
        mean = s["mean"] if kind == "layer" else torch.zeros_like(rstd)
    n = (_restore(codes, scales, dt).float() - mean[:, None]) * rstd[:, None]
    dy = s["dy"].float()
    d = dy * w
    dr = d - n * (d * n).mean(dim=1, keepdim=True)
    if kind == "layer":
        dr = dr - d.mean(dim=1, keepdim=True)
    dr = dr * rstd[:, None] + s["dres"].float()
    out.append(dr.to(DTYPE[dt]))
    if c["branch"]:
        out.append((c["alpha"] * dr).to(DTYPE[dt]))
    out.append((dy * n).sum(dim=0).to(DTYPE[dt]))
    if c["bias"]:
        out.append(dy.sum(dim=0).to(DTYPE[dt]))
    return out


def _plain_weight_grad(s):
    c = s["case"]
    dt = c["dtype"]
    x = _restore(_stored_codes(s["ckpt"][0], c["inner"], c["format"]), s["ckpt"][1], dt).float()
    dy = s["dy"].float()
    dw = dy.t().contiguous() @ x
    if c["accumulate"]:
        dw = dw + s["dweight0"].float()
    out = [dw.to(DTYPE[dt])]
    if c["bias"]:
        db = dy.sum(dim=0)
        if c["accumulate"]:
            db = db + s["dbias0"].float()
        out.append(db.to(DTYPE[dt]))
    return out


# ---------------------------------------------------------------------------
# The framework's calls
# ---------------------------------------------------------------------------

def _own_checkpoint(s):
    from zero_sharded_mixed_flat_amd import abi
    c = s["case"]
    rows, cols, fmt = c["rows"], c["cols"], FORMAT[c["format"]]
    abi.zero_act_save(s["x"], cols + c["pad"], c["dtype"], rows, cols, fmt, s["codes"], s["scales"])
    abi.zero_act_restore(s["codes"], s["scales"], fmt, rows, cols, s["y"], cols, c["dtype"])
    return s["y"]


def _own_glu(s):
    from zero_sharded_mixed_flat_amd import abi
    c = s["case"]
    rows, cols, fmt, fn, dt = c["rows"], c["cols"], FORMAT[c["format"]], FN[c["fn"]], c["dtype"]
    gc, gs = s["ckpt"][0]
    uc, us = s["ckpt"][1] if c["gated"] else (None, None)
    stride = (2 if c["gated"] else 1) * cols
    dgate, dup = s["dx"][:, :cols], s["dx"][:, cols:] if c["gated"] else None
    out = []
    if c["mode"] == "train":
        abi.zero_act_glu_forward(s["gate"], stride, s["up"], stride, dt, rows, cols, fn, fmt, s["h"], cols, gc, gs,
                                 uc, us)
        out.append(s["h"])
    abi.zero_act_glu_backward(gc, gs, uc, us, fmt, rows, cols, fn, s["dh"], cols, dt, dgate, stride, dup, stride,
                              s["h2"], cols)
    return out + [t for t in (dgate, dup, s["h2"]) if t is not None]


def _own_norm(s):
    from zero_sharded_mixed_flat_amd import abi
    c = s["case"]
    rows, cols, fmt, kind, dt = c["rows"], c["cols"], FORMAT[c["format"]], KIND[c["kind"]], c["dtype"]
    codes, scales = s["ckpt"]
    branch = c["branch"]
    out = []
    if c["mode"] == "train":
        abi.zero_act_norm_forward(s["x"], cols, s["branch"], cols, c["alpha"], s["weight"], s["bias"], dt, rows, cols,
                                  kind, EPS, fmt, s["res"] if branch else None, cols, s["y"], cols, codes, scales,
                                  s["mean"], s["rstd"])
        out += ([s["res"]] if branch else []) + [s["y"], s["rstd"]] + ([s["mean"]] if c["kind"] == "layer" else [])
    dbranch = s["dbranch"] if branch else None
    dbias = s["dbias"] if c["bias"] else None
    abi.zero_act_norm_backward(codes, scales, fmt, s["mean"], s["rstd"], s["weight"], rows, cols, kind, s["dy"], cols,
                               s["dres"], cols, c["alpha"], dt, s["dx"], cols, dbranch, cols, False, s["dweight"],
                               dbias, s["ws"])
    return out + [t for t in (s["dx"], dbranch, s["dweight"], dbias) if t is not None]


def _own_weight_grad(s):
    from zero_sharded_mixed_flat_amd import abi
    c = s["case"]
    if c["accumulate"]:
        s["dweight"].copy_(s["dweight0"])
        if c["bias"]:
            s["dbias"].copy_(s["dbias0"])
    codes, scales = s["ckpt"]
    abi.zero_act_weight_grad(s["dy"], c["outer"], c["dtype"], codes, scales, FORMAT[c["format"]], c["rows"],
                             c["inner"], c["outer"], c["accumulate"], s["dweight"], s["dbias"], s["ws"])
    return [t for t in (s["dweight"], s["dbias"]) if t is not None]


_PLAIN = {"checkpoint": _plain_checkpoint, "glu": _plain_glu, "norm": _plain_norm, "weight_grad": _plain_weight_grad}
_OWN = {"checkpoint": _own_checkpoint, "glu": _own_glu, "norm": _own_norm, "weight_grad": _own_weight_grad}


def run(state):
    return (_OWN if own else _PLAIN)[state["case"]["op"]](state)


def work(case):
    """Every input and output once; the checkpoint is written by the forward and read by the backward pass."""
    c, op, rows = case, case["op"], case["rows"]

    def ckpt(cols):
        return rows * (cols + 4 * -(-cols // BLOCK))

    if op == "checkpoint":
        n = rows * c["cols"]
        return {"bytes": 2 * n + 2 * ckpt(c["cols"]) + 2 * n, "flops": 8 * n}
    if op == "glu":
        n, parts = rows * c["cols"], 2 if c["gated"] else 1
        b = parts * ckpt(c["cols"]) + 2 * n + 2 * n * parts + (2 * n if c["recompute"] else 0)
        f = 20 * n
        if c["mode"] == "train":
            b += 2 * n * parts + 2 * n + parts * ckpt(c["cols"])
            f += 20 * n
        return {"bytes": b, "flops": f}
    if op == "norm":
        n, cols = rows * c["cols"], c["cols"]
        b = ckpt(cols) + 4 * rows + 2 * n + 2 * n + 2 * n + (2 * n if c["branch"] else 0) + 4 * cols
        f = 16 * n
        if c["mode"] == "train":
            b += (4 * n if c["branch"] else 0) + 2 * n + 2 * n + ckpt(cols) + 4 * rows + 2 * cols
            f += 12 * n
        if c["kind"] == "layer":
            b += (8 if c["mode"] == "train" else 4) * rows
        if c["bias"]:
            b += (4 if c["mode"] == "train" else 2) * cols
        return {"bytes": b, "flops": f}
    inner, outer = c["inner"], c["outer"]
    grads = inner * outer + (outer if c["bias"] else 0)
    # accumulating reads the earlier gradient and writes the new one
    b = 2 * rows * outer + ckpt(inner) + 2 * grads * (2 if c["accumulate"] else 1)
    return {"bytes": b, "flops": 2 * rows * inner * outer + (rows * outer if c["bias"] else 0)}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_e4m3(q):
    """Nearest 4-bit-exponent, 3-bit-mantissa value, ties to even (q in fp64, |q| <= 448 up to rounding)."""
    e = torch.floor(torch.log2(q.abs().clamp_min(2.0 ** -20))).clamp(-6, 8)
    # log2 may land on the wrong side of a power of two
    e = torch.where(torch.pow(2.0, e) > q.abs(), e - 1, e)
    e = torch.where(torch.pow(2.0, e + 1) <= q.abs(), e + 1, e).clamp(-6, 8)
    step = torch.pow(2.0, e - 3)
    return (torch.round(q / step) * step).clamp(-448.0, 448.0)


def _exact_values(x, fmt):
    """What a checkpoint of the 16-bit x stands for, in fp64: the scale and the quotient are fp32 by definition."""
    rows, cols = x.shape
    out = torch.empty(rows, cols, dtype=torch.float64, device=x.device)
    for a in range(0, cols, BLOCK):
        b = min(a + BLOCK, cols)
        v = x[:, a:b].double()
        scale = (v.abs().max(dim=1, keepdim=True).values / QMAX[fmt]).float().double()
        q = torch.where(scale > 0, v / scale, torch.zeros_like(v)).float().double()
        q = torch.round(q).clamp(-127.0, 127.0) if fmt == "int8" else _exact_e4m3(q)
        out[:, a:b] = q * scale
    return out


def _exact_act(g, fn):
    if fn == "silu":
        return g / (1.0 + torch.exp(-g)), torch.sigmoid(g) * (1.0 + g * torch.sigmoid(-g))
    if fn == "gelu":
        cdf = 0.5 * torch.special.erfc(-g / math.sqrt(2.0))
        return g * cdf, cdf + g * torch.exp(-g * g / 2.0) / math.sqrt(2.0 * math.pi)
    z = math.sqrt(8.0 / math.pi) * (g + 0.044715 * g ** 3)
    sg = torch.sigmoid(z)                        # (1 + tanh(z / 2)) / 2
    return g * sg, sg + g * sg * torch.sigmoid(-z) * math.sqrt(8.0 / math.pi) * (1.0 + 0.134145 * g * g)


def exact(case, seed):
    gen = torch.Generator(device=DEVICE)
    gen.manual_seed(seed)
    c = case
    op, rows, dt, fmt = c["op"], c["rows"], c["dtype"], c["format"]
    half = DTYPE[dt]
    if op == "checkpoint":
        return _exact_values(_activation(gen, rows, c["cols"], dt, stride=c["cols"] + c["pad"]), fmt)
    if op == "glu":
        cols = c["cols"]
        x = _activation(gen, rows, (2 if c["gated"] else 1) * cols, dt)
        dh = _noise(gen, rows, cols, dt, 0.01).double()
        out = []
        if c["mode"] == "train":
            h = _exact_act(x[:, :cols].double(), c["fn"])[0]
            out.append(h * x[:, cols:].double() if c["gated"] else h)
        # the backward pass reads the checkpoint's 16-bit values
        f, df = _exact_act(_exact_values(x[:, :cols], fmt).float().to(half).double(), c["fn"])
        if c["gated"]:
            u = _exact_values(x[:, cols:], fmt).float().to(half).double()
            out += [dh * u * df, dh * f]
            f = f * u
        else:
            out.append(dh * df)
        return out + ([f] if c["recompute"] else [])
    if op == "norm":
        cols = c["cols"]
        r16 = _activation(gen, rows, cols, dt)
        branch = _noise(gen, rows, cols, dt, 0.5) if c["branch"] else None
        w = (1.0 + 0.1 * torch.randn(cols, generator=gen, device=DEVICE)).to(half).double()
        bias = _noise(gen, 1, cols, dt, 0.1)[0].double() if c["bias"] else None
        dy = _noise(gen, rows, cols, dt, 0.01).double()
        dres = _noise(gen, rows, cols, dt, 0.01).double()
        alpha = torch.tensor(c["alpha"], dtype=torch.float32).double().item()
        out = []
        train = c["mode"] == "train"
        if c["branch"] and train:
            # the residual stream is stored in 16 bits; product and sum are fp32 by definition
            r16 = ((r16.double() + (alpha * branch.double()).float().double()).float()).to(half)
            out.append(r16.double())
        r = r16.double()
        mean = r.sum(dim=1, keepdim=True) / cols if c["kind"] == "layer" else torch.zeros_like(r[:, :1])
        rstd = (((r - mean) ** 2).sum(dim=1, keepdim=True) / cols + EPS) ** -0.5
        if train:
            y = (r - mean) * rstd * w
            out += [y + bias if c["bias"] else y, rstd[:, 0]] + ([mean[:, 0]] if c["kind"] == "layer" else [])
        n = (_exact_values(r16, fmt).float().to(half).double() - mean) * rstd
        d = dy * w
        dr = rstd * (d - n * (d * n).sum(dim=1, keepdim=True) / cols
                     - (d.sum(dim=1, keepdim=True) / cols if c["kind"] == "layer" else 0.0)) + dres
        out.append(dr)
        if c["branch"]:
            out.append(alpha * dr)
        out.append((dy * n).sum(dim=0))
        return out + ([dy.sum(dim=0)] if c["bias"] else [])
    inner, outer = c["inner"], c["outer"]
    x = _exact_values(_activation(gen, rows, inner, dt), fmt).float().to(half).double()
    dy = _noise(gen, rows, outer, dt, 0.01).double()
    dw0 = _noise(gen, outer, inner, dt, 0.1).double() if c["accumulate"] else 0.0
    db0 = _noise(gen, 1, outer, dt, 0.1)[0].double() if c["accumulate"] and c["bias"] else 0.0
    out = [torch.mm(dy.t().contiguous(), x) + dw0]
    return out + ([dy.sum(dim=0) + db0] if c["bias"] else [])

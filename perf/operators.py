"""Cases, inputs and plain forms of the 8-bit activation-checkpoint operators.

The operators belong to one training step of a transformer block that keeps
its activations in 8 bits between forward and backward and puts its weight
gradients into the fp32 arena that the compressors take:

  checkpoint       an activation held as int8 codes in groups of 32 columns
                   with a power-of-two step each, and read back
  norm             RMS norm with the residual's addition; the normalised rows
                   are the checkpoint
  norm_backward    its gradient, from the checkpoint
  gated            gated activation (SiLU or tanh-GELU) of two halves of one
                   projection; as a training pass, forward and then backward
                   from the checkpoints of both halves
  gated_backward   the backward alone, which also gives the activation again
                   as a checkpoint for the next weight gradient
  weight_grad      dW = dY^T X from the checkpoint of X

A checkpoint of x[rows, cols] is codes int8[rows, ldc] with
ldc = 32 * ceil(cols / 32) (pad codes 0) and steps uint8[rows, ldc / 32]; the
value is code * 2^(step - 127).  The step of a group is the least power of two
for which its largest magnitude rounds to at most 127; a group holding a NaN
or an infinity has step 255 and reads back as NaN.
"""
import math

import torch

own = False

GROUP = 32
EPS = 1e-5
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # A few tokens' activation, f16, a width that is no multiple of the
        # group: what a short sequence or a small adapter keeps; latency.
        dict(name="checkpoint_few", op="checkpoint", rows=5, cols=1000, dtype="f16"),
        # The residual stream of 32k tokens at the Llama-3-8B width.
        dict(name="checkpoint_stream", op="checkpoint", rows=32768, cols=4096, dtype="bf16"),
        # Serving: one new token through a norm with its residual.
        dict(name="norm_token", op="norm", rows=1, cols=4096, dtype="bf16", residual=True, keep=False),
        # Training forward of a norm over 16k tokens, checkpoint kept.
        dict(name="norm_train", op="norm", rows=16384, cols=4096, dtype="bf16", residual=True, keep=True),
        # Ragged packed batch of a small fp32 model: odd rows, odd width.
        dict(name="norm_backward_odd", op="norm_backward", rows=1031, cols=1001, dtype="f32", residual=False),
        # Training backward of the norm over 16k tokens, with the residual stream's gradient.
        dict(name="norm_backward_train", op="norm_backward", rows=16384, cols=4096, dtype="bf16", residual=True),
        # Serving: one new token through the gated activation of an 8B-sized MLP.
        dict(name="gated_token", op="gated", rows=1, cols=14336, dtype="bf16", kind="silu", train=False),
        # Training pass, forward then backward, over 8k tokens of the same MLP.
        dict(name="gated_train", op="gated", rows=8192, cols=14336, dtype="bf16", kind="silu", train=True),
        # Ragged f16 batch through a GELU gate: backward, and the activation again.
        dict(name="gated_backward_ragged", op="gated_backward", rows=777, cols=4097, dtype="f16", kind="gelu"),
        # Small odd fp32 projection: weight gradient at full fp32 gradients.
        dict(name="weight_grad_odd", op="weight_grad", rows=1000, n=333, k=1001, dtype="f32", scaled=False),
        # Attention projection of a BERT-large / GPT-2-medium width, 8k tokens in
        # f16: a small weight, a long sum.
        dict(name="weight_grad_square", op="weight_grad", rows=8192, n=1024, k=1024, dtype="f16", scaled=False),
        # Up projection of an 8B-sized MLP over 16k tokens, its input the
        # checkpoint of a norm (hence the norm's weight on the columns).
        dict(name="weight_grad_mlp", op="weight_grad", rows=16384, n=14336, k=4096, dtype="bf16", scaled=True),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width over the range: any number, or a multiple of 8 or of 128."""
    w = _log_int(rng, low, high)
    m = rng.choice((1, 8, 128))
    return min(high, max(low, (w + m - 1) // m * m))


def draw(rng):
    op = rng.choice(("checkpoint", "norm", "norm_backward", "gated", "gated_backward", "weight_grad"))
    dtype = rng.choice(("bf16", "bf16", "f16", "f32"))
    case = dict(op=op, dtype=dtype)
    if op == "weight_grad":
        case |= dict(rows=_log_int(rng, 1, 16384), n=_width(rng, 16, 14336), k=_width(rng, 16, 14336),
                     scaled=rng.random() < 0.5)
        most = 16384 * 14336 * 4096 // {"bf16": 1, "f16": 2, "f32": 4}[dtype]
        while case["rows"] * case["n"] * case["k"] > most:
            big = max(("rows", "n", "k"), key=lambda f: case[f])
            case[big] = case[big] * 5 // 8 + 1
        return case
    case |= dict(rows=_log_int(rng, 1, 32768), cols=_width(rng, 32, 16384))
    most = 32768 * 4096 // (2 if dtype == "f32" else 1)
    while case["rows"] * case["cols"] > most:
        big = max(("rows", "cols"), key=lambda f: case[f])
        case[big] = case[big] * 5 // 8 + 1
    if op in ("norm", "norm_backward"):
        case["residual"] = rng.random() < 0.7
    if op == "norm":
        case["keep"] = rng.random() < 0.7
    if op in ("gated", "gated_backward"):
        case["kind"] = rng.choice(("silu", "gelu"))
    if op == "gated":
        case["train"] = rng.random() < 0.7
    return case


def _ldc(cols):
    return (cols + GROUP - 1) // GROUP * GROUP


def work(case):
    s, rows, op = SIZE[case["dtype"]], case["rows"], case["op"]
    if op == "weight_grad":
        n, k = case["n"], case["k"]
        held = rows * _ldc(k) * (1 + 1 / GROUP)
        return {"bytes": int(s * rows * n + held + 4 * n * k), "flops": 2 * rows * n * k}
    e = rows * case["cols"]
    held = rows * _ldc(case["cols"]) * (1 + 1 / GROUP)
    if op == "checkpoint":          # x read, its values written
        return {"bytes": int(2 * s * e), "flops": 4 * e}
    if op == "norm":                # x (and the residual) in, y (and h) out, the checkpoint's values in bf16
        return {"bytes": int((4 if case["residual"] else 2) * s * e + (2 * e if case["keep"] else 0)), "flops": 6 * e}
    if op == "norm_backward":       # dy, dh and the checkpoint in, dx out
        return {"bytes": int((3 if case["residual"] else 2) * s * e + held), "flops": 9 * e}
    if op == "gated":               # gate and up in, a out; then da in, both gradients out
        return {"bytes": int((6 if case["train"] else 3) * s * e), "flops": (25 if case["train"] else 8) * e}
    return {"bytes": int(3 * s * e + 2 * held + 2 * e), "flops": 25 * e}


# ------------------------------------------------------------------------------ inputs

def _activation(gen, rows, cols, dtype, spread):
    """Activations: channels of unequal size (lognormal), tokens of unequal size."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(spread * torch.randn(cols, generator=gen, device="cuda"))
    x *= torch.exp(0.2 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x.to(dtype)


def _gradient(gen, rows, cols, dtype, size):
    """Gradients: small, and zero for the tokens that the loss leaves out."""
    d = size * torch.randn(rows, cols, generator=gen, device="cuda")
    if rows > 1:
        d *= (torch.rand(rows, 1, generator=gen, device="cuda") > 0.1)
    return d.to(dtype)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, rows, dt = case["op"], case["rows"], DTYPES[case["dtype"]]
    st = dict(case)
    if op == "weight_grad":
        n, k = case["n"], case["k"]
        st["dy"] = _gradient(gen, rows, n, dt, 1e-2)
        st["codes"], st["steps"] = _quantise(_activation(gen, rows, k, torch.float32, 0.4))
        st["weight"] = (1 + 0.1 * torch.randn(k, generator=gen, device="cuda")).to(dt) if case["scaled"] else None
        st["dw"] = torch.empty(n, k, device="cuda")
        return st
    cols, ldc = case["cols"], _ldc(case["cols"])
    if op == "checkpoint":
        st["x"] = _activation(gen, rows, cols, dt, 0.4)
        st["out"] = torch.empty_like(st["x"])
    if op in ("norm", "norm_backward"):
        st["weight"] = (1 + 0.1 * torch.randn(cols, generator=gen, device="cuda")).to(dt)
    if op == "norm":
        st["x"] = _activation(gen, rows, cols, dt, 0.4)
        st["r"] = _activation(gen, rows, cols, dt, 0.4) if case["residual"] else None
        st["y"] = torch.empty_like(st["x"])
        st["h"] = torch.empty_like(st["x"]) if case["residual"] else None
        if case["keep"]:
            st["rstd"] = torch.empty(rows, device="cuda")
            st["values"] = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    if op == "norm_backward":
        h = _activation(gen, rows, cols, torch.float32, 0.4)
        st["rstd"] = torch.rsqrt(h.square().mean(1) + EPS)
        st["codes"], st["steps"] = _quantise(h * st["rstd"][:, None])
        st["dy"] = _gradient(gen, rows, cols, dt, 1e-2)
        st["dh"] = _gradient(gen, rows, cols, dt, 1e-2) if case["residual"] else None
        st["dx"] = torch.empty_like(st["dy"])
        st["dw"] = torch.empty(cols, device="cuda")
    if op in ("gated", "gated_backward"):
        both = _activation(gen, rows, 2 * cols, dt, 0.2)   # one projection's output: gate, then up
        da = _gradient(gen, rows, cols, dt, 1e-2)
    if op == "gated":
        st["both"], st["a"] = both, torch.empty(rows, cols, device="cuda", dtype=dt)
        if case["train"]:
            st["da"], st["dboth"] = da, torch.empty_like(both)
    if op == "gated_backward":
        st["da"], st["dboth"] = da, torch.empty_like(both)
        st["codes"], st["steps"] = _quantise(both[:, :cols].float())
        st["codes2"], st["steps2"] = _quantise(both[:, cols:].float())
        st["values"] = torch.empty(rows, cols, device="cuda", dtype=torch.bfloat16)
    if op == "checkpoint" or (op == "norm" and case["keep"]) or (op == "gated" and case["train"]):
        st["codes"] = torch.empty(rows, ldc, device="cuda", dtype=torch.int8)
        st["steps"] = torch.empty(rows, ldc // GROUP, device="cuda", dtype=torch.uint8)
    if op == "gated" and case["train"]:
        st["codes2"], st["steps2"] = torch.empty_like(st["codes"]), torch.empty_like(st["steps"])
    if op == "gated_backward":
        st["codes3"], st["steps3"] = torch.empty_like(st["codes"]), torch.empty_like(st["steps"])
    return st


# ------------------------------------------------------------------------- plain forms

def _quantise(x):
    """Codes and steps of fp32 x[rows, cols]."""
    rows, cols = x.shape
    x = torch.nn.functional.pad(x, (0, _ldc(cols) - cols)).view(rows, -1, GROUP)
    top = x.abs().amax(2)
    fine = torch.isfinite(top)
    bits = torch.where(fine, top, 0.0).view(torch.int32) + 0x10000
    step = ((bits >> 23).clamp(max=254) - 6).clamp(min=1)
    inverse = ((254 - step) << 23).view(torch.float32)
    codes = torch.where(fine[..., None], torch.round(x * inverse[..., None]).clamp(-127, 127), 0.0)
    step = torch.where(fine, step, 255)
    return codes.to(torch.int8).view(rows, -1), step.to(torch.uint8)


def _values(codes, steps, cols):
    """The fp32 values that a checkpoint stands for."""
    scale = (steps.to(torch.int32) << 23).view(torch.float32)
    rows = codes.shape[0]
    return (codes.view(rows, -1, GROUP).float() * scale[..., None]).view(rows, -1)[:, :cols]


def _gate(kind, g):
    """sigmoid(p(g)) and p'(g): the activation is g * sigmoid(p(g))."""
    if kind == "silu":
        return 1 / (1 + torch.exp(-g)), 1.0
    c = 2 * math.sqrt(2 / math.pi)
    return 1 / (1 + torch.exp(-c * (g + 0.044715 * g * g * g))), c * (1 + 3 * 0.044715 * g * g)


def _gate_gradients(kind, g, u, da):
    s, dp = _gate(kind, g)
    return torch.cat((da * u * (s + g * s * (1 - s) * dp), da * (g * s)), 1), g * s * u


def _plain(st):
    op, dt = st["op"], DTYPES[st["dtype"]]
    if op == "checkpoint":
        return _values(*_quantise(st["x"].float()), st["cols"]).to(dt)
    if op == "norm":
        h = st["x"].float() if st["r"] is None else st["x"].float() + st["r"].float()
        rstd = 1 / torch.sqrt(h.square().mean(1) + EPS)
        xh = h * rstd[:, None]
        out = {"y": (xh * st["weight"].float()).to(dt)}
        if st["r"] is not None:
            out["h"] = h.to(dt)
        if st["keep"]:
            out |= {"rstd": rstd, "values": _values(*_quantise(xh), st["cols"]).to(torch.bfloat16)}
        return out
    if op == "norm_backward":
        q, dy = _values(st["codes"], st["steps"], st["cols"]), st["dy"].float()
        gw = dy * st["weight"].float()
        dx = st["rstd"][:, None] * (gw - q * (gw * q).mean(1, keepdim=True))
        if st["dh"] is not None:
            dx = dx + st["dh"].float()
        return {"dx": dx.to(dt), "dw": (dy * q).sum(0)}
    if op == "gated":
        cols = st["cols"]
        g, u = st["both"][:, :cols].float(), st["both"][:, cols:].float()
        out = {"a": (g * _gate(st["kind"], g)[0] * u).to(dt)}
        if st["train"]:
            g, u = _values(*_quantise(g), cols), _values(*_quantise(u), cols)
            out["dboth"] = _gate_gradients(st["kind"], g, u, st["da"].float())[0].to(dt)
        return out
    if op == "gated_backward":
        cols = st["cols"]
        g, u = _values(st["codes"], st["steps"], cols), _values(st["codes2"], st["steps2"], cols)
        d, a = _gate_gradients(st["kind"], g, u, st["da"].float())
        return {"dboth": d.to(dt), "values": _values(*_quantise(a), cols).to(torch.bfloat16)}
    dw = st["dy"].float().T @ _values(st["codes"], st["steps"], st["k"])
    return dw if st["weight"] is None else dw * st["weight"].float()


# ---------------------------------------------------------------- the framework's calls

def _call(st):
    import gradient_compression_gb300 as gc
    op, rows = st["op"], st["rows"]
    if op == "weight_grad":
        if "ws" not in st:
            st["ws"] = gc.act_weight_grad_workspace(rows, st["n"], st["k"], st["dy"].dtype, st["dw"].device)
        kept = gc.ActCheckpoint(rows, st["k"], codes=st["codes"], steps=st["steps"])
        gc.act_weight_grad(st["dy"], kept, st["dw"], st["ws"], col_scale=st["weight"])
        return st["dw"]
    cols = st["cols"]
    if "codes" in st:
        kept = gc.ActCheckpoint(rows, cols, codes=st["codes"], steps=st["steps"])
    if op == "checkpoint":
        gc.act_compress(st["x"], kept)
        gc.act_decompress(kept, st["out"])
        return st["out"]
    if op == "norm":
        out = {"y": st["y"]}
        if st["r"] is not None:
            out["h"] = st["h"]
        if st["keep"]:
            gc.rmsnorm(st["x"], st["weight"], EPS, st["y"], residual=st["r"], h=st["h"], rstd=st["rstd"], ckpt=kept)
            gc.act_decompress(kept, st["values"])
            out |= {"rstd": st["rstd"], "values": st["values"]}
        else:
            gc.rmsnorm(st["x"], st["weight"], EPS, st["y"], residual=st["r"], h=st["h"])
        return out
    if op == "norm_backward":
        if "ws" not in st:
            st["ws"] = gc.rmsnorm_backward_workspace(rows, cols, st["dw"].device)
        gc.rmsnorm_backward(st["dy"], kept, st["rstd"], st["weight"], st["dx"], st["dw"], st["ws"], dh=st["dh"])
        return {"dx": st["dx"], "dw": st["dw"]}
    kind = gc.GC_GATE_SILU if st["kind"] == "silu" else gc.GC_GATE_GELU_TANH
    if op == "gated":
        gate, up = st["both"][:, :cols], st["both"][:, cols:]
        if not st["train"]:
            gc.gated_act(kind, gate, up, st["a"])
            return {"a": st["a"]}
        kept2 = gc.ActCheckpoint(rows, cols, codes=st["codes2"], steps=st["steps2"])
        gc.gated_act(kind, gate, up, st["a"], ckpt_gate=kept, ckpt_up=kept2)
        gc.gated_act_backward(kind, st["da"], kept, kept2, st["dboth"][:, :cols], st["dboth"][:, cols:])
        return {"a": st["a"], "dboth": st["dboth"]}
    kept2 = gc.ActCheckpoint(rows, cols, codes=st["codes2"], steps=st["steps2"])
    again = gc.ActCheckpoint(rows, cols, codes=st["codes3"], steps=st["steps3"])
    gc.gated_act_backward(kind, st["da"], kept, kept2, st["dboth"][:, :cols], st["dboth"][:, cols:], ckpt_out=again)
    gc.act_decompress(again, st["values"])
    return {"dboth": st["dboth"], "values": st["values"]}


def run(state):
    return _call(state) if own else _plain(state)


# ------------------------------------------------------------------- in 64 bits, apart

def _held64(x):
    """What a checkpoint of x holds, from the definition: the least power of
    two for which a group's largest magnitude rounds to at most 127."""
    rows, cols = x.shape
    groups = torch.nn.functional.pad(x, (0, -cols % GROUP)).reshape(rows, -1, GROUP)
    top = groups.abs().amax(-1, keepdim=True)
    exponent = torch.frexp(top)[1].double() - 7              # top / 2^exponent is in [64, 128)
    exponent = exponent + (torch.round(top * torch.exp2(-exponent)) > 127)
    step = torch.exp2(exponent.clamp(min=-126))
    return (torch.round(groups / step) * step).reshape(rows, -1)[:, :cols]


def _read64(codes, steps, cols):
    step = torch.exp2(steps.double() - 127).repeat_interleave(GROUP, 1)
    return (codes.double() * step)[:, :cols]


def _act64(kind, g):
    """The activation and its derivative."""
    if kind == "silu":
        s = torch.sigmoid(g)
        return g * s, s * (1 + g * (1 - s))
    root = math.sqrt(2 / math.pi)
    t = torch.tanh(root * (g + 0.044715 * g ** 3))
    return 0.5 * g * (1 + t), 0.5 * (1 + t) + 0.5 * g * (1 - t * t) * root * (1 + 0.134145 * g * g)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "weight_grad":
        dw = torch.matmul(st["dy"].double().T, _read64(st["codes"], st["steps"], case["k"]))
        return dw if st["weight"] is None else dw * st["weight"].double()
    cols = case["cols"]
    if op == "checkpoint":
        return _held64(st["x"].double())
    if op == "norm":
        h = st["x"].double()
        if st["r"] is not None:
            h = h + st["r"].double()
        rms = torch.sqrt((h * h).sum(1) / cols + EPS)
        out = {"y": h / rms[:, None] * st["weight"].double()}
        if st["r"] is not None:
            out["h"] = h
        if case["keep"]:
            out["rstd"], out["values"] = 1 / rms, _held64(h / rms[:, None])
        return out
    if op == "norm_backward":
        xh, dy = _read64(st["codes"], st["steps"], cols), st["dy"].double()
        dxh = dy * st["weight"].double()
        dx = (dxh - xh * ((dxh * xh).sum(1) / cols)[:, None]) * st["rstd"].double()[:, None]
        return {"dx": dx if st["dh"] is None else dx + st["dh"].double(), "dw": torch.einsum("tc,tc->c", dy, xh)}
    if op == "gated":
        g, u = st["both"].double().split(cols, 1)
        out = {"a": _act64(case["kind"], g)[0] * u}
        if case["train"]:
            f, df = _act64(case["kind"], _held64(g))
            da = st["da"].double()
            out["dboth"] = torch.cat((da * _held64(u) * df, da * f), 1)
        return out
    g, u, da = _read64(st["codes"], st["steps"], cols), _read64(st["codes2"], st["steps2"], cols), st["da"].double()
    f, df = _act64(case["kind"], g)
    return {"dboth": torch.cat((da * u * df, da * f), 1), "values": _held64(f * u)}

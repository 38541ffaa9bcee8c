"""Cases, inputs and plain forms of the gated projection and of the global
gradient norm with its clipping.

They stand at the two ends of what a training step with 8-bit activation
checkpoints and compressed gradients does to a gated feed-forward block:

  gated           out = act(x Wg^T) * (x Wu^T), both projections, the
                  activation (SiLU or tanh-GELU) and the product in one; as a
                  training pass, forward and then backward from the 8-bit
                  checkpoints of both projections' outputs
  gated_backward  the backward alone: dgate, dup and dx = dgate Wg + dup Wu
  norm            the L2 norm of all gradients of a model, tensors of any type
  clip            the norm, then every gradient times min(1, max_norm / norm)
                  into the flat fp32 arena that the compressors take

A checkpoint of x[rows, cols] is codes int8[rows, ldc] with
ldc = 32 * ceil(cols / 32) (pad codes 0) and steps uint8[rows, ldc / 32]; the
value is code * 2^(step - 127).  The step of a group is the least power of two
for which its largest magnitude rounds to at most 127.
"""
import math

import torch

own = False

GROUP = 32
DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
SIZE = {"f32": 4, "bf16": 2, "f16": 2}


# ------------------------------------------------------------------------------- cases

def listed():
    return [
        # Serving: one new token through the gate of an 8B-sized MLP; the weights' bytes.
        dict(name="gated_token", op="gated", rows=1, n=14336, k=4096, dtype="bf16", kind="silu", train=False),
        # Serving: a decode batch of 48 sequences through the same.
        dict(name="gated_batch", op="gated", rows=48, n=14336, k=4096, dtype="bf16", kind="silu", train=False),
        # A small odd f16 layer whose rows start anywhere; latency.
        dict(name="gated_odd", op="gated", rows=77, n=333, k=1001, dtype="f16", kind="gelu", train=False),
        # Training pass, forward then backward, 2k tokens at a BERT-large / GPT-2-medium width in f16.
        dict(name="gated_train_small", op="gated", rows=2048, n=4096, k=1024, dtype="f16", kind="gelu", train=True),
        # Training pass over 8k tokens of the 8B-sized MLP.
        dict(name="gated_train", op="gated", rows=8192, n=14336, k=4096, dtype="bf16", kind="silu", train=True),
        # Backward of a ragged packed batch.
        dict(name="gated_backward_ragged", op="gated_backward", rows=1031, n=4097, k=1000, dtype="f16", kind="silu"),
        # Backward of a micro-batch of 2k tokens of the 8B-sized MLP.
        dict(name="gated_backward_micro", op="gated_backward", rows=2048, n=14336, k=4096, dtype="bf16", kind="gelu"),
        # The gradients of a small adapter: a dozen odd fp32 tensors; latency.
        dict(name="clip_adapter", op="clip", layout="ragged", count=12, numel=100003, dtype="f32", clipped=True),
        # ResNet-50 in fp32: 161 tensors, most of them tiny.
        dict(name="clip_resnet50", op="clip", layout="resnet50", count=161, numel=25557032, dtype="f32", clipped=True),
        # BERT-large, matrices in bf16 and vectors in fp32, as mixed training leaves them.
        dict(name="clip_bert_large", op="clip", layout="bert_large", count=391, numel=335141888, dtype="mixed",
             clipped=True),
        # The norm alone of a Llama-3-8B gradient in bf16: a long sum.
        dict(name="norm_llama3_8b", op="norm", layout="llama3_8b", count=291, numel=8030261248, dtype="bf16"),
    ]


def _log_int(rng, low, high):
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def _width(rng, low, high):
    """A width over the range: any number, or a multiple of 8 or of 128."""
    w = _log_int(rng, low, high)
    m = rng.choice((1, 8, 128))
    return min(high, max(low, (w + m - 1) // m * m))


def draw(rng):
    op = rng.choice(("gated", "gated", "gated", "gated_backward", "gated_backward", "norm", "clip", "clip"))
    if op in ("gated", "gated_backward"):
        case = dict(op=op, dtype=rng.choice(("bf16", "f16")), rows=_log_int(rng, 1, 16384), n=_width(rng, 16, 14336),
                    k=_width(rng, 16, 8192), kind=rng.choice(("silu", "gelu")))
        if op == "gated":
            case["train"] = rng.random() < 0.5
        while case["rows"] * case["n"] * case["k"] > 8192 * 14336 * 4096:
            big = max(("rows", "n", "k"), key=lambda f: case[f])
            case[big] = case[big] * 5 // 8 + 1
        return case
    count = _log_int(rng, 1, 1500)
    case = dict(op=op, layout="ragged", count=count, numel=max(count, _log_int(rng, 1000, 400_000_000)),
                dtype=rng.choice(("f32", "bf16", "f16", "mixed")))
    if op == "clip":
        case["clipped"] = rng.random() < 0.7
    return case


def _resnet50():
    sizes, cin = [64 * 3 * 49, 64, 64], 64
    for planes, blocks in ((64, 3), (128, 4), (256, 6), (512, 3)):
        for b in range(blocks):
            out = 4 * planes
            sizes += [planes * cin, planes, planes, planes * planes * 9, planes, planes, out * planes, out, out]
            sizes += [out * cin, out, out] if b == 0 else []
            cin = out
    return sizes + [1000 * 2048, 1000]


def _bert_large():
    h, f = 1024, 4096
    layer = [h * h, h] * 4 + [h, h, f * h, f, h * f, h, h, h]
    return [30522 * h, 512 * h, 2 * h, h, h] + layer * 24 + [h * h, h]


def _llama3_8b():
    d, f, vocab, kv = 4096, 14336, 128256, 1024
    return [vocab * d] + [d * d, kv * d, kv * d, d * d, f * d, f * d, d * f, d, d] * 32 + [d, vocab * d]


LAYOUTS = {"resnet50": _resnet50, "bert_large": _bert_large, "llama3_8b": _llama3_8b}


def _sizes(case):
    """The tensors' sizes: a model's parameter list, or `count` sizes that
    differ widely, with their sum `numel`."""
    if case["layout"] != "ragged":
        return LAYOUTS[case["layout"]]()
    count, rest = case["count"], case["numel"] - case["count"]
    weight = [math.exp(4.0 * math.sin(1.0 + 2.399963 * i)) for i in range(count)]
    total = sum(weight)
    sizes = [1 + int(rest * w / total) for w in weight]
    sizes[count // 2] += case["numel"] - sum(sizes)
    return sizes


def _types(case, sizes):
    """Each tensor's type: one for all, or bf16 with the small ones in fp32."""
    if case["dtype"] != "mixed":
        return [DTYPES[case["dtype"]]] * len(sizes)
    return [torch.float32 if s <= 4096 else torch.bfloat16 for s in sizes]


def _ldc(cols):
    return (cols + GROUP - 1) // GROUP * GROUP


def work(case):
    if case["op"] in ("norm", "clip"):
        sizes = _sizes(case)
        read = sum(n * t.itemsize for n, t in zip(sizes, _types(case, sizes)))
        if case["op"] == "norm":
            return {"bytes": read, "flops": 2 * sum(sizes)}
        return {"bytes": 2 * read + 4 * sum(sizes), "flops": 3 * sum(sizes)}   # the norm is known after one reading
    s, rows, n, k = SIZE[case["dtype"]], case["rows"], case["n"], case["k"]
    held = 2 * rows * _ldc(n) * (1 + 1 / GROUP)
    forward = {"bytes": s * (rows * k + 2 * n * k + rows * n), "flops": 4 * rows * n * k + 8 * rows * n}
    # dout and the checkpoints in, dgate, dup and dx out, which the product needs whole
    backward = {"bytes": s * (3 * rows * n + 2 * n * k + rows * k) + held, "flops": 4 * rows * n * k + 17 * rows * n}
    if case["op"] == "gated_backward":
        return backward
    if not case["train"]:
        return forward
    return {"bytes": forward["bytes"] + held + backward["bytes"], "flops": forward["flops"] + backward["flops"]}


# ------------------------------------------------------------------------------ inputs

def _activation(gen, rows, cols, spread):
    """Activations: channels of unequal size (lognormal), tokens of unequal size."""
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    x *= torch.exp(spread * torch.randn(cols, generator=gen, device="cuda"))
    x *= torch.exp(0.2 * torch.randn(rows, 1, generator=gen, device="cuda"))
    return x


def _gradients(gen, case):
    """Gradients of a model's tensors: each with a size of its own, the
    elements of a tensor unequal, side by side in one buffer a type."""
    sizes = _sizes(case)
    types = _types(case, sizes)
    room = {t: torch.empty(sum(n for n, u in zip(sizes, types) if u == t), device="cuda", dtype=t) for t in set(types)}
    scale = (1e-3 * torch.exp(torch.randn(len(sizes), generator=gen, device="cuda"))).tolist()
    at, out = dict.fromkeys(room, 0), []
    for n, t, s in zip(sizes, types, scale):
        g = room[t][at[t]:at[t] + n]
        g.normal_(0.0, s, generator=gen)
        out.append(g)
        at[t] += n
    return sizes, out


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    st = dict(case)
    if case["op"] in ("norm", "clip"):
        sizes, st["grads"] = _gradients(gen, case)
        st["norm"] = torch.empty(1, device="cuda")
        if case["op"] == "clip":
            # near what the gradients' sizes give, below it where they are to be clipped
            st["max_norm"] = (0.5 if case["clipped"] else 1e3) * 1e-3 * math.sqrt(sum(sizes))
            st["arena"] = torch.empty(sum(sizes), device="cuda")
            st["views"] = list(st["arena"].split(sizes))
        return st
    rows, n, k, dt = case["rows"], case["n"], case["k"], DTYPES[case["dtype"]]
    st["w"] = (torch.randn(2 * n, k, generator=gen, device="cuda") / math.sqrt(k)).to(dt)   # the gate's rows, then up's
    if case["op"] == "gated":
        st["x"] = _activation(gen, rows, k, 0.3).to(dt)
        st["a"] = torch.empty(rows, n, device="cuda", dtype=dt)
    if case["op"] == "gated_backward" or case["train"]:
        da = 1e-2 * torch.randn(rows, n, generator=gen, device="cuda")
        if rows > 1:                                                            # tokens that the loss leaves out
            da *= (torch.rand(rows, 1, generator=gen, device="cuda") > 0.1)
        st["da"] = da.to(dt)
        st["dboth"] = torch.empty(rows, 2 * n, device="cuda", dtype=dt)
        st["dx"] = torch.empty(rows, k, device="cuda", dtype=dt)
    if case["op"] == "gated_backward":
        st["codes"], st["steps"] = _quantise(_activation(gen, rows, n, 0.2))
        st["codes2"], st["steps2"] = _quantise(_activation(gen, rows, n, 0.2))
    elif case["train"]:
        st["codes"], st["codes2"] = (torch.empty(rows, _ldc(n), device="cuda", dtype=torch.int8) for _ in range(2))
        st["steps"], st["steps2"] = (torch.empty(rows, _ldc(n) // GROUP, device="cuda", dtype=torch.uint8)
                                     for _ in range(2))
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


def _backward(st, g, u):
    dt, da = DTYPES[st["dtype"]], st["da"].float()
    s, dp = _gate(st["kind"], g)
    dboth = torch.cat((da * u * (s + g * s * (1 - s) * dp), da * (g * s)), 1)
    return {"dboth": dboth.to(dt), "dx": (dboth @ st["w"].float()).to(dt)}


def _plain(st):
    op = st["op"]
    if op in ("norm", "clip"):
        norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in st["grads"]]).sum().sqrt().float()
        if op == "norm":
            return {"norm": norm.view(1)}
        c = torch.where(norm > st["max_norm"], st["max_norm"] / norm, 1.0)
        return {"norm": norm.view(1), "arena": torch.cat([g.float() * c for g in st["grads"]])}
    n = st["n"]
    if op == "gated_backward":
        return _backward(st, _values(st["codes"], st["steps"], n), _values(st["codes2"], st["steps2"], n))
    g, u = (st["x"].float() @ st["w"].float().T).split(n, 1)
    out = {"a": (g * _gate(st["kind"], g)[0] * u).to(DTYPES[st["dtype"]])}
    if st["train"]:
        out |= _backward(st, _values(*_quantise(g), n), _values(*_quantise(u), n))
    return out


# ---------------------------------------------------------------- the framework's calls

def _call(st):
    import gradient_compression_gb300 as gc
    op = st["op"]
    if op in ("norm", "clip"):
        if "ws" not in st:
            st["ws"] = gc.grad_norm_workspace(st["grads"])
        gc.grad_norm(st["grads"], st["norm"], st["ws"])
        if op == "norm":
            return {"norm": st["norm"]}
        gc.grad_clip(st["grads"], st["norm"], st["max_norm"], out=st["views"])
        return {"norm": st["norm"], "arena": st["arena"]}
    rows, n, out = st["rows"], st["n"], {}
    kind = gc.GC_GATE_SILU if st["kind"] == "silu" else gc.GC_GATE_GELU_TANH
    wg, wu = st["w"][:n], st["w"][n:]
    both = {}
    if "codes" in st:
        both = dict(ckpt_gate=gc.ActCheckpoint(rows, n, codes=st["codes"], steps=st["steps"]),
                    ckpt_up=gc.ActCheckpoint(rows, n, codes=st["codes2"], steps=st["steps2"]))
    if op == "gated":
        if "ws" not in st:
            st["ws"] = gc.gated_proj_workspace(st["x"], wg, wu)
        gc.gated_proj(kind, st["x"], wg, wu, st["a"], st["ws"], **both)
        out["a"] = st["a"]
    if "da" in st:
        dgate, dup = st["dboth"][:, :n], st["dboth"][:, n:]
        if "ws_back" not in st:
            st["ws_back"] = gc.gated_proj_backward_workspace(dgate, dup, wg, wu)
        gc.gated_proj_backward(kind, st["da"], both["ckpt_gate"], both["ckpt_up"], wg, wu, dgate, dup, st["dx"],
                               st["ws_back"])
        out |= {"dboth": st["dboth"], "dx": st["dx"]}
    return out


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
    if case["op"] in ("norm", "clip"):
        norm = math.sqrt(math.fsum(torch.linalg.vector_norm(g.double()).item() ** 2 for g in st["grads"]))
        out = {"norm": torch.tensor([norm], device="cuda", dtype=torch.float64)}
        if case["op"] == "clip":
            factor = min(1.0, st["max_norm"] / norm)
            out["arena"] = torch.cat([factor * g.double() for g in st["grads"]])
        return out
    n, kind, out = case["n"], case["kind"], {}
    wg, wu = st["w"].double().split(n, 0)
    if case["op"] == "gated":
        x = st["x"].double()
        g, u = torch.einsum("tk,nk->tn", x, wg), torch.einsum("tk,nk->tn", x, wu)
        out["a"] = _act64(kind, g)[0] * u
        if not case["train"]:
            return out
        g, u = _held64(g), _held64(u)
    else:
        g, u = _read64(st["codes"], st["steps"], n), _read64(st["codes2"], st["steps2"], n)
    f, df = _act64(kind, g)
    da = st["da"].double()
    dg, du = da * u * df, da * f
    out["dboth"], out["dx"] = torch.cat((dg, du), 1), torch.matmul(dg, wg) + torch.matmul(du, wu)
    return out

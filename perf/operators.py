"""The layer operators as a training program calls them, for timing and comparison.

Five operators around one pre-norm layer whose matrix the optimizer steps: the
8-bit activation checkpoint (``pack``), the root-mean-square norm with the
residual's addition and its gradient (``norm``, ``norm_backward``), and the
linear layer with bias, activation and residual and its gradient (``linear``,
``linear_backward``).  With ``own`` false every operator runs in its plain form
(torch products, sums and comparisons in 32 bits, rounded once at the end); with
``own`` true it runs through the framework's entry points.

Sizes: 2048, 4096, 8192 and 11008 are the widths of the framework's 1B- and
7B-shaped workloads; the others are generic.
"""
import math

import torch

own = False

ELEM = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
BLOCK = 32   # columns that share one scale in an 8-bit checkpoint
EPS = 1e-6
MOST = 16384 * 4096 * 11008  # tokens x in x out of the largest linear layer


def listed():
    return [
        # The activations of a short ragged micro-batch, kept from a 32-bit layer.
        dict(name="pack_f32_129x1000", op="pack", dtype="f32", tokens=129, cols=1000),
        # The widest activation of a 7B-shaped layer at a full training batch.
        dict(name="pack_bf16_16384x11008", op="pack", dtype="bf16", tokens=16384, cols=11008),
        # One token at a time: the call's latency.
        dict(name="norm_bf16_1x4096", op="norm", dtype="bf16", tokens=1, cols=4096, residual=True, packed=False),
        # The norm before a matrix at a full training batch, its output kept in 8 bits too.
        dict(name="norm_bf16_16384x4096", op="norm", dtype="bf16", tokens=16384, cols=4096, residual=True,
             packed=True),
        # A ragged batch at an odd width, half precision, no residual stream.
        dict(name="norm_bwd_f16_333x2047", op="norm_backward", dtype="f16", tokens=333, cols=2047, stream=False),
        # The same norm's gradient at a full training batch, with the residual stream's own gradient.
        dict(name="norm_bwd_bf16_16384x4096", op="norm_backward", dtype="bf16", tokens=16384, cols=4096,
             stream=True),
        # One token through a 7B-shaped gate matrix: the weights' bytes and the call's latency.
        dict(name="linear_bf16_1x4096x11008", op="linear", dtype="bf16", tokens=1, infeat=4096, outfeat=11008,
             act="silu", bias=True, residual=False, keep="none"),
        # A small ragged training batch through a 1B-shaped matrix, pre-activation and output kept in 8 bits.
        dict(name="linear_bf16_500x2048x8192", op="linear", dtype="bf16", tokens=500, infeat=2048, outfeat=8192,
             act="gelu", bias=True, residual=True, keep="packed"),
        # A full training batch through a 7B-shaped matrix, pre-activation kept.
        dict(name="linear_bf16_16384x4096x11008", op="linear", dtype="bf16", tokens=16384, infeat=4096,
             outfeat=11008, act="silu", bias=True, residual=False, keep="z"),
        # A few tokens at odd widths in half precision, 32-bit gradient.
        dict(name="linear_bwd_f16_61x2047x1001", op="linear_backward", dtype="f16", tokens=61, infeat=2047,
             outfeat=1001, act="none", grad="f32", x8=False, z8=False),
        # A 1B-shaped layer's gradient from 8-bit checkpoints.
        dict(name="linear_bwd_bf16_4096x2048x8192", op="linear_backward", dtype="bf16", tokens=4096, infeat=2048,
             outfeat=8192, act="gelu", grad="bf16", x8=True, z8=True),
        # A 7B-shaped layer's gradient at a full training batch from 8-bit checkpoints.
        dict(name="linear_bwd_bf16_16384x4096x11008", op="linear_backward", dtype="bf16", tokens=16384,
             infeat=4096, outfeat=11008, act="silu", grad="bf16", x8=True, z8=True),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; every other one rounded to a multiple of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 8 and rng.random() < 0.5:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["pack", "norm", "norm_backward", "linear", "linear_backward"])
    tokens = _spread(rng, 1, 16384)
    if op in ("pack", "norm", "norm_backward"):
        c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16", "f32"]), tokens=tokens,
                 cols=_spread(rng, 64, 11008))
        if op == "norm":
            c["residual"], c["packed"] = rng.random() < 0.5, rng.random() < 0.5
        if op == "norm_backward":
            c["stream"] = rng.random() < 0.5
        return c
    infeat, outfeat = _spread(rng, 64, 11008), _spread(rng, 64, 11008)
    tokens = max(1, min(tokens, MOST // (infeat * outfeat)))
    c = dict(op=op, dtype=rng.choice(["bf16", "bf16", "f16"]), tokens=tokens, infeat=infeat, outfeat=outfeat,
             act=rng.choice(["none", "relu", "gelu", "silu"]))
    if op == "linear":
        c["bias"], c["residual"] = rng.random() < 0.5, rng.random() < 0.5
        c["keep"] = rng.choice(["none", "z", "packed"])
    else:
        # The gradient goes where the optimizer reads it: bf16, or 32 bits where nothing is rounded on the way.
        c["grad"] = rng.choice(["f32", "bf16"]) if c["act"] == "none" and tokens <= 4096 else "bf16"
        c["x8"] = rng.random() < 0.5
        c["z8"] = c["act"] != "none" and rng.random() < 0.5
    return c


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _blocks(v):
    """v [tokens, cols] as [tokens, blocks, 32], zeros after the last column."""
    t, n = v.shape
    nb = -(-n // BLOCK)
    p = torch.zeros(t, nb * BLOCK, dtype=v.dtype, device=v.device)
    p[:, :n] = v
    return p.view(t, nb, BLOCK)


def _scale32(byte):
    """2^(byte - 127) in 32 bits."""
    e = byte.to(torch.int32)
    return torch.where(e > 0, e << 23, torch.full_like(e, 1 << 22)).view(torch.float32)


def _pack32(v):
    """Codes and scale bytes of finite v in 32 bits: the smallest power of two that keeps a block within 127."""
    b = _blocks(v)
    bits = b.abs().amax(-1).view(torch.int32)
    byte = ((bits >> 23) - 6 + ((bits & 0x7FFFFF) > 0x7E0000).to(torch.int32)).clamp(min=0)
    inv = ((254 - byte) << 23).view(torch.float32)
    q = torch.round(b * inv[..., None])
    return q.reshape(v.shape[0], -1)[:, :v.shape[1]], byte


def _values32(q, byte):
    """The values that codes and scale bytes stand for."""
    b = _blocks(q.float())
    return (b * _scale32(byte)[..., None]).reshape(q.shape[0], -1)[:, :q.shape[1]]


def _act32(z, act):
    if act == "none":
        return z
    if act == "relu":
        return torch.where(z > 0, z, torch.zeros_like(z))
    u = z if act == "silu" else 1.5957691216057308 * (z + 0.044715 * z * z * z)
    return z / (1 + torch.exp(-u))


def _dact32(z, act):
    if act == "relu":
        return (z > 0).float()
    if act == "silu":
        s = 1 / (1 + torch.exp(-z))
        return s * (1 + z * (1 - s))
    s = 1 / (1 + torch.exp(-1.5957691216057308 * (z + 0.044715 * z * z * z)))
    return s + z * s * (1 - s) * 1.5957691216057308 * (1 + 0.134145 * z * z)


def _plain(c, s):
    e = ELEM[c["dtype"]]
    if c["op"] == "pack":
        return {"values": _values32(*_pack32(s["x"].float())).to(e)}
    if c["op"] == "norm":
        h = s["x"].float()
        out = {}
        if c["residual"]:
            h = h + s["r"].float()
            out["h"] = h.to(e)
        rstd = 1 / torch.sqrt((h * h).mean(-1) + EPS)
        y = h * rstd[:, None] * s["w"].float()
        out["y"], out["rstd"] = y.to(e), rstd
        if c["packed"]:
            out["y8"] = _values32(*_pack32(y)).to(torch.bfloat16)  # a code is exact in bf16
        return out
    if c["op"] == "norm_backward":
        dy, hn = s["dy"].float(), s["h"].float() * s["rstd"][:, None]
        g = dy * s["w"].float()
        dx = s["rstd"][:, None] * (g - hn * (g * hn).mean(-1, keepdim=True))
        if c["stream"]:
            dx = dx + s["dh"].float()
        return {"dx": dx.to(e), "dw": (dy * hn).sum(0)}
    if c["op"] == "linear":
        z = s["x"].float() @ s["w"].float().t()
        if c["bias"]:
            z = z + s["b"]
        y = _act32(z, c["act"])
        if c["residual"]:
            y = y + s["r"].float()
        out = {"y": y.to(e)}
        if c["keep"] == "z":
            out["z"] = z.to(e)
        if c["keep"] == "packed":
            out["z8"], out["y8"] = (_values32(*_pack32(v)).to(torch.bfloat16) for v in (z, y))
        return out
    dz = s["dy"].float()
    if c["act"] != "none":
        z = _values32(*s["z8"]) if c["z8"] else s["z"].float()
        dz = dz * _dact32(z, c["act"])
    x = _values32(*s["x8"]) if c["x8"] else s["x"].float()
    return {"dx": (dz @ s["w"].float()).to(e), "dw": (dz.t() @ x).to(ELEM[c["grad"]]), "db": dz.sum(0)}


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

def _own_setup(c, s):
    """What a training program keeps from call to call: outputs, checkpoints and workspaces."""
    import matrix_orthogonalizing_optimizer_shape_gb300 as d3
    e, dev = ELEM[c["dtype"]], "cuda"
    new = lambda r, n, t=e: torch.empty(r, n, dtype=t, device=dev)  # noqa: E731
    k = {}
    t = c["tokens"]
    if c["op"] == "pack":
        k["p8"], k["values"] = d3.alloc_packed8(t, c["cols"]), new(t, c["cols"])
    elif c["op"] == "norm":
        n = c["cols"]
        k["y"], k["rstd"] = new(t, n), torch.empty(t, dtype=torch.float32, device=dev)
        k["h"] = new(t, n) if c["residual"] else None
        k["p8"] = d3.alloc_packed8(t, n) if c["packed"] else None
        k["y8"] = new(t, n, torch.bfloat16) if c["packed"] else None
    elif c["op"] == "norm_backward":
        n = c["cols"]
        k["dx"], k["dw"] = new(t, n), torch.empty(n, dtype=torch.float32, device=dev)
        k["ws"] = d3.alloc_workspace(d3.rms_norm_backward_workspace_size(t, n))
    elif c["op"] == "linear":
        n = c["outfeat"]
        k["y"] = new(t, n)
        k["z"] = new(t, n) if c["keep"] == "z" else None
        for name in ("z8", "y8"):
            k["p" + name] = d3.alloc_packed8(t, n) if c["keep"] == "packed" else None
            k[name] = new(t, n, torch.bfloat16) if c["keep"] == "packed" else None
        k["act"] = {"none": d3.ACT_NONE, "relu": d3.ACT_RELU, "gelu": d3.ACT_GELU, "silu": d3.ACT_SILU}[c["act"]]
        k["ws"] = d3.alloc_workspace(d3.linear_workspace_size(t, c["infeat"], n, dtype=e))
    else:
        k["x"] = d3.Packed8(*s["x8"]) if c["x8"] else s["x"]
        k["z"] = None if c["act"] == "none" else d3.Packed8(*s["z8"]) if c["z8"] else s["z"]
        k["dx"], k["dw"] = new(t, c["infeat"]), new(c["outfeat"], c["infeat"], ELEM[c["grad"]])
        k["db"] = torch.empty(c["outfeat"], dtype=torch.float32, device=dev)
        k["act"] = {"none": d3.ACT_NONE, "relu": d3.ACT_RELU, "gelu": d3.ACT_GELU, "silu": d3.ACT_SILU}[c["act"]]
        k["ws"] = d3.alloc_workspace(d3.linear_backward_workspace_size(t, c["infeat"], c["outfeat"], dtype=e))
    return k


def _own(c, s):
    import matrix_orthogonalizing_optimizer_shape_gb300 as d3
    k = s["kept"]
    if c["op"] == "pack":
        d3.pack8(s["x"], k["p8"])
        d3.unpack8(k["p8"], k["values"])
        return {"values": k["values"]}
    if c["op"] == "norm":
        d3.rms_norm(s["x"], s["w"], k["y"], residual=s.get("r"), h=k["h"], y8=k["p8"], rstd=k["rstd"], eps=EPS)
        out = {"y": k["y"], "rstd": k["rstd"]}
        if c["residual"]:
            out["h"] = k["h"]
        if c["packed"]:
            d3.unpack8(k["p8"], k["y8"])
            out["y8"] = k["y8"]
        return out
    if c["op"] == "norm_backward":
        d3.rms_norm_backward(s["dy"], s["h"], s["w"], s["rstd"], k["dx"], dh=s.get("dh"), dw=k["dw"], ws=k["ws"])
        return {"dx": k["dx"], "dw": k["dw"]}
    if c["op"] == "linear":
        d3.linear(s["x"], s["w"], k["y"], bias=s.get("b"), residual=s.get("r"), act=k["act"],
                  z=k["pz8"] if c["keep"] == "packed" else k["z"], y8=k["py8"], ws=k["ws"])
        out = {"y": k["y"]}
        if c["keep"] == "z":
            out["z"] = k["z"]
        if c["keep"] == "packed":
            d3.unpack8(k["pz8"], k["z8"])
            d3.unpack8(k["py8"], k["y8"])
            out["z8"], out["y8"] = k["z8"], k["y8"]
        return out
    d3.linear_backward(s["dy"], k["x"], s["w"], dx=k["dx"], dw=k["dw"], db=k["db"], act=k["act"], z=k["z"],
                       ws=k["ws"])
    return {"dx": k["dx"], "dw": k["dw"], "db": k["db"]}


# ---------------------------------------------------------------------------
# Inputs, one pass, its work, and the result in 64 bits
# ---------------------------------------------------------------------------

def prepare(case, seed):
    c = dict(case)
    e, t = ELEM[c["dtype"]], c["tokens"]
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(rows, cols, scale=1.0, outliers=False, dtype=e):
        v = torch.randn(rows, cols, generator=g, device="cuda") * scale
        if outliers:  # a few channels of an activation are much larger than the rest
            v *= 1 + 7 * (torch.rand(cols, generator=g, device="cuda") < 0.01)
        return v.to(dtype)

    def checkpoint(v):
        """8-bit checkpoint of v as it lies in memory: row pitches that are multiples of 16 bytes."""
        q, byte = _pack32(v.float())
        codes = torch.zeros(t, -(-q.shape[1] // 16) * 16, dtype=torch.int8, device="cuda")[:, :q.shape[1]]
        scales = torch.zeros(t, -(-byte.shape[1] // 16) * 16, dtype=torch.uint8, device="cuda")[:, :byte.shape[1]]
        codes.copy_(q)
        scales.copy_(byte)
        return codes, scales

    s = {"case": c}
    if c["op"] == "pack":
        s["x"] = normal(t, c["cols"], outliers=True)
    elif c["op"] == "norm":
        n = c["cols"]
        s["x"], s["w"] = normal(t, n, 0.5), (1 + 0.1 * normal(1, n, dtype=torch.float32))[0].to(e)
        if c["residual"]:
            s["r"] = normal(t, n, outliers=True)
    elif c["op"] == "norm_backward":
        n = c["cols"]
        s["h"], s["w"] = normal(t, n, outliers=True), (1 + 0.1 * normal(1, n, dtype=torch.float32))[0].to(e)
        s["rstd"] = 1 / torch.sqrt((s["h"].float() ** 2).mean(-1) + EPS)
        s["dy"] = normal(t, n, 0.05)
        if c["stream"]:
            s["dh"] = normal(t, n, 0.05)
    elif c["op"] == "linear":
        k, n = c["infeat"], c["outfeat"]
        s["x"], s["w"] = normal(t, k, outliers=True), normal(n, k, 1 / math.sqrt(k))
        if c["bias"]:
            s["b"] = normal(1, n, 0.1, dtype=torch.float32)[0]
        if c["residual"]:
            s["r"] = normal(t, n)
    else:
        k, n = c["infeat"], c["outfeat"]
        s["w"], s["dy"] = normal(n, k, 1 / math.sqrt(k)), normal(t, n, 0.05)
        x = normal(t, k, outliers=True)
        if c["x8"]:
            s["x8"] = checkpoint(x)
        else:
            s["x"] = x
        if c["act"] != "none":
            z = normal(t, n)
            if c["z8"]:
                s["z8"] = checkpoint(z)
            else:
                s["z"] = z
    if own:
        s["kept"] = _own_setup(c, s)
    return s


def run(state):
    return _own(state["case"], state) if own else _plain(state["case"], state)


def work(case):
    c = case
    b, t = BYTES[c["dtype"]], c["tokens"]
    if c["op"] in ("pack", "norm", "norm_backward"):
        n = c["cols"]
        p8 = t * (n + -(-n // BLOCK))  # codes and scale bytes
        if c["op"] == "pack":          # packed, and read back as values
            return {"bytes": 2 * t * n * b + 2 * p8, "flops": 4 * t * n}
        if c["op"] == "norm":
            x = t * n * b * (4 if c["residual"] else 2) + n * b + 4 * t
            return {"bytes": x + (2 * p8 + 2 * t * n if c["packed"] else 0), "flops": 6 * t * n}
        return {"bytes": t * n * b * (4 if c["stream"] else 3) + n * b + 4 * t + 4 * n, "flops": 12 * t * n}
    k, n = c["infeat"], c["outfeat"]
    p8 = lambda w: t * (w + -(-w // BLOCK))  # noqa: E731
    if c["op"] == "linear":
        x = b * (t * k + n * k + t * n) + (4 * n if c["bias"] else 0) + (b * t * n if c["residual"] else 0)
        x += b * t * n if c["keep"] == "z" else 2 * (2 * p8(n) + 2 * t * n) if c["keep"] == "packed" else 0
        return {"bytes": x, "flops": 2 * t * n * k}
    x = b * (t * n + n * k + t * k) + BYTES[c["grad"]] * n * k + 4 * n + (p8(k) if c["x8"] else b * t * k)
    x += 0 if c["act"] == "none" else p8(n) if c["z8"] else b * t * n
    return {"bytes": x, "flops": 4 * t * n * k}


def _two_to(e):
    """2^e in 64 bits, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _exact_values(v):
    """v as 8-bit blocks of 32 columns keep it: whole multiples, at most 127, of the least power of two that allows it."""
    def part(p, width):
        p = p.reshape(p.shape[0], -1, width)
        m, ex = torch.frexp(p.abs().amax(-1, keepdim=True))
        step = _two_to(torch.where(m > 127 / 128, ex - 6, ex - 7).clamp(min=-127))
        return (torch.round(p / step) * step).flatten(1)
    whole = v.shape[1] // 32 * 32
    parts = [part(v[:, :whole], 32)] if whole else []
    return torch.cat(parts + ([part(v[:, whole:], v.shape[1] - whole)] if whole < v.shape[1] else []), 1)


def exact(case, seed):
    """The operator in 64 bits, before its results are rounded to 16 or 8 bits (a checkpoint alone is that rounding)."""
    c, s = dict(case), prepare(case, seed)
    d = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    for k in ("x8", "z8"):
        if k in s:
            codes, byte = s[k]
            step = _two_to(byte.to(torch.int64) - 127).repeat_interleave(32, dim=1)[:, :codes.shape[1]]
            d[k[0]] = codes.double() * step
    if c["op"] == "pack":
        return {"values": _exact_values(d["x"])}
    if c["op"] == "norm":
        h = d["x"] + d["r"] if c["residual"] else d["x"]
        rstd = (h.square().mean(1) + EPS).rsqrt()
        y = torch.einsum("tn,t,n->tn", h, rstd, d["w"])
        return {"y": y, "rstd": rstd, **({"h": h} if c["residual"] else {}), **({"y8": y} if c["packed"] else {})}
    if c["op"] == "norm_backward":
        n = c["cols"]
        a = d["dy"] * d["w"]
        dot = torch.einsum("tn,tn->t", a, d["h"])
        dx = d["rstd"][:, None] * a - (d["rstd"] ** 3 * dot / n)[:, None] * d["h"]
        return {"dx": dx + d["dh"] if c["stream"] else dx, "dw": torch.einsum("tn,tn,t->n", d["dy"], d["h"], d["rstd"])}
    root = math.sqrt(2 / math.pi)
    if c["op"] == "linear":
        z = torch.einsum("tk,nk->tn", d["x"], d["w"])
        if c["bias"]:
            z = z + d["b"]
        y = {"none": lambda: z, "relu": lambda: z.clamp(min=0), "silu": lambda: z * torch.sigmoid(z),
             "gelu": lambda: 0.5 * z * (1 + torch.tanh(root * (z + 0.044715 * z ** 3)))}[c["act"]]()
        if c["residual"]:
            y = y + d["r"]
        return {"y": y, **({"z": z} if c["keep"] == "z" else {}),
                **({"z8": z, "y8": y} if c["keep"] == "packed" else {})}
    dz = d["dy"]
    if c["act"] == "relu":
        dz = dz * (d["z"] > 0)
    elif c["act"] == "silu":
        sg = torch.sigmoid(d["z"])
        dz = dz * (sg + d["z"] * sg * (1 - sg))
    elif c["act"] == "gelu":
        th = torch.tanh(root * (d["z"] + 0.044715 * d["z"] ** 3))
        dz = dz * (0.5 * (1 + th) + 0.5 * d["z"] * (1 - th ** 2) * root * (1 + 3 * 0.044715 * d["z"] ** 2))
    return {"dx": torch.einsum("tn,nk->tk", dz, d["w"]), "dw": torch.einsum("tn,tk->nk", dz, d["x"]), "db": dz.sum(0)}

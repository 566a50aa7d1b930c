"""The operators around a stack of layers as a training program calls them, for timing and comparison.

What a language model trained with the framework's layer operators and its step
needs besides them: the token embedding and its gradient (``embed``,
``embed_grad``), the gated linear recurrence that mixes tokens and its gradient
(``scan``, ``scan_grad``), the log probabilities of given tokens with entropy
and top alternatives and their gradient (``logp``, ``logp_grad``), and the
clipping of all gradients to a global norm (``clip``).  With ``own`` false every
operator runs in its plain form (torch products, sums, exponentials,
comparisons and indexing in 32 bits, rounded once at the end); with ``own`` true
it runs through the framework's entry points.

Sizes: 2048, 4096, 8192 and 11008 are the widths of the framework's 1B- and
7B-shaped workloads; the others are generic.
"""
import math

import torch

own = False

ELEM = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
IGNORED = -100  # a target that is no token


def listed():
    return [
        # A short ragged prompt looked up in a 32-bit table of odd width, handed to 16-bit layers.
        dict(name="embed_f32_777x1001", op="embed", table="f32", dtype="bf16", tokens=777, vocab=50001, cols=1001,
             scale=1.0),
        # The table's gradient at a full training batch: text, whose commonest tokens come thousands of times.
        dict(name="embed_grad_bf16_16384x4096", op="embed_grad", table="bf16", dtype="bf16", tokens=16384,
             vocab=131072, cols=4096, scale=1.0),
        # One new token of each of 64 running sequences, their states carried along.
        dict(name="scan_bf16_64x4096", op="scan", dtype="bf16", tokens=64, channels=4096, sequences=64, states=True),
        # A full training batch of packed sequences.
        dict(name="scan_bf16_16384x4096", op="scan", dtype="bf16", tokens=16384, channels=4096, sequences=5,
             states=False),
        # The gradient of a few ragged sequences at an odd width, with initial and final states.
        dict(name="scan_grad_f16_1000x2047", op="scan_grad", dtype="f16", tokens=1000, channels=2047, sequences=7,
             states=True),
        # The gradient of a full training batch that is one long sequence.
        dict(name="scan_grad_bf16_16384x4096", op="scan_grad", dtype="bf16", tokens=16384, channels=4096,
             sequences=1, states=False),
        # One generated token: its log probability, the entropy and twenty alternatives.
        dict(name="logp_bf16_1x131072", op="logp", dtype="bf16", tokens=1, vocab=131072, entropy=True, top=20,
             scale=1.25, masked=True),
        # A training batch's targets under a large vocabulary.
        dict(name="logp_bf16_8192x131072", op="logp", dtype="bf16", tokens=8192, vocab=131072, entropy=True, top=0,
             scale=1.0, masked=False),
        # Gradient of log probabilities and entropy over an odd vocabulary in 32 bits, some columns masked.
        dict(name="logp_grad_f32_333x32001", op="logp_grad", dtype="f32", tokens=333, vocab=32001, entropy=True,
             scale=1.25, masked=True),
        # Gradient of a training batch's targets.
        dict(name="logp_grad_bf16_8192x131072", op="logp_grad", dtype="bf16", tokens=8192, vocab=131072,
             entropy=False, scale=1.0, masked=False),
        # The gradients of one small layer: matrices and vectors.
        dict(name="clip_bf16_1x128x513", op="clip", dtype="bf16", layers=1, d=128, ffn=513),
        # The gradients of the 1B-shaped set.
        dict(name="clip_bf16_16x2048x8192", op="clip", dtype="bf16", layers=16, d=2048, ffn=8192),
    ]


def _spread(rng, lo, hi):
    """A whole number from lo to hi, spread over its logarithm; every other one rounded to a multiple of 8."""
    v = int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))
    if v > 8 and rng.random() < 0.5:
        v -= v % 8
    return max(lo, min(hi, v))


def draw(rng):
    op = rng.choice(["embed", "embed_grad", "scan", "scan_grad", "logp", "logp_grad", "clip"])
    dtype = rng.choice(["bf16", "bf16", "f16", "f32"])
    if op in ("embed", "embed_grad"):
        cols, vocab = _spread(rng, 64, 8192), _spread(rng, 1000, 131072)
        tokens = min(_spread(rng, 1, 16384), 16384 * 4096 // cols)
        return dict(op=op, table=rng.choice([dtype, "f32"]), dtype=dtype, tokens=tokens,
                    vocab=max(1000, min(vocab, 131072 * 2048 // cols)), cols=cols, scale=rng.choice([1.0, 64.0]))
    if op in ("scan", "scan_grad"):
        channels = _spread(rng, 64, 8192)
        tokens = min(_spread(rng, 1, 16384), 16384 * 2048 // channels)
        return dict(op=op, dtype=dtype, tokens=max(1, tokens), channels=channels,
                    sequences=rng.choice([1, _spread(rng, 1, max(1, tokens))]), states=rng.random() < 0.5)
    if op in ("logp", "logp_grad"):
        vocab = _spread(rng, 1000, 200000)
        c = dict(op=op, dtype=dtype, tokens=max(1, min(_spread(rng, 1, 8192), 8192 * 65536 // vocab)), vocab=vocab,
                 entropy=rng.random() < 0.5, scale=rng.choice([1.0, 1.25]), masked=rng.random() < 0.5)
        if op == "logp":
            c["top"] = rng.choice([0, 1, 5, 20])
        return c
    d = _spread(rng, 64, 2048)
    ffn = _spread(rng, d, 4 * d)
    return dict(op=op, dtype=dtype, layers=max(1, min(_spread(rng, 1, 32), 400_000_000 // (4 * d * d + 3 * d * ffn))),
                d=d, ffn=ffn)


def _shapes(c):
    """The matrices and vectors of a clip case: attention, gate, up and down matrices and two gains a layer."""
    d, f = c["d"], c["ffn"]
    return [(d, d)] * 4 * c["layers"] + [(d, f)] * 2 * c["layers"] + [(f, d)] * c["layers"], [d] * 2 * c["layers"]


# ---------------------------------------------------------------------------
# Plain forms
# ---------------------------------------------------------------------------

def _scan32(a, b):
    """h_t = a_t h_{t-1} + b_t along the rows, by doubling the distance."""
    a, b, k = a.clone(), b.clone(), 1
    while k < a.shape[0]:
        b[k:] += a[k:] * b[:-k]
        a[k:] = a[k:] * a[:-k]
        k *= 2
    return b


def _plain_scan(c, s):
    z, x = s["z"].float(), s["x"].float()
    at, begin, end = s["at"], s["begin"], s["end"]  # non-empty sequences, their first and last rows
    a, na = 1 / (1 + torch.exp(-z)), 1 / (1 + torch.exp(z))
    if c["op"] == "scan":
        b = na * x
        if c["states"]:
            b[begin] += a[begin] * s["first"][at]
        a[begin] = 0
        h = _scan32(a, b)
        out = {"h": h.to(ELEM[c["dtype"]])}
        if c["states"]:
            last = s["first"].clone()
            last[at] = h[end]
            out["last"] = last
        return out
    h, dh = s["h"].float(), s["dh"].float()
    prev = torch.cat([torch.zeros_like(h[:1]), h[:-1]])
    prev[begin] = s["first"][at] if c["states"] else 0
    if c["states"]:
        dh = dh.index_add(0, end, s["dlast"][at])
    down = torch.cat([a[1:], torch.zeros_like(a[:1])])  # what a row's gradient takes from the next row's
    down[end] = 0
    g = _scan32(down.flip(0), dh.flip(0)).flip(0)
    e = ELEM[c["dtype"]]
    out = {"dz": (g * (prev - x) * a * na).to(e), "dx": (g * na).to(e)}
    if c["states"]:
        dfirst = s["dlast"].clone()
        dfirst[at] = a[begin] * g[begin]
        out["dfirst"] = dfirst
    return out


def _order_key(v):
    """Whole numbers in the order of v's values, ties going to the lower column."""
    i = v.float().view(torch.int32).to(torch.int64)
    i = torch.where(i < 0, -(i & 0x7FFFFFFF), i)
    return (i << 32) + (0xFFFFFFFF - torch.arange(v.shape[1], device=v.device))


def _plain_logp(c, s):
    v = s["logits"].float() * c["scale"]
    m = v.amax(1)
    d = v - m[:, None]
    e = torch.exp(d)
    total = e.sum(1)
    logs = torch.log(total)
    there = s["targets"] >= 0
    rows = torch.arange(v.shape[0], device=v.device)
    at = s["targets"].clamp(min=0).long()
    if c["op"] == "logp":
        out = {"logp": torch.where(there, d[rows, at] - logs, 0.0)}
        if c["entropy"]:
            out["entropy"] = logs - torch.where(e > 0, e * d, 0.0).sum(1) / total
        if c["top"]:
            ids = torch.topk(_order_key(s["logits"]), c["top"], dim=1)[1]
            out["top_values"], out["top_ids"] = d.gather(1, ids) - logs[:, None], ids.to(torch.int32)
        return out
    p = e / total[:, None]
    g = torch.where(there, s["dlogp"], 0.0)
    dl = -g[:, None] * p
    dl[rows, at] += g
    if c["entropy"]:
        lp = torch.where(e > 0, d - logs[:, None], 0.0)
        entropy = -(p * lp).sum(1)
        dl -= s["dentropy"][:, None] * p * (lp + entropy[:, None])
    return {"dlogits": (c["scale"] * dl).to(ELEM[c["dtype"]])}


def _plain(c, s):
    if c["op"] in ("scan", "scan_grad"):
        return _plain_scan(c, s)
    if c["op"] in ("logp", "logp_grad"):
        return _plain_logp(c, s)
    if c["op"] == "embed":
        there = (s["ids"] >= 0).float()
        return {"y": (s["table"][s["ids"].clamp(min=0).long()].float() * (there * c["scale"])[:, None])
                .to(ELEM[c["dtype"]])}
    if c["op"] == "embed_grad":
        there = (s["ids"] >= 0).float()
        d = torch.zeros(c["vocab"], c["cols"], device="cuda")
        d.index_add_(0, s["ids"].clamp(min=0).long(), s["dy"].float() * (there * c["scale"])[:, None])
        return {"dtable": d.to(ELEM[c["table"]])}
    norm = torch.stack([g.float().square().sum(dtype=torch.float64) for g in s["grads"]]).sum().sqrt().float()
    coef = (s["max_norm"] / (norm + 1e-6)).clamp(max=1.0)
    # The gradients lie in two pieces of memory, of which `grads` are views.
    return {"matrices": (s["matrices"].float() * coef).to(ELEM[c["dtype"]]), "vectors": s["vectors"] * coef,
            "norm": norm.reshape(1)}


# ---------------------------------------------------------------------------
# The framework's operators
# ---------------------------------------------------------------------------

def _own_setup(c, s):
    """What a training program keeps from call to call: outputs and workspaces."""
    import matrix_orthogonalizing_optimizer_shape_gb300 as d3
    e = ELEM[c["dtype"]]
    new = lambda *n, t=e: torch.empty(*n, dtype=t, device="cuda")  # noqa: E731
    f32 = torch.float32
    k = {}
    if c["op"] == "embed":
        k["y"] = new(c["tokens"], c["cols"])
    elif c["op"] == "embed_grad":
        k["dtable"] = new(c["vocab"], c["cols"], t=ELEM[c["table"]])
        k["ws"] = d3.alloc_workspace(d3.embedding_backward_workspace_size(c["tokens"], c["vocab"], c["cols"]))
    elif c["op"] == "scan":
        k["h"] = new(c["tokens"], c["channels"])
        k["last"] = new(c["sequences"], c["channels"], t=f32) if c["states"] else None
    elif c["op"] == "scan_grad":
        k["dz"], k["dx"] = new(c["tokens"], c["channels"]), new(c["tokens"], c["channels"])
        k["dfirst"] = new(c["sequences"], c["channels"], t=f32) if c["states"] else None
    elif c["op"] == "logp":
        k["logp"] = new(c["tokens"], t=f32)
        k["entropy"] = new(c["tokens"], t=f32) if c["entropy"] else None
        k["top_values"] = new(c["tokens"], c["top"], t=f32) if c["top"] else None
        k["top_ids"] = new(c["tokens"], c["top"], t=torch.int32) if c["top"] else None
    elif c["op"] == "logp_grad":
        k["dlogits"] = new(c["tokens"], c["vocab"])
        # What the forward pass keeps for this one.
        k["stats"] = new(c["tokens"], 3, t=f32)
        d3.log_probs(s["logits"], s["targets"], new(c["tokens"], t=f32), scale=c["scale"], stats=k["stats"])
    else:
        k["matrices"], k["vectors"] = torch.empty_like(s["matrices"]), torch.empty_like(s["vectors"])
        k["out"] = _views(c, k["matrices"], k["vectors"])
        k["norm"] = new(1, t=f32)
        k["ws"] = d3.alloc_workspace(d3.grad_norm_workspace_size())
    return k


def _own(c, s):
    import matrix_orthogonalizing_optimizer_shape_gb300 as d3
    k = s["kept"]
    if c["op"] == "embed":
        d3.embedding(s["ids"], s["table"], k["y"], scale=c["scale"])
        return {"y": k["y"]}
    if c["op"] == "embed_grad":
        d3.embedding_backward(s["dy"], s["ids"], k["dtable"], scale=c["scale"], ws=k["ws"])
        return {"dtable": k["dtable"]}
    if c["op"] == "scan":
        d3.recurrence(s["z"], s["x"], k["h"], offsets=s["offsets"], first=s.get("first"), last=k["last"])
        return {"h": k["h"], **({"last": k["last"]} if c["states"] else {})}
    if c["op"] == "scan_grad":
        d3.recurrence_backward(s["dh"], s["z"], s["x"], s["h"], k["dz"], k["dx"], offsets=s["offsets"],
                               first=s.get("first"), dlast=s.get("dlast"), dfirst=k["dfirst"])
        return {"dz": k["dz"], "dx": k["dx"], **({"dfirst": k["dfirst"]} if c["states"] else {})}
    if c["op"] == "logp":
        d3.log_probs(s["logits"], s["targets"], k["logp"], scale=c["scale"], entropy=k["entropy"],
                     top_values=k["top_values"], top_ids=k["top_ids"])
        return {n: k[n] for n in ("logp", "entropy", "top_values", "top_ids") if k[n] is not None}
    if c["op"] == "logp_grad":
        d3.log_probs_backward(s["logits"], s["targets"], k["stats"], k["dlogits"], dlogp=s["dlogp"],
                              dentropy=s.get("dentropy"), scale=c["scale"])
        return {"dlogits": k["dlogits"]}
    d3.clip_grad_norm(s["grads"], s["max_norm"], k["norm"], out=k["out"], ws=k["ws"])
    return {"matrices": k["matrices"], "vectors": k["vectors"], "norm": k["norm"]}


# ---------------------------------------------------------------------------
# Inputs, one pass, its work, and the result in 64 bits
# ---------------------------------------------------------------------------

def _views(c, matrices, vectors):
    shapes, lens = _shapes(c)
    sizes = [r * n for r, n in shapes]
    return ([v.view(r, n) for v, (r, n) in zip(matrices.split(sizes), shapes)] + list(vectors.split(lens)))


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *n: torch.rand(*n, generator=g, device="cuda")  # noqa: E731
    normal = lambda *n: torch.randn(*n, generator=g, device="cuda")  # noqa: E731
    e = ELEM[c["dtype"]]
    s = {"case": c}
    if c["op"] in ("embed", "embed_grad"):
        # Token frequencies fall off like those of text; one position in 20 is padding.
        u = rand(c["tokens"])
        ids = (torch.exp(u * math.log(c["vocab"])) - 1).long().clamp(max=c["vocab"] - 1)
        s["ids"] = torch.where(rand(c["tokens"]) < 0.05, torch.full_like(ids, -1), ids)
        if c["op"] == "embed":
            s["table"] = (normal(c["vocab"], c["cols"]) * 0.02).to(ELEM[c["table"]])
        else:
            s["dy"] = (normal(c["tokens"], c["cols"]) * 0.05).to(e)
    elif c["op"] in ("scan", "scan_grad"):
        t, n, k = c["tokens"], c["channels"], c["sequences"]
        if k == t:  # one token of each
            offsets = torch.arange(t + 1, dtype=torch.int32, device="cuda")
        else:       # packed, cut anywhere
            cuts = (rand(k - 1) * (t + 1)).long().clamp(max=t).sort()[0]
            offsets = torch.cat([cuts.new_zeros(1), cuts, cuts.new_full((1,), t)]).to(torch.int32)
        s["offsets"] = offsets
        begin, end = offsets[:-1].long(), offsets[1:].long()
        at = torch.nonzero(end > begin)[:, 0]
        s["at"], s["begin"], s["end"] = at, begin[at], end[at] - 1
        # Gates remember over some ten tokens, some channels over hundreds.
        s["z"], s["x"] = (normal(t, n) + 2 + 3 * rand(n)).to(e), normal(t, n).to(e)
        if c["states"]:
            s["first"] = normal(k, n)
        if c["op"] == "scan_grad":
            s["h"], s["dh"] = (0.3 * normal(t, n)).to(e), (0.05 * normal(t, n)).to(e)
            if c["states"]:
                s["dlast"] = 0.05 * normal(k, n)
    elif c["op"] in ("logp", "logp_grad"):
        t, n = c["tokens"], c["vocab"]
        x = 2 * normal(t, n)
        x[torch.arange(t, device="cuda"), (rand(t) * n).long()] += 8  # the model's favourite
        if c["masked"]:  # tokens that may not be generated
            x[:, rand(n) < 0.1] = float("-inf")
        s["logits"] = x.to(e)
        free = s["logits"] > float("-inf")
        targets = (rand(t) * n).long()
        targets = torch.where(free[torch.arange(t, device="cuda"), targets], targets, s["logits"].argmax(1))
        s["targets"] = torch.where(rand(t) < 0.1, torch.full_like(targets, IGNORED), targets)
        if c["op"] == "logp_grad":
            s["dlogp"] = normal(t) / t
            if c["entropy"]:
                s["dentropy"] = 0.01 * normal(t) / t
    else:
        shapes, lens = _shapes(c)
        s["matrices"] = torch.empty(sum(r * n for r, n in shapes), dtype=e, device="cuda")
        for piece in s["matrices"].split(1 << 26):
            piece.copy_(0.01 * torch.randn(piece.shape, generator=g, device="cuda"))
        s["vectors"] = 0.01 * normal(sum(lens))
        s["grads"] = _views(c, s["matrices"], s["vectors"])
        s["max_norm"] = 1.0
    if own:
        s["kept"] = _own_setup(c, s)
    return s


def run(state):
    return _own(state["case"], state) if own else _plain(state["case"], state)


def work(case):
    c = case
    if c["op"] in ("embed", "embed_grad"):
        b, w, t = BYTES[c["dtype"]], BYTES[c["table"]], c["tokens"]
        if c["op"] == "embed":
            return {"bytes": t * c["cols"] * (w + b) + 8 * t, "flops": t * c["cols"]}
        return {"bytes": t * c["cols"] * b + c["vocab"] * c["cols"] * w + 8 * t, "flops": t * c["cols"]}
    if c["op"] in ("scan", "scan_grad"):
        b, n = BYTES[c["dtype"]], c["tokens"] * c["channels"]
        states = 4 * c["sequences"] * c["channels"] if c["states"] else 0
        if c["op"] == "scan":
            return {"bytes": 3 * n * b + 2 * states + 4 * c["sequences"], "flops": 8 * n}
        return {"bytes": 6 * n * b + 3 * states + 4 * c["sequences"], "flops": 14 * n}
    if c["op"] in ("logp", "logp_grad"):
        n, t = c["tokens"] * c["vocab"] * BYTES[c["dtype"]], c["tokens"]
        if c["op"] == "logp":
            return {"bytes": n + (16 + 8 * c["top"]) * t, "flops": 5 * c["tokens"] * c["vocab"]}
        return {"bytes": 2 * n + 28 * t, "flops": 6 * c["tokens"] * c["vocab"]}
    shapes, lens = _shapes(c)
    m, v = sum(r * n for r, n in shapes), sum(lens)
    return {"bytes": 2 * (m * BYTES[c["dtype"]] + 4 * v), "flops": 3 * (m + v)}


def _exact_scan(a, b):
    """h_t = a_t h_{t-1} + b_t: row by row within blocks of rows that are taken side by side, then block by block."""
    t, n = a.shape
    size = max(1, math.isqrt(t))
    blocks = -(-t // size)
    pad = blocks * size - t
    a = torch.cat([a, a.new_ones(pad, n)]).view(blocks, size, n).clone()
    b = torch.cat([b, b.new_zeros(pad, n)]).view(blocks, size, n).clone()
    for i in range(1, size):
        b[:, i].addcmul_(a[:, i], b[:, i - 1])
        a[:, i].mul_(a[:, i - 1])
    for j in range(1, blocks):
        b[j].addcmul_(a[j], b[j - 1, -1:].expand_as(b[j]))
    return b.view(-1, n)[:t]


def exact(case, seed):
    """The operator in 64 bits, before its results are rounded."""
    c, s = dict(case), prepare(case, seed)
    if c["op"] == "embed":
        y = s["table"].double()[s["ids"].clamp(min=0)] * c["scale"]
        return {"y": y.masked_fill((s["ids"] < 0)[:, None], 0.0)}
    if c["op"] == "embed_grad":
        kept = s["ids"] >= 0
        d = torch.zeros(c["vocab"], c["cols"], dtype=torch.float64, device="cuda")
        d.index_put_((s["ids"][kept],), s["dy"][kept].double() * c["scale"], accumulate=True)
        return {"dtable": d}
    if c["op"] in ("scan", "scan_grad"):
        z, x = s["z"].double(), s["x"].double()
        a = torch.sigmoid(z)
        starts = torch.zeros(c["tokens"], dtype=torch.bool, device="cuda")
        starts[s["begin"]] = True
        h0 = torch.zeros_like(z)
        if c["states"]:
            h0[s["begin"]] = s["first"].double()[s["at"]]
        if c["op"] == "scan":
            h = _exact_scan(a.masked_fill(starts[:, None], 0.0), torch.sigmoid(-z) * x + a * h0)
            out = {"h": h}
            if c["states"]:
                out["last"] = s["first"].double().index_copy(0, s["at"], h[s["end"]])
            return out
        prev = torch.where(starts[:, None], h0, s["h"].double().roll(1, 0))
        # The message that a row sends to the one before it: m_t = a_t (dh_t + m_{t+1}).
        ends = torch.zeros(c["tokens"], dtype=torch.bool, device="cuda")
        ends[s["end"]] = True
        into = s["dh"].double()
        if c["states"]:
            into.index_add_(0, s["end"], s["dlast"].double()[s["at"]])
        m = _exact_scan(a.masked_fill(ends[:, None], 0.0).flip(0), (a * into).flip(0)).flip(0)
        g = into + m.roll(-1, 0).masked_fill(ends[:, None], 0.0)
        out = {"dz": g * (prev - x) * a * torch.sigmoid(-z), "dx": g * torch.sigmoid(-z)}
        if c["states"]:
            out["dfirst"] = s["dlast"].double().index_copy(0, s["at"], m[s["begin"]])
        return out
    if c["op"] in ("logp", "logp_grad"):
        out, step = {}, max(1, (1 << 28) // c["vocab"])
        for r in range(0, c["tokens"], step):
            part = _exact_logp(c, {k: v[r:r + step] for k, v in s.items() if isinstance(v, torch.Tensor)})
            for k, v in part.items():
                out.setdefault(k, []).append(v)
        return {k: None if v[0] is None else torch.cat(v) for k, v in out.items()}
    total = sum(float(g.double().square().sum()) for g in s["grads"])
    coef = min(1.0, s["max_norm"] / (math.sqrt(total) + 1e-6))
    return {"matrices": s["matrices"].double() * coef, "vectors": s["vectors"].double() * coef,
            "norm": torch.tensor([math.sqrt(total)], dtype=torch.float64)}


def _exact_logp(c, s):
    lp = torch.log_softmax(s["logits"].double() * c["scale"], 1)
    there = s["targets"] >= 0
    at = s["targets"].clamp(min=0)[:, None]
    p = lp.exp()
    plogp = torch.special.xlogy(p, p)
    if c["op"] == "logp":
        out = {"logp": lp.gather(1, at)[:, 0].masked_fill(~there, 0.0)}
        if c["entropy"]:
            out["entropy"] = -plogp.sum(1)
        if c["top"]:
            out["top_values"], out["top_ids"] = lp.topk(c["top"], 1)[0], None
        return out
    g = (s["dlogp"].double() * there)[:, None]
    d = (torch.zeros_like(p).scatter_(1, at, 1.0) - p) * g
    if c["entropy"]:
        d -= s["dentropy"].double()[:, None] * (plogp - p * plogp.sum(1, keepdim=True))
    return {"dlogits": d * c["scale"]}

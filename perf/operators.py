"""The operators of a training step around the gradient combine, as cases to be measured.

Token embeddings and their gradient, layer norm and its gradient, and activations that are
kept in 8 bits between the forward and the backward pass.  Gradients of parameters come
per worker, in the buffers that the Adasum combine takes: the rows of a call are K workers'
microbatches one after the other, worker k's being [offsets[k], offsets[k+1]).

`run` computes a case with elementary torch operations in 32 bits (`own` false) or through
the package's entry points (`own` true); `exact` computes it in 64 bits from the definition.

Definitions.  Checkpoints: a row of `cols` values is cut into blocks of 128 (the last one
may be shorter); a block with the largest magnitude m holds q = round(x * (127 / m)), ties
to even, and the scale m / 127, and stands for q * scale.  Layer norm: h = (x - mean) * rstd,
rstd = 1 / sqrt(var + eps), y = h * w + b.  Embedding: y = scale * table[token]; a token
outside the table (-1 marks padding) reads zeros and gives no gradient.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
EPS = 1e-5
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}

# The shapes are those of the repository's BERT-Large set (hidden 1024, FFN 4096, vocabulary
# 30522, 16 workers, sequences of 128) and of its GPT-style set (hidden 2048, vocabulary
# 50304, 8 workers), and odd ones.


def listed():
    return [
        # one token each of 8 sequences: what counts is the call's latency
        dict(name="lookup of 8 tokens", op="lookup", rows=8, cols=2048, vocab=50304, type="bf16",
             pad=0.0, scale=1.0, ids="int64"),
        # the microbatches of a whole step; the output is larger than the L2 cache
        dict(name="lookup of a step's tokens", op="lookup", rows=65536, cols=2048, vocab=50304, type="bf16",
             pad=0.0, scale=45.25, ids="int64"),
        # one sequence of 128 added to the gradient that earlier microbatches and the tied
        # output projection left (fp32 accumulation of bf16 activations)
        dict(name="table gradient, 128 added", op="lookup_grad", workers=1, rows=128, cols=1024, vocab=30522,
             type="bf16", grad="fp32", pad=0.1, scale=1.0, add=True, ids="int64"),
        # 16 workers, 32 sequences of 128 each, each worker's whole dense gradient written
        dict(name="table gradient, 16 workers", op="lookup_grad", workers=16, rows=65536, cols=1024, vocab=30522,
             type="bf16", grad="bf16", pad=0.1, scale=1.0, add=False, ids="int64"),
        # a few rows: latency
        dict(name="norm of 8 rows", op="norm", rows=8, cols=1024, type="bf16", weight="bf16"),
        # a step's rows of the GPT-style set, fp32 master weights
        dict(name="norm of a step's rows", op="norm", rows=65536, cols=2048, type="bf16", weight="fp32"),
        # odd sizes, fp32, three workers with unequal rows
        dict(name="norm gradient, odd", op="norm_grad", workers=3, rows=1021, cols=1000, type="fp32",
             weight="fp32", grad="fp32", add=False),
        # 16 workers' rows of the BERT-Large set
        dict(name="norm gradient, 16 workers", op="norm_grad", workers=16, rows=65536, cols=1024, type="bf16",
             weight="bf16", grad="bf16", add=False),
        # an attention output kept in 8 bits and restored for the weight gradient, odd width
        dict(name="8 bits and back, odd", op="keep", rows=513, cols=1000, type="fp32"),
        # the FFN's activation: forward keeping its input in 8 bits, and the backward pass
        # from that, which gives the activation again for the next weight gradient
        dict(name="gelu step from 8 bits", op="keep_gelu", rows=32768, cols=4096, type="bf16", tanh=False, again=True),
        # one sequence of 128: forward keeping h in 8 bits, backward from that
        dict(name="norm step from 8 bits, 128", op="keep_norm", workers=1, rows=128, cols=1024, type="bf16",
             weight="bf16", grad="fp32", add=False, again=False),
        # 8 workers' rows of the GPT-style set
        dict(name="norm step from 8 bits", op="keep_norm", workers=8, rows=65536, cols=2048, type="bf16",
             weight="fp32", grad="bf16", add=False, again=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A usual width, or any odd one."""
    return rng.choice([256, 512, 768, 1024, 1536, 2048, 4096, 8192]) if rng.random() < 0.6 else _log(rng, 65, 5000) | 1


def draw(rng):
    op = rng.choice(["lookup", "lookup_grad", "lookup_grad", "norm", "norm_grad", "norm_grad", "keep", "keep_gelu", "keep_norm"])
    kind, cols = rng.choice(["bf16", "bf16", "fp32"]), _width(rng)
    most = 134_000_000 if kind == "bf16" else 67_000_000  # values of one tensor
    if op in ("lookup", "lookup_grad"):
        cols = min(cols, 4096)
        vocab = _log(rng, 1000, 50304)
        case = dict(op=op, rows=min(_log(rng, 1, 65536), most // cols), cols=cols, vocab=vocab, type=kind,
                    pad=rng.choice([0.0, 0.05, 0.3]), scale=rng.choice([1.0, math.sqrt(cols)]), ids=rng.choice(["int64", "int32"]))
        if op == "lookup_grad":
            grad = rng.choice(["bf16", "fp32"])
            fit = max(1, 1_000_000_000 // (vocab * cols * BYTES[grad]))
            workers = min(rng.choice([1, 1, 3, 8, 16]), fit, case["rows"])
            case.update(workers=workers, grad=grad, add=rng.random() < 0.3, rows=min(case["rows"], 67_000_000 // cols))
        return case
    case = dict(op=op, rows=min(_log(rng, 1, 65536), most // cols), cols=cols, type=kind)
    if op == "keep_norm":
        case.update(type="bf16", rows=min(case["rows"], 67_000_000 // cols))
    if op in ("norm", "norm_grad", "keep_norm"):
        case.update(weight=rng.choice(["bf16", "fp32"]))
    if op in ("norm_grad", "keep_norm"):
        case.update(workers=min(rng.choice([1, 1, 3, 8, 16]), case["rows"]), grad=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.3)
    if op == "keep_gelu":
        case.update(tanh=rng.random() < 0.5)
    if op in ("keep_gelu", "keep_norm"):
        case.update(again=rng.random() < 0.5)
    return case


# ------------------------------------------------------------------------------- inputs


def _offsets(case, seed):
    """K+1 offsets of the workers' rows: equal parts where they divide, else ragged ones."""
    k, rows = case.get("workers", 1), case["rows"]
    if rows % k == 0:
        return [i * (rows // k) for i in range(k + 1)]
    cuts = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, rows + 1, k - 1))
    return [0] + [int(c) for c in cuts] + [rows]


def _activations(rows, cols, gen, kind):
    """Rows of unequal size and mean, with a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= 0.5 + 2 * torch.rand(rows, 1, generator=gen, device=DEV)
    x += 0.3 * torch.randn(rows, 1, generator=gen, device=DEV)
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device=DEV)
    x[:, loud] *= 12.0
    return x.to(TYPES[kind])


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    rows, cols, op = case["rows"], case["cols"], case["op"]
    kind = TYPES[case["type"]]
    s = {"case": case, "offsets": _offsets(case, seed)}

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if op in ("lookup", "lookup_grad"):
        # token frequencies fall off as 1 / rank; ranks are dealt to the ids at random
        vocab = case["vocab"]
        u = torch.rand(rows, generator=gen, device=DEV, dtype=torch.float64)
        rank = (torch.exp(u * math.log(vocab + 1.0)) - 1.0).long().clamp_(0, vocab - 1)
        ids = torch.randperm(vocab, generator=gen, device=DEV)[rank]
        drop = torch.rand(rows, generator=gen, device=DEV) < case["pad"]
        s["ids"] = torch.where(drop, torch.full_like(ids, -1), ids).to(torch.int32 if case["ids"] == "int32" else torch.int64)
    if op == "lookup":
        s["table"] = (0.02 * randn(case["vocab"], cols)).to(kind)
        return s
    if op == "lookup_grad":
        s["dy"] = (1e-3 * randn(rows, cols)).to(kind)
        n = case["vocab"] * cols
        s["flat"] = (1e-3 * randn(case["workers"], n) if case["add"] else torch.zeros(case["workers"], n, device=DEV)).to(TYPES[case["grad"]])
        return s
    s["x"] = _activations(rows, cols, gen, case["type"])
    if "weight" in case:
        s["w"] = (1.0 + 0.1 * randn(cols)).to(TYPES[case["weight"]])
        s["b"] = (0.1 * randn(cols)).to(TYPES[case["weight"]])
    if op in ("norm_grad", "keep_norm", "keep_gelu"):
        s["dy"] = (1e-3 * randn(rows, cols)).to(kind)
    if op == "norm_grad":  # the statistics that the forward pass left
        x = s["x"].float()
        mean = x.mean(1)
        s["mean"], s["rstd"] = mean, torch.rsqrt((x - mean[:, None]).square().mean(1) + EPS)
    if op in ("norm_grad", "keep_norm"):
        k = case["workers"]
        flat = 1e-3 * randn(k, 2 * cols) if case["add"] else torch.zeros(k, 2 * cols, device=DEV)
        s["flat"] = flat.to(TYPES[case["grad"]])
    return s


# ------------------------------------------------------------- the plain forms, in 32 bits


def _by_worker(values, offsets):
    """Sums of the rows of `values` over each worker's rows, K x cols."""
    if len(offsets) == 2:
        return values.sum(0, keepdim=True)
    bounds = torch.tensor(offsets, device=DEV)
    row = torch.arange(values.shape[0], device=DEV)
    mine = (row >= bounds[:-1, None]) & (row < bounds[1:, None])
    return torch.matmul(mine.float(), values)


def _into(flat, new, add):
    """`new` in the type of the gradient buffers, or added to them (rounded once)."""
    if not add:
        return new.to(flat.dtype)
    flat.copy_((flat.float() + new).to(flat.dtype))
    return flat


def _kept(x):
    """The fp32 values that the 8-bit codes of x stand for."""
    rows, cols = x.shape
    blocks = torch.nn.functional.pad(x, (0, -cols % BLOCK)).view(rows, -1, BLOCK)
    top = blocks.abs().amax(2, keepdim=True)
    most = torch.full_like(top, 127.0)  # (a tensor: torch divides by a number, or a number, through reciprocals)
    codes = torch.where(top > 0, torch.round(blocks * (most / top)), torch.zeros_like(blocks))
    return (codes * (top / most)).view(rows, -1)[:, :cols]


def _gelu(x, tanh):
    if tanh:
        return 0.5 * x * (1.0 + torch.tanh(math.sqrt(2.0 / math.pi) * (x + 0.044715 * x * x * x)))
    return 0.5 * x * (1.0 + torch.erf(x * math.sqrt(0.5)))


def _gelu_slope(x, tanh):
    if tanh:
        c = math.sqrt(2.0 / math.pi)
        t = torch.tanh(c * (x + 0.044715 * x * x * x))
        return 0.5 * (1.0 + t) + 0.5 * x * (1.0 - t * t) * c * (1.0 + 3 * 0.044715 * x * x)
    return 0.5 * (1.0 + torch.erf(x * math.sqrt(0.5))) + x * torch.exp(-0.5 * x * x) * (1.0 / math.sqrt(2.0 * math.pi))


def _norm_back(g, h, rstd, w):
    """dx of y = h * w + b."""
    gw = g * w
    return rstd[:, None] * (gw - gw.mean(1, keepdim=True) - h * (gw * h).mean(1, keepdim=True))


def _plain(s):
    c = s["case"]
    op, cols, kind = c["op"], c["cols"], TYPES[c["type"]]
    if op == "lookup":
        ids = s["ids"].long()
        there = (ids >= 0) & (ids < c["vocab"])
        rows = s["table"][torch.where(there, ids, torch.zeros_like(ids))].float() * c["scale"]
        return torch.where(there[:, None], rows, torch.zeros_like(rows)).to(kind)
    if op == "lookup_grad":
        ids, vocab, k = s["ids"].long(), c["vocab"], c["workers"]
        bounds = torch.tensor(s["offsets"], device=DEV)
        worker = torch.bucketize(torch.arange(c["rows"], device=DEV), bounds[1:], right=True)
        there = (ids >= 0) & (ids < vocab)
        total = torch.zeros(k * vocab, cols, device=DEV)
        total.index_add_(0, (worker * vocab + ids)[there], s["dy"][there].float() * c["scale"])
        return list(_into(s["flat"], total.view(k, vocab * cols), c["add"]).unbind(0))
    x = s["x"].float()
    if op == "keep":
        return _kept(x).to(kind)
    if op == "keep_gelu":
        kept = _kept(x)
        out = {"y": _gelu(x, c["tanh"]).to(kind), "dx": (s["dy"].float() * _gelu_slope(kept, c["tanh"])).to(kind)}
        if c["again"]:
            out["again"] = _gelu(kept, c["tanh"]).to(kind)
        return out
    w, b = s["w"].float(), s["b"].float()
    if op == "norm_grad":
        g, h = s["dy"].float(), (x - s["mean"][:, None]) * s["rstd"][:, None]
        both = torch.cat([_by_worker(g * h, s["offsets"]), _by_worker(g, s["offsets"])], 1)
        return {"dx": _norm_back(g, h, s["rstd"], w).to(kind), "flat": _into(s["flat"], both, c["add"])}
    mean = x.mean(1)
    centred = x - mean[:, None]
    rstd = torch.rsqrt(centred.square().mean(1) + EPS)
    h = centred * rstd[:, None]
    y = (h * w + b).to(kind)
    if op == "norm":
        return {"y": y, "mean": mean, "rstd": rstd}
    kept, g = _kept(h), s["dy"].float()
    both = torch.cat([_by_worker(g * kept, s["offsets"]), _by_worker(g, s["offsets"])], 1)
    out = {"y": y, "rstd": rstd, "dx": _norm_back(g, kept, rstd, w).to(kind), "flat": _into(s["flat"], both, c["add"])}
    if c["again"]:
        out["again"] = (kept * w + b).to(kind)
    return out


# ------------------------------------------------------------------- the package's operators


def _own(s):
    import adaptive_gradient_summation_gb300 as ags

    c = s["case"]
    op, cols = c["op"], c["cols"]
    if op == "lookup":
        return ags.embedding(s["table"], s["ids"], scale=c["scale"])
    if op == "lookup_grad":
        return ags.embedding_backward(s["dy"], s["ids"], c["vocab"], scale=c["scale"], worker_offsets=s["offsets"],
                                      grads=list(s["flat"].unbind(0)), accumulate=c["add"])
    if op == "keep":
        return ags.checkpoint_unpack(ags.checkpoint_pack(s["x"]))
    if op == "keep_gelu":
        y, kept = ags.gelu_checkpointed(s["x"], tanh=c["tanh"])
        if c["again"]:
            dx, again = ags.gelu_checkpointed_backward(s["dy"], kept, tanh=c["tanh"], with_output=True)
            return {"y": y, "dx": dx, "again": again}
        return {"y": y, "dx": ags.gelu_checkpointed_backward(s["dy"], kept, tanh=c["tanh"])}
    if op == "norm":
        y, mean, rstd = ags.layer_norm(s["x"], s["w"], s["b"], eps=EPS)
        return {"y": y, "mean": mean, "rstd": rstd}
    dw, db = list(s["flat"][:, :cols].unbind(0)), list(s["flat"][:, cols:].unbind(0))
    if op == "norm_grad":
        dx, _, _ = ags.layer_norm_backward(s["dy"], s["x"], s["mean"], s["rstd"], s["w"], worker_offsets=s["offsets"],
                                           grad_weights=dw, grad_biases=db, accumulate=c["add"])
        return {"dx": dx, "flat": s["flat"]}
    y, kept, rstd = ags.layer_norm_checkpointed(s["x"], s["w"], s["b"], eps=EPS)
    got = ags.layer_norm_checkpointed_backward(s["dy"], kept, rstd, s["w"], s["b"], worker_offsets=s["offsets"],
                                               grad_weights=dw, grad_biases=db, accumulate=c["add"], with_output=c["again"])
    out = {"y": y, "rstd": rstd, "dx": got[0], "flat": s["flat"]}
    if c["again"]:
        out["again"] = got[3]
    return out


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------- work and truth


def work(case):
    """Every input read once and every output written once."""
    rows, cols, op = case["rows"], case["cols"], case["op"]
    e, n = BYTES[case["type"]], rows * cols
    blocks = rows * (-(-cols // BLOCK))
    k = case.get("workers", 1)
    if op in ("lookup", "lookup_grad"):
        # the table's rows that occur, by the frequencies the tokens are drawn with
        r = np.arange(1, case["vocab"] + 1)
        p = np.log1p(1.0 / r) / math.log(case["vocab"] + 1.0)
        used = float(np.sum(1.0 - (1.0 - p) ** (rows * (1.0 - case["pad"]) / k)))
        ids = rows * (4 if case["ids"] == "int32" else 8)
    if op == "lookup":
        return {"bytes": ids + used * cols * e + n * e, "flops": n}
    if op == "lookup_grad":
        g = BYTES[case["grad"]]
        out = 2 * used * k * cols * g if case["add"] else k * case["vocab"] * cols * g
        return {"bytes": ids + n * (1.0 - case["pad"]) * e + out, "flops": 2 * n}
    if op == "keep":
        return {"bytes": 2 * n * e + 2 * (n + 4 * blocks), "flops": 5 * n}
    if op == "keep_gelu":
        return {"bytes": (4 + bool(case["again"])) * n * e + 2 * (n + 4 * blocks), "flops": 40 * n}
    params = 2 * cols * BYTES[case["weight"]]
    if op == "norm":
        return {"bytes": 2 * n * e + 8 * rows + params, "flops": 8 * n}
    grads = 2 * k * cols * BYTES[case["grad"]] * (2 if case["add"] else 1)
    if op == "norm_grad":
        return {"bytes": 3 * n * e + 8 * rows + params // 2 + grads, "flops": 14 * n}
    return {"bytes": (4 + bool(case["again"])) * n * e + 2 * (n + 4 * blocks) + 8 * rows + 2 * params + grads, "flops": 28 * n}


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, cols, k, off = case["op"], case["cols"], case.get("workers", 1), s["offsets"]
    f8 = torch.float64

    def eight(v):  # block by block: the nearest multiple of a 127th of the block's largest
        out = torch.zeros_like(v)
        for at in range(0, cols, BLOCK):
            part = v[:, at:at + BLOCK]
            step = part.abs().max(1, keepdim=True).values / 127
            out[:, at:at + BLOCK] = torch.where(step > 0, torch.round(part / step) * step, torch.zeros_like(part))
        return out

    def phi(v):  # gelu and its slope
        if case["tanh"]:  # x times the logistic function of 2u
            a = 2 * math.sqrt(2 / math.pi)
            q = 1 / (1 + torch.exp(-(a * v + a * 0.044715 * v ** 3)))
            return v * q, q + v * q * (1 - q) * (a + 3 * a * 0.044715 * v ** 2)
        q = 0.5 * torch.special.erfc(-v / math.sqrt(2))
        return v * q, q + v * torch.exp(-v ** 2 / 2) / math.sqrt(2 * math.pi)

    if op == "lookup":
        ok = (s["ids"] >= 0) & (s["ids"] < case["vocab"])
        out = torch.zeros(case["rows"], cols, dtype=f8, device=DEV)
        out[ok] = s["table"].to(f8)[s["ids"][ok].long()] * case["scale"]
        return out
    if op == "lookup_grad":
        outs = []
        for w in range(k):
            ids, dy = s["ids"][off[w]:off[w + 1]].long(), s["dy"][off[w]:off[w + 1]].to(f8)
            ok = (ids >= 0) & (ids < case["vocab"])
            g = torch.zeros(case["vocab"], cols, dtype=f8, device=DEV)
            g.index_put_((ids[ok],), dy[ok] * case["scale"], accumulate=True)
            outs.append(g.view(-1) + (s["flat"][w].to(f8) if case["add"] else 0.0))
        return outs
    x = s["x"].to(f8)
    if op == "keep":
        return eight(x)
    if op == "keep_gelu":
        out = {"y": phi(x)[0]}
        again, slope = phi(eight(x))
        out["dx"] = slope * s["dy"].to(f8)
        if case["again"]:
            out["again"] = again
        return out
    w, b = s["w"].to(f8), s["b"].to(f8)
    if op == "norm_grad":
        mean, r = s["mean"].to(f8)[:, None], s["rstd"].to(f8)[:, None]
    else:
        var, mean = torch.var_mean(x, 1, correction=0, keepdim=True)
        r = 1 / torch.sqrt(var + EPS)
    h = (x - mean) * r
    out = {}
    if op != "norm_grad":
        out["y"], out["rstd"] = w * h + b, r[:, 0]
    if op == "norm":
        out["mean"] = mean[:, 0]
        return out
    g = s["dy"].to(f8)
    if op == "keep_norm":
        h = eight(h)
        if case["again"]:
            out["again"] = w * h + b
    flat = torch.zeros(k, 2 * cols, dtype=f8, device=DEV)
    for i in range(k):
        part = slice(off[i], off[i + 1])
        flat[i, :cols] = torch.einsum("rc,rc->c", g[part], h[part])
        flat[i, cols:] = g[part].sum(0)
    out["flat"] = flat + s["flat"].to(f8) if case["add"] else flat
    dh = g * w
    out["dx"] = r * (dh - dh.sum(1, keepdim=True) / cols - h * (dh * h).sum(1, keepdim=True) / cols)
    return out

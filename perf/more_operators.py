"""More operators of a training step around the gradient combine, as cases to be measured.

Root-mean-square norm with the residual's addition, its gradient and its form that keeps 8
bits between the passes; the learned relative position bias of attention scores by buckets,
with its gradient; and orthogonalised updates: the Newton-Schulz iteration, and the step of
momentum, iteration and weights that follows the combine (as the Muon optimiser does).
Gradients of parameters come per worker, in the buffers that the Adasum combine takes.

`run` computes a case with elementary torch operations in 32 bits (`own` false) or through
the package's entry points (`own` true); `exact` computes it in 64 bits from the definition.

Definitions.
Norm: t = x + residual, rounded to the activations' type; rstd = 1 / sqrt(mean(t^2) + eps);
h = t * rstd; y = h * w.  Its gradient has g = dy * w, dt = d + rstd * (g - h * mean(g h)),
where d is the gradient that reaches t past the norm, and dw = sum of dy * h over a worker's
rows.  8 bits: blocks of 128 columns with the largest magnitude m stand for
round(h * (127 / m)) * (m / 127).
Bias: score (b, h, i, j) gets table[bucket(j - i - offset), h].  With r buckets, n = r / 2 for
each sign where both directions count (the keys ahead take the upper half), else n = r and the
keys ahead take bucket 0; a distance d below e = n / 2 is its own bucket, and beyond it
e + floor((n - e) * ln(d / e) / ln(max_distance / e)), at most n - 1.
Orthogonalised update: X = G / (|G| + eps) (transposed where it has more rows than columns),
then five times A = X X', X <- a X + (b A + c A A) X with (a, b, c) = (3.4445, -4.7750, 2.0315).
Step: v <- mu v + g, X from g + mu v, w <- (1 - lr decay) w - lr sqrt(max(1, rows / cols)) X.
"""
import math

import numpy as np
import torch

own = False

BLOCK = 128
EPS = 1e-6
NS_EPS = 1e-7
COEFFICIENTS = (3.4445, -4.7750, 2.0315)
STEPS = 5
MU, LR, DECAY = 0.95, 0.02, 0.01
DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4}

# The shapes are those of the repository's BERT-Large set (hidden 1024, FFN 4096, 16 workers,
# sequences of 128 and 512) and of its GPT-style set (hidden 2048, 8 workers), and odd ones.


def listed():
    return [
        # one token each of 8 sequences: what counts is the call's latency
        dict(name="norm of 8 rows", op="norm", rows=8, cols=1024, type="bf16", weight="bf16", residual=True),
        # a step's rows of the GPT-style set, fp32 master weights
        dict(name="norm of a step's rows", op="norm", rows=65536, cols=2048, type="bf16", weight="fp32", residual=True),
        # odd sizes, fp32, three workers with unequal rows
        dict(name="norm gradient, odd", op="norm_grad", workers=3, rows=1021, cols=1000, type="fp32", weight="fp32",
             grad="fp32", add=False, residual=True),
        # 8 workers' rows of the GPT-style set: forward keeping h in 8 bits, backward from that
        dict(name="norm step from 8 bits", op="keep_norm", workers=8, rows=65536, cols=2048, type="bf16", weight="fp32",
             grad="bf16", add=False, residual=True, again=True),
        # one new token of 8 sequences against 513 keys
        dict(name="bias of one token", op="bias", batch=8, heads=16, queries=1, keys=513, offset=512, type="fp32",
             table="fp32", buckets=32, distance=128, both=False),
        # a step's attention scores: 64 sequences of 512 with 16 heads
        dict(name="bias of a step's scores", op="bias", batch=64, heads=16, queries=512, keys=512, offset=0, type="bf16",
             table="fp32", buckets=32, distance=128, both=True),
        # a microbatch of 4 sequences of odd length, added to what earlier ones left
        dict(name="bias gradient, odd, added", op="bias_grad", workers=1, batch=4, heads=12, queries=131, keys=131,
             offset=0, type="bf16", grad="fp32", buckets=32, distance=128, both=True, add=True),
        # 16 workers' microbatches of 4 sequences of 512
        dict(name="bias gradient, 16 workers", op="bias_grad", workers=16, batch=64, heads=16, queries=512, keys=512,
             offset=0, type="bf16", grad="bf16", buckets=32, distance=128, both=True, add=False),
        # an odd pair in fp32
        dict(name="orthogonalise two, odd, fp32", op="ortho", batch=2, rows=517, cols=1000, type="fp32"),
        # the updates of the BERT-Large set's FFN matrices of one direction
        dict(name="orthogonalise 24", op="ortho", batch=24, rows=4096, cols=1024, type="bf16"),
        # one layer of a small encoder, hidden 256: latency
        dict(name="step of a small layer", op="step", layers=1, hidden=256, ffn=1024, type="fp32"),
        # the matrices of the BERT-Large set's 24 layers, after the combine
        dict(name="step of 24 layers", op="step", layers=24, hidden=1024, ffn=4096, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _width(rng):
    """A usual width, or any odd one."""
    return rng.choice([256, 512, 768, 1024, 1536, 2048, 4096, 8192]) if rng.random() < 0.6 else _log(rng, 65, 5000) | 1


def draw(rng):
    op = rng.choice(["norm", "norm_grad", "norm_grad", "keep_norm", "bias", "bias", "bias_grad", "bias_grad", "ortho", "ortho", "step", "step"])
    kind = rng.choice(["bf16", "bf16", "fp32"])
    if op in ("norm", "norm_grad", "keep_norm"):
        cols, most = _width(rng), 134_000_000 if kind == "bf16" else 67_000_000  # values of one tensor
        if op != "norm":
            most //= 2
        rows = min(_log(rng, 1, 65536), most // cols)
        case = dict(op=op, rows=rows, cols=cols, type="bf16" if op == "keep_norm" else kind, weight=rng.choice(["bf16", "fp32"]),
                    residual=rng.random() < 0.7)
        if op != "norm":
            case.update(workers=min(rng.choice([1, 1, 3, 8, 16]), rows), grad=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.3)
        if op == "keep_norm":
            # (the weight's gradient in bf16: a value of h next to a tie gets one code or the next by
            # the last bit of its 32, which sums in 32 bits show and have no right answer for)
            case.update(again=rng.random() < 0.5, grad="bf16")
        return case
    if op in ("bias", "bias_grad"):
        heads, batch = rng.choice([1, 8, 12, 16, 20, 32]), _log(rng, 1, 128)
        keys = _log(rng, 1, 2048)
        queries = rng.choice([1, keys, _log(rng, 1, keys)])
        most = 268_000_000 if kind == "bf16" else 134_000_000
        batch = max(1, min(batch, most // (heads * queries * keys)))
        both = rng.random() < 0.6
        case = dict(op=op, batch=batch, heads=heads, queries=queries, keys=keys, offset=keys - queries if rng.random() < 0.7 else 0,
                    type=kind, buckets=rng.choice([8, 16, 32, 32, 64]), distance=rng.choice([64, 128, 128, 100, 300]), both=both)
        if op == "bias":
            case.update(table=rng.choice(["bf16", "fp32"]))
            if rng.random() < 0.3:  # the bias alone, for a caller that adds it
                case.update(batch=0)
        else:
            case.update(workers=min(rng.choice([1, 1, 3, 8, 16]), batch), grad=rng.choice(["bf16", "fp32"]), add=rng.random() < 0.3)
        return case
    if op == "ortho":
        rows, cols = _log(rng, 16, 4096), _log(rng, 16, 4096)
        if rng.random() < 0.5:  # usual sizes
            rows, cols = (max(16, 1 << int(round(math.log2(v)))) for v in (rows, cols))
        m, n = min(rows, cols), max(rows, cols)
        return dict(op=op, batch=max(1, min(_log(rng, 1, 48), 200_000_000_000 // (m * m * (2 * n + m)), 100_000_000 // (m * n))),
                    rows=rows, cols=cols, type=kind)
    hidden = rng.choice([64, 128, 256, 384, 512, 768, 1024, _log(rng, 65, 1023) | 1])
    ffn = 4 * hidden if rng.random() < 0.7 else _log(rng, hidden, 4 * hidden)
    return dict(op=op, layers=min(rng.choice([1, 2, 4, 12]), max(1, 24_000_000 // (hidden * hidden))), hidden=hidden, ffn=ffn, type=kind)


# ------------------------------------------------------------------------------- inputs


def _offsets(count, workers, seed):
    """K+1 offsets of the workers' rows: equal parts where they divide, else ragged ones."""
    if count % workers == 0:
        return [i * (count // workers) for i in range(workers + 1)]
    cuts = np.sort(np.random.RandomState(seed % (1 << 31)).randint(0, count + 1, workers - 1))
    return [0] + [int(c) for c in cuts] + [count]


def _activations(rows, cols, gen, kind):
    """Rows of unequal size, with a few channels far larger than the rest."""
    x = torch.randn(rows, cols, generator=gen, device=DEV)
    x *= 0.5 + 2 * torch.rand(rows, 1, generator=gen, device=DEV)
    loud = torch.randint(0, cols, (max(1, cols // 512),), generator=gen, device=DEV)
    x[:, loud] *= 12.0
    return x.to(TYPES[kind])


def _borders(buckets, distance, both):
    """The smallest distance of every bucket after the first of one direction, in whole numbers:
    (d / e)^p >= (distance / e)^i, without fractions."""
    n = buckets // 2 if both else buckets
    e = n // 2
    p, out = n - e, list(range(1, e + 1))
    for i in range(1, p):
        d = max(e, int(e * (distance / e) ** (i / p)) - 2)
        while d ** p * e ** i < distance ** i * e ** p:
            d += 1
        out.append(d)
    return out


def _slots(case):
    """(start, rows, cols) of a layer's matrices in its slice of the flat vector, and the
    slice's length: four of attention with their bias, a norm's two vectors, the two of the
    FFN with their bias, and a norm's."""
    h, f = case["hidden"], case["ffn"]
    at, found = 0, []
    for rows, cols, after in [(h, h, h)] * 3 + [(h, h, 3 * h), (h, f, f), (f, h, 3 * h)]:
        found.append((at, rows, cols))
        at += rows * cols + after
    return found, at


def _updates(gen, *shape):
    """Matrices of a few strong directions over many weak ones, as gradients have."""
    rows, cols = shape[-2:]
    r = max(1, min(rows, cols) // 16)
    left = torch.randn(*shape[:-1], r, generator=gen, device=DEV) / math.sqrt(r)
    right = torch.randn(*shape[:-2], r, cols, generator=gen, device=DEV)
    return 1e-3 * (torch.matmul(left, right) + 0.5 * torch.randn(*shape, generator=gen, device=DEV))


def prepare(case, seed):
    gen = torch.Generator(device=DEV).manual_seed(int(seed))
    op, kind = case["op"], TYPES[case["type"]]
    s = {"case": case}

    def randn(*shape):
        return torch.randn(*shape, generator=gen, device=DEV)

    if op in ("norm", "norm_grad", "keep_norm"):
        rows, cols = case["rows"], case["cols"]
        s["x"] = _activations(rows, cols, gen, case["type"])
        s["w"] = (1.0 + 0.1 * randn(cols)).to(TYPES[case["weight"]])
        if case["residual"] and op != "norm_grad":
            s["residual"] = (2.0 * randn(rows, cols)).to(kind)
        if op != "norm":
            s["dy"] = (1e-3 * randn(rows, cols)).to(kind)
            if case["residual"]:  # the gradient that reaches the sum past the norm
                s["past"] = (1e-3 * randn(rows, cols)).to(kind)
            s["offsets"] = _offsets(rows, case["workers"], seed)
            flat = 1e-3 * randn(case["workers"], cols) if case["add"] else torch.zeros(case["workers"], cols, device=DEV)
            s["flat"] = flat.to(TYPES[case["grad"]])
        if op == "norm_grad":  # the statistic that the forward pass left
            s["rstd"] = torch.rsqrt(s["x"].float().square().mean(1) + EPS)
        return s
    if op in ("bias", "bias_grad"):
        s["borders"] = torch.tensor(_borders(case["buckets"], case["distance"], case["both"]), device=DEV)
        shape = (case["batch"], case["heads"], case["queries"], case["keys"])
        if op == "bias":
            s["table"] = randn(case["buckets"], case["heads"]).to(TYPES[case["table"]])
            if case["batch"]:
                s["scores"] = (3.0 * randn(*shape)).to(kind)
            return s
        d = randn(*shape)
        d *= 1e-3 * torch.exp(randn(*shape))
        if not case["both"]:  # keys ahead are masked: no gradient comes from them
            d.tril_(case["offset"])
        s["d"] = d.to(kind)
        s["offsets"] = _offsets(case["batch"], case["workers"], seed)
        size = (case["workers"], case["buckets"] * case["heads"])
        s["flat"] = (1e-2 * randn(*size) if case["add"] else torch.zeros(size, device=DEV)).to(TYPES[case["grad"]])
        return s
    if op == "ortho":
        s["x"] = _updates(gen, case["batch"], case["rows"], case["cols"]).to(kind)
        return s
    slots, size = _slots(case)
    n = case["layers"] * size
    s["g"], s["v"] = (1e-3 * randn(n)).to(kind), 5e-3 * randn(n)
    s["w"] = 0.02 * randn(n)
    for at, rows, cols in slots:
        for to, much in (("g", 1.0), ("v", 5.0)):
            part = s[to].view(case["layers"], size)[:, at:at + rows * cols].view(case["layers"], rows, cols)
            part.copy_(much * _updates(gen, case["layers"], rows, cols))
    s["segments"], s["shapes"] = [0], []
    for layer in range(case["layers"]):  # the segments: matrices, and the vectors between them
        for i, (at, rows, cols) in enumerate(slots):
            s["segments"] += [layer * size + at + rows * cols, layer * size + (slots[i + 1][0] if i + 1 < len(slots) else size)]
            s["shapes"] += [(rows, cols), None]
    return s


# ------------------------------------------------------------- the plain forms, in 32 bits


def _by_worker(values, offsets):
    """Sums of the rows of `values` over each worker's rows."""
    if len(offsets) == 2:
        return values.sum(0, keepdim=True)
    bounds = torch.tensor(offsets, device=DEV)
    row = torch.arange(values.shape[0], device=DEV)
    mine = (row >= bounds[:-1, None]) & (row < bounds[1:, None])
    return torch.matmul(mine.float(), values.reshape(values.shape[0], -1)).view(len(offsets) - 1, *values.shape[1:])


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


def _norm_back(s, h, rstd, kind):
    """The gradients of y = h * w."""
    c, dy = s["case"], s["dy"].float()
    g = dy * s["w"].float()
    dt = rstd[:, None] * (g - h * (g * h).mean(1, keepdim=True))
    if "past" in s:
        dt = dt + s["past"].float()
    return {"dx": dt.to(kind), "flat": _into(s["flat"], _by_worker(dy * h, s["offsets"]), c["add"])}


def _bucket(s):
    """Buckets of (query, key)."""
    c = s["case"]
    at = torch.arange(c["keys"], device=DEV)[None, :] - torch.arange(c["queries"], device=DEV)[:, None] - c["offset"]
    if c["both"]:
        return torch.bucketize(at.abs(), s["borders"], right=True) + torch.where(at > 0, c["buckets"] // 2, 0)
    return torch.bucketize((-at).clamp(min=0), s["borders"], right=True)


def _orthogonal(g):
    """A batch of matrices, orthogonalised in their type's precision."""
    x = g if g.shape[1] <= g.shape[2] else g.transpose(1, 2)
    x = x / (x.square().sum((1, 2), keepdim=True).sqrt() + NS_EPS)
    a, b, c = COEFFICIENTS
    for _ in range(STEPS):
        p = torch.matmul(x, x.transpose(1, 2))
        x = a * x + torch.matmul(b * p + c * torch.matmul(p, p), x)
    return x if g.shape[1] <= g.shape[2] else x.transpose(1, 2)


def _plain(s):
    c = s["case"]
    op, kind = c["op"], TYPES[c["type"]]
    if op in ("norm", "keep_norm"):
        t, out = s["x"], {}
        if c["residual"]:
            out["total"] = t = (t.float() + s["residual"].float()).to(kind)
        t = t.float()
        out["rstd"] = rstd = torch.rsqrt(t.square().mean(1) + EPS)
        h = t * rstd[:, None]
        out["y"] = (h * s["w"].float()).to(kind)
        if op == "keep_norm":
            h = _kept(h)
            out.update(_norm_back(s, h, rstd, kind))
            if c["again"]:
                out["again"] = (h * s["w"].float()).to(kind)
        return out
    if op == "norm_grad":
        return _norm_back(s, s["x"].float() * s["rstd"][:, None], s["rstd"], kind)
    if op == "bias":
        bias = s["table"].float()[_bucket(s)].permute(2, 0, 1)
        return (s["scores"].float() + bias).to(kind) if c["batch"] else bias.to(s["table"].dtype).contiguous()
    if op == "bias_grad":
        total = _by_worker(s["d"].float(), s["offsets"]).flatten(2)
        member = (_bucket(s).flatten()[:, None] == torch.arange(c["buckets"], device=DEV)).float()
        return _into(s["flat"], torch.matmul(total, member).transpose(1, 2).flatten(1), c["add"])
    if op == "ortho":
        return _orthogonal(s["x"].float()).to(kind)
    slots, size = _slots(c)
    g, v, w = (s[k].view(c["layers"], size) for k in ("g", "v", "w"))
    for at, rows, cols in slots:
        part = slice(at, at + rows * cols)
        g1 = g[:, part].float()
        v[:, part] = MU * v[:, part] + g1
        o = _orthogonal((g1 + MU * v[:, part]).view(-1, rows, cols))
        w[:, part] = (1.0 - LR * DECAY) * w[:, part] - LR * math.sqrt(max(1.0, rows / cols)) * o.reshape(-1, rows * cols)
    return {"w": s["w"], "v": s["v"]}


# ------------------------------------------------------------------- the package's operators


def _own(s):
    import adaptive_gradient_summation_gb300 as ags

    c = s["case"]
    op = c["op"]
    if op == "norm":
        got = ags.rms_norm(s["x"], s["w"], residual=s.get("residual"), eps=EPS)
        return dict(zip(("y", "total", "rstd") if c["residual"] else ("y", "rstd"), got))
    if op == "norm_grad":
        dx, _ = ags.rms_norm_backward(s["dy"], s["x"], s["rstd"], s["w"], grad_residual=s.get("past"), worker_offsets=s["offsets"],
                                      grad_weights=list(s["flat"].unbind(0)), accumulate=c["add"])
        return {"dx": dx, "flat": s["flat"]}
    if op == "keep_norm":
        got = ags.rms_norm_checkpointed(s["x"], s["w"], residual=s.get("residual"), eps=EPS)
        out = dict(zip(("y", "total", "kept", "rstd") if c["residual"] else ("y", "kept", "rstd"), got))
        back = ags.rms_norm_checkpointed_backward(s["dy"], out.pop("kept"), out["rstd"], s["w"], grad_residual=s.get("past"),
                                                  worker_offsets=s["offsets"], grad_weights=list(s["flat"].unbind(0)),
                                                  accumulate=c["add"], with_output=c["again"])
        out.update(dx=back[0], flat=s["flat"])
        if c["again"]:
            out["again"] = back[2]
        return out
    if op == "bias":
        return ags.relative_position_bias(s["table"], c["queries"], c["keys"], bidirectional=c["both"], max_distance=c["distance"],
                                          offset=c["offset"], scores=s.get("scores"))
    if op == "bias_grad":
        ags.relative_position_bias_backward(s["d"], c["buckets"], bidirectional=c["both"], max_distance=c["distance"],
                                            offset=c["offset"], worker_offsets=s["offsets"], grads=list(s["flat"].unbind(0)),
                                            accumulate=c["add"])
        return s["flat"]
    if op == "ortho":
        return ags.orthogonalize(s["x"], steps=STEPS, coefficients=COEFFICIENTS, eps=NS_EPS)
    ags.muon_step(s["g"], s["segments"], s["shapes"], s["w"], s["v"], lr=LR, mu=MU, weight_decay=DECAY, steps=STEPS,
                  coefficients=COEFFICIENTS, eps=NS_EPS)
    return {"w": s["w"], "v": s["v"]}


def run(state):
    return _own(state) if own else _plain(state)


# -------------------------------------------------------------------------- work and truth


def _products(batch, rows, cols):
    """Operations of the iteration's products, those that give symmetric matrices counted half."""
    m, n = min(rows, cols), max(rows, cols)
    return STEPS * batch * (m * m * n + m * m * m + 2 * m * m * n)


def work(case):
    """Every input read once and every output written once."""
    op, e = case["op"], BYTES[case["type"]]
    if op in ("norm", "norm_grad", "keep_norm"):
        rows, cols, past = case["rows"], case["cols"], bool(case["residual"])
        n, params = rows * cols, cols * BYTES[case["weight"]]
        forward = (2 + 2 * past) * n * e + 4 * rows + params
        if op == "norm":
            return {"bytes": forward, "flops": 5 * n}
        grads = case["workers"] * cols * BYTES[case["grad"]] * (2 if case["add"] else 1)
        codes = n + 4 * rows * (-(-cols // BLOCK))
        if op == "norm_grad":
            return {"bytes": (3 + past) * n * e + 4 * rows + params + grads, "flops": 9 * n}
        return {"bytes": forward + (2 + past + bool(case["again"])) * n * e + 2 * codes + 4 * rows + params + grads, "flops": 20 * n}
    if op in ("bias", "bias_grad"):
        n, table = case["heads"] * case["queries"] * case["keys"], case["buckets"] * case["heads"]
        if op == "bias":
            moved = 2 * case["batch"] * n * e if case["batch"] else n * BYTES[case["table"]]
            return {"bytes": moved + table * BYTES[case["table"]], "flops": max(1, case["batch"]) * n}
        return {"bytes": case["batch"] * n * e + case["workers"] * table * BYTES[case["grad"]] * (2 if case["add"] else 1),
                "flops": case["batch"] * n}
    if op == "ortho":
        n = case["batch"] * case["rows"] * case["cols"]
        return {"bytes": 2 * n * e, "flops": _products(case["batch"], case["rows"], case["cols"])}
    slots = _slots(case)[0]
    n = case["layers"] * sum(rows * cols for _, rows, cols in slots)
    return {"bytes": n * (e + 16), "flops": sum(_products(case["layers"], rows, cols) for _, rows, cols in slots)}


def exact(case, seed):
    """What `run` returns, from the definitions in 64 bits."""
    s = prepare(case, seed)
    op, f8 = case["op"], torch.float64

    def eight(v):  # block by block: the nearest multiple of a 127th of the block's largest
        out = torch.zeros_like(v)
        for at in range(0, v.shape[1], BLOCK):
            part = v[:, at:at + BLOCK]
            step = part.abs().max(1, keepdim=True).values / 127
            out[:, at:at + BLOCK] = torch.where(step > 0, torch.round(part / step) * step, torch.zeros_like(part))
        return out

    if op in ("norm", "norm_grad", "keep_norm"):
        x, w, out = s["x"].to(f8), s["w"].to(f8), {}
        if "residual" in s:  # what follows is of the stored sum
            x = (x + s["residual"].to(f8))
            out["total"] = x
            x = x.to(TYPES[case["type"]]).to(f8)
        r = s["rstd"].to(f8)[:, None] if op == "norm_grad" else 1 / torch.sqrt(torch.einsum("rc,rc->r", x, x)[:, None] / case["cols"] + EPS)
        h = r * x
        if op != "norm_grad":
            out["y"], out["rstd"] = w * h, r[:, 0]
        if op == "norm":
            return out
        dy, off = s["dy"].to(f8), s["offsets"]
        if op == "keep_norm":
            h = eight(h)
            if case["again"]:
                out["again"] = w * h
        flat = s["flat"].to(f8) if case["add"] else torch.zeros(case["workers"], case["cols"], dtype=f8, device=DEV)
        for i in range(case["workers"]):
            flat[i] += torch.einsum("rc,rc->c", dy[off[i]:off[i + 1]], h[off[i]:off[i + 1]])
        along = torch.einsum("rc,c,rc->r", dy, w, h) / case["cols"]
        out["dx"] = r * dy * w - (r[:, 0] * along)[:, None] * h + (s["past"].to(f8) if "past" in s else 0)
        out["flat"] = flat
        return out
    if op in ("bias", "bias_grad"):
        n = case["buckets"] // 2 if case["both"] else case["buckets"]
        e = n // 2
        ahead = torch.arange(case["keys"], device=DEV) - torch.arange(case["queries"], device=DEV)[:, None] - case["offset"]
        d = ahead.abs() if case["both"] else torch.relu(-ahead)
        # (whole values of the logarithms' quotient are rounded away from the floor's edge)
        far = e + torch.floor((n - e) * torch.log(d.clamp(min=1).to(f8) / e) / math.log(case["distance"] / e) + 1e-9).long()
        index = torch.where(d < e, d, far.clamp(max=n - 1))
        if case["both"]:
            index = index + n * (ahead > 0)
        if op == "bias":
            bias = s["table"].to(f8).t()[:, index.flatten()].view(case["heads"], case["queries"], case["keys"])
            if not case["batch"]:
                return bias
            return torch.stack([x.to(f8) + bias for x in s["scores"]]) if s["scores"].numel() < 1 << 26 else s["scores"].to(f8) + bias
        flat, off = s["flat"].to(f8) if case["add"] else torch.zeros(s["flat"].shape, dtype=f8, device=DEV), s["offsets"]
        for i in range(case["workers"]):
            one = torch.zeros(case["heads"], case["queries"], case["keys"], dtype=f8, device=DEV)
            for x in s["d"][off[i]:off[i + 1]]:
                one += x
            for b in range(case["buckets"]):
                flat[i].view(case["buckets"], -1)[b] += one[:, index == b].sum(1)
        return flat
    a, b, c = COEFFICIENTS

    def iterate(u):  # one matrix; the quintic as nested products
        x = u if u.shape[0] <= u.shape[1] else u.t()
        x = x / (torch.linalg.vector_norm(x) + NS_EPS)
        for _ in range(STEPS):
            p = x @ x.t()
            x = p @ (b * x + c * (p @ x)) + a * x
        return x if u.shape[0] <= u.shape[1] else x.t()

    if op == "ortho":
        return torch.stack([iterate(u.to(f8)) for u in s["x"]])
    slots, size = _slots(case)
    w, v = s["w"].to(f8), s["v"].to(f8)
    for layer in range(case["layers"]):
        for at, rows, cols in slots:
            part = slice(layer * size + at, layer * size + at + rows * cols)
            v[part] = MU * v[part] + s["g"][part].to(f8)
            o = iterate((s["g"][part].to(f8) + MU * v[part]).view(rows, cols))
            w[part] = w[part] - LR * (DECAY * w[part] + math.sqrt(max(1.0, rows / cols)) * o.reshape(-1))
    return {"w": w, "v": v}

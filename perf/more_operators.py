"""Cases and plain forms of the operators that answer with several hypotheses and with
adapters.

Three operators join the output head: the choice of a beam search's next hypotheses from
the logits of all beams, the reordering of the beams' states (caches, token histories)
after it, and the low-rank adapters of many requests at once beside a shared classifier.
Each is given here in its plain form, from elementary torch operations, beside the call
of this package that computes the same.

    own = False   run() computes the plain form
    own = True    run() calls vocabulary_cross_entropy_gb300
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
END = 2  # the token that ends a hypothesis


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one request, four hypotheses: the latency of a step
        {"name": "beam 1x4x128256", "op": "beam", "batch": 1, "beams": 4, "vocab": 128256, "dtype": "bf16",
         "count": 4, "ended": 0.0, "masked": 0.0, "penalty": 0.0, "keep": False},
        # a serving batch in mid-search: some hypotheses have ended, some tokens are not allowed;
        # hypotheses stay at their places, so that the caches move as little as possible
        {"name": "beam 64x8x128256 kept", "op": "beam", "batch": 64, "beams": 8, "vocab": 128256, "dtype": "bf16",
         "count": 8, "ended": 0.15, "masked": 0.1, "penalty": 0.8, "keep": True},
        # twice as many candidates as beams, as a search wants that sets ended ones aside; FP32
        # logits of a ragged vocabulary
        {"name": "beam 128x5x50257 f32 pairs", "op": "beam", "batch": 128, "beams": 5, "vocab": 50257,
         "dtype": "f32", "count": 10, "ended": 0.0, "masked": 0.0, "penalty": 0.0, "keep": False},
        # one request's caches of a small model after a few tokens
        {"name": "reorder 1x4 short", "op": "reorder", "batch": 1, "beams": 4, "layout": "heads", "heads": 8,
         "positions": 512, "dim": 64, "dtype": "bf16", "tensors": 12, "history": True, "lengths": True, "inplace": True,
         "moved": 2},
        # a serving batch's caches, half of the beams replaced, in place
        {"name": "reorder 32x8 in place", "op": "reorder", "batch": 32, "beams": 8, "layout": "heads", "heads": 8,
         "positions": 1024, "dim": 128, "dtype": "bf16", "tensors": 8, "history": False, "lengths": True, "inplace": True,
         "moved": 4},
        # ragged sizes, FP32, positions before heads, into a second set of buffers
        {"name": "reorder 24x5 ragged", "op": "reorder", "batch": 24, "beams": 5, "layout": "positions", "heads": 3,
         "positions": 777, "dim": 36, "dtype": "f32", "tensors": 5, "history": True, "lengths": False,
         "inplace": False, "moved": 4},
        # one request's token through its adapter: latency, logits in FP32 as the sampler takes them
        {"name": "adapters 1x4096x128256 r16", "op": "adapters", "rows": 1, "hidden": 4096, "vocab": 128256,
         "rank": 16, "adapters": 8, "none": 0.0, "x": "bf16", "y": "f32"},
        # a decoding batch of many requests, nearly each with an adapter of its own
        {"name": "adapters 64x4096x128256 r16", "op": "adapters", "rows": 64, "hidden": 4096, "vocab": 128256,
         "rank": 16, "adapters": 48, "none": 0.1, "x": "bf16", "y": "f32"},
        # whole prompts are scored: many tokens to an adapter, a larger rank
        {"name": "adapters 2048x4096x128256 r64", "op": "adapters", "rows": 2048, "hidden": 4096, "vocab": 128256,
         "rank": 64, "adapters": 6, "none": 0.1, "x": "bf16", "y": "bf16"},
        # ragged sizes, FP32 hidden states
        {"name": "adapters 257x2056x32001 r8", "op": "adapters", "rows": 257, "hidden": 2056, "vocab": 32001,
         "rank": 8, "adapters": 20, "none": 0.2, "x": "f32", "y": "bf16"},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["beam", "reorder", "adapters"])
    if op == "beam":
        vocab, beams = _spread(rng, 1000, 256000), _spread(rng, 1, 16)
        batch = _spread(rng, 1, min(256, max(1, 60000000 // (vocab * beams))))
        twice = rng.random() < 0.4
        return {"op": op, "batch": batch, "beams": beams, "vocab": vocab, "dtype": rng.choice(["bf16", "f32"]),
                "count": 2 * beams if twice else beams, "ended": rng.choice([0.0, round(rng.uniform(0.05, 0.5), 3)]),
                "masked": rng.choice([0.0, round(rng.uniform(0.01, 0.9), 3)]),
                "penalty": rng.choice([0.0, round(rng.uniform(0.4, 1.2), 3)]),
                "keep": not twice and rng.random() < 0.5}
    if op == "reorder":
        beams, dim = rng.randint(2, 16), rng.choice([32, 36, 64, 80, 96, 128, 256])
        heads, positions = _spread(rng, 1, 32), _spread(rng, 1, 8192)
        dtype = rng.choice(["bf16", "f32"])
        row = heads * positions * dim * (2 if dtype == "bf16" else 4)
        tensors = rng.randint(1, 24)
        batch = _spread(rng, 1, max(1, min(128, 1000000000 // (row * beams * tensors))))
        tensors = max(1, min(tensors, 1000000000 // (row * beams * batch)))
        return {"op": op, "batch": batch, "beams": beams, "layout": rng.choice(["heads", "positions"]), "heads": heads,
                "positions": positions, "dim": dim, "dtype": dtype, "tensors": tensors, "history": rng.random() < 0.5,
                **rng.choice([{"lengths": True, "inplace": True}, {"lengths": False, "inplace": True},
                              {"lengths": False, "inplace": False}]),
                "moved": rng.randint(1, beams - 1)}
    hidden, rank = 8 * _spread(rng, 8, 1024), 8 * _spread(rng, 1, 16)
    vocab, count = _spread(rng, 1000, 202048), _spread(rng, 1, 64)
    count = max(1, min(count, 1000000000 // (rank * vocab)))
    most = min(2048, 200000000 // vocab, max(1, 80000000000 // (vocab * rank * count)))
    return {"op": op, "rows": _spread(rng, 1, most), "hidden": hidden, "vocab": vocab, "rank": rank, "adapters": count,
            "none": rng.choice([0.0, 0.3]), "x": rng.choice(["bf16", "f32"]), "y": rng.choice(["bf16", "f32"])}


def _size(dtype):
    return 2 if dtype == "bf16" else 4


def work(case):
    if case["op"] == "beam":  # each row that goes on is read once
        rows = case["batch"] * case["beams"]
        going = rows - int(rows * case["ended"])
        return {"bytes": going * case["vocab"] * _size(case["dtype"]) + rows * 16 + case["batch"] * case["count"] * 28,
                "flops": 6.0 * going * case["vocab"]}
    if case["op"] == "reorder":
        b, k, m, t = case["batch"], case["beams"], case["moved"], case["positions"]
        places = sum(_lengths(case)) if case["lengths"] else b * t
        each = case["heads"] * case["dim"] * _size(case["dtype"]) * case["tensors"] + 8 * case["history"]
        # in place: the replaced beams are written, and as many others read, if there are as many
        return {"bytes": places * each * ((m + min(m, k - m)) if case["inplace"] else 2 * k), "flops": 0}
    n, h, v, r = case["rows"], case["hidden"], case["vocab"], case["rank"]
    using = n - int(n * case["none"])
    used = min(case["adapters"], using)
    return {"bytes": n * h * _size(case["x"]) + used * r * (h + v) * 2 + 2 * n * v * _size(case["y"]) + 4 * n,
            "flops": 2.0 * using * r * (h + v)}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lengths(case):
    """How many positions each request has filled: from none to all, evenly (one request: a quarter)."""
    b, t = case["batch"], case["positions"]
    return [t // 4] if b == 1 else [t * i // (b - 1) for i in range(b)]


def _some(g, n, share):
    """Truth values [n], int(n * share) of them true."""
    flags = torch.zeros(n, dtype=torch.bool, device="cuda")
    flags[torch.randperm(n, device="cuda", generator=g)[:int(n * share)]] = True
    return flags


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    s = {"case": case}
    if case["op"] == "beam":
        b, k, v = case["batch"], case["beams"], case["vocab"]
        # a bulk of unlikely tokens and a sparse set of likely ones, as a language model's logits have
        z = 2.0 * torch.randn(b * k, v, device="cuda", generator=g)
        z += 8.0 * torch.rand(b * k, v, device="cuda", generator=g) * (
            torch.rand(b * k, v, device="cuda", generator=g) < 3e-4)
        if case["masked"]:
            z.masked_fill_(torch.rand(b * k, v, device="cuda", generator=g) < case["masked"], -math.inf)
        s["logits"] = z.to(DTYPES[case["dtype"]])
        score = -20.0 + 3.0 * torch.randn(b, k, device="cuda", generator=g)
        if b > 1 and k > 1:
            score[b // 2, 1:] = -math.inf  # a request's first step: one hypothesis
            s["logits"][0, :] = -math.inf  # a grammar that allows no token
        s["score"] = score
        s["ended"] = _some(g, b * k, case["ended"]).view(b, k)
        s["length"] = torch.randint(1, 200, (b, k), device="cuda", generator=g, dtype=torch.int32)
    elif case["op"] == "reorder":
        b, k, t, h, d = case["batch"], case["beams"], case["positions"], case["heads"], case["dim"]
        shape = (b * k, h, t, d) if case["layout"] == "heads" else (b * k, t, h, d)
        # (one call of the generator for all of them: preparing many small caches stays quick)
        every = torch.empty(case["tensors"], *shape, dtype=DTYPES[case["dtype"]], device="cuda")
        for part in every:
            part.normal_(generator=g)
        s["states"] = list(every.unbind(0))
        s["dims"] = [2 if case["layout"] == "heads" else 1] * case["tensors"]
        if case["history"]:
            s["states"].append(torch.randint(0, 1 << 40, (b * k, t), device="cuda", generator=g))
            s["dims"].append(1)
        s["out"] = None if case["inplace"] else [torch.zeros_like(x) for x in s["states"]]
        order = torch.rand(b, k, device="cuda", generator=g).argsort(1)
        if case["inplace"]:  # the beams that stay are at their places, the others become copies of some of those
            stay = k - case["moved"]
            parent = torch.arange(k, device="cuda").repeat(b, 1)
            pick = torch.randint(0, stay, (b, k), device="cuda", generator=g)
            parent.scatter_(1, order[:, stay:], order.gather(1, pick)[:, stay:])
        else:
            parent = torch.randint(0, k, (b, k), device="cuda", generator=g)
        s["parent"] = parent
        s["lengths"] = None
        if case["lengths"]:
            filled = torch.tensor(_lengths(case), dtype=torch.int32, device="cuda")
            s["lengths"] = filled[torch.randperm(b, device="cuda", generator=g)]
    else:
        n, h, v, r, c = case["rows"], case["hidden"], case["vocab"], case["rank"], case["adapters"]
        s["x"] = torch.randn(n, h, device="cuda", generator=g).to(DTYPES[case["x"]])
        s["a"] = (torch.randn(c, r, h, device="cuda", generator=g) * h ** -0.5).to(torch.bfloat16)
        s["b"] = torch.empty(c, v, r, dtype=torch.bfloat16, device="cuda").normal_(std=r ** -0.5, generator=g)
        s["y"] = torch.empty(n, v, dtype=DTYPES[case["y"]], device="cuda").normal_(std=2.0, generator=g)
        s["scale"] = 0.25 + torch.rand(c, device="cuda", generator=g)
        index = torch.randint(0, c, (n,), device="cuda", generator=g, dtype=torch.int32)
        s["index"] = torch.where(_some(g, n, case["none"]), torch.full_like(index, -1), index)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_beam(logits, score, ended, length, count, penalty, keep):
    """The next ``count`` hypotheses of every request: token, parent, score, ended, length.

    A hypothesis that goes on offers every token, with its score plus the token's logarithm of
    the softmax; one that has ended offers itself.  The best by score / length^penalty are
    taken, lowest (beam, token) first among equal ones; with ``keep`` the first child of each
    beam takes its parent's place.  In 64 bits: each choice compares sums with one another
    that come from different rows.
    """
    b, k = score.shape
    v = logits.shape[1]
    z = logits.view(b, k, v).double()
    top = z.amax(2, keepdim=True)
    fine = torch.isfinite(top) & torch.isfinite(score)[:, :, None]
    zm = z - torch.where(fine, top, torch.zeros_like(top))
    logp = zm - torch.log(torch.exp(zm).sum(2, keepdim=True))
    c = torch.where(fine, score.double()[:, :, None] + logp, torch.full_like(logp, -math.inf))
    c = torch.where(ended[:, :, None], torch.full_like(c, -math.inf), c)
    c[:, :, END] = torch.where(ended, score.double(), c[:, :, END])
    after = length + (~ended).to(torch.int32)
    value = c / after.clamp(min=1).double().pow(penalty)[:, :, None] if penalty else c
    best, at = torch.sort(value.reshape(b, k * v), dim=1, descending=True, stable=True)
    best, at = best[:, :count], at[:, :count]
    valid = best > -math.inf
    place = torch.arange(count, device=score.device)[None, :] % k
    parent = torch.where(valid, at // v, place)
    if keep:
        # the first child of a parent goes to the parent's place, the others to the free places in order
        first = (parent[:, :, None] == parent[:, None, :]).long().tril(-1).sum(2) == 0
        first = first & valid
        taken = torch.zeros(b, k, dtype=torch.long, device=score.device)
        taken.scatter_add_(1, parent, first.long())
        free = torch.argsort(taken, dim=1, stable=True)  # free places in order, then the others
        nth = torch.cumsum((~first).long(), 1) - 1
        goes = torch.where(first, parent, free.gather(1, nth.clamp(min=0)))
        order = torch.argsort(goes, dim=1)
        at, valid, parent = at.gather(1, order), valid.gather(1, order), parent.gather(1, order)
        parent = torch.where(valid, parent, place)
    token = torch.where(valid, at % v, torch.full_like(at, -1))
    new = torch.where(valid, c.reshape(b, k * v).gather(1, at), torch.full_like(best, -math.inf))
    was = ended.gather(1, parent)
    return (token, parent, new.float(), valid & (was | (token == END)),
            length.gather(1, parent) + (valid & ~was).to(torch.int32))


def _plain_reorder(states, dims, parent, lengths, out):
    b, k = parent.shape
    rows = (torch.arange(b, device=parent.device)[:, None] * k + parent).view(-1)
    res = []
    for i, (x, dim) in enumerate(zip(states, dims)):
        y = torch.index_select(x, 0, rows)
        if lengths is not None:
            shape = [1] * x.dim()
            shape[0], shape[dim] = b * k, x.shape[dim]
            filled = torch.arange(x.shape[dim], device=x.device)[None, :] < lengths.repeat_interleave(k)[:, None]
            y = torch.where(filled.view(shape), y, x)
        res.append((x if out is None else out[i]).copy_(y))
    return res


def _plain_adapters(x, a, b, y, scale, index):
    n, (c, r, h), v = x.shape[0], a.shape, b.shape[1]
    t = (x.float() @ a.view(c * r, h).float().t()).view(n, c, r)
    mine = (index[:, None] == torch.arange(c, device=x.device)[None, :]).float() * scale
    t = (t * mine[:, :, None]).view(n, c * r)
    return (y.float() + t @ b.transpose(1, 2).reshape(c * r, v).float()).to(y.dtype)


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case, s = state["case"], state
    if own:
        import vocabulary_cross_entropy_gb300 as vce
        if case["op"] == "beam":
            r = vce.ce_beam(s["logits"], s["score"], ended=s["ended"], length=s["length"], end=END,
                            length_penalty=case["penalty"], count=case["count"], keep_places=case["keep"])
            return r.token, r.parent, r.score, r.ended, r.length
        if case["op"] == "reorder":
            return vce.beam_reorder(s["states"], s["parent"], lengths=s["lengths"], position_dim=s["dims"], out=s["out"])
        return vce.adapter_linear(s["y"], s["x"], s["a"], s["b"], s["index"], s["scale"])
    if case["op"] == "beam":
        return _plain_beam(s["logits"], s["score"], s["ended"], s["length"], case["count"], case["penalty"], case["keep"])
    if case["op"] == "reorder":
        return _plain_reorder(s["states"], s["dims"], s["parent"], s["lengths"], s["out"])
    return _plain_adapters(s["x"], s["a"], s["b"], s["y"], s["scale"], s["index"])


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_beam(s):
    """Request by request: the scores of its candidates, the best of them, and where they go."""
    case = s["case"]
    b, k = s["score"].shape
    count, p = case["count"], case["penalty"]
    score, ended, length = s["score"].double().tolist(), s["ended"].tolist(), s["length"].tolist()
    out = torch.full((b, count), -math.inf, dtype=torch.float64)
    for i in range(b):
        found = []  # (value, score, beam, token)
        for j in range(k):
            if not math.isfinite(score[i][j]):
                continue
            if ended[i][j]:
                found.append((score[i][j] / length[i][j] ** p, score[i][j], j, END))
                continue
            z = s["logits"][i * k + j].double()
            m = float(z.max())
            if not math.isfinite(m):
                continue
            z = z - m
            lse = float(torch.log(torch.exp(z).sum()))
            # the best of this row; among equal logits any will do, their scores are equal
            best, token = torch.topk(z, min(count, z.numel()))
            found += [((score[i][j] + q - lse) / (length[i][j] + 1) ** p, score[i][j] + q - lse, j, t)
                      for q, t in zip(best.tolist(), token.tolist()) if q > -math.inf]
        found = sorted(found, key=lambda f: (-f[0], f[2]))[:count]
        if case["keep"]:
            places, rest = {}, []
            for f in found:
                if f[2] in places:
                    rest.append(f)
                else:
                    places[f[2]] = f
            for j in range(count):
                if j not in places and rest:
                    places[j] = rest.pop(0)
        else:
            places = dict(enumerate(found))
        for j, f in places.items():
            out[i, j] = f[1]
    return [None, None, out, None, None]


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "beam":
        return _exact_beam(s)
    if case["op"] == "reorder":
        if sum(x.numel() for x in s["states"]) > 100000000:
            return None
        res = []
        for x, dim, into in zip(s["states"], s["dims"], s["out"] or s["states"]):
            if not x.is_floating_point():
                res.append(None)
                continue
            y = (x if s["out"] is None else into).double()
            k = case["beams"]
            for i, row in enumerate(s["parent"].tolist()):
                filled = x.shape[dim] if s["lengths"] is None else int(s["lengths"][i])
                for j, p in enumerate(row):
                    y[i * k + j].narrow(dim - 1, 0, filled).copy_(x[i * k + p].narrow(dim - 1, 0, filled))
            res.append(y)
        return res
    y = s["y"].double()
    for i in range(case["adapters"]):
        rows = torch.nonzero(s["index"] == i)[:, 0]
        if rows.numel():
            t = s["x"][rows].double() @ s["a"][i].double().t()
            y[rows] += float(s["scale"][i]) * (t @ s["b"][i].double().t())
    return y

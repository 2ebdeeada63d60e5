"""Cases and plain forms of the output head's operators.

Four operators sit around the vocabulary cross entropy: the residual addition and
root-mean-square norm before the classifier (forward, 8-bit output, backward), the
microscaled quantisation of hidden states and classifiers, the product of the two
quantised matrices, and the sampling of a token from a row of logits.  Each is
given here in its plain form, from elementary torch operations, beside the call of
this package that computes the same.

    own = False   run() computes the plain form
    own = True    run() calls vocabulary_cross_entropy_gb300

Microscaled tensors hold one power-of-two scale (E8M0, biased by 127) per 32
consecutive columns.  Codes are padded with zeros to a multiple of 128 columns
(E4M3: one byte a value; E2M1: two values a byte, the even column in the low
nibble).  Scales are kept in tiles of 128 rows x 4 blocks, 512 bytes each: the
scale of (row, block) is at tile [row // 128, block // 4], byte
(row % 32) * 16 + (row % 128) // 32 * 4 + block % 4; places outside the matrix are 0.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
E2M1_VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # one sequence's next token: latency of a single row, the usual filters
        {"name": "sample 1x128256 top-k", "op": "sample", "rows": 1, "vocab": 128256, "dtype": "bf16",
         "mode": "topk", "masked": 0.0},
        # a serving batch whose requests each bring their own parameters, some grammar-masked
        {"name": "sample 256x128256 mixed", "op": "sample", "rows": 256, "vocab": 128256, "dtype": "bf16",
         "mode": "mixed", "masked": 0.1},
        # rollouts for training: many rows of a ragged vocabulary, the whole distribution, FP32 logits
        {"name": "sample 1024x50257 unfiltered", "op": "sample", "rows": 1024, "vocab": 50257, "dtype": "f32",
         "mode": "plain", "masked": 0.0},
        # decoding step: one token's final norm, 8-bit output for the quantised classifier
        {"name": "norm 8x4096 to 8 bits", "op": "norm_mx", "rows": 8, "hidden": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True},
        # training step of the linear form's headline width
        {"name": "norm 16384x4096", "op": "norm", "rows": 16384, "hidden": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True},
        # its backward pass
        {"name": "norm backward 16384x4096", "op": "norm_bwd", "rows": 16384, "hidden": 4096, "dtype": "bf16",
         "weight": "bf16", "residual": True},
        # a small FP32 model's backward, odd sizes
        {"name": "norm backward 515x1030 f32", "op": "norm_bwd", "rows": 515, "hidden": 1030, "dtype": "f32",
         "weight": "f32", "residual": False},
        # a classifier quantised when it is loaded
        {"name": "quantise 128256x4096 e2m1", "op": "quantize", "rows": 128256, "cols": 4096, "dtype": "bf16",
         "fmt": "e2m1"},
        # a ragged batch of FP32 hidden states to 8 bits
        {"name": "quantise 301x2056 e4m3", "op": "quantize", "rows": 301, "cols": 2056, "dtype": "f32",
         "fmt": "e4m3"},
        # logits of a decoding batch: the classifier is read once for 8 tokens
        {"name": "product 8x4096x128256", "op": "linear", "rows": 8, "hidden": 4096, "vocab": 128256},
        # a ragged classifier and batch
        {"name": "product 257x2056x32001", "op": "linear", "rows": 257, "hidden": 2056, "vocab": 32001},
        # scoring of whole prompts
        {"name": "product 2048x4096x128256", "op": "linear", "rows": 2048, "hidden": 4096, "vocab": 128256},
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["sample", "sample", "norm", "norm_mx", "norm_bwd", "quantize", "linear", "linear"])
    if op == "sample":
        vocab = _spread(rng, 1000, 256000)
        rows = _spread(rng, 1, min(2048, max(1, 32000000 // vocab)))
        return {"op": op, "rows": rows, "vocab": vocab, "dtype": rng.choice(["bf16", "f32"]),
                "mode": rng.choice(["topk", "nucleus", "minp", "plain", "mixed"]),
                "masked": rng.choice([0.0, round(rng.uniform(0.01, 0.9), 3)])}
    if op in ("norm", "norm_mx", "norm_bwd"):
        hidden = _spread(rng, 64, 16384)
        rows = _spread(rng, 1, min(16384, 64000000 // hidden))
        dtype = rng.choice(["bf16", "f32"])
        return {"op": op, "rows": rows, "hidden": hidden, "dtype": dtype,
                "weight": rng.choice([dtype, "f32"]), "residual": rng.random() < 0.7}
    if op == "quantize":
        cols = _spread(rng, 32, 16384)
        rows = _spread(rng, 1, min(131072, 200000000 // cols))
        return {"op": op, "rows": rows, "cols": cols, "dtype": rng.choice(["bf16", "f32"]),
                "fmt": rng.choice(["e2m1", "e4m3"])}
    hidden = _spread(rng, 64, 8192)
    vocab = _spread(rng, 1000, min(202048, 500000000 // hidden))
    rows = _spread(rng, 1, 2048)
    return {"op": op, "rows": rows, "hidden": hidden, "vocab": vocab}


def work(case):
    n = case["rows"]
    if case["op"] == "sample":
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * case["vocab"] * size + n * 32, "flops": 6.0 * n * case["vocab"]}
    if case["op"] in ("norm", "norm_mx", "norm_bwd"):
        h, size = case["hidden"], 2 if case["dtype"] == "bf16" else 4
        wsize = 2 if case["weight"] == "bf16" else 4
        res = 1 if case["residual"] else 0
        if case["op"] == "norm":  # x, residual -> h, y; without a residual h is x
            return {"bytes": n * h * size * (2 + 2 * res) + h * wsize + 4 * n, "flops": 6.0 * n * h}
        if case["op"] == "norm_mx":
            return {"bytes": n * h * (size * (1 + 2 * res) + 1) + n * h // 32 + h * wsize, "flops": 8.0 * n * h}
        # dy, h, the gradient of h -> dx; the weight's gradient
        return {"bytes": n * h * size * (3 + res) + 2 * h * wsize + 4 * n, "flops": 12.0 * n * h}
    if case["op"] == "quantize":  # read once; the values it stands for are written as bf16
        size = 2 if case["dtype"] == "bf16" else 4
        return {"bytes": n * case["cols"] * (size + 2), "flops": 4.0 * n * case["cols"]}
    h, v = case["hidden"], case["vocab"]
    return {"bytes": n * h * (1 + 1 / 32) + v * h * (1 / 2 + 1 / 32) + n * v * 2, "flops": 2.0 * n * h * v}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _normal(g, *shape, std=1.0):
    return torch.randn(*shape, device="cuda", generator=g) * std


def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    n, s = case["rows"], {"case": case}
    if case["op"] == "sample":
        v = case["vocab"]
        # a bulk of unlikely tokens and a sparse set of likely ones, as a language model's logits have
        z = _normal(g, n, v, std=2.0)
        z += 8.0 * torch.rand(n, v, device="cuda", generator=g) * (
            torch.rand(n, v, device="cuda", generator=g) < 3e-4)
        if case["masked"]:
            z.masked_fill_(torch.rand(n, v, device="cuda", generator=g) < case["masked"], -math.inf)
            if n > 1:
                z[n // 2] = -math.inf  # a grammar that allows no token
        s["logits"] = z.to(DTYPES[case["dtype"]])
        s["uniform"] = torch.rand(n, device="cuda", generator=g)

        def full(value, dtype=torch.float32):
            return torch.full((n,), value, device="cuda", dtype=dtype)

        def either(p, a, b):
            return torch.where(torch.rand(n, device="cuda", generator=g) < p, a, b)

        def between(lo, hi):
            return lo + (hi - lo) * torch.rand(n, device="cuda", generator=g)

        s.update(temperature=None, top_k=None, top_p=None, min_p=None)
        if case["mode"] == "topk":
            s.update(temperature=full(0.8), top_k=full(50, torch.int32), top_p=full(0.95))
        elif case["mode"] == "nucleus":
            s.update(temperature=full(0.9), top_p=full(0.9))
        elif case["mode"] == "minp":
            s.update(temperature=full(1.1), min_p=full(0.02))
        elif case["mode"] == "mixed":
            ks = torch.exp(between(0.0, math.log(5000.0))).to(torch.int32)
            s.update(temperature=either(0.1, full(0.0), between(0.3, 1.5)),
                     top_k=either(0.5, full(0, torch.int32), ks),
                     top_p=either(0.4, full(1.0), between(0.3, 0.99)),
                     min_p=either(0.7, full(0.0), between(0.001, 0.2)))
    elif case["op"] in ("norm", "norm_mx", "norm_bwd"):
        h, dtype = case["hidden"], DTYPES[case["dtype"]]
        s["x"] = _normal(g, n, h).to(dtype)
        s["weight"] = (1.0 + _normal(g, h, std=0.1)).to(DTYPES[case["weight"]])
        s["residual"] = _normal(g, n, h, std=3.0).to(dtype) if case["residual"] else None
        s["eps"] = 1e-6
        if case["op"] == "norm_bwd":  # what the forward pass left, and what arrives from the loss
            hs = s["x"].float() + (s["residual"].float() if case["residual"] else 0.0)
            s["h"] = hs.to(dtype)
            s["rstd"] = torch.rsqrt(s["h"].double().square().mean(1) + s["eps"]).float()
            s["dy"] = _normal(g, n, h, std=0.01).to(dtype)
            s["dh"] = _normal(g, n, h, std=0.01).to(dtype) if case["residual"] else None
            del s["x"], s["residual"]
    elif case["op"] == "quantize":
        # rows of differing size, as a trained classifier's and hidden states' are
        x = _normal(g, n, case["cols"], std=case["cols"] ** -0.5)
        s["x"] = (x * torch.exp(_normal(g, n, 1, std=0.5))).to(DTYPES[case["dtype"]])
    else:
        h, v = case["hidden"], case["vocab"]
        s["x"] = _pack(*_plain_quantize(_normal(g, n, h), "e4m3"), "e4m3")
        s["w"] = _pack(*_plain_quantize(_normal(g, v, h, std=h ** -0.5), "e2m1"), "e2m1")
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _plain_sample(logits, uniform, temperature, top_k, top_p, min_p):
    """The token of each row and the logarithm of the probability it was drawn with.

    Tokens are ordered by descending logit, lowest index first among equal ones.  top_k keeps
    the first k; top_p the shortest head whose mass reaches that share of what top_k kept; min_p
    those whose probability reaches that share of the first one's.  The token is the first whose
    cumulated mass exceeds uniform times the mass of all kept ones.  Masses are in 64 bits: each
    choice compares sums of up to all tokens with a border between two of them.
    """
    n, v = logits.shape
    z, order = torch.sort(logits.float(), dim=1, descending=True, stable=True)
    top = z[:, :1]
    valid = torch.isfinite(top[:, 0]) & ~torch.isnan(logits).any(1)
    t = torch.ones(n, device=z.device) if temperature is None else temperature
    greedy = t <= 0
    t = torch.where(greedy, torch.ones_like(t), t).double()[:, None]
    w = torch.exp((z.double() - top.double()) / t)
    rank = torch.arange(v, device=z.device)[None, :]
    keep = w > 0
    keep = keep & ~(greedy[:, None] & (rank > 0))
    if top_k is not None:
        keep = keep & ((rank < top_k[:, None]) | (top_k[:, None] <= 0))
    w = torch.where(keep, w, torch.zeros_like(w))
    if top_p is not None:
        before = torch.cumsum(w, 1) - w
        border = top_p.double()[:, None] * w.sum(1, keepdim=True)
        keep = keep & ((before < border) | (rank == 0) | (top_p[:, None] >= 1))
    if min_p is not None:
        keep = keep & (w >= min_p.double()[:, None].clamp(max=1.0))
    w = torch.where(keep, w, torch.zeros_like(w))
    cum = torch.cumsum(w, 1)
    mass = cum[:, -1:]
    at = (cum <= uniform.double()[:, None] * mass).sum(1)
    at = torch.minimum(at, keep.sum(1) - 1).clamp(min=0)[:, None]
    token = torch.gather(order, 1, at)[:, 0]
    logprob = (torch.log(torch.gather(w, 1, at)) - torch.log(mass))[:, 0]
    token = torch.where(valid, token, torch.full_like(token, -1))
    logprob = torch.where(valid, logprob, torch.full_like(logprob, math.nan))
    return token, logprob.float()


def _plain_residual(x, residual):
    return x if residual is None else (x.float() + residual.float()).to(x.dtype)


def _plain_norm(h, weight, eps):
    hf = h.float()
    rstd = torch.rsqrt((hf * hf).mean(1) + eps)
    return hf * rstd[:, None] * weight.float(), rstd


def _plain_norm_backward(dy, h, weight, rstd, dh):
    hat = h.float() * rstd[:, None]
    wdy = dy.float() * weight.float()
    dx = rstd[:, None] * (wdy - hat * (wdy * hat).mean(1, keepdim=True))
    if dh is not None:
        dx = dx + dh.float()
    dweight = (dy.float() * hat).sum(0)
    return dx.to(h.dtype), dweight.to(weight.dtype)


def _plain_scale(x, fmt):
    """Exponents of the smallest powers of two under which no value of a block saturates, [n, blocks]; 128
    marks a block that holds an infinity or a NaN."""
    n, c = x.shape
    blocks = torch.nn.functional.pad(x.float(), (0, -c % 32)).view(n, -1, 32)
    amax = blocks.abs().amax(2)
    mant, exp = torch.frexp(amax)  # amax = mant * 2**exp, mant in [0.5, 1)
    most, emax = (0.75, 3) if fmt == "e2m1" else (0.875, 9)  # the largest value: most * 2**emax
    e = exp - emax + (mant > most)
    e = torch.where(amax > 0, e, torch.full_like(e, -127)).clamp(-127, 127)
    e = torch.where(torch.isfinite(amax), e, torch.full_like(e, 128))
    return blocks, e


def _plain_quantize(x, fmt):
    """Codes [n, columns] in their own type of values (float32 of E2M1 or E4M3), and scale exponents."""
    blocks, e = _plain_scale(x, fmt)
    t = blocks * torch.exp2(-e.clamp(max=127).float())[:, :, None]
    if fmt == "e2m1":  # round to the nearest step of the value's octave, ties to even
        a = t.abs()
        step = torch.where(a < 2, 0.5, torch.where(a < 4, 1.0, 2.0))
        q = torch.copysign(torch.round(a / step) * step, t)
    else:
        q = t.to(torch.float8_e4m3fn).float()
    q = torch.where((e == 128)[:, :, None], torch.zeros_like(q), q)
    return q.view(x.shape[0], -1), e


def _plain_dequantize(q, e):
    s = torch.where(e == 128, torch.full_like(e, math.nan, dtype=torch.float32), torch.exp2(e.float()))
    return (q.view(q.shape[0], -1, 32) * s[:, :, None]).view(q.shape[0], -1)


def _tile_scales(e):
    """Scale exponents [n, blocks] as E8M0 bytes in tiles of 128 rows x 4 blocks."""
    n, b = e.shape
    bytes_ = (e + 127).to(torch.uint8)
    bytes_ = torch.nn.functional.pad(bytes_, (0, -b % 4, 0, -n % 128))
    return bytes_.view(-1, 4, 32, bytes_.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()


def _pack(q, e, fmt):
    """(codes, scales) as a microscaled tensor holds them."""
    n = q.shape[0]
    if fmt == "e4m3":
        codes = q.to(torch.float8_e4m3fn).view(torch.uint8)
        return torch.nn.functional.pad(codes, (0, -q.shape[1] % 128)), _tile_scales(e)
    a = q.abs()
    code = torch.where(a < 2, a * 2, torch.where(a < 4, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q).to(torch.uint8) << 3)
    code = torch.nn.functional.pad(code, (0, -q.shape[1] % 128)).view(n, -1, 2)
    return code[:, :, 0] | (code[:, :, 1] << 4), _tile_scales(e)


def _untile_scales(scales, rows, blocks):
    t = scales.permute(0, 3, 2, 1, 4)
    return t.reshape(t.shape[0] * 128, -1)[:rows, :blocks]


def _plain_values(codes, scales, cols, fmt):
    """The float32 values a microscaled tensor stands for, [rows, cols]."""
    n = codes.shape[0]
    if fmt == "e4m3":
        q = codes.view(torch.float8_e4m3fn).float()
    else:
        lut = torch.tensor(E2M1_VALUES + tuple(-x for x in E2M1_VALUES), device=codes.device)
        pair = torch.stack((codes & 15, codes >> 4), 2).view(-1).to(torch.int32)
        q = torch.index_select(lut, 0, pair).view(n, -1)
    e = _untile_scales(scales, n, q.shape[1] // 32).float() - 127.0
    return (q.view(n, -1, 32) * torch.exp2(e)[:, :, None]).view(n, -1)[:, :cols]


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        return _own_run(op, case, state)
    if op == "sample":
        return _plain_sample(state["logits"], state["uniform"], state["temperature"], state["top_k"],
                             state["top_p"], state["min_p"])
    if op == "norm":
        h = _plain_residual(state["x"], state["residual"])
        y, rstd = _plain_norm(h, state["weight"], state["eps"])
        return y.to(h.dtype), h, rstd
    if op == "norm_mx":
        h = _plain_residual(state["x"], state["residual"])
        y, _ = _plain_norm(h, state["weight"], state["eps"])
        codes, scales = _pack(*_plain_quantize(y, "e4m3"), "e4m3")
        return codes.view(torch.float8_e4m3fn), scales.view(torch.float8_e8m0fnu), h
    if op == "norm_bwd":
        return _plain_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"], state["dh"])
    if op == "quantize":
        q, e = _plain_quantize(state["x"], case["fmt"])
        return _plain_dequantize(q, e)[:, :case["cols"]].to(torch.bfloat16)
    x = _plain_values(*state["x"], case["hidden"], "e4m3")
    w = _plain_values(*state["w"], case["hidden"], "e2m1")
    return (x @ w.t()).to(torch.bfloat16)


def _own_run(op, case, state):
    import vocabulary_cross_entropy_gb300 as vce
    if op == "sample":
        r = vce.ce_sample(state["logits"], state["uniform"], state["temperature"], state["top_k"],
                          state["top_p"], state["min_p"])
        return r.token, r.logprob
    if op == "norm":
        r = vce.rms_norm_forward(state["x"], state["weight"], state["eps"], state["residual"])
        return r.y, r.h, r.rstd
    if op == "norm_mx":
        r = vce.rms_norm_mx(state["x"], state["weight"], state["eps"], state["residual"])
        return r.y.codes.view(torch.float8_e4m3fn), r.y.scales.view(torch.float8_e8m0fnu), r.h
    if op == "norm_bwd":
        r = vce.rms_norm_backward(state["dy"], state["h"], state["weight"], state["rstd"], state["dh"])
        return r.dx, r.dweight
    if op == "quantize":
        return vce.mx_dequantize(vce.mx_quantize(state["x"], case["fmt"]), torch.bfloat16)
    x = vce.MXTensor(*state["x"], case["rows"], case["hidden"], "e4m3")
    w = vce.MXTensor(*state["w"], case["vocab"], case["hidden"], "e2m1")
    return vce.mx_linear(x, w, torch.bfloat16)


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------

def _exact_sample(s):
    """Row by row, from sorted values alone: the kept head's length, then the draw in it."""
    out = []
    for r in range(s["logits"].shape[0]):
        z = s["logits"][r].double()
        best = z.max()
        if not bool(torch.isfinite(best)):
            out.append(math.nan)
            continue
        t = 1.0 if s["temperature"] is None else float(s["temperature"][r])
        if t <= 0:
            out.append(0.0)
            continue
        p = torch.exp((torch.sort(z, descending=True).values - best) / t)
        k = 0 if s["top_k"] is None else int(s["top_k"][r])
        p = p[:k] if k > 0 else p
        c = torch.cumsum(p, 0)
        kept = int((p > 0).sum())
        share = 1.0 if s["top_p"] is None else float(s["top_p"][r])
        if share < 1:
            kept = min(kept, 1 + int((c[:-1] < share * c[-1]).sum()))
        least = 0.0 if s["min_p"] is None else float(s["min_p"][r])
        if least > 0:
            kept = min(kept, int((p >= min(least, 1.0)).sum()))
        at = min(int((c[:kept] <= float(s["uniform"][r]) * c[kept - 1]).sum()), kept - 1)
        out.append(float(torch.log(p[at] / c[kept - 1])))
    return [None, torch.tensor(out, dtype=torch.float64)]


def _exact_exponent(amax, most):
    """The least e with amax <= most * 2**e.  A logarithm of an exact power of two may come out a hair above
    it: quotients closer to one than 1e-9 (a float32's neighbours are 1.2e-7 apart) count as one."""
    return torch.ceil(torch.log2(amax / most) - 1e-9).clamp(-127, 127)


def _exact_codes(y):
    """E4M3 values and scales of y [n, c] in 64 bits, padded as a microscaled tensor is."""
    n, c = y.shape
    pad = torch.zeros(n, -(-c // 128) * 128, dtype=torch.float64, device=y.device)
    pad[:, :c] = y
    b = pad.view(n, -1, 32)
    amax = b.abs().amax(2)
    e = _exact_exponent(amax, 448.0)
    e = torch.where(amax > 0, e, torch.full_like(e, -127.0))
    t = b * torch.exp2(-e)[:, :, None]
    octave = torch.floor(torch.log2(t.abs().clamp(min=2.0 ** -6)))
    q = torch.round(t / torch.exp2(octave - 3)) * torch.exp2(octave - 3)
    scales = torch.full((-(-n // 128), pad.shape[1] // 128, 32, 4, 4), 2.0 ** -127, dtype=torch.float64,
                        device=y.device)
    row = torch.arange(n, device=y.device)[:, None]
    blk = torch.arange(-(-c // 32), device=y.device)[None, :]
    scales[row // 128, blk // 4, row % 32, row % 128 // 32, blk % 4] = torch.exp2(e)[:, :blk.shape[1]]
    return q.view(n, -1), scales


def _exact_matrix(codes, scales, cols, fmt):
    n = codes.shape[0]
    if fmt == "e4m3":
        b = codes.int()
        m, x = b & 7, (b >> 3) & 15
        q = torch.where(x > 0, (8 + m).double() * torch.exp2((x - 10).double()), m.double() * 2.0 ** -9)
        q = torch.where(b > 127, -q, q)
    else:
        half = []
        for b in (codes & 15, codes >> 4):
            x, m = ((b & 7) >> 1).double(), (b & 1).double()
            v = torch.where(x > 0, (1 + m / 2) * torch.exp2(x - 1), m / 2)
            half.append(torch.where(b > 7, -v, v))
        q = torch.stack(half, 2).view(n, -1)
    row = torch.arange(n, device=codes.device)[:, None]
    blk = torch.arange(-(-cols // 32), device=codes.device)[None, :]
    e = scales[row // 128, blk // 4, row % 32, row % 128 // 32, blk % 4].double() - 127
    return (q.view(n, -1, 32)[:, :blk.shape[1]] * torch.exp2(e)[:, :, None]).view(n, -1)[:, :cols]


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "sample":
        return _exact_sample(s)
    if op in ("norm", "norm_mx"):
        h = s["x"]
        if s["residual"] is not None:
            h = (s["x"].double() + s["residual"].double()).to(s["x"].dtype)
        hd = h.double()
        rstd = 1.0 / torch.sqrt(hd.square().mean(1) + s["eps"])
        y = hd * s["weight"].double() * rstd[:, None]
        if op == "norm":
            return y, hd, rstd
        return (*_exact_codes(y), hd)
    if op == "norm_bwd":
        h, dy, w, r = s["h"].double(), s["dy"].double(), s["weight"].double(), s["rstd"].double()[:, None]
        proj = (dy * w * h).sum(1, keepdim=True) / h.shape[1]
        dx = r * dy * w - r ** 3 * h * proj
        if s["dh"] is not None:
            dx = dx + s["dh"].double()
        return dx, (dy * h * r).sum(0)
    if op == "quantize":
        x, c = s["x"].double(), case["cols"]
        n = x.shape[0]
        most, low, bits = (6.0, 0.0, 1) if case["fmt"] == "e2m1" else (448.0, -6.0, 3)
        out = torch.empty(n, c, dtype=torch.float64, device=x.device)
        for i in range(0, n, 8192):
            part = torch.zeros(min(8192, n - i), -(-c // 32) * 32, dtype=torch.float64, device=x.device)
            part[:, :c] = x[i:i + 8192]
            b = part.view(part.shape[0], -1, 32)
            amax = b.abs().amax(2, keepdim=True)
            scale = torch.exp2(_exact_exponent(amax, most))
            scale = torch.where(amax > 0, scale, torch.ones_like(scale))
            t = b / scale
            step = torch.exp2(torch.floor(torch.log2(t.abs().clamp(min=2.0 ** low))) - bits)
            out[i:i + 8192] = (torch.round(t / step) * step * scale).view(part.shape[0], -1)[:, :c]
        return out
    x = _exact_matrix(*s["x"], case["hidden"], "e4m3")
    w = _exact_matrix(*s["w"], case["hidden"], "e2m1")
    return x @ w.t()

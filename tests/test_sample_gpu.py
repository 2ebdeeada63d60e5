"""Sampling against its FP64 definition: the same token for every row, and its log probability.

Tokens are whole numbers and have to be equal.  The kernel's weights are within 2^-40 of the
definition's relative to the largest, so a row can differ only where uniform * mass comes
within about 2^-40 V of a border between two tokens' shares: for the row counts here the chance
is below 1e-6 in all, and inputs are fixed.

logprob is x - log(mass), x = (z - m) / T rounded once or twice: off by 4 u (|x| + |log mass|)
+ u |logprob| (log, log1p and the float of the mass: 2 ulp each), u = 2^-24.
"""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import head

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def per_row(value, n, default):
    if value is None:
        return np.full(n, default)
    if isinstance(value, torch.Tensor):
        return value.double().cpu().numpy()
    return np.full(n, np.float32(value), np.float64)


def check(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, status=0):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = vce.ce_sample(logits, uniform, temperature, top_k, top_p, min_p, dev_status=st)
    torch.cuda.synchronize()
    assert int(st) == status
    z = logits.double().cpu().numpy().reshape(-1, logits.shape[-1])
    n = z.shape[0]
    t, p, mp = per_row(temperature, n, 1.0), per_row(top_p, n, 1.0), per_row(min_p, n, 0.0)
    k = np.full(n, top_k or 0) if not isinstance(top_k, torch.Tensor) else top_k.cpu().numpy()
    u = uniform.double().cpu().numpy()
    want = [head.sample_row(z[i], u[i], t[i], int(k[i]), p[i], mp[i]) for i in range(n)]
    tokens = np.array([w[0] for w in want])
    got = r.token.cpu().numpy().reshape(-1)
    bad = np.nonzero(got != tokens)[0]
    assert bad.size == 0, (bad[:5], got[bad[:5]], tokens[bad[:5]])
    lp = np.array([w[1] for w in want])
    glp = r.logprob.double().cpu().numpy().reshape(-1)
    assert np.array_equal(np.isnan(glp), np.isnan(lp))
    for i in np.nonzero(~np.isnan(lp))[0]:
        x = abs(z[i][tokens[i]] - z[i].max()) / max(t[i], 1e-30) if t[i] > 0 else 0.0
        lim = 4 * U * (x + abs(x + lp[i])) + 6 * U * abs(lp[i]) + 1e-12
        assert abs(glp[i] - lp[i]) <= lim, (i, glp[i], lp[i], lim)
    return r


def make(seed, n, v, dtype, std=2.0, mask=0.0, peaks=True, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    z = torch.randn(n, v + pad + offset, generator=g) * std
    if peaks:
        z += 8 * torch.rand(z.shape, generator=g) * (torch.rand(z.shape, generator=g) < 3e-3)
    if mask:
        z.masked_fill_(torch.rand(z.shape, generator=g) < mask, -float("inf"))
        z[:, offset] = torch.where(torch.isfinite(z[:, offset]), z[:, offset], torch.zeros(()))
    u = torch.rand(n, generator=g).to(DEV)
    return z.to(DT[dtype]).to(DEV)[:, offset:offset + v], u


FILTERS = [dict(), dict(temperature=0.7), dict(top_k=1), dict(top_k=5), dict(top_k=50, top_p=0.9, temperature=0.8),
           dict(top_p=0.9), dict(top_p=0.3, temperature=1.3), dict(min_p=0.05), dict(min_p=0.001, temperature=2.0),
           dict(top_k=300, top_p=0.95), dict(top_k=700, min_p=0.01), dict(top_p=0.8, min_p=0.02), dict(temperature=0.0),
           dict(top_k=2500, top_p=0.99, temperature=1.5), dict(top_k=40, top_p=0.7, min_p=0.1)]


@pytest.mark.parametrize("f", range(len(FILTERS)))
@pytest.mark.parametrize("n,v,dtype", [(1, 1000, "f32"), (3, 32001, "bf16"), (1, 128256, "bf16"), (200, 5003, "f32"),
                                       (40, 50257, "f32"), (400, 1024, "bf16")])
def test_filters(n, v, dtype, f):
    z, u = make(100 + f, n, v, dtype)
    check(z, u, **FILTERS[f])


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,v", [(160, 32000), (7, 202048)])
def test_mixed_rows(n, v, dtype):
    z, u = make(5, n, v, dtype, mask=0.3)
    g = torch.Generator().manual_seed(6)
    rnd = lambda: torch.rand(n, generator=g)
    t = torch.where(rnd() < 0.15, torch.zeros(n), 0.3 + 1.2 * rnd()).to(DEV)
    k = torch.where(rnd() < 0.5, torch.zeros(n), torch.exp(rnd() * 9)).to(torch.int32).to(DEV)
    p = torch.where(rnd() < 0.4, torch.ones(n), 0.2 + 0.79 * rnd()).to(DEV)
    m = torch.where(rnd() < 0.6, torch.zeros(n), 0.2 * rnd()).to(DEV)
    check(z, u, t, k, p, m)


@pytest.mark.parametrize("v", [1, 2, 3, 7, 8, 9, 31, 100])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_short_rows(v, dtype):
    z, u = make(v, 50, v, dtype)
    for f in FILTERS:
        check(z, u, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v,pad,offset", [(1000, 3, 1), (4099, 0, 2), (33000, 1, 5)])
def test_strided_rows(v, pad, offset, dtype):
    z, u = make(v, 9, v, dtype, mask=0.1, pad=pad, offset=offset)
    for f in FILTERS[::2]:
        check(z, u, **f)


def test_leading_dimensions():
    z, u = make(1, 12, 500, "f32")
    r = check(z.view(3, 4, 500), u, top_k=20)
    assert r.token.shape == (3, 4) and r.logprob.shape == (3, 4)


@pytest.mark.parametrize("n", [1, 2, 200])
def test_ties(n):
    # few distinct values: equal logits go by index, and a bin holds far more than fits a list
    v = 20000
    g = torch.Generator().manual_seed(n)
    z = torch.randint(0, 3, (n, v), generator=g).float().to(DEV)
    u = torch.rand(n, generator=g).to(DEV)
    for f in FILTERS + [dict(top_k=9000), dict(temperature=1e30), dict(temperature=1e3, top_p=0.5)]:
        check(z, u, **f)
    same = torch.full((n, v), -3.0, device=DEV)
    for f in FILTERS + [dict(top_k=19999)]:
        check(same, u, **f)
    same[:, 5] = float("-inf")
    check(same, torch.zeros(n, device=DEV))


def test_equal_shares_are_split_exactly():
    z = torch.full((8, 8), 1.25, device=DEV)
    u = torch.arange(8, device=DEV) / 8.0        # on the borders: a token's share is closed below
    r = check(z, u)
    assert r.token.tolist() == list(range(8))
    check(z, u, top_p=0.5)
    check(z, u, top_k=4)


def test_negative_zero_is_zero():
    z = torch.tensor([[0.0, -0.0, 0.0, -1.0]], device=DEV).bfloat16()
    z = torch.cat([z, torch.tensor([[-0.0, 0.0, -0.0, -1.0]], device=DEV).bfloat16()])
    u = torch.tensor([0.4, 0.4], device=DEV)
    check(z, u, top_k=2)
    check(z, u, temperature=0.0)


@pytest.mark.parametrize("spread", [1e-6, 1e-3, 1.0, 1e4])
def test_close_and_far_logits(spread):
    # a narrow range puts a whole row in one bin; a wide one leaves one token
    z, u = make(3, 30, 30000, "f32", std=spread, peaks=False)
    for off in (0.0, 1000.0):
        for f in FILTERS[::3]:
            check(z + off, u, **f)


@pytest.mark.parametrize("temperature", [1e-35, 1e-6, 0.01, 100.0, 1e35, float("inf")])
def test_temperatures(temperature):
    z, u = make(4, 20, 3000, "f32")
    check(z, u, temperature=temperature)
    check(z, u, temperature=temperature, top_k=10)
    check(z, u, temperature=temperature, top_p=0.5)


def test_uniform_at_the_ends():
    z, _ = make(5, 6, 4000, "f32")
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 2.0 ** -30, 1e-40, 0.5, -1.0], device=DEV)
    for f in FILTERS:
        check(z, u, **f)
    over = vce.ce_sample(z, torch.full((6,), 1.5, device=DEV), top_k=10)
    last = torch.topk(z, 10, dim=1).indices[:, -1]
    assert torch.equal(over.token, last)


def last_kept(z, top_k=None, top_p=None, min_p=None):
    """The last token of each row's kept head, in FP64."""
    zs, order = torch.sort(z.double(), dim=1, descending=True, stable=True)
    w = torch.exp(zs - zs[:, :1])
    rank = torch.arange(z.shape[1], device=z.device)
    keep = torch.ones_like(w, dtype=torch.bool)
    if top_k is not None:
        keep &= rank < top_k[:, None]
    w = w * keep
    if top_p is not None:
        keep &= (torch.cumsum(w, 1) - w < top_p.double()[:, None] * w.sum(1, keepdim=True)) | (rank == 0)
    if min_p is not None:
        keep &= w >= min_p.double()[:, None]
    return order.gather(1, keep.sum(1, keepdim=True) - 1)[:, 0]


@pytest.mark.parametrize("filters", ["k", "p", "m", "kp", "km", "pm", "kpm"])
@pytest.mark.parametrize("n,v,dtype", [(600, 50257, "f32"), (600, 32001, "bf16"), (40, 128256, "f32")])
def test_uniform_of_one_takes_the_last_kept(n, v, dtype, filters):
    # heads too long for the collecting path: a border's mass and the masses that the draw is
    # looked up in are rounded differently, and the draw must not land behind the border
    z, _ = make(21, n, v, dtype)
    g = torch.Generator(DEV).manual_seed(22)
    rnd = lambda: torch.rand(n, device=DEV, generator=g)
    f = {}
    if "k" in filters:
        f["top_k"] = (257 + 4000 * rnd()).int()
    if "p" in filters:
        f["top_p"] = 0.3 + 0.699 * rnd()
    if "m" in filters:
        f["min_p"] = torch.exp(-12 * rnd())
    want = last_kept(z, **f)
    for u in (1.0, 1.5):
        assert torch.equal(vce.ce_sample(z, torch.full((n,), u, device=DEV), **f).token, want)


@pytest.mark.parametrize("n", [1, 200])
@pytest.mark.parametrize("v", [1500, 5000])
def test_uniform_of_one_among_least_weights(n, v):
    # weights of 1.41 units of the least one: rounded one by one they sum to less than together,
    # and more of them than a list holds
    z = torch.full((n, v), -43.5 * float(np.log(2)), device=DEV)
    z[:, 77] = 0.0
    for u in (1.0, 1.5):
        assert (vce.ce_sample(z, torch.full((n,), u, device=DEV)).token == v - 1).all()


@pytest.mark.parametrize("n,v", [(1, 700), (300, 700), (1, 9000), (300, 9000)])
def test_uniform_of_one_counts_tokens_near_the_least_weight(n, v):
    # 0.55 to 1.6 units each, many of them equal or nearly so: no sum of theirs, rounded together
    # or one by one, tells which is the last
    g = torch.Generator(DEV).manual_seed(v + n)
    z = (-44.8 + 1.5 * (torch.rand(n, v, device=DEV, generator=g) * 20).floor() / 20) * float(np.log(2))
    z[:, v // 3] = 0.0
    k = (2 + (v - 2) * torch.rand(n, device=DEV, generator=g)).int()
    m = torch.full((n,), 1.5 * 2.0 ** -44, device=DEV)
    for dtype in (torch.float32, torch.bfloat16):
        zz = z.to(dtype)
        for u in (1.0, 1.5):
            uu = torch.full((n,), u, device=DEV)
            assert torch.equal(vce.ce_sample(zz, uu).token, last_kept(zz))
            if v > 700:  # (shorter heads are collected as a whole)
                k = k.clamp(min=257)
            assert torch.equal(vce.ce_sample(zz, uu, top_k=k).token, last_kept(zz, top_k=k))
            # one and a half units: where whole units and weights agree on what is kept
            assert torch.equal(vce.ce_sample(zz, uu, min_p=m).token, last_kept(zz, min_p=m))


@pytest.mark.parametrize("n,v", [(1, 1500), (1, 5000), (200, 1500), (200, 5000), (1, 1 << 20)])
def test_least_weights_are_never_drawn(n, v):
    # 0.4 units of the least weight each: below the border, however many there are
    unit = -44 if v <= 1 << 19 else -43
    z = torch.full((n, v), (unit - 1.35) * float(np.log(2)), device=DEV)
    z[:, 77] = 0.0
    for f in (dict(), dict(top_k=v - 1)):
        for u in (1.0, 1.5):
            r = vce.ce_sample(z, torch.full((n,), u, device=DEV), **f)
            assert (r.token == 77).all() and (r.logprob == 0).all()
    z[:, v // 2] = (unit - 0.9) * float(np.log(2))  # 0.54 units
    assert (vce.ce_sample(z, torch.ones(n, device=DEV)).token == v // 2).all()


def test_parameters_that_filter_nothing():
    z, u = make(6, 30, 2000, "bf16")
    want = check(z, u)
    for f in (dict(top_k=0), dict(top_k=-1), dict(top_k=2000), dict(top_k=1 << 30), dict(top_p=1.0), dict(top_p=2.0),
              dict(min_p=0.0), dict(min_p=-1.0), dict(temperature=1.0)):
        assert torch.equal(vce.ce_sample(z, u, **f).token, want.token)
    first = vce.ce_sample(z, u, temperature=-1.0).token
    for f in (dict(top_k=1), dict(top_p=0.0), dict(top_p=-1.0), dict(min_p=1.0), dict(min_p=7.0)):
        got = vce.ce_sample(z, torch.zeros_like(u), **f)
        assert torch.equal(got.token, first), f


def test_numbers_past_their_type():
    z, u = make(6, 30, 2000, "f32")
    want = vce.ce_sample(z, u).token
    for f in (dict(top_k=1 << 40), dict(top_k=float("inf")), dict(top_p=1e39), dict(min_p=-1e39)):
        assert torch.equal(vce.ce_sample(z, u, **f).token, want), f
    assert torch.equal(vce.ce_sample(z, u, temperature=1e39).token, vce.ce_sample(z, u, temperature=1e30).token)
    ones = torch.ones(30, device=DEV)  # numbers of one value for parameters of two types
    assert torch.equal(vce.ce_sample(z, u, 1, 1, 1, 1).token, vce.ce_sample(z, u, ones, ones.int(), ones, ones).token)
    assert torch.equal(vce.ce_sample(z, u, top_k=50.0).token, vce.ce_sample(z, u, top_k=50).token)


@pytest.mark.parametrize("v", [100, 40000])
@pytest.mark.parametrize("f", [dict(), dict(top_k=10), dict(top_p=0.9), dict(min_p=0.1), dict(temperature=0.0)])
def test_masks_and_bad_rows(v, f):
    z, u = make(7, 8, v, "f32", mask=0.9)
    z = z.contiguous()
    z[1] = float("-inf")
    z[2, v // 2] = float("nan")
    z[3, v - 1] = float("inf")
    z[4] = float("-inf")
    z[4, v - 2] = -7.0                       # one token left
    z[5] = torch.finfo(torch.float32).min    # a mask of the lowest value everywhere
    z[6, :] = torch.finfo(torch.float32).min
    z[6, 3] = 2.0
    r = check(z, u, status=vce.DEVSTATUS_BAD_ROW, **f)
    assert r.token.tolist()[1:4] == [-1, -1, -1] and r.token[4] == v - 2 and r.token[6] == 3
    nan = torch.full((8,), float("nan"), device=DEV)
    ok, uu = make(8, 8, v, "f32")
    for g in (dict(temperature=nan), dict(top_p=nan), dict(min_p=nan)):
        assert (vce.ce_sample(ok, uu, **g).token == -1).all()
    assert (vce.ce_sample(ok, nan).token == -1).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_largest_vocabulary(dtype):
    v = vce.SAMPLE_MAX_VOCAB
    z, u = make(9, 2, v, dtype)
    for f in (dict(), dict(top_k=50), dict(top_p=0.9), dict(top_k=3000, top_p=0.9)):
        check(z, u, **f)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("offset", [0, 1, 7])
def test_largest_vocabulary_of_equal_logits(offset, dtype):
    # every token but one in a single step of the exponent, at rows that start off a 16-byte
    # boundary: sums of the largest parts of a row stay within their words
    v, n = vce.SAMPLE_MAX_VOCAB, 6
    z = torch.empty(n, v + 8, device=DEV, dtype=DT[dtype])
    z[:] = -torch.tensor([0.25, 0.00546875, 0.0027, 1.7, 4.03125, 7.9], device=DEV).to(DT[dtype])[:, None]
    z = z[:, offset:offset + v]
    z[:, 0] = 0
    u = torch.rand(n, device=DEV, generator=torch.Generator(DEV).manual_seed(5 + offset))
    check(z, u)
    check(z, u, top_p=0.6)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("v", [1 << 18, 1 << 19, 1 << 20])
def test_rows_of_full_weights(v, dtype):
    # equal logits, and any logits at the highest temperature: the sum of a row is the largest there is
    z = torch.full((3, v), -1.5, dtype=DT[dtype], device=DEV)
    u = torch.tensor([0.0, 0.37, 1.0 - 2.0 ** -24], device=DEV)
    check(z, u)
    check(z, u, top_p=0.3)
    check(z, u, top_k=v - 1)
    g = torch.Generator(DEV).manual_seed(v)
    z = torch.randn(2, v, device=DEV, generator=g).to(DT[dtype])
    check(z, u[:2], temperature=float("inf"))
    check(z, u[1:], temperature=float("inf"), top_p=0.7)


def test_distribution():
    # uniform numbers on a fine grid draw every token in proportion to its probability
    z, _ = make(10, 1, 12, "f32", peaks=False)
    n = 4096
    u = (torch.arange(n, device=DEV) + 0.5) / n
    tok = vce.ce_sample(z.expand(n, 12).contiguous(), u, temperature=0.9).token
    share = torch.bincount(tok, minlength=12).double().cpu() / n
    assert float((share - torch.softmax(z[0].double().cpu() / 0.9, 0)).abs().max()) <= 1.0 / n


def test_streams_graphs_and_two_calls_at_once():
    z, u = make(11, 20, 30000, "bf16")
    kw = dict(temperature=torch.full((20,), 0.9, device=DEV), top_p=torch.full((20,), 0.9, device=DEV))
    want = vce.ce_sample(z, u, **kw)
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams * 4:
        s.wait_stream(torch.cuda.current_stream())
        got.append(vce.ce_sample(z, u, stream=s, **kw))
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r.token, want.token) and torch.equal(r.logprob, want.logprob)
    graph = torch.cuda.CUDAGraph()
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    zs, us = z.contiguous().clone(), u.clone()
    with torch.cuda.graph(graph):
        r = vce.ce_sample(zs, us, dev_status=st, **kw)
    for k in (12, 13):
        z2, u2 = make(k, 20, 30000, "bf16")
        zs.copy_(z2)
        us.copy_(u2)
        graph.replay()
        e = vce.ce_sample(z2, u2, **kw)
        assert torch.equal(r.token, e.token) and torch.equal(r.logprob, e.logprob)


def test_split_does_not_change_results():
    # the same rows alone (split over eight blocks) and among many (one block each)
    z, u = make(14, 330, 20000, "f32")
    for f in FILTERS:
        many = vce.ce_sample(z, u, **f)
        for i in (0, 171, 329):
            alone = vce.ce_sample(z[i:i + 1], u[i:i + 1], **f)
            assert torch.equal(alone.token, many.token[i:i + 1])
            assert torch.equal(alone.logprob, many.logprob[i:i + 1])


@pytest.mark.parametrize("n", [1, 70])
def test_linear_sample(n):
    # norm -> product -> sample as one call, against its parts and the definition
    h, v = 256, 4000
    g = torch.Generator(DEV).manual_seed(n)
    x = torch.randn(2, n, h, device=DEV, generator=g).bfloat16()
    res = torch.randn(2, n, h, device=DEV, generator=g).bfloat16()
    nw = (3 + 0.1 * torch.randn(h, device=DEV, generator=g)).bfloat16()
    w = vce.mx_quantize(torch.randn(v, h, device=DEV, generator=g) * h ** -0.5, "e2m1")
    u = torch.rand(2 * n, device=DEV, generator=g)
    r = vce.linear_sample(x, w, u, 0.8, 50, 0.9, norm_weight=nw, residual=res)
    assert r.token.shape == (2, n)
    q = vce.rms_norm_mx(x.view(-1, h), nw, 1e-6, res.view(-1, h)).y
    logits = vce.mx_linear(q, w, torch.float32)
    check(logits, u, 0.8, 50, 0.9)
    assert torch.equal(vce.ce_sample(logits, u, 0.8, 50, 0.9).token, r.token.view(-1))
    z = vce.mx_dequantize(q, torch.float32).double() @ vce.mx_dequantize(w, torch.float32).double().t()
    assert float((logits.double() - z).abs().max()) <= 1e-4
    plain = vce.linear_sample(x[0], w, u[:n], 0.0)
    zq = vce.mx_linear(vce.mx_quantize(x[0], "e4m3"), w, torch.float32)
    assert torch.equal(plain.token, zq.argmax(1))
    # embeddings of any strides: one row for all (expanded), transposed
    same = vce.linear_sample(x[0, :1].expand(5, h), w, u[:1].expand(5).contiguous(), 0.8, norm_weight=nw)
    one = vce.linear_sample(x[0, :1], w, u[:1], 0.8, norm_weight=nw)
    assert torch.equal(same.token, one.token.expand(5))
    turned = vce.linear_sample(x.transpose(0, 1), w, u, 0.8, norm_weight=nw, residual=res.transpose(0, 1))
    assert turned.token.shape == (n, 2)
    assert torch.equal(turned.token, vce.linear_sample(x.transpose(0, 1).contiguous(), w, u, 0.8, norm_weight=nw,
                                                       residual=res.transpose(0, 1).contiguous()).token)
    none = vce.linear_sample(x[:, :0], w, u[:0], 0.8, norm_weight=nw)
    assert none.token.shape == (2, 0)


def test_linear_sample_reports_a_status():
    g = torch.Generator(DEV).manual_seed(2)
    x = torch.randn(3, 64, device=DEV, generator=g)
    w = vce.mx_quantize(torch.randn(50, 64, device=DEV, generator=g), "e2m1")
    u = torch.rand(3, device=DEV, generator=g)
    r = vce.linear_sample(x, w, u)
    assert r.dev_status.shape == (1,) and int(r.dev_status) == 0
    x[1, 3] = float("nan")
    r = vce.linear_sample(x, w, u, norm_weight=torch.ones(64, device=DEV))
    assert r.token[1] == -1 and int(r.dev_status) == vce.DEVSTATUS_BAD_ROW
    mine = torch.full((1,), 64, dtype=torch.int32, device=DEV)
    r = vce.linear_sample(x, w, u, dev_status=mine)
    assert r.dev_status is mine and int(mine) == 64 | vce.DEVSTATUS_BAD_ROW


@pytest.mark.parametrize("n", [1, 40])
def test_linear_sample_captured(n):
    # numbers as parameters and a status of the call's own, replayed on other inputs
    h, v = 192, 3001
    g = torch.Generator(DEV).manual_seed(n)
    x, res = (torch.randn(n, h, device=DEV, generator=g).bfloat16() for _ in range(2))
    w = vce.mx_quantize(torch.randn(v, h, device=DEV, generator=g) * h ** -0.5, "e2m1")
    u, nw = torch.rand(n, device=DEV, generator=g), torch.full((h,), 3.0, device=DEV)

    def call():
        return vce.linear_sample(x, w, u, 0.8, 50, 0.9, 0.01, norm_weight=nw, residual=res)

    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = call()
    for k in range(3):
        x.copy_(torch.randn(n, h, device=DEV, generator=g))
        u.copy_(torch.rand(n, device=DEV, generator=g))
        if k == 1:
            x[0, 0] = float("nan")
        graph.replay()
        want = call()
        assert torch.equal(r.token, want.token) and torch.equal(r.logprob.nan_to_num(7.0), want.logprob.nan_to_num(7.0))
        assert int(r.dev_status) == int(want.dev_status) == (vce.DEVSTATUS_BAD_ROW if k == 1 else 0)


def test_rows_past_32_bits():
    n, v = 17000, 128257
    z = torch.zeros(n, v, dtype=torch.bfloat16, device=DEV)
    z[-3:] = make(15, 3, v, "bf16")[0]
    u = torch.rand(n, device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    r = vce.ce_sample(z, u, top_p=0.9)
    tail = vce.ce_sample(z[-3:].clone(), u[-3:], top_p=0.9)
    assert torch.equal(r.token[-3:], tail.token)

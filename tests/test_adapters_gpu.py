"""adapter_linear against its FP64 definition, alone and as part of the head.

Tolerances, per logit, with M = s |B| (|A| |x|): a product of the tensor instruction is exact and
every addition is off by at most 2^-22 of what it adds to (cut off, and aligned with one bit to
spare).  t takes 6 additions per 2048 hidden values in a warp (three terms of FP32 states) and 16
between warps and blocks, the second product at most 24, scale and split one each: 2^-22 (6 H / 2048
+ 48) M.  BF16 logits take 16 bits of t, 2^-17 M, and are rounded once, 2^-8 of the result; FP32
ones 2^-24."""
import math

import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import beam as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def make(seed, n, h, v, r, count, xt, yt, none=0.2, pad=0, offset=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(n, h, generator=g).to(xt).to(DEV)
    a = (torch.randn(count, r, h, generator=g) * h ** -0.5).to(BF16).to(DEV)
    b = (torch.randn(count, v, r, generator=g) * r ** -0.5).to(BF16).to(DEV)
    full = (torch.randn(n, v + pad + offset, generator=g) * 2).to(yt).to(DEV)
    index = torch.randint(0, count, (n,), generator=g, dtype=torch.int32)
    index[torch.rand(n, generator=g) < none] = -1
    scale = (0.25 + torch.rand(count, generator=g)).to(DEV)
    return full[:, offset:offset + v], x, a, b, index.to(DEV), scale


def check(got, y, x, a, b, index, scale):
    yd, xd, ad, bd = (t.double().cpu().numpy() for t in (y, x, a, b))
    idx, sc = index.cpu().numpy(), None if scale is None else scale.double().cpu().numpy()
    want = ref.adapter_linear(yd, xd, ad, bd, idx, sc)
    most = ref.adapter_linear(np.zeros_like(yd), np.abs(xd), np.abs(ad), np.abs(bd), idx, sc)
    out = got.double().cpu().numpy()
    tol = 2.0 ** -22 * (6 * math.ceil(xd.shape[1] / 2048) + 48) * most + 2.0 ** -24 * np.abs(want)
    if got.dtype is BF16:
        tol += 2.0 ** -17 * most + 2.0 ** -8 * np.abs(want)
    assert (np.abs(out - want) <= tol).all(), np.abs(out - want).max()
    same = idx < 0
    assert np.array_equal(out[same], yd[same])
    return np.linalg.norm(out - want) / max(np.linalg.norm(want), 1e-300)


@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("xt", [BF16, F32])
@pytest.mark.parametrize("n,h,v,r,count", [(1, 64, 40, 8, 1), (1, 4096, 5000, 16, 3), (3, 8, 8, 8, 2), (17, 136, 257, 24, 5),
                                           (64, 512, 1000, 32, 64), (65, 520, 264, 40, 1), (200, 256, 2001, 64, 3),
                                           (130, 2056, 33, 96, 2), (300, 104, 511, 128, 7), (1, 32, 1, 16, 1),
                                           (5, 8200, 100, 120, 4), (1500, 64, 300, 8, 200)])
def test_adapters(n, h, v, r, count, xt, yt):
    for pad, none in ((0, 0.2), (8 - v % 8, 0.0)):
        y, x, a, b, index, scale = make(n + v, n, h, v, r, count, xt, yt, none, pad)
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        out = vce.adapter_linear(y, x, a, b, index, scale, dev_status=st)
        rel = check(out, y, x, a, b, index, scale)
        assert int(st) == 0 and out.is_contiguous()
        if yt is F32:
            assert rel <= 1e-6, rel
        plain = vce.adapter_linear(y, x, a, b, index)
        check(plain, y, x, a, b, index, None)
        place = y.clone(memory_format=torch.preserve_format) if pad == 0 else y
        assert vce.adapter_linear(place, x, a, b, index, scale, out=place) is place
        assert torch.equal(place, out)  # in place or not: the same bits


@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 0), (1, 4), (8, 8), (2, 7)])
def test_rows_anywhere(pad, offset, yt):
    """Rows off 16-byte boundaries; what lies between rows stays as it was."""
    y, x, a, b, index, scale = make(7, 70, 128, 517, 16, 3, BF16, yt, 0.3, pad, offset)
    around = y._base.clone()
    into = torch.full((70, 517 + 5), 3.0, dtype=yt, device=DEV)
    out = vce.adapter_linear(y, x, a, b, index, scale, out=into[:, 2:519])
    check(out, y, x, a, b, index, scale)
    assert bool((into[:, :2] == 3).all()) and bool((into[:, 519:] == 3).all())
    vce.adapter_linear(y, x, a, b, index, scale, out=y)
    assert torch.equal(y, out)
    around[:, offset:offset + 517] = y
    assert torch.equal(around, y._base)


@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("n,v,r,count,none,pad,offset", [(40, 32001, 8, 40, 0.0, 0, 0), (70, 32000, 16, 40, 0.0, 0, 0),
                                                         (150, 32004, 32, 50, 0.3, 3, 1), (600, 16001, 24, 60, 0.1, 0, 3),
                                                         (600, 16000, 32, 60, 0.1, 8, 8), (128, 40000, 8, 33, 0.5, 8, 0)])
def test_much_work_of_few_tokens(n, v, r, count, none, pad, offset, yt):
    """More logits of more adapters than there are blocks for at once, half of the tokens with one adapter."""
    y, x, a, b, index, scale = make(n + r, n, 264, v, r, count, F32 if n == 128 else BF16, yt, none, pad, offset)
    index[:n // 2:2] = 1
    out = vce.adapter_linear(y, x, a, b, index, scale)
    check(out, y, x, a, b, index, scale)
    for i in (0, 1, n - 1):  # by itself, which is little work
        assert torch.equal(vce.adapter_linear(y[i:i + 1], x[i:i + 1], a, b, index[i:i + 1], scale)[0], out[i])
    base = y.storage_offset(), y._base if y._base is not None else y
    around = base[1].clone()
    place = around[:, offset:offset + v] if pad or offset else around
    vce.adapter_linear(place, x, a, b, index, scale, out=place)
    assert torch.equal(place, out)
    if pad or offset:  # what lies between rows stays
        assert torch.equal(around[:, :offset], base[1][:, :offset]) and torch.equal(around[:, offset + v:], base[1][:, offset + v:])


@pytest.mark.parametrize("n", [1, 2, 31, 127, 128, 129, 255, 256, 257])
def test_tokens_of_one_adapter_and_of_none(n):
    """Tiles that are full, and the border at which the tokens are sorted in another kernel."""
    y, x, a, b, index, scale = make(n, n, 64, 300, 16, 3, BF16, F32, 0.0)
    for which in (torch.full_like(index, 2), torch.full_like(index, -1),
                  torch.where(torch.arange(n, device=DEV) < 65, 1, -1).int(), torch.where(torch.arange(n, device=DEV) < 64, -1, 0).int(),
                  (torch.arange(n, device=DEV) % 4 - 1).int()):
        out = vce.adapter_linear(y, x, a, b, which, scale)
        check(out, y, x, a, b, which, scale)
        place = y.clone()
        assert torch.equal(vce.adapter_linear(place, x, a, b, which, scale, out=place), out)


def test_a_token_does_not_depend_on_its_neighbours():
    y, x, a, b, index, scale = make(3, 300, 264, 1003, 16, 4, BF16, F32)
    out = vce.adapter_linear(y, x, a, b, index, scale)
    order = torch.randperm(300, generator=torch.Generator().manual_seed(1)).to(DEV)
    again = vce.adapter_linear(y[order], x[order], a, b, index[order], scale)
    assert torch.equal(again, out[order])
    for n in (0, 17, 299):
        assert torch.equal(vce.adapter_linear(y[n:n + 1], x[n:n + 1], a, b, index[n:n + 1], scale)[0], out[n])


def test_indexes_outside_the_adapters():
    y, x, a, b, index, scale = make(4, 9, 64, 100, 8, 2, BF16, F32, 0.0)
    index[:] = torch.tensor([0, 1, -1, 2, -2, 1, 2 ** 31 - 1, -2 ** 31, 0], dtype=torch.int32)
    for place in (False, True):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        src = y.clone()
        out = vce.adapter_linear(src, x, a, b, index, scale, out=src if place else None, dev_status=st)
        assert int(st) == vce.DEVSTATUS_BAD_INDEX
        fine = index.clone()
        fine[(index < -1) | (index >= 2)] = -1
        check(out, y, x, a, b, fine, scale)
        st.zero_()
        assert torch.equal(vce.adapter_linear(y, x, a, b, fine, scale, dev_status=st), out) and int(st) == 0
    none = torch.full_like(index, -1)
    assert torch.equal(vce.adapter_linear(y, x, a, b, none, scale), y)
    assert torch.equal(vce.adapter_linear(src, x, a, b, none, scale, out=src), out)
    assert vce.adapter_linear(y[:0], x[:0], a, b, index[:0]).shape == (0, 100)


def test_values_beyond_finite():
    """An infinity or a NaN of one token stays with it; so do the largest finite values."""
    for xt in (BF16, F32):
        y, x, a, b, index, scale = make(5, 40, 64, 200, 8, 2, xt, F32, 0.0)
        clean = vce.adapter_linear(y, x, a, b, index, scale)
        z, u = y.clone(), x.clone()
        u[3, 5], u[4, 6], u[5] = math.inf, math.nan, 0.0
        z[6, 7], z[7, 8] = -math.inf, math.nan
        u[8] = torch.finfo(xt).max * 2.0 ** -20
        out = vce.adapter_linear(z, u, a, b, index, scale)
        assert not torch.isfinite(out[3]).any() and torch.isnan(out[4]).all() and torch.equal(out[5], y[5])
        rest = [i for i in range(40) if i not in (3, 4, 5, 6, 7, 8)]
        assert torch.equal(out[rest], clean[rest])
        assert out[6, 7] == -math.inf and torch.isnan(out[7, 8])
        out[6, 7] = clean[6, 7]
        assert torch.equal(out[6], clean[6]) and torch.isfinite(out[8]).all()


def test_a_nan_whose_leading_half_is_an_infinity():
    y, x, a, b, index, scale = make(6, 3, 64, 40, 8, 1, F32, F32, 0.0)
    x[1, 9:10] = torch.tensor([0x7f800001], dtype=torch.int32, device="cuda").view(F32)
    out = vce.adapter_linear(y, x, a, b, index, scale)
    assert torch.isnan(out[1]).all() and torch.isfinite(out[::2]).all()


def test_captured_and_on_another_stream():
    y, x, a, b, index, scale = make(6, 33, 128, 700, 16, 3, BF16, BF16)
    want = vce.adapter_linear(y, x, a, b, index, scale)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(vce.adapter_workspace_size(33, 3, 16), dtype=torch.uint8, device=DEV)
    got = vce.adapter_linear(y, x, a, b, index, scale, workspace=ws, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    with pytest.raises(vce.VceError):
        vce.adapter_linear(y, x, a, b, index, scale, workspace=ws[:-1])
    yin, iin = torch.zeros_like(y), torch.full_like(index, -1)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vce.adapter_linear(yin, x, a, b, iin, scale)
    for idx in (index, index.flip(0).contiguous(), torch.zeros_like(index)):
        yin.copy_(y), iin.copy_(idx)
        graph.replay()
        assert torch.equal(out, vce.adapter_linear(y, x, a, b, idx, scale))


@pytest.mark.parametrize("n,v,r,count", [(5, 300, 16, 3), (200, 1001, 64, 3), (300, 32001, 16, 70)])
def test_workspace_of_two_graphs(n, v, r, count):
    """Two captured calls of different sizes in one workspace, whatever it holds, replayed in turn."""
    calls = [make(n + i, n - i, 264, v, r, count, BF16, F32) for i in (0, 2)]
    want = [vce.adapter_linear(*c) for c in calls]
    ws = torch.full((vce.adapter_workspace_size(n, count, r),), 255, dtype=torch.uint8, device=DEV)
    outs, graphs = [torch.empty_like(w) for w in want], [torch.cuda.CUDAGraph() for _ in calls]
    for c, o, g in zip(calls, outs, graphs):
        with torch.cuda.graph(g):
            vce.adapter_linear(*c, out=o, workspace=ws)
    for which in (0, 1, 1, 0):
        ws.random_(0, 255)
        outs[which].zero_()
        graphs[which].replay()
        assert torch.equal(outs[which], want[which])


def test_beyond_2_31_elements():
    """Logits and factors of more than 2^31 elements: their last rows."""
    n, v = 17000, 128264
    y = torch.zeros(n, v, dtype=BF16, device=DEV)
    assert y.numel() > 1 << 31
    a = torch.zeros(150, 128, 8, dtype=BF16, device=DEV)
    b = torch.zeros(150, v, 128, dtype=BF16, device=DEV)
    assert b.numel() > 1 << 31
    a[149, 127, 7], b[149, v - 1, 127], b[149, 5, 127] = 2.0, 3.0, -1.0
    x = torch.zeros(n, 8, dtype=BF16, device=DEV)
    x[n - 1, 7], x[3, 7] = 1.0, 2.0
    index = torch.full((n,), -1, dtype=torch.int32, device=DEV)
    index[n - 1], index[3], index[4] = 149, 149, 0
    vce.adapter_linear(y, x, a, b, index, out=y)
    assert y[n - 1, v - 1] == 6 and y[n - 1, 5] == -2 and y[3, v - 1] == 12 and y[3, 5] == -4
    assert int((y != 0).sum()) == 4


# ---------------------------------------------------------------------------
# the head with its adapters
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_head(norm, dtype):
    """linear_sample and linear_beam with adapters are their parts; a search's step with them."""
    g = torch.Generator().manual_seed(11)
    b, k, h, v = 3, 4, 256, 1003
    emb = torch.randn(b, k, h, generator=g).to(dtype).to(DEV)
    res = torch.randn(b, k, h, generator=g).to(dtype).to(DEV) if norm else None
    w = (1 + 0.1 * torch.randn(h, generator=g)).to(DEV) if norm else None
    w4 = vce.mx_quantize((torch.randn(v, h, generator=g) * h ** -0.5).to(DEV), "e2m1")
    _, _, a, bb, index, scale = make(12, b * k, h, v, 16, 5, dtype, F32)
    adapters = vce.Adapters(a, bb, scale)
    flat = emb.view(-1, h)
    if norm:
        q = vce.rms_norm_mx(flat, w, 1e-6, res.view(-1, h))
        x, q = vce.rms_norm_forward(q.h, w).y, q.y
    else:
        x, q = flat, vce.mx_quantize(flat, "e4m3")
    logits = vce.adapter_linear(vce.mx_linear(q, w4, F32), x, a, bb, index, scale)
    kw = dict(norm_weight=w, residual=res, adapters=adapters, adapter_index=index)
    u = torch.rand(b, k, generator=g).to(DEV)
    r = vce.linear_sample(emb, w4, u, 0.9, 40, norm_weight=w, residual=res, adapters=adapters, adapter_index=index)
    want = vce.ce_sample(logits.view(b, k, v), u, 0.9, 40)
    assert torch.equal(r.token, want.token) and torch.equal(r.logprob, want.logprob) and int(r.dev_status) == 0
    score = torch.randn(b, k, generator=g).to(DEV)
    ended = (torch.rand(b, k, generator=g) < 0.2).to(DEV)
    length = torch.randint(1, 9, (b, k), generator=g, dtype=torch.int32).to(DEV)
    for keep in (False, True):
        more = dict(ended=ended, length=length, end=3, length_penalty=0.6, keep_places=keep)
        r = vce.linear_beam(emb, w4, score, **more, **kw)
        want = vce.ce_beam(logits.view(b, k, v), score, **more)
        assert all(torch.equal(p, q) for p, q in zip(r[:5], want[:5])) and int(r.dev_status) == 0
        token, parent, out, done, size = ref.beam_step(logits.double().cpu().numpy().reshape(b, k, v), score.cpu().numpy(),
                                                       ended.cpu().numpy(), length.cpu().numpy(), 3, 0.6, None, keep)
        assert np.array_equal(r.token.cpu().numpy(), token) and np.array_equal(r.parent.cpu().numpy(), parent)
    without = vce.linear_beam(emb, w4, score, norm_weight=w, residual=res)
    want = vce.ce_beam(vce.mx_linear(q, w4, F32), score)
    assert torch.equal(without.token, want.token) and torch.equal(without.score, want.score)


def test_search_with_adapters_captured():
    """Answering as a user would: embeddings of the last tokens, the head with adapters, the choice,
    caches and history reordered; the whole step as one graph, replayed, against the steps one by
    one in plain torch from FP64 logits' order."""
    g = torch.Generator().manual_seed(21)
    b, k, h, v, steps = 2, 3, 128, 401, 6
    table = torch.randn(v, h, generator=g).to(BF16).to(DEV)
    w4 = vce.mx_quantize(table.float() * h ** -0.5, "e2m1")
    _, _, a, bb, _, scale = make(22, b * k, h, v, 8, 2, BF16, F32)
    index = torch.tensor([0, 0, 0, 1, 1, 1], dtype=torch.int32, device=DEV)
    adapters = vce.Adapters(a, bb, scale)

    def fresh():
        score = torch.full((b, k), -math.inf, device=DEV)
        score[:, 0] = 0
        return [score, torch.zeros(b, k, dtype=torch.bool, device=DEV), torch.zeros(b, k, dtype=torch.int32, device=DEV),
                torch.tensor([[1], [2]], device=DEV).repeat(1, k), torch.zeros(b * k, steps, dtype=torch.int64, device=DEV),
                torch.zeros(b * k, h, device=DEV)]

    def step(s, t):
        score, ended, length, last, history, state = s
        state.mul_(0.5).add_(table[last.view(-1)].float())
        r = vce.linear_beam(state.to(BF16).view(b, k, h), w4, score, ended=ended, length=length, end=0, length_penalty=0.7,
                            keep_places=True, adapters=adapters, adapter_index=index, out_score=score, out_ended=ended,
                            out_length=length)
        vce.beam_reorder([history, state], r.parent)
        last.copy_(r.token)
        history.index_copy_(1, t, r.token.view(-1, 1))
        return r

    at = [torch.tensor([t], device=DEV) for t in range(steps)]
    s = fresh()
    for t in at:
        r = step(s, t)
        assert int(r.dev_status) == 0
    # the scores are those of the histories: each hypothesis followed by itself
    state = torch.zeros(b * k, h, device=DEV)
    last = torch.tensor([[1], [2]], device=DEV).repeat(1, k).view(-1)
    total = torch.zeros(b * k, dtype=torch.float64, device=DEV)
    done = torch.zeros(b * k, dtype=torch.bool, device=DEV)
    for t in range(steps):
        state.mul_(0.5).add_(table[last].float())
        q = vce.mx_quantize(state.to(BF16), "e4m3")
        z = vce.adapter_linear(vce.mx_linear(q, w4, F32), state.to(BF16), a, bb, index, scale)
        last = s[4][:, t]
        lp = torch.log_softmax(z.double(), 1).gather(1, last[:, None])[:, 0]
        total += torch.where(done, torch.zeros_like(lp), lp)
        done |= last == 0
    # one rounding of the sum to FP32 per step
    assert (total.view(b, k) - s[0].double()).abs().max() <= steps * (2.0 ** -24 * s[0].abs().max().item() + 1e-6)
    assert torch.equal(done.view(b, k), s[1])
    c = fresh()
    t = at[0].clone()
    step(c, t)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(c, t)
    for x, y in zip(c, fresh()):
        x.copy_(y)
    for now in at:
        t.copy_(now)
        graph.replay()
    assert all(torch.equal(x, y) for x, y in zip(c, s))

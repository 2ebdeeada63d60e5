"""ce_beam and beam_reorder against their FP64 definitions.

Choices (tokens, parents, lengths, ends) are whole and equal the definition's.  A score is one
FP32 rounding (2^-24 of it) off a sum in FP64 whose only inexact part is the logarithm of the
row's sum: at worst every weight has the error of its exponential, 2^-22 for the instruction
and 2^-23 (1 + 20 / 4) for its argument, where weights below e^-20 no longer count: 1e-6."""
import math

import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import beam as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def logits(g, rows, v, dtype, pad=0, offset=0, std=2.0):
    z = torch.randn(rows, v, generator=g) * std + 8.0 * torch.rand(rows, v, generator=g) * (
        torch.rand(rows, v, generator=g) < 3e-3)
    full = torch.zeros(rows, v + pad + offset, dtype=dtype, device=DEV)
    out = full[:, offset:offset + v]
    out.copy_(z)
    return out


def check(z, score, **kw):
    """ce_beam of these inputs against the definition, and its status."""
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = vce.ce_beam(z, score, dev_status=st, **kw)
    b, k = score.shape
    names = dict(ended="ended", length="length", end="end", length_penalty="penalty", count="count", keep_places="keep")
    args = {names[n]: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    token, parent, out, ended, length = ref.beam_step(z.double().cpu().numpy().reshape(b, k, -1), score.cpu().numpy(), **args)
    assert np.array_equal(r.token.cpu().numpy(), token)
    assert np.array_equal(r.parent.cpu().numpy(), parent)
    got = r.score.double().cpu().numpy()
    assert np.array_equal(np.isfinite(got), np.isfinite(out))
    fine = np.isfinite(out)
    assert (np.abs(got[fine] - out[fine]) <= 2.0 ** -24 * np.abs(out[fine]) + 1e-6).all()
    if r.ended is not None:
        assert np.array_equal(r.ended.cpu().numpy(), ended)
    if r.length is not None:
        assert np.array_equal(r.length.cpu().numpy(), length)
    return r, int(st)


SHAPES = [(1, 1, 1), (1, 2, 3), (2, 3, 7), (3, 4, 33), (2, 5, 1001), (1, 4, 128256), (5, 8, 32001), (40, 2, 4099),
          (1, 3, 262145), (1, 1, 1 << 20), (90, 8, 300), (2, 32, 513)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_choice(shape, dtype):
    b, k, v = shape
    g = torch.Generator().manual_seed(b * 1000 + k * 10 + v)
    z = logits(g, b * k, v, dtype)
    score = (-20 + 3 * torch.randn(b, k, generator=g)).to(DEV)
    for count in sorted({1, k, min(64, 2 * k)}):
        assert check(z, score, count=count)[1] == 0
    ended = (torch.rand(b, k, generator=g) < 0.3).to(DEV)
    length = torch.randint(0, 50, (b, k), generator=g, dtype=torch.int32).to(DEV)
    end = v // 2
    for penalty in (0.0, 0.7, -1.0):
        check(z, score, ended=ended, length=length, end=end, length_penalty=penalty)
        check(z, score, ended=ended, length=length, end=end, length_penalty=penalty, keep_places=True)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("pad,offset", [(0, 1), (3, 2), (1, 5), (8, 8), (0, 7)])
def test_strided_rows(pad, offset, dtype):
    g = torch.Generator().manual_seed(pad * 10 + offset)
    for v in (5, 17, 4100, 50257):
        z = logits(g, 6, v, dtype, pad, offset)
        check(z, torch.randn(2, 3, generator=g).to(DEV), count=6)


@pytest.mark.parametrize("v", [64, 1001, 40003])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_beams_take_the_lowest_first(v, dtype):
    """Equal rows at different alignments have equal sums, bit for bit."""
    g = torch.Generator().manual_seed(v)
    for pad in (0, 1, 2, 5):
        z = logits(g, 8, v, dtype, pad)
        z.copy_(z[:1].clone().expand(8, v))
        check(z, torch.full((1, 8), -3.0, device=DEV), count=16)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_equal_logits(dtype):
    """Rows of one value, of two, and of a value that few groups of threads hold."""
    v = 50000
    z = torch.zeros(4, v, dtype=dtype, device=DEV)
    z[1, ::2] = 1.0
    z[2, v // 2:] = -1.0
    z[3] = -math.inf
    z[3, 4096:8192] = 0.5
    for count in (4, 8, 64):
        check(z, torch.zeros(1, 4, device=DEV), count=count)
        check(z, torch.zeros(4, 1, device=DEV), count=count)
    up = torch.linspace(-3, 3, v, device=DEV).to(dtype).repeat(2, 1)  # every element a new best one
    check(up, torch.zeros(2, 1, device=DEV), count=7)
    check(torch.full((2, 9), 0.25, dtype=dtype, device=DEV), torch.zeros(1, 2, device=DEV), count=64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_logits_that_fp64_does_not_tell_apart(dtype):
    """0 and 1e-30 beside a logit of 5: the same sum, but the order of the logits, in any part of the row."""
    v = 40000
    z = torch.zeros(2, v, dtype=dtype, device=DEV)
    z[0, 100], z[1, 5] = 5.0, 5.0
    z[0, 39000], z[0, 17], z[0, 20000] = 2e-30, 1e-30, 1e-30
    z[1, 39999], z[1, 38000] = 1e-30, -1e-30
    for shape in ((1, 2), (2, 1)):
        for count in (3, 6, 40):
            check(z, torch.zeros(shape, device=DEV), count=count)
    wide = z.repeat(16, 1)
    check(wide, torch.zeros(1, 32, device=DEV), count=64)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_masks(dtype):
    """-inf and the type's lowest value as masks; fewer allowed tokens than wanted; no allowed ones."""
    g = torch.Generator().manual_seed(2)
    v, low = 5000, torch.finfo(dtype).min
    for mask in (-math.inf, low):
        z = logits(g, 4, v, dtype)
        z[:, torch.rand(v, generator=g).to(DEV) < 0.95] = mask
        z[2] = mask
        z[2, 77] = 1.0
        assert check(z, torch.randn(2, 2, generator=g).to(DEV), count=4)[1] == 0
        z[1] = mask
        _, st = check(z, torch.randn(2, 2, generator=g).to(DEV), count=4)
        assert st == (vce.DEVSTATUS_BAD_ROW if mask == -math.inf else 0)
        z[:] = mask
        check(z, torch.zeros(2, 2, device=DEV), count=2)
    z = logits(g, 4, v, dtype)
    score = torch.randn(2, 2, generator=g).to(DEV)
    for bad in (math.nan, math.inf):
        y = z.clone()
        y[1, 3000] = bad
        r, st = check_bad(y, score, 1)
        assert st == vce.DEVSTATUS_BAD_ROW and not (r.parent[0] == 1)[r.token[0] >= 0].any()
        s = score.clone()
        s[0, 1] = bad
        r, st = check_bad(z, s, 1)
        assert st == vce.DEVSTATUS_BAD_ROW and not (r.parent[0] == 1)[r.token[0] >= 0].any()


def check_bad(z, score, row):
    """A bad beam offers nothing: as if its score were -inf."""
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    r = vce.ce_beam(z, score, dev_status=st, count=3)
    dead, fine = score.clone(), z.clone()
    dead.view(-1)[row], fine[row] = -math.inf, 0.0
    other = vce.ce_beam(fine, dead, count=3)
    assert all(torch.equal(p, q) for p, q in zip(r[:3], other[:3]))
    return r, int(st)


def test_dead_beams_are_not_read():
    z = torch.full((4, 1000), math.nan, device=DEV)
    z[0] = torch.linspace(0, 5, 1000, device=DEV)
    z[3] = torch.linspace(5, 0, 1000, device=DEV)
    score = torch.tensor([[0.0, -math.inf], [-math.inf, -1.0]], device=DEV)
    assert check(torch.nan_to_num(z), score, count=4)[1] == 0
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    a, c = vce.ce_beam(z, score, count=4, dev_status=st), vce.ce_beam(torch.nan_to_num(z), score, count=4)
    assert int(st) == 0 and all(torch.equal(p, q) for p, q in zip(a[:3], c[:3]))
    every = torch.full((2, 2), -math.inf, device=DEV)
    r, bad = check(torch.nan_to_num(z), every)
    assert bad == 0 and (r.token == -1).all() and r.parent.tolist() == [[0, 1], [0, 1]]
    ended = torch.tensor([[True, False], [True, True]], device=DEV)
    score = torch.tensor([[-1.0, -math.inf], [-math.inf, math.nan]], device=DEV)
    st.zero_()
    r = vce.ce_beam(z, score, ended=ended, end=7, dev_status=st)
    assert int(st) == vce.DEVSTATUS_BAD_ROW  # the NaN
    assert r.token.tolist() == [[7, -1], [-1, -1]] and r.ended.tolist() == [[True, False], [False, False]]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("std", [0.0, 0.1, 1.0, 4.0])
def test_sum_is_good_to_far_more_than_fp32(dtype, std):
    """With the score at minus the chosen token's log probability the result is what is wrong with
    the sum.  The mean square over rows: independent roundings of weights (2^-24 of each and of
    arguments up to 20, 2^-22 of the instruction) average over the weights that count; equal
    weights (std 0) have equal errors, at most those of the instruction at 0, which is exact."""
    g = torch.Generator().manual_seed(5)
    n, v = 64, 128256
    z = logits(g, n, v, dtype, std=std) if std else torch.full((n, v), 1.0, dtype=dtype, device=DEV)
    zd = z.double()
    lp = (zd.amax(1) - zd.logsumexp(1))
    s = -lp.float()
    r = vce.ce_beam(z, s[:, None].contiguous(), count=1)
    err = (r.score[:, 0].double() - (s.double() + lp)).cpu().numpy()
    assert np.sqrt((err ** 2).mean()) <= 1e-7, np.sqrt((err ** 2).mean())
    print(f"rms error of the sum's logarithm: {np.sqrt((err ** 2).mean()):.2e}, mean {err.mean():.2e}")


def test_in_place_and_captured():
    """A search whose state is updated in place, eagerly and as one replayed graph."""
    g = torch.Generator().manual_seed(9)
    b, k, v, steps = 3, 4, 2003, 5
    z = [logits(g, b * k, v, BF16) for _ in range(steps)]
    start = torch.full((b, k), -math.inf)
    start[:, 0] = 0.0

    def state():
        return (start.to(DEV), torch.zeros(b, k, dtype=torch.bool, device=DEV),
                torch.zeros(b, k, dtype=torch.int32, device=DEV))

    def step(zi, s, keep):
        return vce.ce_beam(zi, s[0], ended=s[1], length=s[2], end=5, length_penalty=0.5, keep_places=keep,
                           out_score=s[0], out_ended=s[1], out_length=s[2])

    for keep in (False, True):
        cur, eager = state(), []
        fresh = state()
        for zi in z:
            r = vce.ce_beam(zi, fresh[0], ended=fresh[1], length=fresh[2], end=5, length_penalty=0.5, keep_places=keep)
            fresh = (r.score, r.ended, r.length)
            q = step(zi, cur, keep)
            assert q.score is cur[0] and all(torch.equal(x, y) for x, y in zip(q[:5], r[:5]))
            eager.append([x.clone() for x in q[:5]])
        zin, cur = z[0].clone(), state()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            q = step(zin, cur, keep)
        for t, x in zip(cur, state()):
            t.copy_(x)
        for zi, want in zip(z, eager):
            zin.copy_(zi)
            graph.replay()
            assert all(torch.equal(x, y) for x, y in zip(q[:5], want))


def test_streams_and_workspace():
    g = torch.Generator().manual_seed(3)
    z, score = logits(g, 8, 3001, F32), torch.randn(2, 4, generator=g).to(DEV)
    want = vce.ce_beam(z, score)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    ws = torch.empty(vce.ce_beam_workspace_size(2, 4, 4), dtype=torch.uint8, device=DEV)
    got = vce.ce_beam(z, score, stream=side, workspace=ws)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want[:3], got[:3]))
    with pytest.raises(vce.VceError):
        vce.ce_beam(z, score, workspace=ws[:-1])
    out = vce.ce_beam(torch.zeros(0, 10, device=DEV), torch.zeros(0, 3, device=DEV))
    assert out.token.shape == (0, 3)


@pytest.mark.parametrize("shapes", [((2, 4, 3001), (1, 4, 2000)), ((20, 6, 32001), (3, 8, 128256)), ((1, 1, 300000), (2, 32, 513))])
def test_workspace_of_two_graphs(shapes):
    """Two captured calls in one workspace, whatever it holds, replayed in turn."""
    g = torch.Generator().manual_seed(8)
    calls = [(logits(g, b * k, v, t), torch.randn(b, k, generator=g).to(DEV)) for (b, k, v), t in zip(shapes, (BF16, F32))]
    want = [vce.ce_beam(*c) for c in calls]
    ws = torch.empty(max(vce.ce_beam_workspace_size(*c[1].shape, c[1].shape[1]) for c in calls), dtype=torch.uint8, device=DEV)
    got, graphs = [], [torch.cuda.CUDAGraph() for _ in calls]
    for c, graph in zip(calls, graphs):
        with torch.cuda.graph(graph):
            got.append(vce.ce_beam(*c, workspace=ws))
    for which in (0, 1, 1, 0):
        ws.random_(0, 255)
        got[which].token.zero_(), got[which].parent.zero_(), got[which].score.zero_()
        graphs[which].replay()
        assert all(torch.equal(p, q) for p, q in zip(want[which][:3], got[which][:3]))


# ---------------------------------------------------------------------------
# states
# ---------------------------------------------------------------------------

def fill(g, shape, dtype):
    n = math.prod(shape)
    size = torch.empty(0, dtype=dtype).element_size()
    return torch.randint(0, 2 if dtype is torch.bool else 256, (n * size,), generator=g,
                         dtype=torch.uint8).view(dtype).view(shape).to(DEV)


def same(t, want):
    return np.array_equal(t.contiguous().cpu().view(torch.uint8).numpy(), np.ascontiguousarray(want).view(np.uint8))


def as_bytes(t):  # numpy's view of a state: bytes in the last dimension
    t = t.contiguous().cpu()
    return t.view(torch.uint8).numpy().reshape(*t.shape, t.element_size())


@pytest.mark.parametrize("beams", [1, 2, 4, 5, 8, 13, 16, 31, 32])
@pytest.mark.parametrize("place", [True, False])
def test_reorder(beams, place):
    g = torch.Generator().manual_seed(beams)
    for batch, tail, dim, dtype in ((1, (7,), 1, torch.int64), (3, (2, 9, 24), 2, BF16), (2, (33, 3, 8), 1, F32),
                                    (5, (1, 1), 1, torch.uint8), (2, (3, 5, 7), 2, torch.uint8), (3, (4, 300, 5), 2, BF16),
                                    (2, (), None, F32), (2, (2, 4100, 2), 2, torch.float16), (4, (0, 3), None, F32),
                                    (300, (2, 3), 1, torch.int16), (1, (2, 700, 64), 2, torch.bool)):
        x = fill(g, (batch * beams, *tail), dtype)
        parent = torch.randint(0, beams, (batch, beams), generator=g)
        before = as_bytes(x)
        for lengths in (None,) if dim is None else (None, torch.randint(-1, tail[dim - 1] + 2, (batch,), generator=g,
                                                                        dtype=torch.int32)):
            src = torch.from_numpy(before.copy()).view(-1).to(DEV).view(dtype).view(x.shape)
            out = None if place else fill(g, x.shape, dtype)
            kept = None if place else as_bytes(out)
            st = torch.zeros(1, dtype=torch.int32, device=DEV)
            r = vce.beam_reorder(src, parent.to(DEV), lengths=None if lengths is None else lengths.to(DEV),
                                 position_dim=dim, out=out, dev_status=st)
            assert r is (src if place else out) and int(st) == 0
            moved = ref.reorder(before, parent.numpy(), None if lengths is None else lengths.numpy(), dim)
            if not place and lengths is not None:  # what lies behind the lengths stays as it was in out
                for i in range(batch * beams):
                    n = max(0, int(lengths[i // beams]))
                    at = (slice(None),) * (dim - 1) + (slice(n, None),)
                    moved[i][at] = kept[i][at]
            assert np.array_equal(as_bytes(r), moved)
            if not place:
                assert np.array_equal(as_bytes(src), before)


def test_reorder_many_states_and_layouts():
    g = torch.Generator().manual_seed(1)
    b, k = 3, 4
    parent = torch.tensor([[0, 0, 2, 1], [3, 2, 1, 0], [0, 1, 2, 3]])
    lengths = torch.tensor([5, 9, 3], dtype=torch.int32)
    states, dims, want = [], [], []
    for i in range(140):  # more than one launch takes
        if i % 4 == 0:
            x, dim = fill(g, (b * k, 2, 10, 8), BF16), 2
        elif i % 4 == 1:
            x, dim = fill(g, (2, b * k, 9, 4), F32).transpose(0, 1), 2      # blocks outside rows
        elif i % 4 == 2:
            x, dim = fill(g, (b * k, 3, 16, 6), BF16)[:, 1:, :11], 2         # a part of a larger cache
        else:
            x, dim = fill(g, (b * k, 12), torch.int64)[:, 1:10], 1           # off 16-byte boundaries
        states.append(x), dims.append(dim)
        want.append(ref.reorder(as_bytes(x), parent.numpy(), lengths.numpy(), dim))
    r = vce.beam_reorder(states, parent.to(DEV), lengths=lengths.to(DEV), position_dim=dims)
    assert all(np.array_equal(as_bytes(x), y) for x, y in zip(r, want))
    assert vce.beam_reorder([], parent.to(DEV)) == []


def test_reorder_bad_parents_stay():
    x = torch.arange(12, device=DEV).view(6, 2)
    for place in (True, False):
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        src = x.clone()
        out = None if place else torch.zeros_like(src)
        r = vce.beam_reorder(src, torch.tensor([[-1, 0, 3], [2, 1 << 40, 0]], device=DEV), out=out, dev_status=st)
        assert int(st) == vce.DEVSTATUS_BAD_INDEX
        assert r[:, 0].tolist() == [0, 0, 4, 10, 8, 6]


def test_reorder_beyond_2_31_elements():
    """One state of more than 2^31 elements: the last request's beams."""
    b, k, t, d = 2, 4, 1 << 20, 288
    x = torch.empty(b * k, t, d, dtype=torch.uint8, device=DEV)
    assert x.numel() > 1 << 31
    for i in range(b * k):
        x[i] = i
        x[i, -1] = 100 + i
    vce.beam_reorder(x, torch.tensor([[0, 1, 0, 0], [1, 1, 2, 0]], device=DEV))
    rows = [0, 1, 0, 0, 5, 5, 6, 4]
    assert x[:, -2, 5].tolist() == rows and x[:, -1, d - 1].tolist() == [100 + i for i in rows]
    assert all(bool((x[i, :-1] == r).all()) for i, r in enumerate(rows))


def test_reorder_captured_with_the_choice():
    """The step a search repeats: choice, then caches and history in place, as one graph."""
    g = torch.Generator().manual_seed(4)
    b, k, v, t = 2, 3, 501, 6
    z = logits(g, b * k, v, F32)
    score = torch.randn(b, k, generator=g).to(DEV)
    cache, history = fill(g, (b * k, 2, t, 8), BF16), fill(g, (b * k, t), torch.int64)
    lengths = torch.tensor([4, 6], dtype=torch.int32, device=DEV)
    keep = (score.clone(), cache.clone(), history.clone())

    def step():
        r = vce.ce_beam(z, score, keep_places=True, out_score=score)
        vce.beam_reorder([cache, history], r.parent, lengths=lengths, position_dim=[2, 1])
        return r

    r = step()
    want = [x.clone() for x in (r.parent, score, cache, history)]
    assert np.array_equal(as_bytes(cache), ref.reorder(as_bytes(keep[1]), r.parent.cpu().numpy(), lengths.cpu().numpy(), 2))
    for x, y in zip((score, cache, history), keep):
        x.copy_(y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        r = step()
    for _ in range(2):
        for x, y in zip((score, cache, history), keep):
            x.copy_(y)
        graph.replay()
        assert all(torch.equal(x, y) for x, y in zip((r.parent, score, cache, history), want))

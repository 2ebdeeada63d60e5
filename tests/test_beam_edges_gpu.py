"""ce_beam and beam_reorder where they can go wrong at the edges: equal hypotheses, what a workspace
holds, logits far from zero, penalties and lengths at the border of their types.  Scores are held to
tests/test_beam_gpu.py's bound: one FP32 rounding, and 1e-6 of the sum's logarithm."""
import math

import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import beam as ref

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
BF16, F32 = torch.bfloat16, torch.float32


def logits(g, rows, v, dtype):
    z = torch.randn(rows, v, generator=g) * 2 + 8.0 * torch.rand(rows, v, generator=g) * (
        torch.rand(rows, v, generator=g) < 3e-3)
    return z.to(dtype).to(DEV)


def check(z, score, workspace=None, **kw):
    """ce_beam of these inputs against the definition."""
    r = vce.ce_beam(z, score, workspace=workspace, **kw)
    b, k = score.shape
    names = dict(ended="ended", length="length", end="end", length_penalty="penalty", count="count", keep_places="keep")
    args = {names[n]: v.cpu().numpy() if isinstance(v, torch.Tensor) else v for n, v in kw.items()}
    want = ref.beam_step(z.double().cpu().numpy().reshape(b, k, -1), score.cpu().numpy(), **args)
    assert np.array_equal(r.token.cpu().numpy(), want[0]) and np.array_equal(r.parent.cpu().numpy(), want[1])
    got, out = r.score.double().cpu().numpy(), want[2]
    fine = np.isfinite(out)
    assert np.array_equal(np.isfinite(got), fine)
    assert (np.abs(got[fine] - out[fine]) <= 2.0 ** -24 * np.abs(out[fine]) + 1e-6).all()
    assert r.ended is None or np.array_equal(r.ended.cpu().numpy(), want[3])
    assert r.length is None or np.array_equal(r.length.cpu().numpy(), want[4])
    return r


@pytest.mark.parametrize("fill", [0, 255])
@pytest.mark.parametrize("keep", [False, True])
@pytest.mark.parametrize("k,v", [(2, 9), (4, 1001), (6, 40000), (8, 128256)])
def test_equal_ended_beams_in_any_workspace(k, v, keep, fill):
    """Ended beams of equal score beside live ones, whatever the workspace holds: the lowest beam comes first."""
    g = torch.Generator().manual_seed(k)
    z = logits(g, 4 * k, v, F32)
    z[-1] = -math.inf
    z[-1, 7] = 1.0  # offers one token
    score = torch.full((4, k), -2.0, device=DEV)
    score[1, 0], score[2, -1], score[3, -1] = -30.0, -1.0, -2.5
    ended = torch.ones(4, k, dtype=torch.bool, device=DEV)
    ended[0, -1], ended[1, 0], ended[3, -1] = False, False, False  # two and more ended ones beside a live one
    length = torch.full((4, k), 3, dtype=torch.int32, device=DEV)
    ws = torch.full((vce.ce_beam_workspace_size(4, k, 2 * k),), fill, dtype=torch.uint8, device=DEV)
    for kw in (dict(), dict(length=length, length_penalty=0.8)):
        check(z, score, ended=ended, end=3, keep_places=keep, **kw, workspace=ws)
        ws.fill_(fill)
        if not keep:
            check(z, score, ended=ended, end=3, count=2 * k, **kw, workspace=ws)
            ws.fill_(fill)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", [(3, 4, 1001), (12, 4, 128256), (2, 32, 513), (5, 8, 32001)])
def test_what_the_workspace_holds(shape, dtype):
    """Results do not depend on the workspace's contents: all of every byte value, bytes up to 255 among random ones."""
    b, k, v = shape
    g = torch.Generator().manual_seed(v)
    z = logits(g, b * k, v, dtype)
    score = (-5 + torch.randn(b, k, generator=g)).round().to(DEV)  # some are equal
    ended = (torch.rand(b, k, generator=g) < 0.5).to(DEV)
    length = torch.randint(1, 4, (b, k), generator=g, dtype=torch.int32).to(DEV)
    score[0, -1] = -math.inf
    ws = torch.empty(vce.ce_beam_workspace_size(b, k, k), dtype=torch.uint8, device=DEV)
    kw = dict(ended=ended, length=length, end=2, length_penalty=0.7, keep_places=True)
    for what in (0, 127, 128, 255, None):
        ws.random_(0, 256) if what is None else ws.fill_(what)
        check(z, score, **kw, workspace=ws)


SHIFTS = [3e4, -3e4, 1e5, -1e5, 1e6, -1e6, 1e7, -1e7, 3e7, -3e7, 1e8, 2.6e8, -2.6e8, 2.0 ** 30, -2.0 ** 31, 1e20]


@pytest.mark.parametrize("shift", SHIFTS)
def test_logits_far_from_zero(shift):
    """The sum's logarithm is as good where all logits of a row share a large offset (FP32 rows: a mask that is
    added, a bias), and beams whose rows differ by an offset alone are ranked by their scores.  Without a score the
    result is what the row's sum is made of: one rounding of it and the 1e-6 of the module's derivation."""
    g = torch.Generator().manual_seed(7)
    for v in (4000, 128256):
        z = (torch.randn(4, v, generator=g) * 2 + shift).to(DEV)
        z[3] = shift
        z[3, v // 2] = float(np.nextafter(np.float32(shift), np.float32(np.inf)))
        check(z, torch.zeros(4, 1, device=DEV), count=1)
        zd = z.double()
        lp = -torch.log(torch.exp(zd - zd.amax(1, keepdim=True)).sum(1))
        s = -lp.float()
        st = torch.zeros(1, dtype=torch.int32, device=DEV)
        r = vce.ce_beam(z, s[:, None].contiguous(), count=1, dev_status=st)
        # the score that remains is small: what is wrong with it is wrong with the sum
        err = (r.score[:, 0].double() - (s.double() + lp)).abs().max().item()
        assert err <= 1e-6 and int(st) == 0, err
    # differences of whole steps of the shifted logits: the shift is exact
    step = max(2.0 ** -10, 2.0 ** (math.frexp(abs(shift))[1] - 24))
    base = (torch.randn(1, 4000, generator=g) * 2 / step).round() * step
    far = base.double() + math.trunc(shift / step) * step
    assert (far.float().double() == far).all()
    z = torch.cat([base, far.float(), base, far.float()]).to(DEV)
    for score in ([-1.0, -1.00001, -1.00002, -1.00003], [-1.00003, -1.00002, -1.00001, -1.0], [-1.00002, -1.0, -1.00003, -1.00001]):
        check(z, torch.tensor([score], device=DEV), count=8)


def test_length_penalty_in_64_bits():
    """Two hypotheses whose order is another one under the penalty's nearest 32-bit number."""
    penalty, a, b = 0.8, 10, 200
    near = float(np.float32(penalty))
    pairs = []
    for i in range(400000):
        low = np.float32(-30.0 - i * 1e-5)
        high = np.float32(float(low) * (a / b) ** penalty)
        exact = float(high) / a ** penalty - float(low) / b ** penalty
        if exact * (float(high) / a ** near - float(low) / b ** near) < 0 and abs(exact) > 1e-10:
            pairs.append((high, low))
        if len(pairs) == 8:
            break
    assert len(pairs) == 8
    score = torch.tensor(np.array(pairs), device=DEV)
    length = torch.tensor([[a, b]] * 8, dtype=torch.int32, device=DEV)
    ended = torch.ones(8, 2, dtype=torch.bool, device=DEV)
    check(torch.zeros(16, 5, device=DEV), score, ended=ended, end=1, length=length, length_penalty=penalty)


@pytest.mark.parametrize("penalty", [0.0, 0.9, -0.5])
def test_the_longest_lengths(penalty):
    """A length of 2^31 - 1 is compared as one more than it is, and stays there."""
    most = 2 ** 31 - 1
    z = torch.linspace(0, 1, 10, device=DEV).repeat(4, 1)
    score = torch.tensor([[-3.0, -3.5], [-3.0, -2.0]], device=DEV)
    length = torch.tensor([[most, 4], [most - 1, most]], dtype=torch.int32, device=DEV)
    token, parent, out, _, size = ref.beam_step(z.double().cpu().numpy().reshape(2, 2, 10), score.cpu().numpy(), None,
                                                length.cpu().numpy(), penalty=penalty, count=4)
    r = vce.ce_beam(z, score, length=length, length_penalty=penalty, count=4)
    assert np.array_equal(r.token.cpu().numpy(), token) and np.array_equal(r.parent.cpu().numpy(), parent)
    assert np.array_equal(r.length.cpu().numpy(), np.minimum(size, most))


@pytest.mark.parametrize("length", [2 ** 31 - 1, 1, 0])
def test_reorder_positions_beyond_4_gb(length):
    """Positions of more than 2^32 bytes, whose product with a length does not fit 63 bits."""
    size = 2 ** 32 + 64
    assert (2 ** 31 - 1) * size >= 1 << 63
    x = torch.empty(2, 1, size, dtype=torch.uint8, device=DEV)
    x[0], x[1] = 3, 5
    parent = torch.tensor([[1, 1]], device=DEV)
    lengths = torch.tensor([length], dtype=torch.int32, device=DEV)
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    vce.beam_reorder(x, parent, lengths=lengths, position_dim=1, dev_status=st)
    want = 5 if length else 3
    assert int(st) == 0 and int(x[0].min()) == int(x[0].max()) == want and int(x[1].min()) == int(x[1].max()) == 5

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

"""adapter_linear where it can go wrong at the edges: the bits of tokens without an adapter, the terms that
t = A x is multiplied in, what a workspace holds; and a search with adapters, step by step."""
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


@pytest.mark.parametrize("yt", [BF16, F32])
@pytest.mark.parametrize("n,v,r,count,pad,offset", [(9, 300, 16, 3, 4, 0), (70, 517, 64, 3, 0, 1), (300, 264, 8, 2, 0, 0),
                                                    (70, 32000, 16, 40, 0, 0), (150, 32004, 8, 50, 3, 1)])
def test_tokens_without_an_adapter_keep_their_bits(n, v, r, count, pad, offset, yt):
    """Every bit: -0 stays -0, a NaN keeps its payload, in either form, in place or not."""
    y, x, a, b, index, scale = make(n, n, 64, v, r, count, BF16, yt, 0.0, pad, offset)
    index[::3] = -1
    bits = torch.int16 if yt is BF16 else torch.int32
    y[:, ::5] = -0.0
    y[:, 1::7] = torch.tensor([0x7f81 if yt is BF16 else 0x7f800001], dtype=bits, device=DEV).view(yt)
    want = y.contiguous().view(bits).clone()
    none = index < 0
    for out in (vce.adapter_linear(y, x, a, b, index, scale), vce.adapter_linear(y, x, a, b, index, scale, out=y)):
        assert torch.equal(out.contiguous().view(bits)[none], want[none])


@pytest.mark.parametrize("n,v,r,count,pad,offset", [(40, 264, 8, 1, 0, 0), (40, 261, 64, 2, 0, 1), (70, 32000, 16, 40, 0, 0),
                                                    (150, 32004, 8, 50, 3, 1)])
def test_two_terms_hold_17_bits(n, v, r, count, pad, offset):
    """BF16 logits take t = A x as two BF16 terms, the first rounded to 8 bits: what is left of a t of 17 bits is at
    most half of the first term's last place, 2^8 units, which 8 bits and a sign hold.  With y = -(the first term)
    that is the result, and exact."""
    y, x, a, b, index, scale = make(n, n, 64, v, r, count, F32, BF16, 0.0, pad, offset)
    g = torch.Generator().manual_seed(1)
    t = torch.randint(1 << 16, 1 << 17, (n,), generator=g) * (1 - 2 * torch.randint(0, 2, (n,), generator=g))
    t[:4] = torch.tensor([(1 << 16) + 511, -(1 << 16) - 511, (1 << 17) - 1, (1 << 16) + 257])
    t = (t.float() * 2.0 ** -16).to(DEV)
    x.zero_(), a.zero_(), b.zero_()
    x[:, 9], a[:, 3, 9], b[:, :, 3] = t, 1.0, 1.0
    y.copy_((-t.to(BF16))[:, None].expand(n, v))
    out = vce.adapter_linear(y, x, a, b, index)
    assert torch.equal(out, (t - t.to(BF16).float()).to(BF16)[:, None].expand(n, v))
    # the largest finite values do not round to an infinity
    x[:, 9] = torch.finfo(F32).max
    b[:, :, 3] = 2.0 ** -120
    out = vce.adapter_linear(torch.zeros_like(y), x, a, b, index)
    assert torch.equal(out, torch.full_like(out, 256.0))


@pytest.mark.parametrize("n,v,r,count", [(5, 300, 16, 3), (200, 1001, 64, 3), (300, 32001, 16, 70)])
def test_what_the_workspace_holds(n, v, r, count):
    """Results do not depend on the workspace's contents, bytes up to 255 among them."""
    call = make(n, n, 264, v, r, count, BF16, F32)
    want = vce.adapter_linear(*call)
    ws = torch.empty(vce.adapter_workspace_size(n, count, r), dtype=torch.uint8, device=DEV)
    for what in (0, 255, None):
        ws.random_(0, 256) if what is None else ws.fill_(what)
        assert torch.equal(vce.adapter_linear(*call, workspace=ws), want)


@pytest.mark.parametrize("keep", [False, True])
def test_every_step_of_a_search_against_the_definitions(keep):
    """A search with adapters whose every choice, and every history after it, is the definition's for that step's
    logits: product and adapters by this package, choice and reordering in FP64."""
    g = torch.Generator().manual_seed(31)
    b, k, h, v, steps = 3, 4, 128, 403, 7
    table = torch.randn(v, h, generator=g).to(BF16).to(DEV)
    w4 = vce.mx_quantize(table.float() * h ** -0.5, "e2m1")
    _, _, a, bb, _, scale = make(32, b * k, h, v, 8, 2, BF16, F32)
    index = torch.tensor([0] * k + [-1] * k + [1] * k, dtype=torch.int32, device=DEV)
    score = torch.full((b, k), -math.inf, device=DEV)
    score[:, 0] = 0
    ended = torch.zeros(b, k, dtype=torch.bool, device=DEV)
    length = torch.zeros(b, k, dtype=torch.int32, device=DEV)
    last = torch.arange(1, b + 1, device=DEV)[:, None].repeat(1, k)
    history = torch.zeros(b * k, steps, dtype=torch.int64, device=DEV)
    state = torch.zeros(b * k, h, device=DEV)
    for i in range(steps):
        state.mul_(0.5).add_(table[last.view(-1)].float())
        x = state.to(BF16)
        z = vce.adapter_linear(vce.mx_linear(vce.mx_quantize(x, "e4m3"), w4, F32), x, a, bb, index, scale)
        want = ref.beam_step(z.double().cpu().numpy().reshape(b, k, v), score.cpu().numpy(), ended.cpu().numpy(),
                             length.cpu().numpy(), 0, 0.7, None, keep)
        before = history.cpu().numpy(), state.cpu().numpy()
        r = vce.linear_beam(x.view(b, k, h), w4, score, ended=ended, length=length, end=0, length_penalty=0.7,
                            keep_places=keep, adapters=vce.Adapters(a, bb, scale), adapter_index=index, out_score=score,
                            out_ended=ended, out_length=length)
        assert int(r.dev_status) == 0
        for got, right in zip((r.token, r.parent, r.ended, r.length), (want[0], want[1], want[3], want[4])):
            assert np.array_equal(got.cpu().numpy(), right)
        assert np.allclose(r.score.cpu().numpy(), want[2], rtol=2.0 ** -24, atol=1e-6)
        vce.beam_reorder([history, state], r.parent)
        for got, was in zip((history, state), before):
            assert np.array_equal(got.cpu().numpy(), ref.reorder(was, want[1]))
        last.copy_(r.token)
        history[:, i] = r.token.view(-1)

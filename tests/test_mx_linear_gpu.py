"""The product of an E4M3 and an E2M1 microscaled matrix against the FP64 product of the
values they stand for.

Bound: products of codes are exact and the sum of h of them is FP32.  Whatever its order, a
sum of h terms is off by at most h u times the sum of magnitudes for rounded additions, u = 2^-24,
and by twice that where additions truncate; the output's own half step comes on top.
"""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24


def make(seed, rows, cols, fmt, spread=0.0):
    g = torch.Generator(DEV).manual_seed(seed)
    x = torch.randn(rows, cols, device=DEV, generator=g)
    if spread:  # blocks of very different scales
        x = x * torch.exp2(torch.randint(-int(spread), int(spread) + 1, (rows, cols // 32 + 1), device=DEV, generator=g)
                           .float().repeat_interleave(32, 1)[:, :cols])
    return vce.mx_quantize(x, fmt)


def check(x, w, dtype, out=None):
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = vce.mx_linear(x, w, dtype, out=out, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    xv, wv = vce.mx_dequantize(x, torch.float32).double(), vce.mx_dequantize(w, torch.float32).double()
    ref, mag = xv @ wv.t(), xv.abs() @ wv.abs().t()
    lim = torch.finfo(dtype).eps / 2 * ref.abs() * (1 + 1e-5) + 2 * x.cols * U * mag + 1e-45
    err = (got.double() - ref).abs()
    assert bool((err <= lim).all()), float((err / lim).max())
    return got, err, mag


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,h,v", [(1, 1, 1), (1, 128, 128), (1, 4096, 1000), (5, 96, 40), (16, 256, 129), (17, 384, 300),
                                   (32, 1000, 257), (33, 160, 4000), (64, 2056, 1000), (65, 512, 130), (100, 640, 32001),
                                   (128, 4096, 700), (129, 128, 513), (256, 1024, 5000), (257, 2056, 3001),
                                   (400, 896, 1200), (1000, 300, 2000)])
def test_shapes(n, h, v, dtype):
    check(make(n, n, h, "e4m3"), make(v, v, h, "e2m1"), dtype)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,h,v", [(1290, 384, 29002), (1290, 640, 28929), (2100, 128, 32768), (4096, 260, 32001),
                                   (1537, 1100, 40064)])
def test_many_tiles(n, h, v, dtype):
    # enough tiles for the widest ones, with an odd number of column tiles, a last tile of one
    # row, of one token, and row lengths that are and are not multiples of 16 bytes
    check(make(n, n, h, "e4m3"), make(v, v, h, "e2m1"), dtype)


@pytest.mark.parametrize("n,h,v", [(3, 1024, 300), (300, 2048, 500)])
def test_scales_of_many_sizes(n, h, v):
    check(make(1, n, h, "e4m3", 20), make(2, v, h, "e2m1", 20), torch.float32)


def test_every_scale_reaches_its_block():
    # one-hot rows: out[i, j] = x's value at column c(i) times w's there, exactly
    n, h, v = 256, 512, 384
    g = torch.Generator(DEV).manual_seed(5)
    x = torch.zeros(n, h, device=DEV)
    col = torch.randint(0, h, (n,), device=DEV, generator=g)
    x[torch.arange(n, device=DEV), col] = torch.exp2(torch.randint(-60, 60, (n,), device=DEV, generator=g).float())
    w = torch.exp2(torch.randint(-30, 30, (v, h // 32), device=DEV, generator=g).float()).repeat_interleave(32, 1)
    w = w * torch.randint(-6, 7, (v, h), device=DEV, generator=g)
    xq, wq = vce.mx_quantize(x, "e4m3"), vce.mx_quantize(w, "e2m1")
    got = vce.mx_linear(xq, wq, torch.float32)
    want = vce.mx_dequantize(xq, torch.float32).double() @ vce.mx_dequantize(wq, torch.float32).double().t()
    assert torch.equal(got.double(), want)


def test_strided_and_unaligned_output():
    x, w = make(1, 37, 256, "e4m3"), make(2, 301, 256, "e2m1")
    full = torch.full((37, 310), 7.0, dtype=torch.bfloat16, device=DEV)
    got, _, _ = check(x, w, torch.bfloat16, full[:, 3:304])
    assert torch.equal(got, vce.mx_linear(x, w))
    assert (full[:, :3] == 7).all() and (full[:, 304:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,v", [(37, 301), (200, 1), (300, 290), (300, 129)])
def test_output_rows_at_every_offset(n, v, dtype):
    # rows that start at any element, in steps of any parity: the same bits as in a plain output,
    # and nothing beside them
    x, w = make(3, n, 384, "e4m3"), make(4, v, 384, "e2m1")
    want = vce.mx_linear(x, w, dtype)
    for offset in (0, 1, 2, 7, 8, 16):
        for pad in (17, 18, 24, 32 - v % 16):
            full = torch.full((n, v + pad), 7.0, dtype=dtype, device=DEV)
            vce.mx_linear(x, w, dtype, out=full[:, offset:offset + v])
            assert torch.equal(full[:, offset:offset + v], want), (offset, pad)
            assert (full[:, :offset] == 7).all() and (full[:, offset + v:] == 7).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("n,h,v", [(250, 4700, 38900), (1000, 2100, 43600), (1921, 1300, 24100), (2000, 1300, 24200),
                                   (2048, 1400, 24320)])
def test_pairs_of_tiles(n, h, v, dtype):
    # whole rounds of tiles of 256 tokens x 256 rows on 76 pairs of SMs, long enough to be taken by
    # CTA pairs: last tiles of one token, of few rows (with and without a second tile of scales)
    rounds, k_tiles = -(-n // 256) * -(-v // 256) / 76, -(-h // 128)
    assert rounds == int(rounds) and 0.07 * rounds * k_tiles > 5
    check(make(5, n, h, "e4m3"), make(6, v, h, "e2m1"), dtype)


@pytest.mark.parametrize("n", [4, 200])
def test_nan_scales_stay_in_their_row(n):
    x = torch.randn(n, 256, device=DEV)
    w = torch.randn(300, 256, device=DEV)
    x[1, 40] = float("inf")
    w[7, 200] = float("nan")
    got = vce.mx_linear(vce.mx_quantize(x, "e4m3"), vce.mx_quantize(w, "e2m1"), torch.float32)
    nan = got.isnan()
    assert nan[1].all() and nan[:, 7].all()
    nan[1] = False
    nan[:, 7] = False
    assert not nan.any()


def test_no_tokens_and_bits_repeat():
    w = make(2, 1000, 512, "e2m1")
    assert vce.mx_linear(vce.MXTensor.empty(0, 512, "e4m3", DEV), w).shape == (0, 1000)
    x = make(1, 200, 512, "e4m3")
    a = vce.mx_linear(x, w, torch.float32)
    for _ in range(3):
        assert torch.equal(a, vce.mx_linear(x, w, torch.float32))
    # a token's logits do not depend on the tokens beside it within one width of the kernel
    first = vce.mx_quantize(vce.mx_dequantize(x, torch.float32)[:150].contiguous(), "e4m3")
    assert torch.equal(vce.mx_linear(first, w, torch.float32), a[:150])


def test_graph_replay_and_side_stream():
    x, w = make(1, 20, 512, "e4m3"), make(2, 1000, 512, "e2m1")
    vce.mx_linear(x, w)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = vce.mx_linear(x, w)
    for k in (3, 4):
        y = make(k, 20, 512, "e4m3")
        x.codes.copy_(y.codes)
        x.scales.copy_(y.scales)
        graph.replay()
        assert torch.equal(out, vce.mx_linear(y, w))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vce.mx_linear(x, w, stream=side)
    side.synchronize()
    assert torch.equal(got, vce.mx_linear(x, w))


@pytest.mark.parametrize("n", [1, 300])
def test_norm_product_and_loss_together(n):
    # hidden states -> norm in 8 bits -> product with a 4-bit classifier -> cross entropy
    h, v = 512, 3000
    g = torch.Generator(DEV).manual_seed(9)
    x = torch.randn(n, h, device=DEV, generator=g).bfloat16()
    nw = (1 + 0.1 * torch.randn(h, device=DEV, generator=g)).bfloat16()
    w = make(3, v, h, "e2m1")
    y = torch.randint(0, v, (n,), device=DEV, generator=g)
    q = vce.rms_norm_mx(x, nw).y
    z = vce.mx_linear(q, w, torch.float32)
    f = vce.ce_forward(z, y, 0.0, "mean")
    ref = vce.mx_dequantize(q, torch.float32).double() @ vce.mx_dequantize(w, torch.float32).double().t()
    loss = torch.nn.functional.cross_entropy(ref, y)
    assert abs(float(f.loss) - float(loss)) <= 1e-4 * max(1.0, float(loss))


def test_outputs_past_32_bits():
    n, v, h = 17000, 128257, 128
    x, w = make(1, n, h, "e4m3"), make(2, v, h, "e2m1")
    out = vce.mx_linear(x, w)
    last = vce.mx_quantize(vce.mx_dequantize(x, torch.float32)[-200:].contiguous(), "e4m3")
    assert torch.equal(out[-200:], vce.mx_linear(last, w))

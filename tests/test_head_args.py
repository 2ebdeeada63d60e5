"""Refusals of the operators around the cross entropy, and their FP64 definitions pinned to
torch, without a GPU: a wrong argument is an error before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import head

OK, INVALID, DTYPE, ALIGN, WORKSPACE, ARCH, CUDA = range(7)
FAKE = 0x10000  # never dereferenced: host validation fails first
P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float


@pytest.fixture(scope="module", autouse=True)
def built():
    from vocabulary_cross_entropy_gb300 import build
    build.build()


def _norm(x=FAKE, dtype=0, n=4, h=64, xs=64, res=None, rs=64, w=FAKE, wd=0, eps=1e-6, hp=None, hs=64, y=FAKE,
          ys=64, rstd=FAKE):
    return vce.library().rms_norm_forward(x, dtype, n, h, xs, res, rs, w, wd, eps, hp, hs, y, ys, rstd, None, None)


def test_norm_forward_refusals():
    assert _norm(dtype=2) == DTYPE and _norm(wd=9) == DTYPE
    for bad in (dict(n=-1), dict(h=0), dict(xs=63), dict(eps=-1.0), dict(eps=float("nan")), dict(x=None),
                dict(w=None), dict(y=None), dict(ys=63), dict(res=FAKE, hp=None), dict(res=FAKE, hp=FAKE, rs=3),
                dict(res=FAKE, hp=FAKE, hs=3), dict(n=1 << 40), dict(h=1 << 40, xs=1 << 40, ys=1 << 40)):
        assert _norm(**bad) == INVALID, bad
    for bad in (dict(x=FAKE + 1), dict(y=FAKE + 1), dict(w=FAKE + 1), dict(rstd=FAKE + 2), dict(wd=1, w=FAKE + 2)):
        assert _norm(**bad) == ALIGN, bad


def test_norm_mx_refusals():
    f = vce.library().rms_norm_mx

    def call(codes=FAKE, scales=FAKE, dtype=0):
        return f(FAKE, dtype, 4, 64, 64, None, 0, FAKE, 0, 1e-6, None, 0, codes, scales, None, None, None)

    assert call(dtype=5) == DTYPE
    assert call(codes=None) == INVALID and call(scales=None) == INVALID
    assert call(codes=FAKE + 8) == ALIGN and call(scales=FAKE + 4) == ALIGN


def test_norm_backward_refusals():
    f = vce.library().rms_norm_backward

    def call(dy=FAKE, dtype=0, n=4, h=64, gs=64, hp=FAKE + 256, hs=64, w=FAKE, wd=0, rstd=FAKE, dh=None, ds=64,
             dx=FAKE, xs=64, dw=FAKE, ws=FAKE, size=1 << 30):
        return f(dy, dtype, n, h, gs, hp, hs, w, wd, rstd, dh, ds, dx, xs, dw, ws, size, None, None)

    assert call(dtype=3) == DTYPE and call(wd=3) == DTYPE
    for bad in (dict(n=-1), dict(h=0), dict(gs=1), dict(hs=1), dict(xs=1), dict(dh=FAKE, ds=1), dict(dy=None),
                dict(hp=None), dict(w=None), dict(rstd=None), dict(dx=None), dict(dw=None), dict(dx=FAKE + 256)):
        assert call(**bad) == INVALID, bad
    assert call(dy=FAKE + 1) == ALIGN and call(ws=FAKE + 128) == ALIGN
    assert call(ws=None) == WORKSPACE


def test_mx_refusals():
    lib = vce.library()

    def q(x=FAKE, dtype=0, n=4, c=64, s=64, fmt=0, codes=FAKE, scales=FAKE, fn=lib.mx_quantize):
        if fn is lib.mx_quantize:
            return fn(x, dtype, n, c, s, fmt, codes, scales, None, None)
        return fn(codes, scales, fmt, n, c, x, dtype, s, None, None)

    for fn in (lib.mx_quantize, lib.mx_dequantize):
        assert q(dtype=2, fn=fn) == DTYPE and q(fmt=2, fn=fn) == DTYPE
        for bad in (dict(n=-1), dict(c=0), dict(s=63), dict(x=None), dict(codes=None), dict(scales=None)):
            assert q(**bad, fn=fn) == INVALID, bad
        for bad in (dict(x=FAKE + 1), dict(codes=FAKE + 8), dict(scales=FAKE + 8)):
            assert q(**bad, fn=fn) == ALIGN, bad
    assert vce.mx_codes_size(3, 129, "e4m3") == 3 * 256 and vce.mx_codes_size(3, 129, "e2m1") == 3 * 128
    assert vce.mx_scales_size(129, 129) == 256 * 8 and vce.mx_scales_size(0, 5) == 0


def test_mx_linear_refusals():
    f = vce.library().mx_linear

    def call(xc=FAKE, xs=FAKE, wc=FAKE, ws=FAKE, n=4, h=64, v=100, out=FAKE, dtype=0, stride=100):
        return f(xc, xs, wc, ws, n, h, v, out, dtype, stride, None, None)

    assert call(dtype=2) == DTYPE
    for bad in (dict(n=-1), dict(h=0), dict(v=0), dict(stride=99), dict(xc=None), dict(xs=None), dict(wc=None),
                dict(ws=None), dict(out=None), dict(n=1 << 40), dict(v=1 << 40, stride=1 << 40)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(xc=FAKE + 8), dict(xs=FAKE + 8), dict(wc=FAKE + 8), dict(ws=FAKE + 8), dict(out=FAKE + 1)):
        assert call(**bad) == ALIGN, bad
    x, w = vce.MXTensor.empty(4, 64, "e4m3", "cpu"), vce.MXTensor.empty(9, 64, "e2m1", "cpu")
    with pytest.raises(ValueError, match="CUDA"):
        vce.mx_linear(x, w)
    for pair in ((w, w), (x, x), (x, vce.MXTensor.empty(9, 65, "e2m1", "cpu"))):
        with pytest.raises(ValueError):
            vce.mx_linear(*pair)
    with pytest.raises(ValueError):
        vce.mx_linear(x, w, out=torch.zeros(4, 8, dtype=torch.bfloat16))


def test_sample_refusals():
    f = vce.library().ce_sample

    def call(z=FAKE, dtype=0, n=4, v=100, stride=100, u=FAKE, t=None, k=None, p=None, m=None, tok=FAKE, lp=None):
        return f(z, dtype, n, v, stride, u, t, k, p, m, tok, lp, None, None)

    assert call(dtype=2) == DTYPE
    for bad in (dict(n=-1), dict(v=0), dict(stride=99), dict(z=None), dict(u=None), dict(tok=None),
                dict(v=(1 << 20) + 1, stride=1 << 21)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(z=FAKE + 1), dict(u=FAKE + 2), dict(t=FAKE + 1), dict(k=FAKE + 1), dict(p=FAKE + 1),
                dict(m=FAKE + 1), dict(tok=FAKE + 4), dict(lp=FAKE + 1)):
        assert call(**bad) == ALIGN, bad
    z, u = torch.zeros(4, 10), torch.zeros(4)
    with pytest.raises(ValueError, match="CUDA"):
        vce.ce_sample(z, u)
    for kw in (dict(temperature=torch.zeros(3)), dict(top_k=torch.zeros(4)), dict(top_p=torch.zeros(4).double()),
               dict(min_p=torch.zeros(4, 2)[:, 0]), dict(token=torch.zeros(4, dtype=torch.int32))):
        with pytest.raises(ValueError):
            vce.ce_sample(z, u, **kw)
    with pytest.raises(ValueError):
        vce.ce_sample(z, u[:3])
    with pytest.raises(TypeError):
        vce.ce_sample(z.double(), u)
    with pytest.raises(ValueError):
        vce.linear_sample(z, vce.MXTensor.empty(9, 10, "e2m1", "cpu"), u, residual=z)


def test_linear_sample_checks_before_it_launches(monkeypatch):
    from vocabulary_cross_entropy_gb300 import _head
    x, w = torch.zeros(4, 64), vce.MXTensor.empty(9, 64, "e2m1", "cpu")
    u = torch.zeros(4)

    class Launched(Exception):
        pass

    def launched(*args, **kwargs):
        raise Launched

    for name in ("rms_norm_mx", "mx_quantize", "flat_rows"):
        monkeypatch.setattr(_head, name, launched)
    for norm in (None, torch.ones(64)):
        with pytest.raises(Launched):
            vce.linear_sample(x, w, u, 0.7, 5, torch.ones(4), None, norm_weight=norm)
        for args, kw in (((x, w, u[:3]), {}), ((x, w, u.double()), {}), ((x, w, u, torch.ones(3)), {}),
                         ((x, w, u), dict(top_k=torch.ones(4))), ((x, w, u), dict(top_p=torch.ones(4).double())),
                         ((x, w, u), dict(min_p=torch.ones(4, 2)[:, 0])), ((x, w, u), dict(dev_status=torch.zeros(1))),
                         ((x[:, :63], w, u), {}), ((x, vce.MXTensor.empty(9, 64, "e4m3", "cpu"), u), {}),
                         ((x, vce.MXTensor.empty(0, 64, "e2m1", "cpu"), u), {}),
                         ((x, vce.MXTensor.empty(vce.SAMPLE_MAX_VOCAB + 1, 64, "e2m1", "cpu"), u), {}),
                         ((x, w._replace(codes=w.codes[:8]), u), {}), ((x, w, u), dict(residual=x[:3]))):
            with pytest.raises(ValueError):
                vce.linear_sample(*args, norm_weight=norm, **kw)


def test_sampling_numbers():
    from vocabulary_cross_entropy_gb300._head import _F32_MAX, _params
    u = torch.zeros(4)
    for k in (0.5, 49.9, float("nan")):
        with pytest.raises(ValueError, match="whole"):
            vce.ce_sample(torch.zeros(4, 10), u, top_k=k)
    inf = float("inf")
    for given, taken in ((50, 50), (50.0, 50), (-7, -1), (1 << 40, (1 << 31) - 1), (inf, (1 << 31) - 1)):
        k = _params(u, None, given, None, None, 4, -1)[1]
        assert k == taken and isinstance(k, int)
    for given, taken in ((0.7, 0.7), (1e39, _F32_MAX), (inf, _F32_MAX), (-inf, -_F32_MAX)):
        assert _params(u, given, None, given, given, 4, -1) == (taken, None, taken, taken)
    assert np.isnan(_params(u, float("nan"), None, None, None, 4, -1)[0])


def test_stream_of_another_device():
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    x, w, s = torch.zeros(4, 64), torch.ones(64), Stream()
    q, c = vce.MXTensor.empty(4, 64, "e4m3", "cpu"), vce.MXTensor.empty(9, 64, "e2m1", "cpu")
    for fn, args in ((vce.mx_quantize, (x,)), (vce.mx_dequantize, (q,)), (vce.mx_linear, (q, c)),
                     (vce.rms_norm_forward, (x, w)), (vce.rms_norm_mx, (x, w)),
                     (vce.rms_norm_backward, (x, x, w, w[:4])), (vce.ce_sample, (x, w[:4])),
                     (vce.linear_sample, (x, c, w[:4]))):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            fn(*args, stream=s)


def test_sampling_definition():
    rng = np.random.default_rng(0)
    z = rng.normal(size=50) * 2
    p = np.exp(z - z.max())
    p /= p.sum()
    order = np.argsort(-z, kind="stable")
    us = (np.arange(20000) + 0.5) / 20000
    share = np.bincount([head.sample_row(z, u)[0] for u in us], minlength=50) / len(us)
    assert np.abs(share - p).max() <= 1 / len(us)
    for u in (0.0, 0.3, 0.999999):
        assert head.sample_row(z, u, 0.0)[0] == order[0] and head.sample_row(z, u, top_k=1)[0] == order[0]
        assert head.sample_row(z, u, top_p=0.5)[0] in order[:np.searchsorted(np.cumsum(p[order]), 0.5) + 1]
        assert p[head.sample_row(z, u, min_p=0.2)[0]] >= 0.2 * p.max() * (1 - 1e-12)
    assert head.sample_row(z, 0.999999, top_k=7)[0] == order[6]
    t, lp = head.sample_row(z, 0.6)
    assert abs(lp - np.log(p[t])) <= 1e-12
    assert head.sample_row(np.array([1.0, 1.0, 1.0, 1.0]), 0.5)[0] == 2
    assert head.sample_row(np.array([-np.inf, -np.inf]), 0.5)[0] == -1
    assert head.sample_row(np.array([0.0, np.nan]), 0.5)[0] == -1
    assert head.sample_row(np.array([0.0, np.inf]), 0.5)[0] == -1


def test_python_refusals():
    x, w = torch.zeros(4, 64), torch.ones(64)
    with pytest.raises(ValueError, match="CUDA"):
        vce.rms_norm_forward(x, w)
    with pytest.raises(ValueError, match="CUDA"):
        vce.mx_quantize(x)
    with pytest.raises(TypeError):
        vce.rms_norm_forward(x.half(), w)
    with pytest.raises(TypeError):
        vce.rms_norm_forward(x, w.half())
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x, w[:63])
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x.t(), w)
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x, w, residual=x[:1])          # no broadcasting
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x, w, residual=x.bfloat16())
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x, w, y=torch.zeros(1, 64).expand(4, 64))
    with pytest.raises(ValueError):
        vce.rms_norm_forward(x, w, h=x)                     # h without a residual
    with pytest.raises(ValueError):
        vce.rms_norm(x, w, residual=x[:1])
    with pytest.raises(ValueError):
        vce.linear_cross_entropy(x.bfloat16(), x.bfloat16(), torch.zeros(4, dtype=torch.int64), residual=x)
    with pytest.raises(ValueError):
        vce.mx_quantize(x, "e5m2")
    with pytest.raises(ValueError):
        vce.rms_norm_backward(x, x, w, torch.zeros(3))
    bad = vce.MXTensor(torch.zeros(4, 64, dtype=torch.uint8), torch.zeros(512, dtype=torch.uint8), 4, 64, "e4m3")
    with pytest.raises(ValueError, match="codes"):          # codes are padded to 128 columns
        vce.mx_dequantize(bad)


def test_formats_against_torch():
    vals = head.mx_values("e4m3")
    all8 = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(vals, all8)
    assert np.array_equal(head.mx_values("e2m1"), [0, 0.5, 1, 1.5, 2, 3, 4, 6])
    x = torch.randn(1, 32 * 500, generator=torch.Generator().manual_seed(0)).double()
    codes, e = head.mx_quantize(x.numpy(), "e4m3")
    scaled = x.view(1, -1, 32) * 2.0 ** -torch.from_numpy(e).double()[:, :, None]
    assert scaled.abs().max() <= 448
    want = scaled.float().to(torch.float8_e4m3fn).view(torch.uint8).numpy().reshape(1, -1)
    assert np.array_equal(codes, want)
    assert np.all(np.abs(head.mx_dequantize(codes, e, "e4m3") - x.numpy()) <= 2.0 ** -4 * np.abs(x.numpy()) + 1e-3)


def test_norm_definition_against_torch():
    h = torch.randn(5, 48, dtype=torch.float64, generator=torch.Generator().manual_seed(1), requires_grad=True)
    w = torch.randn(48, dtype=torch.float64, generator=torch.Generator().manual_seed(2), requires_grad=True)
    y = torch.nn.functional.rms_norm(h, (48,), w, 1e-5)
    dy = torch.randn(5, 48, dtype=torch.float64, generator=torch.Generator().manual_seed(3))
    y.backward(dy)
    got, r = head.rms_norm(h.detach().numpy(), w.detach().numpy(), 1e-5)
    dx, dw = head.rms_norm_backward(dy.numpy(), h.detach().numpy(), w.detach().numpy(), r)
    assert np.allclose(got, y.detach().numpy(), rtol=1e-12) and np.allclose(dx, h.grad.numpy(), rtol=1e-10)
    assert np.allclose(dw, w.grad.numpy(), rtol=1e-10)

"""Refusals of beam search and adapters, and their FP64 definitions, without a GPU: a wrong
argument is an error before any launch."""
import ctypes

import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import beam as ref
from vocabulary_cross_entropy_gb300._beam import _layout

OK, INVALID, DTYPE, ALIGN, WORKSPACE, ARCH, CUDA = range(7)
FAKE = 0x10000  # never dereferenced: host validation fails first


@pytest.fixture(scope="module", autouse=True)
def built():
    from vocabulary_cross_entropy_gb300 import build
    build.build()


def test_beam_refusals():
    f = vce.library().ce_beam

    def call(z=FAKE, dtype=0, batch=2, beams=4, v=100, stride=100, score=FAKE, ended=None, length=None, end=-1, pen=0.0,
             count=4, keep=0, tok=FAKE, par=FAKE, sc=FAKE, done=None, size=None, ws=FAKE, nbytes=1 << 30):
        return f(z, dtype, batch, beams, v, stride, score, ended, length, end, pen, count, keep, tok, par, sc, done, size,
                 ws, nbytes, None, None)

    assert call(dtype=2) == DTYPE
    for bad in (dict(batch=-1), dict(beams=0), dict(beams=33), dict(v=0), dict(v=(1 << 20) + 1, stride=1 << 21),
                dict(stride=99), dict(count=0), dict(count=65), dict(keep=1, count=3), dict(end=-2), dict(end=100),
                dict(ended=FAKE, done=FAKE), dict(end=5), dict(ended=FAKE, end=5), dict(pen=17.0, length=FAKE, size=FAKE),
                dict(pen=float("nan"), length=FAKE, size=FAKE), dict(pen=1.0), dict(length=FAKE), dict(size=FAKE),
                dict(z=None), dict(score=None), dict(tok=None), dict(par=None), dict(sc=None), dict(batch=1 << 30),
                dict(count=3), dict(count=3, sc=FAKE + 64, ended=FAKE, end=5, done=FAKE),
                dict(count=3, sc=FAKE + 64, length=FAKE, size=FAKE)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(z=FAKE + 1), dict(score=FAKE + 2), dict(tok=FAKE + 4), dict(par=FAKE + 4), dict(sc=FAKE + 2),
                dict(ws=FAKE + 128), dict(length=FAKE + 2, size=FAKE), dict(length=FAKE, size=FAKE + 2)):
        assert call(**bad) == ALIGN, bad
    assert call(ws=None) == WORKSPACE
    assert call(nbytes=vce.ce_beam_workspace_size(2, 4, 4) - 1) == WORKSPACE
    assert vce.ce_beam_workspace_size(2, 4, 4) >= 8 * (16 + 32) and vce.ce_beam_workspace_size(0, 4, 4) == 0
    if not torch.cuda.is_available():
        assert call() in (ARCH, CUDA) and call(batch=0) in (ARCH, CUDA)


class State(ctypes.Structure):
    _fields_ = [("src", ctypes.c_void_p), ("dst", ctypes.c_void_p), ("src_row", ctypes.c_int64), ("dst_row", ctypes.c_int64),
                ("parts", ctypes.c_int64), ("src_part", ctypes.c_int64), ("dst_part", ctypes.c_int64),
                ("positions", ctypes.c_int64), ("position_bytes", ctypes.c_int64)]


def test_reorder_refusals():
    f = vce.library().beam_reorder

    def call(parent=FAKE, batch=2, beams=4, lengths=None, count=1, states=True, **state):
        s = State(FAKE, FAKE, 1024, 1024, 2, 512, 512, 8, 64)
        for name, value in state.items():
            setattr(s, name, value)
        return f(ctypes.byref(s) if states else None, count, parent, batch, beams, lengths, None, None)

    for bad in (dict(batch=-1), dict(beams=0), dict(beams=33), dict(parent=None), dict(count=-1), dict(states=False),
                dict(src=None), dict(dst=None), dict(parts=-1), dict(positions=-1), dict(position_bytes=-1),
                dict(src_row=-1), dict(dst_part=-5), dict(src_row=1 << 50), dict(positions=1 << 40, position_bytes=1 << 20),
                dict(positions=1 << 62), dict(parts=1 << 46, positions=2), dict(dst_row=2048), dict(dst_part=1024),
                dict(batch=(1 << 23) + 1)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(parent=FAKE + 4), dict(lengths=FAKE + 2)):
        assert call(**bad) == ALIGN, bad
    if not torch.cuda.is_available():
        assert call() in (ARCH, CUDA)


def test_adapter_refusals():
    f = vce.library().adapter_linear

    def call(y=FAKE, yt=0, n=4, v=100, ys=100, x=FAKE, xt=0, h=64, xs=64, a=FAKE, b=FAKE, count=3, r=16, index=FAKE,
             scale=None, out=FAKE + 4096, os=100, ws=FAKE, nbytes=1 << 30):
        return f(y, yt, n, v, ys, x, xt, h, xs, a, b, count, r, index, scale, out, os, ws, nbytes, None, None)

    assert call(yt=2) == DTYPE and call(xt=2) == DTYPE
    for bad in (dict(n=-1), dict(n=1 << 28), dict(v=0), dict(ys=99), dict(os=99), dict(h=0), dict(xs=63), dict(count=0),
                dict(count=4097), dict(r=0), dict(r=12), dict(r=136), dict(y=None), dict(x=None), dict(a=None),
                dict(b=None), dict(index=None), dict(out=None), dict(out=FAKE, os=104)):
        assert call(**bad) == INVALID, bad
    for bad in (dict(y=FAKE + 1), dict(out=FAKE + 1), dict(x=FAKE + 8), dict(a=FAKE + 8), dict(b=FAKE + 8),
                dict(index=FAKE + 2), dict(scale=FAKE + 2), dict(ws=FAKE + 128), dict(h=60), dict(xs=68),
                dict(xt=1, xs=66)):
        assert call(**bad) == ALIGN, bad
    assert call(ws=None) == WORKSPACE and call(nbytes=vce.adapter_workspace_size(4, 3, 16) - 1) == WORKSPACE
    assert vce.adapter_workspace_size(0, 3, 16) == 0
    if not torch.cuda.is_available():
        assert call() in (ARCH, CUDA)


def test_python_refusals():
    z, s = torch.zeros(4, 10), torch.zeros(2, 2)
    flag, size = torch.zeros(2, 2, dtype=torch.bool), torch.ones(2, 2, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vce.ce_beam(z, s)
    for kw in (dict(count=0), dict(count=65), dict(count=1.5), dict(count=3, keep_places=True), dict(end=10), dict(end=-2),
               dict(ended=flag), dict(ended=flag.int(), end=1), dict(ended=flag[:1], end=1), dict(length=size.long()),
               dict(length_penalty=1.0), dict(length_penalty=17.0, length=size), dict(length_penalty=float("nan"), length=size),
               dict(out_ended=flag), dict(out_length=size), dict(out_score=s.double()), dict(token=size),
               dict(parent=torch.zeros(2, 3, dtype=torch.int64)), dict(dev_status=torch.zeros(1))):
        with pytest.raises(ValueError):
            vce.ce_beam(z, s, **kw)
    for args in ((z[:3], s), (z, s.double()), (z, s.t()), (z.t(), torch.zeros(10, 1)), (z, torch.zeros(1, 33)[:, :0])):
        with pytest.raises(ValueError):
            vce.ce_beam(*args)
    with pytest.raises(TypeError):
        vce.ce_beam(z.half(), s)
    parent = torch.zeros(2, 2, dtype=torch.int64)
    x = torch.zeros(4, 3, 8, 2)
    with pytest.raises(ValueError, match="CUDA"):
        vce.beam_reorder(x, parent)
    lengths = torch.ones(2, dtype=torch.int32)
    for args, kw in (((x, parent.int()), {}), ((x, parent.t()[:, ::2]), {}), ((x[:3], parent), {}), (([x, x], parent), dict(out=[x])),
                     ((x, parent), dict(lengths=lengths)), ((x, parent), dict(lengths=lengths.long(), position_dim=2)),
                     ((x, parent), dict(lengths=lengths, position_dim=0)), ((x, parent), dict(lengths=lengths, position_dim=4)),
                     ((x, parent), dict(position_dim=[2, 2])), ((x, parent), dict(out=x.double())),
                     ((x, parent), dict(out=torch.zeros(1, 3, 8, 2).expand(4, 3, 8, 2))),
                     ((x[:, :, ::2], parent), dict(position_dim=2)), ((x[:, :, :, :1], parent), dict(position_dim=2)),
                     ((torch.zeros(4, 4, 3, 8, 2)[:, :, ::2, :5], parent), dict(position_dim=3)),
                     ((x[:1].expand(4, 3, 8, 2), parent), {}), (([x, x], parent), {}),
                     (([x, x.clone()], parent), dict(out=[x.clone(), x])),
                     (([x, x.clone()], parent), dict(out=[y := x.clone(), y]))):
        with pytest.raises(ValueError):
            vce.beam_reorder(*args, **kw)
    y, h = torch.zeros(4, 10), torch.zeros(4, 16)
    a, b = torch.zeros(3, 8, 16).bfloat16(), torch.zeros(3, 10, 8).bfloat16()
    i = torch.zeros(4, dtype=torch.int32)
    with pytest.raises(ValueError, match="CUDA"):
        vce.adapter_linear(y, h, a, b, i)
    for args, kw in (((y, h[:3], a, b, i), {}), ((y, h, a.float(), b, i), {}), ((y, h, a, b.transpose(1, 2), i), {}),
                     ((y, h, a[:2], b, i), {}), ((y, h, a[:, :4].contiguous(), b[:, :, :4].contiguous(), i), {}),
                     ((y, h, a, b, i.long()), {}), ((y, h, a, b, i[:3]), {}), ((y, h, a, b, i, torch.ones(2)), {}),
                     ((y, h, a, b, i), dict(out=y.bfloat16())), ((y, h, a, b, i), dict(out=y[:3])),
                     ((y, h, a, b, i), dict(dev_status=torch.zeros(1)))):
        with pytest.raises(ValueError):
            vce.adapter_linear(*args, **kw)
    with pytest.raises(TypeError):
        vce.adapter_linear(y.half(), h, a, b, i)


def test_head_checks_before_it_launches(monkeypatch):
    from vocabulary_cross_entropy_gb300 import _head
    x, w = torch.zeros(2, 2, 64), vce.MXTensor.empty(9, 64, "e2m1", "cpu")
    score, u = torch.zeros(2, 2), torch.zeros(4)
    adapters = vce.Adapters(torch.zeros(3, 8, 64).bfloat16(), torch.zeros(3, 9, 8).bfloat16())
    index = torch.zeros(4, dtype=torch.int32)

    class Launched(Exception):
        pass

    def launched(*args, **kwargs):
        raise Launched

    for name in ("rms_norm_mx", "mx_quantize", "flat_rows"):
        monkeypatch.setattr(_head, name, launched)
    for kw in ({}, dict(adapters=adapters, adapter_index=index), dict(adapters=tuple(adapters), adapter_index=index)):
        with pytest.raises(Launched):
            vce.linear_beam(x, w, score, **kw)
        with pytest.raises(Launched):
            vce.linear_sample(x, w, u, **kw)
    bad = (dict(adapters=adapters), dict(adapter_index=index), dict(adapters=adapters, adapter_index=index[:3]),
           dict(adapters=adapters._replace(b=adapters.b[:, :8]), adapter_index=index),
           dict(adapters=adapters._replace(scale=torch.ones(2)), adapter_index=index), dict(residual=x))
    for kw in bad:
        with pytest.raises(ValueError):
            vce.linear_beam(x, w, score, **kw)
        with pytest.raises(ValueError):
            vce.linear_sample(x, w, u, **kw)
    for args, kw in (((x, w, score[:1]), {}), ((x, w, score.double()), {}), ((x, w, score), dict(count=65)),
                     ((x, w, score), dict(end=9)), ((x, w, score), dict(out_score=score.double())),
                     ((x, w._replace(codes=w.codes[:8]), score), {})):
        with pytest.raises(ValueError):
            vce.linear_beam(*args, **kw)


def test_stream_of_another_device():
    class Stream:
        device = torch.device("cuda", 1)
        cuda_stream = 0

    s = Stream()
    z, score, parent = torch.zeros(4, 64), torch.zeros(1, 4), torch.zeros(1, 4, dtype=torch.int64)
    a, b = torch.zeros(1, 8, 64).bfloat16(), torch.zeros(1, 64, 8).bfloat16()
    w, i = vce.MXTensor.empty(9, 64, "e2m1", "cpu"), torch.zeros(4, dtype=torch.int32)
    for call in (lambda: vce.ce_beam(z, score, stream=s), lambda: vce.beam_reorder(z, parent, stream=s),
                 lambda: vce.adapter_linear(z, z, a, b, i, stream=s), lambda: vce.linear_beam(z, w, score, stream=s)):
        with pytest.raises(ValueError, match="stream is on cuda:1"):
            call()


def test_layouts():
    full = torch.zeros(6, 4, 10, 8, dtype=torch.bfloat16)

    def of(t, dim=None):
        return _layout(tuple(t.shape), tuple(t.stride()), t.element_size(), dim)

    assert of(full, 2) == ((640, 4, 160, 10, 16), True) and of(full) == ((640, 1, 0, 1, 640), True)
    assert of(full, 1) == ((640, 1, 0, 4, 160), True) and of(full, 3) == ((640, 40, 16, 8, 2), True)
    assert of(full[:, 1:3, :7], 2) == ((640, 2, 160, 7, 16), True) and of(full[:, :, :7]) == ((640, 4, 160, 1, 112), True)
    assert of(full.transpose(0, 1)[:, :4], 2) == ((160, 4, 640, 10, 16), True)
    assert of(full[:1].expand(6, 4, 10, 8), 2)[1] is False and of(full[:, :1].expand(6, 4, 10, 8), 2)[1] is False
    assert of(full[:, :0], 2) == ((0, 0, 0, 0, 0), True) and of(full[:1]) == ((0, 1, 0, 1, 640), True)
    assert isinstance(of(full[:, :, ::2], 2), str) and isinstance(of(full[:, :, :, ::2], 2), str)
    assert isinstance(of(full, 0), str) and isinstance(of(full, 4), str)


def test_definitions():
    rng = np.random.default_rng(0)
    z = rng.normal(size=(2, 3, 7))
    score = np.array([[-1.0, -2.0, -np.inf], [0.0, -0.5, -0.1]])
    t, p, c, _, _ = ref.beam_step(z, score, count=5)
    lp = torch.log_softmax(torch.from_numpy(z), 2).numpy()
    every = (score[:, :, None] + lp).reshape(2, -1)
    order = np.argsort(-every, axis=1, kind="stable")[:, :5]
    assert np.array_equal(p * 7 + t, order) and np.allclose(c, np.take_along_axis(every, order, 1), atol=1e-12)
    ended = np.array([[False, True, False], [True, True, True]])
    length = np.array([[3, 4, 5], [2, 2, 4]])
    t, p, c, e, n = ref.beam_step(z, score, ended, length, 6, 1.0, 3, False)
    assert t[1].tolist() == [6, 6, 6] and p[1].tolist() == [0, 2, 1] and n[1].tolist() == [2, 4, 2] and e[1].all()
    t, p, c, e, n = ref.beam_step(z, score, ended, length, 6, 1.0, 3, True)
    assert p[1].tolist() == [0, 1, 2]
    t, p, c, e, n = ref.beam_step(np.full((1, 2, 3), -np.inf), np.zeros((1, 2)), None, np.array([[5, 6]]), 0)
    assert t.tolist() == [[-1, -1]] and p.tolist() == [[0, 1]] and n.tolist() == [[5, 6]] and not e.any()
    x = np.arange(24).reshape(4, 3, 2)
    y = ref.reorder(x, np.array([[1, 0], [1, 5]]), np.array([2, 9]), 1)
    assert y[0].tolist() == [[6, 7], [8, 9], [4, 5]] and y[1].tolist() == [[0, 1], [2, 3], [10, 11]]
    assert np.array_equal(y[2], x[3]) and np.array_equal(y[3], x[3])

"""Cases of beam search and adapters for the bounds-checking build (libvce_bounds.so, selected
with VCE_LIBRARY by tests/test_beam_bounds_gpu.py in a child process): ragged, unaligned and padded
inputs that reach every kernel shape.  The device status must stay 0, and results must equal
those of plain torch at the loosest bound that tells a wrong element (the other tests hold
them to theirs).  Exit status 0 when everything passes."""
import os
import sys

import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)

import vocabulary_cross_entropy_gb300 as vce  # noqa: E402

DEV = "cuda:0"
G = torch.Generator(DEV).manual_seed(3)


def rand(n, c, dtype, pad=0, offset=0, std=1.0):
    full = (torch.randn(n, c + pad + offset, device=DEV, generator=G) * std).to(dtype)
    return full[:, offset:offset + c]


def status_of(fn):
    st = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = fn(st)
    torch.cuda.synchronize()
    assert int(st) == 0, int(st)
    return out


def beams(b, k, v, dtype, pad, offset, count):
    z = rand(b * k, v, dtype, pad, offset, 2.0)
    score = torch.randn(b, k, device=DEV, generator=G)
    r = status_of(lambda st: vce.ce_beam(z, score, count=count, dev_status=st))
    c = score[:, :, None].double() + torch.log_softmax(z.double(), 1).view(b, k, v)
    n = min(count, k * v)
    best = c.view(b, -1).topk(n, dim=1).values
    assert torch.allclose(r.score[:, :n].double(), best, rtol=1e-5, atol=1e-5)
    at = (r.parent[:, :n] * v + r.token[:, :n])
    assert torch.allclose(c.view(b, -1).gather(1, at), best, rtol=1e-6, atol=1e-6)


def states(b, k, shape, dim, dtype, lengths, place):
    x = (torch.randn(b * k, *shape, device=DEV, generator=G) * 10).to(dtype)
    parent = torch.randint(0, k, (b, k), device=DEV, generator=G)
    n = torch.randint(0, shape[dim - 1] + 1, (b,), device=DEV, generator=G, dtype=torch.int32) if lengths else None
    rows = (torch.arange(b, device=DEV)[:, None] * k + parent).view(-1)
    want = x[rows]
    if lengths:
        size = [1] * x.dim()
        size[0], size[dim] = b * k, x.shape[dim]
        filled = torch.arange(x.shape[dim], device=DEV)[None] < n.repeat_interleave(k)[:, None]
        want = torch.where(filled.view(size), want, x)
    out = x if place else x.clone()
    status_of(lambda st: vce.beam_reorder(x, parent, lengths=n, position_dim=dim, out=None if place else out, dev_status=st))
    assert torch.equal(out, want)


def adapters(n, h, v, r, count, xt, yt, pad, offset):
    y, x = rand(n, v, yt, pad, offset, 2.0), torch.randn(n, h, device=DEV, generator=G).to(xt)
    a, b = rand(count * r, h, torch.bfloat16, std=h ** -0.5).view(count, r, h), rand(count * v, r, torch.bfloat16).view(count, v, r)
    index = torch.randint(-1, count, (n,), device=DEV, generator=G, dtype=torch.int32)
    out = status_of(lambda st: vce.adapter_linear(y, x, a, b, index, dev_status=st))
    want = y.double()
    for i in range(count):
        mine = index == i
        want[mine] += (x[mine].double() @ a[i].double().t()) @ b[i].double().t()
    assert torch.allclose(out.double(), want, rtol=1e-2, atol=1e-2)
    place = y.clone()
    assert torch.equal(status_of(lambda st: vce.adapter_linear(place, x, a, b, index, out=place, dev_status=st)), out)


def main():
    assert vce.vce_bounds_check_build(), "VCE_LIBRARY does not point at the bounds-checking build"
    for dtype in (torch.bfloat16, torch.float32):
        for b, k, v, pad, offset in ((1, 1, 1, 0, 0), (2, 3, 17, 1, 3), (1, 4, 128256, 0, 0), (3, 2, 4099, 2, 5),
                                     (100, 8, 2049, 0, 0), (2, 32, 1001, 0, 1), (1, 2, 600001, 0, 0), (1, 1, 1 << 20, 0, 0)):
            for count in (1, 16, 17, 64):
                beams(b, k, v, dtype, pad, offset, count)
        same = torch.zeros(2, 30000, dtype=dtype, device=DEV)  # more equal elements than a list holds
        r = status_of(lambda st: vce.ce_beam(same, torch.zeros(2, 1, device=DEV), count=5, dev_status=st))
        assert r.token.tolist() == [[0, 1, 2, 3, 4]] * 2
        for n, h, v, r, count in ((1, 64, 9, 8, 1), (70, 136, 1001, 16, 3), (300, 256, 4096, 64, 2), (40, 72, 333, 128, 9),
                                  (257, 2056, 2001, 24, 20), (900, 64, 640, 32, 1), (5, 8, 100000, 16, 5),
                                  (40, 264, 32001, 8, 40), (150, 72, 32000, 32, 50)):
            for pad, offset in ((0, 0), (3, 1), (8 - v % 8, 0)):
                for xt in (torch.bfloat16, torch.float32):
                    adapters(n, h, v, r, count, xt, dtype, pad, offset)
    for place in (False, True):
        for b, k, shape, dim, dtype in ((1, 4, (3, 100, 8), 2, torch.bfloat16), (300, 2, (7,), 1, torch.int64),
                                        (5, 13, (9, 3, 5), 1, torch.uint8), (2, 32, (2, 2000, 2), 2, torch.float32)):
            for lengths in (False, True):
                states(b, k, shape, dim, dtype, lengths, place)
    print("beam bounds cases ok", flush=True)


if __name__ == "__main__":
    main()

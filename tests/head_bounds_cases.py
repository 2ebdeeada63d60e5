"""Cases of the operators around the cross entropy for the bounds-checking build
(libvce_bounds.so, selected with VCE_LIBRARY by tests/test_head_bounds_gpu.py in a child
process): ragged, unaligned and padded inputs that reach every kernel shape.  The device
status must stay 0, and results must equal those of plain torch at the loosest bound that
tells a wrong element (the other tests hold them to theirs).  Exit status 0 when everything
passes."""
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


def norms(n, h, dtype, pad, offset):
    x, res = rand(n, h, dtype, pad, offset), rand(n, h, dtype, pad, offset)
    w = rand(1, h, dtype)[0].contiguous()
    f = status_of(lambda st: vce.rms_norm_forward(x, w, 1e-6, res, dev_status=st))
    m = status_of(lambda st: vce.rms_norm_mx(x, w, 1e-6, res, dev_status=st))
    hh = f.h.float()
    y = hh * (hh.square().mean(1, keepdim=True) + 1e-6).rsqrt() * w.float()
    assert torch.allclose(f.y.float(), y, rtol=1e-2, atol=1e-4)
    assert torch.allclose(vce.mx_dequantize(m.y, torch.float32), y, rtol=0.07, atol=2e-2)
    b = status_of(lambda st: vce.rms_norm_backward(x, f.h, w, f.rstd, res, dev_status=st))
    hat = hh * f.rstd[:, None]
    g = x.float() * w.float()
    dx = f.rstd[:, None] * (g - hat * (g * hat).mean(1, keepdim=True)) + res.float()
    assert torch.allclose(b.dx.float(), dx, rtol=1e-2, atol=1e-2)
    assert torch.allclose(b.dweight.float(), (x.float() * hat).sum(0), rtol=1e-2, atol=5e-2)


def main():
    assert vce.vce_bounds_check_build(), "VCE_LIBRARY does not point at the bounds-checking build"
    for dtype in (torch.bfloat16, torch.float32):
        for n, h, pad, offset in ((3, 7, 2, 1), (130, 256, 0, 0), (33, 1030, 0, 0), (40, 2048, 8, 8), (300, 4096, 0, 0),
                                  (9, 8192, 0, 0), (5, 9001, 2, 1), (2, 40000, 0, 0), (1300, 1031, 0, 0), (3, 515, 0, 0)):
            norms(n, h, dtype, pad, offset)
        for n, c, pad, offset in ((1, 1, 0, 0), (130, 100, 3, 1), (257, 2056, 0, 0)):
            for fmt, tol in (("e2m1", 0.34), ("e4m3", 0.07)):
                x = rand(n, c, dtype, pad, offset)
                q = status_of(lambda st: vce.mx_quantize(x, fmt, dev_status=st))
                for out in (torch.bfloat16, torch.float32):
                    d = status_of(lambda st: vce.mx_dequantize(q, out, dev_status=st))
                    assert torch.allclose(d.float(), x.float(), rtol=tol, atol=0.3 if fmt == "e2m1" else 1e-2)
    for n, h, v in ((1, 128, 1), (5, 96, 300), (33, 1000, 257), (100, 256, 32001), (257, 640, 3001), (1290, 384, 29002), (1921, 1300, 24100)):
        x, w = vce.mx_quantize(rand(n, h, torch.float32), "e4m3"), vce.mx_quantize(rand(v, h, torch.float32), "e2m1")
        ref = vce.mx_dequantize(x, torch.float32) @ vce.mx_dequantize(w, torch.float32).t()
        for dtype in (torch.float32, torch.bfloat16):
            z = status_of(lambda st: vce.mx_linear(x, w, dtype, dev_status=st))
            assert torch.allclose(z.float(), ref, rtol=1e-2, atol=1e-2)
    filters = (dict(), dict(top_k=40, top_p=0.9), dict(top_p=0.9), dict(min_p=0.02), dict(top_k=900, top_p=0.8, min_p=0.01),
               dict(temperature=0.0), dict(top_k=1))
    for n, v, dtype, pad, offset in ((1, 5, torch.float32, 0, 0), (3, 1001, torch.bfloat16, 2, 1),
                                     (1, 128257, torch.bfloat16, 0, 0), (200, 5003, torch.float32, 1, 3),
                                     (2, 1 << 20, torch.float32, 0, 0)):
        z = rand(n, v, dtype, pad, offset, 2.0)
        u = torch.rand(n, device=DEV, generator=G)
        for f in filters:
            r = status_of(lambda st: vce.ce_sample(z, u, dev_status=st, **f))
            assert ((r.token >= 0) & (r.token < v)).all()
            if f.get("top_k") == 1 or f.get("temperature") == 0.0:
                assert torch.equal(z.float().gather(1, r.token[:, None])[:, 0], z.float().max(1).values)
    same = torch.zeros(2, 30000, device=DEV)  # one bin holds the row: it is divided
    r = status_of(lambda st: vce.ce_sample(same, torch.tensor([0.0, 0.5], device=DEV), dev_status=st))
    assert r.token.tolist() == [0, 15000]
    print("head bounds cases ok", flush=True)


if __name__ == "__main__":
    main()

"""The norm before the classifier (forward, 8-bit form, backward) and microscaled
quantisation against their FP64 definitions.

Bounds, with u = 2^-24 (half a step of FP32) and half a step of the output's type:
- a sum of FP32 terms over a row is a chain of at most 64 additions per thread and
  10 levels of tree, so it is off by at most 80 u of the sum of magnitudes;
- rstd: half of that (square root), plus 4 roundings: 44 u;  y: rstd's, plus 2 products;
- dx = r (g - hat c) + dh: c is off by 84 u mean|g hat|, the rest are 6 roundings of
  terms no larger than |r g| + |r hat c| + |dh|;
- dw: a thread adds at most n / parts + 1 rows and the join adds parts / 32 + 32 more
  (parts <= 2432), each term is 3 roundings off: (n / 608 + 120) u of the sum of
  magnitudes (a row's 608 is the least number of parts, unless there are fewer rows).
"""
import numpy as np
import pytest
import torch

import vocabulary_cross_entropy_gb300 as vce
from oracle import head

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
U = 2.0 ** -24
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def f64(t):
    return t.detach().double().cpu().numpy()


def rand(seed, *shape, dtype, std=1.0, pad=0, offset=0):
    """A [.., cols] tensor inside rows of cols + pad + offset elements."""
    g = torch.Generator().manual_seed(seed)
    cols = shape[-1]
    full = (torch.randn(*shape[:-1], cols + pad + offset, generator=g) * std).to(dtype).to(DEV)
    return full[..., offset:offset + cols]


def check_forward(n, h, dtype, wdtype, residual, pad=0, offset=0, eps=1e-6):
    x = rand(1, n, h, dtype=dtype, pad=pad, offset=offset)
    w = rand(2, h, dtype=wdtype).contiguous()
    res = rand(3, n, h, dtype=dtype, std=3.0, pad=pad, offset=offset) if residual else None
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    f = vce.rms_norm_forward(x, w, eps, res, dev_status=status)
    m = vce.rms_norm_mx(x, w, eps, res, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    want_h = x if res is None else (x.float() + res.float()).to(dtype)
    assert torch.equal(f.h, want_h) and torch.equal(m.h, want_h)
    y, r = head.rms_norm(f64(want_h), f64(w), eps)
    assert np.all(np.abs(f64(f.rstd) - r) <= 44 * U * r)
    # y, and its rounding to the output type
    assert np.all(np.abs(f64(f.y) - y) <= (half_step(dtype) * (1 + 1e-5) + 47 * U) * np.abs(y) + 1e-45)
    # the 8-bit form: scales as of the exact y unless a block's maximum is within y's bound of a border
    codes, e = head.mx_quantize(y, "e4m3")
    _, lo = head.mx_quantize(y * (1 - 47 * U), "e4m3")
    _, hi = head.mx_quantize(y * (1 + 47 * U), "e4m3")
    packed, tiles = head.mx_pack(codes, e, h, "e4m3")
    got = m.y.scales.cpu().numpy().reshape(tiles.shape)
    sure = head.mx_pack(codes, lo, h, "e4m3")[1] == head.mx_pack(codes, hi, h, "e4m3")[1]
    assert np.array_equal(got[sure], tiles[sure])
    vals = f64(vce.mx_dequantize(m.y, torch.float32))
    # half a step of E4M3 at the value, or at the least normal value of the block's scale (2^-6)
    scale = np.repeat(2.0 ** np.maximum(e, hi), 32, axis=1)[:, :h]
    lim = np.maximum(np.abs(y) * 2.0 ** -4, scale * 2.0 ** -10) * (1 + 1e-5) + 47 * U * np.abs(y)
    assert np.all(np.abs(vals - y) <= lim)
    return f, m


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32"), ("f32", "bf16")])
@pytest.mark.parametrize("n,h", [(1, 1), (3, 7), (5, 32), (130, 100), (17, 256), (33, 1030), (7, 2048), (9, 4096),
                                 (400, 1024), (2, 7168), (330, 5120), (3, 16384)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward(n, h, dtype, wdtype, residual):
    check_forward(n, h, DT[dtype], DT[wdtype], residual)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h,pad,offset", [(5, 512, 3, 1), (6, 1000, 8, 8), (4, 96, 1, 0), (3, 4098, 0, 2),
                                            (2, 9001, 2, 1), (2, 40000, 0, 0), (3, 70001, 0, 0)])
def test_forward_strided_and_long(n, h, pad, offset, dtype):
    check_forward(n, h, DT[dtype], DT[dtype], True, pad, offset)


@pytest.mark.parametrize("n", [0, 1, 127, 128, 129])
def test_scale_rows_past_the_end_are_zero(n):
    x = rand(5, n, 160, dtype=torch.bfloat16)
    w = torch.ones(160, device=DEV)
    m = vce.rms_norm_mx(x, w).y
    q = vce.mx_quantize(x, "e4m3")
    for t in (m, q):
        flat = t.scales.permute(0, 3, 2, 1, 4).reshape(-1, 8).cpu()
        assert (flat[n:] == 0).all() and (flat[:, 5:] == 0).all()
        assert (t.codes[:, 160:] == 0).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h", [(3000, 1031), (1400, 4097), (2000, 2317), (2500, 301), (1200, 2050), (9, 301)])
@pytest.mark.parametrize("residual", [False, True])
def test_forward_rows_off_16_bytes(n, h, dtype, residual):
    # many rows to a block, every offset of a row from a 16-byte boundary
    check_forward(n, h, DT[dtype], DT[dtype], residual)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("alias", [None, "x", "residual"])
@pytest.mark.parametrize("n,h,pad,offset", [(2600, 1031, 2, 1), (1300, 1024, 5, 3), (3, 2000, 7, 1), (700, 2048, 3, 1)])
def test_forward_of_views_at_one_offset(n, h, pad, offset, alias, dtype):
    # views with one offset and stride, the outputs among them: the same h as plainly added, y
    # within its bound, and nothing beside the views is written
    base = [rand(k, n, h + pad, dtype=DT[dtype]).contiguous() for k in (1, 2, 3, 4)]
    x, res, hh, y = (t[:, offset:offset + h] for t in base)
    w = rand(5, h, dtype=DT[dtype]).contiguous()
    want_h = (x.float() + res.float()).to(DT[dtype])
    want_y, _ = head.rms_norm(f64(want_h), f64(w), 1e-6)
    i = {None: 2, "x": 0, "residual": 1}[alias]
    before = [base[i].clone(), base[3].clone()]
    got = vce.rms_norm_forward(x, w, 1e-6, res, h=(x, res, hh)[i], y=y)
    assert torch.equal(got.h, want_h)
    assert np.all(np.abs(f64(got.y) - want_y) <= (half_step(DT[dtype]) * (1 + 1e-5) + 47 * U) * np.abs(want_y) + 1e-45)
    for full, was, part in ((base[i], before[0], got.h), (base[3], before[1], got.y)):
        was[:, offset:offset + h] = part
        assert torch.equal(full, was)
    plain = vce.rms_norm_forward(want_h[:, :], w, 1e-6, y=y)
    assert np.all(np.abs(f64(plain.y) - want_y) <= (half_step(DT[dtype]) * (1 + 1e-5) + 47 * U) * np.abs(want_y) + 1e-45)


@pytest.mark.parametrize("alias", ["h_is_residual", "h_is_x", "y_is_x", "y_is_residual"])
@pytest.mark.parametrize("h", [4096, 1031, 70001])
def test_forward_in_place(alias, h):
    x, res = rand(1, 6, h, dtype=torch.bfloat16), rand(2, 6, h, dtype=torch.bfloat16)
    w = rand(3, h, dtype=torch.bfloat16).contiguous()
    want = vce.rms_norm_forward(x, w, 1e-5, res)
    x, res = x.clone(), res.clone()
    out = {"h_is_residual": dict(h=res), "h_is_x": dict(h=x), "y_is_x": dict(y=x), "y_is_residual": dict(y=res)}
    got = vce.rms_norm_forward(x, w, 1e-5, res, **out[alias])
    assert torch.equal(got.y, want.y) and torch.equal(got.h, want.h) and torch.equal(got.rstd, want.rstd)


def test_zero_row_and_non_finite_rows():
    x = torch.zeros(4, 256, device=DEV)
    x[1, 3] = float("inf")
    x[2, 200] = float("nan")
    x[3] = 1.0
    w = torch.ones(256, device=DEV)
    f = vce.rms_norm_forward(x, w, 1e-6)
    assert (f.y[0] == 0).all()                      # zero times a finite rstd
    assert f.y[1].isnan().sum() == 1 and (f.y[1].nan_to_num(0.0) == 0).all()   # inf * 0; the rest x * 0
    assert f.y[2].isnan().all()                     # NaN in the sum
    q = vce.rms_norm_mx(x, w, 1e-6).y
    vals = vce.mx_dequantize(q, torch.float32)
    assert (vals[0] == 0).all() and torch.isfinite(vals[3]).all()
    assert vals[1, :32].isnan().all() and (vals[1, 32:] == 0).all() and vals[2].isnan().all()
    # rows of zeros with eps 0 have no norm
    assert vce.rms_norm_forward(x[:1], w, 0.0).y.isnan().all()


def compare_backward(got, dy, hs, w, r, dh):
    n, dtype, wdtype = dy.shape[0], dy.dtype, w.dtype
    dx, dw = head.rms_norm_backward(f64(dy), f64(hs), f64(w), f64(r), None if dh is None else f64(dh))
    rr, g = f64(r)[:, None], f64(dy) * f64(w)
    hat = f64(hs) * rr
    c, cabs = (g * hat).mean(1, keepdims=True), np.abs(g * hat).mean(1, keepdims=True)
    terms = np.abs(rr * g) + np.abs(rr * hat * c) + (0 if dh is None else np.abs(f64(dh)))
    lim = half_step(dtype) * np.abs(dx) * (1 + 1e-5) + 84 * U * np.abs(rr * hat) * cabs + 6 * U * terms
    assert np.all(np.abs(f64(got.dx) - dx) <= lim + 1e-45)
    parts = min(n, 608)
    mag = np.abs(f64(dy) * hat).sum(0)
    lim = half_step(wdtype) * np.abs(dw) * (1 + 1e-5) + (n / max(parts, 1) + 120) * U * mag
    assert np.all(np.abs(f64(got.dweight) - dw) <= lim + 1e-45)


def check_backward(n, h, dtype, wdtype, with_dh, pad=0, offset=0):
    hs = rand(1, n, h, dtype=dtype, std=2.0, pad=pad, offset=offset)
    w = (1 + 0.3 * rand(2, h, dtype=torch.float32)).to(wdtype).contiguous()
    dy = rand(3, n, h, dtype=dtype, std=0.1, pad=pad, offset=offset)
    dh = rand(4, n, h, dtype=dtype, std=0.1, pad=pad, offset=offset) if with_dh else None
    r = torch.from_numpy(head.rms_norm(f64(hs), f64(w), 1e-6)[1]).float().to(DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    got = vce.rms_norm_backward(dy, hs, w, r, dh, dev_status=status)
    again = vce.rms_norm_backward(dy, hs, w, r, dh)
    torch.cuda.synchronize()
    assert int(status) == 0
    assert torch.equal(got.dx, again.dx) and torch.equal(got.dweight, again.dweight)
    compare_backward(got, dy, hs, w, r, dh)


@pytest.mark.parametrize("dtype,wdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("n,h", [(1, 1), (3, 7), (130, 100), (2000, 64), (17, 256), (515, 1030), (33, 1032),
                                 (700, 4096), (5, 7168), (9, 16384)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward(n, h, dtype, wdtype, with_dh):
    check_backward(n, h, DT[dtype], DT[wdtype], with_dh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h,pad,offset", [(5, 512, 3, 1), (6, 1000, 8, 8), (40, 4098, 0, 2), (700, 9001, 2, 1),
                                            (3, 40000, 0, 0)])
def test_backward_strided_and_long(n, h, pad, offset, dtype):
    check_backward(n, h, DT[dtype], DT[dtype], True, pad, offset)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,h", [(3000, 1031), (1500, 2049), (1400, 4097), (2500, 301), (9, 301), (2, 2317)])
@pytest.mark.parametrize("with_dh", [False, True])
def test_backward_rows_off_16_bytes(n, h, dtype, with_dh):
    # many rows to a block, every offset of a row from a 16-byte boundary
    check_backward(n, h, DT[dtype], DT[dtype], with_dh)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("alias", [None, "dy", "dh"])
@pytest.mark.parametrize("n,h,pad,offset", [(1300, 1031, 2, 1), (1300, 1024, 5, 3), (3, 2000, 6, 1)])
def test_backward_of_views_at_one_offset(n, h, pad, offset, alias, dtype):
    # views with one offset and stride, the output among them; nothing beside them is written
    def view(seed):
        return rand(seed, n, h + pad, dtype=DT[dtype]).contiguous()
    base = [view(k) for k in (1, 2, 3, 4)]
    hs, dy, dh, dx = (t[:, offset:offset + h] for t in base)
    w = rand(5, h, dtype=DT[dtype]).contiguous()
    r = vce.rms_norm_forward(hs, w).rstd
    out, full = {None: (dx, base[3]), "dy": (dy, base[1]), "dh": (dh, base[2])}[alias]
    before, given = full.clone(), [t.clone() for t in (dy, hs, dh)]
    got = vce.rms_norm_backward(dy, hs, w, r, dh, dx=out)
    compare_backward(got, given[0], given[1], w, r, given[2])
    before[:, offset:offset + h] = got.dx
    assert torch.equal(full, before)


@pytest.mark.parametrize("h", [1024, 333, 40000])
@pytest.mark.parametrize("alias", ["dy", "dh"])
def test_backward_in_place(h, alias):
    hs, dy, dh = (rand(k, 50, h, dtype=torch.bfloat16) for k in (1, 2, 3))
    w = rand(4, h, dtype=torch.float32).contiguous()
    r = vce.rms_norm_forward(hs, w).rstd
    want = vce.rms_norm_backward(dy, hs, w, r, dh)
    dy, dh = dy.clone(), dh.clone()
    got = vce.rms_norm_backward(dy, hs, w, r, dh, dx=dy if alias == "dy" else dh)
    assert torch.equal(got.dx, want.dx) and torch.equal(got.dweight, want.dweight)


def test_backward_of_no_rows():
    w = torch.ones(64, device=DEV)
    e = torch.empty(0, 64, device=DEV)
    r = vce.rms_norm_backward(e, e, w, torch.empty(0, device=DEV))
    assert (r.dweight == 0).all() and r.dx.shape == (0, 64)


# ---------------------------------------------------------------------------
# autograd
# ---------------------------------------------------------------------------

def test_autograd_against_differences():
    # FP32: central differences of a linear functional of (y, h) along random directions
    n, h = 6, 96
    x, res, w = (rand(k, *s, dtype=torch.float32).contiguous().requires_grad_() for k, s in
                 ((1, (n, h)), (2, (n, h)), (3, (h,))))
    cy, ch = rand(4, n, h, dtype=torch.float32), rand(5, n, h, dtype=torch.float32)

    def value(x, res, w):  # the definition in FP64
        hh = x.double() + res.double()
        r = (hh.square().mean(1, keepdim=True) + 1e-6).rsqrt()
        return ((hh * r * w.double()) * cy.double()).sum() + (hh * ch.double()).sum()

    y, hh = vce.rms_norm(x, w, 1e-6, res)
    ((y * cy).sum() + (hh * ch).sum()).backward()
    for i, t in enumerate((x, res, w)):
        d = rand(10 + i, *t.shape, dtype=torch.float32).double()
        step = 1e-5
        args = [a.detach().double() for a in (x, res, w)]
        hi, lo = list(args), list(args)
        hi[i], lo[i] = hi[i] + step * d, lo[i] - step * d
        diff = float((value(*hi) - value(*lo)) / (2 * step))
        got = float((t.grad.double() * d).sum())
        # step^2 truncation (1e-10 x third derivatives of order 1) and FP32 gradients
        assert abs(got - diff) <= 2e-5 * float((t.grad.double().abs() * d.abs()).sum())
    assert torch.equal(x.grad, res.grad) and x.grad.data_ptr() != res.grad.data_ptr()


def test_autograd_uses_of_either_output():
    x, res = rand(1, 2, 5, 64, dtype=torch.bfloat16), rand(2, 2, 5, 64, dtype=torch.bfloat16)
    w = torch.ones(64, device=DEV)
    for use in ("y", "h", "both", "expanded"):
        xs, rs, ws = (t.clone().requires_grad_() for t in (x, res, w))
        y, h = vce.rms_norm(xs, ws, 1e-6, rs)
        assert y.shape == x.shape and h.shape == x.shape
        if use == "expanded":
            y.sum().backward()  # the gradient of y is one element, expanded
        else:
            g = torch.ones_like(y)
            sum((t * g).sum() for t, skip in ((y, "h"), (h, "y")) if use != skip).backward()
        assert xs.grad.shape == x.shape and torch.equal(xs.grad, rs.grad)
        if use == "h":
            assert (xs.grad == 1).all() and (ws.grad is None or (ws.grad == 0).all())
    xs = x.clone().requires_grad_()
    vce.rms_norm(xs.transpose(0, 1), w).float().square().sum().backward()
    assert xs.grad.shape == x.shape


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("shape", [(64,), (9, 64), (3, 4, 64), (0, 64)])
def test_rms_norm_outputs_change_in_place(shape, residual):
    x, w = rand(1, *shape, dtype=torch.float32), rand(2, 64, dtype=torch.float32)
    res = rand(3, *shape, dtype=torch.float32) if residual else None

    def grads(double):
        leaves = [None if t is None else t.clone().requires_grad_() for t in (x, w, res)]
        out = vce.rms_norm(leaves[0], leaves[1], 1e-6, leaves[2])
        y = out[0] if residual else out
        double(y).square().sum().backward()
        return [t.grad for t in leaves if t is not None]

    for a, b in zip(grads(lambda y: y.mul_(2.0)), grads(lambda y: y * 2.0)):
        assert torch.equal(a, b)
    if residual:  # h may change too, but not before a backward pass that needs it
        a, b, c = (t.clone().requires_grad_() for t in (x, w, res))
        y, h = vce.rms_norm(a, b, 1e-6, c)
        h.add_(1.0)
        h.sum().backward()
        assert torch.equal(a.grad, torch.ones_like(a)) and b.grad is None
        y, h = vce.rms_norm(a, b, 1e-6, c)
        h.add_(1.0)
        if h.numel():
            with pytest.raises(RuntimeError, match="inplace"):
                y.sum().backward()


def test_rms_norm_gradient_has_the_weights_shape():
    x, w = rand(1, 9, 64, dtype=torch.float32), rand(2, 64, dtype=torch.float32)
    flat, row = w.clone().requires_grad_(), w[None].clone().requires_grad_()
    for t in (flat, row):
        vce.rms_norm(x, t).square().sum().backward()
    assert row.grad.shape == (1, 64) and torch.equal(row.grad[0], flat.grad)


@pytest.mark.parametrize("residual", [False, True])
def test_linear_cross_entropy_with_norm(residual):
    b, sq, h, v = 2, 65, 256, 1000
    x = rand(1, b, sq, h, dtype=torch.bfloat16).contiguous()
    res = rand(2, b, sq, h, dtype=torch.bfloat16).contiguous()
    nw = (1 + 0.1 * rand(3, h, dtype=torch.float32)).to(torch.bfloat16)
    w = rand(4, v, h, dtype=torch.bfloat16, std=h ** -0.5).contiguous()
    y = torch.randint(0, v, (b, sq), device=DEV, generator=torch.Generator(DEV).manual_seed(1))
    a = [t.clone().requires_grad_() for t in (x, res, nw, w)]
    loss = vce.linear_cross_entropy(a[0], a[3], y, norm_weight=a[2], norm_eps=1e-5,
                                    residual=a[1] if residual else None, shift=True)
    loss.backward()
    c = [t.clone().requires_grad_() for t in (x, res, nw, w)]
    out = vce.rms_norm(c[0], c[2], 1e-5, c[1] if residual else None)
    want = vce.linear_cross_entropy(out[0] if residual else out, c[3], y, shift=True)
    want.backward()
    assert torch.equal(loss, want)
    for s, t in zip(a, c):
        assert (s.grad is None) == (t.grad is None)
        assert s.grad is None or torch.equal(s.grad, t.grad)
    # and against FP64 autograd of the definition: BF16 roundings of the hidden states (2^-8 each,
    # on the way in and on dX) leave the gradients within 2% in norm
    d = [t.detach().double().requires_grad_() for t in (x, res, nw, w)]
    hh = (x.float() + res.float()).bfloat16().double() if residual else d[0]
    if residual:
        hh = hh + (d[0] - d[0].detach()) + (d[1] - d[1].detach())
    yn = hh * (hh.square().mean(-1, keepdim=True) + 1e-5).rsqrt() * d[2]
    z = (yn @ d[3].t())[:, :-1].reshape(-1, v)
    ref = torch.nn.functional.cross_entropy(z, y[:, 1:].reshape(-1))
    ref.backward()
    assert abs(float(loss) - float(ref)) <= 5e-3
    for s, t in zip(a, d):
        if s.grad is not None:
            assert float((s.grad.double() - t.grad).norm()) <= 0.02 * float(t.grad.norm())


def test_training_step_captured():
    # forward and backward of norm and loss in one graph; refused while an eager graph of the same
    # leaves is alive, and fine once it is gone
    n, h, v = 40, 256, 1000
    leaves = [rand(1, n, h, dtype=torch.bfloat16).contiguous(), (1 + 0.1 * rand(2, h, dtype=torch.float32)).bfloat16(),
              rand(3, v, h, dtype=torch.bfloat16, std=h ** -0.5).contiguous()]
    x, nw, w = [t.requires_grad_() for t in leaves]
    y = torch.randint(0, v, (n,), device=DEV, generator=torch.Generator(DEV).manual_seed(1))

    def step():
        loss = vce.linear_cross_entropy(x, w, y, norm_weight=nw)
        loss.backward()
        return loss

    def grads():
        torch.cuda.synchronize()
        return [t.grad.clone() for t in (x, nw, w)]

    loss = step()
    want, value = grads(), loss.detach().clone()
    x.grad = nw.grad = w.grad = None
    out = vce.rms_norm(x, nw)
    graph = torch.cuda.CUDAGraph()
    with pytest.raises(RuntimeError, match="still alive"):
        with torch.cuda.graph(graph):
            vce.rms_norm(x, nw)
    del out, loss
    # nodes that something else holds (a data-parallel wrapper, say) and made on a side stream: fine
    with torch.cuda.stream(torch.cuda.Stream()):
        held = [torch.autograd.graph.get_gradient_edge(t).node for t in (x, nw)]
    out = vce.rms_norm(x, nw)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = vce.rms_norm(x, nw)
    graph.replay()
    assert torch.equal(got, out)
    del held, out, got, graph
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        loss = step()
    for t in (x, nw, w):
        t.grad.zero_()
    for k in range(1, 3):  # a replay writes the gradients anew
        graph.replay()
        for a, c in zip(grads(), want):
            assert torch.equal(a, c)
        assert torch.equal(loss.detach(), value)


# ---------------------------------------------------------------------------
# quantisation
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("n,c,pad,offset", [(1, 1, 0, 0), (3, 31, 0, 0), (5, 33, 2, 1), (130, 160, 0, 0),
                                            (257, 1000, 8, 0), (64, 2056, 0, 0), (2, 5000, 1, 3)])
def test_quantize_bits(n, c, pad, offset, dtype, fmt):
    x = rand(n + c, n, c, dtype=DT[dtype], std=0.3, pad=pad, offset=offset)
    if n > 2:  # magnitudes over many binades, ties, values at the format's limit, signed zeros
        x[1] = (x[1].double() * torch.exp2(torch.randint(-40, 40, (c,), device=DEV).double())).to(x.dtype)
        x[2] = torch.arange(c, device=DEV).to(x.dtype) * 0.25 - 6.0
    x[0, 0] = -0.0
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    q = vce.mx_quantize(x, fmt, dev_status=status)
    torch.cuda.synchronize()
    assert int(status) == 0
    codes, e = head.mx_quantize(f64(x), fmt)
    packed, tiles = head.mx_pack(codes, e, c, fmt)
    assert np.array_equal(q.scales.cpu().numpy().reshape(tiles.shape), tiles)
    assert np.array_equal(q.codes.cpu().numpy(), packed)
    vals = head.mx_dequantize(codes, e, fmt)[:, :c]
    assert np.array_equal(f64(vce.mx_dequantize(q, torch.float32)), vals)
    half = vce.mx_dequantize(q, torch.bfloat16)
    assert torch.equal(half, torch.from_numpy(vals).to(torch.bfloat16).to(DEV))
    out = torch.full((n, c + 3), 7.0, device=DEV)  # a strided output: its padding stays
    vce.mx_dequantize(q, torch.float32, out=out[:, 1:c + 1])
    assert np.array_equal(f64(out[:, 1:c + 1]), vals) and (out[:, 0] == 7).all() and (out[:, c + 1:] == 7).all()


@pytest.mark.parametrize("fmt", ["e2m1", "e4m3"])
def test_quantize_extremes(fmt):
    big, tiny = torch.finfo(torch.float32).max, 2.0 ** -149
    most = head.FORMATS[fmt][0]
    rows = [[big, -big], [tiny, -tiny], [2.0 ** -126, 2.0 ** -127], [0.0, -0.0], [most, most / 2],
            [float(np.nextafter(np.float32(most), np.float32(1e9))), 1.0], [float("inf"), 1.0],
            [float("nan"), 1.0], [float("-inf"), float("nan")], [2.0 ** 127, 1.0]]
    x = torch.zeros(len(rows), 64, device=DEV)
    x[:, :2] = torch.tensor(rows, device=DEV)
    x[:, 40] = 1.0  # the second block is its own
    q = vce.mx_quantize(x, fmt)
    codes, e = head.mx_quantize(f64(x), fmt)
    packed, tiles = head.mx_pack(codes, e, 64, fmt)
    assert np.array_equal(q.scales.cpu().numpy().reshape(tiles.shape), tiles)
    assert np.array_equal(q.codes.cpu().numpy(), packed)
    got = f64(vce.mx_dequantize(q, torch.float32))
    assert np.array_equal(np.isnan(got[:, :32]).all(1), [False] * 6 + [True] * 3 + [False])
    assert np.array_equal(got[:, 40], np.ones(len(rows)))


def test_mx_from_parts():
    x = rand(3, 150, 200, dtype=torch.float32)
    for fmt in ("e2m1", "e4m3"):
        codes, e = head.mx_quantize(f64(x), fmt)
        raw = codes[:, :200].astype(np.uint8)
        if fmt == "e2m1":
            raw = raw[:, 0::2] | (raw[:, 1::2] << 4)
        t = vce.MXTensor.from_parts(torch.from_numpy(raw).to(DEV),
                                    torch.from_numpy((e + 127).astype(np.uint8)).to(DEV), 200, fmt)
        q = vce.mx_quantize(x, fmt)
        assert torch.equal(t.codes, q.codes) and torch.equal(t.scales, q.scales)


@pytest.mark.parametrize("cols", [256, 255])
def test_every_code(cols):
    # all 256 codes of E4M3, its two NaNs among them, and all 16 of E2M1
    for fmt, codes in (("e4m3", torch.arange(256)[:cols]), ("e2m1", torch.arange(cols) * 7 % 16)):
        raw = codes.to(torch.uint8).numpy()[None]
        want = head.mx_dequantize(np.pad(raw, ((0, 0), (0, 256 - cols))).astype(int), np.full((1, 8), 3), fmt)[:, :cols]
        if fmt == "e2m1":
            raw = np.pad(raw, ((0, 0), (0, cols % 2)))
            raw = raw[:, 0::2] | (raw[:, 1::2] << 4)
        t = vce.MXTensor.from_parts(torch.from_numpy(raw).to(DEV), torch.full((1, 8), 130, dtype=torch.uint8, device=DEV),
                                    cols, fmt)
        for dtype in (torch.float32, torch.bfloat16):
            got = f64(vce.mx_dequantize(t, dtype))
            assert np.array_equal(got, want, equal_nan=True), (fmt, dtype)
            assert np.isnan(got).sum() == (min(2, cols - 254) if fmt == "e4m3" else 0)


def test_streams_and_graphs():
    # another stream than the current one, with outputs and workspace allocated by the call;
    # then a captured chain replayed on new inputs
    x, res = rand(1, 300, 1024, dtype=torch.bfloat16), rand(2, 300, 1024, dtype=torch.bfloat16)
    w = rand(3, 1024, dtype=torch.bfloat16).contiguous()
    want = vce.rms_norm_forward(x, w, 1e-6, res)
    wb = vce.rms_norm_backward(x, want.h, w, want.rstd)
    wq = vce.mx_quantize(want.y, "e2m1")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = vce.rms_norm_forward(x, w, 1e-6, res, stream=side)
    gb = vce.rms_norm_backward(x, got.h, w, got.rstd, stream=side)
    gq = vce.mx_quantize(got.y, "e2m1", stream=side)
    side.synchronize()
    for a, c in ((got.y, want.y), (gb.dx, wb.dx), (gb.dweight, wb.dweight), (gq.codes, wq.codes)):
        assert torch.equal(a, c)
    xs = x.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        f = vce.rms_norm_forward(xs, w, 1e-6, res)
        bk = vce.rms_norm_backward(xs, f.h, w, f.rstd)
        q = vce.mx_dequantize(vce.mx_quantize(f.y, "e4m3"))
    for k in (7, 8):
        xs.copy_(rand(k, 300, 1024, dtype=torch.bfloat16))
        graph.replay()
        e = vce.rms_norm_forward(xs, w, 1e-6, res)
        eb = vce.rms_norm_backward(xs, e.h, w, e.rstd)
        assert torch.equal(f.y, e.y) and torch.equal(bk.dweight, eb.dweight) and torch.equal(bk.dx, eb.dx)
        assert torch.equal(q, vce.mx_dequantize(vce.mx_quantize(e.y, "e4m3")))


def test_offsets_past_32_bits():
    # rows whose elements lie past 2^31: the first and last rows against the same rows alone
    n, h = 70000, 32768
    x = torch.empty(n, h, dtype=torch.bfloat16, device=DEV)
    x[:2].normal_()
    x[-2:].normal_()
    x[2:-2] = 1.0
    w = torch.ones(h, device=DEV)
    f = vce.rms_norm_forward(x, w)
    q = vce.mx_quantize(x, "e2m1")
    d = vce.mx_dequantize(q)
    for s in (slice(0, 2), slice(n - 2, n)):
        part = x[s].contiguous()
        assert torch.equal(f.y[s], vce.rms_norm_forward(part, w).y)
        assert torch.equal(d[s], vce.mx_dequantize(vce.mx_quantize(part, "e2m1")))

"""ctypes marshalling for the operators around the vocabulary cross entropy: the norm
before the classifier, microscaled tensors and their product, and sampling (see include/vce.h for what each
computes).  As in ``_binding``, torch tensors supply memory and the current stream.

A call given ``stream`` allocates what it was not given (outputs and workspace) from
that stream, so memory it drops on return is reused only behind its kernels.
"""
from __future__ import annotations

import contextlib
from collections import namedtuple

import torch

from . import _binding as b

MX_E4M3, MX_E2M1 = 0, 1
SAMPLE_MAX_VOCAB = 1 << 20
_FMT = {"e4m3": MX_E4M3, "e2m1": MX_E2M1}

RMSNormForward = namedtuple("RMSNormForward", "y h rstd")
RMSNormMX = namedtuple("RMSNormMX", "y h rstd")
RMSNormBackward = namedtuple("RMSNormBackward", "dx dweight")
CESample = namedtuple("CESample", "token logprob dev_status")


def _on_stream(stream):
    return contextlib.nullcontext() if stream is None else torch.cuda.stream(stream)


def _float_code(t, name):
    if t.dtype is torch.bfloat16:
        return b.BF16
    if t.dtype is torch.float32:
        return b.F32
    raise TypeError(f"{name} must be bfloat16 or float32, got {t.dtype}")


def _matrix(t, name, shape=None, dtype=None, device=None):
    """Row stride of a [rows, cols] tensor with contiguous rows that do not overlap."""
    if t.dim() != 2 or (t.shape[1] > 1 and t.stride(1) != 1):
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if device is not None and t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    return t.stride(0) if t.shape[0] > 1 else t.shape[1]


def _written(t, name, shape, dtype, device):
    """_matrix of an output: its rows must not overlap."""
    stride = _matrix(t, name, shape, dtype, device)
    if stride < t.shape[1]:
        raise ValueError(f"the rows of {name} overlap")
    return stride


def _vector(t, name, n, dtype, device):
    if t.dtype != dtype or t.numel() != n or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on {device}")
    return t


def _launch(name, device, fn, *args):
    """fn(*args, stream) of the library, once everything about the arguments has been checked."""
    if device.type != "cuda":
        raise ValueError(f"{name}: tensors must be on a CUDA device, got {device}")
    *args, stream = args
    b._check(name, b._on(device, fn, *args, b._stream(device, stream)))


def _status(t, device):
    if t is None:
        return None
    return b._ptr(_vector(t, "dev_status", 1, torch.int32, device))


# ---------------------------------------------------------------------------
# microscaled tensors
# ---------------------------------------------------------------------------

class MXTensor(namedtuple("MXTensor", "codes scales rows cols fmt")):
    """A matrix [rows, cols] of 8-bit (``fmt`` "e4m3") or 4-bit ("e2m1") values with one
    power-of-two scale per 32 columns.

    ``codes`` uint8 [rows, padded] (e4m3) or [rows, padded / 2] (e2m1, even column in the low
    nibble), ``padded`` = cols rounded up to 128; ``scales`` uint8
    [ceil(rows / 128), padded / 128, 32, 4, 4], E8M0 bytes in the tiles of include/vce.h.
    """
    __slots__ = ()

    @staticmethod
    def empty(rows, cols, fmt, device):
        padded = -(-cols // 128) * 128
        codes = torch.empty(rows, padded // (2 if fmt == "e2m1" else 1), dtype=torch.uint8, device=device)
        scales = torch.empty(-(-rows // 128), padded // 128, 32, 4, 4, dtype=torch.uint8, device=device)
        return MXTensor(codes, scales, rows, cols, fmt)

    @staticmethod
    def from_parts(codes, scales, cols, fmt):
        """From codes [rows, cols (/ 2)] and plain row-major E8M0 scales [rows, ceil(cols / 32)],
        as checkpoints hold them: pads the codes and lays the scales out in tiles."""
        rows, per = codes.shape[0], 2 if fmt == "e2m1" else 1
        blocks = -(-cols // 32)
        if _fmt(fmt) is None or codes.dtype != torch.uint8 or scales.dtype != torch.uint8:
            raise TypeError("codes and scales must be uint8")
        if tuple(codes.shape) != (rows, -(-cols // per)) or tuple(scales.shape) != (rows, blocks):
            raise ValueError(f"expected codes {(rows, -(-cols // per))} and scales {(rows, blocks)}, got "
                             f"{tuple(codes.shape)} and {tuple(scales.shape)}")
        out = MXTensor.empty(rows, cols, fmt, codes.device)
        out.codes.zero_()
        out.codes[:, :codes.shape[1]] = codes
        if fmt == "e2m1" and cols % 2:
            out.codes[:, cols // 2] &= 15
        tiles, ct = out.scales.shape[:2]
        padded = torch.nn.functional.pad(scales, (0, ct * 4 - blocks, 0, tiles * 128 - rows))
        out.scales.copy_(padded.view(tiles, 4, 32, ct, 4).permute(0, 3, 2, 1, 4))
        return out


def _fmt(fmt) -> int:
    if fmt not in _FMT:
        raise ValueError(f"fmt must be one of {sorted(_FMT)}, got {fmt!r}")
    return _FMT[fmt]


def _check_mx(t, name):
    code = _fmt(t.fmt)
    n, c = t.codes, t.scales
    if t.rows < 0 or t.cols < 1:
        raise ValueError(f"{name}: rows and cols must be positive")
    for part, what, size in ((n, "codes", mx_codes_size(t.rows, t.cols, t.fmt)),
                             (c, "scales", mx_scales_size(t.rows, t.cols))):
        if part.dtype != torch.uint8 or not part.is_contiguous() or part.numel() != size:
            raise ValueError(f"{name}.{what} must be a contiguous uint8 tensor of {size} bytes")
    if n.device != c.device:
        raise ValueError(f"{name}: codes and scales are on different devices")
    return code


def mx_codes_size(rows: int, cols: int, fmt: str) -> int:
    return int(b.library().mx_codes_size(rows, cols, _fmt(fmt)))


def mx_scales_size(rows: int, cols: int) -> int:
    return int(b.library().mx_scales_size(rows, cols))


def mx_quantize(x, fmt="e2m1", *, out=None, dev_status=None, stream=None) -> MXTensor:
    """``x`` [rows, cols] (bfloat16 or float32) as a microscaled tensor."""
    lib = b.library()
    code, fcode = _float_code(x, "x"), _fmt(fmt)
    stride = _matrix(x, "x")
    rows, cols = x.shape
    if out is None:
        with _on_stream(stream):
            out = MXTensor.empty(rows, cols, fmt, x.device)
    else:
        _check_mx(out, "out")
        if (out.rows, out.cols, out.fmt) != (rows, cols, fmt) or out.codes.device != x.device:
            raise ValueError("out must have x's shape and device, and the format asked for")
    _launch("mx_quantize", x.device, lib.mx_quantize, b._ptr(x), code, rows, cols, stride, fcode, b._ptr(out.codes),
            b._ptr(out.scales), _status(dev_status, x.device), stream)
    return out


def mx_dequantize(t: MXTensor, dtype=torch.bfloat16, *, out=None, dev_status=None, stream=None):
    """The values of a microscaled tensor, [rows, cols] in bfloat16 or float32."""
    lib = b.library()
    fcode = _check_mx(t, "t")
    dev = t.codes.device
    if out is None:
        with _on_stream(stream):
            out = torch.empty(t.rows, t.cols, dtype=dtype, device=dev)
    stride = _written(out, "out", (t.rows, t.cols), dtype, dev)
    _launch("mx_dequantize", dev, lib.mx_dequantize, b._ptr(t.codes), b._ptr(t.scales), fcode, t.rows, t.cols,
            b._ptr(out), _float_code(out, "out"), stride, _status(dev_status, dev), stream)
    return out


def mx_linear(x: MXTensor, w: MXTensor, out_dtype=torch.bfloat16, *, out=None, dev_status=None, stream=None):
    """``x @ w.T`` of the values of x (e4m3, [n, h]) and the classifier w (e2m1, [v, h]):
    logits [n, v] in bfloat16 or float32.  dev_status is None or an int32 [1] tensor."""
    lib = b.library()
    _check_mx(x, "x")
    _check_mx(w, "w")
    dev = x.codes.device
    if x.fmt != "e4m3" or w.fmt != "e2m1":
        raise ValueError(f"x must be e4m3 and w e2m1, got {x.fmt} and {w.fmt}")
    if x.cols != w.cols or w.rows < 1:
        raise ValueError("x and w must share the hidden dimension, and w have rows")
    if w.codes.device != dev:
        raise ValueError("x and w are on different devices")
    if out is None:
        with _on_stream(stream):
            out = torch.empty(x.rows, w.rows, dtype=out_dtype, device=dev)
    stride = _written(out, "out", (x.rows, w.rows), out_dtype, dev)
    _launch("mx_linear", dev, lib.mx_linear, b._ptr(x.codes), b._ptr(x.scales), b._ptr(w.codes), b._ptr(w.scales),
            x.rows, x.cols, w.rows, b._ptr(out), _float_code(out, "out"), stride, _status(dev_status, dev), stream)
    return out


# ---------------------------------------------------------------------------
# the norm before the classifier
# ---------------------------------------------------------------------------

def _norm_inputs(x, weight, residual, h, stream):
    code = _float_code(x, "x")
    xs = _matrix(x, "x")
    n, hidden = x.shape
    if weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"weight must be bfloat16 or float32, got {weight.dtype}")
    _vector(weight, "weight", hidden, weight.dtype, x.device)
    rs = hs = hidden
    if residual is not None:
        rs = _matrix(residual, "residual", x.shape, x.dtype, x.device)
        if h is None:
            with _on_stream(stream):
                h = torch.empty(n, hidden, dtype=x.dtype, device=x.device)
        hs = _written(h, "h", x.shape, x.dtype, x.device)
    elif h is not None:
        raise ValueError("h is written only when a residual is given")
    return code, n, hidden, xs, rs, hs, h


def rms_norm_forward(x, weight, eps=1e-6, residual=None, *, h=None, y=None, rstd=None, dev_status=None,
                     stream=None):
    """Norm of x + residual over the last dimension of ``x`` [n, hidden].  Returns (y, h, rstd):
    h is the rounded sum (``x`` itself without a residual), rstd FP32 [n]."""
    lib = b.library()
    code, n, hidden, xs, rs, hs, h = _norm_inputs(x, weight, residual, h, stream)
    with _on_stream(stream):
        if y is None:
            y = torch.empty(n, hidden, dtype=x.dtype, device=x.device)
        if rstd is None:
            rstd = torch.empty(n, dtype=torch.float32, device=x.device)
    ys = _written(y, "y", x.shape, x.dtype, x.device)
    _vector(rstd, "rstd", n, torch.float32, x.device)
    _launch("rms_norm_forward", x.device, lib.rms_norm_forward, b._ptr(x), code, n, hidden, xs, b._ptr(residual),
            rs, b._ptr(weight), _float_code(weight, "weight"), float(eps), b._ptr(h), hs, b._ptr(y), ys,
            b._ptr(rstd), _status(dev_status, x.device), stream)
    return RMSNormForward(y, x if h is None else h, rstd)


def rms_norm_mx(x, weight, eps=1e-6, residual=None, *, h=None, out=None, rstd=None, dev_status=None, stream=None):
    """rms_norm_forward with y as an E4M3 microscaled tensor, mx_linear's input.  Returns
    (y: MXTensor, h, rstd); rstd only when a tensor is passed for it."""
    lib = b.library()
    code, n, hidden, xs, rs, hs, h = _norm_inputs(x, weight, residual, h, stream)
    if out is None:
        with _on_stream(stream):
            out = MXTensor.empty(n, hidden, "e4m3", x.device)
    else:
        _check_mx(out, "out")
        if (out.rows, out.cols, out.fmt) != (n, hidden, "e4m3") or out.codes.device != x.device:
            raise ValueError("out must be an e4m3 tensor of x's shape and device")
    if rstd is not None:
        _vector(rstd, "rstd", n, torch.float32, x.device)
    _launch("rms_norm_mx", x.device, lib.rms_norm_mx, b._ptr(x), code, n, hidden, xs, b._ptr(residual), rs,
            b._ptr(weight), _float_code(weight, "weight"), float(eps), b._ptr(h), hs, b._ptr(out.codes),
            b._ptr(out.scales), b._ptr(rstd), _status(dev_status, x.device), stream)
    return RMSNormMX(out, x if h is None else h, rstd)


def rms_norm_workspace_size(n: int, hidden: int) -> int:
    return int(b.library().rms_norm_workspace_size(n, hidden))


def rms_norm_backward(dy, h, weight, rstd, dh=None, *, dx=None, dweight=None, workspace=None, dev_status=None,
                      stream=None):
    """Backward of rms_norm_forward.  Returns (dx, dweight): dx is the gradient of x and of the
    residual; ``dh`` is the gradient that reaches h by another way."""
    lib = b.library()
    dev = dy.device
    code = _float_code(dy, "dy")
    gs = _matrix(dy, "dy")
    n, hidden = dy.shape
    hs = _matrix(h, "h", dy.shape, dy.dtype, dev)
    ds = hidden if dh is None else _matrix(dh, "dh", dy.shape, dy.dtype, dev)
    if weight.dtype not in (torch.bfloat16, torch.float32):
        raise TypeError(f"weight must be bfloat16 or float32, got {weight.dtype}")
    _vector(weight, "weight", hidden, weight.dtype, dev)
    _vector(rstd, "rstd", n, torch.float32, dev)
    with _on_stream(stream):
        if dx is None:
            dx = torch.empty(n, hidden, dtype=dy.dtype, device=dev)
        if dweight is None:
            dweight = torch.empty(hidden, dtype=weight.dtype, device=dev)
        if workspace is None:
            size = b._on(dev, lib.rms_norm_workspace_size, n, hidden)
            workspace = torch.empty(max(1, size), dtype=torch.uint8, device=dev)
    xs = _written(dx, "dx", dy.shape, dy.dtype, dev)
    _vector(dweight, "dweight", hidden, weight.dtype, dev)
    _launch("rms_norm_backward", dev, lib.rms_norm_backward, b._ptr(dy), code, n, hidden, gs, b._ptr(h), hs,
            b._ptr(weight), _float_code(weight, "weight"), b._ptr(rstd), b._ptr(dh), ds, b._ptr(dx), xs,
            b._ptr(dweight), b._ptr(workspace), workspace.numel() * workspace.element_size(),
            _status(dev_status, dev), stream)
    return RMSNormBackward(dx, dweight)


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

def _per_row(value, name, n, dtype, device):
    """A sampling parameter: None, a number for all rows, or a tensor with one entry per row."""
    if value is None:
        return None
    if isinstance(value, torch.Tensor):
        return _vector(value, name, n, dtype, device)
    return torch.full((n,), value, dtype=dtype, device=device)


def ce_sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, *, token=None, logprob=None,
              dev_status=None, stream=None):
    """One token per row of ``logits`` [..., V] (bfloat16 or float32) from ``uniform`` (float32 in
    [0, 1), one per row).  temperature, top_p, min_p (float32) and top_k (int32) are None, a
    number, or a tensor with one entry per row.  Returns (token int64, logprob, dev_status), the
    first two shaped like the leading dimensions; logprob is the logarithm of the probability
    the token was drawn with.  A row from which nothing can be drawn gives -1 and NaN."""
    lib = b.library()
    dev = logits.device
    code = _float_code(logits, "logits")
    n, vocab, stride = b._rows_view(logits)
    lead = logits.shape[:-1]
    _vector(uniform, "uniform", n, torch.float32, dev)
    with _on_stream(stream):
        temperature = _per_row(temperature, "temperature", n, torch.float32, dev)
        top_k = _per_row(top_k, "top_k", n, torch.int32, dev)
        top_p = _per_row(top_p, "top_p", n, torch.float32, dev)
        min_p = _per_row(min_p, "min_p", n, torch.float32, dev)
        if token is None:
            token = torch.empty(lead, dtype=torch.int64, device=dev)
        if logprob is None:
            logprob = torch.empty(lead, dtype=torch.float32, device=dev)
        if dev_status is None:
            dev_status = torch.zeros(1, dtype=torch.int32, device=dev)
    _vector(token, "token", n, torch.int64, dev)
    _vector(logprob, "logprob", n, torch.float32, dev)
    _launch("ce_sample", dev, lib.ce_sample, b._ptr(logits), code, n, vocab, stride, b._ptr(uniform),
            b._ptr(temperature), b._ptr(top_k), b._ptr(top_p), b._ptr(min_p), b._ptr(token), b._ptr(logprob),
            _status(dev_status, dev), stream)
    return CESample(token, logprob, dev_status)


def linear_sample(embeddings, classifier: MXTensor, uniform, temperature=None, top_k=None, top_p=None, min_p=None, *,
                  norm_weight=None, norm_eps=1e-6, residual=None, stream=None):
    """The next token after ``embeddings`` [..., H], the counterpart of linear_cross_entropy when a
    model answers: the norm (with ``norm_weight`` [H]; plus ``residual``) in 8 bits, the product
    with the 4-bit ``classifier``, and ce_sample of the logits.  Returns ce_sample's results."""
    lead, h = embeddings.shape[:-1], embeddings.shape[-1]
    x = embeddings.reshape(-1, h)
    if norm_weight is not None:
        res = None if residual is None else residual.reshape(-1, h)
        q = rms_norm_mx(x, norm_weight, norm_eps, res, stream=stream).y
    elif residual is not None:
        raise ValueError("residual is added by the norm: it needs norm_weight")
    else:
        q = mx_quantize(x, "e4m3", stream=stream)
    logits = mx_linear(q, classifier, torch.float32, stream=stream)
    r = ce_sample(logits, uniform, temperature, top_k, top_p, min_p, stream=stream)
    return CESample(r.token.view(lead), r.logprob.view(lead), r.dev_status)

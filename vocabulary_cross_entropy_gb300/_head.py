"""ctypes marshalling for the operators around the vocabulary cross entropy: the norm
before the classifier, microscaled tensors and their product, and sampling (see
include/vce.h for what each computes).  As in ``_binding``, torch tensors supply memory
and the current stream.

A call given ``stream`` runs as if that stream were current: what it was not given
(outputs and workspace) is allocated from it too, so memory it drops on return is reused
only behind its kernels.
"""
from __future__ import annotations

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

_CODES = {torch.bfloat16: b.BF16, torch.float32: b.F32}


def _under(stream, fn, first, *args, **kwargs):
    """fn with ``stream``, a stream of its first argument's device, current."""
    device = first[0].device if isinstance(first, tuple) else first.device
    if stream.device != device:  # its own current stream would be used instead
        raise ValueError(f"stream is on {stream.device}, the tensors are on {device}")
    with torch.cuda.stream(stream):
        return fn(first, *args, **kwargs)


def _float_code(dtype, name):
    code = _CODES.get(dtype)
    if code is None:
        raise TypeError(f"{name} must be bfloat16 or float32, got {dtype}")
    return code


def _rows_of(t, name):
    """(rows, cols, row stride) of a 2-D tensor with contiguous rows."""
    shape = t.shape
    if len(shape) != 2:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    n, c = shape
    rs, cs = t.stride()
    if cs != 1 and c > 1:
        raise ValueError(f"{name} must be a 2-D tensor with contiguous rows")
    return n, c, rs if n > 1 else c


def flat_rows(t):
    """``t`` [..., H] as [rows, H] with contiguous rows that do not overlap (a gradient may be
    expanded, an input transposed)."""
    flat = t.reshape(-1, t.shape[-1])
    return flat if flat.stride(-1) == 1 and flat.stride(0) >= flat.shape[1] else flat.contiguous()


def _same_rows(t, name, like):
    """Row stride of a tensor that has to match ``like`` in shape, type and device."""
    if t.shape != like.shape or t.dtype is not like.dtype or t.get_device() != like.get_device():
        raise ValueError(f"{name} must be a {like.dtype} tensor of shape {tuple(like.shape)} on {like.device}, got "
                         f"{t.dtype}, {tuple(t.shape)} on {t.device}")
    return _rows_of(t, name)[2]


def _written_rows(t, name, shape, dtype, index):
    """Row stride of an output the caller gave: its rows must not overlap."""
    if tuple(t.shape) != shape or t.dtype is not dtype or t.get_device() != index:
        raise ValueError(f"{name} must be a {dtype} tensor of shape {shape} on the inputs' device")
    n, c, stride = _rows_of(t, name)
    if stride < c:
        raise ValueError(f"the rows of {name} overlap")
    return stride


def _vector(t, name, n, dtype, index):
    if t.dtype is not dtype or t.numel() != n or t.get_device() != index or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} tensor of {n} elements on the inputs' device")
    return t


def _weight(t, hidden, index):
    code = _float_code(t.dtype, "weight")
    _vector(t, "weight", hidden, t.dtype, index)
    return code


def _launch(name, device, fn, *args):
    """fn(*args, current stream) of the library, once everything about the arguments has been checked."""
    index = device.index
    if index is None:
        raise ValueError(f"{name}: tensors must be on a CUDA device, got {device}")
    if b._raw_stream is not None and b._raw_device() == index:  # the common case, without detours
        st = fn(*args, b._raw_stream(index))
    else:
        st = b._on(device, fn, *args, b._stream(device, None))
    if st:
        b._check(name, st)


def _status(t, index):
    return None if t is None else _vector(t, "dev_status", 1, torch.int32, index).data_ptr()


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
        tiles = -(-cols // 128)
        codes = torch.empty((rows, tiles * (64 if fmt == "e2m1" else 128)), dtype=torch.uint8, device=device)
        scales = torch.empty((-(-rows // 128), tiles, 32, 4, 4), dtype=torch.uint8, device=device)
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
    """Format code of a microscaled tensor whose buffers have the sizes its shape needs."""
    codes, scales, rows, cols, fmt = t
    code = _fmt(fmt)
    if rows < 0 or cols < 1:
        raise ValueError(f"{name}: rows and cols must be positive")
    padded = -(-cols // 128) * 128
    for part, what, size in ((codes, "codes", rows * padded >> code),
                             (scales, "scales", -(-rows // 128) * padded * 4)):
        if part.dtype is not torch.uint8 or part.numel() != size or not part.is_contiguous():
            raise ValueError(f"{name}.{what} must be a contiguous uint8 tensor of {size} bytes")
    if codes.get_device() != scales.get_device():
        raise ValueError(f"{name}: codes and scales are on different devices")
    return code


def mx_codes_size(rows: int, cols: int, fmt: str) -> int:
    return int(b.library().mx_codes_size(rows, cols, _fmt(fmt)))


def mx_scales_size(rows: int, cols: int) -> int:
    return int(b.library().mx_scales_size(rows, cols))


def mx_quantize(x, fmt="e2m1", *, out=None, dev_status=None, stream=None) -> MXTensor:
    """``x`` [rows, cols] (bfloat16 or float32) as a microscaled tensor."""
    if stream is not None:
        return _under(stream, mx_quantize, x, fmt, out=out, dev_status=dev_status)
    code, fcode = _float_code(x.dtype, "x"), _fmt(fmt)
    rows, cols, stride = _rows_of(x, "x")
    dev, index = x.device, x.get_device()
    if out is None:
        out = MXTensor.empty(rows, cols, fmt, dev)
    else:
        _check_mx(out, "out")
        if out[2:] != (rows, cols, fmt) or out.codes.get_device() != index:
            raise ValueError("out must have x's shape and device, and the format asked for")
    _launch("mx_quantize", dev, b.library().mx_quantize, x.data_ptr(), code, rows, cols, stride, fcode,
            out.codes.data_ptr(), out.scales.data_ptr(), _status(dev_status, index))
    return out


def mx_dequantize(t: MXTensor, dtype=torch.bfloat16, *, out=None, dev_status=None, stream=None):
    """The values of a microscaled tensor, [rows, cols] in bfloat16 or float32."""
    if stream is not None:
        return _under(stream, mx_dequantize, t, dtype, out=out, dev_status=dev_status)
    fcode, code = _check_mx(t, "t"), _float_code(dtype, "dtype")
    codes, scales, rows, cols, _ = t
    dev, index = codes.device, codes.get_device()
    stride = cols
    if out is None:
        out = torch.empty(rows, cols, dtype=dtype, device=dev)
    else:
        stride = _written_rows(out, "out", (rows, cols), dtype, index)
    _launch("mx_dequantize", dev, b.library().mx_dequantize, codes.data_ptr(), scales.data_ptr(), fcode,
            rows, cols, out.data_ptr(), code, stride, _status(dev_status, index))
    return out


def mx_linear(x: MXTensor, w: MXTensor, out_dtype=torch.bfloat16, *, out=None, dev_status=None, stream=None):
    """``x @ w.T`` of the values of x (e4m3, [n, h]) and the classifier w (e2m1, [v, h]):
    logits [n, v] in bfloat16 or float32.  Only ``dev_status`` (an int32 [1] tensor, its bits set
    by the call) tells of a pipeline wait that gave up, after which logits are missing."""
    if stream is not None:
        return _under(stream, mx_linear, x, w, out_dtype, out=out, dev_status=dev_status)
    if (_check_mx(x, "x"), _check_mx(w, "w")) != (MX_E4M3, MX_E2M1):
        raise ValueError(f"x must be e4m3 and w e2m1, got {x.fmt} and {w.fmt}")
    xc, xs, n, h, _ = x
    wc, ws, v, wh, _ = w
    dev, index = xc.device, xc.get_device()
    if h != wh or v < 1:
        raise ValueError("x and w must share the hidden dimension, and w have rows")
    if wc.get_device() != index:
        raise ValueError("x and w are on different devices")
    code, stride = _float_code(out_dtype, "out_dtype"), v
    if out is None:
        out = torch.empty(n, v, dtype=out_dtype, device=dev)
    else:
        stride = _written_rows(out, "out", (n, v), out_dtype, index)
    _launch("mx_linear", dev, b.library().mx_linear, xc.data_ptr(), xs.data_ptr(), wc.data_ptr(),
            ws.data_ptr(), n, h, v, out.data_ptr(), code, stride, _status(dev_status, index))
    return out


# ---------------------------------------------------------------------------
# the norm before the classifier
# ---------------------------------------------------------------------------

def _norm_inputs(x, weight, residual, h):
    """What both norms hand to the library: (x's type, n, hidden, x's stride, residual, its stride,
    weight, its type), then h's pointer and stride, the device's index, and h itself."""
    code = _float_code(x.dtype, "x")
    n, hidden, xs = _rows_of(x, "x")
    index = x.get_device()
    wcode = _weight(weight, hidden, index)
    if residual is None:
        if h is not None:
            raise ValueError("h is written only when a residual is given")
        return (code, n, hidden, xs, None, hidden, weight.data_ptr(), wcode), None, hidden, index, x
    rs, hs = _same_rows(residual, "residual", x), hidden
    if h is None:
        h = torch.empty(n, hidden, dtype=x.dtype, device=x.device)
    else:
        hs = _written_rows(h, "h", (n, hidden), x.dtype, index)
    return (code, n, hidden, xs, residual.data_ptr(), rs, weight.data_ptr(), wcode), h.data_ptr(), hs, index, h


def rms_norm_forward(x, weight, eps=1e-6, residual=None, *, h=None, y=None, rstd=None, dev_status=None,
                     stream=None):
    """Norm of x + residual over the last dimension of ``x`` [n, hidden].  Returns (y, h, rstd):
    h is the rounded sum (``x`` itself without a residual), rstd FP32 [n]."""
    if stream is not None:
        return _under(stream, rms_norm_forward, x, weight, eps, residual, h=h, y=y, rstd=rstd, dev_status=dev_status)
    args, hp, hs, index, h = _norm_inputs(x, weight, residual, h)
    n, hidden = args[1], args[2]
    dev, ys = x.device, hidden
    if y is None:
        y = torch.empty(n, hidden, dtype=x.dtype, device=dev)
    else:
        ys = _written_rows(y, "y", (n, hidden), x.dtype, index)
    if rstd is None:
        rstd = torch.empty(n, dtype=torch.float32, device=dev)
    else:
        _vector(rstd, "rstd", n, torch.float32, index)
    _launch("rms_norm_forward", dev, b.library().rms_norm_forward, x.data_ptr(), *args, eps, hp, hs,
            y.data_ptr(), ys, rstd.data_ptr(), _status(dev_status, index))
    return RMSNormForward(y, h, rstd)


def rms_norm_mx(x, weight, eps=1e-6, residual=None, *, h=None, out=None, rstd=None, dev_status=None, stream=None):
    """rms_norm_forward with y as an E4M3 microscaled tensor, mx_linear's input.  Returns
    (y: MXTensor, h, rstd); rstd only when a tensor is passed for it."""
    if stream is not None:
        return _under(stream, rms_norm_mx, x, weight, eps, residual, h=h, out=out, rstd=rstd, dev_status=dev_status)
    args, hp, hs, index, h = _norm_inputs(x, weight, residual, h)
    n, hidden = args[1], args[2]
    if out is None:
        out = MXTensor.empty(n, hidden, "e4m3", x.device)
    else:
        _check_mx(out, "out")
        if out[2:] != (n, hidden, "e4m3") or out.codes.get_device() != index:
            raise ValueError("out must be an e4m3 tensor of x's shape and device")
    if rstd is not None:
        _vector(rstd, "rstd", n, torch.float32, index)
    _launch("rms_norm_mx", x.device, b.library().rms_norm_mx, x.data_ptr(), *args, eps, hp, hs,
            out.codes.data_ptr(), out.scales.data_ptr(), b._ptr(rstd), _status(dev_status, index))
    return RMSNormMX(out, h, rstd)


def rms_norm_workspace_size(n: int, hidden: int) -> int:
    return int(b.library().rms_norm_workspace_size(n, hidden))


def rms_norm_backward(dy, h, weight, rstd, dh=None, *, dx=None, dweight=None, workspace=None, dev_status=None,
                      stream=None):
    """Backward of rms_norm_forward.  Returns (dx, dweight): dx is the gradient of x and of the
    residual; ``dh`` is the gradient that reaches h by another way."""
    if stream is not None:
        return _under(stream, rms_norm_backward, dy, h, weight, rstd, dh, dx=dx, dweight=dweight, workspace=workspace,
                      dev_status=dev_status)
    lib = b.library()
    dev, index = dy.device, dy.get_device()
    code = _float_code(dy.dtype, "dy")
    n, hidden, gs = _rows_of(dy, "dy")
    hs = _same_rows(h, "h", dy)
    ds = hidden if dh is None else _same_rows(dh, "dh", dy)
    wcode = _weight(weight, hidden, index)
    _vector(rstd, "rstd", n, torch.float32, index)
    xs = hidden
    if dx is None:
        dx = torch.empty(n, hidden, dtype=dy.dtype, device=dev)
    else:
        xs = _written_rows(dx, "dx", (n, hidden), dy.dtype, index)
    if dweight is None:
        dweight = torch.empty(hidden, dtype=weight.dtype, device=dev)
    else:
        _vector(dweight, "dweight", hidden, weight.dtype, index)
    if workspace is None:
        size = b._on(dev, lib.rms_norm_workspace_size, n, hidden)
        workspace = torch.empty(size or 1, dtype=torch.uint8, device=dev)
    elif workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the inputs' device")
    _launch("rms_norm_backward", dev, lib.rms_norm_backward, dy.data_ptr(), code, n, hidden, gs,
            h.data_ptr(), hs, weight.data_ptr(), wcode, rstd.data_ptr(), b._ptr(dh), ds, dx.data_ptr(), xs,
            dweight.data_ptr(), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
            _status(dev_status, index))
    return RMSNormBackward(dx, dweight)


# ---------------------------------------------------------------------------
# sampling
# ---------------------------------------------------------------------------

_I32_MAX, _F32_MAX = 2 ** 31 - 1, torch.finfo(torch.float32).max


def _param(value, name, n, dtype, index):
    """A sampling parameter, checked: None, a tensor with one entry per row, or a number for all rows
    (one that ``dtype`` cannot hold becomes its largest, which filters as it would)."""
    if value is None:
        return None
    if isinstance(value, torch.Tensor):
        return _vector(value, name, n, dtype, index)
    if dtype is torch.float32:
        return max(min(value, _F32_MAX), -_F32_MAX)  # (a NaN stays one)
    value = max(min(value, _I32_MAX), -1)
    if value != value or value != int(value):
        raise ValueError(f"{name} must be a whole number, got {value}")
    return int(value)


def _params(uniform, temperature, top_k, top_p, min_p, n, index):
    """Checks ``uniform`` and the four parameters; returns the latter."""
    _vector(uniform, "uniform", n, torch.float32, index)
    return (_param(temperature, "temperature", n, torch.float32, index), _param(top_k, "top_k", n, torch.int32, index),
            _param(top_p, "top_p", n, torch.float32, index), _param(min_p, "min_p", n, torch.float32, index))


def _per_row(value, n, dtype, device):
    return value if value is None or isinstance(value, torch.Tensor) else \
        torch.full((n,), value, dtype=dtype, device=device)


def _sample(logits, code, n, vocab, stride, uniform, params, token, logprob, status):
    """The library's call, all arguments checked; numbers among ``params`` become tensors."""
    dev, f32 = logits.device, torch.float32
    temperature, top_k, top_p, min_p = params
    t, k = _per_row(temperature, n, f32, dev), _per_row(top_k, n, torch.int32, dev)
    p, m = _per_row(top_p, n, f32, dev), _per_row(min_p, n, f32, dev)
    ptr = b._ptr
    _launch("ce_sample", dev, b.library().ce_sample, logits.data_ptr(), code, n, vocab, stride,
            uniform.data_ptr(), ptr(t), ptr(k), ptr(p), ptr(m), token.data_ptr(), logprob.data_ptr(), status)


def ce_sample(logits, uniform, temperature=None, top_k=None, top_p=None, min_p=None, *, token=None, logprob=None,
              dev_status=None, stream=None):
    """One token per row of ``logits`` [..., V] (bfloat16 or float32) from ``uniform`` (float32 in
    [0, 1), one per row).  temperature, top_p, min_p (float32) and top_k (int32) are None, a
    number, or a tensor with one entry per row.  Returns (token int64, logprob, dev_status), the
    first two shaped like the leading dimensions; logprob is the logarithm of the probability
    the token was drawn with.  A row from which nothing can be drawn gives -1 and NaN, and sets
    a bit of ``dev_status`` (int32 [1]) where one is passed."""
    if stream is not None:
        return _under(stream, ce_sample, logits, uniform, temperature, top_k, top_p, min_p, token=token,
                      logprob=logprob, dev_status=dev_status)
    dev, index = logits.device, logits.get_device()
    code = _float_code(logits.dtype, "logits")
    n, vocab, stride = b._rows_view(logits)
    lead = logits.shape[:-1]
    params = _params(uniform, temperature, top_k, top_p, min_p, n, index)
    if token is None:
        token = torch.empty(lead, dtype=torch.int64, device=dev)
    else:
        _vector(token, "token", n, torch.int64, index)
    if logprob is None:
        logprob = torch.empty(lead, dtype=torch.float32, device=dev)
    else:
        _vector(logprob, "logprob", n, torch.float32, index)
    _sample(logits, code, n, vocab, stride, uniform, params, token, logprob, _status(dev_status, index))
    return CESample(token, logprob, dev_status)


def linear_sample(embeddings, classifier: MXTensor, uniform, temperature=None, top_k=None, top_p=None, min_p=None, *,
                  norm_weight=None, norm_eps=1e-6, residual=None, dev_status=None, stream=None):
    """The next token after ``embeddings`` [..., H], the counterpart of linear_cross_entropy when a
    model answers: the norm (with ``norm_weight`` [H]; plus ``residual``) in 8 bits, the product
    with the 4-bit ``classifier``, and ce_sample of the logits.  Returns ce_sample's results, with
    a zeroed ``dev_status`` of its own where none is passed: mx_linear's bits are in it too."""
    if stream is not None:
        return _under(stream, linear_sample, embeddings, classifier, uniform, temperature, top_k, top_p, min_p,
                      norm_weight=norm_weight, norm_eps=norm_eps, residual=residual, dev_status=dev_status)
    lead, h, v, index = embeddings.shape[:-1], embeddings.shape[-1], classifier.rows, embeddings.get_device()
    n = lead.numel()
    # what the norm and the quantisation do not check themselves, before either is launched
    if _check_mx(classifier, "classifier") != MX_E2M1 or classifier.cols != h:
        raise ValueError(f"classifier must be e2m1 with {h} columns, got {classifier.fmt} with {classifier.cols}")
    if not 1 <= v <= SAMPLE_MAX_VOCAB:
        raise ValueError(f"classifier must have 1 to {SAMPLE_MAX_VOCAB} rows, got {v}")
    if classifier.codes.get_device() != index:
        raise ValueError("embeddings and classifier are on different devices")
    params = _params(uniform, temperature, top_k, top_p, min_p, n, index)
    _status(dev_status, index)
    if residual is not None and norm_weight is None:
        raise ValueError("residual is added by the norm: it needs norm_weight")
    if residual is not None and residual.shape != embeddings.shape:
        raise ValueError("residual must have the shape of embeddings")
    if dev_status is None:
        dev_status = torch.zeros(1, dtype=torch.int32, device=embeddings.device)
    x = flat_rows(embeddings)
    if norm_weight is not None:
        res = None if residual is None else flat_rows(residual)
        q = rms_norm_mx(x, norm_weight, norm_eps, res, dev_status=dev_status).y
    else:
        q = mx_quantize(x, "e4m3", dev_status=dev_status)
    # rows a multiple of 32 bytes apart: mx_linear stores, and ce_sample loads, whole sectors
    logits = torch.empty(n, -(-v // 8) * 8, dtype=torch.float32, device=x.device)
    mx_linear(q, classifier, torch.float32, out=logits[:, :v], dev_status=dev_status)
    token = torch.empty(lead, dtype=torch.int64, device=x.device)
    logprob = torch.empty(lead, dtype=torch.float32, device=x.device)
    _sample(logits, b.F32, n, v, logits.shape[1], uniform, params, token, logprob, dev_status.data_ptr())
    return CESample(token, logprob, dev_status)

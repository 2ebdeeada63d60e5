"""torch.autograd front ends over the C ABI (marshalling only: every step runs in
libvce.so's kernels).

parallel_cross_entropy  the logits form, with the call shape of Transformer
                        Engine's parallel_cross_entropy (API card "Signature")
                        minus the process group; ``overwrite_input`` is the
                        pull request's destructive mode (backward writes the
                        gradient over the saved logits).
linear_cross_entropy    the linear form, loss from embeddings [..., H] and the
                        classifier [V, H] (Cut Cross-Entropy card
                        "what_it_does"), with optional token shifting and
                        per-token entropy, and optionally the norm before
                        the classifier.
rms_norm                that norm with the residual's addition, by itself.
"""
from __future__ import annotations

import torch
from torch.autograd.function import once_differentiable

from . import _binding as b
from . import _head
from ._head import flat_rows


def _grad_tensor(grad, reduce_code, n, device):
    if reduce_code:
        return grad.reshape(1).to(device=device, dtype=torch.float32)
    return grad.reshape(n).to(device=device, dtype=torch.float32).contiguous()


class _LogitsCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, inp, target, label_smoothing, reduce_code, ignore_idx, overwrite_input):
        flat_t = target.reshape(-1).contiguous()
        f = b.ce_forward(inp, flat_t, label_smoothing, reduce_code, ignore_idx)
        ctx.save_for_backward(inp, flat_t, f.stats, f.n_valid)
        ctx.args = (label_smoothing, reduce_code, ignore_idx, overwrite_input)
        return f.loss.reshape(()) if reduce_code else f.loss.reshape(target.shape)

    @staticmethod
    def backward(ctx, grad):
        inp, flat_t, stats, n_valid = ctx.saved_tensors
        eps, reduce_code, ignore_idx, overwrite = ctx.args
        g = _grad_tensor(grad, reduce_code, flat_t.numel(), inp.device)
        dz = b.ce_backward(inp, flat_t, stats, n_valid, g, eps, reduce_code, ignore_idx, inplace=overwrite)
        return dz.detach(), None, None, None, None, None


def parallel_cross_entropy(inp, target, label_smoothing: float = 0.0, reduce_loss: bool = False,
                           dist_process_group=None, ignore_idx: int = -100, is_cg_capturable: bool = False,
                           overwrite_input: bool = False):
    """Cross entropy of logits ``inp`` (B, SQ, V) or (SQ, B, V) against ``target``.

    Returns the mean over non-ignored tokens when ``reduce_loss``, else the per-token
    loss shaped like ``target``.  Every call is CUDA-graph capturable, so
    ``is_cg_capturable`` has no effect.  With ``overwrite_input`` the backward writes
    the gradient over ``inp`` (no extra buffer); ``inp`` must not be used afterwards.
    """
    if dist_process_group is not None:
        raise NotImplementedError("vocabulary-parallel process groups are not supported: one GPU")
    del is_cg_capturable
    code = b._reduce(reduce_loss)
    return _LogitsCE.apply(inp, target, float(label_smoothing), code, int(ignore_idx), bool(overwrite_input))


class _LinearCE(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, w, target, label_smoothing, reduce_code, ignore_idx, want_entropy):
        f = b.lce_forward(x, w, target, label_smoothing, reduce_code, ignore_idx, entropy=want_entropy)
        ctx.save_for_backward(x, w, target, f.lse, f.n_valid)
        ctx.args = (label_smoothing, reduce_code, ignore_idx)
        loss = f.loss.reshape(()) if reduce_code else f.loss
        if want_entropy:
            ctx.mark_non_differentiable(f.entropy)
            return loss, f.entropy
        return loss

    @staticmethod
    def backward(ctx, grad, *unused):
        x, w, target, lse, n_valid = ctx.saved_tensors
        eps, reduce_code, ignore_idx = ctx.args
        g = _grad_tensor(grad, reduce_code, target.numel(), x.device)
        r = b.lce_backward(x, w, target, lse, n_valid, g, eps, reduce_code, ignore_idx)
        return r.dX, r.dW, None, None, None, None, None


_NOTE = "vce_stream"


def _accumulators(*tensors):
    """What adds to the .grad of those ``tensors`` that are leaves; the caller keeps them until
    the graph does.

    torch makes one such node per leaf, which lives as long as any graph of the leaf and works
    on the stream that it was made on.  A graph that is captured while an eager one of the same
    leaves is alive, made on the default stream, would draw that stream into the capture:
    refused here, where nothing has been launched yet, as torch's own failure in the backward
    pass can end the process."""
    nodes = []
    for t in tensors:
        if t is None or not (t.is_leaf and t.requires_grad and t.is_cuda):
            continue
        node = torch.autograd.graph.get_gradient_edge(t).node
        if _NOTE not in node.metadata:
            # the note outlives the node's name here only if something else holds the node,
            # which was then made at an unknown time; otherwise the next one is made now
            node.metadata[_NOTE] = None
            del node
            node = torch.autograd.graph.get_gradient_edge(t).node
            node.metadata.setdefault(_NOTE, torch.cuda.current_stream(t.device).cuda_stream)
        if node.metadata[_NOTE] == 0 and torch.cuda.is_current_stream_capturing():
            raise RuntimeError("an earlier result computed from the same parameters is still alive: drop it "
                               "(or detach it) before the forward and backward pass are captured into a graph")
        nodes.append(node)
    return nodes


class _RMSNorm(torch.autograd.Function):
    # takes and gives back x's own shape: the gradient of x and of the residual is then one
    # tensor with two owners, which autograd copies before it makes it a leaf's .grad (views
    # made outside would each look like the only owner).  The outputs are made in that shape
    # and the library gets views of them: an output that is a view may not be changed in place.
    @staticmethod
    def forward(ctx, x, weight, residual, eps):
        rows = (-1, x.shape[-1])
        y = torch.empty(x.shape, dtype=x.dtype, device=x.device)
        h = None if residual is None else torch.empty_like(y)
        flat = flat_rows(x)
        f = _head.rms_norm_forward(flat, weight, eps, None if residual is None else flat_rows(residual),
                                   h=None if h is None else h.view(rows), y=y.view(rows))
        # h itself, not a view of it, and x likewise unless its rows had to be copied
        kept = h if h is not None else x if flat.data_ptr() == x.data_ptr() else flat
        ctx.save_for_backward(kept, weight, f.rstd)
        ctx.set_materialize_grads(False)
        ctx.with_residual = residual is not None
        return y if h is None else (y, h)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy, dh=None):
        if dy is None:  # only the residual stream was used, or nothing
            dx, dweight = dh, None
        else:
            h, weight, rstd = ctx.saved_tensors
            dx, dweight = _head.rms_norm_backward(flat_rows(dy), flat_rows(h), weight, rstd,
                                                  None if dh is None else flat_rows(dh))
            dx, dweight = dx.view(dy.shape), dweight.view(weight.shape)
        return dx, dweight, dx if ctx.with_residual else None, None


def rms_norm(x, weight, eps: float = 1e-6, residual=None):
    """Root-mean-square norm of ``x`` [..., H] (plus ``residual``, of the same shape) over its
    last dimension, times ``weight`` [H].

    Returns y, or (y, x + residual) when a residual is given; both take part in the backward
    pass.  x and residual are BF16 or FP32, weight either.
    """
    if residual is not None and residual.shape != x.shape:
        raise ValueError("residual must have the shape of x")
    nodes = _accumulators(x, weight, residual) if torch.is_grad_enabled() else None
    out = _RMSNorm.apply(x, weight, residual, float(eps))
    del nodes  # the graph holds them now
    return out


def linear_cross_entropy(embeddings, classifier, labels, ignore_index: int = -100, reduction: str = "mean",
                         label_smoothing: float = 0.0, shift: bool = False, return_entropy: bool = False,
                         norm_weight=None, norm_eps: float = 1e-6, residual=None):
    """Cross entropy of ``embeddings @ classifier.T`` against ``labels`` without the logits.

    embeddings [..., H] and classifier [V, H] are BF16; labels [...] int64.  ``reduction``
    is 'mean' (over non-ignored tokens), 'sum' or 'none'.  ``shift`` scores position t
    of each sequence (the last dimension of ``labels``) against label t + 1.  With
    ``return_entropy`` the per-token entropy of the softmax is returned as well.  With
    ``norm_weight`` [H] the classifier takes rms_norm(embeddings, norm_weight, norm_eps,
    residual): the last norm of a model, whose gradients are part of the backward pass.

    To capture forward and backward in a CUDA graph, first drop every earlier result computed
    from the same parameters on the default stream: torch cannot capture a backward pass beside
    one, and its failure can end the process.  (rms_norm, the norm here included, refuses such a
    capture for its own leaves; to look for the classifier's would add half again to the time
    of a small call.)
    """
    if norm_weight is not None:
        out = rms_norm(embeddings, norm_weight, norm_eps, residual)
        embeddings = out if residual is None else out[0]
    elif residual is not None:
        raise ValueError("residual is added by the norm: it needs norm_weight")
    lead = embeddings.shape[:-1]
    h = embeddings.shape[-1]
    x = embeddings.reshape(-1, h)
    if not x.is_contiguous():
        x = x.contiguous()
    flat = labels.reshape(-1).contiguous()
    if shift:
        flat = b.shift_targets(flat, labels.shape[-1], ignore_index)
    code = b._reduce(reduction)
    out = _LinearCE.apply(x, classifier, flat, float(label_smoothing), code, int(ignore_index),
                          bool(return_entropy))
    loss, ent = (out if return_entropy else (out, None))
    if code == b.REDUCE_NONE:
        loss = loss.reshape(lead)
    if return_entropy:
        return loss, ent.reshape(lead)
    return loss

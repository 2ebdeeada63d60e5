"""FP64 NumPy definitions of beam search's step and of what follows it: the choice of the next
hypotheses, the reordering of the beams' states, and low-rank adapters beside a shared
projection.  Independent of the library and of torch."""
from __future__ import annotations

import numpy as np


def beam_step(z, score, ended=None, length=None, end=-1, penalty=0.0, count=None, keep=False):
    """(token, parent, score, ended, length), each [B, count], of logits z [B, K, V] and score [B, K]."""
    z, score = np.asarray(z, np.float64), np.asarray(score, np.float64)
    bs, k, v = z.shape
    count = k if count is None else count
    ended = np.zeros((bs, k), bool) if ended is None else np.asarray(ended, bool)
    length = np.zeros((bs, k), np.int64) if length is None else np.asarray(length, np.int64)
    token, parent = np.full((bs, count), -1), np.tile(np.arange(count) % k, (bs, 1))
    out, done, size = np.full((bs, count), -np.inf), np.zeros((bs, count), bool), np.zeros((bs, count), np.int64)
    for b in range(bs):
        beam, tok, c, logit = [], [], [], []
        for j in range(k):
            if not np.isfinite(score[b, j]):
                continue
            if ended[b, j]:
                beam.append([j]), tok.append([end]), c.append([score[b, j]]), logit.append([0.0])
                continue
            m = z[b, j].max()
            if not np.isfinite(m):
                continue
            with np.errstate(under="ignore"):
                lp = (z[b, j] - m) - np.log(np.exp(z[b, j] - m).sum())
            allowed = np.flatnonzero(z[b, j] > -np.inf)
            beam.append(np.full(len(allowed), j)), tok.append(allowed), c.append(score[b, j] + lp[allowed])
            logit.append(z[b, j][allowed])
        size[b] = length[b][parent[b]]
        if not c:
            continue
        beam, tok, c, logit = (np.concatenate(x) for x in (beam, tok, c, logit))
        after = length[b][beam] + ~ended[b][beam]
        value = c / np.maximum(after, 1).astype(np.float64) ** penalty
        order = np.lexsort((tok, -logit, beam, -value))[:count]  # (within a beam: the logits' order)
        places = list(range(len(order)))
        if keep:
            free, places = list(range(k)), [None] * len(order)
            for i, o in enumerate(order):
                if beam[o] in free:
                    places[i] = int(beam[o])
                    free.remove(beam[o])
            for i in range(len(order)):
                if places[i] is None:
                    places[i] = free.pop(0)
        for p, o in zip(places, order):
            token[b, p], parent[b, p], out[b, p] = tok[o], beam[o], c[o]
            done[b, p], size[b, p] = ended[b, beam[o]] or tok[o] == end, after[o]
    return token, parent, out, done, size


def reorder(x, parent, lengths=None, position_dim=None):
    """x [B * K, ...] with row (b, k) from (b, parent[b, k]) for the first lengths[b] positions."""
    bs, k = parent.shape
    y = np.array(x)
    for b in range(bs):
        for j in range(k):
            p = parent[b, j] if 0 <= parent[b, j] < k else j
            if lengths is None:
                y[b * k + j] = x[b * k + p]
            else:
                at = (slice(None),) * (position_dim - 1) + (slice(0, max(0, int(lengths[b]))),)
                y[b * k + j][at] = x[b * k + p][at]
    return y


def adapter_linear(y, x, a, b, index, scale=None):
    """y [N, V] + scale_i x A_i^T B_i^T with i = index[n]; rows whose index names no adapter stay."""
    out = np.array(y, np.float64)
    for n, i in enumerate(index):
        if 0 <= i < len(a):
            s = 1.0 if scale is None else np.float64(scale[i])
            out[n] += s * ((np.asarray(x[n], np.float64) @ np.asarray(a[i], np.float64).T) @ np.asarray(b[i], np.float64).T)
    return out

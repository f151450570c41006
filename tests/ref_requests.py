"""Plain 64-bit references, in numpy, of the operators for requests with
adapters and for beam search."""
import numpy as np


def lora(y, x, a, b, scale, ids):
    """(out, bound on the sums' size): what the adapters add, and for each
    element sum_j sum_k |x a b| * scale and max_j |u| * sum_j |b| * scale."""
    out = y.copy()
    size = np.zeros_like(y)
    split = np.zeros_like(y)
    for m, i in enumerate(ids):
        if 0 <= i < len(a):
            s = 1.0 if scale is None else scale[i]
            u = a[i] @ x[m]
            out[m] += s * (b[i] @ u)
            size[m] = abs(s) * (np.abs(b[i]) @ (np.abs(a[i]) @ np.abs(x[m])))
            split[m] = abs(s) * np.abs(u).max() * np.abs(b[i]).sum(-1)
    return out, size, split


def log_softmax(l):
    """Per row; NaN counts as -inf, +inf takes a row's whole probability."""
    l = np.where(np.isnan(l), -np.inf, l)
    top = l.max(-1, keepdims=True)
    with np.errstate(invalid="ignore", over="ignore"):
        d = np.where(l == -np.inf, -np.inf, l - np.where(np.isfinite(top), top, 0.0))
        out = d - np.log(np.exp(d).sum(-1, keepdims=True))
    out = np.where(top == np.inf, np.where(l == np.inf, 0.0, -np.inf), out)
    return np.where(top == -np.inf, -np.inf, out)


def beam_select(logits, scores, eos, anchored):
    """(tokens, parents, scores, ended, gap): gap is the least distance of two
    scores of different beams that decided something."""
    batch, beams, n = logits.shape
    tokens = np.full((batch, beams), -1, np.int64)
    parents = np.full((batch, beams), -1, np.int64)
    best = np.full((batch, beams), -np.inf)
    ended = np.full((batch, beams), -np.inf)
    gap = np.inf
    for i in range(batch):
        c = np.where(np.isfinite(scores[i]), scores[i], -np.inf)
        s = c[:, None] + log_softmax(logits[i])
        end = np.full(beams, -np.inf)
        if eos >= 0:
            end = s[:, eos].copy()
            s[:, eos] = -np.inf
        flat = s.reshape(-1)
        # (score, beam, token): stable, by descending score
        order = np.argsort(-flat, kind="stable")[:beams + 1]
        near = flat[order][np.isfinite(flat[order])]
        who = (order // n)[:len(near)]
        d = np.abs(np.diff(near))
        d = d[(who[1:] != who[:-1]) & (d > 0)]
        gap = min(gap, d.min() if d.size else np.inf)
        order = [int(o) for o in order[:beams] if flat[o] > -np.inf]
        for w in range(beams):
            if end[w] > -np.inf:
                d = np.abs(np.concatenate((flat[order], end)) - end[w])
                d = d[d > 0]
                gap = min(gap, d.min() if d.size else np.inf)
                if (flat[order] > end[w]).sum() + (end > end[w]).sum() < beams:
                    ended[i, w] = end[w]
        slots = list(range(len(order)))
        if anchored:
            slots, free = [None] * len(order), []
            seen = set()
            for r, o in enumerate(order):
                if o // n not in seen:
                    seen.add(o // n)
                    slots[r] = o // n
            free = [j for j in range(beams) if j not in seen]
            slots = [free.pop(0) if v is None else v for v in slots]
        for r, o in zip(slots, order):
            tokens[i, r], parents[i, r], best[i, r] = o % n, o // n, flat[o]
    return tokens, parents, best, ended, gap


def reorder(state, parents, lengths, dim):
    """A copy of state [rows, ...] with its rows moved."""
    new = state.copy()
    batch, beams = parents.shape
    for i in range(batch):
        for j in range(beams):
            p = int(parents[i, j])
            if 0 <= p < beams:
                index = [slice(None)] * (state.ndim - 1)
                if lengths is not None:
                    index[dim - 1] = slice(0, max(0, int(lengths[i])))
                new[(i * beams + j, *index)] = state[(i * beams + p, *index)]
    return new

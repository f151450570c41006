"""64-bit references of the operators around the head (norm, microscaled codes
and their product, sampling), written from the definitions in include/wql.h in
numpy, without any of the library's code."""
from __future__ import annotations

import numpy as np
import torch

EMAX = {0: 2, 1: 8}                       # MX_FP4, MX_FP8
FP4 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def f64(t: torch.Tensor) -> np.ndarray:
    return t.detach().cpu().double().numpy()


def fp8_table() -> np.ndarray:
    """The 256 values of e4m3 ("fn")."""
    c = np.arange(256)
    s, e, m = np.where(c >> 7, -1.0, 1.0), (c >> 3) & 15, (c & 7).astype(float)
    v = np.where(e > 0, (1 + m / 8) * 2.0 ** (e - 7.0), m / 8 * 2.0 ** -6)
    return np.where((c & 127) == 127, np.nan, s * v)


def grid(fmt: int) -> np.ndarray:
    """Non-negative finite elements of a format, by code."""
    return FP4 if fmt == 0 else fp8_table()[:127]


def nearest_code(a: np.ndarray, g: np.ndarray) -> np.ndarray:
    """Code of the element nearest to a >= 0, ties to the even code."""
    hi = np.clip(np.searchsorted(g, a), 0, len(g) - 1)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - g[lo], g[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(a >= g[-1], len(g) - 1, np.where(up, hi, lo))


def mx_quantize(x: np.ndarray, fmt: int):
    """(codes uint8, scale bytes [rows, k/32]) by the definition; finite or not."""
    rows, k = x.shape
    b = x.reshape(rows, k // 32, 32)
    am = np.abs(b).max(-1)
    bad = ~np.isfinite(am)
    e = np.where(am > 0, np.frexp(np.where(bad, 1.0, am))[1] - 1 - EMAX[fmt], -127)
    e = np.maximum(e, -127)
    with np.errstate(invalid="ignore"):
        v = b / (2.0 ** e)[..., None]
        code = nearest_code(np.where(np.isfinite(v), np.abs(v), 0.0), grid(fmt))
    sign = np.signbit(b).astype(np.int64)
    byte = np.where(bad, 255, e + 127).astype(np.uint8)
    if fmt == 0:
        q = (code | (sign << 3)) * ~bad[..., None]
        q = q.reshape(rows, k)
        return (q[:, 0::2] | (q[:, 1::2] << 4)).astype(np.uint8), byte
    q = np.where(bad[..., None], 127, code | (sign << 7))
    return q.reshape(rows, k).astype(np.uint8), byte


def tile(byte: np.ndarray) -> np.ndarray:
    """Scale bytes in the tiled order, one element at a time."""
    rows, nb = byte.shape
    rt, kt = -(-rows // 128), -(-nb // 4)
    out = np.zeros((rt, kt, 512), np.uint8)
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    out[r // 128, b // 4, 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4] = byte
    return out


def untile(tiles: np.ndarray, rows: int, nb: int) -> np.ndarray:
    r, b = np.meshgrid(np.arange(rows), np.arange(nb), indexing="ij")
    return tiles[r // 128, b // 4, 16 * (r % 32) + 4 * (r // 32 % 4) + b % 4]


def mx_values(codes: np.ndarray, byte: np.ndarray, fmt: int) -> np.ndarray:
    if fmt == 0:
        q = np.stack((codes & 15, codes >> 4), -1).reshape(codes.shape[0], -1)
        v = np.where(q & 8, -1.0, 1.0) * FP4[q & 7]
    else:
        v = fp8_table()[codes]
    rows, k = v.shape
    s = np.where(byte == 255, np.nan, 2.0 ** (byte.astype(float) - 127))
    return (v.reshape(rows, k // 32, 32) * s[..., None]).reshape(rows, k)


def rmsnorm(x, residual, gamma, eps):
    h = x + (0.0 if residual is None else residual)
    return h, h / np.sqrt((h * h).mean(-1, keepdims=True) + eps) * gamma


def kept(l: np.ndarray, t: float, top_k: int, top_p: float, min_p: float, slack: float = 0.0):
    """For one row: probabilities (of the temperature alone, times the largest
    one's inverse), rank order, and how many of the first ranks the filters
    keep; `slack` loosens (or, negative, tightens) the nucleus and min-p."""
    l = np.where(np.isnan(l), -np.inf, l)
    order = np.lexsort((np.arange(l.size), -l))
    with np.errstate(invalid="ignore"):
        e = np.where(l == l.max(), 1.0, np.exp((l - l.max()) / t))
    w = e[order]
    keep = l.size if not 0 < top_k < l.size else top_k
    if top_p < 1:
        before = np.concatenate(([0.0], np.cumsum(w[:keep])[:-1])) / w[:keep].sum()
        keep = max(1, int((before < top_p + slack).sum()))
    if min_p > 0:
        keep = min(keep, int((w >= min(min_p, 1.0) * (1 - slack) - 1e-300).sum()))
    return e, order, max(keep, 1)


def sample_exact(l, t, top_k, top_p, min_p, u):
    """One row by the definition with weights that are exact integers: `l` and
    t must make (l - max) * c whole.  Returns (id, weight, sum)."""
    from fractions import Fraction
    l = [float("-inf") if x != x else float(x) for x in l]
    top = max(l)
    if top == float("-inf"):
        return -1, 0, 0
    if not t > 0:
        return l.index(top), 1, 1
    c = float(np.float32(np.float32(1.44269504088896340736) / np.float32(t)))
    w = []
    for x in l:
        d = -1000 if x == float("-inf") else (x - top) * c
        assert d == int(d)
        w.append((1 << 31) >> int(-d) if -d <= 31 else 0)
    order = sorted(range(len(l)), key=lambda i: (-l[i], i))
    if 0 < top_k < len(l):
        order = order[:top_k]
    if top_p < 1:
        total, before, n = sum(w[i] for i in order), 0, 0
        for i in order:
            if n and not before < Fraction(float(np.float32(top_p))) * total:
                break
            before += w[i]
            n += 1
        order = order[:n]
    if min_p > 0:
        order = [i for i in order if w[i] >= Fraction(min(float(np.float32(min_p)), 1.0)) * (1 << 31)]
    total = sum(w[i] for i in order)
    r = min(int(Fraction(float(np.float32(u))) * total), total - 1)
    run = 0
    for i in sorted(order):
        run += w[i]
        if run > r:
            return i, w[i], total
    raise AssertionError("no token")

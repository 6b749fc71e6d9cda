"""Plain 64-bit forms of a serving step's operators: appending to a paged 8-bit
key/value cache, attention over it, and sampling.

A cache here is a dict: codes "k" and "v" (uint8 numpy, [pages][heads][rows][dim]),
scales "ks" and "vs" ([pages][heads]) and a page table "table" ([seqs][columns]).
"""
from __future__ import annotations

import numpy as np

E4M3, INT8 = 0, 1
QMAX = {E4M3: 448.0, INT8: 127.0}
SMALLEST = 2.0 ** -126


def _e4m3_values() -> np.ndarray:
    """The value of each of the 256 codes: sign, 4 exponent bits (bias 7), 3 fraction
    bits; exponent 0 holds the subnormals, S.1111.111 is NaN."""
    c = np.arange(256)
    e, f = (c >> 3) & 15, c & 7
    v = np.where(e == 0, f * 2.0 ** -9, (1 + f / 8) * 2.0 ** (e - 7.0))
    v = np.where((e == 15) & (f == 7), np.nan, v)
    return np.where(c >> 7, -v, v)


_E4M3 = _e4m3_values()


def values(codes: np.ndarray, fmt: int) -> np.ndarray:
    """What codes stand for, before the scale."""
    return _E4M3[codes] if fmt == E4M3 else codes.view(np.int8).astype(np.float64)


def encode(x: np.ndarray, fmt: int) -> np.ndarray:
    """Codes of x: nearest value of the format, ties to the even code, saturating."""
    x = np.asarray(x, dtype=np.float64)
    nan = np.isnan(x)
    x = np.clip(np.where(nan, 0.0, x), -QMAX[fmt], QMAX[fmt])
    if fmt == INT8:
        return np.rint(x).astype(np.int8).view(np.uint8)
    grid = _E4M3[:127]                                  # 0 .. 448, ascending codes
    a = np.abs(x)
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dlo, dhi = a - grid[lo], grid[hi] - a
    code = np.where((dlo < dhi) | ((dlo == dhi) & (lo % 2 == 0)), lo, hi)
    code = np.where(a == 0, 0, code) | (np.signbit(x) * 0x80)
    return np.where(nan, 0x7F, code).astype(np.uint8)


def rotate(x, cos, sin, interleaved, dtype=np.float64):
    """x: [rows][heads][dim]; cos, sin: [rows][pairs].  In fp32 every product and
    sum is rounded by itself, as numpy's operations are."""
    x = np.asarray(x, dtype=dtype)
    pairs = cos.shape[1]
    c, s = np.asarray(cos, dtype)[:, None], np.asarray(sin, dtype)[:, None]
    i = np.arange(0, 2 * pairs, 2) if interleaved else np.arange(pairs)
    j = i + 1 if interleaved else i + pairs
    y = x.copy()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    return y


def append(cache, fmt, q, k, v, cos, sin, base, start, interleaved, dtype=np.float64):
    """Appends in place; returns the rotated queries (not rounded to bf16).  dtype
    float32 follows the rounding of every step, float64 the definition."""
    one = dtype(1)
    page = cache["k"].shape[2]
    q_out = None if q is None else np.zeros(q.shape, dtype)
    for b in range(len(base)):
        rows = slice(int(start[b]), int(start[b + 1]))
        n = rows.stop - rows.start
        if n == 0:
            continue
        pos = int(base[b]) + np.arange(n)
        if q is not None:
            q_out[rows] = rotate(q[rows], cos[pos], sin[pos], interleaved, dtype)
        for name, x in (("k", rotate(k[rows], cos[pos], sin[pos], interleaved, dtype)), ("v", v[rows].astype(dtype))):
            codes, scales = cache[name], cache[name + "s"]
            for col in range(pos[0] // page, pos[-1] // page + 1):
                g, here = int(cache["table"][b, col]), pos // page == col
                held = max(0, int(base[b]) - col * page)
                for h in range(x.shape[1]):
                    a = np.fmin(np.nanmax(np.abs(x[here, h]), initial=0), np.finfo(np.float32).max).astype(dtype)
                    s = a / dtype(QMAX[fmt])
                    s = s if s >= SMALLEST else dtype(0)
                    s0 = scales[g, h].astype(dtype) if held else dtype(0)
                    s = max(s, s0)
                    r = one / s if s >= SMALLEST else dtype(0)
                    if held and s > s0:
                        old = values(codes[g, h, :held], fmt).astype(dtype)
                        codes[g, h, :held] = encode((old * s0) * r, fmt)
                    with np.errstate(invalid="ignore"):
                        codes[g, h, pos[here] % page] = encode(x[here, h] * r, fmt)
                    scales[g, h] = s
    return q_out


def gather(cache, fmt, b, length):
    """Keys and values of sequence b, [heads][length][dim] each."""
    page = cache["k"].shape[2]
    g = cache["table"][b, :-(-length // page)]
    out = []
    for name in ("k", "v"):
        x = values(cache[name][g], fmt) * cache[name + "s"][g].astype(np.float64)[..., None, None]
        out.append(x.transpose(1, 0, 2, 3).reshape(x.shape[1], -1, x.shape[3])[:, :length])
    return out


def attention(cache, fmt, q, lengths, start, scale=None):
    """(O, size): O in 64 bits and the largest sum_j P_j |V_j| of each row and head,
    the scale of its rounding errors."""
    rows, hq, dim = q.shape
    heads = cache["k"].shape[1]
    scale = 1.0 / np.sqrt(dim) if not scale else scale
    out, size = np.zeros((rows, hq, dim)), np.zeros((rows, hq))
    for b in range(len(lengths)):
        n = int(start[b + 1] - start[b])
        length = int(lengths[b])
        if n == 0 or length == 0:
            continue
        k, v = gather(cache, fmt, b, length)
        for i in range(n):
            seen = length - n + i + 1
            if seen <= 0:
                continue
            for h in range(hq):
                kv = h // (hq // heads)
                s = (k[kv, :seen] @ q[start[b] + i, h].astype(np.float64)) * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[start[b] + i, h] = p @ v[kv, :seen]
                size[start[b] + i, h] = (p @ np.abs(v[kv, :seen])).max()
    return out, size


def sample(logits, u, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0, share=0.0):
    """(token, logprob, margin, doubt) of one row, for a reader whose shares of mass
    are known to within `share`.  doubt: the share of mass of the ranks that top-p
    may then keep or not; margin: how far the draw (less the doubt) and the min-p
    cut are from falling the other way."""
    l = np.where(np.isnan(logits), -np.inf, np.asarray(logits, dtype=np.float64))
    order = np.argsort(-l, kind="stable")
    top = l[order[0]]
    if top == -np.inf:
        return -1, -np.inf, 1.0, 0.0
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0, 0.0
    with np.errstate(invalid="ignore"):
        z = np.where(l == top, 0.0, (l - top) / temperature)
    w = np.where(l == -np.inf, 0.0, np.exp(z))
    ranked, margin, doubt = w[order], 1.0, 0.0
    if top_k > 0:
        ranked[top_k:] = 0
    if top_p < 1:
        before = np.cumsum(ranked) - ranked
        bound = top_p * ranked.sum()
        near = np.abs(before - bound) <= share * ranked.sum()
        near[0] = False                                  # the first rank is always kept
        doubt = ranked[near].sum()
        keep = before < bound
        keep[0] = True
        ranked = np.where(keep, ranked, 0)
    if min_p > 0:
        margin = min(margin, np.abs(ranked[ranked > 0] - min_p).min())
        keep = ranked >= min_p
        keep[0] = True
        ranked = np.where(keep, ranked, 0)
    kept = np.zeros_like(w)
    kept[order] = ranked
    running = np.cumsum(kept)
    total = running[-1]
    doubt /= total
    margin = min(margin, np.abs(running / total - u).min() - doubt)
    token = min(int(np.searchsorted(running, u * total, side="right")), len(l) - 1)
    return token, z[token] - np.log(total), margin, doubt

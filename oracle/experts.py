"""Plain 64-bit forms of a layer of routed experts in 8 bits: routing, E4M3 codes with
block scales, their products, and the experts' FFN.

The products come with a bound on what fp32 sums and the stated roundings may add to them,
element by element, so that a test needs no tolerance of its own.
"""
from __future__ import annotations

import numpy as np

from .serving import E4M3, QMAX, SMALLEST, encode, values

BLOCK = 128
SOFTMAX, SIGMOID = 0, 1
U32 = 2.0 ** -24            # half a step of fp32, of fp32 1
U16 = 2.0 ** -8             # half a step of bf16
UH = 2.0 ** -11             # half a step of fp16


def blocks(n: int) -> int:
    return -(-n // BLOCK)


# ------------------------------------------------------------------ routing
def scores(logits, score):
    """Scores of each row in fp64: NaN counts as -inf; softmax rows with +inf share it."""
    l = np.asarray(logits, np.float64)
    l = np.where(np.isnan(l), -np.inf, l)
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        if score == SIGMOID:
            return 1.0 / (1.0 + np.exp(-l)), l
        m = l.max(1, keepdims=True)
        e = np.where(np.isposinf(m), np.isposinf(l), np.where(np.isneginf(l), 0.0, np.exp(l - np.where(np.isinf(m), 0.0, m))))
        total = e.sum(1, keepdims=True)
        return np.where(total > 0, e / np.where(total > 0, total, 1.0), 0.0), l


def route(logits, top_k, bias=None, score=SOFTMAX, groups=1, top_groups=1, group_best=2, renormalise=True, scale=1.0):
    """(ids, weights) of each row, largest choice first, equal ones by lowest index."""
    s, l = scores(logits, score)
    tokens, experts = s.shape
    choice = s
    if bias is not None:
        b = np.asarray(bias, np.float64)
        choice = s + np.where(b < np.inf, b, -np.inf)
    key = l if bias is None else choice
    kept = np.ones((tokens, experts), bool)
    if groups > 1:
        part = -np.sort(-choice.reshape(tokens, groups, -1), axis=2)[:, :, :group_best]
        best = np.argsort(-part.sum(2), axis=1, kind="stable")[:, :top_groups]
        g = np.zeros((tokens, groups), bool)
        np.put_along_axis(g, best, True, 1)
        kept = np.repeat(g, experts // groups, 1)
    # left-out experts after the kept ones, whatever these hold
    order = np.lexsort((-key, ~kept), axis=1)
    ids = order[:, :top_k]
    w = np.take_along_axis(s, ids, 1)
    if renormalise:
        total = w.sum(1, keepdims=True)
        w = np.where(total > 0, w / np.where(total > 0, total, 1.0), 0.0)
    return ids, w * scale


def by_expert(ids, experts):
    """(offsets, order): each expert's slots in ascending order."""
    flat = np.asarray(ids).reshape(-1)
    offsets = np.zeros(experts + 1, np.int64)
    offsets[1:] = np.cumsum(np.bincount(flat, minlength=experts))
    return offsets, np.argsort(flat, kind="stable")


# ------------------------------------------------------------------ codes
def quantise(x, block_rows=1):
    """(codes, scales) of an fp32 matrix; every operation rounded to fp32."""
    x = np.asarray(x, np.float32)
    rows, cols = x.shape
    tall, wide = -(-rows // block_rows), blocks(cols)
    a = np.zeros((tall * block_rows, wide * BLOCK), np.float32)
    a[:rows, :cols] = np.minimum(np.abs(np.where(np.isnan(x), np.float32(0), x)), np.finfo(np.float32).max)
    s = a.reshape(tall, block_rows, wide, BLOCK).max((1, 3)) / np.float32(QMAX[E4M3])
    s = np.where(s >= np.float32(SMALLEST), s, np.float32(0))
    with np.errstate(divide="ignore", invalid="ignore", over="ignore"):
        r = np.where(s > 0, np.float32(1) / s, np.float32(0))
        y = x * spread(r, block_rows, rows, cols)
    return encode(y, E4M3), s


def spread(s, block_rows, rows, cols):
    """A scale for every value."""
    return np.repeat(np.repeat(s, block_rows, 0)[:rows], BLOCK, 1)[:, :cols]


def dequantise(codes, s, block_rows):
    return values(np.asarray(codes, np.uint8), E4M3) * spread(np.asarray(s, np.float64), block_rows, *codes.shape)


# ------------------------------------------------------------------ products
def product_bound(a, b):
    """What fp32 may add to a @ b, for values a and b: in each block of 128 up to 128
    additions inside the tensor core, each off by less than a whole step (2 half steps)
    of the sum of magnitudes; then an addition a block, and the two scales' product."""
    n = 2 * BLOCK + blocks(a.shape[1]) + 4
    return n * U32 * (np.abs(a) @ np.abs(b))


def product(a, b, alpha=1.0, beta=0.0, c=None, bf16=False):
    """(alpha * a @ b + beta * c, bound) for values a, b in fp64."""
    v = alpha * (a @ b)
    e = abs(alpha) * product_bound(a, b) + 2 * U32 * np.abs(v)
    if beta:
        v = v + beta * np.asarray(c, np.float64)
        e = e + 2 * U32 * np.abs(beta * np.asarray(c, np.float64))
    return v, e + (U16 * (np.abs(v) + e) if bf16 else U32 * np.abs(v))


def _silu(g):
    with np.errstate(over="ignore"):
        return g / (1.0 + np.exp(-g))


def held(h, e):
    """Values of h as codes with a scale for each 128, and how far they may be off where
    each h is off by up to e: a code may fall on the other side of a middle."""
    rows, cols = h.shape
    pad = [(0, 0), (0, blocks(cols) * BLOCK - cols)]
    a = np.pad(np.abs(h), pad).reshape(rows, -1, BLOCK)
    ea = np.pad(e, pad).reshape(rows, -1, BLOCK)
    s = (a.max(2) / QMAX[E4M3]).astype(np.float32).astype(np.float64)
    es = ea.max(2) / QMAX[E4M3] + 2 * U32 * s
    S, ES = spread(s, 1, rows, cols), spread(es, 1, rows, cols)
    with np.errstate(divide="ignore", invalid="ignore"):
        t = np.where(S > 0, h / S, 0.0)
        et = np.where(S > 0, e / S + np.abs(t) * (ES / S) + 4 * U32 * np.abs(t), 0.0)
    c, lo, hi = (values(encode(v, E4M3), E4M3) for v in (t, t - et, t + et))
    return c * S, np.maximum(np.abs(hi - c), np.abs(lo - c)) * (S + ES) + np.abs(c) * ES


def ffn(x, gate, up, down):
    """One expert's y of rows x, all values in fp64: (y, bound), y before its rounding."""
    g, u = x @ gate, x @ up
    eg, eu = product_bound(x, gate), product_bound(x, up)
    s = _silu(g)
    es = 1.1 * eg + 8 * U32 * np.abs(s)                      # |silu'| < 1.1
    h = s * u
    eh = es * (np.abs(u) + eu) + np.abs(s) * eu + 2 * U32 * np.abs(h)
    v, ev = held(h, eh)
    return v @ down, ev @ np.abs(down) + product_bound(np.abs(v) + ev, down)


def scaled16_steps(x, gate, up, down):
    """Half a step of fp16's smallest numbers, 2^-25, times the scale of y's blocks, which is up to
    2^-13 * 2^25 times the sum over blocks of K of h's scale times down's.  Down's scales are taken
    from its largest values, as if each block had a code of 448, and twice that."""
    h = _silu(x @ gate) * (x @ up)
    k, n = down.shape

    def largest(v, rows):
        v = np.pad(np.abs(v), [(0, -v.shape[0] % rows), (0, -v.shape[1] % BLOCK)])
        return v.reshape(-1, rows, v.shape[1] // BLOCK, BLOCK).max((1, 3)) / QMAX[E4M3]
    return 2.0 ** -12 * spread(largest(h, 1) @ largest(down, BLOCK), 1, len(x), n)


def experts(x, ids, weights, gate, up, down, y_half_step=U16):
    """(out, bound) of the experts' FFN: x [tokens][hidden] in bf16's values, weights of
    each expert as values; y_half_step: what rounding may take from each y, relative to it."""
    xv = dequantise(*quantise(x), 1)
    ids, w = np.asarray(ids), np.asarray(weights, np.float64)
    out, err = np.zeros(x.shape), np.zeros(x.shape)
    for e in range(len(gate)):
        t, j = np.nonzero(ids == e)
        if len(t) == 0:
            continue
        y, ey = ffn(xv[t], gate[e], up[e], down[e])
        ey = ey + y_half_step * (np.abs(y) + ey)
        if y_half_step == UH:
            ey = ey + scaled16_steps(xv[t], gate[e], up[e], down[e])
        np.add.at(out, t, w[t, j][:, None] * y)
        np.add.at(err, t, np.abs(w[t, j])[:, None] * (ey + ids.shape[1] * U32 * np.abs(y)))
    return out, err + U16 * (np.abs(out) + err)

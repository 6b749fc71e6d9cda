"""A page that is filled a token at a time: its scale grows, and what it holds is rounded
again each time.  The oracle's fp32 form, which the kernels equal bit for bit, stays
within the sum of the half steps that the header states, and does need more than one."""
import numpy as np
import pytest

from oracle import serving as S

ROWS, DIM = 16, 64
NONE = np.zeros((ROWS, 0), np.float32)


def half_step(fmt, s, size):
    return 0.5 * s if fmt == S.INT8 else np.maximum(size * 2.0 ** -4, s * 2.0 ** -10)


def fill(fmt, growth, seed, check):
    rng = np.random.default_rng(seed)
    x = (rng.normal(size=(ROWS, 1, DIM)) * growth ** np.arange(ROWS)[:, None, None]).astype(np.float32)
    c = {"k": np.zeros((1, 1, ROWS, DIM), np.uint8), "v": np.zeros((1, 1, ROWS, DIM), np.uint8),
         "ks": np.zeros((1, 1), np.float32), "vs": np.zeros((1, 1), np.float32), "table": np.array([[0]])}
    err, before, growths = np.zeros((ROWS, DIM)), 0.0, 0
    for t in range(ROWS):
        S.append(c, fmt, None, x[t:t + 1], x[t:t + 1], NONE, NONE, [t], [0, 1], False, np.float32)
        s = float(c["vs"][0, 0])
        assert s >= before
        if t and s > before:
            growths += 1
            err[:t] += half_step(fmt, s, np.abs(x[:t, 0]) + err[:t])
        err[t] = half_step(fmt, s, np.abs(x[t, 0]))
        before = s
        # and a few roundings of fp32 in each step
        check(c, s, x[:t + 1, 0], err[:t + 1] + (growths + 1) * 2.0 ** -20 * S.QMAX[fmt] * s)
    return c, x, growths


@pytest.mark.parametrize("fmt", [S.E4M3, S.INT8])
@pytest.mark.parametrize("growth", [0.9, 1.0, 1.1, 1.5, 8.0])
def test_error_is_the_sum_of_half_steps(fmt, growth):
    def check(c, s, x, err):
        v = S.values(c["v"][0, 0, :len(x)], fmt) * s
        assert (np.abs(v - x) <= err).all()
    for seed in range(5):
        c, x, growths = fill(fmt, growth, seed, check)
        assert growths <= 6 or growth > 1
        assert np.array_equal(c["k"], c["v"])


def test_one_half_step_is_not_enough_where_the_scale_grew():
    c, x, growths = fill(S.INT8, 1.1, 0, lambda *a: None)
    off = np.abs(S.values(c["v"][0, 0], S.INT8) * float(c["vs"][0, 0]) - x[:, 0])
    assert growths > 3 and off.max() > 0.6 * c["vs"][0, 0]
    # the last token was rounded once
    assert off[-1].max() <= 0.5001 * c["vs"][0, 0]

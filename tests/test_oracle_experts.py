"""Pins of the routed experts' 64-bit forms against values worked out by hand, on the CPU."""
import numpy as np
import pytest

from oracle import experts as ox


def test_route_by_hand():
    l = np.log([[0.1, 0.4, 0.2, 0.3]])
    ids, w = ox.route(l, 2, renormalise=False)
    assert ids.tolist() == [[1, 3]] and np.allclose(w, [[0.4, 0.3]], rtol=1e-14)
    ids, w = ox.route(l, 2, scale=2.5)
    assert np.allclose(w, [[2.5 * 4 / 7, 2.5 * 3 / 7]], rtol=1e-14)
    ids, w = ox.route(np.array([[0.0, np.log(3.0)]]), 2, score=ox.SIGMOID, renormalise=False)
    assert ids.tolist() == [[1, 0]] and np.allclose(w, [[0.75, 0.5]], rtol=1e-14)
    # a bias is for the choice alone
    ids, w = ox.route(l, 2, bias=[1.0, 0.0, 0.0, 0.0], renormalise=False)
    assert ids.tolist() == [[0, 1]] and np.allclose(w, [[0.1, 0.4]], rtol=1e-14)
    # equal choices: the lowest index first
    assert ox.route(np.zeros((1, 5)), 3)[0].tolist() == [[0, 1, 2]]


def test_groups_by_hand():
    # scores of the groups' two best: 0.35 + 0.05 = 0.4 and 0.3 + 0.3 = 0.6
    s = np.array([[0.35, 0.05, 0.3, 0.3]])
    ids, w = ox.route(np.log(s), 2, groups=2, top_groups=1, renormalise=False)
    assert ids.tolist() == [[2, 3]] and np.allclose(w, [[0.3, 0.3]])
    # of their single best, the other group
    assert ox.route(np.log(s), 1, groups=2, top_groups=1, group_best=1)[0].tolist() == [[0]]


def test_routes_of_infinities_and_nan():
    inf, nan = np.inf, np.nan
    ids, w = ox.route(np.array([[0.0, inf, 1.0, inf], [-inf] * 4, [nan, 0.0, 0.0, nan]]), 2, renormalise=False)
    assert ids.tolist() == [[1, 3], [0, 1], [1, 2]]
    assert w.tolist() == [[0.5, 0.5], [0.0, 0.0], [0.5, 0.5]]
    # an expert whose bias is no number, or +inf, comes last
    ids, _ = ox.route(np.zeros((1, 4)), 4, bias=[nan, 0.0, inf, 1.0])
    assert ids.tolist() == [[3, 1, 0, 2]]


def test_order_by_expert():
    offsets, order = ox.by_expert([[2, 0], [0, 3], [2, 0]], 5)
    assert offsets.tolist() == [0, 3, 3, 5, 6, 6] and order.tolist() == [1, 2, 5, 0, 4, 3]


@pytest.mark.parametrize("block_rows", [1, 128])
def test_codes_by_hand(block_rows):
    x = np.zeros((2, 130), np.float32)
    x[0, 0], x[0, 1], x[0, 2], x[0, 129] = 448.0, -2.0, 2.0 ** -9, 7.0
    codes, s = ox.quantise(x, block_rows)
    assert s.shape == (2 if block_rows == 1 else 1, 2) and s[0].tolist() == [1.0, 1 / 64]
    assert codes[0, [0, 1, 2, 129]].tolist() == [0x7E, 0xC0, 0x01, 0x7E] and not codes[1].any()
    if block_rows == 1:
        assert s[1].tolist() == [0.0, 0.0]
    # infinities are FLT_MAX, NaN is left out
    codes, s = ox.quantise(np.array([[np.inf, np.nan, 1.0]], np.float32), block_rows)
    assert s[0, 0] == np.finfo(np.float32).max / np.float32(448) and codes[0].tolist() == [0x7E, 0x7F, 0x00]


def test_a_value_is_off_by_half_a_step_of_its_code():
    x = np.random.default_rng(0).normal(size=(5, 300)).astype(np.float32)
    codes, s = ox.quantise(x)
    back = ox.dequantise(codes, s, 1)
    # half a step of e4m3 is 2^-4 of a normal code's value, 2^-10 below; the scale's two roundings
    assert np.all(np.abs(back - x) <= np.maximum(np.abs(x) * 2.0 ** -4, ox.spread(s, 1, 5, 300) * 2.0 ** -10) * (1 + 2.0 ** -20))


def test_product_and_its_bound():
    a, b = np.full((1, 256), 2.0), np.full((256, 1), 0.5)
    v, e = ox.product(a, b, alpha=0.5, beta=2.0, c=np.array([[3.0]]))
    assert v.tolist() == [[134.0]] and 0 < e[0, 0] < 134 * 600 * 2.0 ** -24
    assert ox.product(a, b, bf16=True)[1][0, 0] > 256 * 2.0 ** -8


def test_ffn_by_hand():
    # one value each: x = 1, gate = log 3, up = 2, down = 4: silu = 0.75 log 3, h is its block's
    # largest and held as 448 times its scale
    x, one = np.array([[1.0]]), np.array([[1.0]])
    y, e = ox.ffn(x, one * np.log(3.0), one * 2, one * 4)
    assert abs(y[0, 0] - 6 * np.log(3.0)) < 1e-6 and 0 < e[0, 0] < 1e-3
    out, bound = ox.experts(np.array([[448.0]]), [[1, 0]], [[0.25, 0.5]], [one * 0, one], [one, one], [one, one])
    assert abs(out[0, 0] - 0.25 * 448.0 ** 2) < 0.01 and bound[0, 0] < 0.25 * 448 ** 2 * 0.02


def test_bound_covers_the_other_code():
    # h in the middle of two codes: whichever it falls to is within the bound
    h = np.array([[448.0, 17.0]])
    v, e = ox.held(h, np.full((1, 2), 1e-4))
    assert v[0, 0] == 448.0 and {v[0, 1] - e[0, 1] <= 16.0, v[0, 1] + e[0, 1] >= 18.0} & {True}
    assert e[0, 1] >= 1.9 and e[0, 0] < 0.01

"""Pins of the serving step's 64-bit oracle: hand values, limits and identities."""
import numpy as np
import pytest
import torch

from oracle import serving as S


def test_e4m3_codes_match_torch_and_round_trip():
    c = np.arange(256, dtype=np.uint8)
    v = S.values(c, S.E4M3)
    t = torch.from_numpy(c).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(v, t, equal_nan=True)
    fine = ~np.isnan(v)
    assert np.array_equal(S.encode(v[fine], S.E4M3), c[fine])
    x = np.random.default_rng(0).normal(size=4000) * np.exp(np.random.default_rng(1).normal(size=4000) * 3)
    want = torch.from_numpy(np.clip(x, -448, 448).astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    assert np.array_equal(S.encode(x.astype(np.float32), S.E4M3), want)


def test_int8_codes_round_to_even_and_saturate():
    x = np.array([0.5, 1.5, 2.5, -0.5, -1.5, 126.5, 127.4, 200.0, -127.5, -300.0])
    assert S.encode(x, S.INT8).view(np.int8).tolist() == [0, 2, 2, 0, -2, 126, 127, 127, -127, -127]


def test_rotation_turns_the_plane():
    a = np.array([[0.0, np.pi / 2]])
    x = np.array([[[1.0, 2.0, 3.0, 4.0, 9.0]]])
    half = S.rotate(x, np.cos(a), np.sin(a), False)[0, 0]
    assert np.allclose(half, [1, -4, 3, 2, 9])          # pairs (0, 2) and (1, 3)
    inter = S.rotate(x, np.cos(a), np.sin(a), True)[0, 0]
    assert np.allclose(inter, [1, 2, -4, 3, 9])         # pairs (0, 1) and (2, 3)


def _cache(pages=3, heads=1, rows=4, dim=2, seqs=1):
    return {"k": np.zeros((pages, heads, rows, dim), np.uint8), "v": np.zeros((pages, heads, rows, dim), np.uint8),
            "ks": np.zeros((pages, heads), np.float32), "vs": np.zeros((pages, heads), np.float32),
            "table": np.array([[2, 0, 1]])}


def test_append_worked_example():
    c = _cache()
    none = np.zeros((16, 0))
    x = np.array([[[127.0, -2.0]], [[1.0, 0.0]]])
    S.append(c, S.INT8, None, x, x, none, none, [3], [0, 2], False)
    # token 3 is the last row of the first column's page (2), token 4 the first of page 0
    assert c["ks"][2, 0] == 1.0 and c["k"][2, 0, 3].view(np.int8).tolist() == [127, -2]
    assert c["ks"][0, 0] == np.float32(1 / 127) and c["k"][0, 0, 0].view(np.int8).tolist() == [127, 0]
    # a larger value in page 0: the earlier token is held at the new scale
    S.append(c, S.INT8, None, x[:1] * 3 / 127, x[:1] * 3 / 127, none, none, [5], [0, 1], False)
    assert c["k"][0, 0, 0].view(np.int8).tolist() == [42, 0]     # 127 / 3
    assert c["k"][0, 0, 1].view(np.int8).tolist() == [127, -2]
    # the same again changes nothing
    before = {k: v.copy() for k, v in c.items()}
    S.append(c, S.INT8, None, x[:1] * 3 / 127, x[:1] * 3 / 127, none, none, [5], [0, 1], False)
    assert all(np.array_equal(before[k], c[k]) for k in c)


@pytest.mark.parametrize("fmt", [S.E4M3, S.INT8])
def test_fp32_and_64_bit_appends_agree(fmt):
    rng = np.random.default_rng(fmt)
    x = rng.normal(size=(3, 1, 2)).astype(np.float32)
    a = rng.normal(size=(16, 1))
    got = []
    for dtype in (np.float32, np.float64):
        c = _cache()
        S.append(c, fmt, x, x, x, np.cos(a), np.sin(a), [2], [0, 3], False, dtype)
        got.append(c)
    assert np.allclose(got[0]["ks"], got[1]["ks"], rtol=2.0 ** -21)
    assert np.abs(got[0]["k"].astype(int) - got[1]["k"].astype(int)).max() <= 1


def test_attention_equal_keys_average_values_and_masks():
    c = _cache()
    c["ks"][:] = c["vs"][:] = 0.5
    c["v"][2, 0, :, 0] = np.array([2, 4, 6, 8], np.uint8)
    q = np.ones((2, 1, 2))
    out, size = S.attention(c, S.INT8, q, [4], [0, 2])
    assert np.allclose(out[:, 0, 0], [2.0, 2.5]) and np.allclose(size[:, 0], [2.0, 2.5])
    out, _ = S.attention(c, S.INT8, q, [1], [0, 2])       # the first of two queries sees no key
    assert out[0].tolist() == [[0, 0]] and out[1, 0, 0] == 1.0


def test_sampling_rules_by_hand():
    l = np.log([0.1, 0.4, 0.2, 0.3])
    draw = lambda u, **kw: S.sample(l, u, **kw)[0]  # noqa: E731
    assert [draw(u) for u in (0.0, 0.09, 0.11, 0.49, 0.51, 0.69, 0.71, 0.99)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [draw(u, top_k=2) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]
    assert [draw(u, top_p=0.7) for u in (0.0, 0.57, 0.58, 0.99)] == [1, 1, 3, 3]      # 0.4 + 0.3 reach 0.7
    assert [draw(u, top_p=0.71) for u in (0.43, 0.45, 0.67)] == [1, 2, 3]
    assert draw(0.99, min_p=0.6) == 3 and draw(0.5, min_p=0.76) == 1
    assert draw(0.7, temperature=0.0) == 1
    assert abs(S.sample(l, 0.0, top_k=2)[1] - np.log(0.4 / 0.7)) < 1e-12
    # ties: the lower index ranks first
    assert S.sample(np.zeros(5), 0.99, top_k=2)[0] == 1
    assert S.sample(np.full(3, -np.inf), 0.5)[0] == -1
    assert S.sample(np.array([np.nan, -np.inf, 3.0]), 0.99)[0] == 2

"""Pins of the 8-bit cache's oracle: hand-worked values, closed forms and laws, no formula typed twice."""
import math

import numpy as np
import pytest

from oracle import kvcache8 as O


def test_exponents_hand_worked():
    assert O.exponent(127.0) == 0 and O.exponent(127.0001) == 1 and O.exponent(63.5) == -1
    assert O.exponent(0.0) == O.LOW and O.exponent(1e-30) == O.LOW
    assert O.exponent(3.4028e38) == O.HIGH == 121
    r = np.random.default_rng(0)
    for x in np.exp(r.uniform(-30, 80, 200)):
        e = O.exponent(x)
        assert 63 < x / 2.0 ** e <= 127


def test_rounding():
    x = np.array([0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 0.49, 126.5, 127.5, -500.0])
    assert O.round_even(x).tolist() == [0, 2, 2, 0, -2, -2, 0, 126, 127, -127]
    y = np.random.default_rng(1).uniform(-120, 120, 500)
    assert np.array_equal(O.round_even(y), np.round(y))


@pytest.mark.parametrize("D", [64, 128])
def test_bytes_of_a_block_are_a_permutation(D):
    keys = sorted(O.key_byte(D, i, d) for i in range(16) for d in range(D))
    values = sorted(O.value_byte(D, i, d) for i in range(16) for d in range(D))
    assert keys == list(range(16 * D)) and values == list(range(16 * D, 32 * D))


def test_places_hand_worked():
    assert O.key_byte(128, 0, 17) == 17 and O.key_byte(128, 1, 17) == 128 + 1 and O.key_byte(64, 1, 17) == 81
    # token 5 is the odd one of pair 2: chunk 1 (values 8..15) at place 1 ^ 4
    assert O.value_byte(128, 5, 9) == 2048 + 2 * 256 + 16 * 5 + 3
    assert O.value_byte(64, 0, 0) == 1024


def _empty(pages, H, D, ps):
    return np.zeros((pages, H, ps * (2 * D + 1)), np.uint8)


def test_append_reads_back():
    """Tokens one by one and all at once: each value within half a step of the block's final exponent, or one
    step where it was rounded again; the same where the exponent never grows."""
    r = np.random.default_rng(2)
    H, D, ps = 2, 64, 32
    k, v = r.standard_normal((2, 21, H, D)) * np.exp(r.standard_normal((2, 21, 1, 1)))
    slots = np.arange(21) + 64  # from the start of page 2
    one, all_ = _empty(4, H, D, ps), _empty(4, H, D, ps)
    out = O.append(all_, slots, k, v, ps)
    for t in range(21):
        O.append(one, slots[t:t + 1], k[t:t + 1], v[t:t + 1], ps)
    for h in range(H):
        for cache, room in ((all_, 0.5), (one, 1.0)):
            K, V, E = O.read_head(cache, [2], 21, h, ps, D)
            assert (np.abs(V - v[:, h]) <= room * 2.0 ** E[:, None]).all()
            step = [2.0 ** O.Block(cache[2, h, j:j + 32 * D + 16], D, 0).e for j in (0, 32 * D + 16)]
            assert (np.abs(K - k[:, h]) <= room * np.where(np.arange(21) < 16, *step)[:, None]).all()
        K, V, _ = O.read_head(all_, [2], 21, h, ps, D)
        assert np.array_equal(K, out[0, :, h]) and np.array_equal(V, out[1, :, h])
    # loudest first: no exponent grows, and what came in one call does not show
    order = np.argsort(-np.abs(k[:16, 0]).max(1))
    k2 = k[:16][order][:, :1]
    a, b = _empty(1, 1, D, 16), _empty(1, 1, D, 16)
    O.append(a, np.arange(16), k2, k2, 16)
    for t in range(16):
        O.append(b, [t], k2[t:t + 1], k2[t:t + 1], 16)
    assert np.array_equal(a, b)


def test_append_growth_hand_worked():
    D = 64
    cache = _empty(1, 1, D, 16)
    x = np.zeros((1, 1, D))
    x[0, 0, :4] = [127, 5, -3, 1]
    O.append(cache, [0], x, x, 16)
    assert O.Block(cache[0, 0], D, 0).e == 0
    y = np.full((1, 1, D), 200.0)
    out = O.append(cache, [1], y, y, 16)
    for which in (0, 1):
        b = O.Block(cache[0, 0], D, which)
        assert b.e == 1 and b.codes[0, :4].tolist() == [64, 2, -2, 0] and (b.codes[1] == 100).all()
    assert (out == 200).all()
    O.append(cache, [0], x, x, 16)  # the block starts afresh
    b = O.Block(cache[0, 0], D, 1)
    assert b.e == 0 and b.codes[0, :4].tolist() == [127, 5, -3, 1] and not b.codes[1:].any()


def test_marks():
    D = 64
    cache = _empty(1, 1, D, 16)
    x = np.ones((3, 1, D))
    x[1, 0, 7] = math.inf
    out = O.append(cache, [0, 1, 2], x, np.ones((3, 1, D)), 16)
    K, V, _ = O.read_head(cache, [0], 3, 0, 16, D)
    assert np.isnan(K[1]).all() and (K[[0, 2]] == 1).all() and (V == 1).all() and np.isnan(out[0, 1]).all()
    o = O.attention(np.ones((3, 1, D)), cache, np.array([[0]]), [3], [0, 3], 16, 0.1)
    assert np.isfinite(o["out"][0]).all() and np.isnan(o["out"][1:]).all() and np.isnan(o["lse"][1:]).all()
    O.append(cache, [1], np.ones((1, 1, D)), np.ones((1, 1, D)), 16)  # written anew
    assert (O.read_head(cache, [0], 3, 0, 16, D)[0] == 1).all()


def test_attention_closed_forms():
    r = np.random.default_rng(3)
    D, ps = 64, 16
    cache = _empty(8, 1, D, ps)
    table = np.array([[5, 2], [0, 1], [7, 3]])
    x = r.standard_normal((20, 1, D))
    at = np.arange(20)
    out = O.append(cache, table[0][at // ps] * ps + at % ps, x, x, ps)
    q = np.zeros((2 + 1 + 3, 2, D))
    o = O.attention(q, cache, table, [20, 0, 2], [0, 2, 3, 6], ps, 1.0)
    assert np.allclose(o["out"][0], out[1, :19, 0].mean(0)) and np.allclose(o["out"][1], out[1, :, 0].mean(0))
    assert np.allclose(o["lse"][:2], np.log([[19, 19], [20, 20]]))
    assert (o["out"][2:4] == 0).all() and np.isneginf(o["lse"][2:4]).all()  # nothing to see


def test_prompt_closed_forms():
    r = np.random.default_rng(4)
    T, D = 9, 64
    q, k, v = np.zeros((T, 4, D)), r.standard_normal((T, 2, D)), r.standard_normal((T, 2, D))
    o = O.prompt_attention(q, k, v, [0, 3, 8], 1.0)
    assert np.allclose(o["out"][2, 0], v[:3, 0].mean(0)) and np.allclose(o["out"][7, 3], v[3:8, 1].mean(0))
    assert np.allclose(o["lse"][:8, 0], np.log([1, 2, 3, 1, 2, 3, 4, 5])) and np.isnan(o["out"][8]).all()
    # one token weighs all
    q[7, 0] = 1000 * k[4, 0]
    assert np.allclose(O.prompt_attention(q, k, v, [0, 3, 8], 1.0)["out"][7, 0], v[4, 0])
    # the last row of a prompt is what the cache's attention gives for one new token
    cache = _empty(1, 2, D, 16)
    x = O.append(cache, np.arange(5), k[:5], v[:5], 16)
    q = r.standard_normal((5, 4, D))
    a = O.prompt_attention(q, x[0], x[1], [0, 5], 0.3)
    b = O.attention(q, cache, np.array([[0]]), [5], [0, 5], 16, 0.3)
    assert np.allclose(a["out"], b["out"]) and np.allclose(a["lse"], b["lse"])

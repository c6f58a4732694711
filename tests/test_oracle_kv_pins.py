"""Pins of the cache oracle: formats against torch's own and hand-worked bytes, tables against
hand-worked rounds and conservation of pages, the rotation against its group laws, attention
against closed forms."""
import math

import numpy as np
import pytest

from oracle import kvcache as O


def test_e4m3_against_torch():
    torch = pytest.importorskip("torch")
    b = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(b, O.E4M3, equal_nan=True)


def test_nearest_even_grid():
    for i in range(7):  # midpoints of the code grid go to the even code
        mid = (O.E2M1[i] + O.E2M1[i + 1]) / 2
        assert O.nearest_even(mid, O.E2M1) == (i if i % 2 == 0 else i + 1)
        assert O.nearest_even(mid - 1e-9, O.E2M1) == i
        assert O.nearest_even(mid + 1e-9, O.E2M1) == i + 1
    assert O.nearest_even(100.0, O.E2M1) == 7


def test_quantise_hand_worked():
    x = np.zeros(16, np.float32)
    x[:8] = [6, -3, 0.25, 0.75, -0.25, 1.25, 5, 2.5]
    codes, scale = O.quantise16(x, 1.0)
    assert O.E4M3[scale] == 1.0
    assert codes[:8].tolist() == [7, 13, 0, 2, 8, 2, 6, 4]
    assert O.quantise16(x, 0.5)[1] == scale + 8  # half the tensor scale: twice the block's
    assert O.quantise16(np.zeros(16), 1.0) == (pytest.approx(np.zeros(16)), 0)
    x[3] = math.inf
    assert O.quantise16(x, 1.0)[1] == 0x7F


@pytest.mark.parametrize("D", [64, 128])
def test_value_places_are_a_permutation(D):
    for p in range(8):
        assert sorted(O.value_place(D, p, d) for d in range(D)) == list(range(D))


@pytest.mark.parametrize("D", [64, 128])
def test_put_and_read_round_trip(D):
    """Values on the format's own grid come back as they are, whatever order tokens come in."""
    r = np.random.default_rng(3)
    ps, pages = 32, [2, 0]
    cache = r.integers(0, 256, (3, 2, ps * (D + D // 8)), dtype=np.uint8)
    K = O.E2M1[r.integers(0, 8, (40, D))] * r.choice([-1, 1], (40, D))
    V = O.E2M1[r.integers(0, 8, (40, D))] * r.choice([-1, 1], (40, D))
    K[:, ::16], V[:, ::16] = 6, -6  # every block's largest: a scale of 1
    for t in r.permutation(40):
        O.put_token(cache, pages[t // ps] * ps + t % ps, 1, ps, D, K[t], V[t] * 0.5, 1.0, 0.5)
    k, v = O.read_head(cache, pages, 40, 1, ps, D, 1.0, 0.5)
    assert np.array_equal(k, K) and np.array_equal(v, V * 0.5)


def test_tables_hand_worked():
    table = np.array([[4, 5, -1], [6, -1, -1], [7, 8, 9]])
    ring = np.array([1, 2, 3, 0, -1, -1, -1, -1, -1, -1])
    r = O.block_tables([17, 10, 40], [2, -1, 0], [13, 5, -1], table, [2, 1, 3], ring, [0, 4], 16, 20)
    # 20 + 13 tokens need a third page; 10 + 5 fit; the third sequence ended
    assert r["block_table"].tolist() == [[4, 5, 1], [6, -1, -1], [7, 8, 9]]
    assert r["ring"].tolist() == [1, 2, 3, 0, 7, 8, 9, -1, -1, -1]
    assert r["counters"].tolist() == [1, 7]
    assert r["ctx_lens"].tolist() == [20, 10, 0] and r["held"].tolist() == [3, 1, 0]
    assert r["kv_lens"].tolist() == [33, 15, 0] and r["status"].tolist() == [1, 1, 0]
    assert r["cu_new"].tolist() == [0, 13, 18, 18]
    assert r["slots"][12] == 16 and r["slots"][0] == 5 * 16 + 4
    assert r["slots"][13:].tolist() == [6 * 16 + i for i in range(10, 15)] + [-1, -1]
    assert r["positions"][11:15].tolist() == [31, 32, 10, 11]


def test_tables_pages_are_conserved():
    r = np.random.default_rng(0)
    B, ps, cap = 6, 16, 40
    table, held, ctx = np.full((B, 9), -1), np.zeros(B, int), np.zeros(B, int)
    ring, counters, acc = np.arange(cap), np.array([0, cap]), None
    seen = set()
    for step in range(60):
        new = r.integers(-1, 40, B) * (r.random(B) < 0.8)
        o = O.block_tables(ctx, acc, new, table, held, ring, counters, ps, 90)
        table, held, ctx, ring, counters = (o[k] for k in ("block_table", "held", "ctx_lens", "ring", "counters"))
        live = [int(ring[i % cap]) for i in range(counters[0], counters[1])]
        used = [int(p) for b in range(B) for p in table[b, :held[b]]]
        assert sorted(live + used) == list(range(cap))
        s = o["slots"][o["slots"] >= 0]
        assert len(set(s.tolist())) == len(s) == o["cu_new"][-1] <= 90
        acc = np.array([r.integers(0, n) if n > 0 else -1 for n in np.diff(o["cu_new"])])
        seen |= set(o["status"].tolist())
    assert {1, 0, -1, -3} <= seen


def test_rotation_laws():
    r = np.random.default_rng(1)
    x = r.standard_normal((3, 2, 8))
    freq = [1.0, 0.3, 0.01]
    for inter in (False, True):
        y0, _ = O.qk_norm_rope(x, [0, 0, 0], freq, None, 0.0, inter)
        assert np.allclose((y0 ** 2).mean(-1), 1) and np.allclose(y0 / x, (y0 / x)[..., :1])
        a, _ = O.qk_norm_rope(x, [5, 9, 100], freq, None, 0.0, inter)
        b, _ = O.qk_norm_rope(x, [1005, 1009, 1100], freq, None, 0.0, inter)
        # scores depend on the distance alone
        assert np.allclose(np.einsum("thd,shd->hts", a, a), np.einsum("thd,shd->hts", b, b))
        assert np.array_equal(a[..., 6:], y0[..., 6:])  # past the rotated part


def _filled(D, ps, lens, heads, seed):
    r = np.random.default_rng(seed)
    most = max(1, -(-max(lens) // ps))
    table = r.permutation(len(lens) * most).reshape(len(lens), most)
    cache = r.integers(0, 256, (len(lens) * most, heads, ps * (D + D // 8)), dtype=np.uint8)
    for b, L in enumerate(lens):
        for t in range(L):
            for h in range(heads):
                O.put_token(cache, table[b, t // ps] * ps + t % ps, h, ps, D,
                            r.standard_normal(D), r.standard_normal(D), 1.0, 1.0)
    return cache, table


def test_attention_closed_forms():
    D, ps = 64, 16
    cache, table = _filled(D, ps, [5, 0, 2], 1, 0)
    _, V = O.read_head(cache, table[0], 5, 0, ps, D, 1.0, 1.0)
    q = np.zeros((2 + 1 + 4, 2, D))  # no preference: the mean of what is seen
    o = O.attention(q, cache, table, [5, 0, 2], [0, 2, 3, 7], ps, 1.0, 1.0, 1.0)
    assert np.allclose(o["out"][0], V[:4].mean(0)) and np.allclose(o["out"][1], V.mean(0))
    assert np.allclose(o["lse"][:2], np.log([[4, 4], [5, 5]]))
    empty = [2, 3, 4]  # nothing cached; and the first two of four rows over two tokens
    assert (o["out"][empty] == 0).all() and np.isneginf(o["lse"][empty]).all()
    assert np.allclose(o["lse"][5:], np.log([[1, 1], [2, 2]]))

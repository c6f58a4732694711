"""GPU parity of the cache operators (include/spec_kv.h) with the float64 oracle.

Integers and 4-bit codes are equal. Tolerances count roundings: half a step of the output's type
(2^-8 of a bf16 value, 2^-24 of a float32 one) and, scaled by the magnitudes that enter a sum, those of
the arithmetic in between; each test says which.
"""
import itertools
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from oracle import kvcache as O  # noqa: E402
from speculative_decoding_verification_33_gb300 import _lib  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


# ------------------------------------------------------------------------------ block tables
def _tables_inputs(B, ps, most, seed, spare=None, prompts=0):
    r = np.random.default_rng([seed, B, ps])
    ctx = r.integers(0, max(1, (most - 1) * ps // 2), B)
    held = np.minimum(most, -(-ctx // ps) + r.integers(0, 3, B))
    acc = np.where(r.random(B) < 0.7, np.minimum(r.integers(0, 9, B), held * ps - ctx - 1), -1)
    new = r.integers(0, prompts + 10, B) * (r.random(B) < 0.9)
    new[r.random(B) < 0.1] = -1
    pages = r.permutation(int(held.sum()) + 4 * B + 7)
    table = np.full((B, most), -1)
    table[np.arange(most)[None] < held[:, None]] = pages[:held.sum()]
    left = pages[held.sum():][:spare]
    ring = np.full(len(pages) + 3, -1)
    head = int(r.integers(0, 3 * len(ring)))
    ring[(head + np.arange(len(left))) % len(ring)] = left
    return [ctx, acc, new, table, held, ring, np.array([head, head + len(left)])]


def _check_tables(x, ps, cap, accept=True):
    ctx, acc, new, table, held, ring, counters = x
    ref = O.block_tables(ctx, acc if accept else None, new, table, held, ring, counters, ps, cap)
    tb, rg = dev(table), dev(ring)
    args = (dev(ctx), dev(new), tb, dev(held), rg, dev(counters, torch.int64))
    out = sv.block_tables(*args, page_size=ps, max_tokens=cap,
                          accept_len=dev(acc) if accept else None)
    for again in range(2):  # a second call on the same inputs writes the same
        for name, v in {**out, "block_table": tb, "ring": rg}.items():
            assert np.array_equal(host(v), ref[name]), (name, again)
        sv.block_tables(*args, page_size=ps, max_tokens=cap, accept_len=dev(acc) if accept else None,
                        out=out)
    return ref


@pytest.mark.parametrize("B,ps,most,cap,prompts", [
    (1, 16, 1, 0, 0), (1, 16, 4, 1, 0), (3, 128, 5, 40, 0), (33, 32, 9, 500, 0),
    (256, 16, 40, 2000, 0), (257, 64, 300, 40000, 300), (1000, 16, 30, 3001, 0),
    (8192, 16, 12, 60000, 0)])
def test_tables(B, ps, most, cap, prompts):
    _check_tables(_tables_inputs(B, ps, most, 0, prompts=prompts), ps, cap)


def test_tables_without_outcomes():
    _check_tables(_tables_inputs(50, 16, 20, 1), 16, 400, accept=False)


@pytest.mark.parametrize("spare", [0, 1, 17])
def test_tables_pages_run_out(spare):
    x = _tables_inputs(300, 16, 40, 2, spare=spare, prompts=60)
    ref = _check_tables(x, 16, 20000)
    assert (ref["status"] == -1).any() and ref["counters"][0] - x[6][0] <= spare


def test_tables_tokens_run_out():
    ref = _check_tables(_tables_inputs(300, 16, 40, 3, prompts=60), 16, 2500)
    assert (ref["status"] == -3).any() and ref["cu_new"][-1] <= 2500


def test_tables_lengths_that_do_not_fit():
    x = _tables_inputs(64, 16, 8, 4)
    ctx, acc, new, table, held, ring, _ = x
    ctx[3], held[5], held[6], new[7] = -5, -1, 9, 8 * 16 + 1
    ctx[8], held[8] = 40, 1                       # more tokens than its pages hold
    ctx[9], new[9], held[9] = -3, -1, 2           # ended: only its pages count
    table[9, :2] = [77, 78]
    ctx[10], new[10], acc[10] = 2 ** 31 - 1, 2 ** 31 - 1, 8
    ref = _check_tables(x, 16, 1000)
    assert (ref["status"][[3, 5, 6, 7, 8, 10]] == -2).all() and ref["status"][9] == 0


def test_tables_many_rounds():
    """A loop of rounds in two sets of buffers: pages are conserved, slots never shared."""
    r = np.random.default_rng(5)
    B, ps, cap, most = 40, 16, 260, 20
    table, ring = dev(np.full((B, most), -1)), dev(np.arange(cap))
    ctx, held, counters = dev(np.zeros(B)), dev(np.zeros(B)), dev([0, cap], torch.int64)
    acc, sets = None, [None, None]
    ref = dict(ctx_lens=np.zeros(B, int), held=np.zeros(B, int), counters=[0, cap],
               block_table=np.full((B, most), -1), ring=np.arange(cap))
    for step in range(40):
        new = r.integers(-1, 50, B) * (r.random(B) < 0.8)
        acc_h = None if acc is None else host(acc)
        ref = O.block_tables(ref["ctx_lens"], acc_h, new, ref["block_table"], ref["held"],
                             ref["ring"], ref["counters"], ps, 600)
        out = sv.block_tables(ctx, dev(new), table, held, ring, counters, page_size=ps,
                              max_tokens=600, accept_len=acc, out=sets[step % 2])
        sets[step % 2] = out
        for name, v in {**out, "block_table": table, "ring": ring}.items():
            assert np.array_equal(host(v), ref[name]), (name, step)
        ctx, held, counters = out["ctx_lens"], out["held"], out["counters"]
        n = np.diff(ref["cu_new"])
        acc = dev(np.where(n > 0, r.integers(0, 1 << 20, B) % np.maximum(n, 1), -1))


# ------------------------------------------------------------------------------ norm, rotation
def _check_norm_rope(T, hq, hk, D, rot, inter, dtype, *, far=5000, strided=False, in_place=False,
                     weights=True, seed=0, offset=0):
    g = torch.Generator("cuda").manual_seed(seed + D + T)
    gap = 8 if strided else 0

    def rows(h):
        base = torch.randn(T, h * D + gap + offset, device="cuda", generator=g) * 3
        return base.to(dtype)[:, offset:offset + h * D].unflatten(1, (h, D))
    q, k = rows(hq), rows(hk) if hk else None
    pos = torch.randint(-far, far, (T,), device="cuda", generator=g, dtype=torch.int32)
    freq = torch.tensor([500000.0 ** (-2 * i / max(rot, 1)) for i in range(rot // 2)],
                        dtype=torch.float64, device="cuda")
    w = [torch.randn(D, device="cuda", generator=g).to(dtype) if weights else None for _ in "qk"]
    q0, k0 = host(q), host(k) if hk else None
    out = {"q": q, "k": k} if in_place else None
    out = sv.qk_norm_rope(q, k, pos, freq, q_weight=w[0], k_weight=w[1], eps=1e-5,
                          interleaved=inter, out=out)
    for name, x, wt in (("q", q0, w[0]), ("k", k0, w[1])):
        if x is None:
            continue
        ref, room = O.qk_norm_rope(x, host(pos), host(freq), host(wt) if weights else None, 1e-5, inter)
        # the sum of squares (D terms, half of its relative error reaches its root), root, quotient, weight
        # and rotation: (D / 2 + 8) 2^-24; sine and cosine: 2^-23, and 2^-32 turns of the angle
        tol = room * ((D / 2 + 8) * 2.0 ** -24 + 2.0 ** -23 + 2 * math.pi * 2.0 ** -32)
        tol += (2.0 ** -8 if dtype == BF16 else 2.0 ** -24) * np.abs(ref) + 1e-38
        bad = np.abs(host(out[name]) - ref) > tol
        assert not bad.any(), (name, int(bad.sum()), np.abs(host(out[name]) - ref).max())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,hq,hk,D,rot", [
    (1, 1, 1, 64, 64), (8, 32, 8, 128, 128), (5, 28, 4, 128, 64), (700, 8, 1, 64, 16),
    (3, 16, 16, 256, 256), (2, 3, 2, 96, 32), (4, 2, 1, 80, 6), (1300, 4, 4, 128, 0),
    (9, 1, 0, 64, 64), (2, 2, 1, 2, 2), (3, 1, 1, 512, 130)])
def test_norm_rope(dtype, inter, T, hq, hk, D, rot):
    _check_norm_rope(T, hq, hk, D, rot, inter, dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_norm_rope_views(dtype):
    _check_norm_rope(17, 4, 2, 128, 128, False, dtype, strided=True)
    _check_norm_rope(17, 4, 2, 128, 128, False, dtype, strided=True, in_place=True)
    _check_norm_rope(17, 4, 2, 128, 64, True, dtype, in_place=True, weights=False)
    _check_norm_rope(6, 4, 2, 64, 64, False, dtype, offset=1)   # no 16-byte alignment
    _check_norm_rope(6, 4, 2, 64, 64, True, dtype, offset=3, in_place=True)


def test_norm_rope_far_positions():
    """Angles of up to 2^31 positions keep the tolerance of near ones."""
    _check_norm_rope(64, 2, 1, 64, 64, False, F32, far=2 ** 31 - 1)


def test_norm_rope_values():
    """A zero row stays zero, a NaN stays in its head, nothing to do is nothing launched."""
    q = torch.randn(2, 2, 64, device="cuda")
    q[0, 0] = 0
    q[1, 0, 3] = math.nan
    pos, freq = dev([3, 4]), torch.ones(32, dtype=torch.float64, device="cuda")
    o = sv.qk_norm_rope(q, None, pos, freq)["q"]
    assert (o[0, 0] == 0).all() and o[1, 0].isnan().all() and o[:, 1].isfinite().all()
    e = sv.qk_norm_rope(q[:0], None, pos[:0], freq)["q"]
    assert e.shape == (0, 2, 64)
    with pytest.raises(TypeError):
        sv.qk_norm_rope(q.half(), None, pos, freq)
    with pytest.raises(ValueError):
        sv.qk_norm_rope(q.transpose(1, 2), None, pos, freq)


# ------------------------------------------------------------------------------ append
def _check_append(T, H, D, ps, dtype, slots, *, gk=1.0, gv=0.5, strided=False, spread=1.0, edit=None,
                  seed=0, pages=None):
    r = np.random.default_rng(seed)
    slots = np.asarray(slots)
    pages = pages or int(slots.max()) // ps + 2
    x = r.standard_normal((2, T, H, D)) * np.exp(spread * r.standard_normal((2, T, H, 1)))
    k, v = (torch.from_numpy(a).to("cuda", dtype) for a in x)
    if edit:
        edit(k, v)
    if strided:
        both = torch.cat([k.flatten(1), v.flatten(1)], 1)
        k, v = both[:, :H * D].unflatten(1, (H, D)), both[:, H * D:].unflatten(1, (H, D))
    old = r.integers(0, 256, (pages, H, ps * (D + D // 8)), dtype=np.uint8)
    cache = dev(old, torch.uint8)
    out = sv.kv4_append(k, v, dev(slots, torch.int64), cache, page_size=ps, k_scale=gk, v_scale=gv,
                        values=True)
    ref = old.copy()
    kh, vh = k.float().cpu().numpy(), v.float().cpu().numpy()
    want = np.zeros((2, T, H, D))
    for t in range(T):
        for h in range(H):
            if 0 <= slots[t] < pages * ps:
                O.put_token(ref, slots[t], h, ps, D, kh[t, h], vh[t, h], gk, gv)
            for i, (a, g) in enumerate(((kh, gk), (vh, gv))):
                for s in range(D // 16):
                    c, sc = O.quantise16(a[t, h, 16 * s:16 * s + 16], g)
                    want[i, t, h, 16 * s:16 * s + 16] = O.code_value(c, sc, g)
    assert np.array_equal(host(cache), ref)
    for i, n in enumerate("kv"):
        # code * scale * tensor scale: 6 bits times the tensor scale's, rounded to bf16 once or twice
        w = want[i]
        assert np.array_equal(np.isnan(host(out[n])), np.isnan(w))
        assert (np.nan_to_num(np.abs(host(out[n]) - w)) <= np.nan_to_num(np.abs(w)) * 2.0 ** -7.9).all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,ps,H", [(128, 16, 2), (64, 32, 3), (128, 128, 1), (64, 16, 1)])
def test_append_runs(dtype, D, ps, H):
    """Runs of tokens that start and end at odd and even slots, in pages out of order."""
    at = np.concatenate([np.arange(5, 5 + 23), [100], [103], np.arange(48, 56), [201, 202]])
    page = np.random.default_rng(1).permutation(300 // ps + 1)
    _check_append(len(at), H, D, ps, dtype, page[at // ps] * ps + at % ps)


@pytest.mark.parametrize("D", [64, 128])
def test_append_any_order(D):
    """Both tokens of a byte in one call, in every order and far apart."""
    slots = np.random.default_rng(2).permutation(64)
    _check_append(64, 2, D, 32, BF16, slots)
    _check_append(4, 1, D, 16, BF16, [1, 0, 3, 2])
    _check_append(1, 1, D, 16, F32, [15])


def test_append_views_scales_and_skips():
    _check_append(9, 2, 128, 16, BF16, np.arange(9) + 3, strided=True, spread=4.0)
    _check_append(9, 2, 64, 16, F32, np.arange(9) + 3, gk=0.013, gv=7.3, spread=6.0)
    _check_append(6, 2, 128, 16, BF16, [4, -1, 5, 6, 1 << 40, 7], pages=2)
    _check_append(3, 1, 64, 16, BF16, [30, 31, 32], pages=2)  # the last one is past the cache


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_values(dtype):
    def edit(k, v):
        k[0] = 0
        v[0, 0, :16] = -0.0
        k[1, 0, 5] = math.nan
        v[1, 0, 40] = math.inf
        k[2, 0, 7] = -math.inf
        v[2] *= 1e30
        k[3] *= 1e-30
        k[4, 0, :16] = torch.tensor([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5, -6, -0.25, -0.75,
                                     -1.25, -1.75, -2.5, -3.5, -5.0])  # ties to the even code
        v[4, 0, :16] = k[4, 0, :16] / 2
    _check_append(6, 1, 64, 16, dtype, np.arange(6) + 9, edit=edit)


def test_append_far_pages():
    """Byte offsets past 32 bits."""
    H, D, ps = 8, 128, 128
    pages = (5 << 30) // (H * ps * 144)
    cache = torch.zeros(pages, H, ps * 144, dtype=torch.uint8, device="cuda")
    k = torch.randn(3, H, D, device="cuda").to(BF16)
    v = torch.randn(3, H, D, device="cuda").to(BF16)
    slots = np.array([(pages - 1) * ps + 126, (pages - 1) * ps + 127, 0])
    sv.kv4_append(k, v, dev(slots, torch.int64), cache, page_size=ps)
    ref = np.zeros((2, H, ps * 144), np.uint8)
    for t, s in enumerate([ps + 126, ps + 127, 0]):
        for h in range(H):
            O.put_token(ref, s, h, ps, D, k[t, h].float().cpu().numpy(), v[t, h].float().cpu().numpy(), 1.0, 1.0)
    assert np.array_equal(cache[[0, -1]].cpu().numpy(), ref)
    q = torch.randn(2, 16, D, device="cuda").to(BF16)
    table = dev([[pages - 1], [0]])
    o = sv.kv4_attention(q, cache, table, dev([128, 1]), dev([0, 1, 2]), page_size=ps)
    r = O.attention(host(q), ref, np.array([[1], [0]]), [128, 1], [0, 1, 2], ps, D ** -0.5, 1.0, 1.0)
    assert np.abs(host(o["out"]) - r["out"]).max() < 0.02 and np.abs(host(o["lse"]) - r["lse"]).max() < 1e-3


# ------------------------------------------------------------------------------ attention
def random_cache(pages, H, ps, D, seed):
    """Cache bytes with every code and ordinary scales (2^-4 .. 2 in steps of the format)."""
    r = np.random.default_rng(seed)
    c = r.integers(0, 256, (pages, H, ps // 16, 18 * D), dtype=np.uint8)
    for a, b in ((8 * D, 9 * D), (17 * D, 18 * D)):
        c[..., a:b] = r.integers(24, 65, c[..., a:b].shape)
    return c.reshape(pages, H, -1)


def _tolerance(ref, D):
    """Per value: half a bf16 step; weights rounded to float16 (2^-11 of each, or half its smallest
    step of 2^-24 where the row's largest weight is 2^7, in the numerator alone); scores summed in float32 (2^-24 of the magnitudes a step, D products and the scalings)
    and exponentials (2^-22), each in numerator and denominator; the weighted sum (as much
    again)."""
    dz = (D + 8) * 2.0 ** -24 * ref["zroom"] + np.abs(np.nan_to_num(ref["lse"], neginf=0)) * 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(ref["out"]) + ref["room"] * (2.0 ** -11 + 2 * dz[..., None] + 2.0 ** -19)
    return tol + 2.0 ** -32 * ref["vsum"] + 1e-30, dz + 2.0 ** -20


def _compare(o, ref, D):
    tol, tol_lse = _tolerance(ref, D)
    for name, t in (("out", tol), ("lse", tol_lse)):
        x, y = host(o[name]), ref[name]
        fine = np.isfinite(y)
        assert np.array_equal(np.isnan(x), np.isnan(y)), name
        assert np.array_equal(x[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)]), name
        over = np.abs(x[fine] - y[fine]) / t[fine]
        assert not over.size or over.max() <= 1, (name, over.max())


def _check_attention(lens, news, hq, hk, D, ps, *, seed=0, gk=1.0, gv=0.5, max_new=None, edit=None,
                     sharp=1.0, strided=False, most=None):
    r = np.random.default_rng([seed, D, ps])
    lens, news = np.asarray(lens), np.asarray(news)
    B, T = len(lens), int(sum(news))
    held = -(-np.maximum(lens, 0) // ps)
    most = most or max(1, int(held.max()))
    held = np.minimum(held, most)
    pages = int(held.sum()) + 2
    table = np.full((B, most), -1)
    table[np.arange(most)[None] < held[:, None]] = r.permutation(pages)[:held.sum()]
    cache = random_cache(pages, hk, ps, D, seed)
    q = torch.from_numpy(sharp * r.standard_normal((T, hq, D))).to("cuda", BF16)
    if edit:
        edit(cache, table, q)
    if strided:
        q = torch.cat([q.flatten(1), torch.ones(T, 16, device="cuda", dtype=BF16)], 1)[:, :hq * D].unflatten(1, (hq, D))
    cu = np.concatenate([[0], np.cumsum(news)])
    ref = O.attention(host(q), cache, table, lens, cu, ps, 0.11, gk, gv)
    o = sv.kv4_attention(q, dev(cache, torch.uint8), dev(table), dev(lens), dev(cu), page_size=ps,
                         scale=0.11, k_scale=gk, v_scale=gv,
                         max_new=int(news.max()) if max_new is None else max_new)
    _compare(o, ref, D)
    return o, ref


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 2), (7, 1), (16, 1), (6, 6)])
def test_attention_heads(D, hq, hk):
    _check_attention([1, 17, 70], [1, 3, 5], hq, hk, D, 16, seed=hq)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_attention_pages_end_inside_tiles(ps, D):
    _check_attention([ps - 1, ps, ps + 1, 2 * ps + 5, 15, 16, 31, 33], [1, 2, 3, 4, 5, 6, 7, 8], 4,
                     1, D, ps)


@pytest.mark.parametrize("n", [1, 2, 9, 10, 17, 40])
@pytest.mark.parametrize("hq,hk,D", [(8, 1, 128), (14, 2, 64), (4, 4, 128)])
def test_attention_new_tokens(n, hq, hk, D):
    """From one row a head to several tiles of rows, with every hint."""
    for max_new in {1, n, 64}:
        _check_attention([n, n + 40], [n, n], hq, hk, D, 32, max_new=max_new)


HINTS = pytest.mark.parametrize("hint", [None, 64])  # 64: the kernel for many rows


@HINTS
def test_attention_empty(hint):
    """No tokens cached, no tokens brought, fewer cached than brought: rows that see nothing."""
    o, ref = _check_attention([0, 5, 0, 3, 20], [2, 0, 0, 7, 1], 4, 2, 128, 16, max_new=hint)
    assert (host(o["out"])[:2] == 0).all() and np.isneginf(host(o["lse"])[:6]).all()
    _check_attention([-4, 9], [1, 1], 2, 1, 64, 16, max_new=hint)


@HINTS
def test_attention_sharp_and_flat(hint):
    _check_attention([200, 300], [3, 2], 8, 2, 128, 16, sharp=30.0, max_new=hint)
    _check_attention([200, 90], [3, 2], 8, 2, 128, 16, sharp=0.0, max_new=hint)
    _check_attention([60], [2], 2, 1, 64, 16, sharp=1e-20)
    _check_attention([60], [2], 2, 1, 64, 16, gk=3e-3, gv=200.0, strided=True)


@HINTS
def test_attention_ignores_what_rows_do_not_see(hint):
    """NaN scales past the length, and in the keys and values of later drafts."""
    D, ps = 128, 16

    def edit(cache, table, q):
        c = cache.reshape(cache.shape[0], cache.shape[1], ps // 16, 18 * D)
        last = c[table[0, 2], :, 0]
        for t in (7, 8, 9, 15):  # tokens 39 (seen by all), 40, 41, 47 (past the length) of 42
            last[:, 17 * D + (t // 2) * 16 + t % 2::2][:, :1] = 0x7F if t != 7 else 0x30
        last[:, 8 * D + 9 * 8] = 0x7F       # a key of token 41
        last[:, 8 * D + 15 * 8:9 * D] = 0x7F  # the key of token 47
        c[table[1, 0], :, 0, 17 * D:] = 0xFF  # every value of the second sequence
    o, ref = _check_attention([42, 16], [4, 1], 4, 2, D, ps, edit=edit, max_new=hint)
    x = host(o["out"])
    assert np.isfinite(x[0:2]).all()                       # sees up to 39
    assert np.isnan(x[2, :, :16]).all() and np.isfinite(x[2, :, 16:]).all()  # sees 40's NaN values
    assert np.isnan(x[3:]).all()                           # sees 41's NaN key; all NaN values
    assert np.isfinite(host(o["lse"])[2]).all()


@HINTS
def test_attention_nan_inside_a_prompt(hint):
    """A prompt of several tiles of rows and tokens with a NaN value and a NaN key in its middle: rows
    before them stay what they are."""
    D, ps = 128, 16

    def edit(cache, table, q):
        c = cache.reshape(cache.shape[0], cache.shape[1], ps // 16, 18 * D)
        for tok, block in ((70, 2), (300, 5)):  # a value scale each
            c[table[0, tok // ps], :, 0, 17 * D + (tok % 16 // 2) * 16 + 2 * block + tok % 2] = 0x7F
        c[table[0, 350 // ps], :, 0, 8 * D + (350 % 16) * 8 + 3] = 0xFF  # a key
    o, _ = _check_attention([400], [400], 2, 1, D, ps, edit=edit, max_new=hint)
    x = host(o["out"])
    assert np.isfinite(x[:70]).all() and np.isnan(x[70:, :, 32:48]).all()
    assert np.isfinite(x[70:300, :, 48:]).all() and np.isnan(x[300:, :, 80:96]).all()
    assert np.isfinite(x[300:350, :, 96:]).all() and np.isnan(x[350:]).all()


@HINTS
@pytest.mark.parametrize("D", [64, 128])
def test_attention_infinite_queries(D, hint):
    def edit(cache, table, q):
        q[0, 0, 5] = math.inf
        q[1, 1, 6] = math.nan
        q[2, 2] = 1e36  # scores of up to 8e37: float32 holds them
        q[2, 3] = 1e-38
    o, _ = _check_attention([40], [3], 4, 1, D, 16, edit=edit, max_new=hint)
    assert host(o["out"])[2, 3].any()


@HINTS
@pytest.mark.parametrize("D", [64, 128])
def test_attention_pages_outside_the_cache(D, hint):
    """A page number outside the cache is not read; the rows that see its tokens are NaN."""
    def edit(cache, table, q):
        table[0, 1] = -3
        table[1, 2] = 1 << 30
    o, _ = _check_attention([40, 33, 50], [2, 2, 2], 2, 1, D, 16, edit=edit, max_new=hint)
    x = host(o["out"])
    assert np.isnan(x[:2]).all() and np.isfinite(x[2]).all() and np.isnan(x[3]).all()


@HINTS
def test_attention_lengths_past_the_table(hint):
    _check_attention([500, 20], [1, 3], 2, 1, 128, 16, most=4, max_new=hint)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk", [(2, 2), (6, 1), (16, 2), (14, 1)])
def test_attention_tiles(ps, hq, hk):
    """The kernel for many rows, with few and many of them, lengths around its tiles of 128."""
    _check_attention([127, 128, 129, 255, 260, 1, 16], [1, 2, 3, 9, 5, 1, 4], hq, hk, 128, ps,
                     max_new=64)


@HINTS
@pytest.mark.parametrize("D", [64, 128])
def test_attention_every_order_of_four_pages(D, hint):
    """Blocks that are fetched together, side by side in the cache or not, in every order."""
    orders = list(itertools.permutations(range(4)))

    def edit(cache, table, q):
        table[:] = [[4 * b + i for i in order] for b, order in enumerate(orders)]
    _check_attention([64] * len(orders), [1] * len(orders), 4, 1, D, 16, edit=edit, max_new=hint)


@HINTS
@pytest.mark.parametrize("D,ps", [(64, 16), (128, 32)])
def test_attention_uneven_batches(D, ps, hint):
    """Sequences that cost very different amounts: empty ones, single tokens, many rows, long ones."""
    r = np.random.default_rng(D)
    lens, news = r.integers(1, 300, 60), r.choice([0, 0, 1, 1, 2, 7, 12], 60)
    lens[::9], lens[4], lens[30] = r.integers(0, 20, 7), 2500, 1800
    _check_attention(lens, news, 8, 2, D, ps, max_new=hint)


def wide_cache(B, L, H, D, ps, seed):
    """A cache made on the GPU, and its keys and values [B, H, L, D] in float64."""
    g = torch.Generator("cuda").manual_seed(seed)
    blocks = -(-L // ps)
    pages = torch.randperm(B * blocks + 3, device="cuda", generator=g)[:B * blocks].view(B, blocks)
    cache = sv.kv4_cache(B * blocks + 3, H, D, ps)
    t = torch.arange(L, device="cuda")
    kv = torch.empty(2, B, H, L, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        x = torch.randn(2, L, H, D, device="cuda", generator=g).to(BF16)
        o = sv.kv4_append(x[0], x[1], pages[b, t // ps] * ps + t % ps, cache, page_size=ps,
                          values=True)
        kv[0, b], kv[1, b] = o["k"].double().transpose(0, 1), o["v"].double().transpose(0, 1)
    return cache, pages.to(torch.int32), kv


@pytest.mark.parametrize("B,L,n,hq,hk,D,ps", [
    (1, 50000, 1, 8, 1, 128, 64), (1, 50001, 5, 32, 8, 128, 128), (3, 4097, 9, 28, 4, 128, 16),
    (40, 700, 2, 8, 2, 64, 32), (300, 40, 1, 4, 2, 64, 16), (2, 3000, 70, 8, 1, 64, 16),
    (1, 30000, 9, 8, 1, 128, 64), (70, 500, 9, 14, 2, 128, 16), (2, 2900, 70, 8, 1, 128, 32)])
def test_attention_long_and_many(B, L, n, hq, hk, D, ps):
    """Long sequences and large batches, against float64 on the values that the append reports:
    work split over the tokens of a sequence and joined, and many sequences to a CTA."""
    cache, table, kv = wide_cache(B, L, hk, D, ps, B + L)
    g = torch.Generator("cuda").manual_seed(L)
    lens = torch.randint(max(n, L // 2), L + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    lens[0] = L
    news = torch.randint(1, n + 1, (B,), device="cuda", generator=g)
    news[-1] = n
    cu = torch.cat([news[:1] * 0, news.cumsum(0)]).to(torch.int32)
    T = int(cu[-1])
    q = torch.randn(T, hq, D, device="cuda", generator=g).to(BF16)
    o = sv.kv4_attention(q, cache, table, lens, cu, page_size=ps, max_new=n)
    ref = {"out": np.zeros((T, hq, D)), "lse": np.zeros((T, hq)), "room": np.zeros((T, hq, D)),
           "vsum": np.zeros((T, hq, D)), "zroom": np.zeros((T, hq))}
    G = hq // hk
    for b in range(B):
        r0, r1, m = int(cu[b]), int(cu[b + 1]), int(lens[b])
        for h in range(hq):
            K, V, x = kv[0, b, h // G, :m], kv[1, b, h // G, :m], q[r0:r1, h].double()
            z = x @ K.T * D ** -0.5
            at = m - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
            z.masked_fill_(torch.arange(m, device="cuda") > at[:, None], -math.inf)
            p = z.softmax(-1)
            ref["out"][r0:r1, h], ref["lse"][r0:r1, h] = host(p @ V), host(z.logsumexp(-1))
            ref["room"][r0:r1, h] = host(p @ V.abs())
            ref["vsum"][r0:r1, h] = host(V.abs().sum(0))
            ref["zroom"][r0:r1, h] = host((x.abs() @ K.abs().T).amax(-1) * D ** -0.5)
    _compare(o, ref, D)
    again = sv.kv4_attention(q, cache, table, lens, cu, page_size=ps, max_new=n)
    assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])


def test_attention_rows_of_no_sequence():
    """Rows before the first and past the last sequence keep what they hold."""
    cache, table, _ = wide_cache(1, 20, 1, 64, 16, 0)
    q = torch.randn(6, 2, 64, device="cuda").to(BF16)
    out = {"out": torch.full((6, 2, 64), 7.0, device="cuda", dtype=BF16),
           "lse": torch.full((6, 2), 7.0, device="cuda")}
    sv.kv4_attention(q, cache, table, dev([20]), dev([2, 4]), page_size=16, out=out)
    assert (out["out"][[0, 1, 4, 5]] == 7).all() and (out["lse"][[0, 1, 4, 5]] == 7).all()
    assert (out["out"][2:4] != 7).any()


def test_attention_streams_and_graphs():
    """On two streams at once and replayed from a graph: the eager result."""
    cache, table, _ = wide_cache(3, 3000, 2, 128, 32, 1)
    q = torch.randn(9, 8, 128, device="cuda").to(BF16)
    lens, cu = dev([3000, 1200, 77]), dev([0, 3, 8, 9])

    def call(out=None):
        return sv.kv4_attention(q, cache, table, lens, cu, page_size=32, max_new=5, out=out)
    want = call()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(20):
        for s in streams:
            with torch.cuda.stream(s):
                got.append(call())
    torch.cuda.synchronize()
    assert all(torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"]) for o in got)
    out = {k: torch.zeros_like(v) for k, v in want.items()}
    g = torch.cuda.CUDAGraph()
    with torch.cuda.stream(streams[0]), torch.cuda.graph(g, stream=streams[0]):
        call(out)
    for _ in range(3):
        out["out"].zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out["out"], want["out"]) and torch.equal(out["lse"], want["lse"])
    assert sv.device_error() == 0


def test_binding_refusals():
    cache = sv.kv4_cache(2, 1, 64, 16)
    q = torch.zeros(1, 2, 64, device="cuda", dtype=BF16)
    one, cu, table = dev([1]), dev([0, 1]), dev([[0]])
    with pytest.raises(TypeError):
        sv.kv4_attention(q.float(), cache, table, one, cu, page_size=16)
    with pytest.raises(ValueError):
        sv.kv4_attention(q, cache, table, one, cu, page_size=32)
    with pytest.raises(ValueError):
        sv.kv4_attention(q, cache, table, one, dev([0, 1, 1]), page_size=16)
    with pytest.raises(_lib.SpecVerifyError):
        sv.kv4_attention(q, cache, table, one, cu, page_size=16, scale=math.nan)
    with pytest.raises(ValueError):
        sv.kv4_append(q, q, dev([0, 1], torch.int64), cache, page_size=16)
    with pytest.raises(ValueError):
        sv.kv4_cache(2, 1, 96, 16)

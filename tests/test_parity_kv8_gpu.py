"""GPU parity of the 8-bit cache's operators (include/spec_kv.h) with the float64 oracle.

Codes, exponents and marks are equal, and so are the values that they stand for (a power of two times a
code is a bfloat16). Tolerances of attention count roundings: half a step of the output's type, 2^-11 of a
weight in float16, and those of the arithmetic in between, as each test says.
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
from oracle import kvcache8 as O  # noqa: E402

BF16, F32 = torch.bfloat16, torch.float32


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def random_cache(pages, H, ps, D, seed, low=-9, high=-4):
    """Cache bytes with every code of -127..127, ordinary exponents and no marks."""
    r = np.random.default_rng(seed)
    c = r.integers(1, 256, (pages, H, ps // 16, 32 * D + 16), dtype=np.uint8)
    c[..., 32 * D:] = 0
    c[..., 32 * D:32 * D + 2] = r.integers(low, high + 1, c[..., 32 * D:32 * D + 2].shape) % 256
    return c.reshape(pages, H, -1)


# ------------------------------------------------------------------------------ append
def _check_append(T, H, D, ps, dtype, slots, *, strided=False, spread=1.0, edit=None, seed=0, pages=None,
                  old=None, level=1.0):
    r = np.random.default_rng(seed)
    slots = np.asarray(slots)
    pages = pages or int(slots.max()) // ps + 2
    x = level * r.standard_normal((2, T, H, D)) * np.exp(spread * r.standard_normal((2, T, H, 1)))
    k, v = (torch.from_numpy(a).to("cuda", dtype) for a in x)
    if edit:
        edit(k, v)
    if strided:
        both = torch.cat([k.flatten(1), v.flatten(1)], 1)
        k, v = both[:, :H * D].unflatten(1, (H, D)), both[:, H * D:].unflatten(1, (H, D))
    old = random_cache(pages, H, ps, D, seed) if old is None else old
    cache = dev(old, torch.uint8)
    out = sv.kv8_append(k, v, dev(slots, torch.int64), cache, page_size=ps, values=True)
    ref = old.copy()
    want = O.append(ref, slots, host(k), host(v), ps)
    assert np.array_equal(host(cache), ref)
    for i, n in enumerate("kv"):
        assert np.array_equal(host(out[n]), want[i], equal_nan=True), n
    first = cache.clone()
    sv.kv8_append(k, v, dev(slots, torch.int64), cache, page_size=ps)  # again, and without the values
    assert torch.equal(first, cache)
    return ref


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,ps,H", [(128, 16, 2), (64, 32, 3), (128, 128, 1), (64, 16, 1)])
def test_append_runs(dtype, D, ps, H):
    """Runs of tokens that start and end at odd and even places, in pages out of order; blocks begun
    afresh, blocks gone on with, and single tokens."""
    at = np.concatenate([np.arange(5, 5 + 23), [100], [103], np.arange(48, 56), [201, 202], [64]])
    page = np.random.default_rng(1).permutation(300 // ps + 1)
    for level in (1.0, 0.01):  # exponents that grow, and that stay
        _check_append(len(at), H, D, ps, dtype, page[at // ps] * ps + at % ps, level=level)


@pytest.mark.parametrize("D", [64, 128])
def test_append_any_order_within_a_block(D):
    r = np.random.default_rng(2)
    slots = np.concatenate([16 * b + r.permutation(16)[:r.integers(1, 17)] for b in r.permutation(8)])
    _check_append(len(slots), 2, D, 32, BF16, slots)
    _check_append(4, 1, D, 16, BF16, [1, 0, 3, 2])
    _check_append(1, 1, D, 16, F32, [15])
    _check_append(2, 1, D, 16, F32, [9, 4])


@pytest.mark.parametrize("place", range(16))
def test_append_one_token(place):
    """One token at each place, louder and quieter than what the block holds: the other places' codes are
    rounded again or stay, byte by byte; at place 0 they are cleared."""
    for level, D, dtype in ((100.0, 128, BF16), (1e-3, 128, F32), (100.0, 64, F32), (1e-3, 64, BF16)):
        _check_append(1, 2, D, 16, dtype, [16 + place], level=level, seed=place)


def test_append_many():
    """More than one group of tokens a warp, groups that begin inside a block, many blocks."""
    r = np.random.default_rng(3)
    at = [np.arange(s, s + n) for s, n in zip(r.integers(0, 40, 70), r.integers(1, 60, 70))]
    slots = np.concatenate([112 * i + a for i, a in enumerate(at)])
    _check_append(len(slots), 3, 64, 16, BF16, slots, seed=1)
    _check_append(len(slots), 16, 64, 16, BF16, slots, seed=2)  # over the rule for groups


@pytest.mark.parametrize("H", [2, 24])
def test_append_tokens_that_are_not_written(H):
    """Between the tokens of a block, before the first and behind the last one, up to a block's 32 neighbours."""
    r = np.random.default_rng(4)
    slots = []
    for b in r.permutation(100):
        p = list(16 * b + np.sort(r.permutation(16)[:r.integers(1, 17)]))
        slots += list(r.choice([-1, 1 << 40], r.integers(0, 3)))
        while p:
            slots.append(p.pop(0))
            slots += [-1] * (r.random() < 0.3 if len(p) < 10 else 0)
        slots += [-1] * (40 if b % 20 == 0 else 0)
    _check_append(len(slots), H, 64, 16, BF16, slots, pages=101)
    _check_append(33, H, 128, 16, BF16, [17] + [-1] * 14 + [18] + [-1] * 15 + [20, -1], pages=3)


def test_append_views_and_skips():
    _check_append(9, 2, 128, 16, BF16, np.arange(9) + 3, strided=True, spread=4.0)
    _check_append(9, 2, 64, 16, F32, np.arange(9) + 3, strided=True, spread=6.0)
    _check_append(6, 2, 128, 16, BF16, [4, -1, 5, 6, 1 << 40, 7], pages=2)
    _check_append(5, 2, 64, 16, BF16, [-1, -1, -7, 3, -(1 << 62)], pages=2)
    _check_append(3, 1, 64, 16, BF16, [30, 31, 32], pages=2)  # the last one is past the cache


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_append_values(dtype, D):
    """Zeros, marks, ties, the largest and the smallest magnitudes; each token in a block of its own, and
    all in one."""
    def edit(k, v):
        k[0] = 0
        v[0, 0, :16] = -0.0
        k[1, 0, 5] = math.nan
        v[1, 0, 40] = math.inf
        k[2, 0, 7] = -math.inf
        v[2] *= 1e30
        k[3] *= 1e-30
        v[3] = 1e-40
        k[4] = 0
        k[4, 0, :10] = torch.tensor([127, 0.5, 1.5, 2.5, -0.5, -1.5, 125.5, -126.5, 63.5, -0.25])  # ties
        v[4] = k[4] / 4
        k[5, 0, 0], v[5, 0, 0] = 3.38e38, -3.3e38  # the largest exponent
    _check_append(6, 1, D, 16, dtype, np.arange(6) + 9, edit=edit)
    _check_append(6, 1, D, 16, dtype, np.arange(6), edit=edit)
    _check_append(6, 1, D, 16, dtype, 16 * np.arange(6), edit=edit)
    _check_append(6, 1, D, 16, dtype, 16 * np.arange(6) + 3, edit=edit)


def test_append_exponent_borders():
    """Largest magnitudes at and next to 127 * 2^e, for every exponent."""
    most = np.array([127.0, np.nextafter(np.float32(127), np.float32(200)), 126.99999])
    x = (most[None] * 2.0 ** np.arange(-64, 122)[:, None]).astype(np.float32).reshape(-1)

    def edit(k, v):
        k[:] = torch.from_numpy(x)[:, None, None].cuda() * torch.linspace(-1, 1, 64, device="cuda")
        k[:, 0, 63] = torch.from_numpy(x).cuda()
        v[:] = k.flip(0)
    _check_append(len(x), 1, 64, 16, F32, 16 * np.arange(len(x)), edit=edit)


def test_append_over_any_bytes():
    """A cache that held something else: blocks begun afresh do not depend on it."""
    old = np.random.default_rng(7).integers(0, 256, (3, 2, 16 * 257), dtype=np.uint8)
    clean = np.zeros_like(old)
    for o in (old, clean):
        o[..., 32 * 128 + 2:32 * 128 + 4] = o[..., 32 * 128 + 8:] = 0
    slots = np.concatenate([np.arange(16, 27), [32]])
    a = _check_append(12, 2, 128, 16, BF16, slots, old=old)
    b = _check_append(12, 2, 128, 16, BF16, slots, old=clean)
    assert np.array_equal(a[1:], b[1:])


def test_far_pages():
    """Byte offsets past 32 bits, in the append and in attention."""
    H, D, ps = 8, 128, 128
    pages = (5 << 30) // (H * ps * 257)
    cache = torch.zeros(pages, H, ps * 257, dtype=torch.uint8, device="cuda")
    k = torch.randn(4, H, D, device="cuda").to(BF16)
    v = torch.randn(4, H, D, device="cuda").to(BF16)
    slots = np.array([(pages - 1) * ps + 112, (pages - 1) * ps + 113, (pages - 1) * ps + 114, 0])
    sv.kv8_append(k, v, dev(slots, torch.int64), cache, page_size=ps)
    ref = np.zeros((2, H, ps * 257), np.uint8)
    O.append(ref, [ps + 112, ps + 113, ps + 114, 0], host(k), host(v), ps)
    assert np.array_equal(cache[[0, -1]].cpu().numpy(), ref)
    q = torch.randn(2, 16, D, device="cuda").to(BF16)
    table = dev([[pages - 1], [0]])
    for new in (1, 64, 600):
        o = sv.kv8_attention(q, cache, table, dev([115, 1]), dev([0, 1, 2]), page_size=ps, max_new=new)
        _compare(o, O.attention(host(q), ref, np.array([[1], [0]]), [115, 1], [0, 1, 2], ps, D ** -0.5), D)


# ------------------------------------------------------------------------------ attention
def _tolerance(ref, D):
    """Per value: half a bf16 step; weights times 2^e of their block rounded to float16 (2^-11 of each, or
    half its smallest step of 2^-24 where the row's largest is 2^7, in the numerator alone); scores summed in
    float32 (2^-24 of the magnitudes a step, D products and the scalings), the block's exponent added to them
    (2^-24 of score and exponent, twice) and exponentials (2^-22), each in numerator and denominator; the
    weighted sum (as much again)."""
    dz = (D + 8) * 2.0 ** -24 * ref["zroom"] + np.abs(np.nan_to_num(ref["lse"], neginf=0)) * 2.0 ** -22
    dz = dz + ref.get("emost", 0) * 2.0 ** -23
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


def _check_attention(lens, news, hq, hk, D, ps, *, seed=0, max_new=None, edit=None, sharp=1.0, strided=False,
                     most=None, scale=0.05, exponents=(-9, -4)):
    r = np.random.default_rng([seed, D, ps])
    lens, news = np.asarray(lens), np.asarray(news)
    B, T = len(lens), int(sum(news))
    held = -(-np.maximum(lens, 0) // ps)
    most = most or max(1, int(held.max()))
    held = np.minimum(held, most)
    pages = int(held.sum()) + 2
    table = np.full((B, most), -1)
    table[np.arange(most)[None] < held[:, None]] = r.permutation(pages)[:held.sum()]
    cache = random_cache(pages, hk, ps, D, seed, *exponents)
    q = torch.from_numpy(sharp * r.standard_normal((T, hq, D))).to("cuda", BF16)
    if edit:
        edit(cache.reshape(pages, hk, ps // 16, 32 * D + 16), table, q)
    if strided:
        q = torch.cat([q.flatten(1), torch.ones(T, 16, device="cuda", dtype=BF16)], 1)[:, :hq * D].unflatten(1, (hq, D))
    cu = np.concatenate([[0], np.cumsum(news)])
    ref = O.attention(host(q), cache, table, lens, cu, ps, scale)
    o = sv.kv8_attention(q, dev(cache, torch.uint8), dev(table), dev(lens), dev(cu), page_size=ps, scale=scale,
                         max_new=int(news.max()) if max_new is None else max_new)
    _compare(o, ref, D)
    return o, ref


def mark(c, page, head, token, D, keys):
    """Marks a token's keys or values in blocks [pages, heads, blocks, bytes]."""
    c[page, head, token // 16, 32 * D + (4 if keys else 6) + token % 16 // 8] |= 1 << token % 8


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
    for max_new in {1, n, 64, 600}:
        _check_attention([n, n + 40], [n, n], hq, hk, D, 32, max_new=max_new)


HINTS = pytest.mark.parametrize("hint", [None, 64, 600])  # for a few, some and many rows
DIMS = pytest.mark.parametrize("D", [64, 128])


@HINTS
@DIMS
def test_attention_empty(hint, D):
    """No tokens cached, no tokens brought, fewer cached than brought: rows that see nothing."""
    o, ref = _check_attention([0, 5, 0, 3, 20], [2, 0, 0, 7, 1], 4, 2, D, 16, max_new=hint)
    assert (host(o["out"])[:2] == 0).all() and np.isneginf(host(o["lse"])[:6]).all()
    _check_attention([-4, 9], [1, 1], 2, 1, D, 16, max_new=hint)


@HINTS
@DIMS
def test_attention_sharp_and_flat(hint, D):
    _check_attention([200, 300], [3, 2], 8, 2, D, 16, sharp=30.0, max_new=hint)
    _check_attention([200, 90], [3, 2], 8, 2, D, 16, sharp=0.0, max_new=hint)
    _check_attention([60], [2], 2, 1, D, 16, sharp=1e-20, max_new=hint)
    _check_attention([60], [2], 2, 1, D, 16, strided=True, max_new=hint)
    _check_attention([60, 77], [2, 1], 2, 1, D, 16, scale=-0.05, max_new=hint)
    _check_attention([60, 77], [2, 1], 2, 1, D, 16, scale=0.0, max_new=hint)


@HINTS
@DIMS
def test_attention_exponents_far_apart(hint, D):
    """Blocks whose exponents differ by up to 90, in keys and in values; the loudest values may have the
    smallest weights."""
    _check_attention([330, 50], [3, 2], 4, 1, D, 16, exponents=(-40, 0), max_new=hint, seed=1)

    def edit(c, table, q):
        ev = c[..., 32 * D + 1]
        ev[:] = np.random.default_rng(5).integers(-60, 31, ev.shape) % 256
    _check_attention([330, 50, 200], [3, 2, 1], 4, 1, D, 16, edit=edit, max_new=hint, seed=2)
    _check_attention([330, 50, 200], [3, 2, 1], 4, 1, D, 16, edit=edit, max_new=hint, sharp=20.0, seed=3)

    def empty_values(c, table, q):  # blocks of zeros count in the softmax
        c[table[0, ::2], :, :, 16 * D:32 * D] = 128
        c[table[0, ::2], :, :, 32 * D + 1] = -60 % 256
    _check_attention([330], [3], 4, 1, D, 16, edit=empty_values, max_new=hint, sharp=4.0, seed=4)


@HINTS
@DIMS
def test_attention_ignores_what_rows_do_not_see(hint, D):
    """Marks past the length, and in the keys and values of later drafts."""
    def edit(c, table, q):
        last = table[0, 2]
        for t in (8, 9, 15):  # tokens 40, 41, 47 (past the length) of 42
            mark(c, last, slice(None), t, D, False)
        mark(c, last, slice(None), 9, D, True)
        mark(c, last, slice(None), 15, D, True)
        c[table[1, 0], :, 0, 32 * D + 6:32 * D + 8] = 0xFF  # every value of the second sequence
    o, ref = _check_attention([42, 16], [4, 1], 4, 2, D, 16, edit=edit, max_new=hint)
    x, lse = host(o["out"]), host(o["lse"])
    assert np.isfinite(x[:2]).all() and np.isfinite(lse[:3]).all()  # rows 0 and 1 see up to 39
    assert np.isnan(x[2:]).all() and np.isnan(lse[3]).all()         # 40's value; 41's key; all values
    assert np.isfinite(lse[4]).all()


@HINTS
@DIMS
def test_attention_marks_inside_a_prompt(hint, D):
    """A prompt of several tiles with a marked value in one head and a marked key in the other: rows before
    them stay what they are."""
    def edit(c, table, q):
        for head, token, keys in ((0, 70, False), (1, 300, True)):
            mark(c, table[0, token // 16], head, token % 16, D, keys)
    o, _ = _check_attention([400], [400], 4, 2, D, 16, edit=edit, max_new=hint)
    x, lse = host(o["out"]), host(o["lse"])
    assert np.isfinite(x[:70, :2]).all() and np.isnan(x[70:, :2]).all() and np.isfinite(lse[:, :2]).all()
    assert np.isfinite(x[:300, 2:]).all() and np.isnan(x[300:, 2:]).all() and np.isnan(lse[300:, 2:]).all()


@HINTS
@DIMS
def test_attention_infinite_queries(D, hint):
    def edit(c, table, q):
        q[0, 0, 5] = math.inf
        q[1, 1, 6] = math.nan
        q[2, 2] = 1e30
        q[2, 3] = 1e-38
    o, _ = _check_attention([40], [3], 4, 1, D, 16, edit=edit, max_new=hint)
    assert host(o["out"])[2, 3].any()


@HINTS
@DIMS
def test_attention_pages_outside_the_cache(D, hint):
    """A page number outside the cache is not read; the rows that see its tokens are NaN."""
    def edit(c, table, q):
        table[0, 1] = -3
        table[1, 2] = 1 << 30
    o, _ = _check_attention([40, 33, 50], [2, 2, 2], 2, 1, D, 16, edit=edit, max_new=hint)
    x = host(o["out"])
    assert np.isnan(x[:2]).all() and np.isfinite(x[2]).all() and np.isnan(x[3]).all()


@HINTS
@DIMS
def test_attention_lengths_past_the_table(hint, D):
    _check_attention([500, 20], [1, 3], 2, 1, D, 16, most=4, max_new=hint)


@pytest.mark.parametrize("ps", [16, 32, 64, 128])
@pytest.mark.parametrize("hq,hk", [(2, 2), (6, 1), (16, 2), (14, 1)])
@DIMS
def test_attention_tiles(ps, hq, hk, D):
    """Few and many rows, lengths around tiles of 64 and 128 tokens."""
    for hint in (64, 600):
        _check_attention([127, 128, 129, 255, 260, 1, 16], [1, 2, 3, 9, 5, 1, 4], hq, hk, D, ps, max_new=hint)


@HINTS
@DIMS
def test_attention_every_order_of_four_pages(D, hint):
    """Blocks that are fetched together, side by side in the cache or not, in every order."""
    orders = list(itertools.permutations(range(4)))

    def edit(c, table, q):
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
    """A cache made on the GPU, its keys and values [B, H, L, D] and the values' exponents [B, H, L], all in
    float64."""
    g = torch.Generator("cuda").manual_seed(seed)
    blocks = -(-L // ps)
    pages = torch.randperm(B * blocks + 3, device="cuda", generator=g)[:B * blocks].view(B, blocks)
    cache = sv.kv8_cache(B * blocks + 3, H, D, ps)
    t = torch.arange(L, device="cuda")
    kv = torch.empty(2, B, H, L, D, dtype=torch.float64, device="cuda")
    for b in range(B):
        x = torch.randn(2, L, H, D, device="cuda", generator=g).to(BF16)
        o = sv.kv8_append(x[0], x[1], pages[b, t // ps] * ps + t % ps, cache, page_size=ps, values=True)
        kv[0, b], kv[1, b] = o["k"].double().transpose(0, 1), o["v"].double().transpose(0, 1)
    heads = cache.view(B * blocks + 3, H, ps // 16, -1)[pages][..., 32 * D + 1].view(torch.int8)  # [B, blocks, H, .]
    e = heads.permute(0, 2, 1, 3).flatten(2).repeat_interleave(16, 2)[..., :L].double()
    return cache, pages.to(torch.int32), kv, e


@pytest.mark.parametrize("B,L,n,hq,hk,D,ps", [
    (1, 50000, 1, 8, 1, 128, 64), (1, 50001, 5, 32, 8, 128, 128), (3, 4097, 9, 28, 4, 128, 16),
    (40, 700, 2, 8, 2, 64, 32), (300, 40, 1, 4, 2, 64, 16), (2, 3000, 70, 8, 1, 64, 16),
    (1, 30000, 9, 8, 1, 128, 64), (70, 500, 9, 14, 2, 128, 16), (2, 2900, 70, 8, 1, 128, 32),
    (2, 2500, 800, 8, 2, 128, 64), (3, 1500, 1500, 4, 4, 128, 16), (2, 2000, 900, 16, 2, 64, 32)])
def test_attention_long_and_many(B, L, n, hq, hk, D, ps):
    """Long sequences and large batches, against float64 on the values that the append reports:
    work split over the tokens of a sequence and joined, and many sequences to a CTA."""
    cache, table, kv, ev = wide_cache(B, L, hk, D, ps, B + L)
    g = torch.Generator("cuda").manual_seed(L)
    lens = torch.randint(max(n, L // 2), L + 1, (B,), device="cuda", generator=g, dtype=torch.int32)
    lens[0] = L
    news = torch.randint(1, n + 1, (B,), device="cuda", generator=g)
    news[-1] = n
    cu = torch.cat([news[:1] * 0, news.cumsum(0)]).to(torch.int32)
    T = int(cu[-1])
    q = torch.randn(T, hq, D, device="cuda", generator=g).to(BF16)
    o = sv.kv8_attention(q, cache, table, lens, cu, page_size=ps, max_new=n)
    ref = {"out": np.zeros((T, hq, D)), "lse": np.zeros((T, hq)), "room": np.zeros((T, hq, D)),
           "vsum": np.zeros((T, hq, D)), "zroom": np.zeros((T, hq)), "emost": float(ev.abs().max())}
    G = hq // hk
    for b in range(B):
        r0, r1, m = int(cu[b]), int(cu[b + 1]), int(lens[b])
        for h in range(hq):
            K, V, x = kv[0, b, h // G, :m], kv[1, b, h // G, :m], q[r0:r1, h].double()
            two = ev[b, h // G, :m].exp2()
            z = x @ K.T * D ** -0.5
            at = m - (r1 - r0) + torch.arange(r1 - r0, device="cuda")
            z.masked_fill_(torch.arange(m, device="cuda") > at[:, None], -math.inf)
            p = z.softmax(-1)
            ref["out"][r0:r1, h], ref["lse"][r0:r1, h] = host(p @ V), host(z.logsumexp(-1))
            ref["room"][r0:r1, h] = host(p @ V.abs())
            ref["vsum"][r0:r1, h] = host((p * two).amax(-1)[:, None] * (V.abs() / two[:, None]).sum(0))
            ref["zroom"][r0:r1, h] = host((x.abs() @ K.abs().T).amax(-1) * D ** -0.5)
    _compare(o, ref, D)
    again = sv.kv8_attention(q, cache, table, lens, cu, page_size=ps, max_new=n)
    assert torch.equal(o["out"], again["out"]) and torch.equal(o["lse"], again["lse"])


@HINTS
def test_attention_rows_of_no_sequence(hint):
    """Rows before the first and past the last sequence keep what they hold."""
    cache, table = wide_cache(1, 20, 1, 64, 16, 0)[:2]
    q = torch.randn(6, 2, 64, device="cuda").to(BF16)
    out = {"out": torch.full((6, 2, 64), 7.0, device="cuda", dtype=BF16),
           "lse": torch.full((6, 2), 7.0, device="cuda")}
    sv.kv8_attention(q, cache, table, dev([20]), dev([2, 4]), page_size=16, out=out, max_new=hint or 1)
    assert (out["out"][[0, 1, 4, 5]] == 7).all() and (out["lse"][[0, 1, 4, 5]] == 7).all()
    assert (out["out"][2:4] != 7).any()


@pytest.mark.parametrize("new", [5, 700])
def test_attention_streams_and_graphs(new):
    """On two streams at once and replayed from a graph: the eager result."""
    cache, table = wide_cache(3, 3000, 2, 128, 32, 1)[:2]
    T = new + 6
    q = torch.randn(T, 8, 128, device="cuda").to(BF16)
    lens, cu = dev([3000, 1200, 77]), dev([0, new - 2, new + 5, T])

    def call(out=None):
        return sv.kv8_attention(q, cache, table, lens, cu, page_size=32, max_new=new, out=out)
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


@pytest.mark.parametrize("keys", [True, False])
def test_append_one_output(keys):
    """The values as held of keys alone, or of values alone, for every token, written to the cache or not."""
    from speculative_decoding_verification_33_gb300 import _lib
    T, H, D, ps = 40, 2, 64, 16
    slots = np.where(np.arange(T) % 7 == 3, -1, np.arange(T) + 5)
    k, v = (torch.randn(T, H, D, device="cuda").to(BF16) for _ in range(2))
    caches = [sv.kv8_cache(4, H, D, ps) for _ in range(2)]
    want = sv.kv8_append(k, v, dev(slots, torch.int64), caches[0], page_size=ps, values=True)
    out, s = torch.full_like(k, 7.0), dev(slots, torch.int64)
    st = _lib.load().spec_kv8_append(
        T, H, D, ps, 4, 1, k.data_ptr(), H * D, v.data_ptr(), H * D, s.data_ptr(), caches[1].data_ptr(),
        out.data_ptr() if keys else 0, 0 if keys else out.data_ptr(), torch.cuda.current_stream().cuda_stream)
    assert st == 0
    torch.cuda.synchronize()
    assert torch.equal(out, want["k" if keys else "v"]) and torch.equal(caches[0], caches[1])

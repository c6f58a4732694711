"""Attention over the 8-bit cache at the edges of its definition, in each of its three forms: register operands
(few rows a head), one tile of rows over two streams of tokens, two tiles of rows."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from tests import test_parity_kv8_gpu as K  # noqa: E402
from tests.test_parity_kv8_gpu import BF16, _check_attention, _compare, dev, host, wide_cache  # noqa: E402

DIMS = pytest.mark.parametrize("D", [64, 128])


def dense_reference(q, kv, ev, lens, news, scale):
    """What ``oracle.kvcache8.attention`` gives, in float64 on the GPU, for sequences of much the same size: keys
    and values [2, B, H, L, D], the values' exponents [B, H, L]."""
    B, H, L, D = kv.shape[1:]
    hq, n = q.shape[1], int(news.max())
    G = hq // H
    cu = np.concatenate([[0], np.cumsum(news)])
    at = torch.from_numpy(np.minimum(cu[:-1, None] + np.arange(n), len(q) - 1)).cuda()
    x = q[at].double().view(B, n, H, G, D).permute(0, 2, 3, 1, 4).reshape(B, H, G * n, D)
    z = x @ kv[0].transpose(-1, -2) * scale
    sees = (torch.from_numpy(lens - news).cuda()[:, None] + torch.arange(n, device="cuda") + 1)[:, None, :, None]
    hidden = (torch.arange(L, device="cuda") >= sees).repeat(1, G, 1, 1).view(B, 1, G * n, L)
    z = z.masked_fill(hidden, -math.inf)
    p = z.softmax(-1).nan_to_num(0.0)
    two = ev.exp2()
    o = {"out": p @ kv[1], "lse": z.logsumexp(-1), "room": p @ kv[1].abs(),
         "vsum": (p * two[:, :, None]).amax(-1, keepdim=True) * (kv[1].abs() / two[..., None]).sum(2, keepdim=True),
         "zroom": (x.abs() @ kv[0].abs().transpose(-1, -2)).amax(-1) * abs(scale)}
    there = torch.from_numpy(np.arange(n)[None] < news[:, None]).cuda()
    o = {k: host(y.unflatten(2, (G, n)).permute((0, 3, 1, 2, 4)[:y.dim() + 1]).flatten(2, 3)[there])
         for k, y in o.items()}
    return {**o, "emost": float(ev.abs().max())}


@DIMS
@pytest.mark.parametrize("L", [100, 128, 300])
def test_tiles_without_rows(L, D):
    """Two tiles of rows for sequences of which most bring one token: items of few units, many in a row, whose
    second tile has no rows, between others that fill both."""
    B, hq, H, ps = 330, 8, 2, 16
    cache, table, kv, ev = wide_cache(B, L, H, D, ps, L)
    r = np.random.default_rng([L, D])
    news = np.where(r.random(B) < 0.02, r.integers(33, 80, B), 1)
    lens = np.maximum(news, r.integers(1, L + 1, B))
    q = torch.randn(int(news.sum()), hq, D, device="cuda").to(BF16)
    cu = dev(np.concatenate([[0], np.cumsum(news)]))
    ref = dense_reference(q, kv, ev, lens, news, D ** -0.5)
    for _ in range(20):
        o = sv.kv8_attention(q, cache, table, dev(lens), cu, page_size=ps, max_new=600)
    _compare(o, ref, D)
    assert sv.device_error() == 0


FORMS = pytest.mark.parametrize("rows", [4, 20, 100, 600])  # a head, as the caller says: each form of the kernel


@FORMS
@DIMS
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_scale_of_zero(rows, D, scale):
    """Every token counts alike, however large keys and queries are: their products pass 2^120 and more."""
    def edit(c, table, q):
        c[..., 32 * D] = np.random.default_rng(1).integers(60, 122, c.shape[:3])
        q[3:] *= 1e15
    o, ref = _check_attention([150, 300, 3], [2, 3, 1], 4, 2, D, 16, scale=scale, max_new=rows // 2, edit=edit)
    assert np.allclose(ref["lse"][:, 0], np.log([149, 150, 298, 299, 300, 3]))


def values_exponents(c, which, D):
    """Exponents of the values of blocks [pages, heads, blocks, bytes], from a function of page and block."""
    pages, _, blocks, _ = c.shape
    for p in range(pages):
        for j in range(blocks):
            c[p, :, j, 32 * D + 1] = which(p, j) % 256


@FORMS
@DIMS
@pytest.mark.parametrize("sharp", [1.0, 20.0, 60.0])
def test_exponents_of_the_whole_range(rows, D, sharp):
    """Values of every exponent that the append writes, from -60 to 121, side by side."""
    def edit(c, table, q):
        c[..., 32 * D + 1] = np.random.default_rng(7).integers(-60, 122, c.shape[:3]) % 256
    _check_attention([330, 50, 1200], [3, 2, 4], 4, 1, D, 16, edit=edit, max_new=rows // 4, sharp=sharp)


@FORMS
@DIMS
@pytest.mark.parametrize("order", ["quiet first", "loud first", "in turn", "nothing but zeros beside"])
def test_quiet_and_loud_values(rows, D, order):
    """Whole runs of blocks of the least exponents beside those of the largest: all count in the softmax's sum, in
    whatever order they come and wherever the work is cut."""
    L, ps = 2600, 32
    blocks = -(-L // ps)

    def edit(c, table, q):
        r, at = np.random.default_rng(3), {int(p): i for i, p in enumerate(table[0])}
        late = order == "quiet first"

        def e(p, j):
            i = at.get(p, 0)
            loud = (i >= blocks // 2) == late if order in ("quiet first", "loud first") else (i + j) % 3 == 0
            return int(r.integers(110, 122)) if loud else -60
        values_exponents(c, e, D)
        if order == "nothing but zeros beside":
            c.reshape(-1, 32 * D + 16)[c[..., 32 * D + 1].reshape(-1) == 196, 16 * D:32 * D] = 128
    for sharp in (1.0, 30.0):
        _check_attention([L], [3], 4, 1, D, ps, edit=edit, max_new=rows // 4, sharp=sharp)


@DIMS
@pytest.mark.parametrize("hint", [32, 60])  # 64 to 128 rows a head for groups of two and four
@pytest.mark.parametrize("case", [
    K.test_attention_empty, K.test_attention_sharp_and_flat, K.test_attention_exponents_far_apart,
    K.test_attention_ignores_what_rows_do_not_see, K.test_attention_marks_inside_a_prompt,
    K.test_attention_infinite_queries, K.test_attention_pages_outside_the_cache,
    K.test_attention_lengths_past_the_table, K.test_attention_every_order_of_four_pages],
    ids=lambda f: f.__name__[15:])
def test_one_tile_of_rows(case, hint, D):
    """The cases of the other forms where one tile of rows goes over two streams of tokens: values lag keys by a
    unit, and streams with maxima of their own are joined."""
    case(hint=hint, D=D)


@pytest.mark.parametrize("B,L,n,hq,hk,D,ps", [
    (2, 6000, 16, 16, 2, 64, 32), (40, 900, 25, 8, 2, 64, 16), (1, 20000, 100, 1, 1, 64, 64),
    (3, 4000, 30, 8, 2, 128, 64), (1, 9001, 65, 2, 1, 128, 16), (60, 400, 40, 4, 2, 128, 32)])
def test_one_tile_of_rows_long_and_many(B, L, n, hq, hk, D, ps):
    """Rings of operands and bytes that wrap many times, work cut over a sequence's tokens."""
    K.test_attention_long_and_many(B, L, n, hq, hk, D, ps)


@FORMS
@DIMS
def test_key_exponents_of_the_whole_range(rows, D):
    """Keys of every exponent side by side, with queries that bring the loudest ones' scores to the order of 1."""
    def edit(c, table, q):
        c[..., 32 * D] = np.random.default_rng(11).integers(-60, 122, c.shape[:3]) % 256
    _check_attention([330, 50, 900], [3, 2, 4], 4, 1, D, 16, edit=edit, max_new=rows // 4, sharp=1e-30, scale=1e-9)


@FORMS
@DIMS
def test_append_and_attend_at_every_magnitude(rows, D):
    """Values from 1e-25 to 1e37 and blocks of zeros, appended as they come and attended to."""
    L, H, ps = 700, 2, 32
    r, g = np.random.default_rng(D), torch.Generator("cuda").manual_seed(D)
    k, v = (torch.randn(L, H, D, device="cuda", generator=g) for _ in "kv")
    size = 10.0 ** torch.from_numpy(r.uniform(-25, 37, -(-L // 16))).cuda().repeat_interleave(16)[:L]
    size[::100] *= 0.01
    v = (v * size[:, None, None]).to(BF16)
    v[160:208] = 0.0
    table = r.permutation(-(-L // ps))[None]
    slots = table[0][np.arange(L) // ps] * ps + np.arange(L) % ps
    cache = sv.kv8_cache(table.size, H, D, ps)
    for a, b in ((0, 16), (16, 333), (333, 334), (334, L)):
        sv.kv8_append(k[a:b].to(BF16), v[a:b], dev(slots[a:b], torch.int64), cache, page_size=ps)
    q = torch.randn(6, 4 * H, D, device="cuda", generator=g).to(BF16)
    lens, cu = np.array([L]), np.array([0, 6])
    o = sv.kv8_attention(q, cache, dev(table), dev(lens), dev(cu), page_size=ps, max_new=rows // 4)
    _compare(o, K.O.attention(host(q), cache.cpu().numpy(), table, lens, cu, ps, D ** -0.5), D)

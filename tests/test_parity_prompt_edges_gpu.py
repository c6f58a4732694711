"""Packed prompt attention at the edges of its definition: values that are not finite in every item of work, work
that is taken without an order, repeated calls bit by bit."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from tests.test_parity_prompt_gpu import BF16, DIMS, _compare, dev, host  # noqa: E402


def rows_reference(q, k, v, first, rows, scale):
    """What ``oracle.kvcache8.rows_attention`` gives, in float64 on the GPU: each of ``rows`` of q over the keys
    and values of its sequence, which starts at ``first``, up to itself. Sequences of much the same length."""
    n, (hq, D), H = len(rows), q.shape[1:], k.shape[1]
    L = int((rows - first).max()) + 1
    at = (torch.from_numpy(first).cuda()[:, None] + torch.arange(L, device="cuda")).clamp(max=len(k) - 1)
    hidden = torch.arange(L, device="cuda") > torch.from_numpy(rows - first).cuda()[:, None]
    K, V = (x[at].double().masked_fill_(hidden[..., None, None], 0.0).permute(0, 2, 1, 3) for x in (k, v))
    x = q[torch.from_numpy(rows).cuda()].double().view(n, H, hq // H, D)
    z = (x @ K.transpose(-1, -2) * scale).masked_fill_(hidden[:, None, None], -math.inf)
    p = z.softmax(-1)
    # a weight of 0 is one of a token that the row does not see
    o = {"out": p @ V, "lse": z.logsumexp(-1), "room": p @ V.abs(),
         "zroom": (x.abs() @ K.abs().transpose(-1, -2)).amax(-1) * abs(scale)}
    return {name: host(y.flatten(1, 2)) for name, y in o.items()}


def check(q, k, v, lens, rows=None, scale=None, chunk=4096):
    """A call's ``rows`` (all) with float64, and the call again, bit by bit. Rows of no sequence keep what they hold."""
    T, hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    cu = np.concatenate([[0], np.cumsum(lens)])
    out = {"out": torch.full((T, hq, D), 7.0, device="cuda", dtype=BF16), "lse": torch.full((T, hq), 7.0, device="cuda")}
    o = sv.prompt_attention(q, k, v, dev(cu), scale=scale, out=out)
    assert sv.device_error() == 0
    assert (o["out"][cu[-1]:] == 7).all() and (o["lse"][cu[-1]:] == 7).all()
    first = np.repeat(cu[:-1], lens)
    rows = np.arange(cu[-1]) if rows is None else rows
    for a in range(0, len(rows), chunk):
        r = rows[a:a + chunk]
        _compare({x: o[x][torch.from_numpy(r).cuda()] for x in o}, rows_reference(q, k, v, first[r], r, scale), D)
    again = {x: torch.full_like(y, 7.0) for x, y in o.items()}
    sv.prompt_attention(q, k, v, dev(cu), scale=scale, out=again)
    assert torch.equal(again["out"].view(torch.int16), o["out"].view(torch.int16))
    assert torch.equal(again["lse"].view(torch.int32), o["lse"].view(torch.int32))
    return o


def inputs(T, hq, hk, D, seed):
    g = torch.Generator("cuda").manual_seed(seed)
    return [torch.randn(T, h, D, device="cuda", generator=g).to(BF16) for h in (hq, hk, hk)]


KINDS = (math.nan, math.inf, -math.inf)


@DIMS
@pytest.mark.parametrize("hq,hk", [(8, 8), (20, 10)])
def test_values_not_finite_in_every_sequence(hq, hk, D):
    """More than a hundred items for each CTA, each with some such value, of one kind or of two in a dimension."""
    r = np.random.default_rng([hq, D])
    lens = r.integers(2, 8, 2500)
    cu = np.concatenate([[0], np.cumsum(lens)])
    q, k, v = inputs(cu[-1], hq, hk, D, 1)
    for b in range(len(lens)):
        for h in r.choice(hk, 2, replace=False):
            for _ in range(2):
                v[cu[b] + int(r.integers(lens[b])), int(h), int(r.choice([3, D - 1]))] = KINDS[r.integers(3)]
    o = check(q, k, v, lens)
    assert o["lse"].isfinite().all() and not o["out"].isfinite().all()


@DIMS
@pytest.mark.parametrize("n,hq,hk", [(300, 1, 1), (257, 2, 1), (700, 3, 1), (390, 4, 2), (520, 6, 6)])
def test_kinds_of_values_not_finite(n, hq, hk, D):
    """Each kind at some token of each dimension, the next one later: rows see none, one or both."""
    r = np.random.default_rng(n)
    q, k, v = inputs(n, hq, hk, D, n)
    for d in range(0, D, 3):
        for t in r.choice(n, 2, replace=False):
            v[int(t), int(r.integers(hk)), d] = KINDS[r.integers(3)]
    v[5, 0, D - 1], v[200, 0, D - 1] = math.inf, -math.inf
    o = check(q, k, v, [n])
    x = host(o["out"])[:, 0, D - 1]
    if (D - 1) % 3:  # no other one in that dimension
        assert np.isfinite(x[:5]).all() and (x[5:200] == math.inf).all() and np.isnan(x[200:]).all()


@DIMS
def test_keys_and_values_not_finite(D):
    """A token of infinite keys and values: rows whose score for it is -inf have a weight of 0, and NaN values."""
    q, k, v = inputs(400, 4, 2, D, 3)
    q[..., 0] = q[..., 0].abs() + 0.5
    for t in (70, 200, 333):
        k[t, t % 2, 0], v[t, t % 2, 5], v[t, t % 2, 6] = -math.inf, math.inf, math.nan
    o = check(q, k, v, [400])
    assert o["lse"].isfinite().all() and o["out"][334:, :, 5].isnan().all()


def test_values_not_finite_throughout_a_long_prompt():
    """98304 tokens with an infinity in every item: as fast as any other, and what later rows see is exact."""
    T, hq, hk, D = 98304, 32, 4, 64
    q, k, v = inputs(T, hq, hk, D, 5)
    t = torch.arange(7, T, 32, device="cuda")
    v[t, :, t // 2048] = math.inf
    rows = np.unique(np.concatenate([np.arange(60), np.random.default_rng(2).integers(0, T, 24),
                                     [T - 1, T - 32, 2048, 2054, 2055]]))
    o = check(q, k, v, [T], rows, chunk=2)
    assert o["lse"].isfinite().all()


@DIMS
@pytest.mark.parametrize("scale", [0.0, -0.0])
def test_scale_of_zero(D, scale):
    """Every token counts alike, however large keys and queries are: their products reach 2^125."""
    q, k, v = inputs(290, 4, 2, D, 9)
    q[100:], k[100:] = q[100:] * 1e18, k[100:] * 1e18
    q[50] *= 1e35
    o = check(q, k, v, [90, 200], scale=scale)
    assert np.allclose(host(o["lse"])[:, 0], np.log(np.concatenate([np.arange(90), np.arange(200)]) + 1.0))


@DIMS
@pytest.mark.parametrize("B,empty", [(1023, 0.0), (1024, 0.3), (1025, 0.3), (3000, 0.9), (3000, 0.05)])
def test_sequences_around_the_limit_of_ordering(B, empty, D):
    """Up to 1024 sequences are taken in the order of their cost, more as they come."""
    r = np.random.default_rng([B, D])
    lens = np.where(r.random(B) < empty, 0, r.integers(1, 40, B))
    lens[r.integers(0, B, 3)] = 300
    q, k, v = inputs(int(lens.sum()) + 9, 4, 2, D, B)
    check(q, k, v, lens, chunk=1024)


@DIMS
@pytest.mark.parametrize("lens", [[2046], [2047], [2048], [2049], [2100], [3, 2300, 0, 70, 2050], [1500, 2052, 2400]])
def test_tiles_around_the_limit_of_ordering(lens, D):
    """128 query heads on one: two tokens are an item, and more than 1024 of a sequence are taken as they come."""
    q, k, v = inputs(sum(lens), 128, 1, D, sum(lens))
    check(q, k, v, lens, chunk=64)


@DIMS
def test_more_sequences_than_an_order_holds_and_long_ones(D):
    r = np.random.default_rng(D)
    lens = r.integers(0, 9, 1500)
    lens[[3, 700, 1499]] = 2600, 1900, 3001
    q, k, v = inputs(int(lens.sum()), 14, 2, D, 4)
    check(q, k, v, lens, np.unique(r.integers(0, int(lens.sum()), 700)), chunk=50)

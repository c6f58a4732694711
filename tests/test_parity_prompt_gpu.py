"""GPU parity of packed prompt attention (spec_prompt_attention) with the float64 oracle. Tolerances count
roundings: half a step of the output's type, 2^-8 of a weight in bfloat16, and those of the arithmetic in
between."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from oracle import kvcache8 as O  # noqa: E402

BF16 = torch.bfloat16
DIMS = pytest.mark.parametrize("D", [64, 128])


def dev(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda", dtype)


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def _compare(o, ref, D, rows=slice(None)):
    """Per value: half a bf16 step; weights rounded to bfloat16 in the numerator alone (2^-8 of each; its
    range is float32's, down to which nothing is lost); scores summed in float32 (2^-24 of the magnitudes a
    step, D products and the scaling) and exponentials (2^-22), each in numerator and denominator; the
    weighted sum (as much again)."""
    dz = (D + 8) * 2.0 ** -24 * ref["zroom"] + np.abs(np.nan_to_num(ref["lse"], neginf=0)) * 2.0 ** -22
    tol = 2.0 ** -8 * np.abs(ref["out"]) + ref["room"] * (2.0 ** -8 + 2 * dz[..., None] + 2.0 ** -18) + 1e-30
    for name, t in (("out", tol), ("lse", dz + 2.0 ** -19)):
        x, y, t = host(o[name])[rows], ref[name][rows], t[rows]
        fine = np.isfinite(y)
        assert np.array_equal(np.isnan(x), np.isnan(y)), name
        assert np.array_equal(x[~fine & ~np.isnan(y)], y[~fine & ~np.isnan(y)]), name
        over = np.abs(x[fine] - y[fine]) / t[fine]
        assert not over.size or over.max() <= 1, (name, over.max())


def _check(lens, hq, hk, D, *, seed=0, scale=None, sharp=1.0, edit=None, layout="apart", cu=None, T=None):
    r = np.random.default_rng([seed, D, hq])
    cu = np.concatenate([[0], np.cumsum(lens)]) if cu is None else np.asarray(cu)
    T = int(cu[-1]) if T is None else T
    q, k, v = (torch.from_numpy(s * r.standard_normal((T, h, D))).to("cuda", BF16)
               for h, s in ((hq, sharp), (hk, 1.0), (hk, 1.0)))
    if edit:
        edit(q, k, v)
    if layout == "one":  # views of one projection's output
        x = torch.cat([q.flatten(1), k.flatten(1), v.flatten(1)], 1)
        q, k, v = (y.unflatten(1, (-1, D)) for y in x.split([hq * D, hk * D, hk * D], 1))
    out = {"out": torch.full((T, hq, D), 7.0, device="cuda", dtype=BF16),
           "lse": torch.full((T, hq), 7.0, device="cuda")}
    o = sv.prompt_attention(q, k, v, dev(cu), scale=scale, out=out)
    held = np.clip(cu, 0, T)
    ref = O.prompt_attention(host(q), host(k), host(v), held, D ** -0.5 if scale is None else scale)
    rows = np.zeros(T, bool)
    rows[held[0]:held[-1]] = True
    _compare(o, ref, D, rows)
    assert (host(o["out"])[~rows] == 7).all() and (host(o["lse"])[~rows] == 7).all()
    again = sv.prompt_attention(q, k, v, dev(cu), scale=scale)
    assert torch.equal(again["out"][rows], o["out"][rows]) or o["out"].isnan().any()
    return o, ref


@DIMS
@pytest.mark.parametrize("hq,hk", [(1, 1), (8, 2), (7, 1), (16, 1), (6, 6), (3, 1), (5, 1), (64, 1), (128, 1), (100, 1)])
def test_heads(D, hq, hk):
    """Groups of query heads that divide a tile of 128 rows, and that do not."""
    _check([1, 17, 70, 3], hq, hk, D, seed=hq)


@DIMS
@pytest.mark.parametrize("n", [1, 2, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 256, 257, 300])
def test_lengths(D, n):
    """Lengths around the tiles of rows and tokens."""
    _check([n], 4, 1, D)
    _check([n, n], 1, 1, D)


@DIMS
@pytest.mark.parametrize("seed", range(4))
def test_packed(D, seed):
    r = np.random.default_rng(seed)
    lens = r.choice([0, 1, 2, 5, 40, 130, 260], 20)
    _check(lens, *((8, 2), (4, 4), (7, 1), (12, 2))[seed], D, seed=seed, layout=("apart", "one")[seed % 2])


@DIMS
def test_many_sequences(D):
    _check(np.random.default_rng(1).integers(0, 4, 700), 2, 1, D)


@DIMS
def test_rows_of_no_sequence(D):
    """Rows before the first and past the last sequence keep what they hold, whatever else they hold."""
    def edit(q, k, v):
        for x in (q, k, v):
            x[:3], x[150:] = math.nan, math.inf
    _check(None, 4, 2, D, cu=[3, 3, 50, 150], T=170, edit=edit)
    _check(None, 4, 2, D, cu=[0, 0, 0], T=5)
    _check(None, 2, 1, D, cu=[-4, 9, 400], T=40)  # held to the rows there are


@DIMS
def test_sharp_flat_and_scaled(D):
    _check([200, 90], 8, 2, D, sharp=30.0)
    _check([200, 90], 8, 2, D, sharp=0.0)
    _check([200, 90], 8, 2, D, scale=-0.2)
    _check([200, 90], 8, 2, D, scale=0.0)
    _check([140], 2, 1, D, sharp=1e-20)

    def edit(q, k, v):  # maxima that rise along the tokens, by a lot and by little
        k[:] = k * (0.05 * torch.arange(len(k), device="cuda"))[:, None, None]
    _check([600], 4, 1, D, edit=edit, scale=0.3)

    def falling(q, k, v):
        q[:] = q.abs()
        k[:] = -k.abs() * (0.05 * torch.arange(len(k), device="cuda"))[:, None, None]
    _check([600], 4, 1, D, edit=falling, scale=0.3)


@DIMS
def test_scores_far_from_zero(D):
    """Scores of up to 1e31: the largest decides, in rows and tiles whose maxima differ by a lot."""
    def edit(q, k, v):
        q[3:200] *= 1e30
        q[200:210] *= 1e7
        q[210] *= -1e20
        k[100] *= 3.0
    _check([300, 40], 4, 2, D, edit=edit)
    _check([300, 40], 4, 2, D, edit=edit, scale=-0.1)


@DIMS
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("at", [0, 5, 31, 32, 127, 128, 200, 255, 256, 299])
def test_values_that_rows_do_not_see(D, bad, at):
    """A NaN or an infinity in one value of one token: rows before it stay what they are, as do the other
    dimensions and heads."""
    def edit(q, k, v):
        v[at, 0, 11] = bad
    for hq, hk in ((4, 2), (1, 1)):
        o, ref = _check([300], hq, hk, D, edit=edit, seed=at)
        x = host(o["out"])
        assert np.isfinite(x[:at]).all() and np.isfinite(np.delete(x, 11, 2)).all()
        assert not np.isfinite(x[at:, 0, 11]).any() and np.isfinite(host(o["lse"])).all()


@DIMS
def test_keys_and_queries_that_are_not_finite(D):
    def edit(q, k, v):
        k[100, 0, 3] = math.nan
        q[40, 2, 5] = math.nan
        q[41, 3, 5] = math.inf
        v[250, 1] = math.nan
        v[251, 1] = -math.inf
    o, _ = _check([270, 60], 4, 2, D, edit=edit)
    x = host(o["out"])
    assert np.isfinite(x[:40]).all() and np.isnan(x[40, 2]).all() and np.isnan(x[100:270, :2]).all()
    assert np.isfinite(x[42:250, 2:]).all() and np.isfinite(x[270:]).all()


@DIMS
def test_neighbours_that_are_not_finite(D):
    """Whole sequences of NaN between others."""
    def edit(q, k, v):
        for x in (q, k, v):
            x[33:80] = math.nan
            x[200:201] = math.inf
    o, _ = _check([33, 47, 120, 1, 70], 4, 2, D, edit=edit)
    x = host(o["out"])
    assert np.isfinite(x[:33]).all() and np.isnan(x[33:80]).all() and np.isfinite(x[80:200]).all()
    assert np.isfinite(x[201:]).all()


@pytest.mark.parametrize("lens,hq,hk,D", [
    ([4097], 8, 2, 128), ([5000, 1, 2300, 700], 28, 4, 128), ([6001], 4, 4, 64), ([3000, 2999], 16, 2, 64),
    ([700] * 40, 4, 1, 128), ([20000], 2, 1, 128)])
def test_long(lens, hq, hk, D):
    """Against float64 on the GPU, row by row bounds; the same again on another stream and from a graph."""
    g = torch.Generator("cuda").manual_seed(sum(lens))
    T, G = sum(lens), hq // hk
    q, k, v = (torch.randn(T, h, D, device="cuda", generator=g).to(BF16) for h in (hq, hk, hk))
    cu = dev(np.concatenate([[0], np.cumsum(lens)]))
    o = sv.prompt_attention(q, k, v, cu)
    at = 0
    for n in lens:
        for h in range(hq):
            for r0 in range(0, n, 4096):
                rows = slice(at + r0, min(at + r0 + 4096, at + n))
                m = rows.stop - at
                Q, K, V = q[rows, h].double(), k[at:at + m, h // G].double(), v[at:at + m, h // G].double()
                z = Q @ K.T * D ** -0.5
                z.masked_fill_(torch.arange(m, device="cuda") > torch.arange(r0, m, device="cuda")[:, None], -math.inf)
                p = z.softmax(-1)
                ref = {"out": p @ V, "lse": z.logsumexp(-1), "room": p @ V.abs(),
                       "zroom": (Q.abs() @ K.abs().T).amax(-1) * D ** -0.5}
                _compare({"out": o["out"][rows, h], "lse": o["lse"][rows, h]},
                         {x: host(y) for x, y in ref.items()}, D)
        at += n
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    out = {x: torch.zeros_like(y) for x, y in o.items()}
    with torch.cuda.stream(st):
        second = sv.prompt_attention(q, k, v, cu)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=st):
            sv.prompt_attention(q, k, v, cu, out=out)
    for _ in range(2):
        out["out"].zero_()
        graph.replay()
        torch.cuda.synchronize()
        for x in o:
            assert torch.equal(second[x], o[x]) and torch.equal(out[x], o[x])
    assert sv.device_error() == 0


def test_two_calls_at_once():
    """On two streams, with different inputs."""
    calls = []
    for i in range(2):
        g = torch.Generator("cuda").manual_seed(i)
        q, k, v = (torch.randn(3000, h, 128, device="cuda", generator=g).to(BF16) for h in (8, 2, 2))
        calls.append((q, k, v, dev([0, 1000 + i, 3000])))
    want = [sv.prompt_attention(*c) for c in calls]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(10):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                got[i].append(sv.prompt_attention(*calls[i]))
    torch.cuda.synchronize()
    for w, outs in zip(want, got):
        assert all(torch.equal(o[x], w[x]) for o in outs for x in w)


def test_without_log_sums_and_nothing_to_do():
    q = torch.randn(5, 2, 64, device="cuda").to(BF16)
    out = {"out": torch.empty_like(q)}
    full = sv.prompt_attention(q, q, q, dev([0, 5]))
    assert torch.equal(sv.prompt_attention(q, q, q, dev([0, 5]), out=out)["out"], full["out"])
    assert sv.prompt_attention(q[:0], q[:0], q[:0], dev([0, 0]))["out"].shape == (0, 2, 64)
    assert sv.prompt_attention(q, q, q, dev([3]))["out"].shape == (5, 2, 64)  # no sequence


@DIMS
def test_output_at_half_a_sector(D):
    """An output that begins 16 bytes behind a line: the same values, and nothing beside them."""
    T, hq, hk = 150, 4, 2
    q, k, v = (torch.randn(T, h, D, device="cuda").to(BF16) for h in (hq, hk, hk))
    cu = dev(np.array([0, 130, 150]))
    want = sv.prompt_attention(q, k, v, cu)
    room = torch.full((T * hq * D + 16,), 7.0, device="cuda", dtype=BF16)
    o = {"out": room[8:-8].view(T, hq, D), "lse": torch.empty((T, hq), device="cuda")}
    sv.prompt_attention(q, k, v, cu, out=o)
    assert torch.equal(o["out"], want["out"]) and torch.equal(o["lse"], want["lse"])
    assert bool((room[:8] == 7).all()) and bool((room[-8:] == 7).all())


@DIMS
@pytest.mark.parametrize("n", [63, 64, 65, 190, 191, 192, 193])
@pytest.mark.parametrize("hq,hk", [(4, 2), (6, 1), (1, 1)])
def test_half_tiles(n, hq, hk, D):
    """Lengths whose last tile of tokens is half seen, in one of a CTA's tiles of rows or in both, with values
    behind them that are not finite."""
    def edit(q, k, v):
        v[n:] = float("nan")
        k[n:] = float("inf")
    _check([n, 70], hq, hk, D, seed=n)
    _check([n], hq, hk, D, seed=n, edit=edit, cu=[0, n], T=n + 80)

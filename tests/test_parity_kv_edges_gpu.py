"""Cache operators at the edges of their definitions: NaN values in prompts of many tiles, signed zeros
and the smallest scales, angles of far positions."""
import math

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from tests.test_parity_kv_gpu import BF16, F32, _check_append, dev, host  # noqa: E402


@pytest.mark.parametrize("news", [[2500, 2300], [250, 640, 129, 510, 700, 384, 260, 255] * 4])
def test_attention_nan_values_in_prompts_of_many_tiles(news):
    """Prompts whose tiles of tokens are nearly all masked for some row, dozens of them in a CTA's run, with
    NaN values in several: the rows that see one are NaN in its 16 values, all others are what they are
    without it, and every call says the same."""
    H, G, D, ps = 2, 2, 128, 32
    g = torch.Generator("cuda").manual_seed(len(news))
    r = np.random.default_rng(len(news))
    T, B, blocks = sum(news), len(news), -(-max(news) // ps)
    table = torch.randperm(B * blocks, device="cuda", generator=g).view(B, blocks)
    cu = np.concatenate([[0], np.cumsum(news)])
    seq = torch.repeat_interleave(torch.arange(B, device="cuda"), torch.tensor(news, device="cuda"))
    at = torch.arange(T, device="cuda") - dev(cu)[seq]
    slots = table[seq, at // ps] * ps + at % ps
    k, v = (torch.randn(T, H, D, device="cuda", generator=g).to(BF16) for _ in "kv")
    cache, clean = (sv.kv4_cache(B * blocks, H, D, ps) for _ in range(2))
    sv.kv4_append(k, v, slots, clean, page_size=ps)
    want = torch.zeros(T, H, D // 16, dtype=torch.bool, device="cuda")
    for b in range(B):
        for _ in range(12):
            t, h, s = int(r.integers(0, news[b])), int(r.integers(H)), int(r.integers(D // 16))
            v[cu[b] + t, h, 16 * s + int(r.integers(16))] = math.nan
            want[cu[b] + t:cu[b + 1], h, s] = True
    sv.kv4_append(k, v, slots, cache, page_size=ps)
    want = want.repeat_interleave(G, 1).repeat_interleave(16, 2)
    assert 0.1 < float(want.float().mean()) < 0.9
    q = torch.randn(T, H * G, D, device="cuda", generator=g).to(BF16)
    lens, cu, table = dev(np.array(news)), dev(cu), table.int()

    def call(c):
        return sv.kv4_attention(q, c, table, lens, cu, page_size=ps, max_new=max(news))
    ref = call(clean)
    for _ in range(20):
        o = call(cache)
        assert torch.equal(o["out"].isnan(), want)
        assert torch.equal(o["out"][~want], ref["out"][~want]) and torch.equal(o["lse"], ref["lse"])
    # the clean call against float64, a few rows of each sequence
    for b in range(min(B, 8)):
        n, c0 = news[b], int(cu[b])
        out = sv.kv4_append(k[c0:c0 + n], v[c0:c0 + n].nan_to_num(0.0), slots[c0:c0 + n],
                            torch.empty_like(clean), page_size=ps, values=True)
        for i in sorted({0, n - 1, *r.integers(0, n, 6).tolist()}):
            for h in range(H * G):
                K, V = out["k"][:i + 1, h // G].double(), out["v"][:i + 1, h // G].double()
                fine = ~want[c0 + i, h]
                p = (K @ q[c0 + i, h].double() * D ** -0.5).softmax(0)
                y = p @ V
                tol = 2.0 ** -8 * y.abs() + (p @ V.abs()) * 2.0 ** -9 + 2.0 ** -32 * V.abs().sum(0)
                assert ((ref["out"][c0 + i, h].double() - y).abs() <= tol)[fine].all()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D", [64, 128])
def test_append_keeps_the_sign_of_zero(dtype, D):
    """-0.0 beside other values has the code of -0, as the quotient -0 / scale has: in pairs of tokens and
    alone, with scales in and out of the range of the quotient's short form, and held at 448."""
    def edit(k, v):
        k[:, :, 1::3] = -0.0
        v[:, :, ::2] = -0.0
        v[:, :, 1::4] = 0.0
        v[5, 0] *= 1e6  # scales held at 448
    slots = [0, 1, 2, 5, 8, 9, 31]
    for gk, gv in ((1.0, 0.5), (2.0 ** -70, 2.0 ** 70)):
        _check_append(len(slots), 2, D, 16, dtype, slots, gk=gk, gv=gv, edit=edit)
    k = torch.full((1, 1, D), -0.0, device="cuda", dtype=dtype)
    k[..., ::16] = 3.0
    out = sv.kv4_append(k, -k, dev([0], torch.int64), sv.kv4_cache(1, 1, D, 16), page_size=16, values=True)
    for n, x in (("k", k), ("v", -k)):
        assert torch.equal(out[n].float(), x.float()) and torch.equal(out[n].signbit(), x.signbit())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_smallest_scales(dtype):
    """Blocks whose scale is one of the smallest, 2^-9 to 2^-6: there the largest value may be almost nine
    times the scale, or nothing is left of the block."""
    r = np.random.default_rng(4)
    most = 6 * 2.0 ** -9 * np.array([0.4, 0.499, 0.501, 0.9, 1.2, 1.49, 1.51, 2.49, 2.51, 3.5, 7.4, 7.9])

    def edit(k, v):
        for x in (k, v):
            y = r.uniform(-1, 1, (len(most), 1, 4, 16)) * most[:, None, None, None]
            y[..., 3] = most[:, None, None]
            x[:] = torch.from_numpy(y.reshape(len(most), 1, 64)).to(x)
    _check_append(len(most), 1, 64, 16, dtype, np.arange(len(most)) + 1, gk=1.0, gv=1.0, edit=edit)


def _inverse_of_two_pi(bits):
    """1 / (2 pi) * 2^bits, from pi = 16 atan(1/5) - 4 atan(1/239) in integers."""
    one = 1 << (bits + 64)

    def atan(n):
        total = term = one // n
        k = 1
        while term:
            term //= -n * n
            k += 2
            total += term // k
        return total
    return (one << bits) // (2 * (16 * atan(5) - 4 * atan(239)))


def _exact_turns(position, freq, bits=256):
    """position * freq / (2 pi), less the nearest whole number of turns."""
    n, d = float(freq).as_integer_ratio()
    x = position * n * _INVERSE // d % (1 << bits)
    return (x - (1 << bits) if x >> (bits - 1) else x) / 2 ** bits


_INVERSE = _inverse_of_two_pi(256)


@pytest.mark.parametrize("offset", [0, 1])  # 1: rows that are not 16-byte aligned, the general kernel
@pytest.mark.parametrize("far", [1 << 16, 1 << 24, (1 << 31) - 1])
def test_angles_of_far_positions(far, offset):
    """Sines next to their zeros show the angle itself: off by at most 2^-32 turns at every position, with
    frequencies above one too."""
    r = np.random.default_rng(far % 1000 + offset)
    T, half, D = 4096, 32, 64
    pos = r.integers(-far, far + 1, T)
    pos[:4] = [far, -far, far - 1, 1]
    freq = np.array([10000.0 ** (-j / 28) for j in range(28)] + [3.7, 123.456, 1e5 / 3, 7e8])
    base = torch.zeros(T, D + offset, device="cuda")
    base[:, offset:offset + half] = 1.0
    q = base[:, offset:].unflatten(1, (1, D))
    o = host(sv.qk_norm_rope(q, None, dev(pos), torch.from_numpy(freq).cuda(), eps=0.0)["q"])[:, 0]
    turns = np.array([[_exact_turns(int(p), f) for f in freq] for p in pos])
    y = math.sqrt(2)
    for x, want in ((o[:, :half], y * np.cos(2 * math.pi * turns)), (o[:, half:], y * np.sin(2 * math.pi * turns))):
        # the norm and the rotation's own roundings as in test_norm_rope; 2^-32 turns of the angle
        tol = np.abs(want) * ((D / 2 + 8) * 2.0 ** -24 + 2.0 ** -23) + y * 2 * math.pi * 2.0 ** -32
        assert (np.abs(x - want) <= tol).all(), (np.abs(x - want) / tol).max()
    assert (np.abs(turns) < 2.0 ** -12).sum() > 10  # places where the sine tells

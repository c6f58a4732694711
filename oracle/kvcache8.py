"""float64 CPU definitions of the 8-bit cache and of packed prompt attention (numpy; test infrastructure).

Written from the definitions in include/spec_kv.h, block by block and row by row; shares no code with
the CUDA path.
"""
from __future__ import annotations

import math

import numpy as np

LOW, HIGH = -60, 121


def exponent(most: float) -> int:
    """The smallest exponent of LOW..HIGH whose 127 steps reach ``most``, or HIGH."""
    for e in range(LOW, HIGH):
        if most <= 127 * 2.0 ** e:
            return e
    return HIGH


def round_even(x):
    """To the nearest integer, ties to even, held at +-127."""
    down = np.floor(x)
    up = (x - down > 0.5) | ((x - down == 0.5) & (down % 2 == 1))
    return np.clip(down + up, -127, 127)


def key_byte(D, i, d):
    """Byte of value d of token i in a block."""
    chunk = d // 16
    if D == 128:
        chunk ^= i % 2
    return i * D + 16 * chunk + d % 16


def value_byte(D, i, d):
    pair, chunk = i // 2, d // 8
    return 16 * D + pair * 2 * D + 16 * (chunk ^ (2 * (pair % 4))) + 2 * (d % 8) + i % 2


def _signed(b):
    return int(b) - 256 if b > 127 else int(b)


class Block:
    """Keys (0) or values (1) of one block: codes [16, D], exponent, marks [16], read from its bytes."""

    def __init__(self, raw, D, which):
        place = value_byte if which else key_byte
        self.at = np.array([[place(D, i, d) for d in range(D)] for i in range(16)])
        self.raw, self.D, self.which = raw, D, which
        self.codes = raw[self.at].astype(np.int64) - 128
        self.e = _signed(raw[32 * D + which])
        bits = int(raw[32 * D + 4 + 2 * which]) | int(raw[32 * D + 5 + 2 * which]) << 8
        self.marks = np.array([bits >> i & 1 for i in range(16)], bool)

    def write(self):
        self.raw[self.at] = (self.codes + 128).astype(np.uint8)
        self.raw[32 * self.D + self.which] = self.e % 256
        bits = sum(1 << i for i in range(16) if self.marks[i])
        self.raw[32 * self.D + 4 + 2 * self.which] = bits & 255
        self.raw[32 * self.D + 5 + 2 * self.which] = bits >> 8

    def values(self):
        v = self.codes * 2.0 ** self.e
        v[self.marks] = np.nan
        return v


def bring(block, places, rows):
    """Rows [n, D] to these places of a block, in memory (``block.write`` stores it)."""
    rows = np.asarray(rows, np.float64)
    bad = ~np.isfinite(rows).all(-1)
    e = exponent(np.abs(rows[~bad]).max(initial=0.0))
    if 0 in places:
        block.codes[:], block.marks[:] = 0, False
    else:
        old = min(max(block.e, LOW), HIGH)
        e = max(e, old)
        if e > old:
            block.codes = round_even(block.codes * 2.0 ** (old - e)).astype(np.int64)
    block.e = e
    for p, row, b in zip(places, rows, bad):
        block.marks[p] = b
        block.codes[p] = 0 if b else round_even(row * 2.0 ** -e)


def append(cache, slots, k, v, page_size):
    """Into the cache bytes (uint8 [pages, heads, bytes]), in place -> the values that they now stand
    for, (keys, values) [T, H, D]."""
    T, H, D = np.shape(k)
    P, size = cache.shape[0], 32 * D + 16
    blocks = {}  # block of a page -> tokens; a token that is not written is alone
    for t, s in enumerate(slots):
        inside = 0 <= s < P * page_size
        blocks.setdefault(int(s) // 16 if inside else ("alone", t), []).append(t)
    out = np.zeros((2, T, H, D))
    for name, tokens in blocks.items():
        for h in range(H):
            if isinstance(name, tuple):
                raw, places = np.full(size, 128, np.uint8), [0]
            else:
                page, j = divmod(name, page_size // 16)
                raw = cache[page, h, j * size:(j + 1) * size]
                places = [int(slots[t]) % 16 for t in tokens]
            for which, x in enumerate((k, v)):
                b = Block(raw, D, which)
                bring(b, places, np.asarray(x)[tokens, h])
                b.write()
                out[which, tokens, h] = b.values()[places]
    return out


def read_head(cache, pages, length, head, page_size, D):
    """Keys, values [length, D] and the values' exponents [length] of the sequence whose blocks are
    ``pages``. A page outside the cache reads as NaN."""
    size = 32 * D + 16
    K, V, E = np.full((length, D), np.nan), np.full((length, D), np.nan), np.zeros(length, int)
    for t in range(0, length, 16):
        page, n = int(pages[t // page_size]), min(16, length - t)
        if not 0 <= page < cache.shape[0]:
            continue
        j = t % page_size // 16
        raw = cache[page, head, j * size:(j + 1) * size]
        keys, values = Block(raw, D, 0), Block(raw, D, 1)
        K[t:t + n], V[t:t + n], E[t:t + n] = keys.values()[:n], values.values()[:n], values.e
    return K, V, E


def rows_attention(q, K, V, seen, scale, E=None):
    """q [n, D], row i over the first seen[i] tokens -> dict of out [n, D], lse [n], and for error bounds
    room = sum p |v|, vsum = (largest p 2^E) sum |v| 2^-E, zroom = the largest sum |q k| * scale."""
    n, D = q.shape
    E = np.zeros(len(K)) if E is None else E
    o = {"out": np.zeros((n, D)), "lse": np.full(n, -math.inf), "room": np.zeros((n, D)),
         "vsum": np.zeros((n, D)), "zroom": np.zeros(n)}
    for i in range(n):
        k, v, two = K[:seen[i]], V[:seen[i]], 2.0 ** E[:seen[i]]
        if not seen[i]:
            continue
        with np.errstate(invalid="ignore"):
            z = k @ q[i] * scale
            m = z.max()
            p = np.exp(z - m)
            o["lse"][i] = m + math.log(p.sum()) if p.sum() > 0 else math.nan
            p = p / p.sum()
            o["out"][i] = p @ v
            o["room"][i] = p @ np.abs(v)
            o["vsum"][i] = (p * two).max() * (np.abs(v) / two[:, None]).sum(0)
            o["zroom"][i] = (np.abs(k) @ np.abs(q[i])).max() * abs(scale)
    return o


def attention(q, cache, block_table, kv_lens, cu_new, page_size, scale):
    """q [T, Hq, D] -> the dict of ``rows_attention`` with a dimension of heads. Rows of no sequence
    are NaN in ``out`` and ``lse``."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    H, most = cache.shape[1], block_table.shape[1] * page_size
    res = {"out": np.full(q.shape, np.nan), "lse": np.full((T, Hq), np.nan), "room": np.zeros(q.shape),
           "vsum": np.zeros(q.shape), "zroom": np.zeros((T, Hq)), "emost": np.zeros((T, Hq))}
    for b in range(len(kv_lens)):
        r0, r1 = int(cu_new[b]), int(cu_new[b + 1])
        n, L = r1 - r0, min(max(int(kv_lens[b]), 0), most)
        seen = [max(0, min(L, L - n + i + 1)) for i in range(n)]
        for h in range(Hq if n else 0):
            K, V, E = read_head(cache, block_table[b], L, h * H // Hq, page_size, D)
            for name, x in rows_attention(q[r0:r1, h], K, V, seen, scale, E).items():
                res[name][r0:r1, h] = x
            res["emost"][r0:r1, h] = np.abs(E).max(initial=0)
    return res


def prompt_attention(q, k, v, cu, scale):
    """q [T, Hq, D], k, v [T, Hkv, D] -> the dict of ``rows_attention`` with a dimension of heads; rows
    of no sequence are NaN in ``out`` and ``lse``."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    res = {"out": np.full(q.shape, np.nan), "lse": np.full((T, Hq), np.nan), "room": np.zeros(q.shape),
           "vsum": np.zeros(q.shape), "zroom": np.zeros((T, Hq))}
    for a, b in zip(cu[:-1], cu[1:]):
        a, b = int(a), int(b)
        for h in range(Hq):
            o = rows_attention(q[a:b, h], k[a:b, h // G], v[a:b, h // G], range(1, b - a + 1), scale)
            for name, x in o.items():
                res[name][a:b, h] = x
    return res

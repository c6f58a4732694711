"""float64 CPU definitions of the paged key/value cache operators (numpy; test infrastructure).

Written from the definitions in include/spec_kv.h, sequence by sequence and token by token; shares
no code with the CUDA path. Arithmetic is in float64 except where the definition itself names
float32 (the append's block scale and quotient).
"""
from __future__ import annotations

import math

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])


def e4m3_value(byte: int) -> float:
    """Value of an e4m3 byte: sign, 4 exponent bits (bias 7), 3 mantissa bits; no infinities."""
    s, e, m = byte >> 7, (byte >> 3) & 15, byte & 7
    if e == 15 and m == 7:
        return math.nan
    v = m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
    return -v if s else v


E4M3 = np.array([e4m3_value(b) for b in range(256)])


def nearest_even(x: float, grid: np.ndarray) -> int:
    """Index of the value of the ascending ``grid`` nearest to x >= 0; a tie goes to the even
    index, what lies above the last value to the last one."""
    if x >= grid[-1]:
        return len(grid) - 1
    hi = int(np.searchsorted(grid, x, side="right"))
    lo = hi - 1
    a, b = x - grid[lo], grid[hi] - x
    return hi if b < a or (a == b and hi % 2 == 0) else lo


# ------------------------------------------------------------------------------ block tables
def block_tables(ctx_lens, accept_len, new_lens, block_table, held, ring, counters, page_size,
                 max_tokens):
    """Sequence by sequence, in ascending order. Returns a dict; the inputs are left alone."""
    B, most = np.shape(block_table)
    table, ring = np.array(block_table), np.array(ring)
    cap = len(ring)
    head, tail = int(counters[0]), int(counters[1])
    live = min(max(tail - head, 0), cap)
    asked = taken = back = tokens = placed = 0
    r = {k: [] for k in ("ctx_lens", "held", "kv_lens", "status")}
    cu, slots, positions, seq_ids = [0], [], [], []
    freed = []
    for b in range(B):
        ctx, h = int(ctx_lens[b]), int(held[b])
        a = -1 if accept_len is None else int(accept_len[b])
        done = new_lens[b] < 0
        c = 0 if done else ctx + (a + 1 if a >= 0 else 0)
        n = max(int(new_lens[b]), 0)
        need = -(-(c + n) // page_size)
        status, now = None, need
        if not 0 <= h <= most or (not done and (ctx < 0 or c > h * page_size or need > most)):
            status, now, n, c = -2, h, 0, ctx
        elif need > h:
            asked += need - h
            if asked > live:
                status, now, n = -1, h, 0
            else:
                for j in range(h, need):
                    table[b, j] = ring[(head + taken) % cap]
                    taken += 1
        elif need < h:
            for j in range(need, h):
                freed.append((tail + back, table[b, j]))
                back += 1
        if n > 0:
            tokens += n
            if tokens > max_tokens:
                status, n = -3, 0
        for i in range(n):
            p = c + i
            page = int(table[b, p // page_size])
            slots.append(-1 if page < 0 else page * page_size + p % page_size)
            positions.append(p)
            seq_ids.append(b)
        placed += n
        cu.append(placed)
        r["ctx_lens"].append(c)
        r["held"].append(now)
        r["kv_lens"].append(c + n)
        r["status"].append(status if status is not None else int(n > 0))
    for at, page in freed:
        ring[at % cap] = page
    pad = max_tokens - placed
    r.update(counters=[head + taken, tail + back], cu_new=cu, slots=slots + [-1] * pad,
             positions=positions + [0] * pad, seq_ids=seq_ids + [-1] * pad, block_table=table,
             ring=ring)
    return {k: np.array(v) for k, v in r.items()}


# ------------------------------------------------------------------------------ norm, rotation
def qk_norm_rope(x, positions, inv_freq, weight, eps, interleaved):
    """x [T, H, D] -> (y [T, H, D], room [T, H, D]): y in float64, and the sum of the magnitudes
    that enter each value (what rounding errors scale with)."""
    x = np.asarray(x, np.float64)
    T, H, D = x.shape
    half = len(inv_freq)
    y = x / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    if weight is not None:
        y = y * np.asarray(weight, np.float64)
    out, room = y.copy(), np.abs(y)
    for j in range(half):
        i0, i1 = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        angle = np.asarray(positions, np.float64)[:, None] * float(inv_freq[j])
        c, s = np.cos(angle), np.sin(angle)
        out[..., i0] = y[..., i0] * c - y[..., i1] * s
        out[..., i1] = y[..., i1] * c + y[..., i0] * s
        room[..., i0] = room[..., i1] = np.abs(y[..., i0]) + np.abs(y[..., i1])
    return out, room


# ------------------------------------------------------------------------------ 4-bit cache
def quantise16(x, g):
    """16 float32 values -> (codes [16], scale byte)."""
    x = np.asarray(x, np.float32)
    if not np.isfinite(x).all():
        return np.zeros(16, np.int64), 0x7F
    with np.errstate(over="ignore"):
        m = np.float32(np.abs(x).max()) * np.float32(1.0 / (6.0 * float(np.float32(g))))
    scale = nearest_even(float(m), E4M3[:127])
    s = np.float32(E4M3[scale]) * np.float32(g)
    if not s > 0:
        return np.zeros(16, np.int64), scale
    with np.errstate(over="ignore"):
        t = np.abs(x) / s
    codes = np.array([nearest_even(float(v), E2M1) for v in t])
    return codes + 8 * np.signbit(x), scale


def code_value(code, scale, g):
    v = E2M1[np.asarray(code) & 7] * E4M3[scale] * float(g)
    return np.where(np.asarray(code) & 8, -v, v)


def value_place(D, pair, d):
    """Byte of value d among the D code bytes of a token pair."""
    w = D // 8
    g = d // w
    g ^= 2 * (pair % 4) if D == 128 else 4 * (pair // 2 % 2)
    return g * w + d % w


def _block(cache, slot, head, page_size, D):
    page, at = divmod(int(slot), page_size)
    start = at // 16 * 18 * D
    return cache[page, head, start:start + 18 * D], at % 16


def put_token(cache, slot, head, page_size, D, k, v, gk, gv):
    """Write one token of one head into the cache bytes (uint8 [pages, heads, bytes])."""
    blk, i = _block(cache, slot, head, page_size, D)
    S, p, odd = D // 16, i // 2, i % 2
    for s in range(S):
        codes, scale = quantise16(k[16 * s:16 * s + 16], gk)
        blk[8 * D + i * S + s] = scale
        for j in range(8):
            blk[i * (D // 2) + 8 * s + j] = codes[2 * j] | codes[2 * j + 1] << 4
        codes, scale = quantise16(v[16 * s:16 * s + 16], gv)
        blk[17 * D + (p * S + s) * 2 + odd] = scale
        for j in range(16):
            at = 9 * D + p * D + value_place(D, p, 16 * s + j)
            keep = blk[at] & (0x0F if odd else 0xF0)
            blk[at] = keep | codes[j] << (4 if odd else 0)


def read_head(cache, pages, length, head, page_size, D, gk, gv):
    """Keys and values [length, D] in float64 of the sequence whose blocks are ``pages``. A page
    outside the cache reads as NaN."""
    S = D // 16
    d = np.arange(D)
    K, V = np.full((length, D), np.nan), np.full((length, D), np.nan)
    place = np.array([[value_place(D, p, x) for x in range(D)] for p in range(8)])
    for t in range(length):
        page = int(pages[t // page_size])
        if not 0 <= page < cache.shape[0]:
            continue
        blk, i = _block(cache, page * page_size + t % page_size, head, page_size, D)
        p, odd = i // 2, i % 2
        kc = blk[i * (D // 2) + d // 2].astype(np.int64) >> (4 * (d % 2)) & 15
        vc = blk[9 * D + p * D + place[p]].astype(np.int64) >> (4 * odd) & 15
        K[t] = code_value(kc, blk[8 * D + i * S + d // 16], gk)
        V[t] = code_value(vc, blk[17 * D + (p * S + d // 16) * 2 + odd], gv)
    return K, V


# ------------------------------------------------------------------------------ attention
def attention(q, cache, block_table, kv_lens, cu_new, page_size, scale, gk, gv):
    """q [T, Hq, D] -> dict of out [T, Hq, D], lse [T, Hq], and for error bounds room [T, Hq, D]
    = sum p |v|, vsum [T, Hq, D] = sum |v| and zroom [T, Hq] = the largest sum |q k| * scale of a
    token seen. Rows of no sequence are NaN in ``out`` and ``lse``."""
    q = np.asarray(q, np.float64)
    T, Hq, D = q.shape
    H, most = cache.shape[1], block_table.shape[1] * page_size
    G = Hq // H
    out, lse = np.full(q.shape, np.nan), np.full((T, Hq), np.nan)
    room, vsum, zroom = np.zeros(q.shape), np.zeros(q.shape), np.zeros((T, Hq))
    for b in range(len(kv_lens)):
        r0, r1 = int(cu_new[b]), int(cu_new[b + 1])
        n, L = r1 - r0, min(max(int(kv_lens[b]), 0), most)
        for hk in range(H):
            K, V = read_head(cache, block_table[b], L, hk, page_size, D, gk, gv) if n else (0, 0)
            for i in range(n):
                seen = max(0, min(L, L - n + i + 1))
                for h in range(hk * G, hk * G + G):
                    row = r0 + i
                    z = K[:seen] @ q[row, h] * scale
                    if not seen or (np.isneginf(z)).all():
                        out[row, h], lse[row, h] = 0.0, -math.inf
                        continue
                    with np.errstate(invalid="ignore"):
                        m = z.max()
                        p = np.exp(z - m)
                        out[row, h] = p @ V[:seen] / p.sum()
                        lse[row, h] = m + math.log(p.sum()) if p.sum() > 0 else math.nan
                        room[row, h] = p @ np.abs(V[:seen]) / p.sum()
                        vsum[row, h] = np.abs(V[:seen]).sum(0)
                        zroom[row, h] = (np.abs(K[:seen]) @ np.abs(q[row, h])).max() * abs(scale)
    return {"out": out, "lse": lse, "room": room, "vsum": vsum, "zroom": zroom}

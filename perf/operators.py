"""Measured cases of the key/value-cache operators around the verify step.

Four operators carry a draft-and-verify round of a target model up to its logits:

- ``tables``: page allocation, rollback and slot maps of a paged cache, from request lengths;
- ``norm_rope``: root-mean-square norms of queries and keys per head, and the position rotation;
- ``append``: keys and values written into the paged cache in 4 bits (e2m1 codes, an e4m3 scale
  for each 16 values);
- ``attend``: causal attention of each sequence's new tokens over that cache.

``own`` chooses between the plain form (elementary torch operations) and the library's calls. Both
read the same cache bytes; the layout of a block of 16 tokens of one head, D values a token, is

    key codes    [16 tokens][D / 2]      byte j: value 2j in the low four bits, 2j + 1 in the high
    key scales   [16 tokens][D / 16]     e4m3
    value codes  [8 token pairs][D]      one byte a value: the even token low, the odd token high;
                                         the D bytes of pair p lie in 8 chunks, chunk g at place
                                         g ^ 2 (p % 4) for D = 128 and g ^ 4 (p / 2 % 2) for D = 64
    value scales [8 token pairs][D / 16][2]

and a page holds, head by head, its page_size / 16 blocks. A stored value is code * scale * (the
tensor's scale).
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
E2M1 = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
HEADS = ((32, 8, 128), (28, 4, 128), (16, 2, 64), (8, 1, 64), (8, 8, 128), (12, 12, 64))
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # a small server's round: every request brings a draft of up to 5 tokens
        {"name": "tables_b8", "op": "tables", "B": 8, "ps": 64, "ctx": 2000, "n": 6, "prompts": 0},
        # a large batch's verify round, after the outcome of the last one
        {"name": "tables_b1024", "op": "tables", "B": 1024, "ps": 16, "ctx": 8192, "n": 9,
         "prompts": 0},
        # admission: part of the batch brings whole prompts
        {"name": "tables_prompts", "op": "tables", "B": 256, "ps": 32, "ctx": 4096, "n": 9,
         "prompts": 16384},
        # decoding, 8 requests, one token each, heads of a 4096-wide model
        {"name": "norm_rope_t8", "op": "norm_rope", "T": 8, "hq": 32, "hkv": 8, "D": 128,
         "rot": 128, "inter": False, "dtype": "bf16", "far": 100000},
        # verify rows of 256 ragged drafts in float32, interleaved pairs, half of each head rotated
        {"name": "norm_rope_f32", "op": "norm_rope", "T": 1153, "hq": 16, "hkv": 2, "D": 64,
         "rot": 32, "inter": True, "dtype": "f32", "far": 1000000},
        # a prompt of 32k tokens, heads of a 3584-wide model
        {"name": "norm_rope_prompt", "op": "norm_rope", "T": 32767, "hq": 28, "hkv": 4, "D": 128,
         "rot": 128, "inter": False, "dtype": "bf16", "far": 40000},
        # verify rows of 64 drafts of 5
        {"name": "append_verify", "op": "append", "B": 64, "n": 6, "ps": 64, "hkv": 8, "D": 128,
         "dtype": "bf16"},
        # prompts of some thousand tokens
        {"name": "append_prompt", "op": "append", "B": 13, "n": 5001, "ps": 32, "hkv": 8, "D": 128,
         "dtype": "bf16"},
        # one request, one token, 4k behind it: latency
        {"name": "attend_b1", "op": "attend", "B": 1, "n": 1, "ctx": 4097, "ps": 64, "hq": 32,
         "hkv": 8, "D": 128, "ragged": False},
        # one request far into a long document, drafts of 4
        {"name": "attend_long", "op": "attend", "B": 1, "n": 5, "ctx": 524301, "ps": 128, "hq": 32,
         "hkv": 8, "D": 128, "ragged": False},
        # 64 requests, drafts of up to 5, lengths up to 8k
        {"name": "attend_b64", "op": "attend", "B": 64, "n": 6, "ctx": 8192, "ps": 32, "hq": 32,
         "hkv": 8, "D": 128, "ragged": True},
        # 256 requests, drafts of up to 8, lengths up to 8k: many rows on each cached head
        {"name": "attend_b256", "op": "attend", "B": 256, "n": 9, "ctx": 8192, "ps": 16, "hq": 28,
         "hkv": 4, "D": 128, "ragged": True},
    ]


def _log(rng, lo, hi):
    v = min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))
    return v + 1 if v == 3072 else v


def draw(rng):
    op = rng.choice(("tables", "norm_rope", "append", "attend", "attend"))
    ps = rng.choice((16, 32, 64, 128))
    if op == "tables":
        prompts = rng.choice((0, 0, _log(rng, 64, 16384)))
        B = _log(rng, 1, 1024 if not prompts else 200)
        return {"op": op, "B": B, "ps": ps, "ctx": _log(rng, 16, 8192), "n": rng.randint(1, 9),
                "prompts": prompts}
    hq, hkv, D = rng.choice(HEADS)
    if op == "norm_rope":
        rot = rng.choice((D, D, D // 2, D // 4))
        dt = rng.choice(("bf16", "bf16", "f32"))
        T = _log(rng, 1, 32000 * 32 // (hq + hkv) if dt == "bf16" else 12000)
        return {"op": op, "T": T, "hq": hq, "hkv": hkv, "D": D, "rot": rot,
                "inter": rng.random() < 0.3, "dtype": dt, "far": _log(rng, 100, 1000000)}
    if op == "append":
        B = _log(rng, 1, 256)
        n = rng.choice((rng.randint(1, 9), _log(rng, 10, 8191)))
        n = max(1, min(n, 60000 // B))
        n = n + 1 if n == 3072 else n
        return {"op": op, "B": B, "n": n, "ps": ps, "hkv": hkv, "D": D,
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
    n = rng.choice((1, rng.randint(2, 9), rng.randint(2, 9), rng.randint(10, 64)))
    B = _log(rng, 1, 256 if n < 10 else 16)
    most = min(262144, 4_000_000 // (B * hkv), 100_000_000 // (B * hq * n))
    ctx = _log(rng, 1, max(2, most))
    return {"op": op, "B": B, "n": n, "ctx": max(n, ctx), "ps": ps, "hq": hq, "hkv": hkv, "D": D,
            "ragged": rng.random() < 0.6}


# ---------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------
def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    return g


def _news(case):
    """New tokens of the sequences of a case, in no order yet: the same for every seed, so that
    outputs keep their shapes."""
    B, n = case["B"], case["n"]
    r = np.random.default_rng([B, n])
    if case["op"] == "attend":
        return r.integers(max(1, min(2, n)), n + 1, B) if case["ragged"] else np.full(B, n)
    new = r.integers(1, n + 1, B)
    fresh = r.random(B) < (0.5 if case["prompts"] else 0.02)  # admitted now: nothing cached yet
    if case["prompts"]:
        long = np.exp(r.uniform(math.log(16), math.log(case["prompts"]), B)).astype(np.int64) + 1
        new = np.where(fresh, long, new)
    new[(r.random(B) < 0.03) & ~fresh] = 0    # waits this round
    new[(r.random(B) < 0.03) & ~fresh] = -1   # finished: gives its pages back
    return np.stack([new, fresh], 1)


def _lens(case, seed):
    """Host-side lengths of a case: (new tokens, tokens in the cache with them) per sequence."""
    r = np.random.default_rng([seed, 7])
    B, ctx = case["B"], case["ctx"]
    news = r.permutation(_news(case))
    if not case["ragged"]:
        return news, np.full(B, ctx)
    lens = np.exp(r.uniform(math.log(max(1, ctx // 16)), math.log(ctx), B)).astype(np.int64)
    lens[r.integers(B)] = ctx
    return news, np.maximum(news, lens)


def _prep_tables(case, seed):
    r = np.random.default_rng([seed, 1])
    B, ps, n = case["B"], case["ps"], case["n"]
    new, fresh = r.permutation(_news(case)).T
    ctx = np.maximum(1, np.exp(r.uniform(math.log(max(1, case["ctx"] // 16)), math.log(case["ctx"]), B))).astype(np.int64)
    last = r.integers(1, n + 1, B)           # tokens of the last round
    acc = r.integers(0, n, B) % last         # its accepted drafts
    held = -(-(ctx + last) // ps)
    fresh = fresh > 0
    ctx[fresh], held[fresh], acc[fresh] = 0, 0, -1
    most = -(-(max(case["ctx"], case["prompts"] + 1) + 2 * n) // ps)
    grown = np.maximum(0, -(-(ctx + acc + 1 + np.maximum(new, 0)) // ps) - held)
    used, spare = int(held.sum()), int(grown.sum()) + 8
    ring = np.full(B * most + 8, -1, np.int32)
    pages = r.permutation(ring.size)[:used + spare]
    table = np.full((B, most), -1, np.int32)
    table[np.arange(most)[None, :] < held[:, None]] = pages[:used]
    head = int(r.integers(0, 2 * ring.size))
    ring[(head + np.arange(spare)) % ring.size] = pages[used:]
    cap = int(np.maximum(new, 0).sum()) + 5

    def dev(a, t=torch.int32):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, t)
    i32 = {"dtype": torch.int32, "device": DEV}
    out = {"ctx_lens": torch.empty(B, **i32), "held": torch.empty(B, **i32),
           "counters": torch.empty(2, dtype=torch.int64, device=DEV),
           "cu_new": torch.empty(B + 1, **i32), "kv_lens": torch.empty(B, **i32),
           "status": torch.empty(B, **i32),
           "slots": torch.empty(cap, dtype=torch.int64, device=DEV),
           "positions": torch.empty(cap, **i32), "seq_ids": torch.empty(cap, **i32)}
    return {"op": "tables", "ctx": dev(ctx), "acc": dev(acc), "new": dev(new), "held": dev(held),
            "table": dev(table), "ring": dev(ring), "counters": dev([head, head + spare], torch.int64),
            "ps": ps, "cap": cap, "out": out}


def _prep_norm_rope(case, seed):
    g = _gen(seed)
    T, hq, hkv, D = case["T"], case["hq"], case["hkv"], case["D"]
    dt = DT[case["dtype"]]
    # the projection's output: queries, keys and values of a token side by side
    qkv = torch.randn(T, (hq + 2 * hkv) * D, device=DEV, generator=g)
    qkv *= torch.exp(torch.randn(T, 1, device=DEV, generator=g) * 0.5)
    qkv = qkv.to(dt)
    q = qkv[:, :hq * D].view(T, hq, D)
    k = qkv[:, hq * D:(hq + hkv) * D].view(T, hkv, D)
    pos = torch.randint(0, case["far"], (T,), device=DEV, generator=g, dtype=torch.int32)
    half = case["rot"] // 2
    freq = torch.tensor([10000.0 ** (-i / half) for i in range(half)], dtype=torch.float64, device=DEV)
    w = [(1 + 0.2 * torch.randn(D, device=DEV, generator=g)).to(dt) for _ in range(2)]
    return {"op": "norm_rope", "q": q, "k": k, "pos": pos, "freq": freq, "wq": w[0], "wk": w[1],
            "eps": 1e-6, "inter": case["inter"],
            "out": {"q": torch.empty(T, hq, D, dtype=dt, device=DEV),
                    "k": torch.empty(T, hkv, D, dtype=dt, device=DEV)}}


def _block_bytes(D):
    return 16 * (D + D // 8)


def _prep_append(case, seed):
    g = _gen(seed)
    B, n, ps, H, D = case["B"], case["n"], case["ps"], case["hkv"], case["D"]
    dt = DT[case["dtype"]]
    r = np.random.default_rng([seed, 2])
    start = r.integers(0, 4 * ps, B)  # tokens that the sequence has already
    blocks = -(-(4 * ps + n) // ps)
    pages = r.permutation(B * blocks + 3)[:B * blocks].reshape(B, blocks)
    at = start[:, None] + np.arange(n)[None, :]
    slots = (pages[np.arange(B)[:, None], at // ps] * ps + at % ps).reshape(-1)
    T = B * n
    k = torch.randn(T, H, D, device=DEV, generator=g).to(dt)
    v = (torch.randn(T, H, D, device=DEV, generator=g)
         * torch.exp(torch.randn(T, H, 1, device=DEV, generator=g))).to(dt)
    cache = torch.zeros(B * blocks + 3, H, ps // 16 * _block_bytes(D), dtype=torch.uint8, device=DEV)
    return {"op": "append", "k": k, "v": v, "slots": torch.from_numpy(slots).to(DEV),
            "cache": cache, "ps": ps, "ks": 1.0, "vs": 0.5,
            "out": {"k": torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV),
                    "v": torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)}}


def _prep_attend(case, seed):
    g = _gen(seed)
    B, ps, hq, H, D = case["B"], case["ps"], case["hq"], case["hkv"], case["D"]
    news, lens = _lens(case, seed)
    r = np.random.default_rng([seed, 3])
    held = -(-lens // ps)
    P = int(held.sum()) + 5
    pages = r.permutation(P)
    most = int(held.max()) + 1
    table = np.full((B, most), -1, np.int32)
    table[np.arange(most)[None, :] < held[:, None]] = pages[:P - 5]
    cache = torch.empty(P, H, ps // 16 * _block_bytes(D), dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (H * ps * D))
    ch = torch.exp(0.5 * torch.randn(2, H, 1, D, device=DEV, generator=g))  # channels differ
    for p in range(0, P, step):  # pages of quantised keys and values
        m = min(step, P - p)
        x = torch.randn(2, m, H, ps, D, device=DEV, generator=g) * ch[:, None]
        _encode_pages(x[0], x[1], cache[p:p + m])
    T = int(news.sum())
    q = (1.5 * torch.randn(T, hq, D, device=DEV, generator=g)).to(torch.bfloat16)
    cu = np.concatenate([[0], np.cumsum(news)])

    def dev(a):
        return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, torch.int32)
    return {"op": "attend", "q": q, "cache": cache, "table": dev(table), "lens": dev(lens),
            "cu": dev(cu), "ps": ps, "scale": 1 / math.sqrt(D), "ks": 1.0, "vs": 0.5,
            "most_new": int(news.max()), "most_len": int(lens.max()),
            "out": {"out": torch.empty_like(q),
                    "lse": torch.empty(T, hq, dtype=torch.float32, device=DEV)}}


def prepare(case, seed):
    return {"tables": _prep_tables, "norm_rope": _prep_norm_rope, "append": _prep_append,
            "attend": _prep_attend}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------
# the 4-bit format, in elementary operations
# ---------------------------------------------------------------------------------------------
def _quantise(x, g):
    """x [..., D] in float32 -> (codes 0..15 [..., D], scales e4m3 [..., D / 16], values)."""
    b = x.unflatten(-1, (-1, 16))
    most = b.abs().amax(-1)
    most = torch.where(torch.isfinite(b).all(-1), most, torch.full_like(most, math.nan))
    s8 = (most * (1 / (6 * g))).clamp(max=448).to(torch.float8_e4m3fn)
    s = (s8.float() * g).unsqueeze(-1)
    t = torch.where(s > 0, b.abs() / s, torch.zeros_like(b))
    # nearest, ties to the even code: the codes stand for 0, 1/2, 1, 3/2, 2, 3, 4, 6
    c = ((t > 0.25).byte() + (t >= 0.75).byte() + (t > 1.25).byte() + (t >= 1.75).byte()
         + (t > 2.5).byte() + (t >= 3.5).byte() + (t > 5).byte())
    neg = (torch.signbit(b) & (s > 0)).byte()
    mag = torch.tensor(E2M1, device=x.device)[c.int()]
    val = torch.where(neg > 0, -mag, mag) * s
    return (c + 8 * neg).flatten(-2), s8.view(torch.uint8), val.flatten(-2)


def _places(D):
    """Byte of value d of pair p among the D bytes of the pair: [8, D]."""
    p, d = torch.arange(8, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    w = D // 8
    swap = 2 * (p % 4) if D == 128 else 4 * (p // 2 % 2)
    return ((d // w) ^ swap) * w + d % w


def _encode_pages(k, v, to):
    """Whole pages [m, H, ps, D] of keys and values into the bytes `to` [m, H, bytes]."""
    m, H, ps, D = k.shape
    nb, s = ps // 16, D // 16
    to = to.view(m, H, nb, _block_bytes(D))
    c, s8, _ = _quantise(k, 1.0)
    c = c.view(m, H, nb, 16, D // 2, 2)
    to[..., :8 * D] = (c[..., 0] + 16 * c[..., 1]).flatten(-2)
    to[..., 8 * D:9 * D] = s8.view(m, H, nb, 16 * s)
    c, s8, _ = _quantise(v, 0.5)
    c = c.view(m, H, nb, 8, 2, D)
    both = c[..., 0, :] + 16 * c[..., 1, :]
    place = _places(D).expand(m, H, nb, 8, D)
    to[..., 9 * D:17 * D] = torch.empty_like(both).scatter_(-1, place, both).flatten(-2)
    to[..., 17 * D:] = s8.view(m, H, nb, 8, 2, s).transpose(-1, -2).flatten(-3)


def _decode(raw, D, ks, vs):
    """Blocks [..., bytes] -> keys and values [..., 16, D] in float32."""
    one = torch.tensor(E2M1 + tuple(-x for x in E2M1), device=raw.device)
    two = torch.stack([one.repeat(16), one.repeat_interleave(16)], -1)  # byte -> its two values
    s = D // 16

    def scales(b):
        return b.contiguous().view(torch.float8_e4m3fn).float()
    k = two[raw[..., :8 * D].int()].unflatten(-2, (16, s, 8)).flatten(-2)
    k = k * (scales(raw[..., 8 * D:9 * D]) * ks).unflatten(-1, (16, s)).unsqueeze(-1)
    b = raw[..., 9 * D:17 * D].unflatten(-1, (8, D))
    b = torch.gather(b, -1, _places(D).expand(b.shape))
    v = two[b.int()].transpose(-1, -2).unflatten(-1, (s, 16))  # [..., 8, 2, s, 16]
    sv = (scales(raw[..., 17 * D:]) * vs).unflatten(-1, (8, s, 2)).transpose(-1, -2)
    v = v * sv.unsqueeze(-1)
    return k.flatten(-2), v.flatten(-2).flatten(-3, -2)


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _plain_tables(s):
    ps, cap, table, ring = s["ps"], s["cap"], s["table"], s["ring"]
    B, most = table.shape
    ctx, acc, new, held = s["ctx"].long(), s["acc"].long(), s["new"].long(), s["held"].long()
    head, tail = s["counters"][0], s["counters"][1]
    zero = torch.zeros_like(ctx)
    done = new < 0
    c = torch.where(done, zero, ctx + torch.where(acc >= 0, acc + 1, zero))
    n = new.clamp(min=0)
    need = (c + n + ps - 1) // ps
    bad = (held < 0) | (held > most) | (~done & ((ctx < 0) | (c > held * ps) | (need > most)))
    grow = torch.where(bad, zero, (need - held).clamp(min=0))
    grown = grow.cumsum(0)
    short = (grow > 0) & (grown > tail - head)
    n1 = torch.where(bad | short, zero, n)
    full = (n1 > 0) & (n1.cumsum(0) > cap)
    n2 = torch.where(full, zero, n1)
    c = torch.where(bad, ctx, c)
    now = torch.where(bad | short, held, need)
    cu = torch.cat([zero[:1], n2.cumsum(0)])
    shrink = (held - now).clamp(min=0)
    got = torch.where(short, zero, grow).sum()
    col = torch.arange(most, device=table.device)[None, :]
    take = (head + (grown - grow)[:, None] + col - held[:, None]) % ring.numel()
    fresh = (col >= held[:, None]) & (col < now[:, None])
    table2 = torch.where(fresh, ring[take], table)
    back = (col >= now[:, None]) & (col < held[:, None])
    put = (tail + (shrink.cumsum(0) - shrink)[:, None] + col - now[:, None]) % ring.numel()
    put = torch.where(back, put, torch.full_like(put, ring.numel()))
    ring2 = torch.cat([ring, ring[:1]]).scatter_(0, put.flatten(), table.flatten())[:-1]
    status = torch.where(bad, -2, torch.where(short, -1, torch.where(full, -3, (n2 > 0).long())))
    t = torch.arange(cap, device=table.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    valid = seq < B
    b = seq.clamp(max=B - 1)
    pos = torch.where(valid, c[b] + t - cu[b], torch.zeros_like(t))
    slot = table2[b, (pos // ps).clamp(max=most - 1)].long() * ps + pos % ps
    i32 = torch.int32
    return {"table": table2, "ring": ring2, "ctx_lens": c.to(i32), "held": now.to(i32),
            "counters": torch.stack([head + got, tail + shrink.sum()]), "cu_new": cu.to(i32),
            "kv_lens": (c + n2).to(i32), "status": status.to(i32),
            "slots": torch.where(valid, slot, -1), "positions": pos.to(i32),
            "seq_ids": torch.where(valid, seq, -1).to(i32)}


def _plain_norm_rope(s):
    rot = 2 * s["freq"].numel()
    angle = s["pos"].double()[:, None] * s["freq"]
    cos, sin = angle.cos().float()[:, None], angle.sin().float()[:, None]

    def one(x, w):
        y = x.float()
        y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + s["eps"]) * w.float()
        r = y[..., :rot]
        if s["inter"]:
            a, b = r[..., 0::2], r[..., 1::2]
            r = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
        else:
            a, b = r[..., :rot // 2], r[..., rot // 2:]
            r = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
        return torch.cat([r, y[..., rot:]], -1).to(x.dtype)
    return {"q": one(s["q"], s["wq"]), "k": one(s["k"], s["wk"])}


def _plain_append(s):
    k, v, cache, ps = s["k"].float(), s["v"].float(), s["cache"], s["ps"]
    T, H, D = k.shape
    P, nb, sb = cache.shape[0], ps // 16, D // 16
    slots = s["slots"]
    page, blk, i = slots // ps, slots % ps // 16, slots % 16
    whole = cache.view(P, H, nb, _block_bytes(D))
    kc, ks8, kval = _quantise(k, s["ks"])
    kc = kc.unflatten(-1, (-1, 2))
    whole[..., :8 * D].view(P, H, nb, 16, D // 2)[page, :, blk, i] = kc[..., 0] + 16 * kc[..., 1]
    whole[..., 8 * D:9 * D].view(P, H, nb, 16, sb)[page, :, blk, i] = ks8
    vc, vs8, vval = _quantise(v, s["vs"])
    whole[..., 17 * D:].view(P, H, nb, 8, sb, 2)[page, :, blk, i // 2, :, i % 2] = vs8
    place = _places(D)
    codes = whole[..., 9 * D:17 * D].view(P, H, nb, 8, D)
    for odd in (0, 1):  # the two tokens of a byte, one after the other
        at = (slots % 2 == odd).nonzero()[:, 0]
        old = codes[page[at], :, blk[at], i[at] // 2]
        mine = torch.empty_like(old).scatter_(-1, place[i[at] // 2][:, None].expand(old.shape), vc[at])
        codes[page[at], :, blk[at], i[at] // 2] = (old & (15 if odd else 240)) + mine * (16 if odd else 1)
    return {"k": kval.to(torch.bfloat16), "v": vval.to(torch.bfloat16), "cache": cache}


def _plain_attend(s):
    q, cache, ps, lens, cu = s["q"], s["cache"], s["ps"], s["lens"].long(), s["cu"].long()
    T, hq, D = q.shape
    P, H = cache.shape[:2]
    B, G, n = lens.numel(), hq // H, s["most_new"]
    pages = s["table"][:, :-(-s["most_len"] // ps)].long().clamp(min=0)
    L = pages.shape[1] * ps
    raw = cache.view(P, H, ps // 16, _block_bytes(D))[pages]           # [B, pages, H, blocks, bytes]
    k, v = _decode(raw.transpose(1, 2), D, s["ks"], s["vs"])           # [B, H, pages, blocks, 16, D]
    k, v = k.reshape(B, H, L, D), v.reshape(B, H, L, D)
    there = torch.arange(L, device=q.device)[None, :] < lens[:, None]
    v = torch.where(there[:, None, :, None], v, torch.zeros((), device=q.device))
    news = cu[1:] - cu[:-1]
    i = torch.arange(n, device=q.device)
    row = (cu[:-1, None] + i).clamp(max=T - 1)
    qs = q.float()[row].view(B, n, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, n * G, D)
    z = torch.matmul(qs, k.transpose(-1, -2)) * s["scale"]
    at = (lens - news)[:, None] + i                                   # position of a new token
    sees = torch.arange(L, device=q.device)[None, None, :] <= at[..., None]
    sees = (sees & there[:, None]).repeat_interleave(G, 1)[:, None]   # [B, 1, n G, L]
    z = torch.where(sees, z, torch.full((), -math.inf, device=q.device))
    m = z.amax(-1, keepdim=True)
    m0 = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.exp(z - m0)
    sums = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v) / torch.where(sums > 0, sums, torch.ones_like(sums))
    lse = (m0 + torch.log(sums)).squeeze(-1)
    seq = torch.searchsorted(cu[1:].contiguous(), torch.arange(T, device=q.device), right=True)
    j = torch.arange(T, device=q.device) - cu[seq]
    o = o.view(B, H, n, G, D)[seq, :, j].reshape(T, hq, D)
    return {"out": o.to(q.dtype), "lse": lse.view(B, H, n, G)[seq, :, j].reshape(T, hq)}


def run(s):
    op = s["op"]
    if not own:
        return {"tables": _plain_tables, "norm_rope": _plain_norm_rope, "append": _plain_append,
                "attend": _plain_attend}[op](s)
    import speculative_decoding_verification_33_gb300 as sv
    if op == "tables":
        out = sv.block_tables(s["ctx"], s["new"], s["table"], s["held"], s["ring"], s["counters"],
                              page_size=s["ps"], max_tokens=s["cap"], accept_len=s["acc"],
                              out=s["out"])
        return {"table": s["table"], "ring": s["ring"], **out}
    if op == "norm_rope":
        return sv.qk_norm_rope(s["q"], s["k"], s["pos"], s["freq"], q_weight=s["wq"],
                               k_weight=s["wk"], eps=s["eps"], interleaved=s["inter"],
                               out=s["out"])
    if op == "append":
        out = sv.kv4_append(s["k"], s["v"], s["slots"], s["cache"], page_size=s["ps"],
                            k_scale=s["ks"], v_scale=s["vs"], out=s["out"])
        return {**out, "cache": s["cache"]}
    return sv.kv4_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], page_size=s["ps"],
                            scale=s["scale"], k_scale=s["ks"], v_scale=s["vs"],
                            max_new=s["most_new"], out=s["out"])


# ---------------------------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "tables":
        # per request: four lengths in, five out; per token its slot, position and sequence; the
        # new pages' ids from the ring into the table
        B, new = case["B"], np.maximum(_news(case)[:, 0], 0)
        T = float(new.sum())
        return {"bytes": 36 * B + 16 * T + 8 * T / case["ps"] + 36, "flops": 0}
    if op == "norm_rope":
        e = 2 if case["dtype"] == "bf16" else 4
        v = case["T"] * (case["hq"] + case["hkv"]) * case["D"]
        return {"bytes": 2 * e * v + 4 * case["T"], "flops": 6 * v}
    if op == "append":
        e = 2 if case["dtype"] == "bf16" else 4
        v = 2 * case["B"] * case["n"] * case["hkv"] * case["D"]
        return {"bytes": v * (e + 2 + 0.5 + 1 / 16) + 8 * case["B"] * case["n"], "flops": 3 * v}
    B, n, ctx, hq, H, D = (case[x] for x in ("B", "n", "ctx", "hq", "hkv", "D"))
    if case["ragged"]:  # mean of the lengths' and the drafts' distributions
        lo = max(1, ctx // 16)
        ctx = (ctx - lo) / math.log(ctx / lo) if ctx > lo else ctx
        n = float(_news(case).mean())
    kv = B * ctx * H * (D + D // 8)
    return {"bytes": kv + B * n * hq * (4 * D + 4), "flops": 4 * B * n * hq * D * ctx}


def _exact_norm_rope(s):
    rot = 2 * s["freq"].numel()
    res = {}
    for name, w in (("q", s["wq"]), ("k", s["wk"])):
        x = s[name].double()
        y = x / (x.pow(2).sum(-1, keepdim=True) / x.shape[-1] + s["eps"]).sqrt() * w.double()
        if s["inter"]:
            first, second = torch.arange(0, rot, 2), torch.arange(1, rot, 2)
        else:
            first, second = torch.arange(rot // 2), torch.arange(rot // 2, rot)
        z = torch.complex(y[..., first], y[..., second])
        a = torch.outer(s["pos"].double(), s["freq"])
        z = z * torch.polar(torch.ones_like(a), a)[:, None]
        y[..., first], y[..., second] = z.real, z.imag
        res[name] = y
    return res


def _exact_append(s):
    grid = torch.tensor(E2M1, dtype=torch.float64, device=DEV)
    # every non-negative e4m3 number but the NaN
    e4m3 = torch.tensor([(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
                         for e in range(16) for m in range(8)][:127], dtype=torch.float64, device=DEV)

    def nearest(x, values):  # to the nearest of ascending values, a tie to the even index
        hi = torch.searchsorted(values, x).clamp(1, values.numel() - 1)
        lo = hi - 1
        a, b = x - values[lo], values[hi] - x
        up = (b < a) | ((a == b) & (hi % 2 == 0))
        return values[torch.where(up, hi, lo)]
    res = {"cache": None}
    for name, g in (("k", s["ks"]), ("v", s["vs"])):
        parts = []
        for x in s[name].split(8192):
            b = x.double().unflatten(-1, (-1, 16))
            scale = nearest(b.abs().amax(-1, keepdim=True) / (6 * g), e4m3) * g
            mag = torch.where(scale > 0, nearest(b.abs() / torch.where(scale > 0, scale, 1.0), grid), 0.0)
            parts.append((b.sign() * mag * scale).flatten(-2))
        res[name] = torch.cat(parts)
    return res


def _exact_attend(s):
    q, cache, ps = s["q"], s["cache"], s["ps"]
    T, hq, D = q.shape
    H, G = cache.shape[1], hq // cache.shape[1]
    out = torch.zeros(T, hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].cpu()
    lut = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6, -0., -.5, -1, -1.5, -2, -3, -4, -6],
                       dtype=torch.float64, device=DEV)
    t16, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    w = D // 8
    swap = (t16 // 2 % 4) * 2 if D == 128 else (t16 // 4 % 2) * 4
    k_at = t16 * (D // 2) + d // 2
    v_at = 9 * D + (t16 // 2) * D + ((d // w) ^ swap) * w + d % w
    ks_at = 8 * D + t16 * (D // 16) + d // 16
    vs_at = 17 * D + (t16 // 2) * (D // 8) + (d // 16) * 2 + t16 % 2
    e4m3 = torch.arange(256, dtype=torch.uint8, device=DEV).view(torch.float8_e4m3fn).double()
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], lens[b]
        if not n or not L:
            continue
        pages = table[b, :-(-L // ps)].long().to(DEV)
        at = L - n + torch.arange(n, device=DEV)
        hidden = torch.arange(L, device=DEV)[None, :] > at[:, None]
        for h in range(H):
            raw = cache[pages, h].reshape(-1, _block_bytes(D))
            kc = raw[:, k_at.flatten()].long().view(-1, 16, D)
            kc = torch.where(d % 2 == 0, kc & 15, kc >> 4)
            vc = raw[:, v_at.flatten()].long().view(-1, 16, D)
            vc = torch.where(t16 % 2 == 0, vc & 15, vc >> 4)
            k = (lut[kc] * e4m3[raw[:, ks_at.flatten()].int()].view(-1, 16, D) * s["ks"]).view(-1, D)[:L]
            v = (lut[vc] * e4m3[raw[:, vs_at.flatten()].int()].view(-1, 16, D) * s["vs"]).view(-1, D)[:L]
            for g in range(G):
                z = (q[cu[b]:cu[b + 1], h * G + g].double() @ k.T) * s["scale"]
                z = z.masked_fill(hidden, -math.inf)
                lse[cu[b]:cu[b + 1], h * G + g] = torch.logsumexp(z, -1)
                out[cu[b]:cu[b + 1], h * G + g] = torch.softmax(z, -1) @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "tables":
        return None
    if case["op"] == "attend" and case["B"] * case["hkv"] > 600 and case["ctx"] * case["B"] * case["hq"] > 1 << 28:
        return None  # over the 20 seconds
    s = prepare(case, seed)
    return {"norm_rope": _exact_norm_rope, "append": _exact_append, "attend": _exact_attend}[case["op"]](s)

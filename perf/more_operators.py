"""Measured cases of the operators around a prompt and a key/value cache held in 8 bits.

Three operators take a request from its prompt to its verify rounds:

- ``prompt``: causal attention over whole prompts, packed one behind the other, grouped heads;
- ``append8``: keys and values into the paged cache in 8 bits, with a scale for each block of 16
  tokens and head;
- ``attend8``: causal attention of each sequence's new tokens over that cache.

``own`` chooses between the plain form (elementary torch operations) and the library's calls. Both
read the same cache bytes. A page of one head is page_size / 16 blocks of 32 D + 16 bytes:

    key codes    [16 tokens][D]          one byte a value, code + 128; the D bytes of token i are
                                         chunks of 16, for D = 128 chunk j at place j ^ (i % 2)
    value codes  [8 token pairs][D][2]   one byte a value, code + 128; the 2 D bytes of pair p are
                                         chunks of 16, chunk j at place j ^ 2 (p % 4)
    head         int8 key exponent, int8 value exponent, 2 bytes, uint16 key marks, uint16 value
                 marks, 8 bytes

A stored value is code * 2^exponent, codes from -127 to 127. The exponent is the smallest, of -60 to
121, whose codes reach the largest magnitude among the block's 16 tokens. A call that writes a block's
first token starts the block afresh; any other keeps what the block holds, and rounds it again where
the exponent grows. A mark says that a token's key or value held a NaN or an infinity; there is none
in the inputs here.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda"
LOW, HIGH = -60, 121  # exponents
HEADS = ((32, 8, 128), (28, 4, 128), (16, 2, 64), (8, 1, 64), (8, 8, 128), (12, 12, 64))
DT = {"bf16": torch.bfloat16, "f32": torch.float32}


# ---------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------
def listed():
    return [
        # three short questions: latency
        {"name": "prompt_short", "op": "prompt", "B": 3, "n": 70, "hq": 16, "hkv": 2, "D": 64,
         "ragged": True},
        # prompts of a busy server's step, packed: few to a thousand tokens each
        {"name": "prompt_batch", "op": "prompt", "B": 24, "n": 1000, "hq": 28, "hkv": 4, "D": 128,
         "ragged": True},
        # one long document, heads of a 4096-wide model
        {"name": "prompt_long", "op": "prompt", "B": 1, "n": 8191, "hq": 32, "hkv": 8, "D": 128,
         "ragged": False},
        # two documents, heads of 64 that share no keys
        {"name": "prompt_d64", "op": "prompt", "B": 2, "n": 5003, "hq": 12, "hkv": 12, "D": 64,
         "ragged": False},
        # verify rows of 64 drafts of 5
        {"name": "append8_verify", "op": "append8", "B": 64, "n": 6, "ps": 64, "hkv": 8, "D": 128,
         "dtype": "bf16"},
        # one token of each of 256 requests, in float32, heads of 64
        {"name": "append8_f32", "op": "append8", "B": 256, "n": 1, "ps": 16, "hkv": 12, "D": 64,
         "dtype": "f32"},
        # prompts of some thousand tokens
        {"name": "append8_prompt", "op": "append8", "B": 13, "n": 5001, "ps": 32, "hkv": 8, "D": 128,
         "dtype": "bf16"},
        # one request, one token, 4k behind it: latency
        {"name": "attend8_b1", "op": "attend8", "B": 1, "n": 1, "ctx": 4097, "ps": 64, "hq": 32,
         "hkv": 8, "D": 128, "ragged": False},
        # one request far into a long document, drafts of 4
        {"name": "attend8_long", "op": "attend8", "B": 1, "n": 5, "ctx": 524301, "ps": 128, "hq": 32,
         "hkv": 8, "D": 128, "ragged": False},
        # 64 requests, drafts of up to 5, lengths up to 8k
        {"name": "attend8_b64", "op": "attend8", "B": 64, "n": 6, "ctx": 8192, "ps": 32, "hq": 32,
         "hkv": 8, "D": 128, "ragged": True},
        # 100 requests, drafts of up to 3, eight heads of 64 on each cached one
        {"name": "attend8_d64", "op": "attend8", "B": 100, "n": 4, "ctx": 4000, "ps": 16, "hq": 16,
         "hkv": 2, "D": 64, "ragged": True},
        # two long prompts, the next part of each
        {"name": "attend8_part", "op": "attend8", "B": 2, "n": 1500, "ctx": 16384, "ps": 64, "hq": 32,
         "hkv": 8, "D": 128, "ragged": False},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 1)))))))


def draw(rng):
    op = rng.choice(("prompt", "prompt", "append8", "attend8", "attend8"))
    ps = rng.choice((16, 32, 64, 128))
    hq, hkv, D = rng.choice(HEADS)
    if op == "prompt":
        B = _log(rng, 1, 64)
        n = _log(rng, 1, max(2, 8000 // B))
        return {"op": op, "B": B, "n": n, "hq": hq, "hkv": hkv, "D": D, "ragged": rng.random() < 0.6}
    if op == "append8":
        B = _log(rng, 1, 256)
        n = rng.choice((rng.randint(1, 9), _log(rng, 10, 8191)))
        return {"op": op, "B": B, "n": max(1, min(n, 60000 // B)), "ps": ps, "hkv": min(hkv, 8), "D": D,
                "dtype": rng.choice(("bf16", "bf16", "f32"))}
    n = rng.choice((1, rng.randint(2, 9), rng.randint(2, 9), rng.randint(10, 64), _log(rng, 65, 1500)))
    B = _log(rng, 1, 256 if n < 10 else 16 if n < 65 else 3)
    most = min(262144, 4_000_000 // (B * hkv), 500_000_000 // (B * hq * n))
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


def _ints(a, dtype=torch.int32):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV, dtype)


def _prompts(case):
    """Lengths of a case's prompts, in no order yet: the same for every seed, so that outputs keep
    their shapes."""
    B, n = case["B"], case["n"]
    if not case["ragged"]:
        return np.full(B, n)
    r = np.random.default_rng([B, n, 11])
    lens = np.exp(r.uniform(math.log(max(1, n // 64)), math.log(n), B)).astype(np.int64)
    lens[0] = n
    return np.maximum(1, lens)


def _news(case):
    """New tokens of the sequences of an ``attend8`` case, the same for every seed."""
    B, n = case["B"], case["n"]
    r = np.random.default_rng([B, n])
    return r.integers(max(1, min(2, n)), n + 1, B) if case["ragged"] else np.full(B, n)


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


def _prep_prompt(case, seed):
    g = _gen(seed)
    hq, H, D = case["hq"], case["hkv"], case["D"]
    lens = np.random.default_rng([seed, 5]).permutation(_prompts(case))
    T = int(lens.sum())
    # queries and keys come from their norms, values are part of the projection's output
    qkv = torch.randn(T, (hq + 2 * H) * D, device=DEV, generator=g).to(torch.bfloat16)
    q = (1.5 * torch.randn(T, hq, D, device=DEV, generator=g)).to(torch.bfloat16)
    k = torch.randn(T, H, D, device=DEV, generator=g).to(torch.bfloat16)
    v = qkv[:, (hq + H) * D:].view(T, H, D)
    return {"op": "prompt", "q": q, "k": k, "v": v,
            "cu": _ints(np.concatenate([[0], np.cumsum(lens)])), "scale": 1 / math.sqrt(D),
            "out": {"out": torch.empty_like(q),
                    "lse": torch.empty(T, hq, dtype=torch.float32, device=DEV)}}


def _prep_append8(case, seed):
    g = _gen(seed)
    B, n, ps, H, D = case["B"], case["n"], case["ps"], case["hkv"], case["D"]
    dt = DT[case["dtype"]]
    r = np.random.default_rng([seed, 2])
    start = r.integers(0, 4 * ps, B)  # tokens that the sequence has already
    blocks = -(-(4 * ps + n) // ps)
    P = B * blocks + 3
    pages = r.permutation(P)[:B * blocks].reshape(B, blocks)
    at = start[:, None] + np.arange(n)[None, :]
    slots = (pages[np.arange(B)[:, None], at // ps] * ps + at % ps).reshape(-1)
    T = B * n
    k = torch.randn(T, H, D, device=DEV, generator=g).to(dt)
    v = (torch.randn(T, H, D, device=DEV, generator=g)
         * torch.exp(torch.randn(T, H, 1, device=DEV, generator=g))).to(dt)
    cache = torch.empty(P, H, ps // 16 * _block_bytes(D), dtype=torch.uint8, device=DEV)
    _fill(cache, ps, D, g)
    return {"op": "append8", "k": k, "v": v, "slots": _ints(slots, torch.int64), "cache": cache,
            "ps": ps, "out": {"k": torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV),
                              "v": torch.empty(T, H, D, dtype=torch.bfloat16, device=DEV)}}


def _prep_attend8(case, seed):
    g = _gen(seed)
    ps, hq, H, D = case["ps"], case["hq"], case["hkv"], case["D"]
    news, lens = _lens(case, seed)
    held = -(-lens // ps)
    P = int(held.sum()) + 5
    pages = np.random.default_rng([seed, 3]).permutation(P)
    most = int(held.max()) + 1
    table = np.full((case["B"], most), -1, np.int32)
    table[np.arange(most)[None, :] < held[:, None]] = pages[:P - 5]
    cache = torch.empty(P, H, ps // 16 * _block_bytes(D), dtype=torch.uint8, device=DEV)
    _fill(cache, ps, D, g)
    T = int(news.sum())
    q = (1.5 * torch.randn(T, hq, D, device=DEV, generator=g)).to(torch.bfloat16)
    return {"op": "attend8", "q": q, "cache": cache, "table": _ints(table), "lens": _ints(lens),
            "cu": _ints(np.concatenate([[0], np.cumsum(news)])), "ps": ps, "scale": 1 / math.sqrt(D),
            "most_new": int(news.max()), "most_len": int(lens.max()),
            "out": {"out": torch.empty_like(q),
                    "lse": torch.empty(T, hq, dtype=torch.float32, device=DEV)}}


def _fill(cache, ps, D, g):
    """Pages of quantised keys and values: channels and tokens differ in magnitude."""
    P, H = cache.shape[:2]
    step = max(1, (1 << 25) // (H * ps * D))
    ch = torch.exp(0.5 * torch.randn(2, H, 1, D, device=DEV, generator=g))
    for p in range(0, P, step):
        m = min(step, P - p)
        x = torch.randn(2, m, H, ps, D, device=DEV, generator=g) * ch[:, None]
        x *= torch.exp(0.3 * torch.randn(2, m, H, ps, 1, device=DEV, generator=g))
        _store(cache[p:p + m].view(m, H, ps // 16, _block_bytes(D)), *_fresh(x[0]), *_fresh(x[1]))


def prepare(case, seed):
    return {"prompt": _prep_prompt, "append8": _prep_append8, "attend8": _prep_attend8}[case["op"]](case, seed)


# ---------------------------------------------------------------------------------------------
# the 8-bit format, in elementary operations
# ---------------------------------------------------------------------------------------------
def _block_bytes(D):
    return 32 * D + 16


def _two(e):
    """2^e in float32, e from -126 to 127."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _exponent(most):
    """The smallest exponent whose codes reach `most` (float32, not negative)."""
    bits = most.view(torch.int32)
    return ((bits >> 23) - 127 - 6 + ((bits & 0x7FFFFF) > 0x7E0000).int()).clamp(LOW, HIGH)


def _codes(x, e):
    return torch.round(x * _two(-e)).clamp(-127, 127)


def _fresh(x):
    """Pages [m, H, ps, D] in float32 -> codes [m, H, blocks, 16, D], exponents [m, H, blocks]."""
    x = x.unflatten(2, (-1, 16))
    e = _exponent(x.abs().amax((-1, -2)))
    return _codes(x, e[..., None, None]), e


def _key_places(D):
    """Place of value d of token i among a block's key codes: [16, D]."""
    i, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    return i * D + (((d // 16) ^ (i % 2)) * 16 if D == 128 else d // 16 * 16) + d % 16


def _value_places(D):
    """Place of value d of token i among a block's value codes: [16, D]."""
    i, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    return (i // 2) * 2 * D + ((d // 8) ^ (i // 2 % 4 * 2)) * 16 + 2 * (d % 8) + i % 2


def _store(to, kc, ke, vc, ve):
    """Codes [..., 16, D] and exponents [...] into blocks `to` [..., bytes], no marks."""
    D = kc.shape[-1]
    for c, place, at in ((kc, _key_places(D), 0), (vc, _value_places(D), 16 * D)):
        back = torch.empty_like(place.flatten()).scatter_(0, place.flatten(), torch.arange(16 * D, device=DEV))
        to[..., at:at + 16 * D] = (c + 128).byte().flatten(-2)[..., back]
    to[..., 32 * D:] = 0
    to[..., 32 * D] = (ke & 255).byte()
    to[..., 32 * D + 1] = (ve & 255).byte()


def _load(raw, D):
    """Blocks [..., bytes] -> key codes, key exponents, value codes, value exponents."""
    def signed(b):
        return (b.int() ^ 128) - 128
    kc = raw[..., :16 * D][..., _key_places(D)].float() - 128
    vc = raw[..., 16 * D:32 * D][..., _value_places(D)].float() - 128
    return kc, signed(raw[..., 32 * D]), vc, signed(raw[..., 32 * D + 1])


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def _plain_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].long()
    T, hq, D = q.shape
    H = k.shape[1]
    t = torch.arange(T, device=q.device)
    seq = torch.searchsorted(cu[1:].contiguous(), t, right=True)
    sees = (seq[:, None] == seq[None, :]) & (t[None, :] <= t[:, None])
    z = torch.matmul(q.float().view(T, H, hq // H, D).permute(1, 2, 0, 3),
                     k.float().permute(1, 2, 0)[:, None]) * s["scale"]     # [H, G, T, T]
    z = torch.where(sees, z, torch.full((), -math.inf, device=q.device))
    m = z.amax(-1, keepdim=True)
    p = torch.exp(z - m)
    sums = p.sum(-1, keepdim=True)
    o = torch.matmul(p, v.float().permute(1, 0, 2)[:, None]) / sums
    lse = (m + torch.log(sums)).squeeze(-1)
    return {"out": o.permute(2, 0, 1, 3).reshape(T, hq, D).to(q.dtype),
            "lse": lse.permute(2, 0, 1).reshape(T, hq)}


def _plain_append8(s):
    cache, slots, ps = s["cache"], s["slots"], s["ps"]
    T, H, D = s["k"].shape
    P, nb = cache.shape[0], ps // 16
    blk, i = slots // 16, slots % 16                            # blocks in page order, place in one
    whole = cache.view(P, H, nb, -1).transpose(1, 2).clone(memory_format=torch.contiguous_format).view(P * nb, H, -1)
    kc, ke, vc, ve = _load(whole, D)
    afresh = torch.zeros(P * nb, dtype=torch.bool, device=DEV).index_fill_(0, blk[i == 0], True)[:, None]
    out = {}

    def write(x, c, e):
        x = x.float()
        need = torch.zeros(P * nb, H, device=DEV)
        need = _exponent(need.scatter_reduce_(0, blk[:, None].expand(T, H), x.abs().amax(-1), "amax"))
        new = torch.where(afresh, need, torch.maximum(e, need))
        untouched = torch.ones(P * nb, dtype=torch.bool, device=DEV).index_fill_(0, blk, False)
        new = torch.where(untouched[:, None], e, new)
        down = _two((e - new).clamp(min=-126))[..., None, None]
        c = torch.where(afresh[..., None, None], torch.zeros((), device=DEV), torch.round(c * down))
        mine = _codes(x, new[blk][..., None])
        c[blk, :, i] = mine
        return c, new, (mine * _two(new[blk])[..., None]).to(torch.bfloat16)
    kc, ke, out["k"] = write(s["k"], kc, ke)
    vc, ve, out["v"] = write(s["v"], vc, ve)
    _store(whole, kc, ke, vc, ve)
    cache.view(P, H, nb, -1)[:] = whole.view(P, nb, H, -1).transpose(1, 2)
    return {**out, "cache": cache}


def _plain_attend8(s):
    q, cache, ps, lens, cu = s["q"], s["cache"], s["ps"], s["lens"].long(), s["cu"].long()
    T, hq, D = q.shape
    P, H = cache.shape[:2]
    B, G, n = lens.numel(), hq // H, s["most_new"]
    pages = s["table"][:, :-(-s["most_len"] // ps)].long().clamp(min=0)
    L = pages.shape[1] * ps
    raw = cache.view(P, H, ps // 16, _block_bytes(D))[pages].transpose(1, 2)  # [B, H, pages, blocks, bytes]
    kc, ke, vc, ve = _load(raw, D)
    k = (kc * _two(ke)[..., None, None]).reshape(B, H, L, D)
    v = (vc * _two(ve)[..., None, None]).reshape(B, H, L, D)
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
        return {"prompt": _plain_prompt, "append8": _plain_append8, "attend8": _plain_attend8}[op](s)
    import speculative_decoding_verification_33_gb300 as sv
    if op == "prompt":
        return sv.prompt_attention(s["q"], s["k"], s["v"], s["cu"], scale=s["scale"], out=s["out"])
    if op == "append8":
        out = sv.kv8_append(s["k"], s["v"], s["slots"], s["cache"], page_size=s["ps"], out=s["out"])
        return {**out, "cache": s["cache"]}
    return sv.kv8_attention(s["q"], s["cache"], s["table"], s["lens"], s["cu"], page_size=s["ps"],
                            scale=s["scale"], max_new=s["most_new"], out=s["out"])


# ---------------------------------------------------------------------------------------------
# work and the definition in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "prompt":
        hq, H, D = case["hq"], case["hkv"], case["D"]
        lens = _prompts(case).astype(np.float64)
        pairs = float((lens * (lens + 1) / 2).sum())
        return {"bytes": float(lens.sum()) * (4 * (hq + H) * D + 4 * hq), "flops": 4 * hq * D * pairs}
    if op == "append8":
        # values in, codes out, and the values that the cache then stands for
        e = 2 if case["dtype"] == "bf16" else 4
        tokens = case["B"] * case["n"]
        v = 2 * tokens * case["hkv"] * case["D"]
        return {"bytes": v * (e + 2 + 1) + 8 * tokens, "flops": 3 * v}
    B, n, ctx, hq, H, D = (case[x] for x in ("B", "n", "ctx", "hq", "hkv", "D"))
    if case["ragged"]:  # mean of the lengths' and the drafts' distributions
        lo = max(1, ctx // 16)
        ctx = (ctx - lo) / math.log(ctx / lo) if ctx > lo else ctx
        n = float(_news(case).mean())
    kv = B * ctx * H * (2 * D + 1)
    seen = max(ctx - (n - 1) / 2, 1.0)  # a row does not see the new tokens behind it
    return {"bytes": kv + B * n * hq * (4 * D + 4), "flops": 4 * B * n * hq * D * seen}


def _exact_prompt(s):
    q, k, v, cu = s["q"], s["k"], s["v"], s["cu"].tolist()
    T, hq, D = q.shape
    G = hq // k.shape[1]
    out = torch.empty(T, hq, D, dtype=torch.float64, device=DEV)
    lse = torch.empty(T, hq, dtype=torch.float64, device=DEV)
    for a, b in zip(cu[:-1], cu[1:]):
        later = torch.ones(b - a, b - a, dtype=torch.bool, device=DEV).triu(1)
        for h in range(hq):
            z = q[a:b, h].double() @ k[a:b, h // G].double().T
            z = z.mul_(s["scale"]).masked_fill_(later, -math.inf)
            lse[a:b, h] = torch.logsumexp(z, -1)
            out[a:b, h] = torch.softmax(z, -1) @ v[a:b, h // G].double()
    return {"out": out, "lse": lse}


def _exponents64(raw, D):
    return raw[..., 32 * D:32 * D + 2].contiguous().view(torch.int8).double().unbind(-1)


def _exact_append8(s):
    cache, slots, ps = s["cache"], s["slots"], s["ps"]
    T, H, D = s["k"].shape
    P, nb = cache.shape[0], ps // 16
    had = _exponents64(cache.view(P, H, nb, -1), D)
    page, j, first = slots // ps, slots % ps // 16, slots % 16 == 0
    blk = page * nb + j
    begun = torch.zeros(P * nb, dtype=torch.float64, device=DEV).scatter_add_(0, blk, first.double()) > 0
    res = {"cache": None}
    powers = torch.tensor([2.0 ** i for i in range(LOW, HIGH + 1)], dtype=torch.float64, device=DEV)
    for name, old in (("k", had[0]), ("v", had[1])):
        x = s[name].double()
        most = torch.zeros(P * nb, H, dtype=torch.float64, device=DEV)
        most.scatter_reduce_(0, blk[:, None].expand(T, H), x.abs().amax(-1), "amax")
        frac, exp = torch.frexp(most)  # the smallest e with most <= 127 2^e
        e = (exp - 7 + (frac > 127 / 128)).double()
        e = torch.where(most > 0, e, torch.full_like(e, LOW)).clamp(LOW, HIGH)
        e = torch.where(begun[:, None], e, torch.maximum(e, old.transpose(1, 2).reshape(P * nb, H)))
        step = powers[e[blk].long() - LOW][..., None]
        res[name] = torch.round(x / step).clamp(-127, 127) * step
    return res


def _exact_attend8(s):
    q, cache, ps = s["q"], s["cache"], s["ps"]
    T, hq, D = q.shape
    H = cache.shape[1]
    G = hq // H
    out = torch.zeros(T, hq, D, dtype=torch.float64, device=DEV)
    lse = torch.full((T, hq), -math.inf, dtype=torch.float64, device=DEV)
    cu, lens, table = s["cu"].tolist(), s["lens"].tolist(), s["table"].cpu()
    t, d = torch.arange(16, device=DEV)[:, None], torch.arange(D, device=DEV)[None, :]
    turn = (t & 1) * 16 if D == 128 else 0 * t
    k_at = (t * D + (d ^ turn)).flatten()
    v_at = (16 * D + (t >> 1) * 2 * D + ((2 * d + (t & 1)) ^ (((t >> 1) & 3) * 32))).flatten()
    for b in range(len(lens)):
        n, L = cu[b + 1] - cu[b], lens[b]
        if not n or not L:
            continue
        pages = table[b, :-(-L // ps)].long().to(DEV)
        at = L - n + torch.arange(n, device=DEV)
        hidden = (torch.arange(L, device=DEV)[None, :] > at[:, None]).repeat(G, 1)
        for h in range(H):
            raw = cache[pages, h].reshape(-1, _block_bytes(D))
            ek, ev = _exponents64(raw, D)
            k = ((raw[:, k_at].double() - 128) * torch.exp2(ek)[:, None]).view(-1, D)[:L]
            v = ((raw[:, v_at].double() - 128) * torch.exp2(ev)[:, None]).view(-1, D)[:L]
            rows = q[cu[b]:cu[b + 1], h * G:h * G + G].double().transpose(0, 1).reshape(G * n, D)
            z = ((rows @ k.T) * s["scale"]).masked_fill_(hidden, -math.inf)
            lse[cu[b]:cu[b + 1], h * G:h * G + G] = torch.logsumexp(z, -1).view(G, n).T
            out[cu[b]:cu[b + 1], h * G:h * G + G] = (torch.softmax(z, -1) @ v).view(G, n, D).transpose(0, 1)
    return {"out": out, "lse": lse}


def exact(case, seed):
    if case["op"] == "attend8" and case["B"] * case["hkv"] > 1200:
        return None  # over the 20 seconds
    s = prepare(case, seed)
    return {"prompt": _exact_prompt, "append8": _exact_append8, "attend8": _exact_attend8}[case["op"]](s)

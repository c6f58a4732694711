"""The 8-bit cache's operators together: prompts and rounds as examples/cache_rounds.py runs them, and each step
against the float64 oracle."""
import importlib.util
import os

import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from oracle import kvcache8 as O  # noqa: E402

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("cache_rounds", os.path.join(ROOT, "examples", "cache_rounds.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)

I32 = {"dtype": torch.int32, "device": "cuda"}


def host(t):
    return t.double().cpu().numpy() if t.is_floating_point() else t.cpu().numpy()


def test_rounds_keep_the_tokens_and_the_pages():
    K = 4
    spec_run, accepted = ex.main(rounds=12, K=K, bits=8)
    assert accepted.shape[0] == 12 and 0 <= accepted.min() and accepted.max() <= K
    for b, toks in enumerate(spec_run.out):  # a first token, and each round's accepted drafts and one more
        assert len(toks) == 1 + 12 + int(accepted[:, b].sum())
        assert all(0 <= t < 2000 for t in toks)
    # pages: each is free or held once
    live = [int(spec_run.ring[i % len(spec_run.ring)]) for i in range(*spec_run.counters.tolist())]
    held = [int(p) for b in range(len(spec_run.out)) for p in spec_run.table[b, :spec_run.held[b]]]
    assert sorted(live + held) == list(range(len(spec_run.ring)))


def _close(o, ref, D, weight):
    """Half a bf16 step; weights off by `weight` of each; scores as float32 sums (2^-24 of the magnitudes a step,
    D products, scalings and exponents) and exponentials (2^-22), in numerator and denominator; the weighted sum;
    2^-32 of the row's largest weight where the cache's values have exponents."""
    dz = (D + 8) * 2.0 ** -24 * ref["zroom"] + np.abs(ref["lse"]) * 2.0 ** -22 + ref.get("emost", 0) * 2.0 ** -23
    tol = 2.0 ** -8 * np.abs(ref["out"]) + ref["room"] * (weight + 2 * dz[..., None] + 2.0 ** -18)
    tol = tol + 2.0 ** -32 * ref["vsum"] if "vsum" in ref else tol
    assert (np.abs(host(o["out"]) - ref["out"]) <= tol + 1e-30).all()
    assert (np.abs(host(o["lse"]) - ref["lse"]) <= dz + 2.0 ** -19).all()


@pytest.mark.parametrize("hq,hk,D,ps", [(8, 2, 64, 16), (14, 2, 128, 32)])
def test_steps(hq, hk, D, ps):
    """Prompts, then two rounds whose rejected drafts the next one writes over: after each, the cache's bytes
    are the oracle's, and outputs those of the attention over them. Rows of the prompts get from
    ``prompt_attention`` what ``kv8_attention`` gives them."""
    lens, K, pages = [1, 40, 150, 16], 5, 64
    B = len(lens)
    g = torch.Generator("cuda").manual_seed(D)
    cache, want = sv.kv8_cache(pages, hk, D, ps), np.zeros((pages, hk, sv.kv8_page_bytes(ps, D)), np.uint8)
    assert tuple(cache.shape) == want.shape
    cache.zero_()
    table, ring = torch.full((B, 24), -1, **I32), torch.arange(pages, **I32)
    ctx, held, counters = torch.zeros(B, **I32), torch.zeros(B, **I32), torch.tensor([0, pages], device="cuda")
    freq = 10000.0 ** (-torch.arange(D // 2, dtype=torch.float64, device="cuda") / (D // 2))
    accept = None
    for step in range(3):
        new = torch.tensor(lens, **I32) if step == 0 else torch.full((B,), K + 1, **I32)
        T, most = int(new.sum()), int(new.max())
        r = sv.block_tables(ctx, new, table, held, ring, counters, page_size=ps, max_tokens=T, accept_len=accept)
        ctx, held, counters = r["ctx_lens"], r["held"], r["counters"]
        assert bool((r["status"] >= 0).all())
        q, k, v = (torch.randn(T, h, D, device="cuda", generator=g).to(torch.bfloat16) for h in (hq, hk, hk))
        sv.qk_norm_rope(q, k, r["positions"], freq, out={"q": q, "k": k})
        got = sv.kv8_append(k, v, r["slots"], cache, page_size=ps, values=True)
        stand = O.append(want, host(r["slots"]), host(k), host(v), ps)
        assert np.array_equal(host(cache), want)
        assert np.array_equal(host(got["k"]), stand[0]) and np.array_equal(host(got["v"]), stand[1])
        ref = O.attention(host(q), want, host(table), host(r["kv_lens"]), host(r["cu_new"]), ps, D ** -0.5)
        _close(sv.kv8_attention(q, cache, table, r["kv_lens"], r["cu_new"], page_size=ps, max_new=most), ref, D,
               2.0 ** -11)
        if step == 0:
            _close(sv.prompt_attention(q, got["k"], got["v"], r["cu_new"]), ref, D, 2.0 ** -8)
        accept = new - 1 if step == 0 else torch.tensor([0, K, 2, 1], **I32)
    assert sv.device_error() == 0

"""Rounds of greedy self-speculative decoding over the 4-bit or the 8-bit paged cache, end to end.

A small decoder with random weights drafts with its first layers and the shared head (an early
exit) and verifies with all of them (LayerSkip guide, "Verification Phase"): each round is one
``block_tables`` call, the drafts' single-token passes through the first layers, one pass of all
layers over every sequence's last token and drafts (``qk_norm_rope``, ``kv4_append``,
``kv4_attention``), and ``verify_hidden``, whose accepted lengths roll the cache back in the next
round's ``block_tables``. With 8 bits (``kv8_append``, ``kv8_attention``) the prompts' pass runs
``prompt_attention`` over the keys and values as the cache holds them, without reading it. Projections
are plain matrix products.

    python examples/cache_rounds.py [rounds] [draft length] [bits]
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import speculative_decoding_verification_33_gb300 as sv  # noqa: E402

BF16 = torch.bfloat16


class Decoder:
    """``layers`` layers of attention and a gated product, the first ``exit`` of which draft."""

    def __init__(self, d=512, hq=8, hkv=2, head=64, vocab=2000, layers=4, exit=2, seed=0):
        g = torch.Generator("cuda").manual_seed(seed)

        def w(*shape, scale=1.0):
            x = torch.randn(*shape, generator=g, device="cuda") * (scale * shape[-1] ** -0.5)
            return x.to(BF16)
        self.d, self.hq, self.hkv, self.head, self.exit = d, hq, hkv, head, exit
        self.embed, self.lm_head = w(vocab, d, scale=d ** 0.5), w(vocab, d)
        # later layers change less, as in a trained model, so that early exits are often right
        self.layers = [{"qkv": w((hq + 2 * hkv) * head, d), "o": w(d, hq * head, scale=0.7 ** i),
                        "up": w(4 * d, d), "gate": w(4 * d, d), "down": w(d, 4 * d, scale=0.7 ** i),
                        "qn": (1 + 0.1 * torch.randn(head, generator=g, device="cuda")).to(BF16),
                        "kn": (1 + 0.1 * torch.randn(head, generator=g, device="cuda")).to(BF16)}
                       for i in range(layers)]
        self.freq = 10000.0 ** (-torch.arange(head // 2, dtype=torch.float64, device="cuda") / (head // 2))

    @staticmethod
    def norm(x):
        y = x.float()
        return (y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)).to(BF16)

    def forward(self, tokens, positions, slots, caches, table, kv_lens, cu_new, max_new, page_size,
                layers, bits=4, prompts=False):
        """Hidden states [T, d] of ``tokens`` after the first ``layers`` layers; their keys and values
        go into ``caches`` at ``slots``. ``prompts``: nothing is cached before these tokens."""
        x = self.embed[tokens.long()]
        T, qw, kw = x.shape[0], self.hq * self.head, self.hkv * self.head
        for w, cache in zip(self.layers[:layers], caches):
            qkv = self.norm(x) @ w["qkv"].T
            q = qkv[:, :qw].unflatten(1, (self.hq, self.head))
            k = qkv[:, qw:qw + kw].unflatten(1, (self.hkv, self.head))
            v = qkv[:, qw + kw:].unflatten(1, (self.hkv, self.head))
            sv.qk_norm_rope(q, k, positions, self.freq, q_weight=w["qn"], k_weight=w["kn"],
                            out={"q": q, "k": k})
            if bits == 8:
                held = sv.kv8_append(k, v, slots, cache, page_size=page_size, values=prompts)
            else:
                sv.kv4_append(k, v, slots, cache, page_size=page_size)
            if bits == 8 and prompts:
                a = sv.prompt_attention(q, held["k"], held["v"], cu_new)
            else:
                attend = sv.kv8_attention if bits == 8 else sv.kv4_attention
                a = attend(q, cache, table, kv_lens, cu_new, page_size=page_size, max_new=max_new)
            x = x + a["out"].view(T, qw) @ w["o"].T
            y = self.norm(x)
            x = x + (torch.nn.functional.silu(y @ w["gate"].T) * (y @ w["up"].T)) @ w["down"].T
        return self.norm(x)

    def next_token(self, hidden):
        return sv.lmhead_stats(hidden, self.lm_head)["argmax"]


class Session:
    """Sequences that decode together: their lengths, pages and caches."""

    def __init__(self, model, prompts, page_size=16, pages=512, max_blocks=64, bits=4):
        self.m, self.ps, self.bits, B = model, page_size, bits, len(prompts)
        i32 = {"dtype": torch.int32, "device": "cuda"}
        empty = sv.kv8_cache if bits == 8 else sv.kv4_cache
        self.caches = [empty(pages, model.hkv, model.head, page_size) for _ in model.layers]
        self.table = torch.full((B, max_blocks), -1, **i32)
        self.ring = torch.arange(pages, **i32)
        self.ctx, self.held = torch.zeros(B, **i32), torch.zeros(B, **i32)
        self.counters = torch.tensor([0, pages], device="cuda")
        self.accept = None
        # the prompts, all but whose last tokens are context
        new = torch.tensor([len(p) for p in prompts], **i32)
        r = self.tables(new, int(new.sum()))
        tokens = torch.tensor([t for p in prompts for t in p], **i32)
        h = model.forward(tokens, r["positions"], r["slots"], self.caches, self.table, r["kv_lens"],
                          r["cu_new"], int(new.max()), self.ps, len(model.layers), bits, prompts=True)
        self.last = model.next_token(h[(r["cu_new"][1:] - 1).long()])
        self.accept = new - 1
        self.out = [[int(t)] for t in self.last]

    def tables(self, new, most):
        r = sv.block_tables(self.ctx, new, self.table, self.held, self.ring, self.counters,
                            page_size=self.ps, max_tokens=most, accept_len=self.accept)
        self.ctx, self.held, self.counters = r["ctx_lens"], r["held"], r["counters"]
        assert bool((r["status"] >= 0).all()), "out of pages"
        return r

    def round(self, K):
        """One round with K drafts a sequence (K = 0: plain decoding). Returns the accepted lengths."""
        m, B = self.m, self.last.shape[0]
        new = torch.full_like(self.last, K + 1)
        r = self.tables(new, B * (K + 1))
        slots, positions = r["slots"].view(B, K + 1), r["positions"].view(B, K + 1)
        tokens = self.last.new_empty(B, K + 1)
        tokens[:, 0] = self.last
        one = torch.arange(B + 1, dtype=torch.int32, device="cuda")
        for j in range(K):  # drafts: the first layers, a token at a time
            h = m.forward(tokens[:, j], positions[:, j].contiguous(), slots[:, j].contiguous(),
                          self.caches, self.table, positions[:, j] + 1, one, 1, self.ps, m.exit,
                          self.bits)
            tokens[:, j + 1] = m.next_token(h)
        h = m.forward(tokens.view(-1), r["positions"], r["slots"], self.caches, self.table,
                      r["kv_lens"], r["cu_new"], K + 1, self.ps, len(m.layers), self.bits)
        if K == 0:
            self.last, self.accept = m.next_token(h), torch.zeros_like(self.last)
            for b, t in enumerate(self.last.tolist()):
                self.out[b].append(t)
            return self.accept
        v = sv.verify_hidden(h.view(B, K + 1, -1), None, m.lm_head, tokens[:, 1:].contiguous(),
                             new - 1, mode="greedy")
        self.accept = v["accept_len"]
        self.last = v["tokens"].gather(1, self.accept[:, None].long())[:, 0].contiguous()
        for b, (a, row) in enumerate(zip(self.accept.tolist(), v["tokens"].tolist())):
            self.out[b] += row[:a + 1]
        return self.accept


def main(rounds=12, K=4, bits=4):
    model = Decoder()
    g = torch.Generator().manual_seed(1)
    prompts = [torch.randint(0, 2000, (n,), generator=g).tolist() for n in (1, 7, 16, 33, 90, 127)]
    s = Session(model, prompts, bits=bits)
    accepted = torch.stack([s.round(K) for _ in range(rounds)]).float()
    torch.cuda.synchronize()
    assert sv.device_error() == 0
    return s, accepted


if __name__ == "__main__":
    args = [int(a) for a in sys.argv[1:4]]
    session, acc = main(*args)
    print(f"{acc.shape[0]} rounds, {acc.mean():.2f} drafts accepted a round and sequence")
    for b, toks in enumerate(session.out):
        print(f"sequence {b}: {len(toks)} tokens, the first {toks[:8]}")

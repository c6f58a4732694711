"""First calls on a stream while the default stream is busy: what a stream's workspace starts from is
set in that stream's own order, so results do not depend on what other streams have queued."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402

BF16 = torch.bfloat16


def first_calls(call, want, streams=3):
    """``call`` on streams that no other test uses, each with some 30 ms queued on the default stream; none
    of them waits for that. Its tensors must equal ``want``'s, on the first call and on a second one after
    the default stream has run dry."""
    a = torch.zeros(8192, 8192, device="cuda", dtype=BF16)
    for _ in range(streams):
        s = torch.cuda.Stream(priority=-1)  # another set of streams than the usual priority's
        torch.cuda.synchronize()
        b = a
        for _ in range(40):
            b = b @ a
        with torch.cuda.stream(s):
            first = call()
        s.synchronize()
        torch.cuda.synchronize()
        with torch.cuda.stream(s):
            second = call()
        torch.cuda.synchronize()
        for got in (first, second):
            assert got.keys() == want.keys()
            assert all(torch.equal(got[k], want[k]) for k in want)
        with torch.cuda.stream(s):
            assert sv.device_error() == 0


@pytest.mark.parametrize("max_new", [3, 64])
def test_attention(max_new):
    """Few heads and long sequences: every head is cut, and its pieces are joined by arrival counts."""
    B, L, H, D, ps = 2, 6000, 2, 128, 32
    g = torch.Generator("cuda").manual_seed(3)
    blocks = -(-L // ps)
    table = torch.randperm(B * blocks, device="cuda", generator=g).view(B, blocks)
    cache = sv.kv4_cache(B * blocks, H, D, ps)
    t = torch.arange(L, device="cuda")
    for b in range(B):
        x = torch.randn(2, L, H, D, device="cuda", generator=g).to(BF16)
        sv.kv4_append(x[0], x[1], table[b, t // ps] * ps + t % ps, cache, page_size=ps)
    i32 = {"dtype": torch.int32, "device": "cuda"}
    table, lens, cu = table.int(), torch.tensor([L, L - 77], **i32), torch.tensor([0, 3, 5], **i32)
    q = torch.randn(5, 8, D, device="cuda", generator=g).to(BF16)
    out = iter([{"out": torch.full_like(q, 7.0), "lse": torch.full((5, 8), 7.0, device="cuda")}
                for _ in range(7)])  # rows that nobody writes show

    def call():
        return sv.kv4_attention(q, cache, table, lens, cu, page_size=ps, max_new=max_new, out=next(out))
    first_calls(call, call())


@pytest.mark.parametrize("B,K,V,mode,beta", [
    (64, 8, 152064, "stochastic", 1.0),   # the walk, its draws deferred to two more launches
    (64, 8, 152064, "stochastic", 0.5),   # the walk behind its prepass
    (64, 8, 152064, "greedy", 1.0),       # the greedy walk
    (8, 5, 32000, "stochastic", 1.0),     # every row at once
    (8, 5, 32000, "greedy", 1.0)])
def test_verify(B, K, V, mode, beta):
    g = torch.Generator("cuda").manual_seed(B + K)
    tgt = torch.randn(B, K + 1, V, device="cuda", generator=g).mul_(2).to(BF16)
    dft = (tgt[:, :K].float() + torch.randn(B, K, V, device="cuda", generator=g) * 0.3).to(BF16)
    tokens = dft.argmax(-1).int()
    uniforms = torch.rand(B, K + 1, device="cuda", generator=g)

    def call():
        return sv.verify(tgt, None if mode == "greedy" else dft, tokens, None,
                         None if mode == "greedy" else uniforms, mode=mode, beta=beta,
                         bias_k=4 if beta < 1 else 0)
    first_calls(call, call())


def test_rows():
    """The row steps' queues."""
    B, K, V = 40, 6, 32000
    g = torch.Generator("cuda").manual_seed(1)
    tgt = torch.randn(B, K + 1, V, device="cuda", generator=g).to(BF16)
    dft = torch.randn(B, K, V, device="cuda", generator=g).to(BF16)
    uniforms = torch.rand(B * K, device="cuda", generator=g)

    def call():
        return {**sv.draft_sample(dft.view(B * K, V), uniforms, beta=0.5, bias_k=4),
                **sv.residual_topf(tgt, dft, None, [4] * K)}
    first_calls(call, call())

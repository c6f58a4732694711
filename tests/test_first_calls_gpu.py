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

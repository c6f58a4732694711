"""First calls of the 8-bit cache's attention and of prompt attention on a stream while the default stream is
busy: the workspace's counters and queue start in that stream's own order."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from tests.test_first_calls_gpu import first_calls  # noqa: E402

BF16 = torch.bfloat16
I32 = {"dtype": torch.int32, "device": "cuda"}


@pytest.mark.parametrize("max_new", [3, 64])
def test_cache8(max_new):
    """Few heads and long sequences: every head is cut, and its pieces are joined by arrival counts."""
    B, L, H, D, ps = 2, 6000, 2, 128, 32
    g = torch.Generator("cuda").manual_seed(3)
    blocks = -(-L // ps)
    table = torch.randperm(B * blocks, device="cuda", generator=g).view(B, blocks)
    cache = sv.kv8_cache(B * blocks, H, D, ps)
    t = torch.arange(L, device="cuda")
    for b in range(B):
        x = torch.randn(2, L, H, D, device="cuda", generator=g).to(BF16)
        sv.kv8_append(x[0], x[1], table[b, t // ps] * ps + t % ps, cache, page_size=ps)
    table, lens, cu = table.int(), torch.tensor([L, L - 77], **I32), torch.tensor([0, 3, 5], **I32)
    q = torch.randn(5, 8, D, device="cuda", generator=g).to(BF16)
    out = iter([{"out": torch.full_like(q, 7.0), "lse": torch.full((5, 8), 7.0, device="cuda")}
                for _ in range(7)])  # rows that nobody writes show

    def call():
        return sv.kv8_attention(q, cache, table, lens, cu, page_size=ps, max_new=max_new, out=next(out))
    first_calls(call, call())


@pytest.mark.parametrize("hq,hk,D", [(28, 4, 128), (8, 8, 64)])
def test_prompts(hq, hk, D):
    """More items than CTAs: later ones come from the queue."""
    lens = [700, 3, 1300, 0, 64]
    T = sum(lens)
    g = torch.Generator("cuda").manual_seed(5)
    q, k, v = (torch.randn(T, h, D, device="cuda", generator=g).to(BF16) for h in (hq, hk, hk))
    cu = torch.tensor([0] + lens, **I32).cumsum(0).int()
    out = iter([{"out": torch.full_like(q, 7.0), "lse": torch.full((T, hq), 7.0, device="cuda")} for _ in range(7)])

    def call():
        return sv.prompt_attention(q, k, v, cu, out=next(out))
    first_calls(call, call())

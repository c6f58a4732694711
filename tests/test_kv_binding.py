"""Devices of the cache operators' tensors: the library launches on the current one, so a tensor on
another is refused before any call. Tensors here are host memory that says where it would be."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from speculative_decoding_verification_33_gb300 import kvcache  # noqa: E402

BF16, I32, I64 = torch.bfloat16, torch.int32, torch.int64


class On(torch.Tensor):
    """A tensor that says it is on the CUDA device ``at``."""
    at = 0
    is_cuda = property(lambda self: True)

    def get_device(self):
        return self.at


def on(at, *shape, dtype=I32):
    t = torch.zeros(*shape, dtype=dtype).as_subclass(On)
    t.at = at
    return t


def tables(at):
    out = {n: on(at("out " + n), k, dtype=d) for n, k, d in (
        ("ctx_lens", 2, I32), ("held", 2, I32), ("counters", 2, I64), ("cu_new", 3, I32),
        ("kv_lens", 2, I32), ("status", 2, I32), ("slots", 4, I64), ("positions", 4, I32),
        ("seq_ids", 4, I32))}
    sv.block_tables(on(at("ctx_lens"), 2), on(at("new_lens"), 2), on(at("block_table"), 2, 3),
                    on(at("held"), 2), on(at("ring"), 8), on(at("counters"), 2, dtype=I64), page_size=16,
                    max_tokens=4, accept_len=on(at("accept_len"), 2), out=out)


def norm_rope(at):
    sv.qk_norm_rope(on(at("q"), 3, 2, 64, dtype=BF16), on(at("k"), 3, 1, 64, dtype=BF16), on(at("positions"), 3),
                    on(at("inv_freq"), 32, dtype=torch.float64), q_weight=on(at("q_weight"), 64, dtype=BF16),
                    k_weight=on(at("k_weight"), 64, dtype=BF16),
                    out={"q": on(at("out q"), 3, 2, 64, dtype=BF16), "k": on(at("out k"), 3, 1, 64, dtype=BF16)})


def append(at):
    sv.kv4_append(on(at("k"), 3, 1, 64, dtype=BF16), on(at("v"), 3, 1, 64, dtype=BF16),
                  on(at("slots"), 3, dtype=I64), on(at("cache"), 2, 1, 16 * 72, dtype=torch.uint8), page_size=16,
                  out={n: on(at("out " + n), 3, 1, 64, dtype=BF16) for n in "kv"})


def attention(at):
    sv.kv4_attention(on(at("q"), 3, 2, 64, dtype=BF16), on(at("cache"), 2, 1, 16 * 72, dtype=torch.uint8),
                     on(at("block_table"), 2, 3), on(at("kv_lens"), 2), on(at("cu_new"), 3), page_size=16,
                     out={"out": on(at("out"), 3, 2, 64, dtype=BF16), "lse": on(at("lse"), 3, 2, dtype=torch.float32)})


CALLS = {tables: ["ctx_lens", "new_lens", "block_table", "held", "ring", "counters", "accept_len", "out ctx_lens",
                  "out held", "out counters", "out cu_new", "out kv_lens", "out status", "out slots",
                  "out positions", "out seq_ids"],
         norm_rope: ["q", "k", "positions", "inv_freq", "q_weight", "k_weight", "out q", "out k"],
         append: ["k", "v", "slots", "cache", "out k", "out v"],
         attention: ["q", "cache", "block_table", "kv_lens", "cu_new", "out", "lse"]}


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_all_on_a_device_that_is_not_current(call, monkeypatch):
    monkeypatch.setattr(kvcache, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kvcache, "_several", True, raising=False)
    with pytest.raises(ValueError, match="device 1"):
        call(lambda name: 1)


@pytest.mark.parametrize("call,name", [(c, n) for c, ns in CALLS.items() for n in ns],
                         ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_one_on_another_device(call, name, monkeypatch):
    monkeypatch.setattr(kvcache, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kvcache, "_several", True, raising=False)
    with pytest.raises(ValueError, match="device"):
        call(lambda n: 1 if n == name else 0)


def test_host_tensors():
    x = torch.zeros(3, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.kv4_append(x, x, torch.zeros(3, dtype=I64), torch.zeros(2, 1, 16 * 72, dtype=torch.uint8), page_size=16)

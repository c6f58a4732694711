"""Devices, types and shapes of the tensors of the 8-bit cache's and the prompt's calls: what does not fit is
refused before any call. Tensors here are host memory that says where it would be."""
import pytest

torch = pytest.importorskip("torch")

import speculative_decoding_verification_33_gb300 as sv  # noqa: E402
from speculative_decoding_verification_33_gb300 import kvcache  # noqa: E402
from tests.test_kv_binding import BF16, I64, on  # noqa: E402


def append(at):
    sv.kv8_append(on(at("k"), 3, 1, 64, dtype=BF16), on(at("v"), 3, 1, 64, dtype=BF16),
                  on(at("slots"), 3, dtype=I64), on(at("cache"), 2, 1, 16 * 129, dtype=torch.uint8), page_size=16,
                  out={n: on(at("out " + n), 3, 1, 64, dtype=BF16) for n in "kv"})


def attention(at):
    sv.kv8_attention(on(at("q"), 3, 2, 64, dtype=BF16), on(at("cache"), 2, 1, 16 * 129, dtype=torch.uint8),
                     on(at("block_table"), 2, 3), on(at("kv_lens"), 2), on(at("cu_new"), 3), page_size=16,
                     out={"out": on(at("out"), 3, 2, 64, dtype=BF16), "lse": on(at("lse"), 3, 2, dtype=torch.float32)})


def prompt(at):
    sv.prompt_attention(on(at("q"), 3, 2, 64, dtype=BF16), on(at("k"), 3, 1, 64, dtype=BF16),
                        on(at("v"), 3, 1, 64, dtype=BF16), on(at("cu"), 3),
                        out={"out": on(at("out"), 3, 2, 64, dtype=BF16),
                             "lse": on(at("lse"), 3, 2, dtype=torch.float32)})


CALLS = {append: ["k", "v", "slots", "cache", "out k", "out v"],
         attention: ["q", "cache", "block_table", "kv_lens", "cu_new", "out", "lse"],
         prompt: ["q", "k", "v", "cu", "out", "lse"]}


@pytest.fixture
def two_devices(monkeypatch):
    monkeypatch.setattr(kvcache, "_current_device", lambda: 0, raising=False)
    monkeypatch.setattr(kvcache, "_several", True, raising=False)


@pytest.mark.parametrize("call", CALLS, ids=lambda f: f.__name__)
def test_all_on_a_device_that_is_not_current(call, two_devices):
    with pytest.raises(ValueError, match="device 1"):
        call(lambda name: 1)


@pytest.mark.parametrize("call,name", [(c, n) for c, ns in CALLS.items() for n in ns],
                         ids=lambda x: x if isinstance(x, str) else x.__name__)
def test_one_on_another_device(call, name, two_devices):
    with pytest.raises(ValueError, match="device"):
        call(lambda n: 1 if n == name else 0)


def test_shapes_and_types():
    q, k, cu = on(0, 3, 2, 64, dtype=BF16), on(0, 3, 1, 64, dtype=BF16), on(0, 3)
    with pytest.raises(TypeError):
        sv.prompt_attention(q.float(), k, k, cu)
    with pytest.raises(TypeError):
        sv.prompt_attention(q, k, k, on(0, 3, dtype=I64))
    for bad in (on(0, 2, 1, 64, dtype=BF16), on(0, 3, 1, 32, dtype=BF16), on(0, 3, 64, dtype=BF16)):
        with pytest.raises(ValueError):
            sv.prompt_attention(q, bad, bad, cu)
    with pytest.raises(ValueError):
        sv.prompt_attention(q, k, on(0, 3, 2, 64, dtype=BF16), cu)
    with pytest.raises(ValueError):
        sv.prompt_attention(on(0, 3, 64, 2, dtype=BF16).transpose(1, 2), k, k, cu)
    slots, cache = on(0, 3, dtype=I64), on(0, 2, 1, 16 * 129, dtype=torch.uint8)
    with pytest.raises(ValueError, match="cache"):
        sv.kv8_append(k, k, slots, on(0, 2, 1, 16 * 72, dtype=torch.uint8), page_size=16)  # the 4-bit one's size
    with pytest.raises(ValueError, match="cache"):
        sv.kv8_append(k, k, slots, cache, page_size=32)
    with pytest.raises(ValueError):
        sv.kv8_append(k, on(0, 3, 1, 128, dtype=BF16), slots, cache, page_size=16)
    with pytest.raises(TypeError):
        sv.kv8_append(k.half(), k.half(), slots, cache, page_size=16)
    with pytest.raises(TypeError):
        sv.kv8_attention(q.float(), cache, on(0, 2, 3), on(0, 2), cu, page_size=16)
    with pytest.raises(ValueError):
        sv.kv8_cache(2, 1, 96, 16)


def test_host_tensors():
    x = torch.zeros(3, 1, 64, dtype=BF16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.kv8_append(x, x, torch.zeros(3, dtype=I64), torch.zeros(2, 1, 16 * 129, dtype=torch.uint8), page_size=16)
    with pytest.raises(ValueError, match="CUDA tensor"):
        sv.prompt_attention(x, x, x, torch.zeros(2, dtype=torch.int32))

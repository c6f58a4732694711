"""The cache operators together: examples/cache_rounds.py decodes with drafts what it decodes without."""
import importlib.util
import os

import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():  # pragma: no cover - collected on CPU machines too
    pytest.skip("needs a CUDA GPU", allow_module_level=True)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
spec = importlib.util.spec_from_file_location("cache_rounds", os.path.join(ROOT, "examples", "cache_rounds.py"))
ex = importlib.util.module_from_spec(spec)
spec.loader.exec_module(ex)


def test_rounds_keep_the_tokens_and_the_pages():
    K = 4
    spec_run, accepted = ex.main(rounds=12, K=K)
    assert 0 <= accepted.min() and accepted.max() <= K and accepted.mean() > 0.3
    plain, _ = ex.main(rounds=40, K=0)
    # greedy verification keeps the model's own tokens; the two runs round differently (other
    # tiles, other matrix products), so a near-tie may part a sequence from there on
    same = total = 0
    for a, b in zip(spec_run.out, plain.out):
        n = min(len(a), len(b))
        same += next((i for i in range(n) if a[i] != b[i]), n)
        total += n
    assert same >= 0.8 * total, (same, total)
    # pages: each is free or held once
    live = [int(spec_run.ring[i % len(spec_run.ring)]) for i in range(*spec_run.counters.tolist())]
    held = [int(p) for b in range(len(spec_run.out)) for p in spec_run.table[b, :spec_run.held[b]]]
    assert sorted(live + held) == list(range(len(spec_run.ring)))

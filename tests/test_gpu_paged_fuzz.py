"""Random paged caches under random sequences of calls, against the float64 oracle: head
layouts, page sizes and types, batches in any order, prompts and single tokens, weights
with decay, evictions of one token and of many. Tolerances as in test_gpu_paged."""
import numpy as np
import pytest

from tests.gpu_common import device
from tests.test_gpu_paged import Pair

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


@pytest.mark.parametrize("case", range(48))
def test_random_calls(case):
    rng = np.random.default_rng(9000 + case)
    kv = int(rng.choice([1, 2, 3, 4, 5, 8, 16]))
    group = int(rng.integers(1, 17))
    d = int(rng.choice([64, 128]))
    page = int(rng.choice([16, 32, 48, 64, 80, 128, 1024]))
    n = int(rng.integers(1, 10))
    cap = int(np.exp(rng.uniform(np.log(page), np.log(6000))))
    max_pages = max(1, cap // page)
    p = Pair(kv * group, kv, d, page, n, max_pages, e4m3=bool(rng.integers(0, 2)), seed=case,
             junk=float(rng.choice([np.nan, np.inf, 0.0])))
    cap = max_pages * page
    for _ in range(8):
        seqs = rng.permutation(n)[: int(rng.integers(1, n + 1))].tolist()
        room = [cap - int(p.ora.length[s]) for s in seqs]
        kind = rng.choice(["prompt", "token", "none"])
        counts = [int(rng.integers(0, r + 1)) if kind == "prompt" else min(r, 1) if kind == "token" else 0 for r in room]
        p.append(seqs, counts)
        decay = None if rng.random() < 0.4 else float(rng.choice([0.0, 0.5, 1.0]))
        p.attend(seqs, decay=decay, qs=float(rng.choice([0.1, 1.5, 4.0])))
        top = max(int(p.ora.length[s]) for s in seqs)
        if rng.random() < 0.6 and top > 1:
            budget = int(rng.choice([top - 1, rng.integers(1, top)]))
            sink = int(rng.integers(0, budget // 2 + 1))
            recent = int(rng.integers(0, budget - sink + 1))
            p.cache.evict(budget, sink, recent, seqs=seqs)
            p.ora.evict(seqs, budget, sink, recent)
        if rng.random() < 0.1:
            p.cache.reset(seqs[:1])
            p.ora.reset(seqs[:1])
        p.check_state(range(n))
    p.ok()

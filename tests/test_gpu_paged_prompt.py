"""Attention of several new tokens per sequence over the paged cache, against the float64 oracle.

Tolerances as in test_gpu_paged, with a weight's rounding for its product with V: half a step of bf16 (2^-8, bf16
pages) or of fp16 (2^-11, or 2^-31 of the largest weight; e4m3 and 4-bit pages)."""
import numpy as np
import pytest
import torch

from tests.gpu_common import device
from tests.test_gpu_paged import E, U, f64
from tests.test_gpu_paged_int4 import _pair

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "int4"]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


def compare(p, kind, seqs, counts, q, o, lse, causal, visible=None):
    q64, g = f64(q), p.heads // p.kv
    ref, ref_lse, wv = p.ora.prompt_attention(seqs, counts, q64, causal, visible)
    o, lse = f64(o), f64(lse)
    r = 0
    for i, (s, m) in enumerate(zip(seqs, counts)):
        L = int(p.ora.length[s])
        seen = np.ones(L, bool) if visible is None else visible[i]
        ka, va = np.abs(p.ora.k[s, :L])[seen], np.abs(p.ora.v[s, :L])[seen]
        qa = np.abs(q64[r: r + m]).reshape(m, p.kv, g, p.d)
        dot = np.einsum("rhgd,thd->rhgt", qa, ka).max(3, initial=0.0).reshape(m, p.heads)
        dx = (p.d + 8) * U * p.ora.scale * dot
        rel = 2 * dx + L * U + 2.0 ** -20
        W = 2.0 ** -8 if kind == "bf16" else 2.0 ** -11
        bound = E * np.abs(ref[r: r + m]) + (W + rel[..., None]) * wv[r: r + m] + L * 2.0 ** -31 * va.max(initial=0.0) + 1e-30
        err = np.abs(o[r: r + m] - ref[r: r + m])
        assert np.all(err <= bound), (s, L, m, float((err / bound).max()))
        none = np.isinf(ref_lse[r: r + m])
        assert np.all(lse[r: r + m][none] == -np.inf) and np.all(o[r: r + m][none] == 0)
        with np.errstate(invalid="ignore"):
            tol = dx + L * U + 2.0 ** -20 + 4 * U * np.abs(ref_lse[r: r + m])
            off = np.abs(lse[r: r + m] - ref_lse[r: r + m])
        assert np.all((off <= tol) | none), (s, L, m)
        r += m


def prompt(p, kind, seqs, counts, causal=True, qs=1.5, visible=None):
    q = p.randn(sum(counts), p.heads, p.d, s=qs)
    out = torch.full_like(q, float("nan"))
    o, lse = p.cache.prompt_attention(q, counts, seqs=seqs, out=out, lse=True, causal=causal)
    assert o is out
    torch.cuda.synchronize()
    compare(p, kind, seqs, counts, q, o, lse, causal, visible)
    return q, o, lse


SHAPES = [  # heads, kv heads, d, page tokens
    (4, 4, 64, 16), (8, 1, 128, 64), (40, 8, 128, 64), (16, 1, 64, 48), (10, 5, 64, 32), (32, 2, 128, 16), (6, 2, 128, 128),
    (1, 1, 128, 16), (7, 1, 64, 64), (34, 2, 128, 32),
]
LENGTHS = [0, 1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 255, 257, 300, 511]


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_prompts_of_every_length(shape, kind, causal):
    """New tokens after others and none before them; one, a few and many; some sequences take no part."""
    heads, kv, d, page = shape
    n = len(LENGTHS)
    p = _pair(kind, heads, kv, d, page, n, -(-600 // page), seed=heads + d)
    p.append(list(range(n)), LENGTHS)
    seqs = p.rng.permutation(n).tolist()
    prompt(p, kind, seqs, [LENGTHS[s] if s % 2 else min(LENGTHS[s], 3) for s in seqs], causal)     # some from the first token on
    counts = [int(x) for x in p.rng.permutation([1, 1, 2, 3, 5, 7, 16, 17, 33, 40, 64, 80, 0, 4, 1, 2])]
    p.append(seqs, counts)
    prompt(p, kind, seqs, counts, causal)
    prompt(p, kind, seqs[:3], [min(9, int(p.ora.length[s])) for s in seqs[:3]], causal)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv,d,length,count,causal", [
    (8, 2, 128, 5003, 4, True), (5, 1, 64, 9001, 1, True), (16, 1, 128, 2500, 130, True), (4, 4, 64, 3001, 700, True),
    (2, 1, 128, 1100, 1100, True), (8, 8, 128, 2300, 300, False), (12, 3, 64, 4100, 33, False), (64, 1, 128, 1025, 40, True)])
def test_long_sequences_are_split_and_joined(kind, heads, kv, d, length, count, causal):
    p = _pair(kind, heads, kv, d, 64, 2, -(-length // 64), seed=length)
    p.append([0, 1], [length, 1])
    prompt(p, kind, [1, 0], [1, count], causal)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_many_ragged_sequences(kind):
    rng = np.random.default_rng(5)
    n = 70
    p = _pair(kind, 8, 2, 64, 16, n, 45, seed=3)
    lengths = [int(x) for x in rng.integers(0, 700, n)]
    p.append(list(range(n)), lengths)
    seqs = rng.permutation(n).tolist()
    prompt(p, kind, seqs, [int(rng.integers(0, min(lengths[s], 20) + 1)) for s in seqs])
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_sequences_shorter_than_their_rows(kind):
    """More query rows than the sequence has tokens: the first rows see nothing; not so without the mask."""
    p = _pair(kind, 8, 2, 64, 16, 3, 20, seed=4)
    p.append([0, 1, 2], [5, 0, 200])
    prompt(p, kind, [0, 1, 2], [9, 4, 260])
    prompt(p, kind, [2, 0, 1], [260, 9, 4], causal=False)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_bad_pages_are_left_out_and_reported(kind):
    from chunked_kv_cache_gb300 import _native as N
    p = _pair(kind, 8, 2, 128, 16, 3, 20, seed=7)
    p.append([0, 1, 2], [300, 100, 40])
    p.cache.block_table[0, 3] = -1
    p.cache.block_table[0, 17] = p.cache.n_pages
    p.cache.block_table[2] = -7
    seen = np.ones(300, bool)
    seen[48:64] = seen[272:288] = False
    prompt(p, kind, [0, 1, 2], [31, 100, 40], visible=[seen, np.ones(100, bool), np.zeros(40, bool)])
    assert p.cache.error_status() == N.SR_ERR_INVALID_ARG


@pytest.mark.parametrize("length", [40, 1500])
def test_rows_whose_scores_are_all_minus_infinity(length):
    p = _pair("bf16", 2, 2, 64, 16, 2, 100, seed=8)
    k, v, q = p.randn(length, 2, 64), p.randn(length, 2, 64), p.randn(20, 2, 64)
    k[:, 0, 0] = float("-inf")
    q[:, :, 0] = 1.0
    p.cache.append(k, v, counts=[length, 0])
    o, lse = p.cache.prompt_attention(q, [20, 0], lse=True)
    assert torch.all(o[:, 0] == 0) and torch.all(lse[:, 0] == float("-inf"))
    assert torch.isfinite(o[:, 1]).all() and torch.isfinite(lse[:, 1]).all()
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_numbers_that_are_none_stay_behind_the_mask(kind):
    """NaN among the last new tokens' values and keys reaches the rows that see them and no others; NaN in a query its row."""
    p = _pair(kind, 4, 2, 64, 16, 1, 20, seed=9)
    k, v, q = p.randn(200, 2, 64), p.randn(200, 2, 64), p.randn(100, 4, 64)
    v[190, 0] = float("nan")
    k[180, 1] = float("nan")
    q[50, 0] = float("nan")
    p.cache.append(k, v, counts=[200])
    o = p.cache.prompt_attention(q, [100])
    bad = torch.isnan(o).all(-1)
    want = torch.zeros(100, 4, dtype=torch.bool, device=o.device)
    want[90:, :2] = True
    want[80:, 2:] = True
    want[50, 0] = True
    assert torch.equal(bad, want) and torch.equal(torch.isnan(o).any(-1), want)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,heads,kv,length", [(64, 4, 2, 200), (128, 6, 2, 63), (128, 4, 1, 1500), (64, 1, 1, 7)])
def test_numbers_that_are_none_stay_behind_the_mask_of_a_few_rows(kind, d, heads, kv, length):
    """The same for drafts of 4 tokens; an infinity too, where pages hold it."""
    p = _pair(kind, heads, kv, d, 16, 2, 100, seed=9)
    k, v, q = p.randn(length, kv, d), p.randn(length, kv, d), p.randn(4, heads, d)
    v[length - 2] = float("nan")
    k[length - 1] = float("nan")
    v[length - 3, :, 5] = float("inf")
    p.cache.append(k, v, counts=[length, 0])
    o = p.cache.prompt_attention(q, [4, 0])
    nan, inf = torch.isnan(o), torch.isinf(o)
    assert not nan[:2].any() and nan[2:].all()
    assert not inf[0].any()
    if kind == "bf16":
        assert (o[1, :, 5] == float("inf")).all() and inf[1].sum() == heads
    else:
        assert not inf[1].any()                    # these pages saturate
    o = p.cache.prompt_attention(q, [4, 0], causal=False)
    assert torch.isnan(o).all()
    p.ok()


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("heads,kv,d,page,m", [(4, 4, 64, 16, 16), (32, 8, 128, 64, 4), (8, 1, 64, 48, 2), (5, 1, 128, 16, 3), (34, 2, 128, 32, 1),
                                               (3, 1, 64, 32, 5), (10, 2, 128, 128, 3)])
def test_a_few_rows_of_every_length(heads, kv, d, page, m, kind, causal):
    """Drafts whose heads fit one product: every number of rows up to m, lengths of one tile and several, empty ones."""
    n = len(LENGTHS)
    p = _pair(kind, heads, kv, d, page, n + 1, -(-2100 // page), seed=heads + d)
    seqs = p.rng.permutation(n + 1).tolist()
    p.append(list(range(n + 1)), LENGTHS + [2000])
    counts = [int(x) for x in p.rng.integers(0, m + 1, n + 1)]
    counts[0] = m
    prompt(p, kind, seqs, counts, causal)          # some sequences are shorter than their rows
    p.append(seqs, counts)
    prompt(p, kind, seqs, counts, causal)
    prompt(p, kind, seqs[:1], [m], causal, qs=30.0)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_large_scores_and_tiny_queries(kind):
    p = _pair(kind, 8, 2, 128, 32, 2, 20, seed=10, scale=0.7)
    p.append([0, 1], [600, 33])
    prompt(p, kind, [0, 1], [150, 33], qs=40.0)
    prompt(p, kind, [0, 1], [150, 33], qs=2.0 ** -80)
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_in_pieces_and_then_tokens(kind):
    """A run of the cache's calls as they are used: a prompt in three pieces, its attention each time, then single tokens by
    prompt_attention and by attention, weights, eviction, more tokens, reading back."""
    p = _pair(kind, 8, 2, 128, 16, 3, 30, seed=11)
    seqs = [2, 0, 1]
    for counts in ([100, 30, 0], [60, 129, 200], [1, 17, 64]):
        p.append(seqs, counts)
        prompt(p, kind, seqs, counts)
    for step in range(4):
        p.append(seqs, [1, 1, 1])
        prompt(p, kind, seqs, [1, 1, 1])
        p.attend(seqs, decay=1.0)
        p.cache.evict(150, 4, 20)
        p.ora.evict([0, 1, 2], 150, 4, 20)
    p.append(seqs, [5, 3, 8])
    prompt(p, kind, seqs, [5, 3, 8])
    p.check_state([0, 1, 2])
    k, v = p.cache.read([5, 3, 8], seqs=seqs)
    want = p.ora.read(seqs, [5, 3, 8])
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_captured_prompts(kind):
    """Captured on one stream, replayed later over longer sequences; two graphs and eager calls share the workspace."""
    p = _pair(kind, 16, 2, 128, 64, 4, 40, seed=12)
    seqs = [0, 1, 2, 3]
    p.append(seqs, [1000, 3, 0, 700])
    counts = [[4, 4, 4, 4], [130, 0, 70, 1]]
    qs = [p.randn(sum(c), 16, 128) for c in counts]
    ks = [p.randn(sum(c), 2, 128) for c in counts]
    side = torch.cuda.Stream(p.dev)
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [torch.cuda.CUDAGraph() for _ in counts], []
    with torch.cuda.stream(side):
        for graph, c, q, k in zip(graphs, counts, qs, ks):
            with torch.cuda.graph(graph, stream=side):
                p.cache.append(k, k, counts=c)
                outs.append(p.cache.prompt_attention(q, c, lse=True))
    torch.cuda.current_stream().wait_stream(side)
    for turn in (0, 1, 0, 0, 1):
        for x in (qs[turn], ks[turn]):
            x.copy_(p.randn(*x.shape))
        graphs[turn].replay()
        p.ora.append(seqs, counts[turn], f64(ks[turn]), f64(ks[turn]))
        torch.cuda.synchronize()
        compare(p, kind, seqs, counts[turn], qs[turn], *outs[turn], causal=True)
        o, lse = p.cache.prompt_attention(qs[turn], counts[turn], lse=True)
        assert torch.equal(o, outs[turn][0]) and torch.equal(lse, outs[turn][1])
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_results_do_not_depend_on_the_run_and_o_may_be_q(kind):
    p = _pair(kind, 40, 8, 128, 64, 5, 80, seed=13)
    p.append(list(range(5)), [5000, 100, 640, 64, 2222])
    counts = [37, 100, 260, 1, 4]
    q = p.randn(sum(counts), 40, 128)
    first = p.cache.prompt_attention(q, counts, lse=True)
    for _ in range(10):
        again = p.cache.prompt_attention(q, counts, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    same = q.clone()
    p.cache.prompt_attention(same, counts, out=same)
    assert torch.equal(same, first[0])
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
def test_nothing_is_written_outside_the_outputs(kind):
    p = _pair(kind, 10, 2, 64, 16, 3, 20, seed=14)
    p.append([0, 1, 2], [300, 77, 5])
    counts = [33, 77, 1]
    rows = sum(counts)
    buf = torch.full((rows + 64, 10, 64), -7.0, dtype=torch.bfloat16, device=p.dev)
    lse = torch.full((rows + 64, 10), -7.0, device=p.dev)
    q = p.randn(rows, 10, 64)
    before = [t.clone() for t in (p.cache.k_pages.view(torch.uint8), p.cache.v_pages.view(torch.uint8), p.cache.token_mass, p.cache.seq_len)]
    p.cache.prompt_attention(q, counts, out=buf[32: 32 + rows], lse=lse[32: 32 + rows])
    for t in (buf, lse):
        assert bool((t[:32] == -7).all()) and bool((t[32 + rows:] == -7).all()) and not bool((t[32: 32 + rows] == -7).any())
    after = (p.cache.k_pages.view(torch.uint8), p.cache.v_pages.view(torch.uint8), p.cache.token_mass, p.cache.seq_len)
    assert all(torch.equal(a, b) for a, b in zip(before, after))
    p.ok()


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("case", range(12))
def test_random_prompts(case, kind):
    rng = np.random.default_rng(700 + case)
    kv, group, d = int(rng.choice([1, 2, 3, 8])), int(rng.integers(1, 20)), int(rng.choice([64, 128]))
    page, n = int(rng.choice([16, 48, 64, 1024])), int(rng.integers(1, 9))
    pages = max(1, int(np.exp(rng.uniform(np.log(64), np.log(3000)))) // page)
    p = _pair(kind, kv * group, kv, d, page, n, pages, seed=case)
    cap = pages * page
    for _ in range(4):
        seqs = rng.permutation(n)[: int(rng.integers(1, n + 1))].tolist()
        counts = [int(rng.integers(0, min(cap - int(p.ora.length[s]), 300 // group + 3) + 1)) for s in seqs]
        p.append(seqs, counts)
        prompt(p, kind, seqs, counts, causal=bool(rng.integers(0, 2)), qs=float(rng.choice([0.1, 1.5, 4.0])))
    p.ok()

"""Attention of several new tokens on the paths that few calls take, against a plain form in 64 bits: numbers that are
none in whole, cut and merged blocks, many blocks to a CTA, outputs on any 16 bytes, batches of every size, prompts among
single tokens, one workspace for several caches.

The plain form computes from the tokens as the cache reads them back (exact, test_gpu_paged_int4). Tolerances are
test_gpu_paged_prompt's. Which outputs are NaN or infinite has to agree element by element."""
import numpy as np
import pytest
import torch

from tests.gpu_common import device

pytestmark = pytest.mark.gpu

KINDS = ["bf16", "e4m3", "int4"]
U, E = 2.0 ** -24, 2.0 ** -8
INF, NAN = float("inf"), float("nan")


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


class Calls:
    """A cache whose pages lie in no order, and what its attention should give."""

    def __init__(self, kind, heads, kv, d, n, cap, page=16, seed=0):
        import chunked_kv_cache_gb300 as sr
        self.kind, self.heads, self.kv, self.d, self.n = kind, heads, kv, d, n
        self.dev = device()
        self.g = torch.Generator(device=self.dev).manual_seed(seed)
        pages = -(-cap // page)
        table = torch.randperm(n * pages, generator=self.g, device=self.dev).to(torch.int32).view(n, pages)
        dtype = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn, "int4": "int4"}[kind]
        self.cache = sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=n * pages, max_seqs=n, max_pages=pages,
                                   page_dtype=dtype, device=self.dev, buffers=dict(block_table=table))
        self.len = [0] * n

    def randn(self, *shape, s=1.0):
        return (torch.randn(shape, generator=self.g, device=self.dev) * s).to(torch.bfloat16)

    def append(self, k, v, counts, seqs=None):
        self.cache.append(k, v, counts=counts, seqs=seqs)
        for i, c in enumerate(counts):
            self.len[i if seqs is None else seqs[i]] += c

    def plain(self, q, counts, seqs=None, causal=True):
        """o, lse and the bounds of their errors, fp64: [rows][heads][d], [rows][heads]."""
        out, r = [], 0
        scale, g = self.d ** -0.5, self.heads // self.kv
        for i, m in enumerate(counts):
            s = i if seqs is None else seqs[i]
            L = self.len[s]
            k, v = (x.double() for x in self.cache.read([L], seqs=[s]))
            x = q[r: r + m].double().view(m, self.kv, g, self.d)
            r += m
            t = torch.arange(L, device=self.dev)
            sees = t[None] <= torch.arange(m, device=self.dev)[:, None] + (L - m) if causal else torch.ones(m, L, dtype=torch.bool, device=self.dev)
            score = torch.einsum("rhgd,thd->rhgt", x, k) * scale
            score = torch.where(sees[:, None, None], score, -INF)
            lse = torch.logsumexp(score, -1) if L else torch.full(score.shape[:3], -INF, dtype=torch.float64, device=self.dev)
            w = torch.where((lse == -INF)[..., None], 0.0, torch.exp(score - lse[..., None]))
            vf = torch.where(torch.isfinite(v), v, 0.0)
            o = torch.einsum("rhgt,thd->rhgd", w, vf)
            wv = torch.einsum("rhgt,thd->rhgd", w, vf.abs())
            for j in torch.nonzero(~torch.isfinite(v).all(2).all(1)).flatten().tolist():
                odd = torch.where(torch.isfinite(v[j]), 0.0, v[j])[None, :, None]
                there = sees[:, j, None, None, None] & (lse != -INF)[..., None] & (odd != 0)
                o = o + torch.where(there, w[..., j, None] * odd, 0.0)
            dot = torch.einsum("rhgd,thd->rhgt", x.abs(), torch.where(torch.isfinite(k), k, 0.0).abs()).amax(-1) if L else torch.zeros_like(lse)
            dx = (self.d + 8) * U * scale * dot
            W = 2.0 ** -8 if self.kind == "bf16" else 2.0 ** -11
            bound = E * o.abs() + (W + 2 * dx + L * U + 2.0 ** -20)[..., None] * wv + L * 2.0 ** -31 * (vf.abs().max() if L else 0.0) + 1e-30
            tol = dx + L * U + 2.0 ** -20 + 4 * U * lse.abs()
            out.append([y.reshape(m, self.heads, *y.shape[3:]) for y in (o, lse, bound, tol)])
        return [torch.cat(y) for y in zip(*out)]

    def compare(self, q, counts, o, lse, seqs=None, causal=True):
        ref, ref_lse, bound, tol = self.plain(q, counts, seqs, causal)
        o = o.double()
        assert torch.equal(torch.isnan(o), torch.isnan(ref)), "NaN elsewhere"
        for inf in (INF, -INF):
            assert torch.equal(o == inf, ref == inf), "infinite elsewhere"
        fine = torch.isfinite(ref)
        err = (o - ref).abs()
        assert bool((err[fine] <= bound[fine]).all()), float((err / bound)[fine].max())
        none = ref_lse == -INF
        assert bool((lse.double() == ref_lse)[none].all()) and bool((o[none] == 0).all())
        assert bool(((lse.double() - ref_lse).abs() <= tol)[~none].all())

    def prompt(self, q, counts, seqs=None, causal=True):
        o, lse = self.cache.prompt_attention(q, counts, seqs=seqs, lse=True, causal=causal)
        self.compare(q, counts, o, lse, seqs, causal)
        assert self.cache.error_status() == 0
        return o, lse


@pytest.mark.parametrize("low", [0, 1])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,kv,n", [(64, 1, 1), (128, 1, 1), (64, 16, 40), (128, 8, 40)])
def test_nan_under_scores_that_leave_its_weight_at_zero(d, kv, n, kind, low):
    """Rows of one query tile: the groups that share the key tiles merge sums of which one is lighter by far more than
    2^-126. A NaN among its values is still one."""
    p = Calls(kind, kv, kv, d, n, 320, seed=d + n)
    length, m = 256 + 40, 40
    k, v, q = p.randn(n * length, kv, d, s=0.1), p.randn(n * length, kv, d), p.randn(n * m, kv, d, s=0.1)
    q[..., 0] = 256.0
    tile = torch.arange(length, device=p.dev) // 128
    k.view(n, length, kv, d)[..., 0] = torch.where(tile % 2 == low, -8.0, 8.0)[None, :, None]
    v.view(n, length, kv, d)[::2, 128 * low + 10, :, 3] = NAN
    p.append(k, v, [length] * n)
    o, _ = p.prompt(q, [m] * n)
    assert bool(torch.isnan(o[:m]).any(-1).all())


# d, key heads, query heads of each, sequences, tokens before the new ones, new ones
SHAPES = [
    (64, 16, 1, 128, 60, 40),       # one query tile, 13 blocks to a CTA
    (128, 16, 1, 128, 126, 256),    # two, and new tokens in three key tiles
    (64, 16, 1, 96, 254, 256),
    (128, 8, 4, 64, 100, 50),
    (64, 2, 8, 256, 0, 33),         # as many sequences as a call takes
    (128, 4, 3, 20, 300, 130),      # several blocks to a sequence
    (128, 1, 2, 3, 1000, 200),      # cut blocks
]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("shape", SHAPES)
def test_numbers_that_are_none_among_the_new_tokens(shape, kind):
    """NaN and infinities in some sequences' new values reach the rows that see them, and no row of a sequence without."""
    d, kv, group, n, base, m = shape
    p = Calls(kind, kv * group, kv, d, n, base + m, seed=base + m)
    length = base + m
    k, v, q = p.randn(n * length, kv, d), p.randn(n * length, kv, d), p.randn(n * m, kv * group, d)
    each = v.view(n, length, kv, d)
    rng = np.random.default_rng(n)
    for s in range(n):
        for j in rng.integers(1, m, 3 if s % 3 else 0).tolist() + ([m - 1, m - 2] if s % 3 == 2 else []):
            each[s, base + j, int(rng.integers(kv)), int(rng.integers(d))] = [NAN, INF, -INF][int(rng.integers(3))]
    p.append(k, v, [length] * n)
    o, lse = p.prompt(q, [m] * n)
    p.prompt(q, [m] * n, causal=False)
    same = q.clone()                                  # in the queries' place
    p.cache.prompt_attention(same, [m] * n, out=same)
    assert torch.equal(same.view(torch.int16), o.view(torch.int16))


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("d,kv,group,m", [(64, 2, 4, 4), (128, 1, 1, 5), (128, 2, 8, 2)])
def test_numbers_that_are_none_among_a_few_rows(d, kv, group, m, kind):
    """The same where the rows are few enough for the kernel of single tokens; 256 sequences."""
    n, length = 256, 70
    p = Calls(kind, kv * group, kv, d, n, length, seed=d + m)
    k, v, q = p.randn(n * length, kv, d), p.randn(n * length, kv, d), p.randn(n * m, kv * group, d)
    each = v.view(n, length, kv, d)
    for s in range(n):
        if s % 2:
            each[s, length - 1 - s // 2 % (m - 1), s % kv, s % d] = [NAN, INF, -INF][s % 3]
    p.append(k, v, [length] * n)
    o, _ = p.prompt(q, [m] * n)
    same = q.clone()
    p.cache.prompt_attention(same, [m] * n, out=same)
    assert torch.equal(same.view(torch.int16), o.view(torch.int16))


@pytest.mark.parametrize("length,m", [(40, 1), (40, 4), (40, 20), (3000, 1), (3000, 4), (3000, 40), (600, 300)])
def test_rows_whose_scores_are_all_minus_infinity_over_values_that_are_none(length, m):
    """o = 0 and lse = -inf whatever the values are, in sequences taken whole and in ones cut into parts; by prompt_attention
    and, for one token, by attention."""
    p = Calls("bf16", 4, 2, 64, 5, length, seed=length + m)
    k, v, q = p.randn(5 * length, 2, 64), p.randn(5 * length, 2, 64), p.randn(5 * m, 4, 64)
    k[:, 0, 0] = -INF
    q[:, :, 0] = 1.0
    v.view(5, length, 2, 64)[:, :, 0, 7] = NAN
    v.view(5, length, 2, 64)[:, length // 2, 0, 9] = INF
    p.append(k, v, [length] * 5)
    calls = [lambda: p.cache.prompt_attention(q, [m] * 5, lse=True), lambda: p.cache.prompt_attention(q, [m] * 5, lse=True, causal=False)]
    if m == 1:
        calls += [lambda: p.cache.attention(q, lse=True), lambda: p.cache.attention(q, lse=True, mass_decay=1.0),
                  lambda: p.cache.attention(q[:1], lse=True)]
    for call in calls:
        o, lse = call()
        assert bool((o[:, :2] == 0).all()) and bool((lse[:, :2] == -INF).all())
        assert bool(torch.isfinite(o[:, 2:]).all()) and bool(torch.isfinite(lse[:, 2:]).all())


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("counts", [[200, 77, 33, 300], [4, 1, 0, 3]])
def test_queries_and_outputs_on_any_16_bytes(counts, kind):
    p = Calls(kind, 8, 2, 128, 4, 700, seed=3)
    p.append(p.randn(4 * 400, 2, 128), p.randn(4 * 400, 2, 128), [400] * 4)
    rows = sum(counts)
    q = p.randn(rows, 8, 128)
    want, want_lse = p.prompt(q, counts)
    for shift in (8, 16, 24):
        flat = [torch.full((rows * 1024 + 64,), -7.0, dtype=torch.bfloat16, device=p.dev) for _ in range(2)]
        qs, out = (x[shift: shift + rows * 1024].view(rows, 8, 128) for x in flat)
        lse = torch.full((rows * 8 + 3,), -7.0, device=p.dev)
        qs.copy_(q)
        p.cache.prompt_attention(qs, counts, out=out, lse=lse[1: 1 + rows * 8].view(rows, 8))
        assert torch.equal(out, want) and torch.equal(lse[1: 1 + rows * 8].view(rows, 8), want_lse)
        assert bool((flat[1][:shift] == -7).all()) and bool((flat[1][shift + rows * 1024:] == -7).all())
        assert float(lse[0]) == -7 and bool((lse[1 + rows * 8:] == -7).all())
    assert p.cache.error_status() == 0


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("kind", KINDS)
def test_a_prompt_among_single_tokens_and_drafts(kind, causal):
    """What a server's step holds: one prompt, single tokens, drafts, a sequence that waits; the same rows alone agree to
    the bounds of both kernels."""
    p = Calls(kind, 16, 4, 128, 40, 1300, page=64, seed=6)
    before = [int(x) for x in np.random.default_rng(6).integers(0, 700, 40)]
    p.append(p.randn(sum(before), 4, 128), p.randn(sum(before), 4, 128), before)
    counts = [1] * 40
    counts[7], counts[8], counts[9], counts[21] = 513, 4, 0, 3
    p.append(p.randn(sum(counts), 4, 128), p.randn(sum(counts), 4, 128), counts)
    q = p.randn(sum(counts), 16, 128)
    p.prompt(q, counts, causal=causal)
    seqs = [s for s in range(40) if s != 7]
    few = [counts[s] for s in seqs]
    alone = torch.cat([q[:7], q[7 + 513:]])
    p.prompt(alone, few, seqs, causal)


def test_caches_whose_calls_do_not_overlap_share_a_workspace():
    """Layers of several shapes and page types on one workspace, their calls in turn, captured ones among them: bit for bit what
    each gives on its own."""
    import chunked_kv_cache_gb300 as sr
    dev = device()
    g = torch.Generator(device=dev).manual_seed(1)
    shapes = [(32, 8, 128, torch.bfloat16, 64), (4, 4, 64, "int4", 16), (8, 1, 128, torch.float8_e4m3fn, 32), (16, 2, 64, torch.bfloat16, 16)]

    def layers(shared):
        out = []
        for heads, kv, d, dtype, page in shapes:
            own = {} if not shared or not out else dict(workspace=out[0].workspace)
            out.append(sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=4 * (4096 // page), max_seqs=4, max_pages=4096 // page,
                                     page_dtype=dtype, device=dev, buffers=own))
            for s in range(4):
                out[-1].reserve(s, 4096)
        return out

    both = [layers(False), layers(True)]
    need = [c.workspace.numel() for c in both[0]]
    assert need[0] == max(need) and all(c.workspace is both[1][0].workspace for c in both[1])
    with pytest.raises(ValueError):
        heads, kv, d, dtype, page = shapes[0]
        sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=4 * (4096 // page), max_seqs=4, max_pages=4096 // page,
                      device=dev, buffers=dict(workspace=both[1][0].workspace[256:]))

    def step(c, k, v, q, counts):
        c.append(k, v, counts=counts)
        out = list(c.prompt_attention(q, counts, lse=True))
        out += c.attention(q[:4], lse=True, mass_decay=0.5)
        c.evict(1500, n_sink=4, n_recent=64)
        return out + [c.seq_len.clone(), c.token_mass.clone()]

    for counts in ([1700, 33, 0, 600], [130, 1, 70, 900], [4, 4, 4, 4], [1, 1, 1, 1]):
        for i, (heads, kv, d, _, _) in enumerate(shapes):
            rows = sum(counts)
            k, v, q = ((torch.randn(rows, h, d, generator=g, device=dev)).to(torch.bfloat16) for h in (kv, kv, heads))
            for a, b in zip(step(both[0][i], k, v, q, counts), step(both[1][i], k, v, q, counts)):
                assert torch.equal(a, b)
    x = [torch.randn(4, h, d, generator=g, device=dev).to(torch.bfloat16) for h, d in [(8, 128), (32, 128), (4, 64), (4, 64)]]
    side, graph = torch.cuda.Stream(dev), torch.cuda.CUDAGraph()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        got = step(both[1][0], x[0], x[0], x[1], [1] * 4) + step(both[1][1], x[2], x[2], x[3], [1] * 4)
    torch.cuda.current_stream().wait_stream(side)
    graph.replay()
    want = step(both[0][0], x[0], x[0], x[1], [1] * 4) + step(both[0][1], x[2], x[2], x[3], [1] * 4)
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    for c in both[0] + both[1]:
        assert c.error_status() == 0
        c.close()

"""The paged token cache on the GPU against its float64 oracle.

Tolerances, from the arithmetic (u = 2^-24, e = 2^-8 the half step of bf16):
* an output is rounded to bf16 (e |o|). A weight meets V as two bf16 numbers, the first
  rounded from (1 - 2^-8) of it, so that at most 2^-8 + 2^-8 of it is left for the second, whose
  rounding loses 2^-8 of that: 2^-15 of the weight (bf16 pages); or as fp16, which rounds it by 2^-11 of itself or, below
  fp16's normal numbers, by 2^-31 of the largest weight (e4m3 pages): W sum w|v| and
  L 2^-31 max|v|. fp32 scores, exponentials and sums add
  (2 dx + L u + 2^-20) sum w|v|, with dx the error of a scaled score:
  (d + 8) u * scale * max_t sum_i |q_i k_i(t)|, and 2^-22 for the exponential.
* the log-sum-exp is off by dx + L u + 2^-20 + 4 u |lse|.
* a weight is off by (2 dx + L u + 2^-20) of itself, and the accumulated weight by
  that and 4 u of itself.
Copies (pages, positions), lengths and the choice of what to evict are exact; the
choice is made by the oracle from the weights that the GPU holds.
"""
import numpy as np
import pytest
import torch

from oracle.paged import OraclePagedCache
from tests.gpu_common import device

pytestmark = pytest.mark.gpu

U, E = 2.0 ** -24, 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


def f64(t):
    return t.detach().double().cpu().numpy() if t.dtype != torch.float8_e4m3fn else t.float().double().cpu().numpy()


class Pair:
    """A GPU cache and its oracle; stale pages are filled with `junk`."""

    def __init__(self, heads, kv, d, page, max_seqs, max_pages, e4m3=False, seed=0, spare=3, junk=float("nan"),
                 mass=True, scale=0.0):
        import chunked_kv_cache_gb300 as sr
        self.dev = device()
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator(device=self.dev).manual_seed(seed)
        self.page, self.kv, self.d, self.heads = page, kv, d, heads
        n_pages = max_seqs * max_pages + spare
        exps = torch.from_numpy(self.rng.integers(-5, 3, (2, kv)).astype(np.int32)).to(self.dev)
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        pool = [torch.full((n_pages, page, kv, d), junk, device=self.dev).to(dtype) for _ in range(2)]
        self.table = self.rng.permutation(n_pages)[: max_seqs * max_pages].reshape(max_seqs, max_pages)
        self.cache = sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=max_seqs,
                                   max_pages=max_pages, page_dtype=dtype, device=self.dev, mass=mass,
                                   softmax_scale=scale,
                                   buffers=dict(k_pages=pool[0], v_pages=pool[1], kv_exp=exps, block_table=torch.from_numpy(
                                       self.table.astype(np.int32)).to(self.dev)))
        self.ora = OraclePagedCache(heads, kv, d, max_seqs, max_pages * page, e4m3, exps.cpu().numpy(),
                                    scale if scale > 0 else None)
        self.exps = exps.cpu().numpy()

    def randn(self, *shape, s=1.0):
        return (torch.randn(shape, generator=self.g, device=self.dev) * s).to(torch.bfloat16)

    def append(self, seqs, counts):
        rows = int(sum(counts))
        k, v = self.randn(rows, self.kv, self.d), self.randn(rows, self.kv, self.d)
        self.cache.append(k, v, seqs=seqs, counts=counts)
        self.ora.append(seqs, counts, f64(k), f64(v))

    def check_state(self, seqs):
        torch.cuda.synchronize()
        length, nxt = self.cache.seq_len.cpu().numpy(), self.cache.seq_pos.cpu().numpy()
        pos = self.cache.token_pos.cpu().numpy()
        k, v = f64(self.cache.k_pages), f64(self.cache.v_pages)
        if self.ora.e4m3:
            k, v = k * (2.0 ** self.exps[0])[:, None], v * (2.0 ** self.exps[1])[:, None]
        for s in seqs:
            n = int(self.ora.length[s])
            assert length[s] == n and nxt[s] == self.ora.next_pos[s], s
            assert np.array_equal(pos[s, :n], self.ora.pos[s, :n]), s
            t = np.arange(n)
            pg = self.table[s][t // self.page]
            assert np.array_equal(k[pg, t % self.page], self.ora.k[s, :n], equal_nan=True), s
            assert np.array_equal(v[pg, t % self.page], self.ora.v[s, :n], equal_nan=True), s

    def attend(self, seqs, decay=None, qs=1.5, visible=None):
        n = len(seqs)
        q = self.randn(n, self.heads, self.d, s=qs)
        out = torch.full_like(q, float("nan"))
        o, lse = self.cache.attention(q, seqs=seqs, out=out, lse=True, mass_decay=decay)
        torch.cuda.synchronize()
        q64, g = f64(q), self.heads // self.kv
        ref, ref_lse, wv = self.ora.attention(seqs, q64, decay, visible)
        o, lse = f64(o), f64(lse)
        mass = f64(self.cache.token_mass) if decay is not None else None
        for i, s in enumerate(seqs):
            L = int(self.ora.length[s])
            qa = np.abs(q64[i]).reshape(self.kv, g, self.d)
            ka = np.abs(self.ora.k[s, :L])
            if visible is not None:
                ka = ka[visible[i]]
            dot = np.einsum("hgd,thd->hgt", qa, ka).max(2, initial=0.0).reshape(self.heads)
            dx = (self.d + 8) * U * self.ora.scale * dot
            rel = 2 * dx + L * U + 2.0 ** -20
            W = 2.0 ** -11 if self.ora.e4m3 else 2.0 ** -15
            top_v = np.abs(self.ora.v[s, :L]).max(initial=0.0) if visible is None else np.abs(self.ora.v[s, :L][visible[i]]).max(initial=0.0)
            bound = E * np.abs(ref[i]) + (W + rel[:, None]) * wv[i] + L * 2.0 ** -31 * top_v + 1e-30
            err = np.abs(o[i] - ref[i])
            assert np.all(err <= bound), (s, L, float((err / bound).max()))
            if L == 0 or (visible is not None and not visible[i].any()):
                assert np.all(lse[i] == -np.inf)
            else:
                tol = dx + L * U + 2.0 ** -20 + 4 * U * np.abs(ref_lse[i])
                assert np.all(np.abs(lse[i] - ref_lse[i]) <= tol), (s, L, float((np.abs(lse[i] - ref_lse[i]) / tol).max()))
            if decay is not None:
                m = self.ora.mass[s, :L]
                tol = (float(rel.max()) + 4 * U) * np.abs(m) + 1e-30
                assert np.all(np.abs(mass[s, :L] - m) <= tol), (s, L)
        if mass is not None:      # what the oracle chooses by from here on
            for s in seqs:
                L = int(self.ora.length[s])
                self.ora.mass[s, :L] = mass[s, :L]
        return o, lse

    def ok(self):
        assert self.cache.error_status() == 0


SHAPES = [  # heads, kv heads, d, page tokens
    (4, 4, 64, 16), (8, 1, 128, 64), (40, 8, 128, 64), (16, 1, 64, 48), (10, 5, 64, 32), (32, 2, 128, 16),
    (6, 2, 128, 128), (1, 1, 128, 16),
]
LENGTHS = [0, 1, 2, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 300, 511]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("shape", SHAPES)
def test_append_and_attend_every_length(shape, e4m3):
    heads, kv, d, page = shape
    n = len(LENGTHS)
    p = Pair(heads, kv, d, page, n, -(-512 // page), e4m3, seed=heads * 7 + d)
    seqs = p.rng.permutation(n).tolist()
    p.append(seqs, [LENGTHS[s] for s in seqs])
    p.check_state(range(n))
    p.attend(seqs)
    p.attend(seqs[::-1][:5], decay=1.0)
    p.append(seqs[:7], [1] * 7)                 # token by token
    p.attend(seqs[:7], decay=0.5)
    p.check_state(range(n))
    p.ok()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv,d,length", [(5, 1, 128, 20011), (16, 2, 64, 9001), (4, 4, 128, 4097)])
def test_one_long_sequence_is_split_and_joined(heads, kv, d, length, e4m3):
    p = Pair(heads, kv, d, 64, 2, -(-length // 64), e4m3, seed=5)
    p.append([1], [length])
    p.attend([1], decay=1.0)
    p.attend([1], decay=0.25)
    p.ok()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv,d", [(4, 1, 128), (8, 1, 64), (16, 1, 64), (6, 3, 64)])
def test_one_long_sequence_among_many_short_ones(heads, kv, d, e4m3):
    """The long one is cut into far more parts than the batch's size lets expect."""
    n, long = 48, 20011
    p = Pair(heads, kv, d, 64, n, -(-long // 64), e4m3, seed=22)
    counts = [s % 4 for s in range(n)]
    counts[17] = long
    p.append(list(range(n)), counts)
    p.attend(list(range(n)), decay=1.0)
    p.attend(list(range(n)), decay=0.5)
    p.ok()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("heads,kv,d,lengths", [
    (32, 1, 128, [300, 0, 17, 1000]), (34, 2, 64, [65, 129, 1]), (71, 1, 64, [500, 40]), (128, 4, 128, [2000, 1, 333]),
    (96, 3, 128, [9000]), (40, 2, 64, [700] * 20), (512, 1, 128, [130, 70]), (1024, 1, 64, [90]),
])
def test_more_query_heads_than_one_read_serves(heads, kv, d, lengths, e4m3):
    n = len(lengths)
    p = Pair(heads, kv, d, 64, n, -(-max(lengths) // 64) + 1, e4m3, seed=heads + n)
    seqs = p.rng.permutation(n).tolist()
    p.append(seqs, [lengths[s] for s in seqs])
    p.attend(seqs, decay=1.0)
    p.append(seqs, [1] * n)
    p.attend(seqs[::-1], decay=0.5)
    p.cache.evict(max(lengths) // 2, 3, 5)
    p.ora.evict(range(n), max(lengths) // 2, 3, 5)
    p.check_state(range(n))
    p.attend(seqs)
    p.ok()


def test_many_sequences_of_unequal_length():
    n = 256
    p = Pair(8, 2, 64, 16, n, 20, seed=6)
    counts = [int(x) for x in p.rng.integers(0, 320, n)]
    counts[:6] = [0, 320, 1, 0, 0, 319]
    p.append(list(range(n)), counts)
    p.check_state(range(n))
    p.attend(list(range(n)), decay=1.0)
    p.ok()


@pytest.mark.parametrize("e4m3,d", [(False, 128), (True, 128), (False, 64), (True, 64)])
@pytest.mark.parametrize("heads,kv,lengths", [
    (32, 8, [512] * 32),                             # one item for each CTA
    (32, 8, [512] * 20 + [0] * 3 + [1, 500] + [0] * 7),
    (8, 8, [70] * 100 + [0, 0, 71, 1] * 3),          # several items for each
    (4, 1, [33] * 256),
    (3, 3, [40] * 251 + [0] * 5),
    (8, 2, [2500] * 12),                             # items in equal pieces
    (8, 2, [2500] * 9 + [0, 1, 130]),                # and some that have fewer tiles than pieces
    (40, 8, [768, 0, 767, 500, 700, 768] * 2),
    (5, 1, [6000]), (5, 1, [6000, 5990]), (16, 1, [0, 9000, 0]),
    (12, 4, [1200, 1, 1199, 64, 0, 1000, 650]),      # neither
])
def test_batches_of_nearly_equal_sequences(heads, kv, lengths, e4m3, d):
    n = len(lengths)
    p = Pair(heads, kv, d, 64, n, -(-max(lengths) // 64) + 1, e4m3, seed=sum(lengths) % 97)
    seqs = list(range(n))
    p.append(seqs, lengths)
    p.attend(seqs, decay=1.0)
    p.append(seqs, [1] * n)                          # lengths of one tile more, empty ones that have a token now
    p.attend(seqs)
    p.attend(seqs[::-1], decay=0.5)
    p.ok()


@pytest.mark.parametrize("e4m3,d,heads,kv,n,pages", [(False, 128, 8, 8, 16, 256), (False, 64, 16, 1, 40, 52), (True, 128, 5, 1, 48, 144),
                                                      (True, 64, 12, 4, 64, 44)])
def test_weights_of_large_batches(e4m3, d, heads, kv, n, pages):
    """Batches from 2^21 scores on drop them from the cache once read: every later call stores them anew."""
    cap = 64 * pages
    assert n * cap * heads >= 1 << 21
    p = Pair(heads, kv, d, 64, n, pages, e4m3, seed=d + n)
    lengths = [int(x) for x in p.rng.integers(1, 400, n)]
    lengths[:4] = [cap - 3, 0, 128, 1000]
    seqs = list(range(n))
    p.append(seqs, lengths)
    p.attend(seqs, decay=1.0)
    p.attend(seqs[::-1], decay=0.5)
    p.append(seqs[:4], [1, 1, 1, 129])
    p.attend(seqs[:n // 2], decay=1.0)
    p.attend(seqs, decay=0.75)
    p.ok()


def test_large_scores_and_scale():
    """Scores of several hundred: one token holds nearly all weight."""
    p = Pair(4, 2, 128, 32, 3, 8, seed=7, scale=0.7)
    p.append([0, 1, 2], [200, 1, 77])
    p.attend([0, 1, 2], decay=1.0, qs=8.0)
    p.ok()


def test_results_do_not_depend_on_the_run():
    p = Pair(40, 8, 128, 64, 5, 40, seed=8)
    p.append([0, 1, 2, 3, 4], [2500, 0, 3, 64, 1111])
    q = p.randn(5, 40, 128)
    first = None
    for _ in range(6):
        p.cache.token_mass.zero_()
        o, lse = p.cache.attention(q, lse=True, mass_decay=1.0)
        got = (o.clone(), lse.clone(), p.cache.token_mass.clone())
        first = first or got
        assert all(torch.equal(a, b) for a, b in zip(first, got))
    o2 = p.cache.attention(q)
    assert torch.equal(o2, first[0])


def test_empty_batch_of_empty_sequences():
    p = Pair(4, 1, 64, 16, 3, 2, seed=9)
    o, lse = p.attend([0, 1, 2], decay=1.0)
    assert not o.any() and np.all(lse == -np.inf)
    p.cache.evict(4)
    p.check_state(range(3))
    p.ok()


def test_values_in_unused_rows_do_not_matter():
    for junk in (float("inf"), float("-inf"), float("nan"), torch.finfo(torch.bfloat16).min):
        p = Pair(8, 2, 128, 64, 2, 3, seed=10, junk=junk)
        p.append([0, 1], [65, 130])
        p.attend([0, 1], decay=1.0)
        p.ok()


def test_bad_pages_are_left_out_and_reported():
    """Entries that are no page of the pool: their tokens are not seen, err_word says so."""
    p = Pair(4, 2, 64, 16, 2, 6, seed=11)
    p.append([0, 1], [90, 40])
    p.cache.block_table[0, 1] = -1
    p.cache.block_table[0, 4] = p.cache.n_pages
    vis0 = np.ones(90, bool)
    vis0[16:32] = vis0[64:80] = False
    p.attend([0, 1], visible=[vis0, np.ones(40, bool)])
    from chunked_kv_cache_gb300 import _native as N
    assert p.cache.error_status() == N.SR_ERR_INVALID_ARG
    assert int(p.cache.err_word.item()) == N.SR_DEVERR_BAD_PAGE
    # nothing but bad pages: an empty row
    p.cache.block_table[1, :] = -7
    p.attend([1], visible=[np.zeros(40, bool)])


def test_append_is_all_or_nothing():
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 2, 64, 16, 3, 4, seed=12)
    p.append([0, 1, 2], [60, 10, 63])
    before = [t.clone() for t in (p.cache.k_pages, p.cache.v_pages)]
    k, v = p.randn(8, 2, 64), p.randn(8, 2, 64)
    p.cache.append(k, v, seqs=[0, 2], counts=[5, 3])       # 65 of 64; 66 of 64
    assert p.cache.error_status() == N.SR_ERR_STATE and int(p.cache.err_word.item()) == N.SR_DEVERR_CACHE_FULL
    assert p.cache.seq_len.tolist() == [60, 10, 63] and p.cache.seq_pos.tolist() == [60, 10, 63]
    for a, b in zip(before, (p.cache.k_pages, p.cache.v_pages)):
        assert torch.equal(a.view(torch.int16), b.view(torch.int16))
    p.cache.err_word.zero_()
    p.cache.block_table[1, 2] = -1
    p.cache.append(k, v, seqs=[1, 0], counts=[6, 2])       # tokens 10..15 fit, 60 and 61 do
    assert p.cache.error_status() == 0 and p.cache.seq_len.tolist() == [62, 16, 63]
    k, v = p.randn(40, 2, 64), p.randn(40, 2, 64)
    p.cache.append(k, v, seqs=[1], counts=[40])            # 16 .. 55 touches the unmapped page 2
    assert int(p.cache.err_word.item()) == N.SR_DEVERR_BAD_PAGE and p.cache.seq_len.tolist() == [62, 16, 63]


@pytest.mark.parametrize("n,budget,sink,recent", [
    (300, 128, 4, 32), (300, 299, 0, 0), (300, 1, 0, 1), (300, 1, 0, 0), (65, 64, 8, 56), (1500, 1024, 100, 300),
    (5000, 17, 3, 5), (2049, 2048, 0, 2048), (33, 32, 32, 0),
])
@pytest.mark.parametrize("kind", ["spread", "ties", "odd"])
def test_evict_is_exact(n, budget, sink, recent, kind):
    p = Pair(2, 1, 64, 16, 3, -(-n // 16), seed=n + budget)
    p.append([0, 2], [n, budget])               # sequence 2 is already within the budget, 1 is empty
    m = p.rng.lognormal(0, 2, (3, p.cache.capacity)).astype(np.float32)
    if kind == "ties":
        m = np.floor(p.rng.random(m.shape) * 4).astype(np.float32)
        m[m == 0] = np.where(p.rng.random((m == 0).sum()) < 0.5, 0.0, -0.0)
    if kind == "odd":
        pick = p.rng.integers(0, 9, m.shape)
        m[pick == 0], m[pick == 1], m[pick == 2], m[pick == 3] = np.nan, np.inf, -np.inf, -3.0
        m[pick == 4], m[pick == 5] = -np.nan, 1e-42
    p.cache.token_mass.copy_(torch.from_numpy(m))
    p.ora.mass[:] = m
    behind = p.cache.token_pos.clone()
    p.cache.evict(budget, sink, recent)
    p.ora.evict(range(3), budget, sink, recent)
    p.check_state(range(3))
    got = p.cache.token_mass.cpu().numpy()
    new = int(p.ora.length[0])
    assert np.array_equal(got[0, :new], p.ora.mass[0, :new].astype(np.float32), equal_nan=True)
    # nothing behind the new length was touched
    assert np.array_equal(got[0, new:], m[0, new:], equal_nan=True) and np.array_equal(got[1:], m[1:], equal_nan=True)
    assert torch.equal(p.cache.token_pos[:, new:], behind[:, new:])
    p.ok()


@pytest.mark.parametrize("kind", ["spread", "ties", "protected"])
@pytest.mark.parametrize("lengths,budget", [([2, 1, 3, 2], 1), ([257, 256, 300, 257], 256), ([4608, 4607, 4608], 4607),
                                            ([4609, 4608, 4700, 4609], 4608), ([9001, 9000, 9001], 9000)])
def test_evict_one_token(lengths, budget, kind):
    """One token too many takes a path of its own, in one CTA or a cluster, beside sequences that lose more or none."""
    n = len(lengths)
    p = Pair(2, 1, 64, 16, n, -(-max(lengths) // 16), seed=budget)
    p.append(list(range(n)), lengths)
    m = p.rng.lognormal(0, 2, (n, p.cache.capacity)).astype(np.float32)
    if kind == "ties":
        m = np.floor(p.rng.random(m.shape) * 3).astype(np.float32)
    p.cache.token_mass.copy_(torch.from_numpy(m))
    p.ora.mass[:] = m
    sink, recent = (budget // 2, budget - budget // 2) if kind == "protected" else (min(4, budget), 0)
    p.cache.evict(budget, sink, recent)
    p.ora.evict(range(n), budget, sink, recent)
    p.check_state(range(n))
    got = p.cache.token_mass.cpu().numpy()
    for s in range(n):
        new = int(p.ora.length[s])
        assert np.array_equal(got[s, :new], p.ora.mass[s, :new].astype(np.float32))
        assert np.array_equal(got[s, new:], m[s, new:])
    p.ok()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("n0,n1,budget", [(70000, 66001, 60000), (40000, 33007, 32500), (9000, 8999, 8192)])
def test_evict_long_sequences(n0, n1, budget, odd):
    p = Pair(1, 1, 64, 64, 2, -(-n0 // 64), seed=13, spare=0)
    p.append([0, 1], [n0, n1])
    m = p.rng.exponential(1.0, (2, p.cache.capacity)).astype(np.float32)
    if odd:      # so few that may go below NaN that some of the NaN go too, and many ties
        m[:] = np.where(p.rng.random(m.shape) < 0.99, np.nan, np.float32(2.0))
    p.cache.token_mass.copy_(torch.from_numpy(m))
    p.ora.mass[:] = m
    p.cache.evict(budget, 16, 1000, seqs=[1, 0])
    p.ora.evict([1, 0], budget, 16, 1000)
    p.check_state([0, 1])
    p.ok()


def test_evict_from_a_sequence_longer_than_shared_memory_holds():
    """Half a million tokens: their keys are read again from global memory. Copies are checked by position."""
    import chunked_kv_cache_gb300 as sr
    dev = device()
    n, budget, sink, recent = 400_003, 300_000, 10, 5000
    c = sr.PagedCache(1, 1, 64, page_tokens=1024, n_pages=400, max_seqs=1, max_pages=400, device=dev)
    c.reserve(0, n)
    g = torch.Generator(device=dev).manual_seed(2)
    k = torch.randn(n, 1, 64, device=dev, generator=g).to(torch.bfloat16)
    c.append(k, -k, counts=[n])
    m = torch.floor(torch.rand(c.capacity, device=dev, generator=g) * 50000)     # ties among them
    c.token_mass[0] = m
    c.evict(budget, sink, recent)
    assert c.seq_len.tolist() == [budget] and c.error_status() == 0
    t = torch.arange(n, device=dev)
    free = (t >= sink) & (t < n - recent)
    key = torch.where(free, m[:n].double(), torch.inf)
    order = torch.sort(key, descending=True, stable=True).indices          # a tie: the lower index stays
    keep = torch.zeros(n, dtype=torch.bool, device=dev).index_fill_(0, order[:budget], True)
    want = t[:budget].clone()
    want[~keep[:budget]] = t[budget:][keep[budget:]]
    got = c.token_pos[0, :budget].long()
    assert torch.equal(got, want) and torch.equal(c.token_mass[0, :budget], m[want])
    rows = c.block_table[0].long()[t[:budget] // 1024] * 1024 + t[:budget] % 1024
    assert torch.equal(c.k_pages.view(-1, 1, 64)[rows], k[want]) and torch.equal(c.v_pages.view(-1, 1, 64)[rows], -k[want])


def test_all_that_may_go_goes():
    """NaN weights only, and exactly the protected tokens stay."""
    for n, budget, sink, recent in ((300, 100, 40, 60), (9000, 5000, 1000, 4000)):
        p = Pair(1, 1, 64, 64, 1, -(-n // 64), seed=n)
        p.append([0], [n])
        p.cache.token_mass.fill_(float("nan"))
        p.ora.mass[:] = np.nan
        p.cache.evict(budget, sink, recent)
        p.ora.evict([0], budget, sink, recent)
        p.check_state([0])
        p.ok()


def test_positions_that_protect_more_than_the_budget():
    """Positions a caller restored wrongly (all recent): nothing may go, and nothing is written."""
    for n, budget in ((300, 290), (300, 20), (9000, 100)):
        p = Pair(1, 1, 64, 64, 1, -(-n // 64), seed=n)
        p.append([0], [n])
        p.cache.token_pos.fill_(n - 1)
        p.cache.token_pos[0, :5] = 1
        p.ora.pos[:] = n - 1
        p.ora.pos[0, :5] = 1
        p.cache.evict(budget, 0, 1)
        p.ora.evict([0], budget, 0, 1)
        p.check_state([0])
        p.ok()


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_loop_at_a_budget(e4m3):
    """Prompts, then token by token with weights and eviction, two budgets; lengths never exceed them."""
    p = Pair(8, 2, 64, 16, 4, 8, e4m3, seed=14)
    p.append([0, 1, 2, 3], [70, 5, 0, 100])
    for step in range(40):
        seqs = [3, 0, 1, 2] if step % 3 else [1, 3]
        p.append(seqs, [1] * len(seqs))
        p.attend(seqs, decay=0.9)
        p.cache.evict(64, n_sink=4, n_recent=16, seqs=seqs)
        p.ora.evict(seqs, 64, 4, 16)
        if step % 8 == 7:
            p.check_state(range(4))
    assert p.ora.length.max() == 64
    p.ok()


def test_captured_step_serves_later_tokens():
    p = Pair(8, 2, 128, 16, 3, 8, seed=15)
    p.append([0, 1, 2], [60, 63, 3])
    k, v, q = (torch.zeros(3, h, 128, dtype=torch.bfloat16, device=p.dev) for h in (2, 2, 8))
    out, lse = torch.empty_like(q), torch.empty(3, 8, device=p.dev)

    def step():
        p.cache.append(k, v)
        p.cache.attention(q, out=out, lse=lse, mass_decay=1.0)
        p.cache.evict(64, 2, 8)

    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    twin = Pair(8, 2, 128, 16, 3, 8, seed=15)
    twin.append([0, 1, 2], [60, 63, 3])
    for t in range(10):
        kk, vv, qq = p.randn(3, 2, 128), p.randn(3, 2, 128), p.randn(3, 8, 128)
        for dst, src in ((k, kk), (v, vv), (q, qq)):
            dst.copy_(src)
        graph.replay()
        twin.cache.append(kk, vv)
        o, l = twin.cache.attention(qq, lse=True, mass_decay=1.0)
        twin.cache.evict(64, 2, 8)
        torch.cuda.synchronize()
        assert torch.equal(out, o) and torch.equal(lse, l)
        for name in ("seq_len", "seq_pos", "token_pos", "token_mass"):
            assert torch.equal(getattr(p.cache, name), getattr(twin.cache, name)), (t, name)
    assert p.cache.seq_len.tolist() == [64, 64, 13]
    p.ok()


def test_two_graphs_of_one_cache_replayed_in_turn():
    """Two captured sequences and eager calls share a workspace; one after the other they do not disturb each other."""
    p = Pair(32, 8, 128, 64, 6, 20, seed=24)
    seqs = list(range(6))
    p.append(seqs, [1200, 1100, 0, 64, 1279, 700])
    q, k = p.randn(6, 32, 128), p.randn(3, 8, 128)
    p.cache.attention(q, mass_decay=0.0)                      # warm
    want = p.cache.attention(q)
    side = torch.cuda.Stream(p.dev)
    side.wait_stream(torch.cuda.current_stream())
    graphs, outs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()], []
    with torch.cuda.stream(side):
        with torch.cuda.graph(graphs[0], stream=side):
            outs.append(p.cache.attention(q, lse=True))
        with torch.cuda.graph(graphs[1], stream=side):
            p.cache.append(k, k, seqs=[2, 3, 5])
            outs.append(p.cache.attention(q, lse=True, mass_decay=1.0))
            p.cache.evict(1150, 4, 100)
    torch.cuda.current_stream().wait_stream(side)
    graphs[0].replay()
    assert torch.equal(outs[0][0], want)
    for step in range(3):
        graphs[1].replay()
        mass = p.cache.token_mass.clone()
        graphs[0].replay()
        torch.cuda.synchronize()
        assert torch.equal(outs[0][0], p.cache.attention(q)) and torch.isfinite(mass).all()
        assert p.cache.seq_len.tolist() == [1150, 1100, step + 1, 65 + step, 1150, 701 + step]
    p.ok()


def test_a_closed_cache_is_refused():
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 2, 64, 16, 2, 4, seed=25)
    p.append([0, 1], [3, 3])
    p.cache.close()
    p.cache.close()
    q, k = p.randn(2, 4, 64), p.randn(2, 2, 64)
    for call in (lambda: p.cache.attention(q), lambda: p.cache.append(k, k), lambda: p.cache.reset(), lambda: p.cache.evict(1)):
        with pytest.raises(N.SrError):
            call()


def test_other_stream_and_reserved_pages():
    import chunked_kv_cache_gb300 as sr
    dev = device()
    c = sr.PagedCache(4, 4, 64, page_tokens=16, n_pages=6, max_seqs=4, max_pages=4, device=dev)
    st = torch.cuda.Stream(dev)
    st.wait_stream(torch.cuda.current_stream(dev))
    with torch.cuda.stream(st):
        c.reserve(2, 33)
        c.reserve(0, 16)
        with pytest.raises(RuntimeError):
            c.reserve(1, 48)
        with pytest.raises(ValueError):
            c.reserve(1, 80)
        g = torch.Generator(device=dev).manual_seed(1)
        k = torch.randn(33, 4, 64, device=dev, generator=g).to(torch.bfloat16)
        c.append(k, k, seqs=[2], counts=[33])
        o = c.attention(torch.zeros(2, 4, 64, dtype=torch.bfloat16, device=dev), seqs=[2, 0])
    st.synchronize()
    assert c.error_status() == 0
    want = k.double().mean(0)
    assert (o[0].double() - want).abs().max() <= 2 * E * k.double().abs().mean(0).max()
    assert not o[1].any()
    c.release(2)
    c.reserve(1, 48)                            # the pages came back
    assert c.seq_len.tolist() == [0, 0, 0, 0]


def test_pages_past_4_gigabytes():
    """Rows whose offsets pass 32 bits, in elements and in bytes, on every path."""
    import chunked_kv_cache_gb300 as sr
    dev = device()
    kv, d, page, n_pages = 32, 128, 64, 10240          # 5.4 GB of keys, as much of values
    k_pages = torch.empty(n_pages, page, kv, d, dtype=torch.bfloat16, device=dev)
    v_pages = torch.empty_like(k_pages)
    table = torch.tensor([[n_pages - 1, 0, n_pages - 7], [n_pages - 2, n_pages - 3, 5]], dtype=torch.int32, device=dev)
    c = sr.PagedCache(kv, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=2, max_pages=3, device=dev,
                      buffers=dict(k_pages=k_pages, v_pages=v_pages, block_table=table))
    o = OraclePagedCache(kv, kv, d, 2, 192)
    g = torch.Generator(device=dev).manual_seed(3)
    k, v = (torch.randn(300, kv, d, device=dev, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, kv, d, device=dev, generator=g).to(torch.bfloat16)
    c.append(k, v, counts=[180, 120])
    o.append([0, 1], [180, 120], f64(k), f64(v))
    out = f64(c.attention(q, mass_decay=1.0))
    ref, _, wv = o.attention([0, 1], f64(q), 1.0)
    assert np.all(np.abs(out - ref) <= E * np.abs(ref) + (E + 1e-4) * wv)
    o.mass = f64(c.token_mass)
    c.evict(100, 2, 30)
    o.evict([0, 1], 100, 2, 30)
    assert c.seq_len.tolist() == [100, 100] and c.error_status() == 0
    for s in range(2):
        t = torch.arange(100, device=dev)
        rows = table[s].long()[t // page], t % page
        assert np.array_equal(f64(k_pages[rows]), o.k[s, :100]) and np.array_equal(f64(v_pages[rows]), o.v[s, :100])


def test_sequences_that_share_pages():
    """Reading shared pages is fine; weights and eviction need room for every token once, and say so."""
    import chunked_kv_cache_gb300 as sr
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 1, 64, 16, 1, 64, seed=17, spare=0)
    p.append([0], [1024])
    n = 8
    table = torch.from_numpy(np.repeat(p.table, n, 0).astype(np.int32)).to(p.dev)
    i32 = dict(dtype=torch.int32, device=p.dev)
    shared = sr.PagedCache(4, 1, 64, page_tokens=16, n_pages=64, max_seqs=n, max_pages=64, device=p.dev,
                           buffers=dict(k_pages=p.cache.k_pages, v_pages=p.cache.v_pages, block_table=table,
                                        seq_len=torch.full((n,), 1024, **i32), seq_pos=torch.full((n,), 1024, **i32),
                                        token_pos=torch.arange(1024, **i32).repeat(n, 1)))
    q = p.randn(n, 4, 64)
    want = torch.cat([p.cache.attention(q[i:i + 1]) for i in range(n)])
    got = shared.attention(q)
    assert (got.double() - want.double()).abs().max() <= 4 * E * want.double().abs().max()
    assert shared.error_status() == 0
    got = shared.attention(q, mass_decay=1.0)
    assert int(shared.err_word.item()) == N.SR_DEVERR_WORKSPACE and shared.error_status() == N.SR_ERR_STATE
    assert (got.double() - want.double()).abs().max() <= 4 * E * want.double().abs().max()
    shared.err_word.zero_()
    shared.token_mass.uniform_()
    shared.evict(512)
    assert int(shared.err_word.item()) == N.SR_DEVERR_WORKSPACE
    shared.err_word.zero_()
    shared.seq_len.fill_(100)                  # the counters are whole again
    o = shared.attention(q, mass_decay=1.0)
    assert shared.error_status() == 0 and torch.isfinite(o.float()).all()


def test_two_caches_read_the_same_pages_at_once():
    import chunked_kv_cache_gb300 as sr
    p = Pair(8, 2, 128, 64, 4, 40, seed=18)
    p.append([0, 1, 2, 3], [2500, 700, 64, 1999])
    q = p.randn(4, 8, 128)
    want = p.cache.attention(q)
    bufs = {k: getattr(p.cache, k) for k in ("k_pages", "v_pages", "block_table", "seq_len", "seq_pos", "token_pos")}
    others = [sr.PagedCache(8, 2, 128, page_tokens=64, n_pages=p.cache.n_pages, max_seqs=4, max_pages=40, mass=False,
                            buffers=bufs, device=p.dev) for _ in range(2)]
    streams = [torch.cuda.Stream(p.dev) for _ in others]
    torch.cuda.synchronize()
    outs = [[], []]
    for _ in range(20):
        for i, st in enumerate(streams):
            with torch.cuda.stream(st):
                outs[i].append(others[i].attention(q))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want) for both in outs for o in both)


def test_lengths_the_caller_spoilt_stay_in_bounds():
    """Lengths outside [0, cap] are read as the nearest end; an append to them is refused."""
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 2, 64, 16, 3, 4, seed=19)
    p.append([0, 1, 2], [64, 64, 10])
    p.cache.seq_len[0] = 1 << 30
    p.cache.seq_len[2] = -5
    p.ora.length[2] = 0
    p.attend([0, 1, 2], decay=1.0)
    k = p.randn(2, 2, 64)
    p.cache.append(k, k, seqs=[0, 2])
    assert int(p.cache.err_word.item()) == N.SR_DEVERR_CACHE_FULL
    assert p.cache.seq_len.tolist() == [1 << 30, 64, -5]
    p.cache.seq_len[1] = 20
    p.cache.seq_pos[1] = 2 ** 31 - 2
    p.cache.err_word.zero_()
    p.cache.append(k, k, seqs=[1], counts=[2])               # positions would pass 2^31 - 1
    assert int(p.cache.err_word.item()) == N.SR_DEVERR_CACHE_FULL and int(p.cache.seq_len[1]) == 20


@pytest.mark.parametrize("e4m3", [False, True])
def test_infinities_and_nan_of_live_tokens_are_not_hidden(e4m3):
    p = Pair(4, 2, 64, 16, 3, 4, e4m3, seed=20)
    k, v = p.randn(120, 2, 64), p.randn(120, 2, 64)
    k[5, 0, 3] = float("nan")                                 # sequence 0, head 0
    v[45, 1, 7] = float("nan")                                # sequence 1, head 1, one output column
    p.cache.append(k, v, counts=[40, 40, 40])
    p.ora.append([0, 1, 2], [40, 40, 40], f64(k), f64(v))
    o, lse = p.cache.attention(p.randn(3, 4, 64), lse=True)
    o, lse = f64(o), f64(lse)
    assert np.isnan(o[0, :2]).all() and np.isnan(lse[0, :2]).all() and np.isfinite(o[0, 2:]).all()
    assert np.isnan(o[1, 2:, 7]).all() and np.isnan(o[1]).sum() == 2 and np.isfinite(lse[1]).all()
    assert np.isfinite(o[2]).all()


@pytest.mark.parametrize("length", [1, 40, 2000])
def test_infinite_values_stay_infinite(length):
    """softmax weights are positive, so an infinite value of one sign is the output; of both, NaN."""
    p = Pair(4, 2, 64, 16, 1, 128, seed=22)
    k, v = p.randn(length, 2, 64), p.randn(length, 2, 64)
    v[length // 2, 0, 3] = float("inf")
    v[length - 1, 1, 9] = -float("inf")
    v[0, 1, 11], v[length - 1, 1, 11] = float("inf"), -float("inf")
    p.cache.append(k, v, counts=[length])
    o, lse = p.cache.attention(p.randn(1, 4, 64, s=0.25), lse=True)
    o = f64(o)[0]
    assert (o[:2, 3] == np.inf).all() and (o[2:, 9] == -np.inf).all() and np.isfinite(f64(lse)).all()
    if length > 1:
        assert np.isnan(o[2:, 11]).all()
    assert np.isfinite(np.delete(o, [3, 9, 11], 1)).all()


@pytest.mark.parametrize("heads,kv,n,length", [(8, 8, 3, 70), (16, 1, 2, 5000), (32, 8, 60, 900)])
def test_the_output_may_take_the_place_of_the_queries(heads, kv, n, length):
    p = Pair(heads, kv, 128, 64, n, -(-length // 64), seed=23)
    p.append(list(range(n)), [length - i for i in range(n)])
    q = p.randn(n, heads, 128)
    want, lse = p.cache.attention(q, lse=True, mass_decay=0.0)
    mass = p.cache.token_mass.clone()
    same, lse2 = p.cache.attention(q, out=q, lse=True, mass_decay=0.0)
    assert same is q and torch.equal(q, want) and torch.equal(lse, lse2) and torch.equal(mass, p.cache.token_mass)


def test_a_scale_that_underflows():
    p = Pair(4, 2, 64, 16, 2, 4, True, seed=21, scale=1e-38)
    p.append([0, 1], [37, 64])
    q = p.randn(2, 4, 64, s=1e-30)
    o = f64(p.cache.attention(q))
    for i in range(2):
        want = np.repeat(p.ora.v[i, : p.ora.length[i]].mean(0), 2, 0)
        assert np.abs(o[i] - want).max() <= 2 * E * np.abs(p.ora.v[i]).max()


def test_nothing_is_written_outside_the_buffers():
    """Every buffer between canary bands, through prompts, single tokens, weights, both joins and evictions."""
    import chunked_kv_cache_gb300 as sr
    from chunked_kv_cache_gb300 import _native as N
    from tests.test_gpu_guards import Guarded
    dev = device()
    for heads, kv, d, page, e4m3 in ((8, 2, 64, 16, False), (16, 1, 128, 48, True), (5, 5, 128, 64, False)):
        n, pages_each = 3, -(-4200 // page)
        n_pages, cap = n * pages_each, pages_each * page
        cfg = N.SrPagedConfig(heads, kv, d, page, n_pages, n, pages_each, 1 if e4m3 else 0, 0.0)
        row = n_pages * page * kv * d * (1 if e4m3 else 2)
        g = {name: Guarded(size, dev) for name, size in dict(
            k=row, v=row, table=n * pages_each * 4, length=n * 4, pos=n * 4, tpos=n * cap * 4, mass=n * cap * 4,
            exp=2 * kv * 4, err=4, ws=N.sr_paged_workspace_bytes(cfg, True), q=n * heads * d * 2, o=n * heads * d * 2,
            lse=n * heads * 4).items()}
        for name in ("length", "pos", "exp", "mass"):
            g[name].inner.zero_()
        g["table"].view(torch.int32, (n, pages_each)).copy_(
            torch.randperm(n_pages, device=dev).to(torch.int32).view(n, pages_each))
        ptr = {name: x.inner.data_ptr() for name, x in g.items()}
        stream = torch.cuda.current_stream(dev).cuda_stream
        h = N.sr_paged_init(cfg, N.SrPagedBuffers(ptr["k"], ptr["v"], ptr["table"], ptr["length"], ptr["pos"], ptr["tpos"],
                                                  ptr["mass"], ptr["exp"], ptr["err"], ptr["ws"]), stream)
        try:
            import ctypes
            for counts in ([4100, 0, 77], [1, 1, 1], [1, 130, 1]):
                rows = sum(counts)
                x = torch.randn(rows, kv, d, device=dev).to(torch.bfloat16)
                N.sr_paged_append(h, None, (ctypes.c_int32 * n)(*counts), n, x.data_ptr(), x.data_ptr(), stream)
                g["q"].view(torch.bfloat16, (n, heads, d)).normal_()
                N.sr_paged_attention(h, None, n, ptr["q"], ptr["o"], ptr["lse"], 1.0, stream)
                N.sr_paged_attention(h, (ctypes.c_int32 * 1)(0), 1, ptr["q"], ptr["o"], ptr["lse"], 0.5, stream)
            N.sr_paged_evict(h, None, n, 4101, 4, 100, stream)      # one token too many
            N.sr_paged_evict(h, None, n, 3000, 4, 100, stream)
            N.sr_paged_evict(h, None, n, 60, 4, 10, stream)
            N.sr_paged_attention(h, None, n, ptr["q"], ptr["o"], 0, -1.0, stream)
            torch.cuda.synchronize()
            assert int(g["err"].view(torch.int32, (1,)).item()) == 0
            assert g["length"].view(torch.int32, (n,)).tolist() == [60, 60, 60]
            assert torch.isfinite(g["o"].view(torch.bfloat16, (n, heads, d)).float()).all()
            assert {name: x.intact() for name, x in g.items()} == {name: True for name in g}
        finally:
            N.sr_paged_free(h)


def test_numbers_past_32_bits_are_not_cut():
    import chunked_kv_cache_gb300 as sr
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 2, 64, 16, 2, 4, seed=23)
    p.append([0, 1], [40, 40])
    q = p.randn(1, 4, 64)
    for call in (lambda: p.cache.attention(q, seqs=[1 << 32]), lambda: p.cache.reset([1 << 32]),
                 lambda: p.cache.evict(10, n_sink=1 << 32), lambda: p.cache.evict(10, n_recent=(1 << 32) + 3),
                 lambda: p.cache.evict(-((1 << 32) - 5))):
        with pytest.raises(sr.SrError) as e:
            call()
        assert e.value.status == N.SR_ERR_INVALID_ARG
    p.cache.evict((1 << 32) + 5)                              # above every length: nothing to do
    p.check_state([0, 1])
    p.ok()


def test_refusals():
    import chunked_kv_cache_gb300 as sr
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(4, 2, 64, 16, 3, 4, seed=16, mass=False)
    q, k = p.randn(3, 4, 64), p.randn(3, 2, 64)

    def refused(status, f, *a, **kw):
        with pytest.raises(sr.SrError) as e:
            f(*a, **kw)
        assert e.value.status == status

    refused(N.SR_ERR_STATE, p.cache.attention, q, mass_decay=1.0)
    refused(N.SR_ERR_STATE, p.cache.evict, 8)
    p = Pair(4, 2, 64, 16, 3, 4, seed=16)
    refused(N.SR_ERR_INVALID_ARG, p.cache.attention, q, seqs=[0, 1, 1])      # the same row twice
    refused(N.SR_ERR_INVALID_ARG, p.cache.append, k, k, seqs=[0, 1, 0])
    refused(N.SR_ERR_INVALID_ARG, p.cache.attention, q, seqs=[0, 1, 3])
    refused(N.SR_ERR_INVALID_ARG, p.cache.attention, q, seqs=[0, -1, 2])
    refused(N.SR_ERR_INVALID_ARG, p.cache.append, k, k, counts=[4, -2, 1])
    refused(N.SR_ERR_INVALID_ARG, p.cache.attention, q, mass_decay=float("nan"))
    refused(N.SR_ERR_INVALID_ARG, p.cache.evict, 0)
    refused(N.SR_ERR_INVALID_ARG, p.cache.evict, 8, 5, 4)
    refused(N.SR_ERR_INVALID_ARG, p.cache.evict, 8, -1, 4)
    refused(N.SR_ERR_INVALID_ARG, p.cache.evict, 8, seqs=[])
    for bad in (q.float(), q[:, :2], q.transpose(0, 1).contiguous().transpose(0, 1), q.cpu()):
        with pytest.raises(ValueError):
            p.cache.attention(bad)
    with pytest.raises(ValueError):
        p.cache.attention(q, seqs=[0, 1])
    with pytest.raises(ValueError):
        p.cache.append(k, k, counts=[1, 1])
    with pytest.raises(ValueError):
        p.cache.attention(q, mass_decay=-1.0)
    p.cache.append(k[:0], k[:0], counts=[0, 0, 0])            # nothing to do
    p.cache.evict(1 << 20)                                     # above every length
    assert p.cache.seq_len.tolist() == [0, 0, 0]
    p.ok()

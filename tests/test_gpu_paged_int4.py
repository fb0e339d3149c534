"""4-bit pages on the GPU against the float64 oracle: what is stored, attention of one token per sequence, eviction,
and reading back, which serves pages of every type.

Tolerances are test_gpu_paged's with the weights in fp16 (2^-11 of a weight, 2^-31 of the largest), as for e4m3
pages: a decoded value is exact in fp16, the queries are held as there. What is stored and read back is exact."""
import ctypes

import numpy as np
import pytest
import torch

from oracle.paged import OraclePagedCache
from tests.gpu_common import device
from tests.test_gpu_paged import LENGTHS, SHAPES, Pair, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


def unpack(pages, kv, page, d, exps):
    """4-bit pages as float64 [n_pages][page][kv][d], byte by byte from the layout's description."""
    rec = pages.cpu().numpy().reshape(-1, kv, page // 16, 9 * d)
    codes = rec[..., : 8 * d].reshape(*rec.shape[:3], d // 32, 16, 8, 2).astype(np.int64)
    unit = codes[..., 0] + 256 * codes[..., 1]
    unit = (unit >> 1) | ((unit & 1) << 15)
    n = np.stack([(unit >> (4 * i)) & 15 for i in range(4)], -1) - 8
    n = n.transpose(0, 2, 4, 1, 3, 5, 6).reshape(-1, page, kv, d)
    scales = rec[..., 8 * d:].reshape(*rec.shape[:3], 16, d // 16).transpose(0, 2, 3, 1, 4).reshape(-1, page, kv, d // 16)
    s = (scales.astype(np.uint16) << 7).view(np.float16).astype(np.float64)
    return n * np.repeat(s, 16, -1) * (2.0 ** exps)[:, None]


class Pair4(Pair):
    """Pair with 4-bit pages; stale pages are filled with the byte `junk`."""

    def __init__(self, heads, kv, d, page, max_seqs, max_pages, seed=0, spare=3, junk=255, mass=True, scale=0.0, exps=None):
        import chunked_kv_cache_gb300 as sr
        self.dev = device()
        self.rng = np.random.default_rng(seed)
        self.g = torch.Generator(device=self.dev).manual_seed(seed)
        self.page, self.kv, self.d, self.heads = page, kv, d, heads
        n_pages = max_seqs * max_pages + spare
        self.exps = self.rng.integers(-5, 3, (2, kv)).astype(np.int32) if exps is None else exps
        exps = torch.from_numpy(self.exps).to(self.dev)
        pool = [torch.full((n_pages, page * kv * 9 * d // 16), junk, device=self.dev, dtype=torch.uint8) for _ in range(2)]
        self.table = self.rng.permutation(n_pages)[: max_seqs * max_pages].reshape(max_seqs, max_pages)
        self.cache = sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=max_seqs, max_pages=max_pages,
                                   page_dtype="int4", device=self.dev, mass=mass, softmax_scale=scale,
                                   buffers=dict(k_pages=pool[0], v_pages=pool[1], kv_exp=exps,
                                                block_table=torch.from_numpy(self.table.astype(np.int32)).to(self.dev)))
        self.ora = OraclePagedCache(heads, kv, d, max_seqs, max_pages * page, kv_exp=self.exps, scale=scale if scale > 0 else None,
                                    int4=True)
        self.ora.e4m3 = True                     # Pair's tolerance of weights held in fp16

    def check_state(self, seqs):
        torch.cuda.synchronize()
        length, nxt = self.cache.seq_len.cpu().numpy(), self.cache.seq_pos.cpu().numpy()
        pos = self.cache.token_pos.cpu().numpy()
        k, v = (unpack(t, self.kv, self.page, self.d, e) for t, e in zip((self.cache.k_pages, self.cache.v_pages), self.exps))
        for s in seqs:
            n = int(self.ora.length[s])
            assert length[s] == n and nxt[s] == self.ora.next_pos[s], s
            assert np.array_equal(pos[s, :n], self.ora.pos[s, :n]), s
            t = np.arange(n)
            pg = self.table[s][t // self.page]
            assert np.array_equal(k[pg, t % self.page], self.ora.k[s, :n], equal_nan=True), s
            assert np.array_equal(v[pg, t % self.page], self.ora.v[s, :n], equal_nan=True), s

    def check_read(self, seqs, counts, first=None):
        k, v = self.cache.read(counts, seqs=seqs, first=first)
        want = self.ora.read(seqs, counts, first)
        assert k.dtype == torch.bfloat16
        assert np.array_equal(f64(k), want[0], equal_nan=True) and np.array_equal(f64(v), want[1], equal_nan=True)


@pytest.mark.parametrize("shape", SHAPES)
def test_append_read_and_attend_every_length(shape):
    heads, kv, d, page = shape
    n = len(LENGTHS)
    p = Pair4(heads, kv, d, page, n, -(-513 // page), seed=heads + d)
    seqs = p.rng.permutation(n).tolist()
    p.append(seqs, [LENGTHS[s] for s in seqs])
    p.check_state(range(n))
    p.attend(seqs)
    p.check_read(seqs, [LENGTHS[s] for s in seqs])
    p.append(list(range(n)), [1] * n)                      # one token each, wherever its page begins or ends
    p.check_state(range(n))
    p.attend(list(range(n)), decay=0.5)
    p.ok()


def special_rows(kv, d):
    """Rows whose blocks of 16 hold what rounding can get wrong: ties of scales and of values, zeros, tiny and huge
    numbers, infinities, NaN."""
    blocks = []
    for b in list(range(1, 20)) + [59, 60, 95, 96, 119, 127, 128, 199, 207, 213, 214]:
        s, nxt = ((1 + x % 8 / 8) * 2.0 ** (x // 8 - 15) if x >= 8 else x * 2.0 ** -17 for x in (b, b + 1))
        blocks.append([7 * (s + nxt) / 2] + [0.0] * 15)
        blocks.append([0.0] * 15 + [-7 * (s + nxt) / 2 * (1 - 2.0 ** -8)])
        blocks.append([7 * s] + [s * (k + 0.5) for k in range(7)] + [-s * (k + 0.5) for k in range(7)] + [-0.0])
        blocks.append([-7 * s] + [s * (k + 0.5) * (1 - 2.0 ** -8) for k in range(7)] + [s * k for k in range(8)])
    inf, nan = float("inf"), float("nan")
    blocks += [[0.0] * 16, [-0.0] * 16, [1e-38] * 16, [2.0 ** -18] * 16, [1e-40, 1.0] * 8, [1e38] * 16, [26880.0] * 16,
               [27000.0, 1.0] * 8, [inf] + [1.0] * 15, [-inf, inf] * 8, [nan] + [1.0] * 15, [1.0] * 15 + [nan], [nan, inf] * 8,
               [1920.0] * 8 + [-1920.0] * 8]
    blocks += [[3.0] * 16] * (-len(blocks) % (kv * d // 16))
    return torch.tensor(blocks, dtype=torch.float64).to(torch.bfloat16).view(-1, kv, d)


@pytest.mark.parametrize("kv,d,page", [(1, 64, 16), (3, 128, 48), (2, 64, 32)])
def test_blocks_that_lie_on_borders(kv, d, page):
    rows = special_rows(kv, d).to(device())
    n = rows.shape[0]
    p = Pair4(kv, kv, d, page, 2, -(-2 * n // page), exps=np.zeros((2, kv), np.int32))
    for counts in ([n, 0], [0, n], [n, 1]):
        k, v = (x[: sum(counts)].contiguous() for x in (torch.cat([rows, rows[:1]]), torch.cat([rows.flip(0), rows[-1:]])))
        p.cache.append(k, v, counts=counts)
        p.ora.append([0, 1], counts, f64(k), f64(v))
    p.check_state([0, 1])
    p.check_read([1, 0], [n + 1, 2 * n])
    p.ok()


@pytest.mark.parametrize("e", [-64, -20, 0, 17, 64])
def test_exponents_of_heads(e):
    p = Pair4(4, 2, 64, 16, 1, 4, exps=np.array([[e, 0], [0, e]], np.int32))
    k, v = p.randn(50, 2, 64), p.randn(50, 2, 64)
    k[:, 0] *= 2.0 ** e
    v[:, 1] *= 2.0 ** e
    p.cache.append(k, v, counts=[50])
    p.ora.append([0], [50], f64(k), f64(v))
    p.check_state([0])
    p.check_read([0], [50])
    if abs(e) < 40:
        p.attend([0], qs=1.5 * 2.0 ** min(-e, 0))
    p.ok()


@pytest.mark.parametrize("heads,kv,d,length", [(5, 1, 128, 20011), (16, 2, 64, 9001), (4, 4, 128, 4097), (64, 2, 128, 3001)])
def test_one_long_sequence_is_split_and_joined(heads, kv, d, length):
    p = Pair4(heads, kv, d, 64, 1, -(-length // 64), seed=length)
    p.append([0], [length])
    p.attend([0], decay=1.0)
    p.attend([0], decay=0.25)
    p.ok()


@pytest.mark.parametrize("heads,kv,d", [(40, 8, 128), (8, 1, 64), (12, 3, 64), (17, 1, 128)])
def test_many_sequences_of_unequal_length(heads, kv, d):
    lengths = [1 + (i * 397) % 1500 for i in range(40)] + [0, 6001, 0]
    p = Pair4(heads, kv, d, 32, len(lengths), 188, seed=heads)
    p.append(list(range(len(lengths))), lengths)
    seqs = p.rng.permutation(len(lengths)).tolist()
    p.attend(seqs, decay=1.0)
    p.attend(seqs[:7])
    p.ok()


@pytest.mark.parametrize("length", [1, 40, 257, 2000])
def test_large_queries_and_scales(length):
    p = Pair4(8, 2, 128, 16, 2, 126, seed=length, scale=0.9)
    p.append([0, 1], [length, 7])
    p.attend([0, 1], qs=60.0)
    p.attend([0, 1], qs=2.0 ** -90)
    p.ok()


@pytest.mark.parametrize("junk", [0, 0x7F, 0xF8, 0xFF])
def test_bytes_in_unused_rows_do_not_matter(junk):
    got = []
    for j in (junk, 0x55):
        p = Pair4(8, 2, 64, 16, 3, 20, seed=5, junk=j)
        p.append([0, 1, 2], [17, 1, 300])
        got.append(p.attend([0, 1, 2], decay=1.0))
        p.ok()
    assert all(np.array_equal(a, b) for a, b in zip(*got))


def test_numbers_that_are_none_reach_the_output():
    """A block with a NaN among the tokens seen; in a row behind the sequence it does not."""
    p = Pair4(2, 2, 64, 16, 2, 4, seed=6)
    k, v = p.randn(40, 2, 64), p.randn(40, 2, 64)
    v[7, 0, 20] = float("nan")
    v[39, 1, 0] = float("nan")
    p.cache.append(k, v, counts=[40, 0])
    o = f64(p.cache.attention(p.randn(2, 2, 64)))
    assert np.isnan(o[0, 0, 16:32]).all() and np.isfinite(o[0, 0, :16]).all() and np.isfinite(o[0, 0, 32:]).all()
    assert np.isnan(o[0, 1, :16]).all() and np.all(o[1] == 0)
    p.cache.seq_len[0] = 39
    o = f64(p.cache.attention(p.randn(2, 2, 64)))
    assert np.isfinite(o[0, 1]).all()
    p.ok()


def test_bad_pages_are_left_out_and_reported():
    from chunked_kv_cache_gb300 import _native as N
    p = Pair4(8, 2, 128, 16, 2, 20, seed=7)
    p.append([0, 1], [300, 100])
    p.cache.block_table[0, 3] = -1
    p.cache.block_table[0, 17] = p.cache.n_pages
    seen = np.ones(300, bool)
    seen[48:64] = seen[272:288] = False
    p.attend([0, 1], decay=1.0, visible=[seen, np.ones(100, bool)])
    assert p.cache.error_status() == N.SR_ERR_INVALID_ARG
    p.cache.err_word.zero_()
    k, v = p.cache.read([300, 100])
    want = p.ora.read([0, 1], [300, 100])
    want[0][:300][~seen] = want[1][:300][~seen] = 0
    assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1])
    assert p.cache.error_status() == N.SR_ERR_INVALID_ARG
    p.cache.err_word.zero_()
    before = p.cache.k_pages.clone()
    k = p.randn(21, 2, 128)
    p.cache.block_table[1, 7] = -5
    p.cache.append(k, k, counts=[0, 21])                    # its last token would lie there
    assert p.cache.error_status() == N.SR_ERR_INVALID_ARG and p.cache.seq_len.tolist() == [300, 100]
    assert torch.equal(before, p.cache.k_pages)


@pytest.mark.parametrize("n,budget,sink,recent", [(300, 299, 4, 16), (300, 200, 0, 0), (1000, 64, 10, 20), (5009, 5008, 3, 7), (5009, 4000, 64, 512)])
@pytest.mark.parametrize("kv,d,page", [(1, 64, 16), (8, 128, 64), (5, 64, 48)])
def test_evict_is_exact(n, budget, sink, recent, kv, d, page):
    p = Pair4(kv, kv, d, page, 3, -(-n // page), seed=n + budget)
    p.append([0, 1, 2], [n, n // 2, n - 1])
    p.attend([0, 1, 2], decay=1.0)
    p.cache.evict(budget, sink, recent)
    p.ora.evict([0, 1, 2], budget, sink, recent)
    p.check_state([0, 1, 2])
    p.attend([2, 1, 0])
    p.ok()


def test_serving_loop_at_a_budget():
    """Prompts, then token by token with weights, eviction and reading back; the other rows of the pool stay."""
    p = Pair4(8, 2, 64, 16, 4, 8, seed=14)
    p.append([0, 1, 2, 3], [70, 5, 0, 100])
    used = np.zeros(p.cache.n_pages, bool)
    used[p.table.ravel()] = True
    for step in range(30):
        seqs = [3, 0, 1, 2] if step % 3 else [1, 3]
        p.append(seqs, [1] * len(seqs))
        p.attend(seqs, decay=0.9)
        p.cache.evict(64, n_sink=4, n_recent=16, seqs=seqs)
        p.ora.evict(seqs, 64, 4, 16)
        if step % 8 == 7:
            p.check_state(range(4))
            p.check_read([2, 0], [3, 64])
    assert p.ora.length.max() == 64
    assert bool((p.cache.k_pages[torch.from_numpy(~used).to(p.dev)] == 255).all())
    p.ok()


def test_captured_step_serves_later_tokens():
    p, twin = (Pair4(8, 2, 128, 16, 3, 8, seed=15) for _ in range(2))
    for x in (p, twin):
        x.append([0, 1, 2], [60, 63, 3])
    k, v, q = (torch.zeros(3, h, 128, dtype=torch.bfloat16, device=p.dev) for h in (2, 2, 8))
    outs = [torch.empty_like(q), torch.empty(3, 8, device=p.dev)]
    back = [torch.empty(6, 2, 128, dtype=torch.bfloat16, device=p.dev) for _ in range(2)]

    def step(x, k, v, q, outs, back):
        x.cache.append(k, v)
        x.cache.attention(q, out=outs[0], lse=outs[1], mass_decay=1.0)
        x.cache.read([2, 2, 2], k=back[0], v=back[1])
        x.cache.evict(64, 2, 8)

    side = torch.cuda.Stream(p.dev)
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side), torch.cuda.graph(graph, stream=side):
        step(p, k, v, q, outs, back)
    torch.cuda.current_stream().wait_stream(side)
    for t in range(8):
        new = p.randn(3, 2, 128), p.randn(3, 2, 128), p.randn(3, 8, 128)
        for dst, src in zip((k, v, q), new):
            dst.copy_(src)
        graph.replay()
        o2, b2 = [torch.empty_like(x) for x in outs], [torch.empty_like(x) for x in back]
        step(twin, *new, o2, b2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs + back, o2 + b2))
        for name in ("seq_len", "seq_pos", "token_pos", "token_mass", "k_pages", "v_pages"):
            assert torch.equal(getattr(p.cache, name), getattr(twin.cache, name)), (t, name)
    assert p.cache.seq_len.tolist() == [64, 64, 11]
    p.ok()


def test_results_do_not_depend_on_the_run():
    p = Pair4(40, 8, 128, 64, 8, 80, seed=16)
    p.append(list(range(8)), [5000, 1, 640, 64, 4999, 3000, 17, 2222])
    q = p.randn(8, 40, 128)
    first = p.cache.attention(q, lse=True)
    for _ in range(20):
        again = p.cache.attention(q, lse=True)
        assert torch.equal(first[0], again[0]) and torch.equal(first[1], again[1])
    p.ok()


def test_pages_past_4_gigabytes():
    import chunked_kv_cache_gb300 as sr
    dev = device()
    kv, d, page = 16, 128, 1024
    per = page * kv * 9 * d // 16
    n_pages = (9 << 29) // per + 2                          # 4.5 GB of keys and as much of values
    cache = sr.PagedCache(16, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=2, max_pages=2, page_dtype="int4", device=dev,
                          mass=False, buffers=dict(block_table=torch.tensor([[n_pages - 1, 0], [1, n_pages - 2]], dtype=torch.int32,
                                                                            device=dev)))
    g = torch.Generator(device=dev).manual_seed(1)
    k, v = (torch.randn(2100, kv, d, device=dev, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, 16, d, device=dev, generator=g).to(torch.bfloat16)
    many = torch.randn(40, 16, d, device=dev, generator=g).to(torch.bfloat16)
    cache.append(k, v, counts=[1050, 1050])
    small = sr.PagedCache(16, kv, d, page_tokens=page, n_pages=4, max_seqs=2, max_pages=2, page_dtype="int4", device=dev, mass=False,
                          buffers=dict(block_table=torch.tensor([[3, 0], [1, 2]], dtype=torch.int32, device=dev)))
    small.append(k, v, counts=[1050, 1050])
    assert torch.equal(cache.attention(q), small.attention(q))
    assert torch.equal(cache.prompt_attention(many, [3, 37]), small.prompt_attention(many, [3, 37]))
    assert all(torch.equal(a, b) for a, b in zip(cache.read([1050, 7]), small.read([1050, 7])))
    assert torch.equal(cache.k_pages[n_pages - 1], small.k_pages[3]) and cache.error_status() == small.error_status() == 0


# ------------------------------------------------------------------ reading back, pages of every type
def _pair(kind, *a, **kw):
    return Pair4(*a, **kw) if kind == "int4" else Pair(*a, e4m3=kind == "e4m3", **kw)


@pytest.mark.parametrize("kind", ["bf16", "e4m3", "int4"])
@pytest.mark.parametrize("kv,d,page", [(1, 64, 16), (3, 128, 32), (8, 128, 64), (40, 128, 1024)])
def test_read_any_rows(kind, kv, d, page):
    p = _pair(kind, kv, kv, d, page, 4, max(2, 400 // page), seed=kv + d)
    p.append([0, 1, 2, 3], [min(391, 2 * page if page < 300 else 391), 9, 0, 31])
    L = [int(x) for x in p.ora.length]
    for seqs, counts, first in (([0, 1, 2, 3], L, None), ([3, 0], [1, 1], None), ([1, 3, 0], [20, 0, 3], None), ([2], [5], None),
                                ([0, 1, 3], [13, 9, 40], [5, 0, 2]), ([0, 2], [7, 2], [L[0] - 3, 0]), ([3], [4], [(1 << 31) - 2])):
        k, v = p.cache.read(counts, seqs=seqs, first=first)
        want = p.ora.read(seqs, counts, first)
        assert np.array_equal(f64(k), want[0]) and np.array_equal(f64(v), want[1]), (seqs, counts, first)
    a, b = p.cache.read()                                   # the last token of every sequence
    assert a.shape == (4, kv, d) and np.array_equal(f64(b), p.ora.read([0, 1, 2, 3], [1] * 4)[1])
    p.ok()


def test_refusals():
    import chunked_kv_cache_gb300 as sr
    p = Pair4(4, 2, 64, 16, 3, 4, seed=1)
    c, lib, dev = p.cache, p.cache._lib, p.dev
    p.append([0, 1, 2], [3, 3, 3])
    q, k = p.randn(3, 4, 64), p.randn(3, 2, 64)
    for call in (lambda: c.read([1, 1], seqs=[0]), lambda: c.read([1], first=[0, 1]), lambda: c.prompt_attention(q, [1, 1]),
                 lambda: c.prompt_attention(q.float()), lambda: c.prompt_attention(q, out=q[:2]), lambda: c.read([2], k=k),
                 lambda: c.prompt_attention(q.transpose(0, 1)), lambda: c.prompt_attention(q, lse=torch.zeros(3, 4, 1, device=dev)),
                 lambda: c.read([3], k=k.float(), v=k)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: c.read([1, -1]), lambda: c.read([1], seqs=[3]), lambda: c.read([1, 1], seqs=[1, 1]), lambda: c.read([1], first=[-1]),
                 lambda: c.prompt_attention(q, seqs=[0, 1, 1]), lambda: c.prompt_attention(q, seqs=[0, 1, 7]), lambda: c.read([]),
                 lambda: c.read([1], first=[1 << 31]), lambda: c.prompt_attention(q, [4, -1, 0]),
                 lambda: c.prompt_attention(torch.zeros(4, 4, 64, dtype=torch.bfloat16, device=dev))):
        with pytest.raises(sr.SrError):
            call()
    with pytest.raises(TypeError):
        c.read([1], k=3, v=k)
    s = c._stream()
    ok, inv, align = 0, -1, -3
    assert lib.sr_paged_read(c.handle, None, None, None, 3, k.data_ptr() + 2, k.data_ptr(), s) == align
    assert lib.sr_paged_read(c.handle, None, None, None, 3, 0, k.data_ptr(), s) == inv
    assert lib.sr_paged_read(c.handle, None, None, None, 0, k.data_ptr(), k.data_ptr(), s) == inv
    assert lib.sr_paged_prompt_attention(c.handle, None, None, 3, q.data_ptr() + 8, q.data_ptr(), None, 1, s) == align
    assert lib.sr_paged_prompt_attention(c.handle, None, None, 3, q.data_ptr(), q.data_ptr(), 2, 1, s) == align
    assert lib.sr_paged_prompt_attention(c.handle, None, None, 3, 0, q.data_ptr(), None, 1, s) == inv
    zeros = (ctypes.c_int32 * 3)(0, 0, 0)
    assert lib.sr_paged_prompt_attention(c.handle, None, zeros, 3, 0, 0, None, 1, s) == ok
    assert lib.sr_paged_read(c.handle, None, None, zeros, 3, 0, 0, s) == ok
    p.ok()

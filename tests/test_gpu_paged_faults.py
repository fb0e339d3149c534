"""The paged cache where a call cannot be carried out, or where the numbers leave nothing to
weigh: what it then leaves untouched, and what it says. Against the float64 oracle; tolerances
as derived in test_gpu_paged."""
import numpy as np
import pytest
import torch

from oracle.paged import OraclePagedCache
from tests.gpu_common import device
from tests.test_gpu_paged import E, U, Pair, f64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from chunked_kv_cache_gb300 import build
    build.build()
    device()


# ------------------------------------------------------------------ eviction over a page that is none of the pool's
@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n,length,budget,sink,recent", [
    (4, 33, 32, 0, 1), (4, 300, 299, 4, 16), (8, 4608, 4607, 4, 256),       # one token, one CTA
    (4, 5001, 5000, 4, 256),                                                # one token, a cluster
    (4, 300, 200, 4, 16), (4, 5000, 4000, 16, 500), (8, 9000, 4700, 0, 4),  # a block of them, a cluster
    (96, 120, 64, 4, 16),                                                   # a block of them, one CTA
])
def test_an_eviction_that_cannot_move_its_tokens_changes_nothing(n, length, budget, sink, recent, e4m3):
    """Sequences in turn: sound; the lightest token on an unmapped page; the last token, which is protected, on
    one; an unmapped page whose tokens stay in place. The second and third kind are left as they were."""
    from chunked_kv_cache_gb300 import _native as N
    p = Pair(2, 1, 64, 16, n, -(-length // 16), e4m3, seed=length + n)
    seqs = list(range(n))
    p.append(seqs, [length] * n)
    m = p.rng.lognormal(0, 2, (n, p.cache.capacity)).astype(np.float32)
    table = p.cache.block_table.clone()
    mid = (sink + 16) // 16                         # a page without sinks, below the budget
    assert 16 * (mid + 1) <= min(budget, length - recent)
    for s in seqs:
        bad = [-1, p.cache.n_pages, -(1 << 31), (1 << 31) - 1][s // 4 % 4]
        if s % 4 == 1:
            m[s, 16 * mid + 5] = 1e-9
            p.cache.block_table[s, mid] = bad
        elif s % 4 == 2:
            p.cache.block_table[s, (length - 1) // 16] = bad
        elif s % 4 == 3:
            m[s, 16 * mid: 16 * mid + 16] = 1e9
            p.cache.block_table[s, mid] = bad
    p.cache.token_mass.copy_(torch.from_numpy(m))
    p.ora.mass[:] = m
    before = p.cache.token_pos.clone()
    p.cache.evict(budget, sink, recent)
    sound = [s for s in seqs if s % 4 in (0, 3)]
    spoilt = [s for s in seqs if s % 4 in (1, 2)]
    p.ora.evict(sound, budget, sink, recent)
    assert int(p.cache.err_word.item()) == N.SR_DEVERR_BAD_PAGE
    p.check_state(seqs)
    mass = p.cache.token_mass.cpu().numpy()
    assert np.array_equal(mass[spoilt], m[spoilt]) and torch.equal(p.cache.token_pos[spoilt], before[spoilt])
    for s in sound:
        assert np.array_equal(mass[s, :budget], p.ora.mass[s, :budget].astype(np.float32))
    # with the pages back, the same call does what it could not do
    p.cache.block_table.copy_(table)
    p.cache.err_word.zero_()
    p.cache.evict(budget, sink, recent)
    p.ora.evict(seqs, budget, sink, recent)
    p.check_state(seqs)
    assert np.array_equal(p.cache.token_mass.cpu().numpy()[:, :budget], p.ora.mass[:, :budget].astype(np.float32))
    p.ok()


@pytest.mark.parametrize("length,budget", [(300, 299), (300, 288), (5009, 5008), (5009, 5000)])
def test_tokens_at_the_end_go_without_a_move(length, budget):
    """Nothing moves where the lightest tokens are the last: their page need not be there any more."""
    p = Pair(2, 1, 64, 16, 2, -(-length // 16), seed=length - budget)
    p.append([0, 1], [length, length])
    m = p.rng.lognormal(0, 1, (2, p.cache.capacity)).astype(np.float32)
    m[:, budget:] = 1e-9
    p.cache.token_mass.copy_(torch.from_numpy(m))
    p.ora.mass[:] = m
    p.cache.block_table[0, (length - 1) // 16] = -1
    p.cache.evict(budget, 4)
    p.ora.evict([0, 1], budget, 4)
    p.check_state([0, 1])
    p.ok()


# ------------------------------------------------------------------ weights that there is no room for
@pytest.mark.parametrize("kv,d,cap", [(1, 64, 1024), (2, 128, 256)])
def test_weights_of_a_batch_that_does_not_fit_are_left_as_they_were(kv, d, cap):
    """Sequences that share pages and hold more tokens than the pool: no sequence's weights change, so that the
    caller can take them in smaller batches. Outputs are written all the same."""
    import chunked_kv_cache_gb300 as sr
    from chunked_kv_cache_gb300 import _native as N
    n, page, heads = 8, 16, 4 * kv
    p = Pair(heads, kv, d, page, 1, cap // page, seed=d, spare=0)
    p.append([0], [cap])
    i32 = dict(dtype=torch.int32, device=p.dev)
    c = sr.PagedCache(heads, kv, d, page_tokens=page, n_pages=cap // page, max_seqs=n, max_pages=cap // page, device=p.dev,
                      buffers=dict(k_pages=p.cache.k_pages, v_pages=p.cache.v_pages,
                                   block_table=torch.from_numpy(np.repeat(p.table, n, 0).astype(np.int32)).to(p.dev),
                                   seq_len=torch.full((n,), cap, **i32), seq_pos=torch.full((n,), cap, **i32),
                                   token_pos=torch.arange(cap, **i32).repeat(n, 1)))
    q = p.randn(n, heads, d)
    c.token_mass.uniform_(generator=p.g)
    old = c.token_mass.clone()
    want, want_lse = c.attention(q, lse=True)
    o, lse = c.attention(q, lse=True, mass_decay=0.5)
    assert int(c.err_word.item()) == N.SR_DEVERR_WORKSPACE
    assert torch.equal(c.token_mass, old)
    assert torch.equal(o, want) and torch.equal(lse, want_lse)
    c.err_word.zero_()
    for seqs in ([0, 1], [5, 4], [2, 3], [7, 6]):
        c.attention(q[seqs], seqs=seqs, mass_decay=0.5)
    assert c.error_status() == 0
    got, rows = f64(c.token_mass), f64(old)
    for s in range(n):
        _, w, _ = p.ora.weights(0, f64(q[s]))
        ref = 0.5 * rows[s] + w.sum(0)
        qa, ka = np.abs(f64(q[s])).reshape(kv, 4, d), np.abs(p.ora.k[0])
        dx = (d + 8) * U * p.ora.scale * np.einsum("hgd,thd->hgt", qa, ka).max()
        assert np.all(np.abs(got[s] - ref) <= (2 * dx + cap * U + 2.0 ** -20 + 4 * U) * ref), s


# ------------------------------------------------------------------ scores that leave nothing
@pytest.mark.parametrize("heads,kv,length", [(4, 2, 40), (8, 2, 4000), (2, 2, 20011), (32, 2, 3000), (40, 2, 700)])
def test_tokens_whose_scores_are_all_minus_infinity_draw_no_weight(heads, kv, length):
    """Keys of -inf under positive queries: ln of a sum of zeros is -inf, the output 0 and the weight drawn 0, as for
    an empty sequence; the heads of other keys are not affected. Held whole, joined by the last CTA, by a launch."""
    d = 64
    p = Pair(heads, kv, d, 64, 2, -(-length // 64), seed=length)
    k, v = p.randn(2 * length, kv, d), p.randn(2 * length, kv, d)
    k[:length, 0] = -float("inf")                                 # sequence 0, key head 0
    p.cache.append(k, v, counts=[length, length])
    p.ora.append([0, 1], [length, length], f64(k), f64(v))
    q = p.randn(2, heads, d).abs() + 0.125
    p.cache.token_mass.uniform_(generator=p.g)
    old = f64(p.cache.token_mass)
    o, lse = p.cache.attention(q, lse=True, mass_decay=0.5)
    g = heads // kv
    assert not o[0, :g].any() and torch.all(lse[0, :g] == -np.inf)
    assert torch.isfinite(o.float()).all() and torch.isfinite(lse[0, g:]).all() and torch.isfinite(lse[1]).all()
    mass = f64(p.cache.token_mass)
    p.ora.k[0, :length, 0] = 0.0                                  # the other heads' weights; these are not counted
    for s in (0, 1):
        _, w, _ = p.ora.weights(s, f64(q[s]))
        ref = 0.5 * old[s, :length] + w[g if s == 0 else 0:].sum(0)
        ka = np.abs(p.ora.k[s, :length])
        dot = np.einsum("hgd,thd->hgt", np.abs(f64(q[s])).reshape(kv, g, d), ka).max()
        dx = (d + 8) * U * p.ora.scale * dot
        assert np.all(np.abs(mass[s, :length] - ref) <= (2 * dx + length * U + 2.0 ** -20 + 4 * U) * ref), s
    p.ok()


# ------------------------------------------------------------------ far rows, to the stated bounds
def test_far_rows_meet_the_stated_bounds():
    """Offsets past 32 bits with outputs, log-sum-exp and weights held to the bounds that near rows are held to."""
    import chunked_kv_cache_gb300 as sr
    dev = device()
    kv, d, page, n_pages = 32, 128, 64, 10240          # 5.4 GB of keys, as much of values
    k_pages = torch.empty(n_pages, page, kv, d, dtype=torch.bfloat16, device=dev)
    v_pages = torch.empty_like(k_pages)
    table = torch.tensor([[n_pages - 1, 1, n_pages - 9], [n_pages - 2, n_pages - 5, 4]], dtype=torch.int32, device=dev)
    c = sr.PagedCache(kv, kv, d, page_tokens=page, n_pages=n_pages, max_seqs=2, max_pages=3, device=dev,
                      buffers=dict(k_pages=k_pages, v_pages=v_pages, block_table=table))
    ora = OraclePagedCache(kv, kv, d, 2, 192)
    g = torch.Generator(device=dev).manual_seed(31)
    counts = [180, 120]
    k, v = (torch.randn(300, kv, d, device=dev, generator=g).to(torch.bfloat16) for _ in range(2))
    q = torch.randn(2, kv, d, device=dev, generator=g).to(torch.bfloat16)
    c.append(k, v, counts=counts)
    ora.append([0, 1], counts, f64(k), f64(v))
    o, lse = c.attention(q, lse=True, mass_decay=1.0)
    ref, ref_lse, wv = ora.attention([0, 1], f64(q), 1.0)
    o, lse, mass = f64(o), f64(lse), f64(c.token_mass)
    for s, n in enumerate(counts):
        dot = np.einsum("hd,thd->ht", np.abs(f64(q[s])), np.abs(ora.k[s, :n])).max(1)
        dx = (d + 8) * U * ora.scale * dot
        rel = 2 * dx + n * U + 2.0 ** -20
        bound = E * np.abs(ref[s]) + (2.0 ** -15 + rel[:, None]) * wv[s] + n * 2.0 ** -31 * np.abs(ora.v[s, :n]).max()
        assert np.all(np.abs(o[s] - ref[s]) <= bound), s
        assert np.all(np.abs(lse[s] - ref_lse[s]) <= dx + n * U + 2.0 ** -20 + 4 * U * np.abs(ref_lse[s])), s
        m = ora.mass[s, :n]
        assert np.all(np.abs(mass[s, :n] - m) <= (rel.max() + 4 * U) * np.abs(m)), s
    assert c.error_status() == 0

"""The paged cache's oracle against closed forms, brute force and invariants (CPU)."""
import itertools

import numpy as np
import pytest
import torch

from oracle.paged import OraclePagedCache, round_e4m3


def test_round_e4m3_is_the_nearest_value():
    # every finite e4m3 value, from its bits
    bits = np.arange(256, dtype=np.uint8)
    grid = torch.from_numpy(bits).view(torch.float8_e4m3fn).double().numpy()
    grid = np.unique(grid[np.isfinite(grid)])
    assert np.array_equal(round_e4m3(grid), grid)
    rng = np.random.default_rng(0)
    x = np.concatenate([rng.normal(size=4000) * 2.0 ** rng.integers(-12, 10, 4000), (grid[1:] + grid[:-1]) / 2])
    y = round_e4m3(x)
    near = np.abs(grid[None, :] - x[:, None]).min(1)
    assert np.array_equal(np.abs(y - x), near)
    # ties, infinities and NaN as the library of the tests rounds them (saturating)
    t = torch.from_numpy(x).clamp(-448, 448).to(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(y, t)
    assert round_e4m3(np.array([np.inf, -np.inf, 1e9])).tolist() == [448.0, -448.0, 448.0]
    assert np.isnan(round_e4m3(np.array([np.nan]))).all()


def _filled(rng, n, heads=4, kv=2, d=8):
    o = OraclePagedCache(heads, kv, d, 2, 64)
    o.append([1], [n], rng.normal(size=(n, kv, d)), rng.normal(size=(n, kv, d)))
    return o


def test_attention_against_brute_force_and_permutation():
    rng = np.random.default_rng(1)
    o = _filled(rng, 13)
    q = rng.normal(size=(1, 4, 8))
    out, lse, _ = o.attention([1], q)
    for h in range(4):
        x = [float(q[0, h] @ o.k[1, t, h // 2]) / np.sqrt(8) for t in range(13)]
        z = sum(np.exp(a) for a in x)
        want = sum(np.exp(a) / z * o.v[1, t, h // 2] for t, a in enumerate(x))
        assert np.allclose(out[0, h], want, atol=1e-13) and np.isclose(lse[0, h], np.log(z), atol=1e-13)
    perm = rng.permutation(13)
    o.k[1, :13], o.v[1, :13] = o.k[1, :13][perm], o.v[1, :13][perm]
    again, _, _ = o.attention([1], q)
    assert np.allclose(out, again, atol=1e-13)


def test_equal_keys_give_the_mean_and_an_empty_sequence_nothing():
    rng = np.random.default_rng(2)
    o = _filled(rng, 9)
    o.k[1, :] = o.k[1, 0]
    out, _, _ = o.attention([1], rng.normal(size=(1, 4, 8)))
    assert np.allclose(out[0].reshape(2, 2, 8), o.v[1, :9].mean(0)[:, None], atol=1e-13)
    out, lse, _ = o.attention([0], rng.normal(size=(1, 4, 8)))
    assert not out.any() and np.all(lse == -np.inf)


def test_mass_sums_to_the_heads_and_decays():
    rng = np.random.default_rng(3)
    o = _filled(rng, 11)
    o.attention([1], rng.normal(size=(1, 4, 8)), mass_decay=0.0)
    assert np.isclose(o.mass[1, :11].sum(), 4)
    before = o.mass[1, :11].copy()
    o.attention([1], np.zeros((1, 4, 8)), mass_decay=0.5)
    assert np.allclose(o.mass[1, :11], 0.5 * before + 4 / 11) and not o.mass[1, 11:].any()


@pytest.mark.parametrize("seed", range(6))
def test_evict_keeps_the_heaviest_set(seed):
    """Against all subsets: the kept tokens hold the sinks, the recent ones and the largest possible weight."""
    rng = np.random.default_rng(seed)
    n, budget = 10, int(rng.integers(4, 10))
    o = _filled(rng, n)
    o.mass[1, :n] = rng.integers(0, 4, n)      # ties among them
    sink, recent = int(rng.integers(0, 3)), int(rng.integers(0, 3))
    k0, m0 = o.k[1].copy(), o.mass[1].copy()
    o.evict([1], budget, sink, recent)
    assert o.length[1] == budget
    kept = sorted(o.pos[1, :budget].tolist())
    assert len(set(kept)) == budget
    must = set(range(sink)) | set(range(n - recent, n))
    assert must <= set(kept)
    rest = [t for t in range(n) if t not in must]
    best = max(m0[list(c)].sum() for c in itertools.combinations(rest, budget - len(must)))
    assert m0[[t for t in kept if t not in must]].sum() == best
    for i in range(budget):      # rows travel with their positions; those in place have not moved
        t = o.pos[1, i]
        assert np.array_equal(o.k[1, i], k0[t]) and o.mass[1, i] == m0[t] and (t == i or t >= budget)

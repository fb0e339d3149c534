"""4-bit pages, prompts and reading back, without a GPU: the oracle's rounding against its definition, and calls
that are refused before anything is launched."""
import ctypes
import fractions

import numpy as np
import pytest
import torch

from chunked_kv_cache_gb300 import _native as N
from chunked_kv_cache_gb300 import build as B
from oracle.paged import OraclePagedCache, round_int4


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.lib()


def _cfg(**kw):
    base = dict(n_heads=8, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=12, max_seqs=3, max_pages=5,
                page_type=N.SR_PAGE_INT4, softmax_scale=0.0)
    base.update(kw)
    return N.SrPagedConfig(**base)


# every scale there is: bytes 0 .. 215 as fp16 numbers with the bits b << 7
SCALES = [fractions.Fraction(b % 8, 1 << 17) if b < 8 else fractions.Fraction(8 + b % 8, 8) * fractions.Fraction(2) ** (b // 8 - 15)
          for b in range(216)]


def _round_slowly(block):
    """The definition in rational numbers, by search over the scales."""
    x = [fractions.Fraction(float(v)) for v in block]
    want = max(abs(v) for v in x) / 7
    s = next((a for a, b in zip(SCALES, SCALES[1:]) if want < (a + b) / 2), SCALES[-1])
    if s == 0:
        return [0.0] * 16
    out = []
    for v in x:
        n = (abs(v) / s + fractions.Fraction(1, 2)).__floor__()
        out.append(float(max(-8, min(7, n if v >= 0 else -n)) * s))
    return out


@pytest.mark.parametrize("top", [1e-7, 2.0 ** -16, 1e-4, 0.03, 1.0, 7.0, 300.0, 30000.0, 1e30])
def test_the_oracle_rounds_as_defined(top):
    rng = np.random.default_rng(int(top * 1000) % 997)
    x = rng.standard_normal((40, 16)) * top
    x = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    x[0] = 0.0
    x[1, 3:] = 0.0
    assert np.array_equal(round_int4(x), [_round_slowly(b) for b in x])


def test_halves_of_scales_and_of_values():
    """Quotients that lie on a border: 7 times the middle of two scales, and scales times halves."""
    rows = []
    for b in (1, 5, 8, 9, 60, 119, 121, 200, 214):
        s, nxt = float(SCALES[b]), float(SCALES[b + 1])
        rows.append([7 * (s + nxt) / 2] + [0.0] * 15)                          # goes up to the next scale
        rows.append([7 * s] + [s * (k + 0.5) for k in range(7)] + [-s * (k + 0.5) for k in range(7)] + [0.0])
    x = np.array(rows)
    assert np.array_equal(torch.from_numpy(x).to(torch.bfloat16).double().numpy(), x)   # all of them are bf16 numbers
    y = round_int4(x)
    assert np.array_equal(y, [_round_slowly(r) for r in x])
    for i, b in enumerate((1, 5, 8, 9, 60, 119, 121, 200)):
        k = y[2 * i, 0] / float(SCALES[b + 1])                                 # in steps of the larger scale
        assert k == round(k) and k <= 7
    assert y[3, 1] == float(SCALES[5]) and y[3, 8] == -float(SCALES[5])        # away from zero


def test_blocks_that_are_no_numbers():
    x = np.full((4, 32), 7.0)
    x[0, 3], x[1, 20], x[2, 0] = np.inf, -np.inf, np.nan
    y = round_int4(x)
    assert y[0, 3] == 7 * 3840 and np.all(np.delete(y[0, :16], 3) == 0) and np.all(y[0, 16:] == 7)
    assert y[1, 20] == -8 * 3840 and np.isnan(y[2, :16]).all() and np.all(y[2, 16:] == 7)


def test_the_oracle_of_prompts_is_that_of_tokens():
    rng = np.random.default_rng(3)
    o = OraclePagedCache(4, 2, 64, 2, 40, int4=True)
    k, v = rng.standard_normal((2, 30, 2, 64))
    o.append([0, 1], [20, 10], k, v)
    q = rng.standard_normal((9, 4, 64))
    out, lse, _ = o.prompt_attention([1, 0], [4, 5], q)
    o.length[0] -= 3                                        # row 5 of the call sees two tokens of the new five
    ref, ref_lse, _ = o.attention([0], q[5:6])
    assert np.allclose(out[5], ref[0]) and np.allclose(lse[5], ref_lse[0])
    o.length[1] = 2
    assert np.all(o.prompt_attention([1], [4], q[:4])[1][:2] == -np.inf)


INV, UNS, ALIGN = N.SR_ERR_INVALID_ARG, N.SR_ERR_UNSUPPORTED, N.SR_ERR_ALIGN


def test_null_arguments(lib):
    assert lib.sr_paged_prompt_attention(None, None, None, 1, 16, 16, None, 1, None) == INV
    assert lib.sr_paged_read(None, None, None, None, 1, 16, 16, None) == INV


@pytest.mark.parametrize("change,status", [
    (dict(), N.SR_OK), (dict(head_dim=128), N.SR_OK), (dict(head_dim=32), UNS), (dict(page_tokens=24), UNS),
    (dict(n_heads=7), INV), (dict(page_type=3), UNS), (dict(page_type=5), UNS),
])
def test_shapes(lib, change, status):
    n = ctypes.c_uint64()
    assert lib.sr_paged_workspace_bytes(ctypes.byref(_cfg(**change)), 1, ctypes.byref(n)) == status


def test_python_refuses_before_allocating(lib):
    import chunked_kv_cache_gb300 as sr
    for bad in ("int8", "INT4", torch.uint8):
        with pytest.raises(ValueError, match="page_dtype"):
            sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, page_dtype=bad, device="cpu")
    with pytest.raises(ValueError, match="k_pages"):
        sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, page_dtype="int4", device="cpu",
                      buffers={"k_pages": torch.zeros(4, 64, 4, 64, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match="v_pages"):
        sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, page_dtype="int4", device="cpu",
                      buffers={"v_pages": torch.zeros(4, 64 * 4 * 36 - 1, dtype=torch.uint8)})

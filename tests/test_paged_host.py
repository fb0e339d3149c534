"""The paged cache's refusals and its page arithmetic, without a GPU: every call here
is refused before anything is launched, or is host arithmetic."""
import ctypes

import numpy as np
import pytest

from chunked_kv_cache_gb300 import _native as N
from chunked_kv_cache_gb300 import build as B


@pytest.fixture(scope="module")
def lib():
    B.build()
    return N.lib()


def _cfg(**kw):
    base = dict(n_heads=8, n_kv_heads=2, head_dim=64, page_tokens=16, n_pages=12, max_seqs=3, max_pages=5,
                page_type=N.SR_PAGE_BF16, softmax_scale=0.0)
    base.update(kw)
    return N.SrPagedConfig(**base)


def _bufs(**kw):
    base = dict(k_pages=0x10000, v_pages=0x20000, block_table=0x30000, seq_len=0x40000, seq_pos=0x50000,
                token_pos=0x60000, token_mass=0x70000, kv_exp=0, err_word=0x80000, workspace=0x90000)
    base.update(kw)
    return N.SrPagedBuffers(**base)


def _init(cfg, bufs):
    out = ctypes.c_void_p(0x1234)
    return N.lib().sr_paged_init(ctypes.byref(cfg), ctypes.byref(bufs), None, ctypes.byref(out)), out.value


INV, UNS, ALIGN = N.SR_ERR_INVALID_ARG, N.SR_ERR_UNSUPPORTED, N.SR_ERR_ALIGN


@pytest.mark.parametrize("change,status", [
    (dict(n_heads=0), INV), (dict(n_kv_heads=0), INV), (dict(n_heads=7), INV),
    (dict(head_dim=96), UNS), (dict(head_dim=256), UNS), (dict(page_type=2), UNS), (dict(page_type=-1), UNS),
    (dict(page_tokens=0), INV), (dict(page_tokens=8), UNS), (dict(page_tokens=24), UNS),
    (dict(page_tokens=1040), UNS), (dict(n_pages=0), INV), (dict(max_seqs=0), INV), (dict(max_seqs=65537), INV),
    (dict(max_pages=0), INV), (dict(max_pages=(1 << 20) + 1), INV), (dict(n_pages=(1 << 27) + 1), INV),
    (dict(n_heads=1040, n_kv_heads=1040), INV), (dict(softmax_scale=float("nan")), INV),
])
def test_bad_shapes(lib, change, status):
    st, out = _init(_cfg(**change), _bufs())
    assert st == status and out is None
    n = ctypes.c_uint64()
    assert lib.sr_paged_workspace_bytes(ctypes.byref(_cfg(**change)), 1, ctypes.byref(n)) == status


@pytest.mark.parametrize("heads,kv", [(34, 2), (32, 1), (1024, 1), (71, 1), (512, 16)])
def test_any_share_of_a_key_head_has_a_workspace(lib, heads, kv):
    """More query heads than a read serves are split; the weights' scores need the same room however they are."""
    n, m = ctypes.c_uint64(), ctypes.c_uint64()
    shape = dict(n_heads=heads, n_kv_heads=kv, head_dim=64, n_pages=1000, max_seqs=1)
    assert lib.sr_paged_workspace_bytes(ctypes.byref(_cfg(**shape)), 1, ctypes.byref(n)) == N.SR_OK
    assert lib.sr_paged_workspace_bytes(ctypes.byref(_cfg(**dict(shape, n_kv_heads=heads))), 1, ctypes.byref(m)) == N.SR_OK
    tokens = 1000 * _cfg(**shape).page_tokens
    assert n.value >= tokens * heads * 4 and n.value <= 4 * m.value


@pytest.mark.parametrize("name,value,status", [
    ("k_pages", 0, INV), ("v_pages", 0, INV), ("block_table", 0, INV), ("seq_len", 0, INV), ("seq_pos", 0, INV),
    ("token_pos", 0, INV), ("err_word", 0, INV), ("workspace", 0, INV), ("k_pages", 0x10008, ALIGN),
    ("v_pages", 0x20001, ALIGN), ("block_table", 0x30002, ALIGN), ("token_mass", 0x70001, ALIGN),
    ("kv_exp", 0x3, ALIGN), ("workspace", 0x90080, ALIGN),
])
def test_bad_buffers(lib, name, value, status):
    st, out = _init(_cfg(), _bufs(**{name: value}))
    assert st == status and out is None


def test_null_arguments(lib):
    assert lib.sr_paged_init(None, None, None, None) == INV
    assert lib.sr_paged_workspace_bytes(None, 0, None) == INV
    assert lib.sr_paged_free(None) == N.SR_OK
    assert lib.sr_paged_reset(None, None, 1, None) == INV
    assert lib.sr_paged_append(None, None, None, 1, 16, 16, None) == INV
    assert lib.sr_paged_attention(None, None, 1, 16, 16, None, -1.0, None) == INV
    assert lib.sr_paged_evict(None, None, 1, 16, 0, 0, None) == INV
    assert lib.sr_paged_locate(None, None, 0, None) == INV


def test_workspace_grows_with_mass_only(lib):
    a, b = N.sr_paged_workspace_bytes(_cfg(), False), N.sr_paged_workspace_bytes(_cfg(), True)
    assert 0 < a < b and a % 256 == b % 256 == 0


@pytest.mark.parametrize("page_tokens", [16, 48, 64, 1024])
def test_locate_follows_the_table_and_refuses_bad_pages(lib, page_tokens):
    cfg = _cfg(page_tokens=page_tokens, n_pages=7, max_pages=5)
    table = [3, 6, -1, 7, 0]          # page 2 is unmapped, 7 is past the pool
    cap = 5 * page_tokens
    for i in sorted({-1, 0, 1, page_tokens - 1, page_tokens, 2 * page_tokens - 1, 2 * page_tokens,
                     3 * page_tokens, 4 * page_tokens - 1, 4 * page_tokens, cap - 1, cap, cap + 5, 1 << 40}):
        want = -1
        if 0 <= i < cap and 0 <= table[i // page_tokens] < 7:
            want = table[i // page_tokens] * page_tokens + i % page_tokens
        assert N.sr_paged_locate(cfg, table, i) == want


def test_rows_past_32_bits_are_not_cut(lib):
    cfg = _cfg(page_tokens=1024, n_pages=1 << 21, max_pages=4)
    assert N.sr_paged_locate(cfg, [(1 << 21) - 1, 0, 0, 0], 1023) == (1 << 31) - 1


def test_device_codes_map_to_statuses(lib):
    assert N.sr_device_error_status(N.SR_DEVERR_BAD_PAGE) == N.SR_ERR_INVALID_ARG
    assert N.sr_device_error_status(N.SR_DEVERR_CACHE_FULL) == N.SR_ERR_STATE
    assert N.sr_device_error_status(N.SR_DEVERR_WORKSPACE) == N.SR_ERR_STATE
    assert N.sr_device_error_status(N.SR_DEVERR_WAIT_TIMEOUT | (3 << 8)) == N.SR_ERR_TIMEOUT


def test_python_refuses_before_allocating(lib):
    import torch

    import chunked_kv_cache_gb300 as sr
    with pytest.raises(ValueError, match="page_dtype"):
        sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, page_dtype=torch.float16, device="cpu")
    with pytest.raises(sr.SrError):
        sr.PagedCache(4, 4, 80, n_pages=4, max_seqs=1, max_pages=4, device="cpu")
    with pytest.raises(ValueError, match="k_pages"):
        sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, device="cpu",
                      buffers={"k_pages": torch.zeros(4, 64, 4, 32, dtype=torch.bfloat16)})
    with pytest.raises(ValueError, match="unknown"):
        sr.PagedCache(4, 4, 64, n_pages=4, max_seqs=1, max_pages=4, device="cpu",
                      buffers={"pages": torch.zeros(1)})
    assert np.dtype(np.int32).itemsize == ctypes.sizeof(ctypes.c_int32)

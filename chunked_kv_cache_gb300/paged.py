"""The paged token cache: sequences served token by token over a shared pool of pages.

``PagedCache`` allocates the cache's device buffers with torch (or takes the
caller's), hands out pages of the pool, and marshals tensors into the sr_paged_*
calls of libsr.so. Nothing here computes.
"""
from __future__ import annotations

from array import array
from collections.abc import Sequence

import torch

from . import _native as N

_BF16 = torch.bfloat16
_PAGE_TYPES = {torch.bfloat16: N.SR_PAGE_BF16, torch.float8_e4m3fn: N.SR_PAGE_E4M3, "int4": N.SR_PAGE_INT4}


class PagedCache:
    """Keys and values of up to max_seqs sequences in pages of page_tokens tokens.

    Tensors, all on one device: k_pages, v_pages [n_pages][page_tokens][n_kv_heads][head_dim]
    (bf16, or e4m3 with value = e4m3 * 2^kv_exp[0 or 1][head]), or, with page_dtype="int4" (codes of 4 bits and
    a scale for each 16 values, also times 2^kv_exp; the layout stands at sr_paged_cache in include/sr.h),
    [n_pages][page_tokens * n_kv_heads * 9 * head_dim // 16] uint8; block_table
    [max_seqs][max_pages] int32; seq_len, seq_pos [max_seqs] int32; token_pos
    [max_seqs][max_pages * page_tokens] int32; token_mass, the same shape in fp32 (mass=True);
    kv_exp [2][n_kv_heads] int32.

    buffers: a dict with any of these names, used in place and as found. Sequences
    whose block table the caller does not fill get their pages from reserve(). Also
    "workspace", uint8, another cache's that is as long at least (sr_paged_workspace_bytes; most of
    it is room for the parts of cut prompts, 21 MB for heads of 64 and 43 MB for heads of 128, whatever the
    pool): caches whose calls never run at the same time, as a model's layers, may share one.

    Calls run on the current stream of the cache's device, which must be the current device, and
    two of one cache must not run at the same time (they share a workspace). The cache is
    made on the current stream too: whoever goes on with it on another stream orders that one
    behind, and keeps the cache until the work there is done (its memory returns to torch's
    allocator, as a tensor's does). seqs: distinct rows of the block table (host integers), at
    most SR_MAX_PAGED_SEQS; None stands for the first rows, as many as the call has.
    """

    def __init__(self, n_heads: int, n_kv_heads: int, head_dim: int, *, page_tokens: int = 64, n_pages: int,
                 max_seqs: int, max_pages: int, page_dtype: torch.dtype | str = _BF16, softmax_scale: float = 0.0,
                 mass: bool = True, buffers: dict | None = None, device="cuda"):
        self.handle = None
        if page_dtype not in _PAGE_TYPES:
            raise ValueError(f"page_dtype must be one of {list(_PAGE_TYPES)}, got {page_dtype}")
        self.device = torch.device(device)
        if self.device.type == "cuda" and self.device.index is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        dev = self.device
        self.n_heads, self.n_kv_heads, self.head_dim = n_heads, n_kv_heads, head_dim
        self.page_tokens, self.n_pages, self.max_seqs, self.max_pages = page_tokens, n_pages, max_seqs, max_pages
        self.capacity = max_pages * page_tokens
        self.cfg = N.SrPagedConfig(n_heads, n_kv_heads, head_dim, page_tokens, n_pages, max_seqs, max_pages,
                                   _PAGE_TYPES[page_dtype], softmax_scale)
        given = dict(buffers or {})
        mass = mass or "token_mass" in given
        nbytes = N.sr_paged_workspace_bytes(self.cfg, mass)     # refuses a bad shape before anything is allocated

        def take(name, shape, dtype, fill):
            t = given.pop(name, None)
            if t is None:
                return torch.full(shape, fill, dtype=dtype, device=dev) if fill is not None else \
                    torch.empty(shape, dtype=dtype, device=dev)
            if not isinstance(t, torch.Tensor):
                raise TypeError(f"{name} must be a torch.Tensor")
            if t.dtype != dtype or tuple(t.shape) != tuple(shape) or not t.is_contiguous() or t.device != dev:
                raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {dev}, "
                                 f"got {t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")
            return t

        pages, stored = (n_pages, page_tokens, n_kv_heads, head_dim), page_dtype
        if page_dtype == "int4":
            pages, stored = (n_pages, page_tokens * n_kv_heads * 9 * head_dim // 16), torch.uint8
        per_token = (max_seqs, self.capacity)
        i32 = torch.int32
        own_table = "block_table" not in given
        self.k_pages = take("k_pages", pages, stored, None)
        self.v_pages = take("v_pages", pages, stored, None)
        self.block_table = take("block_table", (max_seqs, max_pages), i32, -1)
        self.seq_len = take("seq_len", (max_seqs,), i32, 0)
        self.seq_pos = take("seq_pos", (max_seqs,), i32, 0)
        self.token_pos = take("token_pos", per_token, i32, 0)
        self.token_mass = take("token_mass", per_token, torch.float32, 0.0) if mass else None
        self.kv_exp = take("kv_exp", (2, n_kv_heads), i32, 0)
        space = self._workspace(given.pop("workspace", None), nbytes, dev)
        if given:
            raise ValueError(f"unknown buffers: {sorted(given)}")
        self.err_word = torch.zeros((1,), dtype=i32, device=dev)
        self.workspace = torch.empty((nbytes,), dtype=torch.uint8, device=dev) if space is None else space
        # pages not handed out yet (only when the cache owns its block table)
        self._free = list(range(n_pages - 1, -1, -1)) if own_table else None
        self._pages: list[list[int]] = [[] for _ in range(max_seqs)] if own_table else []
        bufs = N.SrPagedBuffers(self.k_pages.data_ptr(), self.v_pages.data_ptr(), self.block_table.data_ptr(),
                                self.seq_len.data_ptr(), self.seq_pos.data_ptr(), self.token_pos.data_ptr(),
                                self.token_mass.data_ptr() if mass else None, self.kv_exp.data_ptr(),
                                self.err_word.data_ptr(), self.workspace.data_ptr())
        self._lib = N.lib()
        with torch.cuda.device(dev):
            self.handle = N.sr_paged_init(self.cfg, bufs, self._stream())

    # ---------------------------------------------------------------- helpers
    @staticmethod
    def _workspace(t, nbytes: int, dev):
        """A given workspace, checked; None stays."""
        if t is None:
            return None
        if not isinstance(t, torch.Tensor):
            raise TypeError("workspace must be a torch.Tensor")
        if t.dtype != torch.uint8 or t.dim() != 1 or t.numel() < nbytes or not t.is_contiguous() or t.device != dev:
            raise ValueError(f"workspace: expected contiguous torch.uint8 of {nbytes} bytes or more on {dev}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")
        return t

    def _stream(self) -> int:
        # the handle itself: a Stream object costs two microseconds, as much as a launch
        return torch._C._cuda_getCurrentRawStream(self.device.index)

    @staticmethod
    def _ids(seqs: Sequence[int] | None):
        """The numbers as 32-bit ones, to be kept while their address is used, and that address."""
        if seqs is None:
            return None, None
        if isinstance(seqs, (bytes, bytearray)):
            seqs = list(seqs)                        # an array would take them for its raw memory
        try:
            ids = array("i", seqs)
        except OverflowError:
            raise N.SrError(N.SR_ERR_INVALID_ARG, "sequence or count") from None
        return ids, ids.buffer_info()[0]

    # The calls below go to the library without N's wrappers: a call is a few microseconds on the host.
    @staticmethod
    def _done(status: int, what: str) -> None:
        if status != N.SR_OK:
            raise N.SrError(status, what)

    def _check(self, name: str, t: torch.Tensor, shape, dtype=_BF16) -> None:
        if not isinstance(t, torch.Tensor):
            raise TypeError(f"{name} must be a torch.Tensor")
        if t.dtype != dtype or t.shape != shape or t.device != self.device or not t.is_contiguous():
            raise ValueError(f"{name}: expected contiguous {dtype} {tuple(shape)} on {self.device}, "
                             f"got {t.dtype} {tuple(t.shape)} on {t.device} (contiguous={t.is_contiguous()})")

    @staticmethod
    def _seqs_of(what: str, rows: int, seqs, counts) -> int:
        """The sequences of a call whose tensors have `rows` rows."""
        n = len(seqs) if seqs is not None else len(counts) if counts is not None else rows
        if counts is not None and len(counts) != n:
            raise ValueError(f"{len(counts)} counts for {n} sequences")
        takes = n if counts is None else sum(counts)
        if takes != rows:
            raise ValueError(f"{what} {rows} rows, the sequences take {takes}")
        return n

    # ---------------------------------------------------------------- pages
    def reserve(self, seq: int, n_tokens: int) -> None:
        """Give sequence `seq` the pages it needs to hold n_tokens tokens (those it has stay)."""
        if self._free is None:
            raise RuntimeError("the caller's block table is the caller's to fill")
        if not 0 <= seq < self.max_seqs:
            raise ValueError(f"sequence {seq} of {self.max_seqs}")
        have = self._pages[seq]
        need = -(-n_tokens // self.page_tokens)
        if need > self.max_pages:
            raise ValueError(f"{n_tokens} tokens are {need} pages, more than max_pages = {self.max_pages}")
        more = need - len(have)
        if more <= 0:
            return
        if more > len(self._free):
            raise RuntimeError(f"the pool has {len(self._free)} free pages, {more} are needed")
        new = self._free[:-more - 1:-1]
        self.block_table[seq, len(have):need] = torch.tensor(new, dtype=torch.int32, device=self.device)
        del self._free[-more:]                       # theirs once the table has them
        have.extend(new)

    def release(self, seq: int) -> None:
        """Empty sequence `seq` and give its pages back to the pool (the only way back: a sequence
        that tokens were evicted from keeps its pages, since the host does not know its length)."""
        if self._free is None:
            raise RuntimeError("the caller's block table is the caller's to fill")
        self.reset([seq])
        self.block_table[seq].fill_(-1)
        self._free.extend(reversed(self._pages[seq]))
        self._pages[seq] = []

    # ---------------------------------------------------------------- calls
    def reset(self, seqs: Sequence[int] | None = None) -> None:
        """Empty sequences (None: the first SR_MAX_PAGED_SEQS rows, or all where there are fewer)."""
        n = min(self.max_seqs, N.SR_MAX_PAGED_SEQS) if seqs is None else len(seqs)
        ids, at = self._ids(seqs)
        self._done(self._lib.sr_paged_reset(self.handle, at, n, self._stream()), "sr_paged_reset")

    def append(self, k: torch.Tensor, v: torch.Tensor, seqs: Sequence[int] | None = None,
               counts: Sequence[int] | None = None) -> None:
        """Append rows [rows][n_kv_heads][head_dim] bf16: one per sequence, or counts[i] for sequence seqs[i]."""
        rows = k.shape[0]
        shape = (rows, self.n_kv_heads, self.head_dim)
        self._check("k", k, shape)
        self._check("v", v, shape)
        n = self._seqs_of("k and v have", rows, seqs, counts)
        ids, at = self._ids(seqs)
        each, each_at = self._ids(counts)
        self._done(self._lib.sr_paged_append(self.handle, at, each_at, n, k.data_ptr(), v.data_ptr(), self._stream()),
                   "sr_paged_append")

    def attention(self, q: torch.Tensor, seqs: Sequence[int] | None = None, out: torch.Tensor | None = None,
                  lse: torch.Tensor | bool | None = None, mass_decay: float | None = None):
        """Attention of one new token per sequence, q [n][n_heads][head_dim]; returns out, or (out, lse)
        when lse is True or a tensor [n][n_heads] fp32. mass_decay: a number >= 0 also accumulates
        token_mass = mass_decay * token_mass + the tokens' weights summed over heads (of all sequences or, where
        they share pages and hold more tokens than the pool, of none: error_status() tells)."""
        n = q.shape[0]
        shape = (n, self.n_heads, self.head_dim)
        self._check("q", q, shape)
        if seqs is not None and len(seqs) != n:
            raise ValueError(f"q has {n} rows for {len(seqs)} sequences")
        if mass_decay is not None and mass_decay < 0:
            raise ValueError("mass_decay must be >= 0")
        if out is None:
            out = torch.empty_like(q)
        else:
            self._check("out", out, shape)
        if lse is True:
            lse = torch.empty((n, self.n_heads), dtype=torch.float32, device=self.device)
        elif isinstance(lse, torch.Tensor):
            self._check("lse", lse, (n, self.n_heads), torch.float32)
        else:
            lse = None
        ids, at = self._ids(seqs)
        self._done(self._lib.sr_paged_attention(self.handle, at, n, q.data_ptr(), out.data_ptr(),
                                                None if lse is None else lse.data_ptr(),
                                                -1.0 if mass_decay is None else mass_decay, self._stream()),
                   "sr_paged_attention")
        return out if lse is None else (out, lse)

    def prompt_attention(self, q: torch.Tensor, counts: Sequence[int] | None = None, seqs: Sequence[int] | None = None,
                         out: torch.Tensor | None = None, lse: torch.Tensor | bool | None = None, causal: bool = True):
        """Attention of the last counts[i] tokens of sequence seqs[i] (None: one each), appended before: q
        [rows][n_heads][head_dim], the sequences' rows back to back. causal: a row sees the tokens up to its own, else all
        that its sequence holds. Returns out, or (out, lse) when lse is True or a tensor [rows][n_heads] fp32. Calls of a
        few rows to each sequence and calls with more take different kernels (sr_paged_prompt_attention in include/sr.h
        has the rule and the times): over 4-bit pages single tokens are faster in a call without prompts."""
        rows = q.shape[0]
        shape = (rows, self.n_heads, self.head_dim)
        self._check("q", q, shape)
        n = self._seqs_of("q has", rows, seqs, counts)
        if out is None:
            out = torch.empty_like(q)
        else:
            self._check("out", out, shape)
        if lse is True:
            lse = torch.empty((rows, self.n_heads), dtype=torch.float32, device=self.device)
        elif isinstance(lse, torch.Tensor):
            self._check("lse", lse, (rows, self.n_heads), torch.float32)
        else:
            lse = None
        ids, at = self._ids(seqs)
        each, each_at = self._ids(counts)
        self._done(self._lib.sr_paged_prompt_attention(self.handle, at, each_at, n, q.data_ptr(), out.data_ptr(),
                                                       None if lse is None else lse.data_ptr(), 1 if causal else 0,
                                                       self._stream()), "sr_paged_prompt_attention")
        return out if lse is None else (out, lse)

    def read(self, counts: Sequence[int] | None = None, seqs: Sequence[int] | None = None,
             first: Sequence[int] | None = None, k: torch.Tensor | None = None, v: torch.Tensor | None = None):
        """Tokens back in bf16: counts[i] of sequence seqs[i] (None: one each), from index first[i] on, or (None) its
        last ones. Returns k, v [rows][n_kv_heads][head_dim] (the given tensors, or new ones), the sequences' rows back to
        back; rows that a sequence does not hold are zero."""
        n = len(counts) if counts is not None else len(seqs) if seqs is not None else len(first) if first is not None \
            else min(self.max_seqs, N.SR_MAX_PAGED_SEQS)
        for name, given in (("seqs", seqs), ("first", first)):
            if given is not None and len(given) != n:
                raise ValueError(f"{len(given)} {name} for {n} sequences")
        if counts is not None and n > 0 and min(counts) < 0:
            raise N.SrError(N.SR_ERR_INVALID_ARG, "sr_paged_read")
        shape = (n if counts is None else int(sum(counts)), self.n_kv_heads, self.head_dim)
        if k is None:
            k = torch.empty(shape, dtype=_BF16, device=self.device)
        else:
            self._check("k", k, shape)
        if v is None:
            v = torch.empty(shape, dtype=_BF16, device=self.device)
        else:
            self._check("v", v, shape)
        ids, at = self._ids(seqs)
        start, start_at = self._ids(first)
        each, each_at = self._ids(counts)
        self._done(self._lib.sr_paged_read(self.handle, at, start_at, each_at, n, k.data_ptr(), v.data_ptr(),
                                           self._stream()), "sr_paged_read")
        return k, v

    def evict(self, budget: int, n_sink: int = 0, n_recent: int = 0, seqs: Sequence[int] | None = None) -> None:
        """Keep at most `budget` tokens per sequence: positions below n_sink, the last n_recent
        positions, and the tokens with the largest token_mass (None: the first
        SR_MAX_PAGED_SEQS rows, or all where there are fewer). A sequence whose moves meet an entry that
        is no page of the pool stays as it is: error_status() tells."""
        if not (0 <= n_sink < 1 << 31 and 0 <= n_recent < 1 << 31 and budget >= 0):
            raise N.SrError(N.SR_ERR_INVALID_ARG, "sr_paged_evict")
        budget = min(budget, (1 << 31) - 1)                      # no sequence is longer
        n = min(self.max_seqs, N.SR_MAX_PAGED_SEQS) if seqs is None else len(seqs)
        ids, at = self._ids(seqs)
        self._done(self._lib.sr_paged_evict(self.handle, at, n, budget, n_sink, n_recent, self._stream()),
                   "sr_paged_evict")

    # ---------------------------------------------------------------- state
    def error_status(self) -> int:
        """Synchronises and maps the device error word to a status."""
        return N.sr_device_error_status(int(self.err_word.item()))

    def close(self) -> None:
        if self.handle is not None:
            N.sr_paged_free(self.handle)
            self.handle = None

    def __del__(self):
        try:
            self.close()
        except Exception:
            pass

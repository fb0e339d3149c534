"""The paged token cache in float64 (test infrastructure only).

Sequences are kept by logical index: pages are a matter of the layout, so the
tests read the GPU's pages back through the block table and compare them with
the rows held here. Values are float64; what the cache stores in 8 bits is
rounded here by its definition.
"""
import numpy as np


def round_e4m3(x: np.ndarray) -> np.ndarray:
    """Nearest e4m3 value (3 fraction bits, exponents 2^-6 .. 2^8, subnormals below), ties
    to even, saturating at 448; NaN stays."""
    x = np.asarray(x, np.float64)
    a = np.abs(x)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.floor(np.log2(np.where(a > 0, a, 1.0)))
    step = 2.0 ** (np.maximum(e, -6.0) - 3.0)
    with np.errstate(invalid="ignore"):
        y = np.rint(np.where(np.isfinite(a), a, 0.0) / step) * step
    y = np.minimum(np.where(np.isinf(a), 448.0, y), 448.0)
    return np.where(np.isnan(x), np.nan, np.copysign(y, x))


def round_int4(x: np.ndarray) -> np.ndarray:
    """What 4-bit pages hold for values x [..., 16 n]: blocks of 16 as integers -8 .. 7 times a scale of four
    significant bits (a multiple of 2^-17), max |x| / 7 rounded with halves up, at most 3840; quotients round with halves
    away from zero. A block with a NaN is NaN."""
    x = np.asarray(x, np.float64)
    b = x.reshape(*x.shape[:-1], x.shape[-1] // 16, 16)
    nan = np.isnan(b).any(-1, keepdims=True)
    b = np.where(nan, 0.0, b)
    want = np.minimum(np.abs(b).max(-1, keepdims=True) / 7.0, 3840.0)
    _, e = np.frexp(np.maximum(want, 2.0 ** -14))
    step = np.ldexp(1.0, e - 4)
    scale = np.floor(want / step + 0.5) * step
    with np.errstate(invalid="ignore"):
        t = np.where(scale > 0, b / np.where(scale > 0, scale, 1.0), 0.0)
    c = np.clip(np.copysign(np.floor(np.abs(t) + 0.5), t), -8, 7)
    return np.where(nan, np.nan, c * scale).reshape(x.shape)


class OraclePagedCache:
    """k, v: [max_seqs][cap][n_kv][d]; pos, mass: [max_seqs][cap]; length, next_pos: [max_seqs]."""

    def __init__(self, n_heads, n_kv, d, max_seqs, cap, e4m3=False, kv_exp=None, scale=None,
                 int4=False):
        self.n_heads, self.n_kv, self.d, self.cap = n_heads, n_kv, d, cap
        self.scale = 1.0 / np.sqrt(d) if scale is None else float(scale)
        self.e4m3, self.int4 = e4m3, int4
        self.exp = np.zeros((2, n_kv)) if kv_exp is None else np.asarray(kv_exp, np.float64)
        self.k = np.zeros((max_seqs, cap, n_kv, d))
        self.v = np.zeros((max_seqs, cap, n_kv, d))
        self.pos = np.zeros((max_seqs, cap), np.int64)
        self.mass = np.zeros((max_seqs, cap))
        self.length = np.zeros(max_seqs, np.int64)
        self.next_pos = np.zeros(max_seqs, np.int64)

    def reset(self, seqs):
        for s in seqs:
            self.length[s] = self.next_pos[s] = 0

    def stored(self, x, which):
        """What the cache holds for rows x [n][n_kv][d] of the keys (which 0) or the values (1)."""
        x = np.asarray(x, np.float64)
        if not self.e4m3 and not self.int4:
            return x
        s = (2.0 ** self.exp[which])[:, None]
        return (round_int4 if self.int4 else round_e4m3)(x / s) * s

    def append(self, seqs, counts, k, v):
        r = 0
        for s, n in zip(seqs, counts):
            a, b = self.length[s], self.length[s] + n
            assert b <= self.cap
            self.k[s, a:b] = self.stored(k[r:r + n], 0)
            self.v[s, a:b] = self.stored(v[r:r + n], 1)
            self.pos[s, a:b] = self.next_pos[s] + np.arange(n)
            self.mass[s, a:b] = 0.0
            self.length[s] = b
            self.next_pos[s] += n
            r += n

    def weights(self, s, q, visible=None):
        """x [n_heads][len] scaled scores, w their softmax, lse; visible: a mask of the tokens."""
        n = self.length[s]
        g = self.n_heads // self.n_kv
        x = np.einsum("hgd,thd->hgt", np.asarray(q, np.float64).reshape(self.n_kv, g, self.d), self.k[s, :n])
        x = (x * self.scale).reshape(self.n_heads, n)
        if visible is not None:
            x = np.where(visible[None, :], x, -np.inf)
        if n == 0 or (visible is not None and not visible.any()):
            return x, np.zeros_like(x), np.full(self.n_heads, -np.inf)
        top = x.max(1, keepdims=True)
        e = np.exp(x - top)
        total = e.sum(1, keepdims=True)
        return x, e / total, (top + np.log(total))[:, 0]

    def attention(self, seqs, q, mass_decay=None, visible=None):
        """Returns o [n][n_heads][d], lse [n][n_heads], and sum w|v| [n][n_heads][d] (for error bounds)."""
        out, lses, bounds = [], [], []
        g = self.n_heads // self.n_kv
        for i, s in enumerate(seqs):
            n = self.length[s]
            vis = None if visible is None else visible[i]
            _, w, lse = self.weights(s, q[i], vis)
            v = self.v[s, :n]
            if vis is not None:
                v = np.where(vis[:, None, None], v, 0.0)
            wg = w.reshape(self.n_kv, g, n)
            out.append(np.einsum("hgt,thd->hgd", wg, v).reshape(self.n_heads, self.d))
            bounds.append(np.einsum("hgt,thd->hgd", wg, np.abs(v)).reshape(self.n_heads, self.d))
            lses.append(lse)
            if mass_decay is not None:
                seen = slice(0, n) if vis is None else np.nonzero(vis)[0]
                self.mass[s, seen] = mass_decay * self.mass[s, seen] + w.sum(0)[seen if vis is not None else slice(None)]
        return np.stack(out), np.stack(lses), np.stack(bounds)

    def prompt_attention(self, seqs, counts, q, causal=True, visible=None):
        """As attention, for the last counts[i] tokens of each sequence; q [rows][n_heads][d]. visible: masks of the
        tokens, one per sequence."""
        out, lses, bounds = [np.zeros((0, self.n_heads, self.d))], [np.zeros((0, self.n_heads))], [np.zeros((0, self.n_heads, self.d))]
        r = 0
        for i, (s, m) in enumerate(zip(seqs, counts)):
            n = int(self.length[s])
            for j in range(m):
                mask = np.arange(n) < n - m + j + 1 if causal else np.ones(n, bool)
                if visible is not None:
                    mask &= visible[i]
                for dst, x in zip((out, lses, bounds), self.attention([s], q[r + j: r + j + 1], visible=[mask])):
                    dst.append(x)
            r += m
        return np.concatenate(out), np.concatenate(lses), np.concatenate(bounds)

    def read(self, seqs, counts, first=None):
        both = [np.zeros((sum(counts), self.n_kv, self.d)) for _ in range(2)]
        r = 0
        for i, (s, m) in enumerate(zip(seqs, counts)):
            n = int(self.length[s])
            t0 = n - m if first is None else first[i]
            for j in range(m):
                if 0 <= t0 + j < n:
                    both[0][r + j], both[1][r + j] = self.k[s, t0 + j], self.v[s, t0 + j]
            r += m
        return both

    def evict(self, seqs, budget, n_sink=0, n_recent=0):
        for s in seqs:
            n = int(self.length[s])
            if n <= budget:
                continue
            free = [t for t in range(n) if n_sink <= self.pos[s, t] < self.next_pos[s] - n_recent]
            # lightest first, of equal ones the last index; NaN is the heaviest
            free.sort(key=lambda t: (np.isnan(self.mass[s, t]), 0.0 if np.isnan(self.mass[s, t]) else self.mass[s, t], -t))
            gone = set(free[:n - budget])
            new = n - len(gone)
            holes = sorted(t for t in gone if t < new)
            back = [t for t in range(new, n) if t not in gone]
            assert len(holes) == len(back)
            for h, b in zip(holes, back):
                for x in (self.k, self.v, self.pos, self.mass):
                    x[s, h] = x[s, b]
            self.length[s] = new

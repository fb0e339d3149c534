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


class OraclePagedCache:
    """k, v: [max_seqs][cap][n_kv][d]; pos, mass: [max_seqs][cap]; length, next_pos: [max_seqs]."""

    def __init__(self, n_heads, n_kv, d, max_seqs, cap, e4m3=False, kv_exp=None, scale=None):
        self.n_heads, self.n_kv, self.d, self.cap = n_heads, n_kv, d, cap
        self.scale = 1.0 / np.sqrt(d) if scale is None else float(scale)
        self.e4m3 = e4m3
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
        if not self.e4m3:
            return x
        s = (2.0 ** self.exp[which])[:, None]
        return round_e4m3(x / s) * s

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

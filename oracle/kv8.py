"""Plain replay of the 8-bit paged cache's append -- TEST INFRASTRUCTURE ONLY
(see oracle/__init__.py).

Holds the cache as logical pages of float64 values: every value is an e4m3
number (`x`) with the page's power-of-two scale beside it.  Rows are taken one
page group at a time, in call order, in loops; the rotation is evaluated in
float32 with every product and sum rounded by itself, as the interface states.
"""
import numpy as np

E_MIN, E_MAX = -40, 40


def e4m3(x):
    """float64 -> nearest e4m3 value (ties to even), saturating at 448; NaN
    stays."""
    x = np.asarray(x, np.float64)
    with np.errstate(invalid="ignore"):
        y = np.clip(x, -448.0, 448.0)
        _, e = np.frexp(y)
        step = np.ldexp(1.0, np.maximum(e - 1, -6) - 3)
        return np.round(y / step) * step


def scale_for(amax):
    """Smallest power of two 2^e, e in [E_MIN, E_MAX], with amax <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and amax > np.ldexp(448.0, e):
        e += 1
    return np.ldexp(1.0, e)


def rotate(x, pos, cos_sin, interleaved):
    """x [heads, d] float32 turned by position pos."""
    rot = cos_sin.shape[1]
    c = cos_sin[pos, :rot // 2].astype(np.float32)
    s = cos_sin[pos, rot // 2:].astype(np.float32)
    ia = np.arange(rot // 2) * 2 if interleaved else np.arange(rot // 2)
    ib = ia + 1 if interleaved else ia + rot // 2
    y = x.astype(np.float32).copy()
    with np.errstate(invalid="ignore"):
        a, b = y[:, ia].copy(), y[:, ib].copy()
        y[:, ia] = a * c - b * s
        y[:, ib] = b * c + a * s
    return y


class Kv8Replay:
    """k, v [n_pages, H, page, d] float64 e4m3 values; k_scale, v_scale
    [n_pages, H]."""

    def __init__(self, H, d, page, n_pages, pos0, doc_table, seg_table):
        self.H, self.d, self.page, self.pos0 = H, d, page, pos0
        self.doc_table, self.seg_table = np.asarray(doc_table), np.asarray(seg_table)
        self.n_pages = n_pages
        self.k = np.zeros((n_pages, H, page, d))
        self.v = np.zeros((n_pages, H, page, d))
        self.k_scale = np.ones((n_pages, H))
        self.v_scale = np.ones((n_pages, H))

    def place(self, sid, pos):
        """(page, slot in page) of a token, or None where it has none."""
        slot = pos if sid == 0 else pos - self.pos0
        if pos < 0 or slot < 0 or sid > len(self.seg_table):
            return None
        tab = self.doc_table if sid == 0 else self.seg_table[sid - 1]
        if slot // self.page >= len(tab):
            return None
        pg = int(tab[slot // self.page])
        return (pg, slot % self.page) if 0 <= pg < self.n_pages else None

    def append(self, k, v, sid, pos, cos_sin=None, interleaved=False):
        """k, v [n, H, d] float32.  Returns the indices of dropped rows."""
        n = len(sid)
        dropped, runs_seen, groups = [], {}, {}
        for i in range(n):
            s, p = int(sid[i]), int(pos[i])
            if s < 0:
                continue
            if i == 0 or sid[i - 1] != s:
                start = runs_seen.setdefault(s, i)      # first run of the stream
                run, whole = i, True
            fits = p - int(pos[run]) == i - run
            afresh = (p if s == 0 else p - self.pos0) % self.page == 0
            whole = fits and (whole or afresh)          # no break in this page so far
            ok = start == run and whole
            at = self.place(s, p) if ok else None
            if at is None or (cos_sin is not None and p >= len(cos_sin)):
                dropped.append(i)
                continue
            groups.setdefault((s, at[0]), []).append((i, at[1], p))
        for (s, pg), rows in groups.items():
            for name, src in (("k", k), ("v", v)):
                pool, scale = getattr(self, name), getattr(self, name + "_scale")
                x = []
                for i, _, p in rows:
                    y = src[i].astype(np.float32)
                    if name == "k" and cos_sin is not None:
                        y = rotate(y, p, cos_sin, interleaved)
                    x.append(y.astype(np.float64))
                first = rows[0][1]
                for h in range(self.H):
                    vals = np.concatenate([y[h] for y in x])
                    vals = np.abs(vals[np.isfinite(vals)])
                    need = scale_for(vals.max() if vals.size else 0.0)
                    new = need if first == 0 else max(scale[pg, h], need)
                    if new > scale[pg, h] and first > 0:
                        pool[pg, h, :first] = e4m3(pool[pg, h, :first] * (scale[pg, h] / new))
                    scale[pg, h] = new
                    for (i, off, _), y in zip(rows, x):
                        pool[pg, h, off] = e4m3(y[h] / new)
            for i, off, _ in rows:          # a NaN value is kept by its key
                bad = np.isnan(self.v[pg, :, off])
                self.k[pg, bad.any(-1), off, 0] = np.nan
                self.v[pg, :, off][bad] = 0.0
        return dropped

    def rows(self, sid, count):
        """Dequantised (k, v) [count, H, d] of a stream's first tokens."""
        base = 0 if sid == 0 else self.pos0
        out = [[], []]
        for t in range(count):
            pg, off = self.place(sid, base + t)
            out[0].append(self.k[pg, :, off] * self.k_scale[pg][:, None])
            out[1].append(self.v[pg, :, off] * self.v_scale[pg][:, None])
        z = np.zeros((0, self.H, self.d))
        return tuple(np.stack(o) if o else z for o in out)

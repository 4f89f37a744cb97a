"""Plain numpy implementations, in 64 bits, of the MXFP4 and 8-bit cache operators."""
import numpy as np

E2M1 = np.array([0, 0.5, 1, 1.5, 2, 3, 4, 6], np.float64)
E2M1_ALL = np.concatenate([E2M1, -E2M1])


def _e4m3_table():
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m / 8.0 * 2.0 ** -6, (1 + m / 8.0) * 2.0 ** (e - 7.0))
    v = np.where(c & 128, -v, v)
    v[[127, 255]] = np.nan
    return v


E4M3 = _e4m3_table()


def _nearest(a, table):
    """Index of the nearest table value (ascending, from 0); ties to the even index, past the end the last."""
    hi = np.clip(np.searchsorted(table, a), 1, len(table) - 1)
    lo = hi - 1
    dl, dh = a - table[lo], table[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return np.where(up, hi, lo)


def e8m0(e):
    e = np.asarray(e).astype(np.int64)
    return np.where(e == 255, np.nan, np.ldexp(1.0, e - 127))


def encode_mxfp4(x):
    """x [rows, n] float64 -> codes uint8 [rows, n/2], scales uint8 [rows, n/32]."""
    rows, n = x.shape
    b = np.asarray(x, np.float64).reshape(rows, n // 32, 32)
    bad = ~np.isfinite(b).all(-1)
    b = np.where(bad[..., None], 0.0, b)
    _, e = np.frexp(np.abs(b).max(-1))
    scale = np.clip(e - 1 - 2 + 127, 0, 254)
    scale = np.where(np.abs(b).max(-1) == 0, 0, scale)
    a = np.abs(b) / np.ldexp(1.0, scale - 127)[..., None]
    codes = _nearest(np.minimum(a, 6.0), E2M1) + 8 * np.signbit(b)
    codes = np.where(bad[..., None], 0, codes).astype(np.uint8).reshape(rows, n)
    return codes[:, 0::2] | codes[:, 1::2] << 4, np.where(bad, 255, scale).astype(np.uint8)


def decode_mxfp4(codes, scales):
    c = np.stack([codes & 15, codes >> 4], -1).reshape(codes.shape[0], -1)
    return E2M1_ALL[c] * np.repeat(e8m0(scales), 32, axis=1)


def page_exponent(x):
    """Smallest biased exponent with every finite |x| / 2^(e-127) <= 448, 0 at least."""
    a = np.abs(x[np.isfinite(x)])
    e = 0
    if a.size and a.max() > 0:
        m, p = np.frexp(a.max())  # a = m 2^p, m in [1/2, 1)
        e = max(0, p - 1 - 8 + (1 if m > 0.875 else 0) + 127)
    return e


def encode_e4m3(a):
    """Values of at most 448 -> codes; NaN and infinities -> NaN codes."""
    finite = np.isfinite(a)
    v = np.where(finite, a, 0.0)
    c = _nearest(np.abs(v), E4M3[:127]) + 128 * np.signbit(v)
    return np.where(finite, c, 127).astype(np.uint8)


class Cache:
    """Pages as the library lays them out: k [pages, heads, page, dim], v [pages, heads, dim, page]."""

    def __init__(self, pages, heads, dim, page, rng=None):
        self.k = np.zeros((pages, heads, page, dim), np.uint8)
        self.v = np.zeros((pages, heads, dim, page), np.uint8)
        self.ks = np.zeros((pages, heads), np.uint8)
        self.vs = np.zeros((pages, heads), np.uint8)
        if rng is not None:  # whatever the pool held before, NaN codes and scales among it
            for t in (self.k, self.v, self.ks, self.vs):
                t[...] = rng.integers(0, 256, t.shape)
        self.page = page

    def append(self, k, v, table, lens, starts):
        for s in range(len(lens)):
            for i, t in enumerate(range(starts[s], starts[s + 1])):
                if lens[s] < 0:
                    break
                pos = lens[s] + i
                slot = pos % self.page
                if i and slot:
                    continue  # its page is done
                p = pos // self.page
                if p >= table.shape[1] or not 0 <= table[s, p] < len(self.k):
                    continue
                n = min(self.page - slot, starts[s + 1] - t)
                for x, codes, scales in ((k, self.k, self.ks), (v, self.v.transpose(0, 1, 3, 2), self.vs)):
                    for h in range(x.shape[1]):
                        self._put(codes[table[s, p], h], scales, (table[s, p], h), x[t:t + n, h], slot)

    @staticmethod
    def _put(page, scales, at, x, slot):
        e = page_exponent(x)
        if slot:
            old = int(scales[at])
            e = max(e, old)
            if e > old:
                page[:slot] = encode_e4m3_keeping_nan(page[:slot], old - e)
        page[slot:slot + len(x)] = encode_e4m3(x / np.ldexp(1.0, e - 127))
        scales[at] = e

    def rows(self, table, s, n):
        """K and V of the first n positions of a sequence: [heads, n, dim] each."""
        ids = table[s, :-(-n // self.page)]
        k = E4M3[self.k[ids]] * e8m0(self.ks[ids])[..., None, None]
        v = E4M3[self.v[ids].transpose(0, 1, 3, 2)] * e8m0(self.vs[ids])[..., None, None]
        heads, dim = k.shape[1], k.shape[3]
        return (k.transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n],
                v.transpose(1, 0, 2, 3).reshape(heads, -1, dim)[:, :n])


def encode_e4m3_keeping_nan(codes, shift):
    v = E4M3[codes] * np.ldexp(1.0, shift)
    return np.where(np.isnan(v), codes, encode_e4m3(np.where(np.isnan(v), 0.0, v))).astype(np.uint8)


def attend(q, cache, table, lens, scale, window=0):
    """q [seqs, q_len, heads, dim] float64 -> (out, sum of p|v|, bound on a score's sum of |q k|)."""
    seqs, q_len, heads, dim = q.shape
    out, weight, size = np.zeros(q.shape), np.zeros(q.shape), np.zeros(q.shape[:3] + (1,))
    group = heads // cache.k.shape[1]
    for s in range(seqs):
        n = int(lens[s])
        if n <= 0:
            continue
        k, v = cache.rows(table, s, n)
        for t in range(q_len):
            hi = n - q_len + t + 1
            lo = max(0, hi - window) if window else 0
            if hi <= lo:
                continue
            for h in range(heads):
                kk, vv = k[h // group, lo:hi], v[h // group, lo:hi]
                x = kk @ q[s, t, h] * scale
                p = np.exp(x - x.max())
                p /= p.sum()
                out[s, t, h], weight[s, t, h] = p @ vv, p @ np.abs(vv)
                size[s, t, h] = (np.abs(kk) @ np.abs(q[s, t, h])).max() * abs(scale)
    return out, weight, size

"""The attention operators of a tensor-parallel layer in fp64, written out
plainly (test infrastructure only), each result with a bound on the error of
the GPU's arithmetic.

Readings taken (the common forms):

  norm and rotation of a head x:  n = x / sqrt(mean(x^2) + eps), y = n w,
      (y_j, y_j') -> (y_j cos a - y_j' sin a, y_j' cos a + y_j sin a),
      a = pos freq_j, for the pairs (j, j + rot / 2) or (2 j, 2 j + 1);
      backward: g = dout turned back, dn = g w,
      dx = (dn - n mean(dn n)) / sqrt(mean(x^2) + eps), dw = sum g n
  cache: codes of e4m3 (bias 7, NaN 0x7f) times 2^(b - 127), b the smallest
      that brings a page's largest value to 448
  attention: z = scale q k, softmax over what the row sees, times v

The bounds count roundings: one is off by at most half a step, e = 2^-24
relative in fp32, `step` = 2^-8 in bf16 (e again where the payload is fp32).
"""

import numpy as np

from .layer import E, TINY, step


# ---- norms and rotation ----


def turn(y, pos, freq, pairs, back=False):
    """[rows, heads, dim] turned by pos * freq, and the same of magnitudes."""
    rot = 2 * len(freq)
    a = pos.astype(np.float64)[:, None] * freq.astype(np.float64)[None]
    c, s = np.cos(a)[:, None], np.sin(a)[:, None] * (-1 if back else 1)
    out, size = y.copy(), np.abs(y)
    first = np.s_[..., 0:rot:2] if pairs else np.s_[..., :rot // 2]
    second = np.s_[..., 1:rot:2] if pairs else np.s_[..., rot // 2:rot]
    p, q = y[first], y[second]
    out[first], out[second] = p * c - q * s, q * c + p * s
    size[first] = np.abs(p * c) + np.abs(q * s)
    size[second] = np.abs(q * c) + np.abs(p * s)
    # an angle is off by 2^-25 half turns of its fraction in fp32: 1e-7
    whole = np.zeros_like(y)
    whole[first] = whole[second] = np.abs(p) + np.abs(q)
    return out, size, whole


def norm_rope(x, w, pos, freq, pairs, eps, dt):
    """(out, bound)"""
    d = x.shape[-1]
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    y = x * inv * w
    out, size, whole = turn(y, pos, freq, pairs)
    # inv: a sum of d squares and some roundings; y two more, the turn two more
    err = size * ((d / 2 + 12) * E) + whole * (8 * E) + TINY
    return out, err + step(dt) * (np.abs(out) + err)


def norm_rope_backward(dout, x, w, pos, freq, pairs, eps, dt):
    """((dx, bound), (dw, bound))"""
    d = x.shape[-1]
    inv = 1.0 / np.sqrt((x * x).mean(-1, keepdims=True) + eps)
    n = x * inv
    g, size, whole = turn(dout, pos, freq, pairs, back=True)
    eg = size * (3 * E) + whole * (8 * E)
    dn, edn = g * w, eg * np.abs(w) + np.abs(g * w) * E
    rn = (d / 2 + 12) * E  # of n and inv, relative
    dot = (dn * n).mean(-1, keepdims=True)
    edot = (edn * np.abs(n)).mean(-1, keepdims=True) + np.abs(dn * n).mean(-1, keepdims=True) * (rn + (d + 4) * E)
    dx = inv * (dn - n * dot)
    parts = np.abs(dn) + np.abs(n * dot)
    edx = inv * (edn + np.abs(n) * edot + parts * (2 * rn + 6 * E)) + TINY
    dw = (g * n).sum((0, 1))
    terms = x.shape[0] * x.shape[1]
    edw = (eg * np.abs(n)).sum((0, 1)) + np.abs(g * n).sum((0, 1)) * (rn + (terms + 2) * E) + TINY
    return (dx, edx + step(dt) * (np.abs(dx) + edx)), (dw, edw + step(dt) * (np.abs(dw) + edw))


# ---- the cache ----


def code_values():
    """The value of every e4m3 code."""
    c = np.arange(256)
    e, m = (c >> 3) & 15, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    v = np.where((c & 127) == 127, np.nan, v)
    return np.where(c >= 128, -v, v)


VALUES = code_values()


def scale_byte(m):
    """The smallest b in [1, 254] with m <= 448 * 2^(b - 127)."""
    b = 1
    while b < 254 and m > 448.0 * 2.0 ** (b - 127):
        b += 1
    return b


def encode(y):
    """Nearest codes of |y| <= 448, ties to even; NaN for what is not finite."""
    grid = VALUES[:127]
    a = np.abs(np.where(np.isfinite(y), y, 0.0))
    hi = np.clip(np.searchsorted(grid, a), 1, 126)
    lo = hi - 1
    dl, dh = a - grid[lo], grid[hi] - a
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    code = np.where(np.signbit(y), code | 128, code)
    return np.where(np.isfinite(y), code, 0x7f).astype(np.uint8)


class Cache:
    """One rank's cache: k and v codes [pages, heads, page, dim], scales [pages, heads]."""

    def __init__(self, pages, heads, page, dim, rng=None):
        self.page, self.heads, self.dim, self.pages = page, heads, dim, pages
        make = (lambda *s: rng.integers(0, 256, s, dtype=np.uint8)) if rng is not None else (lambda *s: np.zeros(s, np.uint8))
        self.codes = [make(pages, heads, page, dim) for _ in range(2)]
        self.scale = [np.full((pages, heads), 120, np.uint8) if rng is None else
                      rng.integers(110, 130, (pages, heads), dtype=np.uint8) for _ in range(2)]

    def write(self, new, table, first, at):
        """new: (k, v) [rows, heads, dim] in fp64."""
        for s in range(len(at)):
            n, start = int(first[s + 1] - first[s]), max(int(at[s]), 0)
            for j in range(start // self.page, (start + n - 1) // self.page + 1 if n > 0 else 0):
                if j >= table.shape[1] or not 0 <= table[s, j] < self.pages:
                    continue
                lo, hi = max(start, j * self.page), min(start + n, (j + 1) * self.page)
                row, a, b = first[s] + lo - start, lo - j * self.page, hi - j * self.page
                for i in range(2):
                    for h in range(self.heads):
                        x = new[i][row:row + hi - lo, h]
                        codes, old = self.codes[i][table[s, j], h], int(self.scale[i][table[s, j], h])
                        fin = np.abs(x[np.isfinite(x)])
                        byte = scale_byte(fin.max() if fin.size else 0.0)
                        if a > 0:
                            byte = max(byte, old)
                            if byte > old:
                                codes[:a] = encode(VALUES[codes[:a]] * 2.0 ** (old - byte))
                        codes[a:b] = encode(x / 2.0 ** (byte - 127))
                        self.scale[i][table[s, j], h] = byte

    def tokens(self, i, s, table, start, n):
        """([n, heads, dim] values, [n] on a page) of sequence s."""
        out, there = np.zeros((n, self.heads, self.dim)), np.zeros(n, bool)
        for t in range(n):
            j = (start + t) // self.page
            if j < table.shape[1] and 0 <= table[s, j] < self.pages:
                p = table[s, j]
                out[t] = VALUES[self.codes[i][p, :, (start + t) % self.page]] * 2.0 ** (self.scale[i][p].astype(float) - 127)[:, None]
                there[t] = True
        return out, there


# ---- attention ----


def attention(q, cache, table, first, length, scale, causal, window, dt, terms):
    """((out, bound), (lse, bound)); rows of no sequence are NaN.  terms: bf16
    terms of the weights (1: 2^-8 relative, 2: 2^-16, 3: 2^-24)."""
    rows, heads, dim = q.shape
    group = heads // cache.heads
    out, eout = np.full(q.shape, np.nan), np.zeros(q.shape)
    lse, elen = np.full((rows, heads), np.nan), np.zeros((rows, heads))
    pr = 2.0 ** (-8 * terms)
    for s in range(len(length)):
        n = int(first[s + 1] - first[s])
        if n <= 0:
            continue
        total = max(0, min(int(length[s]), table.shape[1] * cache.page))
        k, there = cache.tokens(0, s, table, 0, total)
        v, _ = cache.tokens(1, s, table, 0, total)
        at = np.arange(total)
        for i in range(n):
            see = there.copy()
            if causal:
                p = total - n + i
                see &= at <= p
                if window:
                    see &= at > p - window
            r = first[s] + i
            for h in range(heads):
                kk, vv, x = k[see, h // group], v[see, h // group], q[r, h]
                if not len(kk):
                    out[r, h], lse[r, h] = 0.0, -np.inf
                    continue
                z = kk @ x * scale
                size = np.abs(kk) @ np.abs(x) * abs(scale)
                # a product of dim terms, each in up to three parts, in any order; what
                # three bf16 terms leave of a query is at most 2^-24 of it
                ez = size * (3 * dim + 6) * E
                m = z.max()
                w = np.exp(z - m)
                w /= w.sum()
                # the exponent is rounded (factor, product, difference), and rescaled
                rel = ez + (np.abs(z) + abs(m) + 8) * 4 * E + 8 * E
                o = w @ vv
                mag = w @ np.abs(vv)
                both = np.abs(vv) + np.abs(o)[None]
                err = (w * rel) @ both + (w @ rel) * np.abs(o) + pr * (w @ both) + (len(kk) + 20) * 3 * E * (mag + np.abs(o)) + TINY
                out[r, h], eout[r, h] = o, err + step(dt) * (np.abs(o) + err)
                lse[r, h] = m + np.log(np.exp(z - m).sum())
                elen[r, h] = w @ rel + (len(kk) + 20) * E + 4 * E * (abs(lse[r, h]) + abs(m) + 1)
    return (out, eout), (lse, elen)

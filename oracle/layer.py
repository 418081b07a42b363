"""The operators of a tensor-parallel layer in fp64, written out plainly (test
infrastructure only), each result with a bound on the error of the GPU's
arithmetic.

"NCCL collectives, ring all-reduce & launching TP/PP", section "Direct
answer", names the column-then-row split that leaves partial sums; the page
gives no formulas.  Readings taken (the common forms):

  gated feed-forward, one rank:  g = x Wg^T, u = x Wu^T, h = act(g) u,
      out = h Wd^T;  dh = dout Wd, dg = dh u act'(g), du = dh act(g),
      dx = dg Wg + du Wu, dWg = dg^T x, dWu = du^T x, dWd = dout^T h
  cross entropy:  l = x W^T, lse = log sum exp(l), loss = lse - l_target;
      d = (exp(l - lse) - onehot) grad, dx = d W, dW = d^T x

Every function takes and returns fp64 arrays and returns (value, bound)
pairs.  The bounds: a product of k terms summed in fp32 in any order is off by
at most k e S, S the sum of the terms' magnitudes and e = 2^-24 (one rounding
is off by at most half a step: 2^-24 relative in fp32, `step` = 2^-8 in bf16,
2^-24 again where the payload is fp32).  An operand that is itself off by b
adds sum b |w|.  A value rounded to the payload type adds step |value|.  An
activation and its derivative are at most 16 fp32 roundings of values of
magnitude at most 1 + |value| each, and change by at most 1.2 (2 for the
derivative) times a change of their argument.

`terms`: the bf16 terms an intermediate (h, dg, du, d) is kept in.  With two, its
error is at most step^2 |value| (what rounding leaves is exact in fp32, at most
step |value|, and rounded once more), a product sums twice as many terms, and
the result's bound is the sharper `nearest`, under which a lost or misplaced
second term shows.
"""

import math

import numpy as np

E = 2.0 ** -24
TINY = 1e-30  # below any value compared: gradual underflow of single terms


def step(dt):
    return 2.0 ** -8 if dt == "bf16" else E


def _erfc(z):
    return np.vectorize(math.erfc, otypes=[np.float64])(z) if z.size else z


def act(z, name):
    """(act(z), act'(z)) in fp64."""
    if name == "silu":
        s = np.where(z >= 0, 1.0 / (1.0 + np.exp(-np.abs(z))), np.exp(-np.abs(z)) / (1.0 + np.exp(-np.abs(z))))
        return z * s, s + z * s * (1.0 - s)
    if name == "gelu":
        phi = 0.5 * _erfc(-z / math.sqrt(2.0))
        return z * phi, phi + z * np.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    k = math.sqrt(2.0 / math.pi)
    t = np.tanh(k * (z + 0.044715 * z ** 3))
    return 0.5 * z * (1 + t), 0.5 * (1 + t) + 0.5 * z * (1 - t * t) * k * (1 + 3 * 0.044715 * z * z)


def product(a, b, ea=None, eb=None, terms=1):
    """a b^T and the bound on its fp32 evaluation; ea, eb bound the operands,
    one of which is in `terms` terms."""
    k = a.shape[1]
    size = np.abs(a) @ np.abs(b).T
    err = terms * k * E * size * (1 + 2.0 ** -7 * (terms - 1)) + TINY
    if ea is not None:
        err = err + ea @ np.abs(b).T
    if eb is not None:
        err = err + np.abs(a) @ eb.T
    return a @ b.T, err


def rounded(v, err, dt, terms=1):
    return v, err + step(dt) ** terms * (np.abs(v) + err)


def bf16_of(v):
    """The bf16 value nearest to an fp64 one, ties to even."""
    m, e = np.frexp(v)
    return np.ldexp(np.rint(np.ldexp(m, 8)), e - 8)


def nearest(v, err):
    """A value y within err of v, rounded to bf16: y's nearest is no further from
    y than v's nearest is, so off v by at most |bf16(v) - v| + 2 err."""
    return v, np.abs(bf16_of(v) - v) + 2 * err


def result(v, err, dt, terms):
    return nearest(v, err) if terms == 2 else rounded(v, err, dt)


def gated_ffn(x, wg, wu, wd, name, dt, terms=1):
    """{"gate", "up", "out"}: (value, bound) of one rank."""
    g, eg = product(x, wg)
    u, eu = product(x, wu)
    a, _ = act(g, name)
    ea = 1.2 * eg + 16 * E * (1 + np.abs(a))
    h = a * u
    _, eh = rounded(h, ea * (np.abs(u) + eu) + np.abs(a) * eu + E * np.abs(h), dt, terms)
    out, eo = product(h, wd, eh, terms=terms)
    return {"gate": (g, eg), "up": (u, eu), "out": result(out, eo, dt, terms)}


def gated_ffn_backward(dout, x, wg, wu, wd, g, u, name, dt, terms=1):
    """{"dx", "dw_gate", "dw_up", "dw_down"} of one rank, given the stored g and u."""
    dh, edh = product(dout, wd.T)
    a, da = act(g, name)
    ea, eda = 16 * E * (1 + np.abs(a)), 16 * E * (1 + np.abs(da))
    dg, du, h = dh * u * da, dh * a, a * u
    _, edg = rounded(dg, edh * np.abs(u) * (np.abs(da) + eda) + np.abs(dh * u) * eda + 2 * E * np.abs(dg), dt, terms)
    _, edu = rounded(du, edh * (np.abs(a) + ea) + np.abs(dh) * ea + E * np.abs(du), dt, terms)
    _, eh = rounded(h, np.abs(u) * ea + E * np.abs(h), dt, terms)
    # dx is one sum of 2 inter terms
    dx, edx = product(np.concatenate([dg, du], 1), np.concatenate([wg, wu], 0).T, np.concatenate([edg, edu], 1), terms=terms)
    dwg, edwg = product(dg.T, x.T, edg.T, terms=terms)
    dwu, edwu = product(du.T, x.T, edu.T, terms=terms)
    dwd, edwd = product(dout.T, h.T, None, eh.T, terms=terms)
    return {"dx": result(dx, edx, dt, terms), "dw_gate": result(dwg, edwg, dt, terms),
            "dw_up": result(dwu, edwu, dt, terms), "dw_down": result(dwd, edwd, dt, terms)}


def cross_entropy(x, w, target):
    """(loss, lse) of the whole vocabulary w, each (value, bound).

    The sum of exponentials: a term is off by the logit's error plus 2 e per
    unit of its distance from the maximum (the exponential's argument is
    rounded, and rescaled again when tiles join) plus a few roundings; the
    terms are joined in a chain of at most 40 + vocab / 128 additions, each
    with 4 roundings."""
    logits, el = product(x, w)
    rows, vocab = logits.shape
    top = logits.max(1) if vocab else np.full(rows, -np.inf)
    p = np.exp(logits - top[:, None])
    total = p.sum(1)
    lse = top + np.log(total)
    share = p / total[:, None]
    rel = (share * (el + 2 * E * np.abs(logits - top[:, None]))).sum(1) + 4 * E * (40 + vocab / 128.0)
    rel = rel + (el * el * share).sum(1)  # second order
    elen = rel + 4 * E * (np.abs(lse) + np.abs(top) + 1)
    live = (target >= 0) & (target < vocab)
    at = np.where(live, target, 0)
    i = np.arange(rows)
    loss = np.where(live, lse - logits[i, at], 0.0)
    eloss = np.where(live, elen + el[i, at] + 2 * E * np.abs(loss), 0.0)
    return (loss, eloss), (lse, elen)


def cross_entropy_backward(grad, x, w, target, lse, dt, first=0, vocab=None, terms=1):
    """(dx, dw) of the vocabulary rows w = W[first : first + len(w)], given the
    stored lse."""
    logits, el = product(x, w)
    rows, n = logits.shape
    vocab = n if vocab is None else vocab
    live = (target >= 0) & (target < vocab)
    g = np.where(live, grad, 0.0)[:, None]
    z = logits - lse[:, None]
    p = np.exp(z)
    hit = np.zeros_like(p)
    mine = live & (target >= first) & (target < first + n)
    hit[np.arange(rows)[mine], (target - first)[mine]] = 1.0
    ez = el + E * np.abs(z)
    ep = p * (np.expm1(ez) + 2 * E * np.abs(z) + 4 * E)
    d = (p - hit) * g
    _, ed = rounded(d, (ep + 2 * E * np.abs(p - hit)) * np.abs(g), dt, terms)
    dx, edx = product(d, w.T, ed, terms=terms)
    dw, edw = product(d.T, x.T, ed.T, terms=terms)
    # dx is added up over pieces of the vocabulary: as many terms, plus one
    # fp32 addition per piece, within the count of terms
    return result(dx, edx, dt, terms), result(dw, edw, dt, terms)

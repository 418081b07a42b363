"""Up to 32 rows, the layer operators keep their bf16 intermediates in two terms,
value and remainder.  Each result is held to the sharp bound of two terms
element by element, and its distance from fp64 to that of the result's own
rounding; on the host the same checks are shown to catch a second term that is
dropped, subtracted, or taken from another row or column.

The distance: an fp32 sum of k terms of random rounding errors is off by about
2^-24 sqrt(k) of the result, below 1e-5 of it here, so that it moves few
roundings to bf16 (2^-8 / sqrt(3) of a value in the mean) and the ratio stays
within a hundredth of 1; an intermediate of one term adds as much again (1.4).
NEAR lies between."""

import sys

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import layer
from tests.test_gpu_layer import f64, ffn_inputs, xent_inputs

NEAR = 1.1

# rows at both ends of the two layouts (second terms 8 and 32 rows below); odd
# widths, several tiles, several K steps
FFN = [(1, 64, 32), (8, 72, 130), (9, 200, 96), (32, 65, 33), (17, 128, 256), (5, 33, 100)]
XENT = [(1, 64, 96), (8, 40, 300), (9, 100, 130), (32, 65, 77), (24, 128, 256)]


def faults(got, want):
    """What is wrong with an fp64 array of results: elements beyond their bounds,
    or a distance beyond the result's own rounding."""
    value, bound = want
    beyond = ~(np.abs(got - value) <= bound)
    off = np.linalg.norm(got - value) / np.linalg.norm(layer.bf16_of(value) - value)
    return ([f"{int(beyond.sum())} of {beyond.size} beyond the bound"] if beyond.any() else []) + \
           ([f"{off:.3f} times the rounding's distance"] if off > NEAR else [])


# ---- the checks, on an emulation of the arithmetic and its mutants ----


def _bf(v):
    return layer.bf16_of(np.asarray(v, np.float64))


def _f32(v):
    return np.asarray(v, np.float32).astype(np.float64)


def _two(v, mutant):
    """(first, second) bf16 terms of an fp32 intermediate."""
    top = _bf(v)
    low = _bf(_f32(v - top))
    return top, {"": low, "dropped": 0 * low, "subtracted": -low, "other row": np.roll(low, 1, 0),
                 "other column": np.roll(low, 1, 1)}[mutant]


def _sum(pairs):
    """bf16 of the fp32 sum of products a b^T."""
    return _bf(sum((a.astype(np.float32) @ b.astype(np.float32).T for a, b in pairs), np.float32(0)))


def emulate_ffn(x, wg, wu, wd, dout, mutants):
    g, u = (_f32(x.astype(np.float32) @ w.astype(np.float32).T) for w in (wg, wu))
    a, da = layer.act(g, "silu")
    h = _f32(_f32(a) * u)
    terms = _two(h, mutants.get("h", ""))
    res = {"out": _sum([(t, wd) for t in terms])}
    dh = _f32(dout.astype(np.float32) @ wd.astype(np.float32))
    dg, du = _two(_f32(dh * u * da), mutants.get("dg", "")), _two(_f32(dh * a), mutants.get("du", ""))
    back = _two(h, mutants.get("h back", ""))
    res["dx"] = _sum([(t, wg.T) for t in dg] + [(t, wu.T) for t in du])
    res["dw_gate"], res["dw_up"] = (_sum([(t.T, x.T) for t in d]) for d in (dg, du))
    res["dw_down"] = _sum([(dout.T, t.T) for t in back])
    return g, u, res


def _numpy_ffn(rows, hidden, inter, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)  # the GPU tests' inputs, kept on the host
    return [f64(v[0]) for v in ffn_inputs(1, rows, hidden, inter, "bf16", rows)]


MUTANTS = ["dropped", "subtracted", "other row", "other column"]
READERS = {"h": ["out"], "dg": ["dx", "dw_gate"], "du": ["dx", "dw_up"], "h back": ["dw_down"]}


@pytest.mark.parametrize("rows,hidden,inter", FFN)
def test_the_checks_catch_a_wrong_second_term_of_the_feed_forward_block(rows, hidden, inter, monkeypatch):
    x, wg, wu, wd, dout = _numpy_ffn(rows, hidden, inter, monkeypatch)

    def wrong(mutants):
        g, u, got = emulate_ffn(x, wg, wu, wd, dout, mutants)
        want = layer.gated_ffn(x, wg, wu, wd, "silu", "bf16", terms=2)
        want.update(layer.gated_ffn_backward(dout, x, wg, wu, wd, g, u, "silu", "bf16", terms=2))
        return {k: faults(got[k], want[k]) for k in got}

    assert not any(wrong({}).values()), wrong({})
    for mid, readers in READERS.items():
        for mutant in MUTANTS:
            if mutant == "other row" and rows == 1:
                continue
            found = wrong({mid: mutant})
            assert all(found[k] for k in readers), (mid, mutant, found)
            assert not any(found[k] for k in found if k not in readers), (mid, mutant, found)


@pytest.mark.parametrize("rows,hidden,vocab", XENT)
def test_the_checks_catch_a_wrong_second_term_of_the_loss(rows, hidden, vocab, monkeypatch):
    monkeypatch.setattr(torch.Tensor, "cuda", lambda t: t)
    x, w, target, grad = xent_inputs(1, rows, hidden, vocab, "bf16", rows, ignored=0.0)
    x, w, grad, target = f64(x[0]), f64(w[0]), f64(grad), target.numpy()
    logits = _f32(x.astype(np.float32) @ w.astype(np.float32).T)
    lse = _f32(np.log(np.exp(logits).sum(1)))
    d = _f32(np.exp(_f32(logits - lse[:, None])))
    d[np.arange(rows), target] -= 1.0
    d = _f32(_f32(d) * grad[:, None])
    want = layer.cross_entropy_backward(grad, x, w, target, lse, "bf16", terms=2)
    for mutant in ["", *MUTANTS]:
        if mutant == "other row" and rows == 1:
            continue
        terms = _two(d, mutant)
        got = _sum([(t, w.T) for t in terms]), _sum([(t.T, x.T) for t in terms])
        for a, b in zip(got, want):
            assert bool(faults(a, b)) == bool(mutant), (mutant, faults(a, b))


def test_bf16_of_rounds_as_torch_does():
    v = np.random.default_rng(0).standard_normal(100000) * np.exp(np.random.default_rng(1).standard_normal(100000) * 9)
    v = np.concatenate([_f32(v), [1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8, -255.5, 0.0, 2.0 ** -100]])
    assert (layer.bf16_of(v) == torch.tensor(v).float().bfloat16().double().numpy()).all()


# ---- the kernels ----


def _say(*what):
    print("CASE", *what, flush=True, file=sys.stderr)


def _hold(got, want, what):
    found = faults(f64(got), want)
    assert not found, (what, found)


# ... with tiles' sums shared among workgroups (long K) as well
@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 3])
@pytest.mark.parametrize("rows,hidden,inter", FFN + [(5, 33, 8000), (30, 100, 4100), (1, 1024, 512)])
def test_feed_forward_results_are_as_near_as_two_terms_put_them(rows, hidden, inter, n):
    _say("ffn", n, rows, hidden, inter)
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, "bf16", rows)
    gate, up = ([torch.empty(rows, inter, device="cuda") for _ in range(n)] for _ in range(2))
    got = {"out": ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up)}
    got.update(zip(("dx", "dw_gate", "dw_up", "dw_down"), ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)))
    torch.cuda.synchronize()
    for r in range(n):
        args = [f64(v[r]) for v in (x, wg, wu, wd)]
        want = layer.gated_ffn(*args, "silu", "bf16", terms=2)
        want.update(layer.gated_ffn_backward(f64(dout[r]), *args, f64(gate[r]), f64(up[r]), "silu", "bf16", terms=2))
        for k in got:
            _hold(got[k][r], want[k], f"{k} rank {r}")


@pytest.mark.gpu
@pytest.mark.parametrize("n,piece", [(1, 0), (3, 0), (1, 256)])
@pytest.mark.parametrize("rows,hidden,vocab", XENT + [(20, 72, 9000), (2, 512, 3001)])
def test_loss_gradients_are_as_near_as_two_terms_put_them(rows, hidden, vocab, n, piece):
    _say("xent", n, rows, hidden, vocab, piece)
    x, w, target, grad = xent_inputs(n, rows, hidden, vocab, "bf16", rows, ignored=0.0)
    _, lse = ar.linear_cross_entropy(x, w, target)
    dx, dw = ar.linear_cross_entropy_backward(grad, x, w, target, lse, piece=piece)
    torch.cuda.synchronize()
    first = 0
    for r in range(n):
        want = layer.cross_entropy_backward(f64(grad), f64(x[0]), f64(w[r]), target.cpu().numpy(), f64(lse[r]), "bf16",
                                            first, vocab, terms=2)
        _hold(dx[r], want[0], f"dx rank {r}")
        _hold(dw[r], want[1], f"dw rank {r}")
        first += w[r].shape[0]

"""GPU: the operators of a tensor-parallel layer against their fp64
definitions, within the error bounds the oracle derives for each element."""

import sys

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import layer

pytestmark = pytest.mark.gpu

TORCH = {"f32": torch.float32, "bf16": torch.bfloat16}


def _say(*what):
    print("CASE", *what, flush=True, file=sys.stderr)


def _poison():
    """Memory the next allocations are likely to reuse, full of NaN."""
    for n in (1 << 14, 1 << 18, 1 << 22):
        t = [torch.full((n,), float("nan"), device="cuda") for _ in range(8)]
        del t


def _rand(gen, shape, dt, scale=1.0):
    return (torch.randn(shape, generator=gen) * scale).to(TORCH[dt]).cuda()


def f64(t):
    return t.detach().cpu().to(torch.float64).numpy()


def check(got, want, what):
    value, bound = want
    g = f64(got)
    assert g.shape == value.shape, (what, g.shape, value.shape)
    bad = ~(np.abs(g - value) <= bound)
    assert not bad.any(), (f"{what}: {int(bad.sum())} of {bad.size} beyond the bound, first at "
                           f"{np.argwhere(bad)[:4].tolist()}: got {g[bad][:4]} want {value[bad][:4]} "
                           f"bound {bound[bad][:4]}")


def ffn_inputs(n, rows, hidden, inter, dt, seed):
    gen = torch.Generator().manual_seed(seed)
    x = [_rand(gen, (rows, hidden), dt) for _ in range(n)]
    wg = [_rand(gen, (inter, hidden), dt, hidden ** -0.5) for _ in range(n)]
    wu = [_rand(gen, (inter, hidden), dt, hidden ** -0.5) for _ in range(n)]
    wd = [_rand(gen, (hidden, inter), dt, inter ** -0.5) for _ in range(n)]
    dout = [_rand(gen, (rows, hidden), dt) for _ in range(n)]
    return x, wg, wu, wd, dout


def run_ffn(n, rows, hidden, inter, dt, act, backward=True, seed=0, ranks=None):
    _say("ffn", n, rows, hidden, inter, dt, act)
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, dt, seed)
    _poison()
    gate = [torch.full((rows, inter), float("nan"), device="cuda") for _ in range(n)]
    up = [torch.full((rows, inter), float("nan"), device="cuda") for _ in range(n)]
    out = ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up, act=act)
    plain = ar.gated_ffn(x, wg, wu, wd, act=act)  # without keeping g and u: the same bits
    torch.cuda.synchronize()
    for r in (ranks or range(n)):
        want = layer.gated_ffn(f64(x[r]), f64(wg[r]), f64(wu[r]), f64(wd[r]), act, dt)
        check(gate[r], want["gate"], f"gate rank {r}")
        check(up[r], want["up"], f"up rank {r}")
        check(out[r], want["out"], f"out rank {r}")
        assert torch.equal(out[r], plain[r])
    if not backward:
        return
    _poison()
    got = dict(zip(("dx", "dw_gate", "dw_up", "dw_down"),
                   ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, act=act)))
    torch.cuda.synchronize()
    for r in (ranks or range(n)):
        want = layer.gated_ffn_backward(f64(dout[r]), f64(x[r]), f64(wg[r]), f64(wu[r]), f64(wd[r]), f64(gate[r]),
                                        f64(up[r]), act, dt)
        for k in got:
            check(got[k][r], want[k], f"{k} rank {r}")


FFN_SHAPES = [
    # rows, hidden, inter
    (1, 64, 32), (1, 1, 1), (2, 8, 8), (3, 7, 5), (16, 128, 64), (17, 200, 96), (5, 65, 33), (64, 256, 72),
    (127, 136, 130), (129, 72, 264), (200, 100, 100), (33, 264, 513), (300, 40, 24),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("rows,hidden,inter", FFN_SHAPES)
def test_ffn_shapes(rows, hidden, inter, dt):
    run_ffn(2, rows, hidden, inter, dt, "silu", seed=rows + hidden)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("n", [1, 3, 8])
def test_ffn_activations_and_ranks(n, act, dt):
    run_ffn(n, 21, 80, 56, dt, act, seed=n)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_ffn_large_tiles(dt):
    # enough 256 x 256 tiles to fill the GPU in every product of both passes;
    # rows, hidden and inner size end inside a tile
    run_ffn(8, 1288, 1160, 1416, dt, "silu", seed=5, ranks=(0, 7))


# Shapes that take the tile classes the ones above do not (n, rows, hidden, inter).
FFN_CLASS_SHAPES = [
    (8, 408, 112, 1160), (8, 776, 280, 1632), (8, 603, 40, 1368), (2, 605, 40, 1704), (8, 586, 1856, 72),
    (8, 763, 752, 32), (1, 1116, 1856, 32), (8, 1730, 432, 32), (2, 44, 1024, 72), (3, 18, 640, 130),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,inter", FFN_CLASS_SHAPES)
def test_ffn_tile_classes(n, rows, hidden, inter, dt):
    run_ffn(n, rows, hidden, inter, dt, "silu", seed=rows, ranks=(0, n - 1))


# Few results and a long K: several workgroups share each tile's sum.
FFN_SHARED_SHAPES = [(1, 11, 40, 7522), (2, 5, 33, 8000), (1, 40, 72, 6001), (1, 130, 64, 9000), (2, 30, 100, 4100)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,inter", FFN_SHARED_SHAPES)
def test_ffn_shared_sums(n, rows, hidden, inter, dt):
    run_ffn(n, rows, hidden, inter, dt, "silu", seed=rows)


# ... in other tile classes, the large one among them.
FFN_SHARED_CLASSES = [(2, 990, 528, 9524), (8, 500, 14, 28612), (8, 43, 110, 2126), (8, 152, 15, 13737), (1, 3, 625, 34035)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,inter", FFN_SHARED_CLASSES)
def test_ffn_shared_sums_of_every_class(n, rows, hidden, inter, dt):
    run_ffn(n, rows, hidden, inter, dt, "silu", seed=rows, ranks=(n - 1,))


def xent_inputs(n, rows, hidden, vocab, dt, seed, ignored=0.2):
    gen = torch.Generator().manual_seed(seed)
    x = _rand(gen, (rows, hidden), dt)
    w = [_rand(gen, (v, hidden), dt, 2.0 * hidden ** -0.5) for v in ar.vocab_shards(vocab, n)]
    target = torch.randint(0, vocab, (rows,), generator=gen)
    target[torch.rand(rows, generator=gen) < ignored] = -100
    grad = torch.rand(rows, generator=gen) + 0.5
    return [x.clone() for _ in range(n)], w, target.cuda(), grad.cuda()


def run_xent(n, rows, hidden, vocab, dt, piece=0, seed=0, inputs=None):
    _say("xent", n, rows, hidden, vocab, dt, piece)
    x, w, target, grad = inputs or xent_inputs(n, rows, hidden, vocab, dt, seed)
    _poison()
    loss, lse = ar.linear_cross_entropy(x, w, target)
    torch.cuda.synchronize()
    t = target.cpu().numpy()
    want_loss, want_lse = layer.cross_entropy(f64(x[0]), np.concatenate([f64(v) for v in w]), t)
    for r in range(n):
        check(lse[r], want_lse, f"lse rank {r}")
        check(loss[r], want_loss, f"loss rank {r}")
    _poison()
    dx, dw = ar.linear_cross_entropy_backward(grad, x, w, target, lse, piece=piece)
    torch.cuda.synchronize()
    first = 0
    for r in range(n):
        want_dx, want_dw = layer.cross_entropy_backward(f64(grad), f64(x[0]), f64(w[r]), t, f64(lse[r]), dt, first, vocab)
        check(dx[r], want_dx, f"dx rank {r}")
        check(dw[r], want_dw, f"dw rank {r}")
        first += w[r].shape[0]


XENT_SHAPES = [
    # ranks, rows, hidden, vocab
    (1, 1, 8, 2), (1, 1, 64, 1), (2, 3, 7, 33), (3, 17, 65, 1000), (8, 5, 64, 3), (1, 64, 200, 511), (2, 129, 136, 513),
    (4, 130, 40, 2050), (8, 260, 72, 4099), (1, 300, 33, 129), (8, 1, 200, 16), (3, 1, 40, 17), (1, 22, 144, 29),
    (3, 1047, 88, 9342), (3, 84, 120, 699), (2, 44, 72, 300),
]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,vocab", XENT_SHAPES)
def test_xent_shapes(n, rows, hidden, vocab, dt):
    run_xent(n, rows, hidden, vocab, dt, seed=rows + vocab)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,vocab", [(1, 1500), (2, 1999), (3, 770)])
def test_xent_in_pieces(n, vocab, dt):
    # several pieces, the last one short; ranks with fewer pieces than others
    run_xent(n, 70, 96, vocab, dt, piece=256, seed=vocab)


# ranks, rows, hidden, vocab: few results of dx, summed over many columns
XENT_SHARED_SHAPES = [(1, 20, 72, 9000), (2, 7, 100, 20011), (1, 40, 136, 30000), (2, 150, 72, 24000)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("piece", [0, 7000])
@pytest.mark.parametrize("n,rows,hidden,vocab", XENT_SHARED_SHAPES)
def test_xent_shared_sums(n, rows, hidden, vocab, piece, dt):
    run_xent(n, rows, hidden, vocab, dt, piece=piece, seed=vocab)


XENT_SHARED_CLASSES = [(1, 394, 767, 11339), (2, 300, 8, 26308), (2, 2, 1100, 15083), (1, 764, 39, 3456)]


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,vocab", XENT_SHARED_CLASSES)
def test_xent_shared_sums_of_every_class(n, rows, hidden, vocab, dt):
    run_xent(n, rows, hidden, vocab, dt, seed=vocab)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_xent_logits_are_the_same_bits_in_every_piece(dt):
    # with one row that counts, dw is that row's d times x whatever the order of
    # the sum over the rows: its bits are those of the recomputed logits
    rows, hidden, vocab = 40, 136, 30000
    x, w, target, grad = xent_inputs(1, rows, hidden, vocab, dt, 4, ignored=0.0)
    grad *= (torch.arange(rows) == 23).cuda()
    _, lse = ar.linear_cross_entropy(x, w, target)
    _, whole = ar.linear_cross_entropy_backward(grad, x, w, target, lse)
    for piece in (64, 1000, 9999):
        _, dw = ar.linear_cross_entropy_backward(grad, x, w, target, lse, piece=piece)
        assert torch.equal(dw[0], whole[0]), piece


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_xent_large_tiles(dt):
    run_xent(2, 1030, 72, 20011 if dt == "bf16" else 16400, dt, seed=9)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_xent_rows_without_loss_and_far_targets(dt):
    n, rows, hidden, vocab = 2, 20, 64, 300
    x, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 3, ignored=0.0)
    target[:] = torch.tensor([-1, -100, vocab, vocab + 5, 2 ** 40, -2 ** 62] + [0, vocab - 1, 149, 150] + [-1] * 10)
    grad[:6] = float("nan")  # not looked at in rows without loss
    run_xent(n, rows, hidden, vocab, dt, inputs=(x, w, target, torch.where(torch.isnan(grad), grad, grad)))
    # every row without loss
    target[:] = -1
    loss, lse = ar.linear_cross_entropy(x, w, target)
    dx, dw = ar.linear_cross_entropy_backward(grad, x, w, target, lse)
    for r in range(n):
        assert not loss[r].any() and not dx[r].any() and not dw[r].any()
        assert torch.isfinite(lse[r]).all()

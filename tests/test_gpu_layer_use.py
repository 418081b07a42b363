"""GPU: the layer operators as programs use them -- a layer's chain through the
collectives, captured graphs, side streams, two calls at once, caller's
buffers, empty inputs, non-finite values, tensors past 4 GiB -- and gradients
against differences of the loss."""

import sys

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import layer
from tests.test_gpu_layer import TORCH, check, f64, ffn_inputs, xent_inputs

pytestmark = pytest.mark.gpu


def _say(*what):
    print("CASE", *what, flush=True, file=sys.stderr)


def _rms64(h, weight, eps):
    return h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * weight


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows", [(1, 3), (4, 37), (8, 200)])
def test_layer_chain_through_the_collectives(n, rows, dt):
    """norm -> feed-forward -> all-reduce + norm -> loss, and back: dx of both
    operators summed by the all-reduce.  Each step is compared with fp64 on the
    values that reached it, so the bounds are those of one operator."""
    hidden, inter, vocab = 128, 96, 1000
    _say("chain", n, rows, dt)
    x, wg, wu, wd, _ = ffn_inputs(n, rows, hidden, inter, dt, rows)
    x = [x[0].clone() for _ in range(n)]
    comm = ar.Comm(n, rows * hidden * 4, 0)
    gate = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
    up = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
    part = ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up)
    res = [t.clone() for t in x]
    h = [torch.empty_like(t) for t in x]
    comm.allreduce_rmsnorm(part, h, torch.ones(hidden, dtype=TORCH[dt], device="cuda"), eps=1e-5, residual=res)
    total = sum(f64(p) for p in part) if dt == "f32" else f64(sum(p.float() for p in part).bfloat16())
    want = _rms64(total + f64(x[0]), np.ones(hidden), 1e-5)
    step = 2.0 ** -8 if dt == "bf16" else 1e-5
    for r in range(n):
        assert np.abs(f64(h[r]) - want).max() <= 2 * step * (1 + np.abs(want).max())
    _, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 5)
    loss, lse = ar.linear_cross_entropy(h, w, target)
    wl, _ = layer.cross_entropy(f64(h[0]), np.concatenate([f64(v) for v in w]), target.cpu().numpy())
    for r in range(n):
        check(loss[r], wl, f"loss rank {r}")
    dh, dw = ar.linear_cross_entropy_backward(grad, h, w, target, lse)
    comm.allreduce(dh, algo="oneshot")  # in place: every rank holds the whole gradient
    firsts = np.cumsum([0] + [v.shape[0] for v in w])
    parts = [layer.cross_entropy_backward(f64(grad), f64(h[0]), f64(w[r]), target.cpu().numpy(), f64(lse[r]), dt,
                                          int(firsts[r]), vocab)[0] for r in range(n)]
    value, bound = sum(p[0] for p in parts), sum(p[1] for p in parts)
    mag = sum(np.abs(p[0]) for p in parts)
    for r in range(n):  # n terms added in fp32, rounded once more
        check(dh[r], (value, bound + layer.step(dt) * (np.abs(value) + bound) + n * layer.E * mag), f"dh rank {r}")
    dx, dwg, dwu, dwd = ar.gated_ffn_backward(dh, x, wg, wu, wd, gate, up)
    comm.allreduce(dx, algo="oneshot")
    want = [layer.gated_ffn_backward(f64(dh[r]), f64(x[r]), f64(wg[r]), f64(wu[r]), f64(wd[r]), f64(gate[r]), f64(up[r]),
                                     "silu", dt) for r in range(n)]
    value, bound = sum(v["dx"][0] for v in want), sum(v["dx"][1] for v in want)
    mag = sum(np.abs(v["dx"][0]) for v in want)
    for r in range(n):
        check(dx[r], (value, bound + layer.step(dt) * (np.abs(value) + bound) + n * layer.E * mag), f"dx rank {r}")
        check(dwd[r], want[r]["dw_down"], f"dw_down rank {r}")
    assert comm.check()[0] == "AR_OK"
    comm.close()


def test_gradients_against_differences():
    """d(loss)/d(one weight) from two forward passes in fp32, the whole layer."""
    n, rows, hidden, inter, vocab = 2, 9, 32, 24, 50
    x, wg, wu, wd, _ = ffn_inputs(n, rows, hidden, inter, "f32", 3)
    x = [x[0].clone() for _ in range(n)]
    gen = torch.Generator().manual_seed(4)
    w = [(torch.randn(v, hidden, generator=gen) * hidden ** -0.5).cuda() for v in ar.vocab_shards(vocab, n)]
    target = torch.randint(0, vocab, (rows,), generator=gen).cuda()
    comm = ar.Comm(n, rows * hidden * 4, 0)

    def forward():
        gate = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
        up = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
        y = ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up, act="gelu")
        comm.allreduce(y, algo="oneshot")
        loss, lse = ar.linear_cross_entropy(y, w, target)
        return gate, up, y, loss, lse

    gate, up, y, loss, lse = forward()
    dy, dw = ar.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), y, w, target, lse)
    comm.allreduce(dy, algo="oneshot")
    dx, dwg, dwu, dwd = ar.gated_ffn_backward(dy, x, wg, wu, wd, gate, up, act="gelu")
    step = 2.0 ** -6
    for t, g in ((wg[0], dwg[0]), (wu[1], dwu[1]), (wd[0], dwd[0]), (w[1], dw[1])):
        at = int(g.abs().argmax())
        old = t.view(-1)[at].item()
        sums = []
        for sign in (1, -1):
            t.view(-1)[at] = old + sign * step
            sums.append(forward()[3][0].double().sum().item())
        t.view(-1)[at] = old
        num, got = (sums[0] - sums[1]) / (2 * step), g.view(-1)[at].item()
        # the sums are off by under 2e-5 (rows x 2e-6 each), the difference by
        # 2e-5 / step = 1.3e-3; the third derivative adds step^2 / 6 of order one
        assert abs(num - got) <= 2.5e-3 + 1e-3 * abs(got), (num, got)
    comm.close()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_graph_replays_match_eager_calls(dt):
    n, rows, hidden, inter, vocab = 3, 70, 100, 52, 700
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, dt, 11)
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 12)

    def program():
        gate = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
        up = [torch.empty(rows, inter, device="cuda") for _ in range(n)]
        out = ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up)
        grads = ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)
        loss, lse = ar.linear_cross_entropy(xs, w, target)
        more = ar.linear_cross_entropy_backward(grad, xs, w, target, lse, piece=256)
        return [*out, *loss, *(t for g in grads for t in g), *(t for g in more for t in g)]

    program()  # warm-up
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = program()
    second = torch.cuda.CUDAGraph()
    with torch.cuda.graph(second):  # a graph of its own workspaces
        captured2 = program()
    for it in range(4):
        for t in x + dout + xs:
            t.copy_(torch.randn(t.shape, device="cuda").to(t.dtype))
        for t in xs[1:]:
            t.copy_(xs[0])
        torch.cuda.synchronize()
        graph.replay()
        second.replay()
        eager = program()  # beside the replays, on the same stream
        torch.cuda.synchronize()
        for a, b, c in zip(captured, captured2, eager):
            assert torch.equal(a, c) and torch.equal(b, c), it


def test_two_graphs_replayed_at_once_on_two_streams():
    dt, n, rows, hidden, vocab = "bf16", 2, 130, 256, 5000
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 21)
    loss, lse = ar.linear_cross_entropy(xs, w, target)
    want = ar.linear_cross_entropy_backward(grad, xs, w, target, lse)
    streams = [torch.cuda.Stream() for _ in range(2)]
    graphs, outs = [], []
    torch.cuda.synchronize()
    for s in streams:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            a = ar.linear_cross_entropy(xs, w, target)
            b = ar.linear_cross_entropy_backward(grad, xs, w, target, a[1])
        graphs.append(g)
        outs.append((a, b))
    for _ in range(3):
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for a, b in outs:
            for r in range(n):
                assert torch.equal(a[0][r], loss[r]) and torch.equal(b[0][r], want[0][r]) and torch.equal(b[1][r], want[1][r])


def test_calls_on_a_stream_argument_and_on_the_current_stream():
    n, rows, hidden, inter = 2, 33, 96, 40
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, "bf16", 31)
    want = ar.gated_ffn(x, wg, wu, wd)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    a = ar.gated_ffn(x, wg, wu, wd, stream=side)  # its workspace comes from the side stream's pool
    with torch.cuda.stream(side):
        b = ar.gated_ffn(x, wg, wu, wd)
    torch.cuda.synchronize()
    for r in range(n):
        assert torch.equal(a[r], want[r]) and torch.equal(b[r], want[r])


@pytest.mark.parametrize("rows,hidden,inter", [(5, 24, 9), (70, 33, 17), (140, 130, 70), (513, 520, 264)])
def test_given_outputs_are_written_and_nothing_else(rows, hidden, inter):
    n, dt, guard = 2, "bf16", 512  # bytes around every output
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, dt, 41)
    xs, w, target, grad = xent_inputs(n, rows, hidden, 3 * inter + 1, dt, 42)
    arenas = []

    def out(shape, dtype):
        nb = int(np.prod(shape)) * torch.empty(0, dtype=dtype).element_size()
        a = torch.full((2 * guard + (nb + 15) // 16 * 16,), 0x5C, dtype=torch.uint8, device="cuda")
        arenas.append((a, nb))
        return a[guard:guard + nb].view(dtype).view(shape)

    many = lambda shape, dtype=torch.bfloat16: [out(shape, dtype) for _ in range(n)]  # noqa: E731
    f32 = torch.float32
    gate, up = many((rows, inter), f32), many((rows, inter), f32)
    y = ar.gated_ffn(x, wg, wu, wd, out=many((rows, hidden)), gate=gate, up=up)
    grads = ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up, dx=many((rows, hidden)), dw_gate=many((inter, hidden)),
                                  dw_up=many((inter, hidden)), dw_down=many((hidden, inter)))
    loss, lse = ar.linear_cross_entropy(xs, w, target, loss=many((rows,), f32), lse=many((rows,), f32))
    more = ar.linear_cross_entropy_backward(grad, xs, w, target, lse, dx=many((rows, hidden)),
                                            dw=[out(v.shape, v.dtype) for v in w])
    torch.cuda.synchronize()
    for a, nb in arenas:
        host = a.cpu().numpy()
        assert (host[:guard] == 0x5C).all() and (host[guard + nb:] == 0x5C).all()
    for got, want in ((y, ar.gated_ffn(x, wg, wu, wd)), (grads[0], ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)[0]),
                      (more[1], ar.linear_cross_entropy_backward(grad, xs, w, target, lse)[1])):
        for a, b in zip(got, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_rows_and_ranks_without_vocabulary(dt):
    n, hidden, inter = 3, 40, 20
    x, wg, wu, wd, dout = ffn_inputs(n, 0, hidden, inter, dt, 51)
    gate = [torch.empty(0, inter, device="cuda") for _ in range(n)]
    assert [tuple(t.shape) for t in ar.gated_ffn(x, wg, wu, wd, gate=gate, up=gate)] == [(0, hidden)] * n
    torch.full((1 << 20,), float("nan"), device="cuda")
    for g in ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, gate)[1:]:
        assert all(not t.any() for t in g)
    w = [torch.randn(v, hidden, device="cuda").to(TORCH[dt]) for v in ar.vocab_shards(2, n)]
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    loss, lse = ar.linear_cross_entropy(x, w, none)
    assert loss[0].numel() == 0
    dx, dw = ar.linear_cross_entropy_backward(torch.empty(0, device="cuda"), x, w, none, lse)
    assert [t.shape[0] for t in dw] == [1, 1, 0] and all(not t.any() for t in dw)


def test_non_finite_values_stay_in_their_rows():
    n, rows, hidden, inter, vocab = 2, 150, 64, 48, 400  # rows share tiles
    x, wg, wu, wd, dout = ffn_inputs(n, rows, hidden, inter, "bf16", 61)
    clean = ar.gated_ffn(x, wg, wu, wd)
    x[0][7, 3] = float("nan")
    x[0][9, 5] = float("inf")
    x[1][149, 0] = float("-inf")
    out = ar.gated_ffn(x, wg, wu, wd)
    for r, bad in ((0, (7, 9)), (1, (149,))):
        ok = torch.ones(rows, dtype=torch.bool, device="cuda")
        ok[list(bad)] = False
        assert torch.equal(out[r][ok], clean[r][ok])
        assert not torch.isfinite(out[r][~ok]).all(1).any()
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, "bf16", 62, ignored=0.0)
    loss, lse = ar.linear_cross_entropy(xs, w, target)
    dx, _ = ar.linear_cross_entropy_backward(grad, xs, w, target, lse)
    for t in xs:
        t[4, 4] = float("nan")
    target[11] = -1
    for t in xs:
        t[11, 1] = float("inf")  # a row without loss
    grad[20] = float("inf")
    l2, z2 = ar.linear_cross_entropy(xs, w, target)
    dx2, _ = ar.linear_cross_entropy_backward(grad, xs, w, target, z2)
    ok = torch.ones(rows, dtype=torch.bool, device="cuda")
    ok[[4, 11, 20]] = False
    for r in range(n):
        assert torch.equal(l2[r][ok], loss[r][ok]) and torch.isnan(l2[r][4]) and l2[r][11] == 0 and l2[r][20] == loss[r][20]
        # the other rows' gradients do not move (their scale is another row's
        # finite one now or the same: within one rounding of d and the result)
        tol = 2 * 2.0 ** -8 * dx[r][ok].float().abs().max()
        assert (dx2[r][ok].float() - dx[r][ok].float()).abs().max() <= tol
        assert torch.isnan(dx2[r][4]).all() and not dx2[r][11].any()


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,vocab", [(2, 5, 64, 300), (3, 150, 63, 400), (1, 300, 128, 2000), (2, 20, 72, 9001)])
def test_rows_without_loss_may_hold_anything(n, rows, hidden, vocab, dt):
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 63, ignored=0.0)
    target[1::3] = torch.tensor([-100, vocab, -1, 2 ** 40], device="cuda").repeat(rows)[: len(target[1::3])]
    dead = (target < 0) | (target >= vocab)
    loss, lse = ar.linear_cross_entropy(xs, w, target)
    want = ar.linear_cross_entropy_backward(grad, xs, w, target, lse)
    before = [t.clone() for t in xs]
    for i, t in enumerate(xs):
        t[dead] = (float("nan"), float("inf"), float("-inf"))[i % 3]
    grad[dead] = float("nan")
    l2, z2 = ar.linear_cross_entropy(xs, w, target)
    got = ar.linear_cross_entropy_backward(grad, xs, w, target, z2)
    for r in range(n):
        assert torch.equal(l2[r], loss[r]) and not l2[r][dead].any()
        assert torch.equal(got[0][r], want[0][r]) and not got[0][r][dead].any()
        assert torch.equal(got[1][r], want[1][r])
        assert torch.equal(xs[r][~dead], before[r][~dead])


def test_vectors_at_any_element():
    # the next token's targets are ids[1:]
    n, rows, hidden, vocab = 2, 70, 64, 500
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, "bf16", 64)
    loss, lse = ar.linear_cross_entropy(xs, w, target)
    want = ar.linear_cross_entropy_backward(grad, xs, w, target, lse)

    def at_one(t):
        return torch.cat([t[:1], t])[1:]

    l2, z2 = ([torch.full((rows + 2,), 7.0, device="cuda") for _ in range(n)] for _ in range(2))
    ar.linear_cross_entropy(xs, w, at_one(target), loss=[t[1:-1] for t in l2], lse=[t[1:-1] for t in z2])
    got = ar.linear_cross_entropy_backward(at_one(grad), xs, w, at_one(target), [t[1:-1] for t in z2])
    for r in range(n):
        assert torch.equal(l2[r][1:-1], loss[r]) and torch.equal(z2[r][1:-1], lse[r])
        assert all(t[0] == 7 and t[-1] == 7 for t in (l2[r], z2[r]))
        assert torch.equal(got[0][r], want[0][r]) and torch.equal(got[1][r], want[1][r])


@pytest.mark.parametrize("scale", [2.0 ** -20, 1.0, 2.0 ** 20])
def test_gradients_scale_with_grad_loss(scale):
    # powers of two move every value alike: the results are the same bits moved
    n, rows, hidden, vocab = 2, 100, 64, 300
    xs, w, target, grad = xent_inputs(n, rows, hidden, vocab, "bf16", 71)
    _, lse = ar.linear_cross_entropy(xs, w, target)
    one = ar.linear_cross_entropy_backward(grad, xs, w, target, lse)
    got = ar.linear_cross_entropy_backward(grad * scale, xs, w, target, lse)
    for a, b in zip(one, got):
        for s, t in zip(a, b):
            assert torch.equal(s.double() * scale, t.double())


def test_vocabulary_past_four_gib():
    rows, hidden = 3, 1024
    vocab = (1 << 22) + (1 << 18) + 5  # w: 9.1 GB, dw the same
    _say("far", vocab)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(rows, hidden, generator=gen, device="cuda").bfloat16()
    w = torch.empty(vocab, hidden, dtype=torch.bfloat16, device="cuda")
    for i in range(0, vocab, 1 << 20):
        part = w[i:i + (1 << 20)]
        part.copy_(torch.randn(part.shape, generator=gen, device="cuda") * 0.03)
    target = torch.tensor([vocab - 1, 5, (1 << 22) + 7], device="cuda")
    loss, lse = ar.linear_cross_entropy([x], [w], target)
    dx, dw = ar.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), [x], [w], target, lse)
    logits = torch.cat([x.double() @ w[i:i + (1 << 20)].double().T for i in range(0, vocab, 1 << 20)], 1)
    want = torch.logsumexp(logits, 1)
    # the logits are off by at most hidden e sum|x w| < 1024 * 6e-8 * 25, as is
    # lse; the sum joins about 2^17 partials in a few hundred roundings
    tol = 1024 * 2.0 ** -24 * (x.double().abs() @ w[:4096].double().abs().T).max().item() * 1.5 + 1e-4
    assert (lse[0].double() - want).abs().max() <= tol
    assert (loss[0].double() - (want - logits[torch.arange(rows), target])).abs().max() <= 2 * tol
    d = torch.exp(logits - lse[0].double()[:, None])
    d[torch.arange(rows), target] -= 1.0
    for rows_of in (slice(0, 64), slice(vocab - 64, vocab), slice((1 << 22) - 8, (1 << 22) + 24)):
        ref = d[:, rows_of].T @ x.double()
        err = (dw[0][rows_of].double() - ref).abs()
        assert (err <= 2.0 ** -8 * ref.abs() * 1.01 + (tol + 2.0 ** -8) * 2.0 ** -8 * (d[:, rows_of].abs().T @ x.double().abs())
                + tol * (d[:, rows_of].abs().T @ x.double().abs())).all()
    ref = sum(d[:, i:i + (1 << 20)] @ w[i:i + (1 << 20)].double() for i in range(0, vocab, 1 << 20))
    assert (dx[0].double() - ref).norm() <= 4e-3 * ref.norm()

"""Layer operators on the host (no GPU): the fp64 oracle against torch's own
operators and against differences, the binding's and the C ABI's refusals, and
the workspace sizes."""

import ctypes

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from all_reduce_reduction_rank_amd import binding
from oracle import layer

F64 = torch.float64
ACTS = {"silu": torch.nn.functional.silu, "gelu": torch.nn.functional.gelu,
        "gelu_tanh": lambda z: torch.nn.functional.gelu(z, approximate="tanh")}


def _t(gen, *shape):
    return torch.randn(*shape, generator=gen, dtype=F64, requires_grad=True)


# ---- the oracle ----


@pytest.mark.parametrize("act", list(ACTS))
def test_oracle_ffn_matches_autograd(act):
    gen = torch.Generator().manual_seed(1)
    x, wg, wu, wd = _t(gen, 5, 7), _t(gen, 4, 7), _t(gen, 4, 7), _t(gen, 7, 4)
    dout = torch.randn(5, 7, generator=gen, dtype=F64)
    g, u = x @ wg.T, x @ wu.T
    out = (ACTS[act](g) * u) @ wd.T
    out.backward(dout)
    n = lambda t: t.detach().numpy()  # noqa: E731
    fwd = layer.gated_ffn(n(x), n(wg), n(wu), n(wd), act, "f32")
    bwd = layer.gated_ffn_backward(n(dout), n(x), n(wg), n(wu), n(wd), n(g), n(u), act, "f32")
    for got, want in ((fwd["out"], out), (fwd["gate"], g), (fwd["up"], u), (bwd["dx"], x.grad), (bwd["dw_gate"], wg.grad),
                      (bwd["dw_up"], wu.grad), (bwd["dw_down"], wd.grad)):
        np.testing.assert_allclose(got[0], n(want), rtol=1e-11, atol=1e-12)


def test_oracle_cross_entropy_matches_autograd():
    gen = torch.Generator().manual_seed(2)
    x, w = _t(gen, 6, 5), _t(gen, 9, 5)
    target = torch.tensor([0, 8, -100, 3, 9, 4])  # -100 and 9: without loss
    grad = torch.rand(6, generator=gen, dtype=F64) + 0.1
    logits = x @ w.T
    live = (target >= 0) & (target < 9)
    loss = torch.nn.functional.cross_entropy(logits, torch.where(live, target, -100), reduction="none", ignore_index=-100)
    (loss * grad).sum().backward()
    n = lambda t: t.detach().numpy()  # noqa: E731
    got_loss, got_lse = layer.cross_entropy(n(x), n(w), n(target))
    np.testing.assert_allclose(got_loss[0], n(loss), rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(got_lse[0], n(torch.logsumexp(logits, 1)), rtol=1e-12)
    dx = np.zeros((6, 5))
    for first, last in ((0, 5), (5, 9)):  # two shards
        part_dx, part_dw = layer.cross_entropy_backward(n(grad), n(x), n(w)[first:last], n(target), got_lse[0], "f32",
                                                        first, 9)
        dx += part_dx[0]
        np.testing.assert_allclose(part_dw[0], n(w.grad)[first:last], rtol=1e-11, atol=1e-13)
    np.testing.assert_allclose(dx, n(x.grad), rtol=1e-11, atol=1e-13)


@pytest.mark.parametrize("act", list(ACTS))
def test_oracle_activation_derivative_against_differences(act):
    z = np.linspace(-8, 8, 321)
    h = 1e-5
    _, d = layer.act(z, act)
    num = (layer.act(z + h, act)[0] - layer.act(z - h, act)[0]) / (2 * h)
    np.testing.assert_allclose(d, num, rtol=0, atol=1e-9)  # h^2 f''' / 6 < 1e-10, and 1e-16 / h of rounding


# ---- the binding ----


def _ffn(n=2, rows=3, hidden=8, inter=4, dtype=torch.float32):
    z = lambda *s: [torch.zeros(*s, dtype=dtype) for _ in range(n)]  # noqa: E731
    return z(rows, hidden), z(inter, hidden), z(inter, hidden), z(hidden, inter)


def test_ffn_refuses_shapes_and_types():
    x, wg, wu, wd = _ffn()
    with pytest.raises(ValueError, match="w_up\\[1\\] has shape \\(5, 8\\)"):
        ar.gated_ffn(x, wg, [wu[0], torch.zeros(5, 8)], wd)
    with pytest.raises(ValueError, match="w_down\\[0\\] has shape \\(4, 8\\)"):
        ar.gated_ffn(x, wg, wu, wg)
    with pytest.raises(ValueError, match="x\\[1\\] has shape"):
        ar.gated_ffn([x[0], torch.zeros(4, 8)], wg, wu, wd)
    with pytest.raises(TypeError, match="w_gate\\[0\\] is torch.bfloat16"):
        ar.gated_ffn(x, [t.bfloat16() for t in wg], wu, wd)
    with pytest.raises(ValueError, match="w_up holds 1 rank buffers"):
        ar.gated_ffn(x, wg, wu[:1], wd)
    with pytest.raises(ValueError, match="1 to 8 ranks"):
        ar.gated_ffn([], [], [], [])
    with pytest.raises(ValueError, match="1 to 8 ranks"):
        ar.gated_ffn(*_ffn(n=9))
    with pytest.raises(ValueError, match="act must be one of"):
        ar.gated_ffn(x, wg, wu, wd, act="relu")
    with pytest.raises(ValueError, match="together"):
        ar.gated_ffn(x, wg, wu, wd, gate=[torch.zeros(3, 4)] * 2)
    with pytest.raises(TypeError, match="gate\\[0\\] is torch.bfloat16; the call needs torch.float32"):
        ar.gated_ffn(*_ffn(dtype=torch.bfloat16), gate=[torch.zeros(3, 4, dtype=torch.bfloat16)] * 2,
                     up=[torch.zeros(3, 4)] * 2)
    with pytest.raises(TypeError, match="unsupported tensor dtype"):
        ar.gated_ffn(*_ffn(dtype=torch.float16))
    with pytest.raises(ValueError, match="contiguous"):
        ar.gated_ffn([torch.zeros(8, 3).T] * 2, wg, wu, wd)
    with pytest.raises(ValueError, match="device tensors"):  # every check passed but the device's
        ar.gated_ffn(x, wg, wu, wd)


def test_ffn_backward_refuses_shapes():
    x, wg, wu, wd = _ffn()
    g = [torch.zeros(3, 4)] * 2
    with pytest.raises(ValueError, match="dout\\[0\\] has shape"):
        ar.gated_ffn_backward(wg, x, wg, wu, wd, g, g)
    with pytest.raises(ValueError, match="up\\[0\\] has shape"):
        ar.gated_ffn_backward(x, x, wg, wu, wd, g, x)
    with pytest.raises(ValueError, match="dw_down\\[0\\] has shape"):
        ar.gated_ffn_backward(x, x, wg, wu, wd, g, g, dw_down=wg)
    with pytest.raises(ValueError, match="device tensors"):
        ar.gated_ffn_backward(x, x, wg, wu, wd, g, g)


def test_cross_entropy_refuses_shapes_and_types():
    x = [torch.zeros(3, 8)] * 2
    w = [torch.zeros(5, 8), torch.zeros(4, 8)]
    t = torch.zeros(3, dtype=torch.int64)
    with pytest.raises(ValueError, match="w\\[0\\] has shape \\(4, 8\\); the call needs \\(5, 8\\)"):
        ar.linear_cross_entropy(x, w[::-1], t)  # shards in blocks of ceil(9 / 2)
    with pytest.raises(TypeError, match="target is torch.int32"):
        ar.linear_cross_entropy(x, w, t.int())
    with pytest.raises(ValueError, match="target must be a contiguous vector of 3"):
        ar.linear_cross_entropy(x, w, t[:2])
    with pytest.raises(TypeError, match="loss\\[0\\] is torch.float64"):
        ar.linear_cross_entropy(x, w, t, loss=[torch.zeros(3, dtype=torch.float64)] * 2)
    z = [torch.zeros(3)] * 2
    with pytest.raises(TypeError, match="grad_loss is"):
        ar.linear_cross_entropy_backward(torch.zeros(3, dtype=torch.bfloat16), x, w, t, z)
    with pytest.raises(ValueError, match="piece"):
        ar.linear_cross_entropy_backward(torch.zeros(3), x, w, t, z, piece=-1)
    with pytest.raises(ValueError, match="dw\\[1\\] has shape"):
        ar.linear_cross_entropy_backward(torch.zeros(3), x, w, t, z, dw=[w[0], w[0]])
    with pytest.raises(ValueError, match="device tensors"):
        ar.linear_cross_entropy(x, w, t)


def test_vocab_shards_are_the_blocks_rule():
    assert ar.vocab_shards(10, 4) == [3, 3, 3, 1]
    assert ar.vocab_shards(3, 8) == [1, 1, 1, 0, 0, 0, 0, 0]
    for v in (1, 7, 8, 1000, 10007):
        for n in range(1, 9):
            s = ar.vocab_shards(v, n)
            assert sum(s) == v and len(s) == n and s == sorted(s, reverse=True)


# ---- the C ABI (argument errors come before any HIP call) ----

P8 = ctypes.c_void_p * 8
LIB = binding.library()


def _ptrs(k):
    return P8(*[(k << 40) + (i << 36) for i in range(8)])


def _call_ffn(n=2, rows=4, hidden=16, inter=8, act=0, dtype=1, x=None, out=None, gate=None, up=None, ws=1 << 60,
              ws_bytes=1 << 40):
    return LIB.ar_gated_ffn(n, x or _ptrs(1), _ptrs(2), _ptrs(3), _ptrs(4), out or _ptrs(5), gate, up, rows, hidden, inter,
                            act, dtype, ctypes.c_void_p(ws), ws_bytes, None)


def test_c_abi_ffn_argument_errors():
    if torch.cuda.device_count() > 0:
        pytest.skip("needs a host without a GPU: the fake pointers below must never reach a kernel")
    assert _call_ffn() == 5                                        # every check passed: the first HIP call fails
    assert _call_ffn(rows=0) == 0
    assert _call_ffn(n=0) == 1 and _call_ffn(n=9) == 1 and _call_ffn(act=3) == 1 and _call_ffn(dtype=3) == 1
    assert _call_ffn(dtype=2) == 2                                 # integers
    assert _call_ffn(hidden=0) == 1 and _call_ffn(inter=0) == 1
    assert _call_ffn(hidden=(1 << 20) + 1) == 4 and _call_ffn(rows=(1 << 30) + 1) == 4
    assert _call_ffn(ws_bytes=LIB.ar_gated_ffn_workspace(2, 4, 16, 8, 1, 0) - 1) == 4
    assert _call_ffn(ws=0) == 1 and _call_ffn(ws=(1 << 60) + 8) == 1   # null, misaligned
    assert _call_ffn(x=P8(*[8 + (i << 36) for i in range(8)])) == 1
    assert _call_ffn(out=_ptrs(1)) == 1                            # an output over an input
    assert _call_ffn(gate=_ptrs(6)) == 1                           # gate without up
    assert _call_ffn(gate=_ptrs(6), up=_ptrs(6)) == 1              # outputs over each other
    assert _call_ffn(gate=_ptrs(6), up=_ptrs(7)) == 5
    same = P8(*[1 << 40] * 8)
    assert _call_ffn(x=same) == 5                                  # one input on several ranks


def test_c_abi_cross_entropy_argument_errors():
    if torch.cuda.device_count() > 0:
        pytest.skip("needs a host without a GPU: the fake pointers below must never reach a kernel")

    def fwd(n=3, rows=4, hidden=16, vocab=100, dtype=1, w=None, target=7 << 40, ws=1 << 60, ws_bytes=1 << 40):
        return LIB.ar_linear_cross_entropy(n, _ptrs(1), w or _ptrs(2), ctypes.c_void_p(target), _ptrs(3), _ptrs(4), rows,
                                           hidden, vocab, dtype, ctypes.c_void_p(ws), ws_bytes, None)

    assert fwd() == 5 and fwd(rows=0) == 0
    assert fwd(n=0) == 1 and fwd(vocab=0) == 1 and fwd(hidden=0) == 1 and fwd(dtype=2) == 2 and fwd(target=0) == 1
    assert fwd(vocab=(1 << 30) + 1) == 4
    assert fwd(ws_bytes=LIB.ar_linear_cross_entropy_workspace(3, 4, 16, 100, 1, 0, 0) - 1) == 4
    assert fwd(target=(7 << 40) + 8) == 5 and fwd(target=(7 << 40) + 4) == 1   # vectors: at their elements
    # ranks past the vocabulary need no buffer, ranks within it do
    assert fwd(n=8, vocab=2, w=P8(2 << 40, 9 << 40, *[0] * 6)) == 5
    assert fwd(n=8, vocab=3, w=P8(2 << 40, 9 << 40, *[0] * 6)) == 1

    def bwd(rows=4, piece=0, ws_bytes=1 << 40, dx=None):
        return LIB.ar_linear_cross_entropy_backward(3, ctypes.c_void_p(8 << 40), _ptrs(1), _ptrs(2),
                                                    ctypes.c_void_p(7 << 40), _ptrs(3), dx or _ptrs(4), _ptrs(5), rows, 16,
                                                    100, 1, piece, ctypes.c_void_p(1 << 60), ws_bytes, None)

    assert bwd() == 5 and bwd(dx=_ptrs(5)) == 1
    assert bwd(ws_bytes=LIB.ar_linear_cross_entropy_workspace(3, 4, 16, 100, 1, 1, 0) - 1) == 4


def test_workspace_sizes():
    ws = LIB.ar_gated_ffn_workspace
    assert ws(8, 0, 64, 64, 1, 0) == 0 and ws(9, 4, 64, 64, 1, 0) == 0 and ws(1, 4, 64, 64, 2, 0) == 0
    assert ws(1, 4096, 5120, 1728, 1, 0) == 4096 * 1728 * 2        # h, one term a value
    assert ws(1, 4096, 5120, 1728, 1, 1) == 3 * 4096 * 1728 * 2    # dg, du, h
    # an odd width: h's rows padded to 16 bytes, and copies of x and the weights
    odd = ws(1, 128, 33, 9, 1, 0)
    assert odd >= 128 * 16 * 2 + 128 * 40 * 2 + 2 * 9 * 40 * 2 + 33 * 16 * 2
    xe = LIB.ar_linear_cross_entropy_workspace
    # the pieces cap what backward needs: d of all ranks within 1 GiB, dx's fp32
    # sum and the copy of x
    whole = xe(1, 8192, 1024, 131072, 1, 1, 0)
    assert whole < (1 << 30) + 8192 * 1024 * (4 + 2) + 4096
    small = xe(1, 8192, 1024, 131072, 1, 1, 256)
    assert small < 8192 * (256 * 2 + 1024 * (4 + 2)) + 4096
    # every piece a caller may name fits the bytes named for it
    for piece in (0, 1, 255, 256, 300, 1000, 1 << 30):
        assert xe(2, 100, 64, 1001, 0, 1, piece) > 0

"""Results that the layer operators allocate: every rank's is a tensor of its
own, that keeps no other alive, is saved by itself and takes part in autograd
like any other."""

import io

import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from all_reduce_reduction_rank_amd import binding

DT = [torch.float32, torch.bfloat16]


def own_tensors(ts):
    for t in ts:
        nb = t.numel() * t.element_size()
        assert t.untyped_storage().nbytes() == nb and t.storage_offset() == 0 and not t._is_view()
        f = io.BytesIO()
        torch.save(t, f)
        assert len(f.getvalue()) < nb + 4096
    assert len({t.data_ptr() for t in ts if t.numel()}) == len([t for t in ts if t.numel()])
    before = [t._version for t in ts]
    ts[0].add_(torch.ones_like(ts[0], requires_grad=True))  # refused for one of several views
    assert [t._version for t in ts[1:]] == before[1:]


@pytest.mark.parametrize("dtype", DT)
@pytest.mark.parametrize("n,shape", [(1, (3, 8)), (2, (3, 8)), (8, (5, 7)), (3, (64,)), (4, (0, 8))])
def test_rank_results_are_tensors_of_their_own(n, shape, dtype):
    binding._torch()
    ts = binding._Scratch(None, "cpu").ranks(n, shape, dtype)
    assert len(ts) == n and all(t.shape == shape and t.dtype is dtype for t in ts)
    own_tensors(ts)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", DT)
def test_the_operators_results_are_tensors_of_their_own(dtype):
    n, rows, hidden, inter, vocab = 3, 40, 64, 32, 96

    def rand(*shape):
        return [torch.randn(*shape, device="cuda").to(dtype) for _ in range(n)]

    x, wg, wu, wd, dout = rand(rows, hidden), rand(inter, hidden), rand(inter, hidden), rand(hidden, inter), rand(rows, hidden)
    gate, up = ([torch.empty(rows, inter, device="cuda") for _ in range(n)] for _ in range(2))
    results = [ar.gated_ffn(x, wg, wu, wd, gate=gate, up=up), *ar.gated_ffn_backward(dout, x, wg, wu, wd, gate, up)]
    w = rand(vocab // n, hidden)
    target = torch.arange(rows, device="cuda")
    x = [x[0]] * n
    loss, lse = ar.linear_cross_entropy(x, w, target)
    results += [*ar.linear_cross_entropy_backward(torch.ones(rows, device="cuda"), x, w, target, lse), loss, lse]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    results.append(ar.gated_ffn(x, wg, wu, wd, stream=side))
    torch.cuda.synchronize()
    for ts in results:
        own_tensors(ts)

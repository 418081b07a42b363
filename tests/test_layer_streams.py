"""The layer operators refuse a stream of another device than their tensors'."""

import types

import pytest
import torch

from all_reduce_reduction_rank_amd import binding


@pytest.mark.parametrize("call", ["gated_ffn", "gated_ffn_backward", "linear_cross_entropy",
                                  "linear_cross_entropy_backward"])
def test_a_stream_of_another_device_is_refused(call, monkeypatch):
    # tensors that say they live on device 1, which is current, and a stream of
    # device 0: the call must end before it allocates or launches
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    monkeypatch.setattr(binding._Scratch, "empty", lambda *a: pytest.fail("the call went on"))
    on_1 = type("OnDevice1", (torch.Tensor,), {"get_device": lambda self: 1})

    def ranks(*shape, dtype=torch.float32):
        return [torch.zeros(*shape, dtype=dtype).as_subclass(on_1) for _ in range(2)]

    x, wide, tall = ranks(4, 16), ranks(8, 16), ranks(16, 8)
    kept, rows = ranks(4, 8), ranks(4)
    target = ranks(4, dtype=torch.int64)[0]
    args = {"gated_ffn": (x, wide, wide, tall), "gated_ffn_backward": (x, x, wide, wide, tall, kept, kept),
            "linear_cross_entropy": (x, wide, target),
            "linear_cross_entropy_backward": (rows[0], x, wide, target, rows)}[call]
    stream = types.SimpleNamespace(device_index=0, cuda_stream=0)
    with pytest.raises(ValueError, match="stream of the rank buffers' device"):
        getattr(binding, call)(*args, stream=stream)

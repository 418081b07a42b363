"""Weight gradients of the norms over many rows: the workgroups' shares are added
without further rounding."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [1, 2, 4])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_sums_of_equal_shares_are_exact(n, dim):
    """x of ones has the norm 1, so every term of dw is g itself.  32768 rows are cut
    evenly: a thread adds T equal terms one after the other (its partial sums 3 g,
    5 g .. are rounded, at most half a step each: T - 2 of them), waves and
    workgroups double equal sums, which is exact, and so is the fp64 sum of up to
    1024 equal shares: dw is off 32768 g, a number of fp32, by (T - 2) 2^-24 of it and
    the last rounding at most, and by nothing where T is 2."""
    rows = 1 << 15
    g = (1 + np.random.default_rng(dim).integers(0, 1 << 23, dim) * 2.0 ** -23).astype(np.float32)
    x = torch.ones(rows, 1, dim, device="cuda")
    dout = torch.from_numpy(g).cuda().expand(rows, 1, dim).contiguous()
    dw = ar.qk_norm_rope_backward([dout] * n, None, [x] * n, None, torch.ones(dim, device="cuda"), None, None, None, eps=0.0)[2]
    terms = 2 * n * (2 if dim == 256 else 1)  # 1024 / n workgroups, 16 rows at a time, 2048 / dim of them side by side
    want = g.astype(np.float64) * rows
    for t in dw:
        off = np.abs(t.double().cpu().numpy() - want) / want
        # (n 1 and heads below 256: T is 2.  A sum that was rounded ends rounded once more.)
        assert off.max() <= (terms - 2 + (terms > 2)) * 2.0 ** -24, off.max() * 2 ** 24

"""max_rows chooses the kernel and with it the bf16 terms of the softmax weights: 1
keeps two of them whatever is in the call."""

import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import heads
from test_gpu_heads import att_case, check, host, ints

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("h,kv,dim,page", [(5, 1, 128, 64), (4, 4, 64, 16), (2, 1, 256, 32)])
def test_two_terms_on_request(h, kv, dim, page, window):
    """A prompt, a chunk and single tokens in one call."""
    length, count = [150, 300, 900, 64], [150, 70, 1, 1]
    ref, cache, table, first, q = att_case(1, h, kv, dim, page, length, count, "bf16", wide=True)
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    args = (cache, ints(table), ints(first), ints(length))
    a, b = int(first[0]), int(first[-1])
    for most, terms in ((1, 2), (150, 1), (0, 1)):
        got = ar.cache_attention(q, *args, window=window, max_rows=most, lse=lse)
        (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, dim ** -0.5, True, window, "bf16", terms)
        check(host(got[0][a:b]), o[a:b], eo[a:b], f"out, max_rows {most}")
        check(host(lse[0][a:b]), z[a:b], ez[a:b], f"lse, max_rows {most}")

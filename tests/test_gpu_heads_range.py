"""Attention and cache at the ends of the number range."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import heads
from test_gpu_heads import att_case, check, host, ints, upload

pytestmark = pytest.mark.gpu

FP32_MAX = float(np.finfo(np.float32).max)


def huge_queries(dt, most, values):
    """One element of every row is huge, keys are below 0.22: no product and no sum
    of them leaves fp32."""
    length, count = [90, 700], [4, 60]
    ref, _, table, first, q = att_case(1, 2, 1, 128, 16, length, count, dt, wide=most > 1)
    ref[0].scale[0][:] = 116
    q = [q[0].clone()]
    for i in range(q[0].shape[0]):
        q[0][i, 0, (7 * i) % 128] = values[i % len(values)]
        q[0][i, 1, (5 * i) % 128] = values[(i + 1) % len(values)]
    return ref, upload(ref), table, first, q, length


@pytest.mark.parametrize("most", [1, 100])
def test_queries_beyond_the_largest_bf16(most):
    """fp32 numbers above 3.39e38 round to infinity in bf16, whose terms they enter the
    products in."""
    ref, cache, table, first, q, length = huge_queries("f32", most, [FP32_MAX, -3.3999e38, 3.3895e38, -FP32_MAX, 3.3896e38])
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), scale=1e-37, max_rows=most, lse=lse)
    (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, float(np.float32(1e-37)), True, 0, "f32", 3)
    a, b = int(first[0]), int(first[-1])
    check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")


@pytest.mark.parametrize("most", [1, 100])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("scale", [0.0, 1e-42, -1e-40, 5e-39, -1.5e-38])
def test_scales_down_to_nothing(scale, dt, most):
    """Products of 1e37 times scales below fp32's normal numbers: scores to 1e-6."""
    ref, cache, table, first, q, length = huge_queries(dt, most, [1e38, -3e38, 2.5e38])
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), scale=scale, max_rows=most, lse=lse)
    (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, float(np.float32(scale)), True, 0, dt,
                                       3 if dt == "f32" else 1)
    # scale times log2 e is rounded to a multiple of 2^-149 (and is not 0): off by 2^-149 of
    # products below 2^127, in units of log2; a score's error moves a weight by its own size twice
    extra = 2.0 ** -22 * np.log(2)
    a, b = int(first[0]), int(first[-1])
    size = 448.0 * 2.0 ** -5  # of any value
    check(host(got[0][a:b]), o[a:b], eo[a:b] + 2 * extra * size, "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b] + extra, "lse")

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


def every_code():
    """A cache that holds every code under every scale byte: page b is of byte b."""
    ref = heads.Cache(256, 1, 16, 64)
    for i in range(2):
        ref.codes[i][:, 0] = np.resize(np.arange(256), (16, 64))  # each code four times
        ref.scale[i][:, 0] = np.arange(256)
    values = heads.VALUES[ref.codes[0]] * 2.0 ** (np.clip(np.arange(256), 1, 254) - 127.0)[:, None, None, None]
    return ref, values.transpose(0, 2, 1, 3).reshape(-1, 1, 64)


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_every_code_and_scale_read_back(dt):
    """Exact, and the dtype's nearest where it has no such number (bf16 below 2^-133,
    infinity from 2^128 on)."""
    ref, values = every_code()
    rows = len(values)
    cache, t = upload([ref]), torch.bfloat16 if dt == "bf16" else torch.float32
    k, v = (torch.full((rows, 1, 64), 5.0, dtype=t, device="cuda") for _ in range(2))
    ar.cache_read(cache, ints(np.arange(256)[None]), ints([0, rows]), ints([0]), [k], [v])
    with np.errstate(over="ignore"):
        want = torch.from_numpy(values.astype(np.float32)).to(t)  # (all of them exact or infinite in fp32)
    assert np.array_equal(values.astype(np.float32).astype(np.float64)[np.abs(values) < 2.0 ** 128], values[np.abs(values) < 2.0 ** 128])
    for got in (k.cpu(), v.cpu()):
        assert torch.equal(got.isnan(), want.isnan())
        assert torch.equal(torch.nan_to_num(got, nan=3.0, posinf=torch.inf, neginf=-torch.inf),
                           torch.nan_to_num(want, nan=3.0, posinf=torch.inf, neginf=-torch.inf))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_written_at_the_ends_of_the_range(dt):
    """Tiny and huge values, a page of each, and pages that grow from one to the other."""
    rng = np.random.default_rng(2)
    ref = heads.Cache(12, 1, 16, 64)
    ref.scale[0][:], ref.scale[1][:] = 1, 254
    for i in range(2):
        ref.codes[i][:] = rng.integers(0, 127, ref.codes[i].shape)
    cache = upload([ref])
    table, first, start = np.arange(12)[:, None], np.arange(0, 37, 3), np.array([0, 5] * 6)
    top = 3.38953139e38 if dt == "bf16" else FP32_MAX
    for size in (2.0 ** -140, top, 2.0 ** -126, top / 2):
        x = [rng.uniform(-1, 1, (36, 1, 64)) * size for _ in range(2)]
        x[0][::3, 0, 5], x[1][1::3, 0, 9] = size, -size
        t = [torch.from_numpy(y).to(torch.float32).to(torch.bfloat16 if dt == "bf16" else torch.float32).cuda() for y in x]
        ref.write([host(y) for y in t], table, first, start)
        ar.cache_write(cache, [t[0]], [t[1]], ints(table), ints(first), ints(start))
        start = start + 1
        for i, (codes, scale) in enumerate(((cache.k[0], cache.k_scale[0]), (cache.v[0].transpose(2, 3), cache.v_scale[0]))):
            np.testing.assert_array_equal(scale.cpu().numpy(), ref.scale[i])
            np.testing.assert_array_equal(codes.cpu().numpy() & 127, ref.codes[i] & 127)  # (the sign of 0 as well as not)
            low = ref.codes[i] & 127
            assert ((codes.cpu().numpy() == ref.codes[i]) | (low == 0)).all()

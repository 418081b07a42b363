"""Values that are no finite numbers in the cache of the attention operators: they
reach the rows that see them and no other, and cost no more than other values."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import heads
from test_gpu_heads import att_case, check, host, ints, upload

pytestmark = pytest.mark.gpu


def seen_by(first, length, causal, window):
    """(row, sequence, tokens it sees: [from, to)) of every row."""
    for s, total in enumerate(length):
        n = int(first[s + 1] - first[s])
        for i in range(n):
            p = total - n + i
            yield int(first[s]) + i, s, (max(0, p + 1 - window) if window else 0) if causal else 0, max(0, p + 1) if causal else total


# the last ones of each: few rows, the kernel of many rows, shares among workgroups
@pytest.mark.parametrize("most,count,length", [(1, [5, 3], [100, 1100]), (200, [90, 100], [300, 1100]), (90, [60, 90], [60, 2000])])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dim,page", [(64, 16), (128, 64), (256, 32)])
def test_nan_values_everywhere(most, count, length, window, dt, dim, page):
    """Values of one token in eight are NaN in a dimension of their own or two, and
    so are pages that no row sees: every row against the oracle without them,
    and NaN exactly where a token of its own holds one."""
    ref, _, table, first, q = att_case(1, 4, 2, dim, page, length, count, dt, seed=3)
    c, rng = ref[0], np.random.default_rng(5)
    held = {}  # (sequence, key head) -> [(token, dimension)]
    for s, total in enumerate(length):
        for h in range(2):
            for t in rng.permutation(total)[:total // 8]:
                d = int(rng.integers(0, dim - 16))  # the last dimensions stay numbers
                c.codes[1][table[s, t // page], h, t % page, d] = 0x7f if t % 2 else 0xff
                held.setdefault((s, h), []).append((int(t), d))
    cache = upload(ref)
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), window=window, max_rows=most, lse=lse)
    c.codes[1][(c.codes[1] & 0x7f) == 0x7f] = 0
    few = (most or max(count)) * 2 <= 96
    (o, eo), (z, ez) = heads.attention(host(q[0]), c, table, first, length, dim ** -0.5, True, window, dt,
                                       3 if dt == "f32" else 2 if few else 1)
    clean = 0
    for row, s, a, b in seen_by(first, length, True, window):
        for h in range(2):
            bad = {d for t, d in held[s, h] if a <= t < b}
            clean += dim - len(bad)
            o[row, 2 * h:2 * h + 2, sorted(bad)] = np.nan
    assert clean
    a, b = int(first[0]), int(first[-1])
    check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")


@pytest.mark.parametrize("most", [1, 100])
@pytest.mark.parametrize("byte", [247, 250, 254])
def test_values_beyond_fp32_reach_only_who_sees_them(most, byte):
    """A page whose scale puts codes at 2^128 and above: rows before it are as
    without it, rows that see it hold no number there."""
    length, count, page, dim = [400], [60], 16, 64
    ref, _, table, first, q = att_case(1, 2, 1, dim, page, length, count, "f32", wide=most > 1)
    c, last = ref[0], table[0, 24]  # tokens 384 .. 399
    c.codes[1][last] = 0
    c.codes[1][last, 0, :, 5] = 0x7e   # the largest code
    c.codes[1][last, 0, :, 6] = 0xfe
    c.scale[1][last] = byte
    cache = upload(ref)
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), max_rows=most)
    c.codes[1][last] = 0
    (o, eo), _ = heads.attention(host(q[0]), c, table, first, length, dim ** -0.5, True, 0, "f32", 3)
    a = int(first[0])
    check(host(got[0][a:a + 44]), o[a:a + 44], eo[a:a + 44], "rows before the page")
    for i in range(44, 60):
        assert not torch.isfinite(got[0][a + i, :, 5:7]).any()
        o[a + i, :, 5:7] = 0
    after = host(got[0][a + 44:a + 60])
    after[:, :, 5:7] = 0
    check(after, o[a + 44:a + 60], eo[a + 44:a + 60], "rows that see the page")


def _time(call):
    """The best of five, of some calls each."""
    for _ in range(2):
        call()
    best = np.inf
    for _ in range(5):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        for _ in range(8):
            call()
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


@pytest.mark.parametrize("count,length,h,kv", [(1500, 1500, 8, 1), (1, 3000, 4, 1), (5, 3000, 8, 2)])
def test_a_nan_that_rows_see_costs_nothing(count, length, h, kv):
    """One NaN among the first values, that nearly every row sees, and one among the
    last: the time of a cache without any (half as much again for what timing adds)."""
    page = 64
    pages = -(-length // page)
    gen = torch.Generator(device="cuda").manual_seed(1)
    x = [torch.randn(length, kv, 128, generator=gen, device="cuda").bfloat16() for _ in range(2)]
    q = [torch.randn(count, h, 128, generator=gen, device="cuda").bfloat16()]
    table = torch.arange(pages, dtype=torch.int32, device="cuda")[None]
    times = []
    for bad in (False, True):
        if bad:
            x[1][5, 0, 7] = float("nan")
            x[1][length - 2, 0, 9] = float("inf")
        cache = ar.KVCache.empty(1, pages, kv, 128, page)
        ar.cache_write(cache, [x[0]], [x[1]], table, ints([0, length]), ints([0]))
        first, total = ints([0, count]), ints([length])
        out = ar.cache_attention(q, cache, table, first, total, max_rows=count)
        sees = max(0, 5 - (length - count))  # the first row at position 5 or behind
        assert out[0][sees:, 0, 7].isnan().all().item() == bad and out[0][:sees, 0, 7].isfinite().all()
        assert out[0][:, 0, 8].isfinite().all()
        times.append(_time(lambda: ar.cache_attention(q, cache, table, first, total, max_rows=count)))
    assert times[1] < 1.5 * times[0], times

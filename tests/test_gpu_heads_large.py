"""Calls of more work items than one axis of a launch holds (2^32 threads along x):
the largest that the documentation allows and the GPU's memory holds."""

import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from test_gpu_heads import ints

pytestmark = pytest.mark.gpu

GIB = 1 << 30


@pytest.fixture(autouse=True)
def own_memory():
    torch.cuda.empty_cache()
    yield
    torch.cuda.empty_cache()


def need(gib):
    if torch.cuda.mem_get_info()[0] < gib * GIB:
        pytest.skip(f"needs {gib} GiB of GPU memory")


def slices(rows, edge):
    """Rows at both ends and around `edge`."""
    for a in (0, edge - 700, edge, rows - 900):
        yield slice(a, a + 900)


def test_rope_rows():
    need(90)
    rows, dim = (1 << 28) + 37, 64  # 16 rows a workgroup: 2^24 + 3 of them
    q = torch.empty(rows, 1, dim, dtype=torch.bfloat16, device="cuda").normal_()
    pos = torch.arange(rows, device="cuda")
    w, freq = torch.rand(dim, device="cuda").bfloat16(), torch.rand(dim // 2, device="cuda")
    out, _ = ar.qk_norm_rope([q], None, w, None, pos, freq)
    for s in slices(rows, (1 << 28) - 16):
        want, _ = ar.qk_norm_rope([q[s]], None, w, None, pos[s].clone(), freq)
        assert torch.equal(out[0][s], want[0]), s


def test_cache_rows():
    need(160)
    page, dim = 16, 64
    rows = (1 << 28) + 37
    pages = -(-rows // page)
    width = (1 << 27) // page - 1   # of a sequence (at most 2^31 tokens; three of them here)
    seqs = -(-pages // width)
    first = [min(s * width * page, rows) for s in range(seqs)] + [rows]
    table = torch.arange(seqs * width, dtype=torch.int32, device="cuda").view(seqs, width)
    start = ints([0] * seqs)
    x = torch.empty(rows, 1, dim, dtype=torch.bfloat16, device="cuda").normal_()
    cache = ar.KVCache.empty(1, seqs * width, 1, dim, page)
    ar.cache_write(cache, [x], [x], table, ints(first), start)
    k, v = torch.empty_like(x), torch.empty_like(x)
    ar.cache_read(cache, table, ints(first), start, [k], [v])
    for s in slices(rows, ((1 << 24) - 1) * page):
        # half a step of e4m3, or of its smallest normal number: 2^-6 of the scale, which is below 2 / 448 of a page's largest value
        bound = 2.0 ** -4 * torch.clamp(x[s].abs().float(), min=x[s].abs().max().item() * 2.0 ** -13)
        assert ((k[s].float() - x[s].float()).abs() <= bound).all(), s
        assert torch.equal(k[s], v[s]), s
    assert torch.equal(k, v)  # keys and values lie differently in the cache


def test_attention_rows():
    """(16 rows a workgroup for so many rows only where max_rows says less than there are.)"""
    need(90)
    rows, heads, dim = (1 << 24) + 5, 16, 64
    cache = ar.KVCache.empty(1, 1, 1, dim, 64)
    kv = torch.randn(64, 1, dim, device="cuda").bfloat16()
    table, start = ints([[0]]), ints([0])
    ar.cache_write(cache, [kv], [kv], table, ints([0, 64]), start)
    q = torch.empty(rows, heads, dim, dtype=torch.bfloat16, device="cuda").normal_()
    out = ar.cache_attention([q], cache, table, ints([0, rows]), ints([64]), causal=False, max_rows=1)
    for s in slices(rows, (1 << 24) - 1):
        want = ar.cache_attention([q[s]], cache, table, ints([0, 900]), ints([64]), causal=False, max_rows=1)
        assert torch.equal(out[0][s], want[0]), s


def test_attention_sequences():
    """2^20 sequences of 2 key heads on 8 ranks, two of them with rows."""
    need(4)
    seqs, n, kv, dim, page, width = 1 << 20, 8, 2, 64, 64, 20
    gen = torch.Generator(device="cuda").manual_seed(3)
    cache = ar.KVCache.empty(n, 2 * width, kv, dim, page)
    two = torch.randperm(2 * width, generator=gen, device="cuda").int().view(2, width)
    k = [torch.randn(2400, kv, dim, generator=gen, device="cuda") for _ in range(n)]
    ar.cache_write(cache, k, k, two, ints([0, 1200, 2400]), ints([0, 0]))
    q = [torch.randn(200, kv, dim, generator=gen, device="cuda") for _ in range(n)]
    want = ar.cache_attention(q, cache, two, ints([0, 100, 200]), ints([1200, 1200]), max_rows=100)
    table = torch.full((seqs, width), -1, dtype=torch.int32, device="cuda")
    table[5], table[-1] = two[0], two[1]
    first = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    first[6:], first[-1] = 100, 200
    length = torch.zeros(seqs, dtype=torch.int32, device="cuda")
    length[5] = length[-1] = 1200
    got = ar.cache_attention(q, cache, table, first, length, max_rows=100)
    for a, b in zip(got, want):  # (fewer shares of the tokens: sums in another order)
        assert ((a - b).abs() <= 2.0 ** -24 * 1200 * b.abs().max()).all()

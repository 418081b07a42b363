"""Calls of very many sequences: every sequence finds its rows, in a time that grows
as the calls do."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from test_gpu_heads import ints

pytestmark = pytest.mark.gpu


def case(seqs, count, page=16, dim=64):
    """One page a sequence; sequence s has count[s] tokens of random values."""
    first = torch.zeros(seqs + 1, dtype=torch.int32, device="cuda")
    first[1:] = count.cumsum(0)
    gen = torch.Generator(device="cuda").manual_seed(seqs)
    x = torch.randn(int(first[-1]), 1, dim, generator=gen, device="cuda").bfloat16()
    table = torch.randperm(seqs, generator=gen, device="cuda").int()[:, None]
    return x, table, first, torch.zeros(seqs, dtype=torch.int32, device="cuda")


def plain_codes(x, table, first, pages, page=16):
    """Codes and scales of the same write by torch's own operators: a page for each
    sequence, tokens from 0 on."""
    owner = torch.repeat_interleave(torch.arange(len(first) - 1, device="cuda"), (first[1:] - first[:-1]).long())
    at = torch.arange(len(x), device="cuda") - first[owner].long()
    values = torch.zeros(pages, page, x.shape[-1], device="cuda")
    where = table[owner, 0].long()
    values[where, at] = x[:, 0].float()
    m = values.abs().amax((1, 2)).double()
    scale = torch.ceil(torch.log2(m / 448)).clamp(min=-126)  # (448 2^e itself does not occur)
    codes = (values.double() / torch.exp2(scale)[:, None, None]).float().to(torch.float8_e4m3fn).view(torch.uint8)
    held = torch.zeros(pages, page, dtype=torch.bool, device="cuda")
    held[where, at] = True
    return codes, scale.int() + 127, held


@pytest.mark.parametrize("seqs", [64, 65, 4096, 4097, 70000, 1 << 20])
@pytest.mark.parametrize("empty", [False, True])
def test_every_sequence_finds_its_rows(seqs, empty):
    rng = np.random.default_rng(seqs)
    count = torch.from_numpy(rng.integers(0, 3 if seqs > 1 << 18 else 5, seqs)).cuda()
    if empty:  # runs of sequences without rows, at both ends too
        count[torch.from_numpy(rng.random(-(-seqs // 40)) < 0.6).cuda().repeat_interleave(40)[:seqs]] = 0
        count[:7] = 0
        count[-9:] = 0
    x, table, first, start = case(seqs, count)
    cache = ar.KVCache.empty(1, seqs, 1, 64, 16)
    for t in (*cache.k, *cache.v, *cache.k_scale, *cache.v_scale):
        t.zero_()
    ar.cache_write(cache, [x], [x], table, first, start)
    codes, scale, held = plain_codes(x, table, first, seqs)
    assert torch.equal(cache.k[0][:, 0][held], codes[held]) and (cache.k[0][:, 0][~held] == 0).all()
    assert torch.equal(cache.v[0][:, 0].transpose(1, 2)[held], codes[held])
    there = held.any(1)
    assert torch.equal(cache.k_scale[0][there, 0].int(), scale[there]) and (cache.k_scale[0][~there] == 0).all()
    k, v = torch.empty_like(x), torch.empty_like(x)
    ar.cache_read(cache, table, first, start, [k], [v])
    assert torch.equal(k, v) and ((k - x).abs() <= 2.0 ** -4 * x.abs() + 2.0 ** -7 * 2.0 ** -6 * 8).all()
    # the last token of each alone, and a row that sees one token is its value
    length = (first[1:] > first[:-1]).int()
    out = ar.cache_attention([x.float()], cache, table, first, length, causal=False, max_rows=4)
    heads = first[:-1][length > 0].long()
    want = v[heads].float()
    assert ((out[0][heads] - want).abs() <= want.abs() * 2.0 ** -22).all()  # weight and sum the same, a few roundings


def _time(seqs):
    x, table, first, start = case(seqs, torch.ones(seqs, dtype=torch.int64, device="cuda"))
    cache = ar.KVCache.empty(1, seqs, 1, 64, 16)
    best = np.inf
    for _ in range(4):
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        a.record()
        ar.cache_write(cache, [x], [x], table, first, start)
        b.record()
        torch.cuda.synchronize()
        best = min(best, a.elapsed_time(b))
    return best


def test_time_grows_as_the_sequences_do():
    """Eight times the sequences in 16 times the time at most (not in 64 times)."""
    few, many = _time(1 << 13), _time(1 << 16)
    assert many < 16 * few, (few, many)

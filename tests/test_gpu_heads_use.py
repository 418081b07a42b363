"""Attention operators in use: a tensor-parallel layer's prompt and decode
steps with the collectives, captured graphs, streams, caches past 4 GiB, many
sequences."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import heads
from test_gpu_heads import att_case, check, dev, host, ints

pytestmark = pytest.mark.gpu


class Layer:
    """The attention half of a layer over n ranks: projection, norms and rotation,
    cache, attention, output projection, all-reduce with the next norm."""

    def __init__(self, n, hidden, h, kv, dim, seqs, width, page=16):
        gen = torch.Generator(device="cuda").manual_seed(5)
        r = lambda *s, f=1.0: (torch.randn(*s, generator=gen, device="cuda") * f).bfloat16()  # noqa: E731
        self.n, self.h, self.kv, self.dim, self.hidden = n, h, kv, dim, hidden
        self.w_qkv = [r((h + 2 * kv) * dim, hidden, f=hidden ** -0.5) for _ in range(n)]
        self.w_out = [r(hidden, h * dim, f=(n * h * dim) ** -0.5) for _ in range(n)]
        self.qw, self.kw, self.nw = r(dim, f=0.1) + 1, r(dim, f=0.1) + 1, r(hidden, f=0.1) + 1
        self.freq = torch.pow(10000.0, -torch.arange(dim // 2, device="cuda") / (dim // 2)).float()
        self.cache = ar.KVCache.empty(n, seqs * width, kv, dim, page)
        self.table = torch.randperm(seqs * width, generator=gen, device="cuda").int().view(seqs, width)
        self.comm = ar.Comm(n, 1 << 20)

    def __call__(self, x, first, start, length, pos, keep=None, stream=None):
        h, kv, d = self.h, self.kv, self.dim
        qkv = [(x @ w.t()).view(-1, h + 2 * kv, d) for w in self.w_qkv]
        q, k = ar.qk_norm_rope([t[:, :h] for t in qkv], [t[:, h:h + kv] for t in qkv], self.qw, self.kw, pos, self.freq, stream=stream)
        ar.cache_write(self.cache, k, [t[:, h + kv:] for t in qkv], self.table, first, start, stream=stream)
        a = ar.cache_attention(q, self.cache, self.table, first, length, stream=stream)
        part = [t.view(-1, h * d) @ w.t() for t, w in zip(a, self.w_out)]
        out = [torch.empty_like(t) for t in part]
        res = [x.clone() for _ in part]
        self.comm.allreduce_rmsnorm(part, out, self.nw, residual=res, stream=stream)
        if keep is not None:
            keep.update(qkv=qkv, q=q, k=k, a=a, part=part, res=res)
        return out


def test_layer_prompt_and_decode():
    n, hidden, h, kv, dim, seqs = 4, 256, 3, 1, 64, 3
    layer = Layer(n, hidden, h, kv, dim, seqs, 8)
    gen = torch.Generator(device="cuda").manual_seed(9)
    past = np.zeros(seqs, int)
    ref = None
    for count in ([40, 1, 17], [1, 1, 1], [1, 5, 1], [1, 1, 1]):
        first = np.concatenate([[0], np.cumsum(count)])
        pos = np.concatenate([p + np.arange(c) for p, c in zip(past, count)])
        x = torch.randn(int(first[-1]), hidden, generator=gen, device="cuda").bfloat16()
        keep = {}
        out = layer(x, ints(first), ints(past), ints(past + count), torch.from_numpy(pos).cuda(), keep)
        if ref is None:  # what the pages held before counts for nothing
            ref = [heads.Cache(24, kv, 16, dim) for _ in range(n)]
        table = layer.table.cpu().numpy()
        total = 0
        for r in range(n):
            qkv = host(keep["qkv"][r])
            check(host(keep["q"][r]), *heads.norm_rope(qkv[:, :h], host(layer.qw), pos, host(layer.freq).astype(np.float32), False, 1e-6, "bf16"), "q")
            check(host(keep["k"][r]), *heads.norm_rope(qkv[:, h:h + kv], host(layer.kw), pos, host(layer.freq).astype(np.float32), False, 1e-6, "bf16"), "k")
            ref[r].write([host(keep["k"][r]), qkv[:, h + kv:]], table, first, past)
            (o, eo), _ = heads.attention(host(keep["q"][r]), ref[r], table, first, past + count, dim ** -0.5, True, 0, "bf16", 1)
            check(host(keep["a"][r]), o, eo, "attention")
            total = total + host(keep["part"][r])
        # the sum over the ranks, one rounding, and the residual's
        want = total + host(x)
        check(host(keep["res"][0]), want, 2.0 ** -8 * (np.abs(total) + np.abs(want)) * 1.1 + 1e-6, "residual")
        assert all(torch.equal(out[0], t) for t in out[1:])
        past = past + count
    layer.comm.close()


def test_captured_decode_step():
    """One decode step as a graph, replayed with new inputs and lengths, eager
    work between the replays: the same bits as eager calls on a copy."""
    n, h, kv, dim, seqs, width = 2, 4, 2, 64, 5, 12
    rng = np.random.default_rng(1)
    caches = [ar.KVCache.empty(n, seqs * width, kv, dim, 16) for _ in range(2)]
    for c in caches:
        for t in (*c.k, *c.v):
            t.zero_()
        for t in (*c.k_scale, *c.v_scale):
            t.fill_(120)
    table = ints(rng.permutation(seqs * width).reshape(seqs, width))
    first, start, length = ints(np.arange(seqs + 1)), ints([0, 3, 40, 150, 15]), ints([1, 4, 41, 151, 16])
    pos = start.long()
    w = torch.ones(dim, device="cuda").bfloat16()
    freq = torch.rand(dim // 2, device="cuda")
    qkv = [torch.randn(seqs, h + 2 * kv, dim, device="cuda").bfloat16() for _ in range(n)]

    def step(cache):
        q, k = ar.qk_norm_rope([t[:, :h] for t in qkv], [t[:, h:h + kv] for t in qkv], w, w, pos, freq)
        ar.cache_write(cache, k, [t[:, h + kv:] for t in qkv], table, first, start)
        return ar.cache_attention(q, cache, table, first, length, max_rows=1)

    step(caches[0])
    for c in caches[0].k + caches[0].v:
        c.zero_()
    for t in caches[0].k_scale + caches[0].v_scale:
        t.fill_(120)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(caches[0])
    for i in range(4):
        for t in qkv:
            t.copy_(torch.randn_like(t.float()) * 2.0 ** i)
        graph.replay()
        torch.cuda.synchronize()
        want = step(caches[1])
        assert all(torch.equal(a, b) for a, b in zip(out, want)), i
        for name in ("k", "v", "k_scale", "v_scale"):
            assert all(torch.equal(a, b) for a, b in zip(getattr(caches[0], name), getattr(caches[1], name)))
        start += 1
        length += 1
        pos += 1


def test_captured_backward():
    x = [torch.randn(300, 5, 128, device="cuda").bfloat16()]
    g = [torch.randn(300, 4, 128, device="cuda").bfloat16()]
    gk = [torch.randn(300, 1, 128, device="cuda").bfloat16()]
    w = torch.ones(128, device="cuda").bfloat16()
    pos, freq = torch.arange(300, device="cuda"), torch.rand(64, device="cuda")
    call = lambda: ar.qk_norm_rope_backward(g, gk, [x[0][:, :4]], [x[0][:, 4:]], w, w, pos, freq)  # noqa: E731
    call()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = call()
    for i in range(3):
        x[0].normal_()
        g[0].normal_()
        graph.replay()
        torch.cuda.synchronize()
        want = call()
        assert all(torch.equal(a[0], b[0]) for a, b in zip(got, want)), i


def test_two_streams_at_once():
    cases = [att_case(2, 5, 1, 128, 64, [3000, 900], [1, 1], "bf16", seed=s) for s in range(2)]
    want = [ar.cache_attention(q, c, ints(t), ints(f), ints([3000, 900]), max_rows=1) for _, c, t, f, q in cases]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    args = [(q, c, ints(t), ints(f), ints([3000, 900])) for _, c, t, f, q in cases]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(6):
        for i, s in enumerate(streams):
            got[i].append(ar.cache_attention(*args[i], max_rows=1, stream=s))
    torch.cuda.synchronize()
    for i in range(2):
        f = cases[i][3]
        for o in got[i]:
            assert all(torch.equal(a[f[0]:f[-1]], b[f[0]:f[-1]]) for a, b in zip(o, want[i]))


@pytest.mark.parametrize("most", [1, 128])
def test_cache_past_4_gib(most):
    kv, dim, page = 8, 256, 128
    pages = (5 << 30) // (kv * page * dim)
    cache = ar.KVCache.empty(1, pages, kv, dim, page)
    ids = [pages - 1, pages // 2, 1, pages - 7]
    table = ints([ids[:2], ids[2:]])
    gen = torch.Generator(device="cuda").manual_seed(2)
    k = [torch.randn(400, kv, dim, generator=gen, device="cuda").bfloat16()]
    v = [torch.randn(400, kv, dim, generator=gen, device="cuda").bfloat16()]
    first, length = ints([0, 200, 400]), ints([200, 200])
    ar.cache_write(cache, k, v, table, first, ints([0, 0]))
    kb, vb = [torch.empty_like(k[0])], [torch.empty_like(k[0])]
    ar.cache_read(cache, table, first, ints([0, 0]), kb, vb)
    for a, b in ((k, kb), (v, vb)):
        # half a step of e4m3: 2^-4 of the value, or of its smallest normal number (2^-6 over 448 of a page's largest)
        bound = 2.0 ** -4 * torch.clamp(a[0].abs().double(), min=a[0].abs().max().item() * 2.0 ** -14)
        assert ((a[0].double() - b[0].double()).abs() <= bound).all()
    n = most
    q = [torch.randn(2 * n, kv, dim, generator=gen, device="cuda").bfloat16()]
    if n > 1:  # room for more tokens: the kernel of many rows
        table = torch.cat([table, torch.full((2, 8), -1, dtype=torch.int32, device="cuda")], 1)
    out = ar.cache_attention(q, cache, table, ints([0, n, 2 * n]), length, causal=False, max_rows=n)
    z = torch.einsum("snhd,sjhd->shnj", q[0].view(2, n, kv, dim).double().cpu(), kb[0].view(2, 200, kv, dim).double().cpu()) / 16
    want = torch.einsum("shnj,sjhd->snhd", torch.softmax(z, -1), vb[0].view(2, 200, kv, dim).double().cpu()).reshape(2 * n, kv, dim)
    mag = torch.einsum("shnj,sjhd->snhd", torch.softmax(z, -1), vb[0].view(2, 200, kv, dim).double().cpu().abs()).reshape(2 * n, kv, dim)
    # weights and result rounded to bf16, scores to 1e-5 of themselves
    assert ((out[0].double().cpu() - want).abs() <= 2.0 ** -8 * 3.1 * mag + 1e-4).all()


def test_many_sequences():
    """More sequences than a wave looks at in one step, most of them empty."""
    rng = np.random.default_rng(8)
    seqs, page, kv, dim, h = 300, 16, 1, 64, 2
    count = np.where(rng.random(seqs) < 0.4, rng.integers(0, 4, seqs), 0)
    past = rng.integers(0, 20, seqs)
    first = np.concatenate([[0], np.cumsum(count)])
    rows, width = int(first[-1]), 3
    ref = [heads.Cache(seqs * width, kv, page, dim)]
    ref[0].codes[0][:] = ref[0].codes[1][:] = 0x31
    from test_gpu_heads import same_cache, upload
    cache = upload(ref)
    table = rng.permutation(seqs * width).reshape(seqs, width)
    k, v, q = (dev(rng.normal(size=(rows, x, dim)), "bf16") for x in (kv, kv, h))
    ref[0].write([host(k), host(v)], table, first, past)
    ar.cache_write(cache, [k], [v], ints(table), ints(first), ints(past))
    same_cache(ref, cache)
    wide = np.concatenate([table, np.full((seqs, 80), -1)], 1)
    for most, pages in ((3, table), (100, wide)):
        out = ar.cache_attention([q], cache, ints(pages), ints(first), ints(past + count), max_rows=most)
        (o, eo), _ = heads.attention(host(q), ref[0], table, first, past + count, 0.125, True, 0, "bf16", 1)
        check(host(out[0]), o, eo, "out")


def test_a_table_cut_out_of_a_wider_one():
    _, cache, table, first, q = att_case(1, 2, 1, 64, 16, [30, 40], [2, 2], "bf16")
    wide = ints(np.concatenate([table, np.full_like(table, 1 << 20)], 1))
    a = ar.cache_attention(q, cache, wide[:, :table.shape[1]], ints(first), ints([30, 40]))
    b = ar.cache_attention(q, cache, ints(table), ints(first), ints([30, 40]))
    assert torch.equal(a[0][first[0]:first[-1]], b[0][first[0]:first[-1]])


def test_no_sequences_and_no_rows():
    _, cache, _, _, _ = att_case(1, 2, 1, 64, 16, [30], [2], "bf16")
    none = torch.zeros(0, 4, dtype=torch.int32, device="cuda")
    q, k = [torch.zeros(0, 2, 64, device="cuda")], [torch.zeros(0, 1, 64, device="cuda")]
    assert ar.cache_attention(q, cache, none, ints([0]), ints([]))[0].shape == (0, 2, 64)
    ar.cache_write(cache, k, k, none, ints([0]), ints([]))
    ar.cache_read(cache, none, ints([0]), ints([]), k, k[:1] and [torch.zeros(0, 1, 64, device="cuda")])
    out = [torch.full((3, 2, 64), 5.0, device="cuda")]
    ar.cache_attention([torch.zeros(3, 2, 64, device="cuda")], cache, none, ints([0]), ints([]), out=out)
    assert (out[0] == 5).all()

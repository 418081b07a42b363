"""Attention operators on the GPU against the fp64 oracle, element by element
within its error bounds: norms with the rotation and their gradients, the
8-bit cache, attention over it."""

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from oracle import heads

pytestmark = pytest.mark.gpu

T = {"bf16": torch.bfloat16, "f32": torch.float32}


def dev(x, dt=None):
    t = torch.from_numpy(np.ascontiguousarray(x)).cuda()
    return t if dt is None else t.to(T[dt])


def host(t):
    return t.detach().double().cpu().numpy()


def ints(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check(got, want, bound, what):
    bad = ~(np.abs(got - want) <= bound) & ~((got == want) | (np.isnan(got) & np.isnan(want)))
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} outside, first at {np.argwhere(bad)[0]}: got {got[bad][0]} want {want[bad][0]} +- {bound[bad][0]}"


# ---- norms and rotation ----

ROPE = [  # ranks, rows, heads, kv_heads, dim, rot, pairs, dtype
    (1, 1, 1, 1, 64, 64, False, "bf16"), (8, 1, 5, 1, 128, 128, False, "bf16"), (2, 37, 7, 3, 128, 64, True, "bf16"),
    (3, 130, 4, 2, 256, 256, False, "bf16"), (1, 19, 3, 0, 64, 16, False, "bf16"), (2, 65, 2, 2, 128, 0, False, "bf16"),
    (1, 33, 9, 1, 256, 48, True, "bf16"), (2, 21, 5, 5, 64, 32, True, "f32"), (1, 257, 3, 1, 128, 112, False, "f32"),
    (3, 9, 2, 1, 256, 256, False, "f32"), (1, 70, 40, 8, 128, 128, False, "bf16"), (8, 3, 1, 1, 64, 64, True, "f32"),
]


def rope_case(n, rows, h, kv, dim, rot, dt, seed=0):
    rng = np.random.default_rng(seed)
    qkv = [dev(rng.normal(size=(rows, h + 2 * kv + 1, dim)) * 1.5, dt) for _ in range(n)]  # one head more than is used
    w = [dev(1 + 0.3 * rng.normal(size=dim), dt) for _ in range(2)]
    pos = rng.integers(0, 1 << 20, rows)
    pos[0] = 0
    freq = (500000.0 ** -(np.arange(rot // 2) / max(1, rot // 2))).astype(np.float32)
    q = [t[:, :h] for t in qkv]
    k = [t[:, h:h + kv] for t in qkv] if kv else None
    return q, k, w, dev(pos), dev(freq) if rot else None, pos, freq


@pytest.mark.parametrize("n,rows,h,kv,dim,rot,pairs,dt", ROPE)
def test_rope(n, rows, h, kv, dim, rot, pairs, dt):
    q, k, w, pos, freq, hpos, hfreq = rope_case(n, rows, h, kv, dim, rot, dt)
    kw = w[1] if kv else None
    qo, ko = ar.qk_norm_rope(q, k, w[0], kw, pos if rot else None, freq, eps=1e-5, pairs=pairs)
    for r in range(n):
        for x, o, weight, what in ((q, qo, w[0], "q"), (k, ko, w[1], "k")):
            if x is None:
                assert o is None
                continue
            check(host(o[r]), *heads.norm_rope(host(x[r]), host(weight), hpos, hfreq, pairs, 1e-5, dt), f"{what}[{r}]")


@pytest.mark.parametrize("n,rows,h,kv,dim,rot,pairs,dt", ROPE)
def test_rope_backward(n, rows, h, kv, dim, rot, pairs, dt):
    q, k, w, pos, freq, hpos, hfreq = rope_case(n, rows, h, kv, dim, rot, dt, 1)
    rng = np.random.default_rng(7)
    dq_out = [dev(rng.normal(size=(rows, h, dim)), dt) for _ in range(n)]
    dk_out = [dev(rng.normal(size=(rows, kv, dim)), dt) for _ in range(n)] if kv else None
    # gradients as columns of one matrix, which keeps what lies between them
    dqkv = [torch.full((rows, h + 2 * kv + 1, dim), 7.0, dtype=T[dt], device="cuda") for _ in range(n)]
    dq, dk = [t[:, :h] for t in dqkv], [t[:, h:h + kv] for t in dqkv] if kv else None
    got = ar.qk_norm_rope_backward(dq_out, dk_out, q, k, w[0], w[1] if kv else None, pos if rot else None, freq, eps=1e-5,
                                   pairs=pairs, dq=dq, dk=dk)
    again = ar.qk_norm_rope_backward(dq_out, dk_out, q, k, w[0], w[1] if kv else None, pos if rot else None, freq, eps=1e-5,
                                     pairs=pairs)
    for r in range(n):
        assert (dqkv[r][:, h + kv:] == 7.0).all()
        for i, (x, d, weight) in enumerate(((q, dq_out, w[0]), (k, dk_out, w[1]))):
            if x is None:
                assert got[i] is None and got[2 + i] is None
                continue
            dx, dw = heads.norm_rope_backward(host(d[r]), host(x[r]), host(weight), hpos, hfreq, pairs, 1e-5, dt)
            check(host(got[i][r]), *dx, f"d{'qk'[i]}[{r}]")
            check(host(got[2 + i][r]), *dw, f"d{'qk'[i]}_weight[{r}]")
            assert torch.equal(got[i][r], again[i][r]) and torch.equal(got[2 + i][r], again[2 + i][r])


def test_rope_backward_against_differences():
    """The GPU's gradient against differences of the GPU's own forward pass."""
    q, k, w, pos, freq, _, _ = rope_case(1, 4, 2, 1, 64, 64, "f32", 3)
    g = [torch.randn(4, 2, 64, device="cuda")]
    gk = [torch.randn(4, 1, 64, device="cuda")]
    dq, dk, dwq, _ = ar.qk_norm_rope_backward(g, gk, q, k, *w, pos, freq)

    def loss(x, weight):
        out, _ = ar.qk_norm_rope([x], k, weight, w[1], pos, freq)
        return (out[0].double() * g[0].double()).sum()

    h = 2.0 ** -6
    size = (dq[0].abs().max() + dwq[0].abs().max()).item()
    for at in ((0, 0, 0), (1, 1, 40), (3, 0, 17)):
        e = torch.zeros_like(q[0])
        e[at] = h
        num = ((loss(q[0] + e, w[0]) - loss(q[0] - e, w[0])) / (2 * h)).item()
        # h^2 / 6 of a third derivative of order size, and fp32 values over h
        assert abs(num - dq[0][at].item()) < size * (h * h + 2.0 ** -24 * 64 / h)
    e = torch.zeros(64, device="cuda")
    e[5] = h
    num = ((loss(q[0], w[0] + e) - loss(q[0], w[0] - e)) / (2 * h)).item()
    assert abs(num - dwq[0][5].item()) < size * 2.0 ** -24 * 512 / h  # linear in the weight


def test_rope_no_rows():
    q, k, w, pos, freq, _, _ = rope_case(2, 1, 2, 1, 64, 64, "bf16")
    q, k, pos = [t[:0] for t in q], [t[:0] for t in k], pos[:0]
    qo, ko = ar.qk_norm_rope(q, k, *w, pos, freq)
    assert qo[0].shape == (0, 2, 64) and ko[1].shape == (0, 1, 64)
    dwq = [torch.full((64,), 3.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    ar.qk_norm_rope_backward([t.contiguous() for t in q], [t.contiguous() for t in k], q, k, *w, pos, freq, dq_weight=dwq)
    assert all((t == 0).all() for t in dwq)


# ---- the cache ----


def make_cache(n, pages, kv, page, dim, seed=0):
    """Oracle caches of arbitrary codes (NaN among them) and their copies."""
    rng = np.random.default_rng(seed)
    ref = [heads.Cache(pages, kv, page, dim, rng) for _ in range(n)]
    return ref, upload(ref)


def upload(ref):
    return ar.KVCache([dev(c.codes[0]) for c in ref], [dev(c.codes[1].transpose(0, 1, 3, 2)) for c in ref],
                      [dev(c.scale[0]) for c in ref], [dev(c.scale[1]) for c in ref])


def same_cache(ref, cache):
    for r, c in enumerate(ref):
        np.testing.assert_array_equal(cache.k[r].cpu().numpy(), c.codes[0])
        np.testing.assert_array_equal(cache.v[r].cpu().numpy().transpose(0, 1, 3, 2), c.codes[1])
        np.testing.assert_array_equal(cache.k_scale[r].cpu().numpy(), c.scale[0])
        np.testing.assert_array_equal(cache.v_scale[r].cpu().numpy(), c.scale[1])


def pages_for(rng, seqs, width, pages):
    return rng.permutation(pages)[:seqs * width].reshape(seqs, width)


CACHE = [  # ranks, kv_heads, dim, page, starts, rows per sequence, dtype
    (1, 1, 64, 16, [0], [1], "bf16"), (8, 1, 128, 64, [0, 63, 64, 130], [1, 1, 1, 1], "bf16"),
    (2, 2, 128, 32, [5, 0, 31], [40, 0, 3], "bf16"), (1, 3, 256, 128, [100, 7], [70, 130], "bf16"),
    (3, 1, 64, 16, [3, 17, 0, 8], [30, 1, 16, 0], "f32"), (2, 1, 128, 128, [1], [200], "f32"), (1, 2, 256, 16, [15, 2], [2, 14], "f32"),
]


@pytest.mark.parametrize("n,kv,dim,page,start,count,dt", CACHE)
def test_cache_write_and_read(n, kv, dim, page, start, count, dt):
    rng = np.random.default_rng(11)
    seqs, width = len(start), 1 + max(s + c for s, c in zip(start, count)) // page + 1
    ref, cache = make_cache(n, seqs * width + 2, kv, page, dim)
    table = pages_for(rng, seqs, width, seqs * width + 2)
    lead = 2  # rows before the first sequence and behind the last
    first = lead + np.concatenate([[0], np.cumsum(count)])
    rows = int(first[-1]) + 3
    size = 2.0 ** rng.integers(-12, 6, (rows, kv, 1))
    new = [[dev(rng.normal(size=(rows, kv, dim)) * size, dt) for _ in range(2)] for _ in range(n)]
    for r in range(n):  # zeros, what is not finite, a value at the border of a scale
        new[r][0][lead, 0, :4] = torch.tensor([float("inf"), float("nan"), 0.0, -float("inf")])
        new[r][1][lead, 0, :3] = torch.tensor([448.0, -0.0, 1e-30])
    wide = [torch.cat([t[0], t[1]], 1) for t in new]  # values as a view of a wider matrix
    for c, t in zip(ref, new):
        c.write([host(t[0]), host(t[1])], table, first, np.array(start))
    ar.cache_write(cache, [t[0] for t in new], [t[:, kv:] for t in wide], ints(table), ints(first), ints(start))
    same_cache(ref, cache)
    # read back all that is there, the tokens before `start` too
    upto = np.array(start) + np.array(count)
    back = np.concatenate([[0], np.cumsum(upto)])
    k = [torch.full((int(back[-1]) + 1, kv, dim), 5.0, dtype=T[dt], device="cuda") for _ in range(n)]
    v = [torch.full_like(t, 5.0) for t in k]
    ar.cache_read(cache, ints(table), ints(back), ints([0] * seqs), k, v)
    for r in range(n):
        assert (k[r][-1] == 5.0).all() and (v[r][-1] == 5.0).all()
        for s in range(seqs):
            for i, t in ((0, k), (1, v)):
                want, _ = ref[r].tokens(i, s, table, 0, int(upto[s]))
                got = host(t[r][int(back[s]):int(back[s + 1])])
                np.testing.assert_array_equal(got, want)


def test_cache_pages_that_grow_step_by_step():
    """One token at a time, magnitudes that rise and fall: scales follow, codes move."""
    rng = np.random.default_rng(4)
    ref, cache = make_cache(1, 3, 2, 16, 64)
    table = np.array([[2, 0]])
    for t in range(20):
        new = [dev(rng.normal(size=(1, 2, 64)) * 2.0 ** rng.integers(-9, 9), "f32") for _ in range(2)]
        ref[0].write([host(x) for x in new], table, np.array([0, 1]), np.array([t]))
        ar.cache_write(cache, [new[0]], [new[1]], ints(table), ints([0, 1]), ints([t]))
    same_cache(ref, cache)


def test_cache_drops_tokens_without_a_page():
    rng = np.random.default_rng(6)
    ref, cache = make_cache(1, 4, 1, 16, 64)
    table = np.array([[1, -1, 3], [4, 0, 1 << 30]])  # no page: -1, 4 (one past the end), 2^30
    first, start = np.array([0, 45, 100]), np.array([8, 0])  # both run past the table too
    new = [dev(rng.normal(size=(100, 1, 64)), "bf16") for _ in range(2)]
    ref[0].write([host(x) for x in new], table, first, start)
    ar.cache_write(cache, [new[0]], [new[1]], ints(table), ints(first), ints(start))
    same_cache(ref, cache)
    k, v = [torch.full((100, 1, 64), 5.0, device="cuda")], [torch.full((100, 1, 64), 5.0, device="cuda")]
    ar.cache_read(cache, ints(table), ints(first), ints(start), k, v)
    for s in range(2):
        for i, t in ((0, k), (1, v)):
            want, _ = ref[0].tokens(i, s, table, start[s], first[s + 1] - first[s])
            np.testing.assert_array_equal(host(t[0][first[s]:first[s + 1]]), want)


@pytest.mark.parametrize("first", [[0, -5, 1 << 30], [7, 3, 1], [-9, -9, -9], [0, 1 << 30, 2]])
def test_rows_out_of_order_stay_inside(first):
    """`first` that is not what the documentation asks for: nothing outside the
    buffers is touched (guard rows around each keep their values)."""
    cache = upload([heads.Cache(6, 1, 16, 64)])
    table, at = ints([[0, 1, 2], [3, 4, 5]]), ints([-4, (1 << 31) - 1])
    big = torch.full((24, 1, 64), 3.0, device="cuda")
    k = [big[8:16]]
    ar.cache_write(cache, k, k, table, ints(first), at)
    out = torch.full((24, 1, 64), 9.0, device="cuda")
    out2 = torch.full((24, 1, 64), 9.0, device="cuda")
    ar.cache_read(cache, table, ints(first), at, [out[8:16]], [out2[8:16]])
    ar.cache_attention(k, cache, table, ints(first), at, out=[out[8:16]], max_rows=1)
    # the kernel of many rows: 16 heads to a key, a table with room for more tokens
    table = torch.cat([table, torch.full((2, 70), 5, dtype=torch.int32, device="cuda")], 1)
    q, wide = torch.ones(8, 16, 64, device="cuda"), torch.full((24, 16, 64), 9.0, device="cuda")
    ar.cache_attention([q], cache, table, ints(first), at, out=[wide[8:16]], max_rows=8)
    torch.cuda.synchronize()
    assert (wide[:8] == 9).all() and (wide[16:] == 9).all()
    for t in (out, out2):
        assert (t[:8] == 9).all() and (t[16:] == 9).all()


# ---- attention ----

ATT = [  # ranks, heads, kv_heads, dim, page, cached tokens, query rows, causal, window, dtype, max_rows
    (1, 1, 1, 64, 16, [1], [1], True, 0, "bf16", 1),
    (8, 5, 1, 128, 64, [63, 64, 65, 700], [1, 1, 1, 1], True, 0, "bf16", 1),
    (2, 8, 2, 64, 16, [33, 5, 200], [3, 5, 1], True, 0, "bf16", 0),
    (1, 6, 3, 128, 32, [90, 300], [2, 7], True, 40, "bf16", 7),
    (1, 4, 1, 256, 128, [129, 1000], [1, 4], True, 0, "bf16", 4),
    (2, 3, 3, 128, 16, [77, 400], [1, 2], True, 0, "f32", 2),
    (1, 16, 2, 64, 64, [130, 9], [4, 1], True, 100, "f32", 4),
    (1, 2, 1, 256, 32, [70, 515], [1, 3], True, 0, "f32", 0),
    (2, 5, 1, 128, 64, [150, 64, 33], [150, 64, 20], True, 0, "bf16", 0),
    (1, 4, 4, 64, 16, [200, 17], [130, 17], True, 50, "bf16", 0),
    (1, 2, 1, 256, 64, [140, 80], [70, 80], True, 0, "bf16", 80),
    (1, 3, 1, 128, 32, [300, 40], [50, 1], False, 0, "bf16", 50),
    (1, 6, 6, 64, 32, [130, 70], [129, 33], True, 0, "f32", 0),
    (1, 8, 2, 128, 16, [50, 199], [50, 3], True, 0, "f32", 50),
    (1, 2, 2, 256, 128, [60], [40], False, 0, "f32", 40),
    (2, 1, 1, 128, 64, [1500], [40], True, 0, "bf16", 40),       # shared among workgroups
    (1, 2, 2, 128, 64, [2000], [1], False, 0, "f32", 1),
    (1, 64, 1, 128, 64, [300], [1], True, 0, "bf16", 1),          # 64 heads to one key
    (8, 3, 1, 128, 64, [700, 1, 640, 90, 513, 1100, 2, 64, 800], [1] * 9, True, 0, "bf16", 1),  # eight waves a tile
    (2, 5, 1, 128, 64, [150, 64, 33], [150, 64, 20], True, 0, "bf16", 150),   # from here on: many rows
    (1, 4, 4, 64, 16, [200, 17], [130, 17], True, 50, "bf16", 130),
    (1, 2, 1, 256, 64, [140, 80], [70, 80], True, 0, "bf16", 80),
    (1, 3, 1, 128, 32, [300, 40], [50, 1], False, 0, "bf16", 50),
    (3, 2, 1, 64, 128, [1, 500], [1, 99], True, 120, "bf16", 99),
    (1, 6, 6, 64, 32, [130, 70], [129, 33], True, 0, "f32", 129),
    (1, 8, 2, 128, 16, [50, 199], [50, 3], True, 0, "f32", 50),
    (1, 3, 1, 256, 128, [60], [40], False, 0, "f32", 40),
    (2, 3, 1, 128, 64, [1500], [40], True, 0, "bf16", 40),
    (1, 7, 1, 64, 64, [700, 5], [20, 5], True, 0, "f32", 20),
    (4, 4, 4, 64, 16, [600, 70, 515, 540, 580], [1, 2, 1, 1, 1], True, 0, "f32", 2),
]


def att_case(n, h, kv, dim, page, length, count, dt, seed=0, wide=False):
    """wide: a table with room for more tokens than the kernel of few rows takes
    whatever the rows (97 packed rows and more then go to the kernel of many)."""
    rng = np.random.default_rng(seed)
    seqs, width = len(length), max(1, -(-max(length) // page)) + 1
    pages = seqs * width + 1
    ref = [heads.Cache(pages, kv, page, dim, rng) for _ in range(n)]
    for c in ref:  # scales of like size; codes without NaN up to a length, anything behind
        for i in range(2):
            c.scale[i][:] = rng.integers(118, 122, c.scale[i].shape)
    table = pages_for(rng, seqs, width, pages)
    for c in ref:
        for i in range(2):
            for s in range(seqs):
                for t in range(length[s]):
                    x = c.codes[i][table[s, t // page], :, t % page]
                    x[(x & 0x7f) == 0x7f] = 0x30
    if wide:
        table = np.concatenate([table, np.full((seqs, 1100 // page), -1)], 1)
    first = np.concatenate([[0], np.cumsum(count)]) + 1
    rows = int(first[-1]) + 2
    q = [dev(rng.normal(size=(rows, h + 1, dim)) * 0.4, dt)[:, 1:] for _ in range(n)]
    return ref, upload(ref), table, first, q


@pytest.mark.parametrize("n,h,kv,dim,page,length,count,causal,window,dt,most", ATT)
def test_attention(n, h, kv, dim, page, length, count, causal, window, dt, most):
    wide = max(count) * h // kv > 96
    ref, cache, table, first, q = att_case(n, h, kv, dim, page, length, count, dt, wide=wide)
    out = [torch.full(q[0].shape, 5.0, dtype=T[dt], device="cuda") for _ in range(n)]
    lse = [torch.full(q[0].shape[:2], 5.0, device="cuda") for _ in range(n)]
    scale = dim ** -0.5
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), causal=causal, window=window, max_rows=most, out=out, lse=lse)
    plain = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), causal=causal, window=window, max_rows=most)
    a, b = int(first[0]), int(first[-1])
    few = (most or -(-q[0].shape[0] // len(length))) * (h // kv) <= 96
    for r in range(n):
        (o, eo), (z, ez) = heads.attention(host(q[r]), ref[r], table, first, length, scale, causal, window, dt,
                                           3 if dt == "f32" else 2 if few else 1)
        assert (got[r][:a] == 5).all() and (got[r][b:] == 5).all() and (lse[r][b:] == 5).all()
        check(host(got[r][a:b]), o[a:b], eo[a:b], f"out[{r}]")
        check(host(lse[r][a:b]), z[a:b], ez[a:b], f"lse[{r}]")
        assert torch.equal(got[r][a:b], plain[r][a:b])  # twice the same bits, lse or not


@pytest.mark.parametrize("most,count", [(1, [2, 6, 2, 3]), (60, [50, 60, 40, 45])])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_attention_rows_that_see_nothing(most, count, dt):
    # no cached token, fewer cached tokens than rows, a page that is missing, a window on missing pages
    length, page = [0, 3, 40, 60], 16
    ref, cache, table, first, q = att_case(1, 4, 2, 64, page, length, count, dt, wide=most > 1)
    table[2, 0] = -1
    table[3, 2:4] = 1 << 20
    for window in (0, 8):
        lse = [torch.empty(q[0].shape[:2], device="cuda")]
        got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), window=window, max_rows=most, lse=lse)
        (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, 0.125, True, window, dt, 3 if dt == "f32" else 1)
        a, b = int(first[0]), int(first[-1])
        assert (o[a:b] == 0).all(axis=(1, 2)).sum() >= 5
        check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
        check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")


@pytest.mark.parametrize("most,count", [(1, 6), (200, 90)])
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_attention_nan_reaches_only_who_sees_it(most, count, dt, dim):
    length, page = [100, 1100], 32
    ref, cache, table, first, q = att_case(1, 2, 1, dim, page, length, [count, count], dt)
    c = ref[0]
    # a value of sequence 0's last token but one, one of sequence 1's fifth (seen by all), a key
    # of sequence 1's last token
    c.codes[1][table[0, 98 // page], 0, 98 % page, 3] = 0x7f
    c.codes[1][table[1, 0], 0, 5, dim - 1] = 0xff
    c.codes[0][table[1, 1099 // page], 0, 1099 % page, 0] = 0x7f
    cache = upload(ref)
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), max_rows=most, lse=lse)
    clean = [x.copy() for x in c.codes]
    for x in c.codes:
        x[(x & 0x7f) == 0x7f] = 0  # the oracle's copy: without NaN, which is put where it is seen
    few = (most or count) * 2 <= 96
    (o, eo), (z, ez) = heads.attention(host(q[0]), c, table, first, length, dim ** -0.5, True, 0, dt, 3 if dt == "f32" else 2 if few else 1)
    c.codes = clean
    a, m, b = (int(x) for x in first)
    o[m - 2:m, :, 3] = np.nan      # rows at positions 98 and 99
    o[m:b, :, dim - 1] = np.nan
    o[b - 1], z[b - 1] = np.nan, np.nan
    check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")


@pytest.mark.parametrize("most", [1, 100])
def test_attention_nan_queries(most):
    """A row of NaN, and one that holds an infinity: NaN themselves, and no other row."""
    length, count = [90, 700], [4, 60]
    ref, cache, table, first, q = att_case(1, 2, 1, 128, 16, length, count, "bf16", wide=most > 1)
    q = [q[0].clone()]
    a, b = int(first[0]), int(first[-1])
    clean = [q[0].clone()]
    q[0][a + 1] = float("nan")
    q[0][b - 3, 1, 7] = float("inf")
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), max_rows=most)
    want = ar.cache_attention(clean, cache, ints(table), ints(first), ints(length), max_rows=most)
    assert got[0][a + 1].isnan().all() and got[0][b - 3, 1].isnan().all()
    got[0][a + 1], got[0][b - 3, 1] = want[0][a + 1], want[0][b - 3, 1]
    assert torch.equal(got[0][a:b], want[0][a:b])


@pytest.mark.parametrize("most", [1, 100])
@pytest.mark.parametrize("scale", [-0.2, 0.0, 1.0])
def test_attention_scales(most, scale):
    length, count = [90, 41], [4, 33]
    ref, cache, table, first, q = att_case(1, 3, 1, 128, 16, length, count, "bf16", wide=most > 1)
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), scale=scale, max_rows=most, lse=lse)
    (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, scale, True, 0, "bf16", 1)
    a, b = int(first[0]), int(first[-1])
    check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")


def test_attention_queries_of_all_sizes():
    """Rows of bf16 queries whose elements span many binades, beside tiny and huge rows."""
    length, count = [130], [60]
    ref, cache, table, first, q = att_case(1, 2, 1, 128, 64, length, count, "bf16", wide=True)
    rng = np.random.default_rng(3)
    spread = 2.0 ** rng.integers(-30, 1, q[0].shape)
    rows = 2.0 ** rng.integers(-40, 3, (q[0].shape[0], 1, 1))
    q = [(q[0].double().cpu() * torch.from_numpy(spread * rows)).to(torch.bfloat16).cuda()]
    lse = [torch.empty(q[0].shape[:2], device="cuda")]
    got = ar.cache_attention(q, cache, ints(table), ints(first), ints(length), scale=1.0, max_rows=60, lse=lse)
    (o, eo), (z, ez) = heads.attention(host(q[0]), ref[0], table, first, length, 1.0, True, 0, "bf16", 1)
    a, b = int(first[0]), int(first[-1])
    check(host(got[0][a:b]), o[a:b], eo[a:b], "out")
    check(host(lse[0][a:b]), z[a:b], ez[a:b], "lse")

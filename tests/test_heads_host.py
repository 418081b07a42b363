"""Attention operators on the host (no GPU): the fp64 oracle against torch's
own operators and against differences, the binding's and the C ABI's refusals,
and the workspace sizes."""

import ctypes

import numpy as np
import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from all_reduce_reduction_rank_amd import binding
from oracle import heads

F64 = torch.float64


# ---- the oracle ----


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("rot", [0, 16, 64])
def test_oracle_rope_matches_autograd(pairs, rot):
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(5, 3, 64, generator=gen, dtype=F64, requires_grad=True)
    w = torch.randn(64, generator=gen, dtype=F64, requires_grad=True)
    dout = torch.randn(5, 3, 64, generator=gen, dtype=F64)
    pos = torch.tensor([0, 1, 7, 100000, -3])
    freq = torch.rand(rot // 2, generator=gen, dtype=torch.float32)
    y = x / torch.sqrt((x * x).mean(-1, keepdim=True) + 1e-5) * w
    a = torch.polar(torch.ones(5, rot // 2, dtype=F64), pos[:, None].double() * freq.double())[:, None]
    if pairs:
        z = torch.view_as_complex(y[..., :rot].reshape(5, 3, rot // 2, 2).contiguous()) * a
        turned = torch.view_as_real(z).reshape(5, 3, rot)
    else:
        z = torch.complex(y[..., :rot // 2], y[..., rot // 2:rot]) * a
        turned = torch.cat([z.real, z.imag], -1)
    out = torch.cat([turned, y[..., rot:]], -1)
    out.backward(dout)
    args = (pos.numpy(), freq.numpy(), pairs, 1e-5, "f32")
    got, _ = heads.norm_rope(x.detach().numpy(), w.detach().numpy(), *args)
    np.testing.assert_allclose(got, out.detach().numpy(), rtol=1e-11, atol=1e-12)
    (dx, _), (dw, _) = heads.norm_rope_backward(dout.numpy(), x.detach().numpy(), w.detach().numpy(), *args)
    np.testing.assert_allclose(dx, x.grad.numpy(), rtol=1e-10, atol=1e-12)
    np.testing.assert_allclose(dw, w.grad.numpy(), rtol=1e-10, atol=1e-12)


def test_oracle_rope_backward_against_differences():
    rng = np.random.default_rng(5)
    x, w, dout = rng.normal(size=(2, 2, 64)), rng.normal(size=64), rng.normal(size=(2, 2, 64))
    args = (np.array([3, 90]), rng.random(8).astype(np.float32), False, 1e-6, "f32")
    (dx, _), _ = heads.norm_rope_backward(dout, x, w, *args)
    h = 1e-6
    for at in ((0, 0, 0), (1, 1, 9), (0, 1, 40), (1, 0, 63)):
        up, down = x.copy(), x.copy()
        up[at] += h
        down[at] -= h
        num = ((heads.norm_rope(up, w, *args)[0] - heads.norm_rope(down, w, *args)[0]) * dout).sum() / (2 * h)
        assert abs(num - dx[at]) < 1e-7  # h^2 of the third derivative, and 1e-16 / h of rounding


def test_oracle_codes_are_torchs_e4m3():
    codes = torch.arange(256, dtype=torch.int32).to(torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    np.testing.assert_array_equal(heads.VALUES, codes)
    rng = np.random.default_rng(1)
    grid = heads.VALUES[:127]
    y = np.concatenate([rng.uniform(-448, 448, 4000), rng.normal(size=4000) * 2.0 ** rng.integers(-14, 6, 4000), grid,
                        -grid, (grid[1:] + grid[:-1]) / 2])
    y = y.astype(np.float32).astype(np.float64)
    want = torch.from_numpy(y).float().to(torch.float8_e4m3fn).view(torch.uint8).numpy()
    np.testing.assert_array_equal(heads.encode(y), want)
    assert list(heads.encode(np.array([np.inf, -np.inf, np.nan]))) == [0x7f] * 3


def test_oracle_scale_byte():
    assert heads.scale_byte(0.0) == 1
    for e in (-100, -3, 0, 5, 100):
        assert heads.scale_byte(448.0 * 2.0 ** e) == 127 + e
        assert heads.scale_byte(448.0 * 2.0 ** e * (1 + 2.0 ** -20)) == 128 + e
    assert heads.scale_byte(3e38) <= 254


def test_oracle_attention_matches_torch():
    rng = np.random.default_rng(2)
    c = heads.Cache(4, 2, 16, 64)
    table = np.array([[2, 0, 3], [1, -1, -1]])
    k = [rng.normal(size=(50, 2, 64)) for _ in range(2)]
    first, start = np.array([0, 40, 50]), np.array([0, 0])
    c.write(k, table, first, start)
    q = rng.normal(size=(7, 4, 64))
    (out, _), (lse, _) = heads.attention(q, c, table, np.array([0, 3, 7]), np.array([40, 10]), 0.125, True, 0, "f32", 3)
    for s, (a, b, length) in enumerate(((0, 3, 40), (3, 7, 10))):
        kk, _ = c.tokens(0, s, table, 0, length)
        vv, _ = c.tokens(1, s, table, 0, length)
        kt, vt = (torch.from_numpy(np.repeat(x, 2, 1)).transpose(0, 1) for x in (kk, vv))
        mask = torch.arange(length)[None] <= (length - (b - a) + torch.arange(b - a))[:, None]
        want = torch.nn.functional.scaled_dot_product_attention(torch.from_numpy(q[a:b]).transpose(0, 1), kt, vt, attn_mask=mask, scale=0.125)
        np.testing.assert_allclose(out[a:b], want.transpose(0, 1).numpy(), rtol=1e-10, atol=1e-12)


# ---- the binding ----


def _rope(n=2, rows=3, h=2, kv=1, dim=64, dtype=torch.float32):
    z = lambda *s: [torch.zeros(*s, dtype=dtype) for _ in range(n)]  # noqa: E731
    w = torch.zeros(dim, dtype=dtype)
    return [z(rows, h, dim), z(rows, kv, dim), w, w, torch.zeros(rows, dtype=torch.int64), torch.zeros(16)]


def test_rope_refuses_shapes_and_types():
    good = _rope()

    def bad(i, value, error, match, **more):
        args = list(good)
        args[i] = value
        with pytest.raises(error, match=match):
            ar.qk_norm_rope(*args, **more)

    bad(0, [torch.zeros(3, 2, 64), torch.zeros(3, 3, 64)], ValueError, "q\\[1\\] has shape")
    bad(0, [torch.zeros(3, 128)] * 2, ValueError, "q must be \\[rows, heads")
    bad(1, good[1][:1], ValueError, "k holds 1 rank buffers")
    bad(1, [torch.zeros(4, 1, 64)] * 2, ValueError, "k\\[0\\] has shape \\(4, 1, 64\\)")
    bad(1, [t.bfloat16() for t in good[1]], TypeError, "k\\[0\\] is torch.bfloat16")
    bad(1, None, ValueError, "together")
    bad(2, torch.zeros(32), ValueError, "q_weight must be a contiguous vector of 64")
    bad(4, torch.zeros(3, dtype=torch.int32), TypeError, "pos is torch.int32")
    bad(4, None, ValueError, "freq needs pos")
    bad(5, torch.zeros(16, dtype=F64), TypeError, "freq is torch.float64")
    bad(0, [torch.zeros(3, 64, 2).transpose(1, 2)] * 2, ValueError, "side by side")
    bad(0, [torch.zeros(3, 2, 64), torch.zeros(3, 4, 64)[:, :2]], ValueError, "strides of q\\[0\\]")
    bad(0, good[0], ValueError, "k_out\\[0\\] has shape", k_out=good[0])
    bad(0, good[0], ValueError, "device tensors")
    with pytest.raises(ValueError, match="1 to 8 ranks"):
        ar.qk_norm_rope([], [], *good[2:])
    with pytest.raises(TypeError, match="unsupported tensor dtype"):
        ar.qk_norm_rope(*_rope(dtype=torch.float16))
    with pytest.raises(ValueError, match="dq_out\\[0\\] has shape"):
        ar.qk_norm_rope_backward(good[1], good[1], *good)
    with pytest.raises(ValueError, match="dk_weight\\[0\\] has shape"):
        ar.qk_norm_rope_backward(good[0], good[1], *good, dk_weight=[torch.zeros(3)] * 2)
    with pytest.raises(ValueError, match="need k"):
        ar.qk_norm_rope_backward(good[0], good[1], good[0], None, good[2], None, *good[4:])
    with pytest.raises(ValueError, match="device tensors"):
        ar.qk_norm_rope_backward(good[0], good[1], *good)


def _cache(n=2, pages=4, kv=1, page=16, dim=64):
    z = lambda *s: [torch.zeros(*s, dtype=torch.uint8) for _ in range(n)]  # noqa: E731
    return ar.KVCache(z(pages, kv, page, dim), z(pages, kv, dim, page), z(pages, kv), z(pages, kv))


def _ints(*v):
    return torch.tensor(v, dtype=torch.int32)


def test_cache_refuses_shapes_and_types():
    z = torch.zeros(4, 1, 16, 64, dtype=torch.uint8)
    with pytest.raises(ValueError, match="v\\[0\\] has shape"):
        ar.KVCache([z], [z], [z[..., 0, 0].contiguous()], [z[..., 0, 0].contiguous()])
    with pytest.raises(TypeError, match="k\\[0\\] is torch.int8"):
        ar.KVCache([z.view(torch.int8)], [z], [z], [z])
    c = _cache()
    k = [torch.zeros(3, 1, 64)] * 2
    table, first, at = torch.zeros(2, 2, dtype=torch.int32), _ints(0, 1, 3), _ints(0, 0)

    def write(cache=c, k=k, v=k, table=table, first=first, at=at):
        ar.cache_write(cache, k, v, table, first, at)

    for error, match, kw in (
            (ValueError, "k holds 1 rank buffers; the cache has 2", dict(k=k[:1])),
            (ValueError, "v\\[0\\] has shape", dict(v=[torch.zeros(4, 1, 64)] * 2)),
            (ValueError, "k\\[0\\] has shape", dict(k=[torch.zeros(3, 2, 64)] * 2)),
            (TypeError, "table is torch.int64", dict(table=table.long())),
            (TypeError, "first is torch.int64", dict(first=first.long())),
            (ValueError, "table must be an int32 tensor of 2", dict(table=table[0])),
            (ValueError, "first has 3 entries and start 2; got 2 and 2", dict(first=first[:2])),
            (ValueError, "start must be an int32 tensor of 1", dict(at=table)),
            (ValueError, "overlap", dict(table=table[:1].expand(2, 2))),
            (ValueError, "device tensors", dict())):
        with pytest.raises(error, match=match):
            write(**kw)
    with pytest.raises(ValueError, match="k\\[0\\] must be a contiguous"):
        ar.cache_read(c, table, first, at, [torch.zeros(3, 2, 64)[:, :1]] * 2, k)
    q = [torch.zeros(3, 2, 64)] * 2
    for error, match, kw in (
            (ValueError, "heads must be a multiple of the cache's 2", dict(cache=_cache(kv=2), q=[torch.zeros(3, 3, 64)] * 2)),
            (ValueError, "q\\[0\\] has shape", dict(q=[torch.zeros(3, 2, 128)] * 2)),
            (ValueError, "window needs causal", dict(window=4, causal=False)),
            (ValueError, "not be negative", dict(window=-1)),
            (ValueError, "not be negative", dict(max_rows=-1)),
            (TypeError, "lse\\[0\\] is torch.bfloat16", dict(lse=[torch.zeros(3, 2, dtype=torch.bfloat16)] * 2)),
            (ValueError, "length 2", dict(length=_ints(1))),
            (ValueError, "device tensors", dict())):
        args = dict(q=q, cache=c, table=table, first=first, length=at)
        args.update(kw)
        with pytest.raises(error, match=match):
            ar.cache_attention(**args)


def test_compiled_checks_agree_with_pythons():
    """The checks in C++ pass what those in Python pass, with the same addresses
    and strides, and leave to Python whatever they do not pass."""
    m = binding._MARSHAL
    if m is None:
        pytest.skip("built with the library")
    wide = [torch.zeros(3, 7, 64) for _ in range(2)]
    views = [t[:, 1:3] for t in wide]
    addresses = lambda ts: b"".join(t.data_ptr().to_bytes(8, "little") for t in ts)  # noqa: E731
    f32, i32 = torch.float32, torch.int32
    assert m.rows(views, f32, -1, 3, 2, 64) == (addresses(views), 7 * 64)
    assert m.rows([t[:1] for t in views], f32, -1, 1, 2, 64) == (addresses(views), 2 * 64)
    assert m.contiguous(wide, f32, -1, (3, 7, 64)) == addresses(wide)
    assert m.contiguous(tuple(wide), f32, -1, wide[0].shape) == addresses(wide)
    vec = torch.arange(5)
    assert m.vector(vec, torch.int64, -1, 5) == vec.data_ptr()
    table, first, at = torch.zeros(2, 9, dtype=i32)[:, :4], _ints(0, 1, 2), _ints(5, 6)
    assert m.sequences(table, first, at, -1) == (table.data_ptr(), first.data_ptr(), at.data_ptr(), 9, 4, 2)
    for refused in (m.rows(views, torch.bfloat16, -1, 3, 2, 64), m.rows(views, f32, 0, 3, 2, 64), m.rows(views, f32, -1, 4, 2, 64),
                    m.rows([views[0], views[1].contiguous()], f32, -1, 3, 2, 64), m.rows([], f32, -1, 3, 2, 64),
                    m.rows(views * 5, f32, -1, 3, 2, 64), m.rows([t.transpose(1, 2) for t in wide], f32, -1, 3, 64, 7),
                    m.rows([None, 3], f32, -1, 3, 2, 64), m.rows(views, "f32", -1, 3, 2, 64), m.rows(iter(views), f32, -1, 3, 2, 64),
                    m.contiguous(views, f32, -1, (3, 2, 64)), m.contiguous(wide, f32, -1, (3, 7)), m.contiguous(wide, f32, -1, 3),
                    m.vector(vec[::2], torch.int64, -1, 3),
                    m.vector(vec, torch.int64, -1, 4), m.vector(vec.to_sparse(), torch.int64, -1, 5), m.vector(None, f32, -1, 5),
                    m.sequences(table.long(), first, at, -1), m.sequences(table, first[:2], at, -1), m.sequences(table, first, table, -1),
                    m.sequences(table[:1].expand(2, 4), first, at, -1), m.sequences(table.t(), first, at, -1)):
        assert refused is None
    meta = [t.to("meta") for t in wide]  # no device and no address: Python passes them on too
    assert m.contiguous(meta, f32, -1, (3, 7, 64)) == bytes(binding._layer_list(meta, 2, (3, 7, 64), f32, -1, "x"))
    with pytest.raises((TypeError, OverflowError)):
        m.rows(views, f32, -1, "3", 2, 64)


# ---- the C ABI (argument errors come before any HIP call) ----

P8 = ctypes.c_void_p * 8
LIB = binding.library()


def _ptrs(k, step=1 << 36):
    return P8(*[(k << 40) + i * step for i in range(8)])


def _need_no_gpu():
    if torch.cuda.device_count() > 0:
        pytest.skip("needs a host without a GPU: the fake pointers below must never reach a kernel")


def test_c_abi_rope_argument_errors():
    _need_no_gpu()

    def fwd(n=2, q=None, qs=512, k=None, ks=256, w=9 << 40, pos=10 << 40, freq=11 << 40, qo=None, ko=None, rows=4, h=4, kv=2,
            dim=128, rot=64, pairs=0, dt=1):
        return LIB.ar_qk_norm_rope(n, q or _ptrs(1), qs, k or _ptrs(2), ks, ctypes.c_void_p(w), ctypes.c_void_p(w + 4096),
                                   ctypes.c_void_p(pos), ctypes.c_void_p(freq), qo or _ptrs(3), ko or _ptrs(4), rows, h, kv,
                                   dim, rot, pairs, 1e-6, dt, None)

    assert fwd() == 5                                              # every check passed: the first HIP call fails
    assert fwd(rows=0) == 0
    assert fwd(n=0) == 1 and fwd(n=9) == 1 and fwd(dt=3) == 1 and fwd(pairs=2) == 1 and fwd(h=0) == 1
    assert fwd(dt=2) == 2 and fwd(dim=96) == 2 and fwd(dim=512) == 2
    assert fwd(rot=8) == 1 and fwd(rot=144) == 1 and fwd(rot=0, pos=0, freq=0) == 5
    assert fwd(rows=1 << 29) == 4 and fwd(h=1025) == 4
    assert fwd(qs=511) == 1 and fwd(qs=516) == 1 and fwd(qs=768) == 5 and fwd(qs=1 << 31) == 1   # too short, not whole chunks
    assert fwd(w=0) == 1 and fwd(w=(9 << 40) + 8) == 1 and fwd(pos=0) == 1 and fwd(pos=(10 << 40) + 4) == 1
    assert fwd(qo=_ptrs(1)) == 1 and fwd(ko=_ptrs(3)) == 1         # outputs over an input, over each other
    assert fwd(kv=0, k=P8(), ko=P8()) == 5
    # queries and keys in one matrix
    assert fwd(qs=1024, ks=1024, k=P8(*[(1 << 40) + (i << 36) + 1024 for i in range(8)])) == 5

    def bwd(dq=None, dqs=512, dk=None, dks=256, ws=30 << 40, ws_bytes=1 << 30, rows=4):
        return LIB.ar_qk_norm_rope_backward(2, _ptrs(5), _ptrs(6), _ptrs(1), 512, _ptrs(2), 256, ctypes.c_void_p(9 << 40),
                                            ctypes.c_void_p(10 << 40), ctypes.c_void_p(11 << 40), ctypes.c_void_p(12 << 40),
                                            dq or _ptrs(7), dqs, dk or _ptrs(8), dks, _ptrs(13), _ptrs(14), rows, 4, 2, 128, 64, 0,
                                            1e-6, 1, ctypes.c_void_p(ws), ws_bytes, None)

    assert bwd() == 5 and bwd(ws=0) == 1
    need = LIB.ar_qk_norm_rope_workspace(2, 4, 4, 2, 128)
    assert need > 0 and bwd(ws_bytes=need - 1) == 4
    # gradients as columns of one matrix, side by side; overlapping by one chunk; of two pitches
    beside = lambda off: P8(*[(7 << 40) + (i << 36) + off for i in range(8)])  # noqa: E731
    assert bwd(dqs=768, dks=768, dk=beside(1024)) == 5
    assert bwd(dqs=768, dks=768, dk=beside(1008)) == 1
    assert bwd(dqs=768, dks=768, dk=beside(1536 + 1024)) == 5     # a row further down
    assert bwd(dqs=768, dks=768, dk=beside(1040)) == 1            # runs into the next row's queries
    assert bwd(dqs=768, dks=1024, dk=beside(1024)) == 1
    assert bwd(dq=_ptrs(1)) == 1


def _record(**kw):
    v = dict(k=_ptrs(1), v=_ptrs(2), ks=_ptrs(3), vs=_ptrs(4), pages=100, page=16, kv=2, dim=64, n=2)
    v.update(kw)
    return binding.CacheRecord(*[ctypes.cast(v[x], ctypes.c_void_p) for x in ("k", "v", "ks", "vs")], v["pages"], v["page"],
                               v["kv"], v["dim"], v["n"])


def _paged(**kw):
    v = dict(table=20 << 40, first=21 << 40, at=22 << 40, stride=8, width=8, seqs=3, rows=10)
    v.update(kw)
    return binding.PagedRows(*[v[x] for x in ("table", "first", "at", "stride", "width", "seqs", "rows")])


def test_c_abi_cache_argument_errors():
    _need_no_gpu()

    def write(cache=None, k=None, ks=128, v=None, vs=128, rows=None, dt=1):
        return LIB.ar_cache_write(cache or _record(), k or _ptrs(5), ks, v or _ptrs(6), vs, rows or _paged(), dt, None)

    assert write() == 5 and write(rows=_paged(rows=0)) == 0 and write(rows=_paged(seqs=0)) == 0
    assert write(cache=_record(n=0)) == 1 and write(cache=_record(n=9)) == 1 and write(cache=_record(kv=0)) == 1
    assert write(cache=_record(page=48)) == 2 and write(cache=_record(page=256)) == 2 and write(cache=_record(dim=80)) == 2
    assert write(cache=_record(pages=1 << 31)) == 4 and write(cache=_record(kv=1025), ks=1025 * 64, vs=1025 * 64) == 4
    assert write(dt=2) == 2 and write(dt=3) == 1
    assert write(ks=127) == 1 and write(ks=132) == 1 and write(vs=192) == 5
    assert write(k=_ptrs(1)) == 1                                  # new keys over the cache
    assert write(cache=_record(v=_ptrs(1))) == 1                   # keys over values
    assert write(rows=_paged(table=0)) == 1 and write(rows=_paged(first=2)) == 1 and write(rows=_paged(stride=7)) == 1
    assert write(rows=_paged(width=1 << 27)) == 4 and write(rows=_paged(seqs=(1 << 20) + 1)) == 4
    assert write(rows=_paged(table=0, width=0)) == 5               # no pages at all: nothing to read
    assert LIB.ar_cache_read(_record(), _ptrs(5), _ptrs(6), _paged(), 0, None) == 5
    assert LIB.ar_cache_read(_record(), _ptrs(5), _ptrs(5), _paged(), 0, None) == 1
    assert LIB.ar_cache_read(None, _ptrs(5), _ptrs(6), _paged(), 0, None) == 1


def test_c_abi_attention_argument_errors():
    _need_no_gpu()

    def att(cache=None, q=None, qs=256, rows=None, out=None, lse=None, h=4, scale=0.125, causal=1, window=0, most=0, dt=1, ws=30 << 40,
            nbytes=1 << 40):
        return LIB.ar_cache_attention(cache or _record(), q or _ptrs(5), qs, rows or _paged(), out or _ptrs(6), lse, h, scale, causal,
                                      window, most, dt, ctypes.c_void_p(ws), nbytes, None)

    assert att() == 5 and att(lse=_ptrs(7)) == 5 and att(rows=_paged(rows=0)) == 0
    assert att(h=3) == 1 and att(h=0) == 1 and att(h=1026) == 4 and att(qs=255) == 1
    assert att(scale=float("inf")) == 1 and att(scale=float("nan")) == 1 and att(scale=-1.0) == 5 and att(scale=0.0) == 5
    assert att(causal=2) == 1 and att(causal=0, window=5) == 1 and att(window=5) == 5
    assert att(out=_ptrs(5)) == 1 and att(out=_ptrs(1)) == 1 and att(lse=_ptrs(6)) == 1
    long = _paged(width=4096, stride=4096)
    need = LIB.ar_cache_attention_workspace(_record(), 3, 10, 4096, 4, 0, 0, 1)
    assert need > 0 and att(rows=long, nbytes=need - 1) == 4 and att(rows=long, nbytes=need) == 5 and att(rows=long, ws=0) == 1
    assert LIB.ar_cache_attention_workspace(_record(), 3, 10, 8, 4, 0, 0, 1) == 0   # short: not shared
    assert att(ws=0, nbytes=0) == 5
    assert LIB.ar_cache_attention_workspace(_record(dim=80), 3, 10, 4096, 4, 0, 0, 1) == 0

"""Limits of the attention operators that the host checks (no GPU)."""

import ctypes
import os
import subprocess

from test_heads_host import LIB, _need_no_gpu, _paged, _ptrs, _record

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_work_items_fit_a_launch(tmp_path):
    """Compiles tests/fold_check.hip against the kernels' header: no launch has 2^32
    threads along x, and its layers hold every item."""
    exe = str(tmp_path / "fold_check")
    res = subprocess.run(["hipcc", "--offload-arch=gfx950", "-O2", "-std=c++17", os.path.join(ROOT, "tests", "fold_check.hip"), "-o", exe],
                         capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout


def test_attention_numbers_its_tiles_in_32_bits():
    _need_no_gpu()

    def att(seqs, kv, n):
        cache, heads = _record(kv=kv, n=n, pages=1), kv
        need = LIB.ar_cache_attention_workspace(cache, seqs, 10, 4, heads, 0, 0, 1)
        st = LIB.ar_cache_attention(cache, _ptrs(5), heads * 64, _paged(seqs=seqs, width=4), _ptrs(6), None, heads, 0.125, 1, 0, 0, 1,
                                    ctypes.c_void_p(30 << 40), need, None)
        return st

    assert att(1 << 20, 256, 8) == 5 and att(1 << 20, 1024, 2) == 5   # 2^31 tiles: the first HIP call fails
    assert att(1 << 20, 257, 8) == 4 and att(1 << 20, 1024, 3) == 4

"""The joining of partial softmax statistics (CPU only: a host build of the
kernels' own merge_stats) against fp64: sets far from 0, empty sets, infinities
and NaN, in every order of three."""

import itertools
import os
import subprocess

import numpy as np
import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
E = 2.0 ** -24


@pytest.fixture(scope="module")
def join(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("stats") / "check")
    res = subprocess.run(["hipcc", "--offload-arch=gfx950", "-O3", "-std=c++17",
                          os.path.join(ROOT, "tests", "merge_stats_check.hip"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

    def run(sets):
        text = "\n".join(f"{len(s)} " + " ".join(f"{x:.9g} {y:.9g}" for x, y in s) for s in sets)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        return [tuple(map(float, line.split())) for line in out.stdout.splitlines()]

    return run


EMPTY = (-np.inf, 0.0)
# what a tile hands on: its maximum, and a sum of 1 to 256 exponentials up to 1
TILES = [(np.float32(top), np.float32(total)) for top, total in
         [(-1e4, 1.0), (-200.5, 31.25), (-150.0, 1.0), (-88.75, 7.5), (-60.0, 256.0), (0.0, 2.0), (3.25, 17.0), (90.5, 1.0),
          (200.0, 90.0), (1e4, 3.0)]]


def _lse(sets):
    tops = np.array([float(t) for t, _ in sets])
    sums = np.array([float(s) for _, s in sets])
    top = tops.max()
    return top, float((sums * np.exp(tops - top)).sum())


@pytest.mark.parametrize("count", [1, 2, 3])
def test_sets_of_any_magnitude_and_empty_ones(join, count):
    sets = [s for s in itertools.product([EMPTY, *TILES], repeat=count) if any(x != EMPTY for x in s)]
    for s, (top, total) in zip(sets, join(sets)):
        want_top, want = _lse(s)
        assert top == want_top, s
        # a join rounds each side's exponential (argument exact to E |distance|,
        # result 2 E), its product and the sum: 6 E and E |distance|, at most
        # 2e4 from the maximum, where it weighs nothing; within 104 of it E 104
        assert abs(total - want) <= count * (6 + 104) * E * want, (s, total, want)


def test_empty_sets_alone_and_infinities(join):
    inf = np.inf
    assert join([(EMPTY, EMPTY)]) == [(-inf, 0.0)]
    for low in (EMPTY, (-1e4, 1.0), (-100.0, 2.0), (0.0, 1.0), (200.0, 5.0)):
        for s in ((low, (inf, inf)), ((inf, inf), low)):
            assert join([s]) == [(inf, inf)], s


def test_nan_is_kept(join):
    # a tile of NaN alone has the maximum of an empty one
    for bad in ((-np.inf, np.nan), (0.0, np.nan), (-200.0, np.nan), (np.inf, np.nan)):
        for other in (EMPTY, (-1e4, 1.0), (-100.0, 2.0), (0.0, 1.0), (200.0, 5.0), (np.inf, np.inf)):
            for s in ((bad, other), (other, bad)):
                assert np.isnan(join([s])[0][1]), s

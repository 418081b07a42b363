"""The product kernels' tile classes (CPU only: a host build of the rule, and the
kernels' assembly): the GPU tests' shapes reach every class of every kernel, the
rule's choices at the two ends, and no kernel spills registers."""

import os
import re
import subprocess

import pytest

from all_reduce_reduction_rank_amd import vocab_shards
from tests.test_gpu_layer import (FFN_CLASS_SHAPES, FFN_SHAPES, FFN_SHARED_CLASSES, FFN_SHARED_SHAPES, XENT_SHAPES,
                                  XENT_SHARED_CLASSES, XENT_SHARED_SHAPES)

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "all_reduce_reduction_rank_amd", "csrc")
FLAGS = ["--offload-arch=gfx950", "-O3", "-std=c++17", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
KINDS = ("gated", "store", "stats", "dlogits", "gated_bwd", "grads")
CLASSES = ("large", "small", "tall", "flat", "split", "thin")
ONLY = {"large": "bf16", "flat": "bf16", "tall": "f32"}
DT = {"f32": 0, "bf16": 1}
GRAD_TN = 1


@pytest.fixture(scope="module")
def classes(tmp_path_factory):
    exe = str(tmp_path_factory.mktemp("tiles") / "check")
    res = subprocess.run(["hipcc", *FLAGS, os.path.join(ROOT, "tests", "product_tile_check.hip"),
                          os.path.join(CSRC, "products.hip"), "-o", exe], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr

    def choose(plans):
        text = "\n".join(f"{KINDS.index(kind)} {DT[dt]} {head} {_may_share(kind, head, probs):d} {parts} {len(probs)} " +
                         " ".join(" ".join(map(str, p)) for p in probs) for (kind, dt, head, probs), parts in plans)
        out = subprocess.run([exe], input=text, capture_output=True, text=True, timeout=60)
        assert out.returncode == 0
        got = [line.split() for line in out.stdout.splitlines()]
        return [(CLASSES[int(tile)], int(shares)) for tile, shares in got]

    def run(plans, shares=False):
        """The classes (and shares) of a list of plans; a dlogits plan follows
        its stats plan and adds up K in the same order."""
        got = choose([(p, 0) for p in plans])
        for i, p in enumerate(plans):
            if p[0] == "dlogits":
                got[i] = choose([(p, 4 if got[i - 1][0] in ("split", "thin") else 1)])[0]
        return got if shares else [tile for tile, _ in got]

    return run


def _may_share(kind, head, probs):
    """Results of the first launch's problems small enough for shares of K."""
    first = probs[:head] if head else probs
    if not (kind == "store" or kind == "grads" and first[0][5] != GRAD_TN):
        return False
    return sum((m - fold) * n for m, n, _, _, fold, _ in first) <= 128 * 64 * 128


def _fold(rows, dt):
    return 0 if dt == "f32" or rows == 0 or rows > 32 else 8 if rows <= 8 else 32


def _split(dt, fold, n, dx, dw):
    """The gradients' launches: one, or two where dx has second terms."""
    return [("grads", dt, 0, dx), ("grads", dt, 0, dw)] if fold else [("grads", dt, n, dx + dw)]


def ffn_plans(n, rows, hidden, inter, dt):
    f = _fold(rows, dt)
    two = 2 if f else 1
    dw = [(inter, hidden, rows, two, 0, GRAD_TN)] * 2 + [(hidden, inter, rows, two, 0, GRAD_TN)]
    return [("gated", dt, 0, [(rows, inter, hidden, 1, f, 0)] * n),
            ("store", dt, 0, [(f + rows, hidden, inter, 1, f, 0)] * n),
            ("gated_bwd", dt, 0, [(rows, inter, hidden, 1, f, 0)] * n),
            *_split(dt, f, n, [(f + rows, hidden, inter, 2, f, 0)] * n, dw * n)]


def xent_plans(n, rows, hidden, vocab, dt):
    f = _fold(rows, dt)
    two = 2 if f else 1
    shards = vocab_shards(vocab, n)
    some = [v for v in shards if v]
    return [("stats", dt, 0, [(rows, v, hidden, 1, 0, 0) for v in some]),
            ("dlogits", dt, 0, [(rows, v, hidden, 1, f, 0) for v in some]),
            *_split(dt, f, n, [(f + rows, hidden, v, 1, f, 0) for v in shards],
                    [(v, hidden, rows, two, 0, GRAD_TN) for v in some])]


def test_gpu_tests_reach_every_class_of_every_kernel(classes):
    plans = []
    for dt in ("bf16", "f32"):
        for rows, hidden, inter in FFN_SHAPES:
            plans += ffn_plans(2, rows, hidden, inter, dt)
        for n, rows, hidden, inter in [*FFN_CLASS_SHAPES, (8, 1288, 1160, 1416)]:
            plans += ffn_plans(n, rows, hidden, inter, dt)
        for n, rows, hidden, vocab in XENT_SHAPES:
            plans += xent_plans(n, rows, hidden, vocab, dt)
        plans += xent_plans(2, 1030, 72, 20011 if dt == "bf16" else 16400, dt)
    seen = {(p[0], p[1], c) for p, c in zip(plans, classes(plans))}
    missing = {(k, dt, c) for k in KINDS for dt in DT for c in CLASSES if ONLY.get(c, dt) == dt} - seen
    assert not missing, sorted(missing)


def test_gpu_tests_share_sums(classes):
    for dt in ("bf16", "f32"):
        for shape in FFN_SHARED_SHAPES:
            got = classes(ffn_plans(*shape, dt), shares=True)
            assert got[1][1] > 1 and got[3][1] > 1, (dt, shape, got)
            assert all(n == 1 for i, (_, n) in enumerate(got) if i not in (1, 3)), (dt, shape, got)
        for shape in XENT_SHARED_SHAPES:
            got = classes(xent_plans(*shape, dt), shares=True)
            assert got[2][1] > 1 and all(n == 1 for i, (_, n) in enumerate(got) if i != 2), (dt, shape, got)


def test_gpu_tests_share_sums_in_every_class(classes):
    seen = set()
    for dt in ("bf16", "f32"):
        for shape in [*FFN_SHARED_SHAPES, *FFN_SHARED_CLASSES]:
            got = classes(ffn_plans(*shape, dt), shares=True)
            seen |= {(kind, dt, got[i][0]) for kind, i in (("store", 1), ("grads", 3)) if got[i][1] > 1}
        for shape in [*XENT_SHARED_SHAPES, *XENT_SHARED_CLASSES]:
            got = classes(xent_plans(*shape, dt), shares=True)
            seen |= {("grads", dt, got[2][0])} if got[2][1] > 1 else set()
    want = {(kind, "bf16", c) for kind in ("store", "grads") for c in ("large", "small", "split", "thin")}
    want |= {("grads", "bf16", "flat"), ("grads", "f32", "small")}
    want |= {(kind, "f32", c) for kind in ("store", "grads") for c in ("tall", "split")} | {("store", "f32", "thin")}
    assert not want - seen, sorted(want - seen)


def test_recomputed_logits_are_summed_in_the_order_of_the_forward_pass(classes):
    def order(tile):
        return tile in ("split", "thin")

    for dt in ("bf16", "f32"):
        for shape in [*XENT_SHAPES, *XENT_SHARED_SHAPES]:
            got = classes(xent_plans(*shape, dt))
            assert order(got[0]) == order(got[1]), (dt, shape, got)


def test_choices_at_both_ends(classes):
    one = ffn_plans(8, 1, 5120, 1728, "bf16")
    assert classes(one[:2]) == ["thin", "thin"]
    step = ffn_plans(8, 8192, 5120, 1728, "bf16")
    assert classes(step) == ["large"] * 4
    # second terms fix the reader's tile: both terms of every row in one tile
    for rows, want in ((1, {"thin"}), (8, {"thin"}), (9, {"flat", "split"}), (32, {"flat", "split"})):
        got = classes([p for p in ffn_plans(4, rows, 2048, 1408, "bf16") if p[0] == "store" or p[3][0][4]])
        assert got[1] in want, (rows, got)
    # nor may the large tile write them
    assert "large" not in classes(ffn_plans(8, 32, 8192, 8192, "bf16")[:4])


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_kernel_uses_scratch_memory(tmp_path, dt):
    out = str(tmp_path / "k.s")
    res = subprocess.run(["hipcc", *FLAGS, "-S", "--cuda-device-only", "-o", out,
                          os.path.join(CSRC, f"products_{dt}.hip")], capture_output=True, text=True)
    assert res.returncode == 0, res.stderr
    text = open(out).read()
    kernels = re.findall(r"^(_ZN2ar\S*product_kernel\S*):", text, re.M)
    # 4 kinds + 2 gated kinds x 3 activations, in every class of the type
    assert len(kernels) == (4 + 2 * 3) * (5 if dt == "bf16" else 4)
    spills = re.findall(r"\.vgpr_spill_count:\s+(\d+)", text)
    assert spills and all(int(x) == 0 for x in spills)
    assert all(int(x) == 0 for x in re.findall(r"\.private_segment_fixed_size:\s+(\d+)", text))

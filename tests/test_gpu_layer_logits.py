"""GPU: the linear cross entropy where its logits are far from 0 or far apart,
in every tile class, with tiles that end in a single column and ranks with few
tiles or none, against the fp64 definition."""

import pytest
import torch

import all_reduce_reduction_rank_amd as ar
from tests.test_gpu_layer import XENT_SHAPES, run_xent, xent_inputs

pytestmark = pytest.mark.gpu


def moved(inputs, by):
    """The same logits plus `by`[v] (one value, or one per vocabulary row) in
    every row: one column of x at 1, and that column of w."""
    x, w, target, grad = inputs
    first = 0
    for t in w:
        t[:, 0] = by if isinstance(by, float) else by[first:first + len(t)].to(t)
        first += len(t)
    for t in x:
        t[:, 0] = 1.0
    return x, w, target, grad


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,vocab", XENT_SHAPES)  # every tile class
def test_all_logits_near_minus_200(n, rows, hidden, vocab, dt):
    run_xent(n, rows, hidden, vocab, dt, inputs=moved(xent_inputs(n, rows, hidden, vocab, dt, 7), -200.0))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("by", [-10000.0, -150.0, -90.0, 90.0, 200.0])
@pytest.mark.parametrize("n,rows,hidden,vocab", [(2, 5, 64, 300), (8, 5, 64, 3), (3, 130, 40, 2050), (1, 300, 33, 129)])
def test_a_constant_moves_the_logits(n, rows, hidden, vocab, by, dt):
    run_xent(n, rows, hidden, vocab, dt, inputs=moved(xent_inputs(n, rows, hidden, vocab, dt, 8), by))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_large_tiles_near_minus_200(dt):
    vocab = 20011 if dt == "bf16" else 16400
    run_xent(2, 1030, 72, vocab, dt, inputs=moved(xent_inputs(2, 1030, 72, vocab, dt, 9), -200.0))


# rows that take the Thin, Split or Flat, and larger tiles; each rank's last
# tile holds one column at any width of a tile
@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,vocab", [(1, 3, 257), (2, 20, 514), (3, 150, 2307), (1, 1030, 16385)])
def test_a_last_tile_of_one_far_column(n, rows, vocab, dt):
    by = torch.zeros(vocab)
    end = 0
    for v in ar.vocab_shards(vocab, n):
        assert v % 256 == 1
        end += v
        by[end - 1] = -150.0
    run_xent(n, rows, 72, vocab, dt, inputs=moved(xent_inputs(n, rows, 72, vocab, dt, 10), by))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,vocab", [(1, 3, 700), (3, 40, 2000), (8, 300, 4099), (1, 1030, 16384)])
def test_parts_of_the_vocabulary_far_below_the_rest(n, rows, vocab, dt):
    by = torch.full((vocab,), -300.0)
    by[vocab // 2:] = 0.0
    by[-5:] = -120.0
    run_xent(n, rows, 64, vocab, dt, inputs=moved(xent_inputs(n, rows, 64, vocab, dt, 11), by))


@pytest.mark.parametrize("dt", ["bf16", "f32"])
@pytest.mark.parametrize("n,rows,hidden,vocab", [(1, 3, 64, 500), (2, 20, 64, 900), (4, 130, 40, 2050), (1, 300, 32, 129)])
def test_logits_far_apart(n, rows, hidden, vocab, dt):
    x, w, target, grad = xent_inputs(n, rows, hidden, vocab, dt, 12)
    run_xent(n, rows, hidden, vocab, dt, inputs=(x, [t * 50 for t in w], target, grad))  # a standard deviation of 100

"""The loss's forward workspace holds the partial statistics of the narrowest
tiles its rows may take, and no more (CPU only)."""

import pytest

from all_reduce_reduction_rank_amd import binding
from tests.test_product_tiles import classes, xent_plans  # noqa: F401 (classes: a fixture)

COLS = {"large": 256, "small": 128, "tall": 64, "flat": 128, "split": 64, "thin": 32}
THIN_ROWS = 64  # rows up to which a product may take Thin tiles


def align(x):
    return (x + 255) // 256 * 256


def narrowest(rows):
    return 32 if rows <= THIN_ROWS else 64


@pytest.mark.parametrize("dt", [0, 1])
@pytest.mark.parametrize("n,rows,vocab", [(1, 1, 131072), (4, 48, 32000), (2, 64, 1000), (2, 65, 1000), (8, 4096, 131072),
                                          (1, 8192, 131072), (3, 65536, 100003)])
def test_partials_of_the_narrowest_tile(n, rows, vocab, dt):
    shard = -(-vocab // n)
    tiles = -(-shard // narrowest(rows))
    # the targets' logits, then (max, sum) per rank, tile and row; no copies at this width
    want = align(rows * 4) + n * align(tiles * rows * 8)
    assert binding.library().ar_linear_cross_entropy_workspace(n, rows, 1024, vocab, dt, 0, 0) == want


@pytest.mark.parametrize("dt", ["bf16", "f32"])
def test_no_choice_is_narrower(classes, dt):  # noqa: F811
    shapes = [(n, rows, hidden, vocab) for n in (1, 3, 8) for rows in (1, 16, 17, 64, 65, 66, 100, 500, 5000, 70000)
              for hidden in (8, 200, 5120) for vocab in (3, 300, 5000, 131072)]
    got = classes([xent_plans(*s, dt)[0] for s in shapes])
    for (n, rows, hidden, vocab), tile in zip(shapes, got):
        assert COLS[tile] >= narrowest(rows), (n, rows, hidden, vocab, tile)
    assert {"thin"} < set(got)


@pytest.mark.parametrize("n,rows,hidden,vocab", [(2, 100000, 16, 100000), (8, 400000, 8, 131072), (1, 5000, 1024, 700)])
def test_pieces_are_as_documented(n, rows, hidden, vocab):
    shard = -(-vocab // n)

    def d_bytes(piece):  # fp32: d, and the copy of x; dx is summed in place
        total = binding.library().ar_linear_cross_entropy_workspace(n, rows, hidden, vocab, 0, 1, piece)
        return total - n * align(rows * hidden * 4)

    def of(columns):
        return n * align(rows * min(columns, (shard + 7) // 8 * 8) * 4)

    for piece, columns in ((1, 256), (255, 256), (256, 256), (300, 256), (1023, 768), (1 << 40, 1 << 20)):
        assert d_bytes(piece) == of(columns), piece
    # chosen by the library: within 1 GiB, but no fewer than 256 columns
    assert d_bytes(0) == of(max(256, (1 << 30) // (n * rows * 4) // 256 * 256))
    assert d_bytes(0) <= max(1 << 30, of(256))

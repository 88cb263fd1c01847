"""Shared-prefix groups of more sequences than a row tile holds (128 / G),
whose members at the tiles' heads are empty, short, or padding: every tile's
prefix is the group's, wherever its own first sequence's table points.

Tolerances: tests/attention64.py.
"""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu

# dtype, Hq, Hkv, D, block size, sequences, prefix; sequences per row tile
SHAPES = [(("bf16", 32, 8, 128, 16), 64, 512, 32), (("f16", 14, 2, 64, 32), 40, 700, 18),
          (("bf16", 8, 1, 128, 64), 50, 300, 16)]


def _batch(shape, n, prefix, short, seed):
    return Batch(*shape, [(prefix, [1 + 7 * i % 90 for i in range(n)])], seed=seed, short=short)


@pytest.mark.parametrize("shape, n, prefix, tile", SHAPES, ids=str)
def test_an_ended_sequence_at_the_head_of_a_row_tile(shape, n, prefix, tile):
    t = _batch(shape, n, prefix, {tile: 0, 2 * tile: 0} if 2 * tile < n else {tile: 0}, seed=41)
    assert int(t.tables[tile].max()) == -1
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)


@pytest.mark.parametrize("shape, n, prefix, tile", SHAPES, ids=str)
def test_a_short_sequence_with_other_blocks_at_the_head_of_a_row_tile(shape, n, prefix, tile):
    bs = shape[4]
    t = _batch(shape, n, prefix, {tile: bs + 3}, seed=42)
    # its two blocks are the group's in another order, the rest of its row holds other sequences' blocks
    row = t.tables[tile].clone()
    row[:2] = row[[1, 0]]
    row[2:] = t.tables[n - 1].flip(0).clamp(min=0)[2:]
    t.tables[tile] = row
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)


@pytest.mark.parametrize("shape, n, prefix, tile", SHAPES, ids=str)
def test_padding_from_the_head_of_a_row_tile_on(shape, n, prefix, tile):
    """The batch's last rows are padding; nothing is recorded for them."""
    t = _batch(shape, n, prefix, {b: 0 for b in range(tile, n)}, seed=43)
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    check_batch(t)


def test_sequences_that_end_under_a_captured_graph():
    """A decode loop's graph: sequence by sequence of the group ends, the
    tiles' heads first, the group's first one last."""
    shape, n, prefix, tile = SHAPES[0]
    t = _batch(shape, n, prefix, {}, seed=44)
    ws = pk.shared_prefix_workspace(n, 32, 8, 128, 16, max(t.lens), torch.bfloat16, "cuda")
    t.run(workspace=ws)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        t.run(workspace=ws)
    pk.device_error()
    for b in (tile, tile + 1, 5, n - 1, 0):
        t.seq_lens[b] = 0
        t.tables[b] = -1
        t.lens[b] = 0
        g.replay()
        assert pk.device_error() == 0
        check_batch(t)

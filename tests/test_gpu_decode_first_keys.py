"""Plain decode attention over sequences whose first keys score -inf: they
weigh nothing, on the tensor-core kernels and on the SIMT kernel, whose warps
each take blocks from the sequence's first ones on.

Tolerances: tests/attention64.py.
"""

import pytest

import paged_kv_cache_128_gb300 as pk
from tests.attention64 import check_batch
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("first", [1, 16, 100])
@pytest.mark.parametrize("shape, bps", [(("f32", 8, 2, 128, 16), 0), (("f32", 6, 2, 64, 16), 4), (("f16", 8, 2, 80, 16), 0),
                                        (("bf16", 8, 2, 128, 16), 0), (("f16", 8, 2, 64, 32), 2)], ids=str)
def test_first_keys_that_weigh_nothing(shape, bps, first):
    t = Batch(*shape, [(0, [n]) for n in (900, 130, 101)], seed=121)
    t.q[..., 0] = t.q[..., 0].abs() + 0.5
    for b, L in enumerate(t.lens):
        for pos in range(min(first, L - 1)):
            t.kc[int(t.tables[b, pos // t.bs]), pos % t.bs, :, 0] = float("-inf")
    pk.device_error()
    pk.paged_decode_attention(t.out, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, max(t.lens), blocks_per_split=bps)
    assert pk.device_error() == 0
    check_batch(t)

"""The block manager's prefix groups, and the refusals of the shared-prefix
attention's entry points (host-side checks, no GPU needed)."""

import ctypes

import numpy as np
import pytest

import paged_kv_cache_128_gb300 as pk


def _groups(m, ids):
    start, prefix = m.prefix_groups(ids)
    return start.tolist(), prefix.tolist()


def test_forked_children_share_whole_blocks():
    m = pk.KVBlockManager(64, 4)
    m.allocate_for_prefill(0, 10)          # blocks of 4, 4 and 2 tokens
    m.fork(0, 1, 10)
    m.fork(0, 2, 7)                        # shares 2 blocks, the second one partly filled for it
    assert _groups(m, [0, 1]) == ([0, 2], [8])
    # 2 joins: one block read by three saves two reads, as two blocks read by two do
    assert _groups(m, [0, 1, 2]) == ([0, 3], [4])
    m.fork(0, 3, 10)
    assert _groups(m, [0, 1, 3, 2]) == ([0, 3, 4], [8, 0])  # two blocks by three save four, one by four three
    m.free_sequence(3)
    m.append_slots(2, 1)                   # writes into the shared block: copied, so only block 0 is common
    assert _groups(m, [2, 0, 1]) == ([0, 3], [4])           # 1 * 2 >= 1 * 1
    assert _groups(m, [0]) == ([0, 1], [0])
    assert _groups(m, []) == ([0], [])


def test_unrelated_neighbours_are_groups_of_one():
    m = pk.KVBlockManager(64, 4)
    for i in range(4):
        m.allocate_for_prefill(i, 9)
    assert _groups(m, [0, 1, 2, 3]) == ([0, 1, 2, 3, 4], [0, 0, 0, 0])
    m.fork(2, 7, 8)
    assert _groups(m, [0, 2, 7, 3]) == ([0, 1, 3, 4], [0, 8, 0])
    assert _groups(m, [2, 0, 7]) == ([0, 1, 2, 3], [0, 0, 0])  # neighbours only


def test_rule_against_a_plain_restatement():
    rng = np.random.default_rng(3)
    m = pk.KVBlockManager(4096, 4)
    m.allocate_for_prefill(0, 40)
    ids = [0]
    for i in range(1, 60):
        parent = int(rng.choice(ids))
        n = int(rng.integers(1, m.seq_len(parent) + 1))
        m.fork(parent, i, n)
        m.append_slots(i, int(rng.integers(1, 20)))
        ids.append(i)
    assert m.check_invariants()
    order = rng.permutation(ids).tolist()
    tables = {i: m.block_table(i).tolist()[:m.seq_len(i) // 4] for i in ids}

    def common(a, b):
        n = 0
        while n < min(len(a), len(b)) and a[n] == b[n]:
            n += 1
        return n

    start, prefix, i = [0], [], 0
    while i < len(order):
        shared, j = tables[order[i]], i + 1
        while j < len(order):
            q, n, p = common(shared, tables[order[j]]), j - i, len(shared)
            if q == 0 or q * n < p * (n - 1):
                break
            shared, j = shared[:q], j + 1
        prefix.append(4 * len(shared) if j - i > 1 else 0)
        start.append(j)
        i = j
    assert _groups(m, order) == (start, prefix)
    for g in range(len(prefix)):
        rows = {tuple(tables[x][:prefix[g] // 4]) for x in order[start[g]:start[g + 1]]}
        assert len(rows) == 1 or prefix[g] == 0


def test_unknown_and_bad_arguments():
    m = pk.KVBlockManager(8, 4)
    m.allocate_for_prefill(0, 4)
    with pytest.raises(pk.KVError) as e:
        m.prefix_groups([0, 5])
    assert e.value.code == "UNKNOWN_SEQ"
    fn, h = pk.lib().kvbm_prefix_groups, m._h
    ids = (ctypes.c_int64 * 1)(0)
    out = (ctypes.c_int32 * 2)()
    n = ctypes.c_int64()
    assert fn(h, ids, 1, out, out, ctypes.byref(n)) == 0
    for args in ((None, ids, 1, out, out), (h, None, 1, out, out), (h, ids, -1, out, out), (h, ids, 1, None, out),
                 (h, ids, 1, out, None)):
        assert fn(*args, ctypes.byref(n)) == 1
    assert fn(h, ids, 1, out, out, None) == 1


BUF = (ctypes.c_char * 4096)()
PTR = (ctypes.addressof(BUF) + 255) // 256 * 256


def _call(**over):
    a = dict(out=PTR, q=PTR, k_cache=PTR, v_cache=PTR, block_tables=PTR, seq_lens=PTR, group_start=PTR,
             prefix_lens=PTR, num_seqs=4, num_groups=2, num_heads=8, num_kv_heads=2, head_dim=128, block_size=16,
             num_blocks=8, max_blocks_per_seq=4, max_seq_len=64, scale=0.1, dtype=2, workspace=PTR,
             workspace_bytes=1 << 40, stream=None)
    assert set(over) <= set(a)
    a.update(over)
    return pk.lib().paged_decode_attention_shared_prefix(*a.values())


def test_an_empty_batch_passes():
    assert _call(num_seqs=0, num_groups=0) == 0


@pytest.mark.parametrize("bad", [
    dict(num_seqs=-1), dict(num_groups=-1), dict(num_groups=5), dict(num_heads=0), dict(num_heads=7),
    dict(num_kv_heads=0), dict(head_dim=0), dict(head_dim=260), dict(head_dim=60), dict(block_size=0),
    dict(num_blocks=0), dict(num_blocks=2 ** 31 - 1), dict(max_blocks_per_seq=0), dict(max_seq_len=-1),
    dict(scale=float("nan")), dict(scale=float("inf")), dict(dtype=5), dict(out=None), dict(q=None),
    dict(k_cache=None), dict(v_cache=None), dict(block_tables=None), dict(seq_lens=None), dict(group_start=None),
    dict(prefix_lens=None), dict(q=PTR + 2), dict(out=PTR + 8), dict(k_cache=PTR + 4), dict(workspace=PTR + 16),
], ids=str)
def test_bad_arguments_are_refused(bad):
    assert _call(**bad) == 1


def test_small_or_missing_workspaces_are_refused():
    n = ctypes.c_size_t()
    assert pk.lib().paged_shared_prefix_workspace_size(4, 8, 2, 128, 16, 64, 2, ctypes.byref(n)) == 0 and n.value > 0
    assert _call(workspace_bytes=n.value - 1) == 9
    assert _call(workspace=None) == 9
    assert pk.lib().paged_shared_prefix_workspace_size(4, 8, 2, 128, 16, 64, 2, None) == 1
    assert pk.lib().paged_shared_prefix_workspace_size(4, 7, 2, 128, 16, 64, 2, ctypes.byref(n)) == 1

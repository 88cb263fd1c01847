"""Decode attention over shared prefixes against float64 attention.

Every sequence's output is plain attention over its own whole table, whatever
the grouping; the float64 reference here reads each sequence's logical K and
V and knows nothing of groups.

Tolerance, from the arithmetic.  With weights p_j (summing to 1) and result o:
the probabilities are rounded to the type (relative u: 2^-8 bf16, 2^-11 fp16)
and the sum is taken over the rounded ones, so the result moves by at most
u sum_j p_j |V_j - o| / (1 - u); a score is off by at most
(D + 4) 2^-23 A with A = |scale| sum_d |q_d k_d| (float32 products and sums, each
addition allowed a whole step), plus 2^-22 |s| for the exponential, and moves
the result by at most 2 max_j(that) sum_j p_j |V_j|; the float32 sums of the
values themselves and the joining of the parts add (64 + 16) 2^-23 sum p |V|
(a tile's 64 products, then tiles and pieces, each rescaled: relative errors
of partial sums that are no larger than the whole of |p V|), for up to 1024
tiles 1100 2^-23; the output's own rounding is u |o|.
"""

import math

import numpy as np
import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from tests.helpers import TORCH, sentinel_tensor

pytestmark = pytest.mark.gpu

U = {"f16": 2.0 ** -11, "bf16": 2.0 ** -8, "f32": 2.0 ** -24}


class Batch:
    """groups: list of (prefix tokens, [rest lengths]); a sequence's length is
    the group's prefix in whole blocks plus its rest.  Sequences of a group
    hold the same blocks for that part; `short` overrides lengths."""

    def __init__(self, dtype, hq, hkv, d, bs, groups, seed, short=None, spread=1.0, declared=None):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.dtype, self.hq, self.hkv, self.d, self.bs = dtype, hq, hkv, d, bs
        dev = torch.device("cuda")
        tables, lens, start = [], [], [0]
        nxt = 0
        for prefix, rests in groups:
            whole = prefix // bs
            common = list(range(nxt, nxt + whole))
            nxt += whole
            for rest in rests:
                L = whole * bs + rest
                own = -(-L // bs) - whole
                tables.append(common + list(range(nxt, nxt + own)))
                nxt += own
                lens.append(L)
            start.append(start[-1] + len(rests))
        for b, L in (short or {}).items():
            lens[b] = L
            if L == 0:
                tables[b] = []
        self.lens = lens
        self.nb = nxt + 2
        place = rng.permutation(self.nb).astype(np.int32)
        self.cols = max([len(t) for t in tables] + [1]) + 2
        tab = np.full((len(lens), self.cols), -1, np.int32)
        for b, t in enumerate(tables):
            tab[b, :len(t)] = place[np.array(t, dtype=np.int64)] if t else []
        dt = TORCH[dtype]
        # every slot holds NaN but those a sequence owns
        self.kc = sentinel_tensor((self.nb, bs, hkv, d), dtype, dev)
        self.vc = sentinel_tensor((self.nb, bs, hkv, d), dtype, dev)
        used = torch.zeros(self.nb, bs, dtype=torch.bool, device=dev)
        for b, L in enumerate(lens):
            pos = np.arange(L)
            used.view(-1)[torch.from_numpy(tab[b, pos // bs].astype(np.int64) * bs + pos % bs).to(dev)] = True
        for c in (self.kc, self.vc):
            x = (torch.randn(self.nb, bs, hkv, d, generator=g, device=dev) * spread).to(dt)
            c[used] = x[used]
        self.q = (torch.randn(len(lens), hq, d, generator=g, device=dev) * 1.5).to(dt)
        self.out = sentinel_tensor((len(lens), hq, d), dtype, dev)
        self.tables = torch.from_numpy(tab).to(dev)
        self.seq_lens = torch.tensor(lens, dtype=torch.int32, device=dev)
        self.start = torch.tensor(start, dtype=torch.int32, device=dev)
        self.prefix = torch.tensor([p for p, _ in groups] if declared is None else declared, dtype=torch.int32,
                                   device=dev)
        self.scale = 1.0 / math.sqrt(d)

    def run(self, **over):
        a = dict(out=self.out, q=self.q, k_cache=self.kc, v_cache=self.vc, block_tables=self.tables,
                 seq_lens=self.seq_lens, group_start=self.start, prefix_lens=self.prefix, scale=self.scale,
                 max_seq_len=max(max(self.lens), 1))
        a.update(over)
        return pk.paged_decode_attention_shared_prefix(**a)

    def check(self, out=None):
        out = self.out if out is None else out
        u, G = U[self.dtype], self.hq // self.hkv
        for b, L in enumerate(self.lens):
            got = out[b].double()
            if L == 0:
                assert not got.any(), b
                continue
            blocks = self.tables[b, :-(-L // self.bs)].long()
            k = self.kc[blocks].double().reshape(-1, self.hkv, self.d)[:L].transpose(0, 1)
            v = self.vc[blocks].double().reshape(-1, self.hkv, self.d)[:L].transpose(0, 1)
            q = self.q[b].double().view(self.hkv, G, self.d)
            s = q @ k.transpose(1, 2) * self.scale
            p = torch.softmax(s, -1)
            o = p @ v
            spread = torch.stack([(p[:, g, :, None] * (v - o[:, g, None]).abs()).sum(1) for g in range(G)], 1)
            pv = p @ v.abs()
            sabs = (q.abs() @ k.abs().transpose(1, 2)).amax(-1, keepdim=True) * abs(self.scale)
            tol = u / (1 - u) * spread + u * o.abs() + pv * 2.0 ** -23 * (
                2 * ((self.d + 4) * sabs + 2 * s.abs().amax(-1, keepdim=True)) + 1100) + 1e-7
            err = (got.view_as(o) - o).abs()
            good = bool(torch.isfinite(got).all()) and bool((err <= tol).all())
            assert good, (b, L, float(err.max()), float((err / tol).max()))


CASES = [  # dtype, Hq, Hkv, D, bs, groups
    ("bf16", 8, 2, 128, 16, [(64, [1, 1])]),
    ("bf16", 8, 2, 128, 16, [(1, [1])]),                        # one token, one sequence
    ("f16", 4, 4, 64, 16, [(16, [1, 2, 3])]),                   # a prefix shorter than a tile
    ("bf16", 32, 8, 128, 16, [(500, [17, 1, 333, 64, 65, 63])]),
    ("f16", 14, 2, 64, 16, [(1000, [5] * 40)]),                 # G 7: three row tiles of 18 sequences
    ("bf16", 28, 4, 128, 32, [(700, [0, 31, 700]), (0, [45]), (95, [1, 2]), (31, [40, 50]), (320, [0, 0])]),
    ("bf16", 8, 1, 128, 64, [(640, list(range(0, 170, 10)))]),  # sequences that end with the prefix
    ("f16", 8, 2, 128, 128, [(300, [200, 1]), (128, [64, 65, 3])]),
    ("bf16", 5, 1, 64, 32, [(97, [3] * 60)]),                   # G 5: 25 sequences a tile
    ("f16", 128, 1, 64, 16, [(80, [9, 70, 1])]),                # G 128: one sequence a tile
    ("bf16", 16, 16, 64, 16, [(2000, [100, 30, 4])]),           # one head per kv head
    ("bf16", 8, 2, 128, 16, [(0, [1]), (0, [700]), (0, [64])]),  # nothing shared
    ("f16", 6, 2, 128, 32, [(6000, [1500, 3, 40])]),            # units cut many times over
    ("bf16", 32, 8, 128, 16, [(256, [1 + i % 7 for i in range(150)])]),  # many units of a tile each
    ("f16", 8, 8, 128, 16, [(48, [2, 1])] * 30),
    ("bf16", 16, 2, 128, 32, [(1000, [20] * 33), (64, [3, 1] * 9)]),  # a pair of row tiles and one more; split units
    ("f16", 8, 1, 64, 16, [(77, [1] * 31), (500, [9] * 17), (33, [4, 4])]),
    ("bf16", 32, 2, 128, 16, [(300, [40, 2, 9] * 9)]),          # G 16: two n8 blocks
    ("bf16", 64, 16, 64, 64, [(64, [5] * 3)] * 20),             # many units of one tile, split
]


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{c[0]}-{c[1]}x{c[2]}x{c[3]}-bs{c[4]}-{len(c[5])}g")
def test_shared_prefix_is_attention(case):
    t = Batch(*case, seed=case[1] + case[3])
    pk.device_error()
    assert t.run() is t.out
    assert pk.device_error() == 0
    t.check()


def test_large_scores_move_the_reference():
    """Scores up to hundreds, the largest in the last tiles: the running
    reference has to move and the parts to be rescaled."""
    t = Batch("bf16", 8, 2, 128, 16, [(400, [90, 200, 1, 64])], seed=7, spread=4.0)
    last = t.tables[0, 24].long()                      # the prefix's last block
    t.kc[last] = t.kc[last] * 4
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    t.check()
    t.scale = -t.scale * 3
    t.run()
    t.check()
    t.scale = 0.0
    t.run()
    t.check()


def test_lowest_values_and_infinities_in_slots_nobody_reads():
    t = Batch("f16", 8, 2, 128, 32, [(100, [10, 1, 50])], seed=8)
    nan = torch.isnan(t.kc[..., :1]).expand_as(t.kc)
    for value in (float("inf"), torch.finfo(torch.float16).min):
        for c in (t.kc, t.vc):
            c[nan] = value
        t.run()
        t.check()


def test_empty_and_short_sequences_in_a_group():
    """Padded rows of a batch, and a sequence shorter than its group's prefix,
    whose table differs from the first one's."""
    groups = [(200, [30, 5, 1, 80, 0]), (64, [3, 9])]
    t = Batch("bf16", 8, 2, 128, 16, groups, seed=9, short={1: 0, 3: 70, 6: 0})
    t.tables[3, :5] = t.tables[3, [4, 3, 2, 1, 0]]
    pk.device_error()
    t.run()
    assert pk.device_error() == 0
    t.check()
    # the group's first sequence empty: nothing is shared, the answers are the same
    t = Batch("bf16", 8, 2, 128, 16, groups, seed=10, short={0: 0, 5: 0, 6: 0})
    t.run()
    assert pk.device_error() == 0
    t.check()
    t = Batch("bf16", 8, 2, 128, 16, [(0, [5, 6])], seed=10, short={0: 0, 1: 0})
    t.run()
    t.check()


def test_prefix_longer_or_shorter_than_what_is_shared_in_whole_blocks():
    # declared past the first sequence's end: cut to its whole blocks
    t = Batch("bf16", 8, 2, 128, 16, [(96, [0, 40, 7])], seed=11, declared=[5000])
    t.run()
    assert pk.device_error() == 0
    t.check()
    for declared in (0, 15, 16, 33, 95):
        t.prefix.fill_(declared)
        t.run()
        t.check()
    t.prefix.fill_(-3)
    t.run()
    assert pk.device_error() == 8
    t.check()


@pytest.mark.parametrize("start", [[1, 3, 5], [0, 3, 4], [0, 6, 5], [0, -1, 5], [0, 2 ** 30, 5], [5, 0, 5]], ids=str)
def test_group_bounds_that_are_none_are_recorded_and_nothing_is_shared(start):
    t = Batch("bf16", 8, 2, 128, 16, [(96, [4, 40, 7]), (32, [1, 2])], seed=12)
    t.start.copy_(torch.tensor(start, dtype=torch.int32))
    pk.device_error()
    t.run()
    assert pk.device_error() == 8
    t.check()


def test_empty_group_and_no_group():
    t = Batch("bf16", 8, 2, 128, 16, [(96, [4, 40, 7]), (32, [1, 2])], seed=13)
    t.start = torch.tensor([0, 0, 3, 3, 5], dtype=torch.int32, device="cuda")
    t.prefix = torch.tensor([77, 96, 5, 32], dtype=torch.int32, device="cuda")
    t.run()
    t.check()
    t.start, t.prefix = t.start[:1].contiguous(), t.prefix[:0].contiguous()
    t.run()
    assert pk.device_error() == 0
    t.check()


def test_out_of_range_table_entries_and_lengths_are_recorded():
    t = Batch("f16", 8, 2, 64, 16, [(64, [4, 40])], seed=14)
    good = t.tables.clone()
    for entry in (-1, t.nb, 2 ** 30):
        t.tables.copy_(good)
        t.tables[1, 5] = entry
        t.run()
        assert pk.device_error() == 8
    t.tables.copy_(good)
    for L in (-5, t.cols * t.bs + 1, 2 ** 31 - 1):
        t.seq_lens[1] = L
        t.tables.copy_(good.clamp(min=0))
        t.run()
        assert pk.device_error() == 8


@pytest.mark.parametrize("shape", [("f32", 8, 2, 128, 16), ("bf16", 8, 2, 256, 16), ("f16", 8, 2, 80, 16),
                                   ("bf16", 8, 2, 128, 8), ("f32", 2, 1, 8, 5)], ids=str)
def test_other_shapes_are_the_plain_call(shape):
    t = Batch(*shape, [(100, [3, 60, 1]), (0, [9])], seed=15)
    t.run()
    want = torch.empty_like(t.out)
    pk.paged_decode_attention(want, t.q, t.kc, t.vc, t.tables, t.seq_lens, t.scale, max(t.lens))
    assert torch.equal(t.out, want) and pk.device_error() == 0
    t.check()


def test_repeated_calls_are_identical_and_workspaces_need_no_clearing():
    t = Batch("bf16", 32, 8, 128, 16, [(900, [17, 300, 64, 1] * 6), (100, [50] * 9)], seed=16)
    ws = pk.shared_prefix_workspace(len(t.lens), 32, 8, 128, 16, max(t.lens), torch.bfloat16, "cuda")
    t.run(workspace=ws)
    t.check()
    want = t.out.clone()
    for fill in (0xFF, 0x7F, 0x00):
        ws.fill_(fill)
        t.out.zero_()
        t.run(workspace=ws)
        assert torch.equal(t.out, want)
    for _ in range(30):
        t.run(workspace=ws)
        assert torch.equal(t.out, want)


def test_captured_graphs_that_share_a_workspace_and_another_stream():
    a = Batch("bf16", 8, 2, 128, 16, [(300, [17, 30, 64, 1])], seed=17)
    b = Batch("bf16", 8, 2, 128, 16, [(0, [500]), (80, [9, 7, 200])], seed=18)
    ws = pk.shared_prefix_workspace(4, 8, 2, 128, 16, 4096, torch.bfloat16, "cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    a.run(workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    b.run(workspace=ws)
    want = a.out.clone(), b.out.clone()
    a.check()
    b.check()
    graphs = []
    for t in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            t.run(workspace=ws)
        graphs.append(g)
    for _ in range(3):
        for t in (a, b):
            t.out.zero_()
        for g in graphs:
            g.replay()
        assert torch.equal(a.out, want[0]) and torch.equal(b.out, want[1])
    # lengths and groups are read at the replay: one sequence ends, the prefix is cut
    a.seq_lens[2] = 0
    a.lens[2] = 0
    a.prefix.fill_(40)
    graphs[0].replay()
    a.check()
    # no workspace given, another stream
    side.wait_stream(torch.cuda.current_stream())
    a.run(stream=side)
    torch.cuda.current_stream().wait_stream(side)
    a.check()


def test_two_calls_at_once_on_two_streams():
    ts = [Batch("bf16", 32, 8, 128, 16, [(600, [40 + i, 3, 100] * 4)], seed=20 + i) for i in range(2)]
    wss = [pk.shared_prefix_workspace(12, 32, 8, 128, 16, 4096, torch.bfloat16, "cuda") for _ in ts]
    streams = [torch.cuda.Stream() for _ in ts]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for _ in range(10):
        for t, ws, s in zip(ts, wss, streams):
            t.run(workspace=ws, stream=s)
    torch.cuda.synchronize()
    for t in ts:
        t.check()
    assert pk.device_error() == 0


def test_wide_batches():
    for n, hkv, groups in ((1700, 1, 1), (2048, 1, 512), (2048, 2, 2), (4096, 1, 512), (4100, 1, 2)):
        t = Batch("bf16", 4 * hkv, hkv, 128, 16, [(64, [1 + i % 3 for i in range(n // groups)])] * groups, seed=23)
        # every sequence a row of its own: check a spread of them
        t.run()
        assert pk.device_error() == 0
        keep = sorted(set(range(0, len(t.lens), 97)) | {len(t.lens) - 1})
        lens = t.lens
        sub = object.__new__(Batch)
        sub.__dict__.update(t.__dict__)
        sub.lens, sub.tables, sub.q = [lens[i] for i in keep], t.tables[keep], t.q[keep]
        sub.check(t.out[keep])


def test_many_groups_of_one():
    t = Batch("bf16", 8, 2, 128, 16, [(40, [3 + i]) for i in range(100)], seed=24)
    t.run()
    assert pk.device_error() == 0
    t.check()


def test_offsets_past_32_bits():
    """A pool of more than 2^32 bytes and 2^31 elements: the blocks used lie at its end."""
    nb, bs, hkv, d = 70000, 32, 8, 128
    kc = torch.zeros(nb, bs, hkv, d, dtype=torch.bfloat16, device="cuda")
    vc = torch.zeros_like(kc)
    assert kc.numel() > 2 ** 31
    t = Batch("bf16", 32, hkv, d, bs, [(100, [5, 70])], seed=25)
    n = t.nb
    kc[-n:], vc[-n:] = t.kc, t.vc
    t.kc, t.vc = kc, vc
    t.tables = torch.where(t.tables >= 0, t.tables + (nb - n), -1)
    t.run()
    assert pk.device_error() == 0
    t.check()


def test_fork_rope_write_and_shared_attention_together():
    """A prompt, five samples forked from it, four decode steps: the manager's
    groups, copy-on-write copies, rotated writes and shared attention, each
    step against attention over the sequence's logical rotated keys."""
    bs, hq, hkv, d, prompt, steps = 16, 8, 2, 128, 150, 4
    dev = torch.device("cuda")
    g = torch.Generator(device="cuda").manual_seed(30)
    mgr = pk.KVBlockManager(64, bs)
    kc = torch.zeros(64, bs, hkv, d, dtype=torch.bfloat16, device=dev)
    vc = torch.zeros_like(kc)
    ang = torch.arange(512, device=dev, dtype=torch.float64)[:, None] * \
        10000.0 ** (-torch.arange(0, d, 2, device=dev, dtype=torch.float64) / d)
    table = torch.cat([ang.cos(), ang.sin()], 1).float()

    def draw(n, h):
        return torch.randn(n, h, d, generator=g, device=dev).bfloat16()

    def turned(x, pos):
        c, s = table[pos, :d // 2][:, None], table[pos, d // 2:][:, None]
        a, b = x.float()[..., :d // 2], x.float()[..., d // 2:]
        return torch.cat([a * c - b * s, b * c + a * s], -1).bfloat16()

    k, v = draw(prompt, hkv), draw(prompt, hkv)
    pos = torch.arange(prompt, device=dev, dtype=torch.int32)
    slots = torch.from_numpy(mgr.allocate_for_prefill(0, prompt)).to(dev)
    pk.rope_and_cache(None, None, k, v, pos, table, kc, vc, slots)
    logical = {0: [(turned(k, pos.long()), v)]}
    for child in range(1, 6):
        mgr.fork(0, child, prompt)
        logical[child] = list(logical[0])
    ids = list(range(6))
    for step in range(steps):
        tab = mgr.decode_step(ids, 16)
        src, dst = mgr.take_copies()
        if len(src):
            pk.copy_blocks(kc, vc, torch.from_numpy(src).to(dev), torch.from_numpy(dst).to(dev))
        slots, tables, lens = (torch.from_numpy(np.ascontiguousarray(x)).to(dev) for x in tab)
        q, k, v = draw(6, hq), draw(6, hkv), draw(6, hkv)
        pos = lens - 1
        q_out = torch.empty_like(q)
        pk.rope_and_cache(q_out, q, k, v, pos, table, kc, vc, slots)
        for b in ids:
            logical[b].append((turned(k[b:b + 1], pos[b:b + 1].long()), v[b:b + 1]))
        start, prefix = mgr.prefix_groups(ids)
        assert start.tolist() == [0, 6] and prefix.tolist() == [prompt // bs * bs]
        out = torch.empty_like(q)
        pk.paged_decode_attention_shared_prefix(out, q_out, kc, vc, tables, lens, torch.from_numpy(start).to(dev),
                                                torch.from_numpy(prefix).to(dev), d ** -0.5, 512)
        assert pk.device_error() == 0
        plain = torch.empty_like(q)
        pk.paged_decode_attention(plain, q_out, kc, vc, tables, lens, d ** -0.5, 512)
        qt = turned(q, pos.long())
        assert torch.equal(q_out, qt)
        for b in ids:
            K = torch.cat([x for x, _ in logical[b]]).double().transpose(0, 1)
            V = torch.cat([y for _, y in logical[b]]).double().transpose(0, 1)
            p = torch.softmax(qt[b].double().view(hkv, -1, d) @ K.transpose(1, 2) * d ** -0.5, -1)
            ref = (p @ V).reshape(hq, d)
            # p rounded and the output rounded, each 2^-8 of at most sum p |V| (twice: the sum is over rounded p too)
            tol = 2.0 ** -8 * 1.05 * (2 * (p @ V.abs()).reshape(hq, d) + ref.abs())
            for o in (out, plain):
                assert bool(((o[b].double() - ref).abs() <= tol).all())


def test_wrapper_refusals():
    t = Batch("f16", 4, 2, 64, 16, [(32, [1, 2])], seed=31)
    t.run()
    ws = pk.shared_prefix_workspace(2, 4, 2, 64, 16, 64, torch.float16, "cuda")
    bad = dict(out=[t.out[:1], t.out.float(), t.out.cpu()], q=[t.q.bfloat16(), t.q[:, :, :32]],
               k_cache=[t.kc.float(), t.kc[:, :, :1], t.kc.cpu()], v_cache=[t.vc[:1]],
               block_tables=[t.tables.long(), t.tables[:1], t.tables[:, :1]], seq_lens=[t.seq_lens.long(),
                                                                                       t.seq_lens[:1]],
               group_start=[t.start.long(), t.start[:1]], prefix_lens=[t.prefix.long(), t.start],
               scale=[float("nan"), float("inf")], workspace=[ws[:100], ws[256:], ws[1:], ws.cpu()])
    for name, values in bad.items():
        for x in values:
            with pytest.raises(pk.KVError) as e:
                t.run(**{name: x})
            assert e.value.code in ("INVALID_ARG", "WORKSPACE"), name

"""Calls that allocate their own workspace and run on a stream of the
caller's choice: the memory is that stream's, so that earlier work on the
current stream cannot still be using it and later work there is not given it
while the call runs."""

import pytest
import torch

import paged_kv_cache_128_gb300 as pk
from paged_kv_cache_128_gb300 import kernels
from tests.test_gpu_shared_prefix import Batch

pytestmark = pytest.mark.gpu


def _calls(t):
    n = len(t.lens)
    slots = torch.full((n,), -1, dtype=torch.int32, device="cuda")      # a step that writes nothing
    rows = slots.clone()
    k, v = t.kc.view(-1, t.hkv, t.d)[:n], t.vc.view(-1, t.hkv, t.d)[:n]
    at = (t.block_tables, t.seq_lens, t.scale, max(t.lens))
    codes = torch.zeros(t.kc.shape, dtype=torch.uint8, device="cuda")
    scales = torch.ones(t.nb, t.hkv, t.bs, device="cuda")
    fp8 = (codes, codes.clone(), scales, scales.clone())
    return {
        "shared": lambda s: t.run(stream=s),
        "decode": lambda s: pk.paged_decode_attention(t.out, t.q, t.kc, t.vc, *at, stream=s),
        "split": lambda s: pk.paged_decode_attention(t.out, t.q, t.kc, t.vc, *at, blocks_per_split=4, stream=s),
        "step": lambda s: pk.paged_decode_step(t.out, t.q, k, v, slots, rows, t.kc, t.vc, *at, stream=s),
        "decode_fp8": lambda s: pk.paged_decode_attention_fp8(t.out, t.q, *fp8, *at, stream=s),
        "step_fp8": lambda s: pk.paged_decode_step_fp8(t.out, t.q, k, v, slots, rows, *fp8, *at, stream=s),
    }


@pytest.mark.parametrize("name", ["shared", "decode", "split", "step", "decode_fp8", "step_fp8"])
def test_the_workspace_belongs_to_the_calls_stream(name, monkeypatch):
    t = Batch("bf16", 32, 8, 128, 16, [(600, [40, 300, 100])], seed=97)
    t.block_tables = t.tables
    taken = []
    for fn in ("alloc_workspace", "shared_prefix_workspace"):
        def spy(*args, _real=getattr(kernels, fn)):
            ws = _real(*args)
            taken.append((torch.cuda.current_stream(), ws))
            return ws
        monkeypatch.setattr(kernels, fn, spy)
    call = _calls(t)[name]
    pk.device_error()
    call(None)
    torch.cuda.synchronize()
    want = t.out.clone()
    side = torch.cuda.Stream()
    t.out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    call(side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(t.out, want) and pk.device_error() == 0
    (first, a), (second, b) = taken
    assert a is not None and b is not None
    assert first == torch.cuda.current_stream() and second == side

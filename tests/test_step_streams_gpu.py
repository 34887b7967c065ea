"""Serving-step calls on a stream other than the current one, which is busy with work of its own."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from sparse_decode_attention_02_gb300 import inputs
from test_rope_gpu import make, scales

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
def test_rotated_queries_while_the_current_stream_is_busy(fp8):
    """The output that the call makes is zero in padding rows and whole in the others, although what
    was enqueued on the current stream before is not done by then."""
    q, k, v, pos, inv, slots, cache = make(3000, 8, 2, 192, 192, fp8=fp8)
    slots[::7] = -1
    want_cache = cache.clone()
    want = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, want_cache, **scales(fp8))
    kw = scales(fp8)
    busy = torch.empty(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(400):                                      # some 100 milliseconds
        busy.add_(1.0)
    got = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, stream=side, **kw)
    side.synchronize()
    assert not torch.cuda.current_stream().query()            # the current stream still had work
    with torch.cuda.stream(side):
        same = torch.equal(got, want) and not got[slots < 0].any()
    torch.cuda.synchronize()
    assert same and torch.equal(cache, want_cache)


def test_split_attention_and_selection_while_the_current_stream_is_busy():
    """The older entries likewise: the default workspace, uploaded scales and outputs that they make."""
    w = inputs.make_workload(inputs.scaled("gqa", requests=3, ctx=(4000, 9000)), "cuda:0", fill="all")
    scores = torch.randn(64, 5000, device="cuda")
    current = torch.full((64,), 4000, dtype=torch.int32, device="cuda")
    want = torch.zeros_like(w.query)
    kw = dict(scale=w.scale, query_len=w.query_len, splits=4, k_scale=w.k_scale, v_scale=w.v_scale, gate=w.gate,
              region_tokens=w.region_tokens)
    args = w.query, w.cache, w.regions, w.block_table, w.positions, w.active
    sda.sparse_decode_attention(*args, want, **kw)
    want_ids = sda.sparse_decode_select_regions(scores, current, 100)
    got = torch.zeros_like(want)
    busy = torch.empty(1 << 28, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(400):
        busy.add_(1.0)
    sda.sparse_decode_attention(*args, got, stream=side, **kw)
    ids = sda.sparse_decode_select_regions(scores, current, 100, stream=side)
    side.synchronize()
    assert not torch.cuda.current_stream().query()
    with torch.cuda.stream(side):
        same = torch.equal(got, want) and torch.equal(ids, want_ids)
    assert same

"""Serving-step calls on a stream other than the current one, which is busy with work of its own."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
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
    for _ in range(100):                                      # tens of milliseconds
        busy.add_(1.0)
    got = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, stream=side, **kw)
    side.synchronize()
    assert not torch.cuda.current_stream().query()            # the current stream still had work
    with torch.cuda.stream(side):
        same = torch.equal(got, want) and not got[slots < 0].any()
    torch.cuda.synchronize()
    assert same and torch.equal(cache, want_cache)

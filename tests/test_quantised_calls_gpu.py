"""Ways to call the quantised cache's entries: waits that run out, flags without a workspace, host threads,
the two ways a call is made, one stream for a chain of them."""
import threading

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from test_quantised_attention_gpu import Problem
from test_quantised_cache_gpu import Cache, filled, slots_of

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


LONG = [20000, 30000, 9000] * 4


@pytest.mark.parametrize("lens,regions,ql,D,int8", [(LONG, None, 1, 192, False), (LONG, None, 2, 192, True), (LONG, (2500, 8), 1, 192, False),
                                                    (LONG, (1200, 64), 2, 64, True), ([6000, 300], None, 1, 192, False),
                                                    ([7000], (80, 64), 1, 256, True)])
def test_a_wait_that_runs_out_is_flagged_and_recoverable(lens, regions, ql, D, int8):
    """Stages and their scales are still on their way when every wait gives up at once: the flag is raised, the
    copies land before the blocks end, and the next call is right.  (Whether a stage is late is a matter of time:
    more calls where none was.)"""
    p = Problem(lens, G=4, H=16, D=D, block=64, span=32, ql=ql, int8=int8, regions=regions)
    by = regions is not None
    ws = p.workspace()
    out, lse, other = torch.empty_like(p.query), torch.empty(p.query.shape[:2], device="cuda"), torch.empty(1 << 28, dtype=torch.uint8, device="cuda")
    kw = dict(scale=p.scale, query_len=p.ql, lse=lse, workspace=ws)
    flags = 0
    sda.set_wait_limit_ns(0)
    try:
        for _ in range(50):
            other.fill_(1)                      # nothing of the cache lies in L2
            if by:
                sda.sparse_decode_quantised_attention(p.query, p.cache, p.scales, p.regions, p.table, p.positions, p.active, out,
                                                      region_tokens=p.rt, **kw)
            else:
                sda.sparse_decode_quantised_paged_attention(p.query, p.cache, p.scales, p.table, p.seq_lens, out, **kw)
            torch.cuda.synchronize()
            flags |= sda.read_errors(ws, clear=True)
            if flags:
                break
    finally:
        sda.set_wait_limit_ns(10 ** 9)
    assert flags == sda.FLAG_TIMEOUT
    p.check(*p.run(regions=by, workspace=ws), regions=by)


def test_flags_without_a_workspace():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        c = Cache(pages=4, B=16, S=16)
        x = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
        at = torch.arange(3, device="cuda")
        assert sda.read_errors(sda.step_workspace(DEV)) == 0
        sda.sparse_decode_quantised_append(x, x, at, c.cache, c.scales)
        assert sda.read_errors(sda.step_workspace(DEV)) == 0
        sda.sparse_decode_quantised_append(x * float("inf"), x, at, c.cache, c.scales)
        assert sda.read_errors(sda.step_workspace(DEV), clear=True) == sda.FLAG_NONFINITE
        sda.sparse_decode_quantised_append(x, x, at + 63, c.cache, c.scales)
        assert sda.read_errors(sda.step_workspace(DEV), clear=True) == sda.FLAG_BOUNDS
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        sda.sparse_decode_quantised_read(c.cache, c.scales, i32([[9]]), i32([0, 3]), x, None)
        assert sda.read_errors(sda.step_workspace(DEV), clear=True) == sda.FLAG_BOUNDS


def test_both_ways_of_a_call_are_the_same():
    """Made natively, or (on a stream that is passed) through ctypes."""
    def one(stream):
        c = Cache(pages=8, G=2, B=32, S=16, D=64, int8=True)
        x = torch.randn(40, 4, 64, generator=torch.Generator().manual_seed(1)).bfloat16().cuda()
        i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        table, lens = i32([[2, 0]]), i32([40])
        out = [torch.zeros(40, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        rows = [torch.zeros(2, 4, 64, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        lse = [torch.zeros(2, 4, device="cuda") for _ in range(2)]
        query = x[:2, :2].repeat(1, 2, 1).contiguous()
        kw = {} if stream is None else dict(stream=stream)
        sda.sparse_decode_quantised_append(x[:, :2], x[:, 2:], torch.tensor(slots_of([2, 0], 0, 40, 32), device="cuda"), c.cache,
                                           c.scales, **kw)
        sda.sparse_decode_quantised_read(c.cache, c.scales, table, i32([0, 35]), *out, first_tokens=i32([5]), **kw)
        sda.sparse_decode_quantised_paged_attention(query, c.cache, c.scales, table, lens, rows[0], scale=0.125, lse=lse[0], **kw)
        sda.sparse_decode_quantised_attention(query, c.cache, c.scales, i32([[0, 4], [3, -1]]), table, i32([39, 39]),
                                              torch.tensor([True, True], device="cuda"), rows[1], scale=0.125, region_tokens=8,
                                              lse=lse[1], clear_inactive=False, **kw)
        torch.cuda.synchronize()
        return [c.store, c.scale_store, *out, *rows, *lse]

    for a, b in zip(one(None), one(torch.cuda.current_stream())):
        assert torch.equal(a, b)
    with pytest.raises(OverflowError):
        sda.sparse_decode_quantised_attention(*[torch.zeros(1, 1, 64, device="cuda")] * 8, scale=1.0, region_tokens=1 << 40)


@pytest.mark.parametrize("regions", [None, (128, 8)])
def test_host_threads_share_a_stream_and_its_workspace(regions):
    p = Problem([3000, 900, 5000, 40], G=2, H=8, D=128, block=32, span=16, regions=regions)
    want, _ = p.run(regions=regions is not None)
    outs = [[torch.zeros_like(p.query) for _ in range(20)] for _ in range(6)]
    torch.cuda.synchronize()
    stream = torch.cuda.current_stream()

    def work(mine):
        with torch.cuda.stream(stream):
            for out in mine:
                if regions:
                    sda.sparse_decode_quantised_attention(p.query, p.cache, p.scales, p.regions, p.table, p.positions, p.active, out,
                                                          scale=p.scale, region_tokens=8)
                else:
                    sda.sparse_decode_quantised_paged_attention(p.query, p.cache, p.scales, p.table, p.seq_lens, out, scale=p.scale)

    threads = [threading.Thread(target=work, args=(x,)) for x in outs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert all(torch.equal(x, want) for mine in outs for x in mine)


def test_a_chain_needs_no_waits():
    """Many appends, reads and attentions one behind another on a stream: each sees what the ones before it wrote."""
    B, S, D, G = 32, 16, 128, 2
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(200, 1, 2 * G, D, generator=gen).bfloat16().cuda()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    table, pages = i32([list(range(7))]), list(range(7))
    at = torch.tensor(slots_of(pages, 0, 200, B), device="cuda").view(200, 1)
    lens, starts = [i32([t + 1]) for t in range(200)], [i32([0, t + 1]) for t in range(200)]
    query = torch.randn(G, 4, D, generator=gen).bfloat16().cuda()

    def chain(wait):
        c = Cache(pages=8, G=G, B=B, S=S, D=D, int8=True)
        outs = [torch.zeros_like(query) for _ in range(200)]
        keys = [torch.zeros(t + 1, G, D, dtype=torch.bfloat16, device="cuda") for t in range(200)]
        torch.cuda.synchronize()
        for t in range(200):
            sda.sparse_decode_quantised_append(x[t, :, :G], x[t, :, G:], at[t], c.cache, c.scales)
            wait()
            sda.sparse_decode_quantised_read(c.cache, c.scales, table, starts[t], keys[t], None)
            sda.sparse_decode_quantised_paged_attention(query, c.cache, c.scales, table, lens[t], outs[t], scale=0.09)
            wait()
        torch.cuda.synchronize()
        return outs + keys + [c.store, c.scale_store]

    for a, b in zip(chain(lambda: None), chain(torch.cuda.synchronize)):
        assert torch.equal(a, b)


def test_a_full_cache_of_short_requests():
    """More runs than a CTA's warps take at a time, in one chunk and across chunks, with padding between requests."""
    c = Cache(pages=300, G=3, B=16, S=8, D=64)
    filled(c, [[1 + q % 3 for q in range(120)], [1] * 120, [7] * 120], torch.Generator().manual_seed(4))

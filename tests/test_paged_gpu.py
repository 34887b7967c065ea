"""Attention over the whole paged cache, against float64 attention over the gathered tokens.
Bounds: step_util.attention_bound, element by element."""
import itertools
import random

import numpy as np
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import step_util

pytestmark = pytest.mark.gpu
KS, VS = 8.0 / 448.0, 6.0 / 448.0


class Problem:
    def __init__(self, lens, *, G=1, H=8, D=192, block=16, ql=1, fp8=False, gate=False, seed=0, spare=0, width=None,
                 q_std=2.0):
        r = random.Random(seed)
        gen = torch.Generator().manual_seed(seed + 17 * D + H)
        self.lens, self.G, self.H, self.D, self.block, self.ql, self.fp8 = list(lens), G, H, D, block, ql, fp8
        need = [-(-max(n, 0) // block) for n in lens]
        pages = sum(need) + 2
        ids = list(range(pages))
        r.shuffle(ids)
        W = width or max(1, max(need, default=0)) + spare
        table = np.full((len(lens), W), -1)
        at = 0
        for q, n in enumerate(need):
            table[q, :n] = ids[at:at + n]
            at += n
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda").view(len(lens), W)
        rows = len(lens) * ql * G
        kv = torch.randn(pages, G, block, 2 * D, generator=gen)
        if fp8:
            kv = (kv / KS).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        else:
            kv = kv.bfloat16()
        # what no request's token holds is not a number
        bad = 0x7F if fp8 else float("nan")
        used = torch.zeros(pages, block, dtype=torch.bool)
        for q, n in enumerate(lens):
            for c in range(need[q]):
                used[table[q, c], :max(0, min(block, n - c * block))] = True
        kv.permute(0, 2, 1, 3)[~used] = bad
        self.cache = kv.cuda()
        self.query = (torch.randn(rows, H, D, generator=gen) * q_std).bfloat16().cuda()
        self.gate = (torch.randn(rows // G, G * H, generator=gen) * 2).bfloat16().cuda() if gate else None
        self.scale = D ** -0.5
        self.seq_lens = torch.tensor(list(lens), dtype=torch.int32, device="cuda")

    def kw(self):
        k = dict(scale=self.scale, query_len=self.ql, gate=self.gate)
        if self.fp8:
            k |= dict(k_scale=torch.tensor([KS], device="cuda"), v_scale=torch.tensor([VS], device="cuda"))
        return k

    def workspace(self):
        return torch.zeros(sda.paged_workspace_bytes(self.H, self.ql, self.D), dtype=torch.uint8, device="cuda")

    def run(self, *, out=None, lse=None, workspace=None, flags=0, query=None, cache=None, table=None, **kw):
        out = torch.full_like(self.query, float("nan")) if out is None else out
        lse = torch.full(self.query.shape[:2], float("nan"), device="cuda") if lse is None else lse
        ws = self.workspace() if workspace is None else workspace
        sda.sparse_decode_paged_attention(self.query if query is None else query, self.cache if cache is None else cache,
                                          self.table if table is None else table, self.seq_lens, out, lse=lse, workspace=ws,
                                          **{**self.kw(), **kw})
        torch.cuda.synchronize()
        assert sda.read_errors(ws, clear=True) == flags
        return out, lse

    def exact(self):
        f = float(torch.tensor(KS)), float(torch.tensor(VS))
        return step_util.paged_attention(self.query.cpu(), self.cache.cpu(), self.table.cpu(), self.lens,
                                         scale=float(np.float32(self.scale)), query_len=self.ql,
                                         k_scale=f[0] if self.fp8 else 1.0, v_scale=f[1] if self.fp8 else 1.0,
                                         gate=None if self.gate is None else self.gate.cpu())

    def check(self, out, lse, rows=None):
        o, l, spread, slack = self.exact()
        got, got_l = out.cpu().double(), lse.cpu().double()
        pick = torch.ones(o.shape[0], dtype=torch.bool)
        for q, n in enumerate(self.lens):
            if n < 0:
                pick[q * self.ql * self.G:(q + 1) * self.ql * self.G] = False
        bound = step_util.attention_bound(o, spread, slack, self.fp8, self.gate is not None)
        err = (got - o).abs()
        assert torch.isfinite(got[pick]).all()
        worst = (err / bound)[pick].max().item()
        assert worst <= 1.0, f"error {worst:.2f} times its bound"
        dead = pick[:, None] & torch.isinf(l)
        assert (out.cpu().view(torch.int16)[dead] == 0).all() and (lse.cpu()[dead] == -float("inf")).all()
        live = pick[:, None] & ~torch.isinf(l)
        assert ((got_l - l).abs() <= slack + l.abs() * 2.0 ** -22 + 2.0 ** -18)[live].all()


def check(*a, **kw):
    p = Problem(*a, **kw)
    out, lse = p.run()
    p.check(out, lse)
    return p


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,ql", [(1, 1), (8, 1), (16, 1), (16, 2), (5, 3), (40, 1), (16, 4)])
def test_shapes(D, fp8, H, ql):
    check([1, 700, 0, 65, 333, 2], H=H, ql=ql, D=D, fp8=fp8, G=2, block=16, spare=40)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 129, 255, 257, 1023, 1025])
@pytest.mark.parametrize("fp8", [False, True])
def test_lengths_around_tiles(n, fp8):
    check([n], fp8=fp8, D=192, block=64, spare=30)
    check([n], fp8=fp8, D=192, block=64)                       # a narrow table: units are not cut
    check([n, n + 1], fp8=fp8, D=128, block=32, ql=2, spare=90)


@pytest.mark.parametrize("block", [8, 16, 24, 32, 40, 48, 56, 64, 72, 96, 128, 136, 256])
@pytest.mark.parametrize("D,fp8", [(192, True), (128, False), (64, True), (256, False)])
def test_page_sizes(block, D, fp8):
    check([3 * block + 5, 1, block, 2 * block - 1, 0, 1000], D=D, fp8=fp8, block=block, G=2, H=4)


def test_one_long_request_is_shared_by_all_ctas():
    check([40001], G=1, H=16, D=192, block=64, fp8=True)
    check([20011], G=3, H=4, D=64, block=16, ql=4)
    check([30000, 5], G=2, H=16, D=128, block=128, ql=2, fp8=True, gate=True)


def test_many_short_requests():
    r = random.Random(1)
    check([r.choice([0, 1, 5, 30, 64, 200, 900]) for _ in range(400)], G=2, H=4, D=64, block=16, fp8=True)   # more units than CTAs
    check([r.randint(0, 90) for _ in range(500)], G=1, H=16, D=192, block=16)                                # none is cut
    check([r.choice([0, 1, 2, 3]) for _ in range(1000)], G=1, H=2, D=64, block=8, ql=3, spare=100)


@pytest.mark.parametrize("seed", range(24))
def test_drawn(seed):
    r = random.Random(700 + seed)
    fp8, D = r.random() < 0.5, r.choice([64, 128, 192, 256])
    ql = r.choice([1, 1, 2, 3, 4])
    H = r.randint(1, 64 // ql) if r.random() < 0.3 else r.randint(1, 16)
    n = r.choice([1, 2, 5, 33])
    top = r.choice([20, 300, 3000])
    check([r.choice([0, 1, ql, r.randint(1, top)]) if r.random() < 0.3 else r.randint(1, top) for _ in range(n)],
          G=r.choice([1, 2, 3]), H=H, D=D, block=r.choice([8, 16, 24, 64, 80, 128]), ql=ql, fp8=fp8, gate=r.random() < 0.5,
          seed=seed, spare=r.choice([0, 50]))


def test_padding_requests_keep_their_rows():
    p = Problem([100, -1, 0, 70, -1, -5], G=2, H=8, ql=2, D=128, block=16, spare=60)
    out, lse = torch.full_like(p.query, 5.0), torch.full(p.query.shape[:2], 6.0, device="cuda")
    p.run(out=out, lse=lse)
    for q, n in enumerate(p.lens):
        rows = slice(q * 4, q * 4 + 4)
        assert (out[rows] == 5.0).all() == (n < 0) and (lse[rows] == 6.0).all() == (n < 0)
    p.check(out, lse)


def test_all_requests_empty():
    p = Problem([0] * 9, G=2, H=8, spare=50)
    p.check(*p.run())
    p = Problem([-1] * 3, G=2, H=8, spare=50)
    out = torch.full_like(p.query, 5.0)
    p.run(out=out)
    assert (out == 5.0).all()


@pytest.mark.parametrize("fp8", [False, True])
def test_values_that_are_not_numbers_reach_their_readers_only(fp8):
    """The newest token's V is NaN: the last query token reads it, the others do not."""
    p = Problem([130, 64, 33], G=2, H=4, D=128, ql=4, block=16, fp8=fp8, spare=60)
    for q, n in enumerate(p.lens):
        page = p.table[q, (n - 1) // 16]
        p.cache[page, :, (n - 1) % 16, 128:] = 0x7F if fp8 else float("nan")
    out, lse = p.run()
    o, l, spread, slack = p.exact()
    last = (torch.arange(o.shape[0]) // p.G) % p.ql == p.ql - 1
    got = out.cpu().double()
    assert torch.isnan(got[last]).all() and torch.isfinite(got[~last]).all()
    assert ((got - o).abs() <= step_util.attention_bound(o, spread, slack, fp8))[~last].all()


def test_nan_and_infinite_logits():
    p = Problem([300, 40], G=1, H=8, D=64, block=16, spare=40)
    p.query[0, 3, 5] = float("nan")
    p.query[1, 2] = 0
    out, lse = p.run()
    assert torch.isnan(out[0, 3]).all() and torch.isnan(lse[0, 3])
    rest = torch.ones_like(lse, dtype=torch.bool)
    rest[0, 3] = False
    assert torch.isfinite(out[rest]).all() and torch.isfinite(lse[rest]).all()
    o, l, _s, _k = p.exact()
    assert abs(lse[1, 2].item() - np.log(40)) < 1e-5                 # q = 0: the mean of V


def test_large_logits_and_every_query_magnitude():
    """Logits of some hundreds (one token takes nearly all), and FP8 queries far from 1."""
    for fp8 in (False, True):
        check([777, 12], fp8=fp8, q_std=60.0, G=2, spare=40)
    p = Problem([500], fp8=True, H=6, spare=40)
    p.query *= torch.tensor([1e-6, 3e4, 1.0, 1e-3, 2e2, 0.0], device="cuda")[None, :, None].bfloat16()
    p.scale = 192 ** -0.5 * 1e-4
    p.check(*p.run())


def test_strides_and_alignment():
    p = Problem([90, 300], G=2, H=6, D=192, block=16, ql=2, fp8=False, spare=30)
    want, want_lse = p.run()
    rows, H, D = p.query.shape
    # heads first, rows in between, then a base that is off by one element
    q = torch.empty(H, rows, D, dtype=torch.bfloat16, device="cuda").transpose(0, 1)
    q.copy_(p.query)
    raw = torch.full((rows * (H * D + 5) + 1,), 3.0, dtype=torch.bfloat16, device="cuda")
    out = raw[1:].as_strided((rows, H, D), (H * D + 5, D, 1), 1)
    lse = torch.full((H, rows), 9.0, device="cuda").T
    p.run(query=q, out=out, lse=lse)
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    odd = torch.empty(rows * H * D + 1, dtype=torch.bfloat16, device="cuda")[1:].view(rows, H, D)
    odd.copy_(p.query)
    assert torch.equal(p.run(query=odd)[0], want)
    # a cache whose pages lie apart, its groups inside the tokens
    pages, G, B, row = p.cache.shape
    c = torch.full((pages, B, G, row + 8), float("nan"), dtype=torch.bfloat16, device="cuda")
    c[..., :row] = p.cache.transpose(1, 2)
    assert torch.equal(p.run(cache=c[..., :row].transpose(1, 2))[0], want)
    t = torch.full((2, p.table.shape[1] + 3), 99999, dtype=torch.int32, device="cuda")
    t[:, :-3] = p.table
    assert torch.equal(p.run(table=t[:, :-3])[0], want)


def test_bad_pages_and_lengths_are_flagged():
    p = Problem([200, 100], G=2, H=8, D=128, block=16, spare=30)
    t = p.table.clone()
    t[0, 3], t[1, 2] = -1, p.cache.shape[0]
    out, _ = p.run(table=t, flags=sda.FLAG_BOUNDS)
    assert torch.isfinite(out).all()
    p.seq_lens[1] = p.table.shape[1] * 16 + 1                        # past the table
    p.table[1, 7:] = p.table[1, 0]
    p.run(flags=sda.FLAG_BOUNDS)


def test_the_same_bits_every_time_and_in_a_graph():
    p = Problem([5000, 77, 1200], G=2, H=16, D=192, block=64, fp8=True, gate=True)
    want, want_lse = p.run()
    for _ in range(3):
        a, b = p.run()
        assert torch.equal(a, want) and torch.equal(b, want_lse)
    out, lse = torch.empty_like(want), torch.empty_like(want_lse)
    kw = p.kw()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, lse=lse, **kw)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want) and torch.equal(lse, want_lse)
    # the same graph after the requests have moved on
    p.lens = [4000, 78, 0]
    p.cache[p.table[1, 77 // 64], :, 77 % 64] = p.cache[p.table[1, 0], :, 5]     # the token that was added
    p.seq_lens.copy_(torch.tensor(p.lens))
    g.replay()
    torch.cuda.synchronize()
    p.check(out, lse)


def test_two_streams_and_two_graphs():
    a = Problem([3000, 10], G=2, H=16, D=128, block=16, seed=1)
    b = Problem([500] * 8, G=2, H=16, D=128, block=16, seed=2)
    (wa, la), (wb, lb) = a.run(), b.run()
    s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
    oa, ob = torch.empty_like(wa), torch.empty_like(wb)
    ka, kb = a.kw(), b.kw()
    torch.cuda.synchronize()
    for _ in range(20):
        sda.sparse_decode_paged_attention(a.query, a.cache, a.table, a.seq_lens, oa, stream=s1, **ka)
        sda.sparse_decode_paged_attention(b.query, b.cache, b.table, b.seq_lens, ob, stream=s2, **kb)
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)
    graphs = []
    for p, o, k in ((a, oa, ka), (b, ob, kb)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, o, **k)
        graphs.append(g)
    oa.zero_(), ob.zero_()
    torch.cuda.synchronize()
    for _ in range(10):
        for g, s in zip(graphs, (s1, s2)):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    assert torch.equal(oa, wa) and torch.equal(ob, wb)


def test_cache_offsets_past_32_bits():
    """Pages whose byte offset passes 2^32: a 6 GB cache of which a few pages are read."""
    D, B = 192, 64
    pages = 6 * 2 ** 30 // (B * 2 * D)
    cache = torch.empty(pages, 1, B, 2 * D, dtype=torch.uint8, device="cuda")
    use = [pages - 1, 0, pages - 2, 2 ** 32 // (B * 2 * D) + 1, 2 ** 31 // (B * 2 * D)]
    p = Problem([5 * B - 3], fp8=True, block=B, H=16)
    idx = torch.tensor(use, device="cuda")
    cache[idx] = p.cache[p.table[0, :5].long()]
    want, want_lse = p.run()
    got, got_lse = p.run(cache=cache, table=idx.int()[None])
    assert torch.equal(got, want) and torch.equal(got_lse, want_lse)


def test_joins_with_attention_over_other_keys():
    """The log-sum-exp joins two halves of a request into the whole."""
    p = Problem([640], G=2, H=8, D=128, block=64)
    whole, whole_lse = p.run()
    parts = []
    for cols in (slice(0, 4), slice(4, 10)):
        t = p.table[:, cols].contiguous()
        out, lse = torch.empty_like(whole), torch.empty_like(whole_lse)
        sda.sparse_decode_paged_attention(p.query, p.cache, t, torch.tensor([t.shape[1] * 64], dtype=torch.int32, device="cuda"),
                                          out, lse=lse, **p.kw())
        parts.append((out.double(), lse.double()))
    (o1, l1), (o2, l2) = parts
    l = torch.logaddexp(l1, l2)
    o = o1 * torch.exp(l1 - l)[..., None] + o2 * torch.exp(l2 - l)[..., None]
    assert ((l - whole_lse).abs() < 1e-5).all()
    assert ((o - whole.double()).abs() <= 3 * 2.0 ** -8 * (o1.abs() + o2.abs())).all()


def test_a_wait_that_runs_out_is_flagged():
    # all SMs stream from a cold cache: a wait's own hardware suspension is over before the data is there
    p = Problem([30000] * 8, G=2, H=16, D=192, block=64, fp8=True)
    want, _ = p.run()
    ws = p.workspace()
    out = torch.empty_like(want)
    torch.zeros(1 << 29, dtype=torch.uint8, device="cuda")
    sda.set_wait_limit_ns(0)
    try:
        sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, workspace=ws, **p.kw())
        torch.cuda.synchronize()
        assert sda.read_errors(ws, clear=True) & sda.FLAG_TIMEOUT
    finally:
        sda.set_wait_limit_ns(1_000_000_000)
    assert torch.equal(p.run(workspace=ws)[0], want)

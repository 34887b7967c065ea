"""Attention over a quantised cache, whole and by regions, against float64 attention over the decoded
tokens.  Bounds: quant_util.attention_bound, element by element."""
import random

import numpy as np
import pytest
import torch

import quant_util
import sparse_decode_attention_02_gb300 as sda

pytestmark = pytest.mark.gpu


class Problem:
    """Requests of given lengths in a cache whose blocks have scales of their own (spread by e^scale_std); what
    no token holds, element or scale, is not a number."""

    def __init__(self, lens, *, G=1, H=8, D=192, block=16, span=16, ql=1, int8=False, gate=False, seed=0, spare=0, width=None,
                 q_std=1.0, scale_std=0.7, regions=None):
        gen = torch.Generator().manual_seed(seed + 17 * D + H)
        r = random.Random(seed)
        self.lens, self.G, self.H, self.D, self.block, self.span, self.ql, self.int8 = list(lens), G, H, D, block, span, ql, int8
        need = [-(-max(n, 0) // block) for n in lens]
        pages = sum(need) + 2
        ids = list(range(pages))
        r.shuffle(ids)
        W = width or max(1, max(need, default=0)) + spare
        table = np.full((len(lens), W), -1)
        self.pages = []
        for q, n in enumerate(need):
            self.pages.append([ids.pop() for _ in range(n)])
            table[q, :n] = self.pages[-1]
        self.table = torch.tensor(table, dtype=torch.int32, device="cuda").view(len(lens), W)
        if int8:
            raw = (torch.randn(pages, G, block, 2 * D, generator=gen) * 40).round().clamp(-127, 127).to(torch.int8)
            size = 1 / 40
        else:
            raw = (torch.randn(pages, G, block, 2 * D, generator=gen) * 100).clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
            size = 1 / 100
        scales = torch.exp(torch.randn(pages, G, block // span, 2, generator=gen) * scale_std) * size
        held = torch.zeros(pages, block, dtype=torch.bool)
        for q, n in enumerate(lens):
            for c, page in enumerate(self.pages[q]):
                held[page, :max(0, min(block, n - c * block))] = True
        if not int8:
            raw.permute(0, 2, 1, 3)[~held] = 0x7F
        scales.permute(0, 2, 1, 3)[~held.view(pages, -1, span).any(-1)] = float("nan")
        self.cache, self.scales = raw.cuda(), scales.cuda()
        rows = len(lens) * ql * G
        self.query = (torch.randn(rows, H, D, generator=gen) * q_std).bfloat16().cuda()
        self.gate = (torch.randn(rows // G, G * H, generator=gen) * 2).bfloat16().cuda() if gate else None
        self.scale = D ** -0.5
        self.seq_lens = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        if regions:
            self.select(regions[0], regions[1], r)

    def select(self, count, rt, r):
        """Regions of each row: any of its request's and some past its position, in any order, -1 among them, at times one twice."""
        rows = self.query.shape[0]
        pos = [self.lens[k // (self.ql * self.G)] - self.ql + k // self.G % self.ql for k in range(rows)]
        ids = np.full((rows, count), -1)
        for k, p in enumerate(pos):
            have = list(range(-(-max(self.lens[k // (self.ql * self.G)], 0) // rt)))
            r.shuffle(have)
            if len(have) > 2 and r.random() < 0.2:
                have[1] = have[0]
            pick = have[:r.choice((count, count, max(1, count // 3)))][:count]
            pick += [-1] * (count - len(pick))
            r.shuffle(pick)
            ids[k] = pick
        self.rt = rt
        self.regions = torch.tensor(ids, dtype=torch.int32, device="cuda").view(rows, count)
        self.positions = torch.tensor(pos, dtype=torch.int32, device="cuda")
        self.active = torch.tensor([p >= 0 and r.random() < 0.9 for p in pos], device="cuda")

    def workspace(self):
        need = sda.paged_workspace_bytes(self.H, self.ql, self.D)
        need = max(need, sda.quantised_workspace_bytes(self.query.shape[0], self.H, self.D))
        return torch.zeros(need, dtype=torch.uint8, device="cuda")

    def run(self, *, regions=False, out=None, lse=None, workspace=None, flags=0, **kw):
        out = torch.full_like(self.query, float("nan")) if out is None else out
        lse = torch.full(self.query.shape[:2], float("nan"), device="cuda") if lse is None else lse
        ws = self.workspace() if workspace is None else workspace
        kw = dict(scale=self.scale, query_len=self.ql, gate=self.gate, lse=lse, workspace=ws) | kw
        if regions:
            sda.sparse_decode_quantised_attention(self.query, self.cache, self.scales, self.regions, self.table, self.positions,
                                                  self.active, out, region_tokens=self.rt, **kw)
        else:
            sda.sparse_decode_quantised_paged_attention(self.query, self.cache, self.scales, self.table, self.seq_lens, out, **kw)
        torch.cuda.synchronize()
        assert sda.read_errors(ws, clear=True) == flags
        return out, lse

    def row(self, r, regions):
        """Keys and values that row r sees, decoded, and its largest value scale."""
        q, g = r // (self.ql * self.G), r % self.G
        n = self.lens[q]
        if regions:
            ids = self.regions[r].cpu().long()
            t = (ids[ids >= 0][:, None] * self.rt + torch.arange(self.rt)).view(-1)
            t = t[t <= int(self.positions[r])]
            if not self.active[r]:
                t = t[:0]
        else:
            t = torch.arange(max(0, n - self.ql + 1 + r // self.G % self.ql))
        page, off = torch.tensor(self.pages[q] + [0])[t // self.block], t % self.block
        x = torch.from_numpy(quant_util.values(self.host_cache[page, g, off].contiguous(), self.int8)).view(len(t), 2, self.D)
        s = self.host_scales[page, g, off // self.span].double()
        x = x * s[:, :, None]
        return x[:, 0], x[:, 1], s[:, 1].max().item() if len(t) else 0.0

    def check(self, out, lse, *, regions=False, left=None):
        """`left`: what rows that are not computed have to hold still."""
        self.host_cache, self.host_scales = self.cache.cpu(), self.scales.cpu()
        got, got_l = out.cpu().double(), lse.cpu().double()
        query, scale = self.query.cpu().double(), float(np.float32(self.scale))
        gate = None
        if self.gate is not None:
            gate = (1.0 / (1.0 + torch.exp(-self.gate.cpu().float()))).bfloat16().double().view(-1, self.G, self.H).reshape(-1, self.H, 1)
        worst = 0.0
        for r in range(len(query)):
            skipped = (not self.active[r] if regions else self.lens[r // (self.ql * self.G)] < 0)
            if skipped and (not regions or left is not None):
                kept = torch.full_like(got[r], float("nan")) if left is None else left[0][r].cpu().double()
                assert torch.equal(got[r].nan_to_num(7.0), kept.nan_to_num(7.0))
                continue
            k, v, top = self.row(r, regions)
            o, l, spread, slack = quant_util.attend(query[r], k, v, scale)
            if not len(k):
                assert (out[r].view(torch.int16) == 0).all() and (got_l[r] == -float("inf")).all()
                continue
            if gate is not None:
                o, spread = o * gate[r], spread * gate[r]
            assert torch.isfinite(got[r]).all()
            bound = quant_util.attention_bound(o, spread, slack, top * (127 if self.int8 else 448), len(k), gate is not None)
            worst = max(worst, ((got[r] - o).abs() / bound).max().item())
            assert ((got_l[r] - l).abs() <= slack + l.abs() * 2.0 ** -22 + 2.0 ** -18).all()
        assert worst <= 1.0, f"error {worst:.2f} times its bound"


def check(*a, regions=None, **kw):
    p = Problem(*a, regions=regions, **kw)
    p.check(*p.run(regions=regions is not None), regions=regions is not None)
    return p


# ---------------------------------------------------------------------------- whole caches


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("H,ql", [(1, 1), (8, 1), (16, 1), (16, 2), (5, 3), (40, 1), (16, 4)])
def test_shapes(D, int8, H, ql):
    check([1, 700, 0, 65, 333, 2, -1], H=H, ql=ql, D=D, int8=int8, G=2, block=16, spare=40)


@pytest.mark.parametrize("n", [1, 2, 7, 8, 9, 15, 16, 17, 31, 33, 63, 64, 65, 127, 129, 255, 257, 1023, 1025])
@pytest.mark.parametrize("int8", [False, True])
def test_lengths_around_tiles(n, int8):
    check([n], int8=int8, D=192, block=64, span=32, spare=30)
    check([n], int8=int8, D=192, block=64, span=64)            # a narrow table: units are not cut
    check([n, n + 1], int8=int8, D=128, block=32, span=8, ql=2, spare=90)


@pytest.mark.parametrize("block,span", [(8, 8), (16, 8), (24, 24), (24, 8), (32, 16), (40, 40), (48, 24), (56, 8), (64, 64), (72, 24),
                                        (96, 48), (128, 128), (136, 8), (256, 64)])
@pytest.mark.parametrize("D,int8", [(192, True), (128, False), (64, True), (256, False)])
def test_page_and_block_sizes(block, span, D, int8):
    check([3 * block + 5, 1, block, 2 * block - 1, 0, 1000], D=D, int8=int8, block=block, span=span, G=2, H=4)


def test_one_long_request_is_shared_by_all_ctas():
    check([40001], G=1, H=16, D=192, block=64, span=64)
    check([20011], G=3, H=4, D=64, block=16, span=8, ql=4, int8=True)
    check([30000, 5], G=2, H=16, D=128, block=128, span=32, ql=2, int8=True, gate=True)


def test_many_short_requests():
    r = random.Random(1)
    check([r.choice([0, 1, 5, 30, 64, 200, 900]) for _ in range(400)], G=2, H=4, D=64, block=16, int8=True)
    check([r.randint(0, 90) for _ in range(500)], G=1, H=16, D=192, block=16)
    check([r.choice([0, 1, 2, 3]) for _ in range(1000)], G=1, H=2, D=64, block=8, span=8, ql=3, spare=100)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("ql", [1, 3])
def test_scales_far_apart(int8, ql):
    """Value scales over a hundred powers of two, in any order: an output's error goes by the largest."""
    p = Problem([900, 40, 2500], G=2, H=8, D=128, block=32, span=8, ql=ql, int8=int8, spare=20, scale_std=0.0)
    gen = torch.Generator().manual_seed(3)
    p.scales[..., 1] *= torch.exp2(torch.randint(-100, 101, p.scales.shape[:3], generator=gen).double()).float().cuda()
    p.check(*p.run())


@pytest.mark.parametrize("int8", [False, True])
def test_scales_at_the_ends(int8):
    """Zero, the smallest and nearly the largest that a bf16 cache could need."""
    p = Problem([900, 40], G=1, H=4, D=64, block=16, span=16, int8=int8, spare=20, scale_std=0.0)
    held = ~p.scales[..., 1].isnan()
    p.scales[..., 1] = torch.where(held, torch.full_like(p.scales[..., 1], 2.0 ** -126), p.scales[..., 1])
    p.check(*p.run())
    p.scales[..., 1] = torch.where(held, torch.zeros_like(p.scales[..., 1]), p.scales[..., 1])
    out, _ = p.run()
    assert (out == 0).all()
    p.scales[..., 1] = torch.where(held, torch.full_like(p.scales[..., 1], 2.0 ** 118), p.scales[..., 1])
    p.check(*p.run())


def test_peaked_rows():
    """Large logits: nearly all weight on one token, that of another block than the largest value scale."""
    check([3000, 77], G=2, H=16, D=192, block=64, span=16, q_std=12.0, scale_std=1.5)
    check([3000, 77], G=2, H=16, D=192, block=64, span=16, q_std=12.0, scale_std=1.5, int8=True, ql=2)


def test_one_scale_for_all_is_the_plain_cache():
    """E4M3 with one scale everywhere: what sparse_decode_paged_attention gives, up to its own rounding."""
    p = Problem([5000, 300, 41], G=2, H=8, D=192, block=64, span=64, int8=False, spare=3, scale_std=0.0)
    one = torch.tensor([0.01], device="cuda")
    p.scales.fill_(0.01)
    p.cache[(p.cache & 0x7F) == 0x7F] = 0x30
    out, lse = p.run()
    plain, plain_l = torch.empty_like(out), torch.empty_like(lse)
    sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, plain, scale=p.scale, k_scale=one, v_scale=one, lse=plain_l)
    assert ((out.double() - plain.double()).abs() <= 2 * (2.0 ** -8 * plain.double().abs() + 0.01 * 448 * 2.0 ** -11)).all()
    assert ((lse - plain_l).abs() <= 1e-4).all()


@pytest.mark.parametrize("seed", range(16))
def test_drawn(seed):
    r = random.Random(100 + seed)
    block = r.choice((8, 16, 24, 32, 64, 128))
    span = r.choice([s for s in range(8, block + 1, 8) if block % s == 0])
    check([r.choice((0, -1, r.randint(1, 40), r.randint(1, 3000))) for _ in range(r.randint(1, 40))], G=r.choice((1, 2, 4)),
          H=r.randint(1, 16), D=r.choice((64, 128, 192, 256)), block=block, span=span, ql=r.choice((1, 1, 2, 4)), int8=r.random() < 0.5,
          gate=r.random() < 0.5, spare=r.choice((0, 5, 300)), seed=seed)


def test_strided_views():
    """Queries, outputs, cache and scales that are views with gaps and odd alignments."""
    p = Problem([300, 17], G=2, H=4, D=128, block=16, span=8, int8=True, spare=3)
    want, want_l = p.run()
    wide = torch.zeros(p.query.shape[0], 6, 131, dtype=torch.bfloat16, device="cuda")
    wide[:, 1:5, 1:129] = p.query
    p.query = wide[:, 1:5, 1:129]
    cache = torch.zeros(p.cache.shape[0], 3, 18, 272, dtype=torch.int8, device="cuda")
    cache[:, :2, :16, :256] = p.cache
    p.cache = cache[:, :2, :16, :256]
    scales = torch.zeros(p.cache.shape[0], 3, 3, 2, device="cuda")
    scales[:, :2, :2] = p.scales
    p.scales = scales[:, :2, :2]
    out = torch.zeros(p.query.shape[0], 5, 129, dtype=torch.bfloat16, device="cuda")
    lse = torch.zeros(p.query.shape[0], 9, device="cuda")
    p.run(out=out[:, 1:, 1:], lse=lse[:, ::2][:, :4])
    assert torch.equal(out[:, 1:, 1:], want) and torch.equal(lse[:, ::2][:, :4], want_l)


# ---------------------------------------------------------------------------- regions


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("H,ql", [(1, 1), (8, 2), (16, 3)])
@pytest.mark.parametrize("count", [3, 60])
def test_region_shapes(D, int8, H, ql, count):
    check([5, 700, 0, 65, 333, 12], H=H, ql=ql, D=D, int8=int8, G=2, block=16, span=8, regions=(count, 8))


@pytest.mark.parametrize("block,rt", [(8, 8), (16, 8), (16, 64), (16, 40), (24, 8), (24, 24), (48, 24), (32, 32), (64, 64), (64, 8), (64, 128),
                                      (128, 16), (40, 16), (128, 128)])
@pytest.mark.parametrize("D,int8", [(192, False), (128, True), (64, False), (256, True)])
@pytest.mark.parametrize("count", [2, 40])
def test_region_and_page_sizes(block, rt, D, int8, count):
    check([3 * block + 5, 9, block, 2 * block - 1, 2000], D=D, int8=int8, block=block, span=8, G=2, H=4, regions=(count, rt), gate=count == 2)


def test_a_few_rows_with_many_regions():
    check([9000], G=1, H=16, D=192, block=64, span=64, regions=(1024, 8))
    check([20000, 300], G=2, H=4, D=128, block=32, span=32, int8=True, ql=2, regions=(300, 64), gate=True)


def test_many_rows():
    r = random.Random(2)
    check([r.randint(1, 600) for _ in range(300)], G=2, H=4, D=64, block=16, regions=(20, 8))
    check([r.randint(1, 600) for _ in range(150)], G=2, H=8, D=192, block=16, ql=2, int8=True, regions=(40, 16))


@pytest.mark.parametrize("int8", [False, True])
def test_long_lists_of_short_contexts(int8):
    """Rows enough for their lists to be looked at first: most of a list is -1, at its end, at its beginning, between,
    or past the row's position; some rows are full, some empty, some inactive."""
    r = random.Random(7)
    p = Problem([r.choice((1, 30, 200, 900, 1500)) for _ in range(120)], G=2, H=4, D=64, block=16, int8=int8, ql=2, regions=(12, 8))
    ids = torch.full((480, 1100), -1, dtype=torch.int32, device="cuda")
    for k in range(480):
        at = (0, 1088, 500 + k, 128 * (k % 8) + k % 3)[k % 4]
        ids[k, at:at + 12] = p.regions[k]
    ids[5::40, 1099] = 10 ** 8                                          # past any position
    p.regions = ids
    p.active[::7] = False
    p.check(*p.run(regions=True), regions=True)
    left = p.query.clone() * 3, torch.full(p.query.shape[:2], 5.0, device="cuda")
    out, lse = p.run(regions=True, out=left[0].clone(), lse=left[1].clone(), clear_inactive=False)
    p.check(out, lse, regions=True, left=left)
    p.regions = ids.clone()
    p.regions[3, 1090] = -2
    p.active[3] = True
    out, lse = p.run(regions=True, flags=sda.FLAG_BOUNDS)
    p.regions[3, 1090] = -1
    p.check(out, lse, regions=True)
    p.regions[:] = -1
    out, lse = p.run(regions=True)
    assert (out.view(torch.int16) == 0).all() and (lse == -float("inf")).all()


def test_rows_that_see_nothing():
    """Inactive rows, rows without regions, rows whose regions lie past their position, and no regions at all."""
    for count in (6, 70):
        p = Problem([40, 300, 1, 90], G=2, H=4, D=64, block=16, regions=(count, 8), spare=2)
        p.active[:] = torch.tensor([1, 0, 1, 1, 1, 1, 0, 1], device="cuda", dtype=torch.bool)
        p.regions[2] = -1
        p.regions[3] = torch.where(p.regions[3] >= 0, 37, -1)
        p.positions[3] = 290
        p.check(*p.run(regions=True), regions=True)
        left = p.query.clone() * 3, torch.full(p.query.shape[:2], 5.0, device="cuda")
        out, lse = p.run(regions=True, out=left[0].clone(), lse=left[1].clone(), clear_inactive=False)
        p.check(out, lse, regions=True, left=left)
        assert torch.equal(lse[~p.active], left[1][~p.active])
    p.regions = p.regions[:, :0]
    out, lse = p.run(regions=True)
    assert (out.view(torch.int16) == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("count", [4, 80])
def test_bad_regions_and_pages(count):
    p = Problem([900], G=1, H=4, D=64, block=16, regions=(count, 8))
    p.active[:] = True
    want = [x.clone() for x in p.run(regions=True)]
    more = torch.tensor([[-7, -1, -2 ** 31, 0]], dtype=torch.int32, device="cuda")
    ids = p.regions
    p.regions = torch.cat([ids, more[:, :3]], 1)
    out, lse = p.run(regions=True, flags=sda.FLAG_BOUNDS)
    assert torch.allclose(out.float(), want[0].float(), atol=2e-2) and torch.allclose(lse, want[1], atol=1e-4)
    p.regions, p.positions = ids.clone(), p.positions + 100000          # sees all; a region past the table
    p.regions[0, 0] = 12500
    p.run(regions=True, flags=sda.FLAG_BOUNDS)
    p.regions[0, 0] = 2 ** 31 - 1                                       # past any position: not looked at
    p.run(regions=True)
    p.table[0, :] = 10 ** 6                                             # nothing is there: zeros
    out, lse = p.run(regions=True, flags=sda.FLAG_BOUNDS)
    assert (out == 0).all() and (lse == -float("inf")).all()


def test_regions_of_the_plain_cache():
    """E4M3 with one scale everywhere: what sparse_decode_attention gives, up to its own rounding (weights of 11 bits
    that reach 2^8 of the running maximum's, beside one bf16 step)."""
    p = Problem([5000, 300, 41], G=2, H=8, D=192, block=64, span=64, spare=3, scale_std=0.0, regions=(30, 64))
    one = torch.tensor([0.01], device="cuda")
    p.scales.fill_(0.01)
    p.cache[(p.cache & 0x7F) == 0x7F] = 0x30
    out, _ = p.run(regions=True)
    plain = torch.empty_like(out)
    sda.sparse_decode_attention(p.query, p.cache, p.regions, p.table, p.positions, p.active, plain, scale=p.scale, k_scale=one,
                                v_scale=one, region_tokens=64)
    assert ((out.double() - plain.double()).abs() <= 2 * (2.0 ** -8 * plain.double().abs() + 0.01 * 448 * 2.0 ** -11)).all()


# ---------------------------------------------------------------------------- calls


@pytest.mark.parametrize("regions", [None, (64, 8)])
def test_equal_inputs_give_equal_bits(regions):
    """Eager, on another stream, with the default workspace, and captured beside a graph with one of its own."""
    a = Problem([4000, 9, 1200, 800], G=2, H=8, D=128, block=32, span=16, int8=True, regions=regions, gate=True)
    b = Problem([700, 5000], G=1, H=16, D=192, block=64, span=32, regions=regions)
    by = regions is not None
    want = [p.run(regions=by) for p in (a, b)]
    for x, y in zip(want, [p.run(regions=by) for p in (a, b)]):
        assert torch.equal(x[0], y[0]) and torch.equal(x[1], y[1])
    other = torch.cuda.Stream()
    graphs, outs = [], []
    call = lambda p, out, lse, **kw: (                                 # noqa: E731
        sda.sparse_decode_quantised_attention(p.query, p.cache, p.scales, p.regions, p.table, p.positions, p.active, out, lse=lse,
                                              scale=p.scale, query_len=p.ql, gate=p.gate, region_tokens=p.rt, **kw) if by else
        sda.sparse_decode_quantised_paged_attention(p.query, p.cache, p.scales, p.table, p.seq_lens, out, lse=lse, scale=p.scale,
                                                    query_len=p.ql, gate=p.gate, **kw))
    for p in (a, b):
        outs.append([(torch.zeros_like(p.query), torch.zeros(p.query.shape[:2], device="cuda")) for _ in range(3)])
    torch.cuda.synchronize()
    for p, o in zip((a, b), outs):
        call(p, *o[0])
        call(p, *o[1], stream=other)
    torch.cuda.synchronize()
    for p, o in zip((a, b), outs):
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call(p, *o[2])
    for _ in range(3):
        with torch.cuda.stream(other):
            graphs[0].replay()
        graphs[1].replay()
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        assert all(torch.equal(x[0], w[0]) and torch.equal(x[1], w[1]) for x in o)


def test_nothing_to_do():
    p = Problem([], G=2, H=4, D=64)
    p.run()
    p.rt, p.regions = 8, torch.zeros(0, 5, dtype=torch.int32, device="cuda")
    p.positions, p.active = torch.zeros(0, dtype=torch.int32, device="cuda"), torch.zeros(0, dtype=torch.bool, device="cuda")
    p.run(regions=True)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("peak", [0.0, 3.0])
def test_long_contexts_keep_their_mean(int8, peak):
    """Rows that weigh 100,000 tokens nearly alike, each unit one worker's from its first tile to its last: the mean of
    values without one is small beside them, and so is its error (in steps of the elements: 2^-11 of each weight, without
    a sign, and 2^-20 for sums in fp32)."""
    G, D, B, n, requests = 8, 64, 128, 100000, 200
    width = -(-n // B)
    gen = torch.Generator(device="cuda").manual_seed(1)
    # one request's pages for all of them: every unit has the same tokens
    raw = torch.randint(-100, 101, (width, 1, B, 2 * D), generator=gen, device="cuda")
    cache = (raw.to(torch.int8) if int8 else raw.float().to(torch.float8_e4m3fn).view(torch.uint8)).expand(width, G, B, 2 * D).contiguous()
    scales = torch.ones(width, G, 1, 2, device="cuda")
    table = torch.arange(width, dtype=torch.int32, device="cuda").expand(requests, width)
    query = torch.zeros(requests * G, 1, D, dtype=torch.bfloat16, device="cuda")
    query[:, :, 0] = peak
    out = torch.empty_like(query)
    lse = torch.empty(requests * G, 1, device="cuda")
    sda.sparse_decode_quantised_paged_attention(query, cache, scales, table, torch.full((requests,), n, dtype=torch.int32, device="cuda"),
                                                out, scale=0.01, lse=lse)
    x = (cache if int8 else cache.view(torch.float8_e4m3fn).float())[:, 0].double().reshape(-1, 2 * D)[:n]
    w = torch.softmax(x[:, 0] * peak * float(np.float32(0.01)), 0)
    want = w @ x[:, D:]
    far = (out[:, 0].double() - want).abs().amax(0)
    # weights' roundings have no sign of their own: 2^-11 / sqrt(tokens that count) of the values' size, six times over
    spread = torch.sqrt((w * w) @ (x[:, D:] ** 2))
    assert (far <= want.abs() * 2.0 ** -8 + 6 * spread * 2.0 ** -11 + 100 * 2.0 ** -15).all(), far.max().item()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,H,ql", [(64, 16, 1), (128, 5, 1), (192, 16, 2), (192, 8, 1), (256, 3, 4), (256, 16, 2), (64, 1, 1)])
@pytest.mark.parametrize("lens,G", [([1200], 4), ([4000, 0, 3000, 7], 4), ([700, -1, 650], 12), ([2000], 1), ([257, 33], 38), ([9000, 0], 2)])
def test_few_units_by_clusters(lens, G, D, H, ql, int8):
    """From two to eight CTAs a unit, some of them or all of their workers without a tile; lengths of 0 and below."""
    check(lens, G=G, H=H, ql=ql, D=D, int8=int8, block=32, span=16, gate=D == 192, scale_std=1.0)
    check(lens, G=G, H=H, ql=ql, D=D, int8=int8, block=24, span=8, spare=5)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,H", [(64, 16), (128, 5), (192, 16), (256, 1)])
def test_few_rows_of_regions_by_clusters(D, H, int8):
    for count, rt in ((40, 64), (33, 8), (150, 16), (9, 128)):
        check([3000, 500, 9], G=2, H=H, D=D, int8=int8, block=32, span=16, regions=(count, rt), gate=True)
    p = check([5000], G=1, H=H, D=D, int8=int8, block=64, span=64, regions=(64, 64))
    left = p.query.clone() * 3, torch.full(p.query.shape[:2], 5.0, device="cuda")
    for on in (False, True):
        p.active[:] = on
        out, lse = p.run(regions=True, out=left[0].clone(), lse=left[1].clone(), clear_inactive=False)
        p.check(out, lse, regions=True, left=left)
    p.regions[:] = -1
    out, lse = p.run(regions=True)
    assert (out.view(torch.int16) == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,G", [([160, 90], 1), ([1600, 200], 2), ([40000, 3000], 2)])
def test_tables_too_narrow_and_bad_pages(lens, G, int8):
    """A length past the table counts as what the table holds, and a page outside the cache is left out, with a flag: by a
    CTA alone, a cluster and the line."""
    p = Problem(lens, G=G, H=8, D=128, block=16, span=8, int8=int8)
    whole = p.table
    p.table = whole[:, :-2]
    out, lse = p.run(flags=sda.FLAG_BOUNDS)
    held = 16 * p.table.shape[1]
    narrow = p.lens
    p.lens = [min(n, held) for n in narrow]
    p.check(out, lse)
    p.lens, p.table = narrow, whole.clone()
    p.check(*p.run())
    p.table[0, 0], p.table[1, 1] = -1, 10 ** 7
    out, lse = p.run(flags=sda.FLAG_BOUNDS)
    assert torch.isfinite(out).all() and torch.isfinite(lse).all()
    # the same requests without those pages' tokens
    p.host_cache, p.host_scales = p.cache.cpu(), p.scales.cpu()
    for r, gone in ((0, range(0, 16)), (G, range(16, 32))):
        k, v, top = p.row(r, False)
        keep = torch.tensor([t not in gone for t in range(len(k))])
        x = p.query[r].cpu().double()
        o, _, spread, slack = quant_util.attend(x, k[keep], v[keep], float(np.float32(p.scale)))
        bound = quant_util.attention_bound(o, spread, slack, top * (127 if int8 else 448), len(k))
        assert ((out[r].cpu().double() - o).abs() <= bound).all()


@pytest.mark.parametrize("int8", [False, True])
def test_pages_past_32_bits(int8):
    """Pages whose bytes lie more than 2^32 behind the first, whole and by regions."""
    G, B, D, pages, n = 8, 128, 256, 9000, 300                          # 4.7 GB
    cache = torch.zeros(pages, G, B, 2 * D, dtype=torch.int8 if int8 else torch.uint8, device="cuda")
    scales = torch.zeros(pages, G, B // 64, 2, device="cuda")
    gen = torch.Generator(device="cuda").manual_seed(4)
    ids = [8999, 8400, 8998]
    cache[ids] = torch.randint(0, 0x7E, (3, G, B, 2 * D), generator=gen, device="cuda").to(cache.dtype)
    scales[ids] = torch.rand(3, G, B // 64, 2, generator=gen, device="cuda") * 0.02 + 0.01
    near_cache, near_scales = cache[ids].contiguous(), scales[ids].contiguous()
    query = torch.randn(G, 4, D, generator=gen, device="cuda").bfloat16()
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    outs = []
    for c, s, table in ((cache, scales, i32([ids])), (near_cache, near_scales, i32([[0, 1, 2]]))):
        outs.append([torch.zeros_like(query) for _ in range(2)])
        sda.sparse_decode_quantised_paged_attention(query, c, s, table, i32([n]), outs[-1][0], scale=0.06)
        sda.sparse_decode_quantised_attention(query, c, s, i32([[4, 0, 2]] * G), table, i32([n - 1] * G),
                                              torch.ones(G, dtype=torch.bool, device="cuda"), outs[-1][1], scale=0.06, region_tokens=64)
    for a, b in zip(*outs):
        assert torch.equal(a, b) and a.abs().sum() > 0

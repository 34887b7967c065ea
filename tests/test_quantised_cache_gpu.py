"""Keys and values into a quantised cache and back, against the plain forms of quant_util: elements,
scales and what is read have to be equal."""
import random

import numpy as np
import pytest
import torch

import quant_util
import sparse_decode_attention_02_gb300 as sda

pytestmark = pytest.mark.gpu


class Cache:
    """A quantised cache on the GPU (its bytes anything at first) and the plain one that follows it."""

    def __init__(self, *, pages=40, G=2, B=32, S=16, D=64, int8=False, pad=(0, 0, 0), scale_pad=(0, 0, 0), seed=0):
        self.G, self.B, self.S, self.D, self.int8 = G, B, S, D, int8
        gen = torch.Generator().manual_seed(seed)
        raw = torch.randint(0, 256, (pages + pad[0], G + pad[1], B + pad[2], 2 * D), generator=gen, dtype=torch.uint8)
        if not int8:
            raw[(raw & 0x7F) == 0x7F] = 0x55               # NaN codes compare with nothing
        self.store = raw.cuda()
        self.cache = (self.store.view(torch.int8) if int8 else self.store)[:pages, :G, :B]
        self.scale_store = torch.full((pages + scale_pad[0], G + scale_pad[1], B // S + scale_pad[2], 2), 7.5, device="cuda")
        self.scales = self.scale_store[:pages, :G, :B // S]
        self.elements = quant_util.values(raw, int8)[:pages, :G, :B].copy()
        self.plain_scales = self.scales.cpu().numpy().copy()
        self.ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
        self.start = self.store.clone(), self.scale_store.clone()

    def append(self, key, value, slots, flags=None, **kw):
        slots = torch.as_tensor(slots, dtype=torch.int64)
        want = quant_util.append(key, value, slots.tolist(), self.elements, self.plain_scales, self.int8)
        sda.sparse_decode_quantised_append(key.cuda(), value.cuda(), slots.cuda(), self.cache, self.scales, workspace=self.ws, **kw)
        torch.cuda.synchronize()
        got = sda.read_errors(self.ws, clear=True)
        assert got == want and (flags is None or got == flags)
        self.check()

    def check(self):
        assert np.array_equal(self.scales.cpu().numpy(), self.plain_scales, equal_nan=True)
        assert np.array_equal(quant_util.values(self.cache.cpu().contiguous(), self.int8), self.elements, equal_nan=True)
        inside = torch.zeros(self.store.shape[:3], dtype=torch.bool)
        inside[:self.cache.shape[0], :self.G, :self.B] = True
        assert torch.equal(self.store.cpu()[~inside], self.start[0].cpu()[~inside])       # what lies between is as it was
        inside = torch.zeros(self.scale_store.shape[:3], dtype=torch.bool)
        inside[:self.scales.shape[0], :self.G, :self.scales.shape[2]] = True
        assert torch.equal(self.scale_store.cpu()[~inside], self.start[1].cpu()[~inside])

    def rows(self, n, gen, size=1.0):
        """Keys and values of n rows as views of one projection's output, each row of a size of its own."""
        x = torch.randn(n, 3 * self.G * self.D + 8, generator=gen)
        x = (x * torch.exp(torch.randn(n, 1, generator=gen)) * size).bfloat16()
        return (x[:, a * self.G * self.D:(a + 1) * self.G * self.D].unflatten(1, (self.G, self.D)) for a in (0, 2))


def slots_of(page, first, n, B):
    """Slots of tokens first .. first + n - 1 of a request whose pages are `page`."""
    return [page[t // B] * B + t % B for t in range(first, first + n)]


def filled(c, steps, gen):
    """Requests that grow by `steps[k][q]` tokens in step k, packed, with padding rows behind."""
    n = len(steps[0])
    ids = list(range(c.cache.shape[0]))
    random.Random(3).shuffle(ids)
    need = [-(-sum(s[q] for s in steps) // c.B) for q in range(n)]
    pages = [[ids.pop() for _ in range(k)] for k in need]
    lens = [0] * n
    for step in steps:
        slots = []
        for q, k in enumerate(step):
            slots += slots_of(pages[q], lens[q], k, c.B)
            lens[q] += k
        slots += [-1] * 3
        c.append(*c.rows(len(slots), gen), slots)
    return pages, lens


STEPS = [[37, 5, 70, 0], [1, 1, 1, 1], [0, 1, 1, 1], [3, 2, 20, 2], [1, 1, 1, 1], [1, 1, 1, 1]]


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,G,B,S", [(16, 1, 8, 8), (64, 3, 24, 8), (128, 2, 32, 32), (192, 2, 48, 24), (192, 1, 64, 64), (256, 2, 16, 8),
                                     (208, 1, 128, 128), (512, 1, 256, 256), (512, 2, 40, 40)])
def test_requests_grow(D, G, B, S, int8):
    c = Cache(D=D, G=G, B=B, S=S, int8=int8)
    filled(c, STEPS, torch.Generator().manual_seed(D + B))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 63, 64, 65, 200, 1500])
def test_row_counts(rows, int8):
    """From one row to more than CTAs share: every split of rows over CTAs and warps, runs across chunks."""
    c = Cache(pages=70, B=32, S=16, D=128, int8=int8)
    gen = torch.Generator().manual_seed(rows)
    pages = list(range(70))
    c.append(*c.rows(rows, gen), slots_of(pages, 5, rows, 32))
    c.append(*c.rows(1, gen), slots_of(pages, 5 + rows, 1, 32))


@pytest.mark.parametrize("int8", [False, True])
def test_scales_grow_token_by_token(int8):
    """Each token twice as large as the last: the scale grows at every step, and elements are rounded again and again."""
    c = Cache(pages=3, G=1, B=32, S=32, D=64, int8=int8)
    gen = torch.Generator().manual_seed(1)
    for t in range(32):
        key, value = c.rows(1, gen, size=1.7 ** t)
        c.append(key, value, [32 + t])
    c.append(*c.rows(1, gen, size=1e-3), [32])             # the page's next owner begins with a scale of its own
    assert c.plain_scales[1, 0, 0].max() < 1e-2


@pytest.mark.parametrize("int8", [False, True])
def test_sizes_at_the_ends(int8):
    """Zeros, the smallest and the largest bf16 values, and those at a border of the scale."""
    c = Cache(pages=12, G=1, B=8, S=8, D=16, int8=int8)
    sizes = [0.0, 2.0 ** -133, 2.0 ** -126, 1e-30, 448.0, 449.0, 446.0, 127.0, 3.0, 2.0 ** 120, 3.3895313892515355e38]
    key = torch.zeros(len(sizes), 1, 16, dtype=torch.bfloat16)
    key[:, 0, 3] = torch.tensor(sizes, dtype=torch.float64).bfloat16()
    key[:, 0, 4:12] = key[:, 0, 3:4] * (torch.arange(8) / 9).bfloat16()
    c.append(key, -key, [8 * i for i in range(len(sizes))])
    assert (c.plain_scales[:len(sizes)] >= 2.0 ** -126).all()


@pytest.mark.parametrize("int8", [False, True])
def test_what_is_not_finite(int8):
    c = Cache(pages=4, G=2, B=16, S=8, D=64, int8=int8)
    gen = torch.Generator().manual_seed(2)
    c.append(*c.rows(5, gen), range(5), flags=0)
    key, value = c.rows(6, gen)
    key, value = key.clone(), value.clone()
    key[0, 0, 5], key[3, 1, 63], value[2, 0, 0] = float("inf"), float("nan"), float("-inf")
    value[5, 1] = float("nan")
    c.append(key, value, range(5, 11), flags=sda.FLAG_NONFINITE)
    assert np.isfinite(c.scales.cpu().numpy()).all()


@pytest.mark.parametrize("slots", [[3, 5, 6, 7], [4, 4, 5], [3, 2, 1], [3, 4, 1 << 40, 12], [-2, 3, 4], [640, 3], [3, -1, 12],
                                   [0, 1, 2, 9, 10, 8, 16, 17], [639], [15, 16, 17, 40, 42, 48]])
def test_rows_out_of_order_and_out_of_the_cache(slots):
    """Left out with a flag, and the rest is as if they were not there."""
    c = Cache(pages=40, B=16, S=8)
    c.append(*c.rows(len(slots), torch.Generator().manual_seed(4)), slots)


@pytest.mark.parametrize("int8", [False, True])
def test_strides(int8):
    c = Cache(G=2, D=64, int8=int8, pad=(1, 2, 3), scale_pad=(2, 1, 1))
    pages, lens = filled(c, STEPS, torch.Generator().manual_seed(5))
    wide = torch.full((sum(lens) + 4, 5, 3 * 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    key, value = wide[:, 1:3, 64:128], wide[:, 3:5, :64]
    check_read(c, pages, lens, None, key=key, value=value)
    rest = wide.clone()
    rest[:, 1:3, 64:128] = rest[:, 3:5, :64] = float("nan")
    assert rest.isnan().all()


def test_nothing_to_do():
    c = Cache()
    gen = torch.Generator().manual_seed(6)
    c.append(*c.rows(0, gen), [])
    c.append(*c.rows(9, gen), [-1] * 9, flags=0)
    sda.sparse_decode_quantised_read(c.cache, c.scales, torch.zeros(0, 0, dtype=torch.int32, device="cuda"),
                                     torch.zeros(1, dtype=torch.int32, device="cuda"),
                                     *(torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv"))


def check_read(c, pages, lens, first, *, key=None, value=None, rows=None, base=0, flags=0):
    counts = [n - (first[q] if first else 0) for q, n in enumerate(lens)]
    starts = np.concatenate([[base], base + np.cumsum(counts)]).astype(int).tolist()
    rows = starts[-1] + 4 if rows is None else rows
    width = max([1] + [len(p) for p in pages])
    table = torch.tensor([list(p) + [-1] * (width - len(p)) for p in pages], dtype=torch.int32).view(len(pages), width)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    out = {}
    for name, t in (("key", key), ("value", value)):
        out[name] = torch.full((rows, c.G, c.D), float("nan"), dtype=torch.bfloat16, device="cuda") if t is None else t
    sda.sparse_decode_quantised_read(c.cache, c.scales, table.cuda(), i32(starts), out["key"], out["value"],
                                     first_tokens=None if first is None else i32(first), workspace=c.ws)
    torch.cuda.synchronize()
    want, told = quant_util.read(c.elements, c.plain_scales, table.tolist(), starts, first, rows)
    assert sda.read_errors(c.ws, clear=True) == told == flags
    got = torch.cat([out["key"], out["value"]], -1).cpu()
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(), want.nan_to_num())


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,G,B,S", [(16, 1, 8, 8), (64, 3, 24, 8), (128, 2, 32, 32), (192, 2, 48, 24), (208, 1, 128, 128), (512, 2, 40, 40)])
def test_read_back(D, G, B, S, int8):
    c = Cache(D=D, G=G, B=B, S=S, int8=int8)
    pages, lens = filled(c, STEPS, torch.Generator().manual_seed(D))
    check_read(c, pages, lens, None)
    check_read(c, pages, lens, [n // 3 for n in lens], base=5)          # rows before the first request are left as they were
    check_read(c, pages, lens, lens, rows=9)                            # nothing of any request


def test_read_of_one_side():
    c = Cache()
    pages, lens = filled(c, STEPS, torch.Generator().manual_seed(1))
    rows, table = sum(lens), torch.tensor([p + [-1] * (9 - len(p)) for p in pages], dtype=torch.int32, device="cuda")
    starts = torch.tensor([0] + np.cumsum(lens).tolist(), dtype=torch.int32, device="cuda")
    both = [torch.empty(rows, 2, 64, dtype=torch.bfloat16, device="cuda") for _ in range(4)]
    sda.sparse_decode_quantised_read(c.cache, c.scales, table, starts, both[0], both[1])
    sda.sparse_decode_quantised_read(c.cache, c.scales, table, starts, both[2], None)
    sda.sparse_decode_quantised_read(c.cache, c.scales, table, starts, None, both[3])
    assert torch.equal(both[0], both[2]) and torch.equal(both[1], both[3])


@pytest.mark.parametrize("requests,rows", [(1, 900), (239, 700), (300, 2000), (5000, 3000), (70000, 900)])
def test_read_finds_its_requests(requests, rows):
    """Many requests, most of them empty, and long ones between them."""
    c = Cache(pages=64, G=1, B=16, S=16, D=64)
    c.store.copy_(torch.randint(0, 0x7E, c.store.shape, dtype=torch.uint8, device="cuda"))
    c.elements = quant_util.values(c.cache.cpu(), False)
    r = random.Random(requests)
    lens = [0] * requests
    left = rows
    for q in sorted(r.sample(range(requests), min(requests, 60))):
        lens[q] = min(left, r.choice((1, 2, 17, 100, 400)))
        left -= lens[q]
    pages = [[r.randrange(64) for _ in range(-(-n // 16))] for n in lens]
    check_read(c, pages, lens, None, rows=rows)


def test_read_of_bad_pages():
    c = Cache(pages=6, B=16, S=16)
    pages = [[0, -1, 2], [6, 3], [1]]
    check_read(c, pages, [40, 20, 16], None, flags=sda.FLAG_BOUNDS)
    check_read(c, [[0, 1, 2]], [60], None, flags=sda.FLAG_BOUNDS)       # past the table
    check_read(c, [[0, 1, 2]], [20], [-3], flags=sda.FLAG_BOUNDS)       # before the first token


@pytest.mark.parametrize("int8", [False, True])
def test_places_past_32_bits(int8):
    """Pages whose bytes lie more than 2^32 behind the first."""
    G, B, D, pages = 8, 128, 256, 9000                                  # 4.7 GB
    cache = torch.zeros(pages, G, B, 2 * D, dtype=torch.int8 if int8 else torch.uint8, device="cuda")
    scales = torch.zeros(pages, G, B // 64, 2, device="cuda")
    gen = torch.Generator().manual_seed(8)
    x = torch.randn(130, 2, G, D, generator=gen).bfloat16().cuda()
    ids = [8999, 8500]
    slots = torch.tensor(slots_of(ids, 0, 130, B), device="cuda")
    sda.sparse_decode_quantised_append(x[:, 0], x[:, 1], slots, cache, scales)
    out = torch.empty(2, 130, G, D, dtype=torch.bfloat16, device="cuda")
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    sda.sparse_decode_quantised_read(cache, scales, i32([ids]), i32([0, 130]), out[0], out[1])
    want = x.transpose(0, 1).double()
    # half a step of the scale, or of E4M3 (2^-4; 2^-10 scales below its normal numbers), and the bf16 rounding
    top = scales[ids].double().amax()
    bound = (top / 2 if int8 else want.abs() * 2.0 ** -4 + top * 2.0 ** -10) + want.abs() * 2.0 ** -8 + top * 2.0 ** -9
    assert ((out.double() - want).abs() <= bound * (1 + 2.0 ** -20)).all()
    assert not scales[:8500].any()


@pytest.mark.parametrize("int8", [False, True])
def test_elements_are_near(int8):
    """What is read is off by half a step at most, in 64 bits and from the values alone."""
    c = Cache(pages=40, B=64, S=32, D=192, G=2, int8=int8)
    gen = torch.Generator().manual_seed(9)
    key, value = c.rows(1000, gen)
    ids = list(range(40))
    c.append(key, value, slots_of(ids, 0, 1000, 64))
    got = [torch.empty(1000, 2, 192, dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    sda.sparse_decode_quantised_read(c.cache, c.scales, i32([ids]), i32([0, 1000]), *got)
    for kv, x in enumerate((key, value)):
        x = x.double()
        s = torch.from_numpy(c.plain_scales[..., kv]).double().transpose(1, 2).reshape(-1, 2)       # [blocks, G]
        s = s.repeat_interleave(32, 0)[:1000, :, None]
        half = s / 2 if int8 else torch.maximum(x.abs() * 2.0 ** -4, s * 2.0 ** -10)
        far = (got[kv].cpu().double() - x).abs()
        assert (far <= half * (1 + 2.0 ** -8) + x.abs() * 2.0 ** -8).all()


def test_captured_and_on_another_stream():
    """A step captured with the default workspace and replayed on new rows is the same as eager ones; so is a
    call on a stream of its own."""
    def fresh():
        return Cache(pages=8, G=2, B=32, S=16, D=128)

    gen = torch.Generator().manual_seed(10)
    rows = [tuple(x.contiguous().cuda() for x in fresh().rows(20, gen)) for _ in range(3)]
    i32 = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    slots = [torch.tensor(slots_of([3, 1, 5], 20 * k, 20, 32), device="cuda") for k in range(3)]
    eager, c = fresh(), fresh()
    table, starts = i32([[3, 1, 5]]), i32([0, 60])
    outs = [[torch.zeros(60, 2, 128, dtype=torch.bfloat16, device="cuda") for _ in "kv"] for _ in range(3)]
    for (k, v), at in zip(rows, slots):
        sda.sparse_decode_quantised_append(k, v, at, eager.cache, eager.scales)
    sda.sparse_decode_quantised_read(eager.cache, eager.scales, table, starts, *outs[0])
    k, v, at = rows[0][0].clone(), rows[0][1].clone(), slots[0].clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sda.sparse_decode_quantised_append(k, v, at, c.cache, c.scales)
        sda.sparse_decode_quantised_read(c.cache, c.scales, table, starts, *outs[1])
    for j in range(3):
        k.copy_(rows[j][0]), v.copy_(rows[j][1]), at.copy_(slots[j])
        graph.replay()
    other, d = torch.cuda.Stream(), fresh()
    other.wait_stream(torch.cuda.current_stream())
    for (k, v), at in zip(rows, slots):
        sda.sparse_decode_quantised_append(k, v, at, d.cache, d.scales, stream=other)
    sda.sparse_decode_quantised_read(d.cache, d.scales, table, starts, *outs[2], stream=other)
    torch.cuda.synchronize()
    for x in (c, d):
        assert torch.equal(x.store, eager.store) and torch.equal(x.scale_store, eager.scale_store)
    assert all(torch.equal(a, b) for pair in outs[1:] for a, b in zip(pair, outs[0]))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D,G,S,rows", [(64, 4, 16, 6000), (64, 4, 64, 6000), (16, 2, 512, 1500), (16, 8, 512, 3000)])
def test_long_prompts(D, G, S, rows, int8):
    """Rows enough for CTAs of 64 each, and blocks longer than the window that a CTA looks at."""
    c = Cache(pages=rows // S + 3, G=G, B=S, S=S, D=D, int8=int8)
    gen = torch.Generator().manual_seed(rows + D)
    pages = list(range(c.cache.shape[0]))
    random.Random(1).shuffle(pages)
    c.append(*c.rows(rows, gen), slots_of(pages, 3, rows, S))
    c.append(*c.rows(5, gen), slots_of(pages, 3 + rows, 5, S))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("D", [272, 416, 512])
def test_wide_heads_of_many_requests(D, int8):
    """A warp for each of many runs, fewer threads than a row has pieces."""
    c = Cache(pages=60, G=2, B=16, S=16, D=D, int8=int8)
    filled(c, [[2] * 40, [1] * 40, [5 if q % 3 else 0 for q in range(40)]], torch.Generator().manual_seed(D))


def test_a_block_of_two_lists_of_rows():
    """A long run that stops inside the window and one that stops behind it, each followed by rows that are left out."""
    c = Cache(pages=4, G=1, B=512, S=512, D=16)
    gen = torch.Generator().manual_seed(3)
    for stop in (100, 255, 256, 257, 300, 479):
        slots = list(range(512, 512 + stop)) + list(range(512 + stop + 1, 1024)) + [0, 1]
        c.append(*c.rows(len(slots), gen), slots, flags=sda.FLAG_BOUNDS)

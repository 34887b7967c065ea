"""The quantised cache as it is used: tables from lengths, keys turned in place, written with scales that follow
them, attended over whole and by selected regions, and read back for a prompt's attention, step after step."""
import numpy as np
import pytest
import torch

import quant_util
import sparse_decode_attention_02_gb300 as sda
import step_util

pytestmark = pytest.mark.gpu
B, S, G, H, D, RT = 32, 16, 2, 4, 128, 8


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Request slots, a page pool and a quantised cache on the GPU; the plain forms follow on the CPU."""

    def __init__(self, slots, pages, width, int8):
        self.int8, self.n = int8, slots
        order = np.random.default_rng(3).permutation(pages)
        self.lens, self.state = i32([0] * slots), i32([0, pages])
        self.ring, self.table = i32(order.tolist()), i32([[-1] * width] * slots)
        self.cache = torch.full((pages, G, B, 2 * D), 0x7F, dtype=torch.uint8, device="cuda")
        self.cache = self.cache.view(torch.int8) if int8 else self.cache
        self.scales = torch.full((pages, G, B // S, 2), float("nan"), device="cuda")
        self.elements = quant_util.values(self.cache.cpu(), int8)
        self.plain_scales = self.scales.cpu().numpy().copy()
        self.inv = (10000.0 ** (-torch.arange(D // 2).double() / (D // 2))).float().cuda()
        self.plain = dict(context=[0] * slots, ring=order.tolist(), state=[0, pages], table=np.full((slots, width), -1))
        need = max(sda.paged_workspace_bytes(H, 3, D), sda.paged_workspace_bytes(H, 1, D), sda.quantised_workspace_bytes(3 * G * slots, H, D))
        self.ws = torch.zeros(need, dtype=torch.uint8, device="cuda")

    def step(self, new, rows, per_request, gen):
        """Plans, turns and appends; returns the turned queries after checking the cache."""
        want, flags = step_util.plan(self.plain["context"], new, B, self.plain["ring"], self.plain["state"],
                                     self.plain["table"], rows, per_request)
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        _, _, _, pos, _, _ = sda.sparse_decode_plan_step(
            self.lens, i32(new), self.ring, self.state, self.table, block_size=B, slots=slots,
            rows_per_request=per_request, seq_lens=self.lens, free_next=self.state, workspace=self.ws)
        qkv = (torch.randn(rows, (G * H + 2 * G) * D, generator=gen) * torch.exp(torch.randn(rows, 1, generator=gen))).bfloat16().cuda()
        qk, v = (x.unflatten(1, (-1, D)) for x in qkv.split([(G * H + G) * D, G * D], dim=1))
        sda.sparse_decode_rope_append(qk, None, None, pos[None], self.inv, slots, None, qk, workspace=self.ws)
        q, k = qk[:, :G * H], qk[:, G * H:]
        sda.sparse_decode_quantised_append(k, v, slots, self.cache, self.scales, workspace=self.ws)
        torch.cuda.synchronize()
        flags |= quant_util.append(k.cpu(), v.cpu(), want["slots"], self.elements, self.plain_scales, self.int8)
        assert sda.read_errors(self.ws, clear=True) == flags
        assert self.lens.tolist() == want["seq_lens"] and slots.tolist() == want["slots"]
        self.plain = dict(context=want["seq_lens"], ring=want["free_pages"], state=want["free_next"], table=want["table"])
        assert np.array_equal(self.scales.cpu().numpy(), self.plain_scales, equal_nan=True)
        assert np.array_equal(quant_util.values(self.cache.cpu(), self.int8), self.elements, equal_nan=True)
        return q

    def decoded(self, q, g):
        n = self.plain["context"][q]
        pages = self.plain["table"][q, :-(-n // B)].astype(int)
        s = np.repeat(self.plain_scales[pages, g], S, 1).astype(np.float64)[..., None]
        x = torch.from_numpy((self.elements[pages, g].reshape(-1, B, 2, D) * s).reshape(-1, 2, D)[:n])
        return x[:, 0], x[:, 1], float(s[:, :, 1].reshape(-1)[:n].max()) if n else 0.0

    def attend(self, q, query_len, seed):
        """The new tokens over the whole cache, then over every other region and their own."""
        rows = self.n * query_len * G
        query = q.reshape(rows, H, D)
        out, lse = torch.full_like(query, float("nan")), torch.empty(rows, H, device="cuda")
        sda.sparse_decode_quantised_paged_attention(query, self.cache, self.scales, self.table, self.lens, out, scale=D ** -0.5,
                                                    query_len=query_len, lse=lse, workspace=self.ws)
        pos = [self.plain["context"][r // (query_len * G)] - query_len + r // G % query_len for r in range(rows)]
        count = 1 + max(max(pos), 0) // RT
        ids = [[i if i <= p // RT and (i + r + seed) % 2 == 0 or p >= 0 and i == p // RT else -1 for i in range(count)]
               for r, p in enumerate(pos)]
        some = torch.full_like(query, float("nan"))
        sda.sparse_decode_quantised_attention(query, self.cache, self.scales, i32(ids), self.table, i32(pos),
                                              torch.tensor([p >= 0 for p in pos], device="cuda"), some, scale=D ** -0.5,
                                              query_len=query_len, region_tokens=RT, workspace=self.ws)
        torch.cuda.synchronize()
        assert sda.read_errors(self.ws, clear=True) == 0
        query, scale = query.cpu().double(), float(np.float32(D ** -0.5))
        for r, p in enumerate(pos):
            k, v, top = self.decoded(r // (query_len * G), r % G)
            every = torch.arange(max(p + 1, 0))
            chosen = torch.isin(every // RT, torch.tensor([i for i in ids[r] if i >= 0]))
            for got, t in ((out, every), (some, every[chosen])):
                o, _, spread, slack = quant_util.attend(query[r], k[t], v[t], scale)
                bound = quant_util.attention_bound(o, spread, slack, top * (127 if self.int8 else 448), len(t))
                assert ((got[r].cpu().double() - o).abs() <= bound).all()

    def read_back(self, first):
        """What each request holds from `first` on, as a prompt's attention would take it."""
        lens = self.plain["context"]
        first = [min(first, n) for n in lens]
        starts = np.concatenate([[0], np.cumsum([n - a for n, a in zip(lens, first)])]).tolist()
        key, value = (torch.full((starts[-1], G, D), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in "kv")
        sda.sparse_decode_quantised_read(self.cache, self.scales, self.table, i32(starts), key, value, first_tokens=i32(first),
                                         workspace=self.ws)
        torch.cuda.synchronize()
        want, flags = quant_util.read(self.elements, self.plain_scales, self.plain["table"].tolist(), starts, first, starts[-1])
        assert sda.read_errors(self.ws, clear=True) == flags == 0
        assert torch.equal(torch.cat([key, value], -1).cpu(), want)


@pytest.mark.parametrize("int8", [False, True])
def test_requests_come_and_go(int8):
    gen = torch.Generator().manual_seed(11)
    s = Server(6, 40, 12, int8)
    s.step([23, 0, 7, 100, 1, 0], 140, 0, gen)                         # prompts, packed
    for new in ([1, 0, 1, 1, 1, 0], [1, 0, 1, -1, 1, 0], [1, 0, 1, 0, 1, 0], [1, 1, 1, 1, 1, 1]):
        s.attend(s.step(new, 6, 1, gen), 1, 0)                         # one token each; slot 3 is released on the way
    s.read_back(9)
    s.step([0, 60, 0, 33, 0, 17], 120, 0, gen)                         # prompts of new requests, pages used again
    for new in ([3, 3, 1, 2, 3, 3], [1, 3, 2, -1, 3, 1]):              # up to three draft tokens
        s.attend(s.step(new, 18, 3, gen), 3, 1)
    s.read_back(0)
    s.step([0, 0, 0, 190, 0, 150], 400, 0, gen)
    s.attend(s.step([1] * 6, 6, 1, gen), 1, 0)


def test_a_whole_step_in_one_graph():
    """Plan, turn, append and both attentions captured once, replayed while the state on the GPU moves on,
    against the same steps run eagerly."""
    def fresh():
        s = Server(8, 64, 16, True)
        s.step([5, 40, 1, 90, 16, 15, 33, 2], 210, 0, torch.Generator().manual_seed(5))
        return s

    x = torch.randn(5, 8, (G * H + 2 * G) * D, generator=torch.Generator().manual_seed(6)).bfloat16().cuda()
    new, ids = i32([1] * 8), i32([[0, 3, 1, -1, 11]] * 16)
    qkv = torch.empty_like(x[0])
    qk, v = (y.unflatten(1, (-1, D)) for y in qkv.split([(G * H + G) * D, G * D], dim=1))

    def one(s, outs):
        slots = torch.empty(8, dtype=torch.int64, device="cuda")
        _, _, _, pos, _, _ = sda.sparse_decode_plan_step(s.lens, new, s.ring, s.state, s.table, block_size=B, slots=slots,
                                                         rows_per_request=1, seq_lens=s.lens, free_next=s.state)
        sda.sparse_decode_rope_append(qk, None, None, pos[None], s.inv, slots, None, qk)
        sda.sparse_decode_quantised_append(qk[:, G * H:], v, slots, s.cache, s.scales)
        query, at = qk[:, :G * H].reshape(16, H, D), pos.repeat_interleave(G)
        sda.sparse_decode_quantised_paged_attention(query, s.cache, s.scales, s.table, s.lens, outs[0], scale=D ** -0.5)
        sda.sparse_decode_quantised_attention(query, s.cache, s.scales, ids, s.table, at, at >= 0, outs[1], scale=D ** -0.5,
                                              region_tokens=RT)

    eager, captured = fresh(), fresh()
    outs = [[torch.zeros(16, H, D, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2)]
    graph = torch.cuda.CUDAGraph()
    qkv.copy_(x[0])
    with torch.cuda.graph(graph):
        one(captured, outs[1])
    for row in x:
        qkv.copy_(row)
        one(eager, outs[0])
        qkv.copy_(row)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(*outs)) and torch.isfinite(outs[0][0]).all()
        assert torch.equal(eager.cache, captured.cache) and torch.equal(eager.scales.nan_to_num(9), captured.scales.nan_to_num(9))
        assert torch.equal(eager.lens, captured.lens) and torch.equal(eager.table, captured.table)

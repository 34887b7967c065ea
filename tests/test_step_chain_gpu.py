"""The serving-step operators as they are used together: tables from lengths, rotary keys and values
into the pages, attention over them, step after step, requests coming and going."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import step_util

pytestmark = pytest.mark.gpu
KS, VS = 8.0 / 448.0, 6.0 / 448.0
B, G, H, D, ROT = 16, 2, 8, 192, 128


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Server:
    """Request slots, a page pool and a cache, all on the GPU; the plain forms follow on the CPU."""

    def __init__(self, slots, pages, width, fp8):
        self.fp8, self.n = fp8, slots
        self.lens, self.state = i32([0] * slots), i32([0, pages])
        order = np.random.default_rng(3).permutation(pages)
        self.ring, self.table = i32(order.tolist()), i32([[-1] * width] * slots)
        self.cache = torch.zeros(pages, G, B, 2 * D, dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
        self.cache.fill_(0x7F if fp8 else float("nan"))          # what was never written is not a number
        self.inv = (10000.0 ** (-torch.arange(ROT // 2).double() / (ROT // 2))).float().cuda()
        self.scales = dict(k_scale=torch.tensor([KS], device="cuda"), v_scale=torch.tensor([VS], device="cuda")) if fp8 else {}
        self.plain = dict(context=[0] * slots, ring=order.tolist(), state=[0, pages], table=np.full((slots, width), -1))
        self.ws = torch.zeros(sda.paged_workspace_bytes(H, 4, D), dtype=torch.uint8, device="cuda")

    def step(self, new, rows, per_request, gen):
        """Plans, rotates and appends; returns (query_out, tokens) after checking both."""
        want, flags = step_util.plan(self.plain["context"], new, B, self.plain["ring"], self.plain["state"],
                                     self.plain["table"], rows, per_request)
        slots = torch.empty(rows, dtype=torch.int64, device="cuda")
        _, starts, _, pos, owner, _ = sda.sparse_decode_plan_step(
            self.lens, i32(new), self.ring, self.state, self.table, block_size=B, slots=slots,
            rows_per_request=per_request, seq_lens=self.lens, free_next=self.state, workspace=self.ws)
        qkv = torch.randn(rows, (G * H + 2 * G) * D, generator=gen).bfloat16().cuda()
        q, k, v = (x.view(rows, -1, D) for x in qkv.split([G * H * D, G * D, G * D], dim=1))
        out = torch.zeros(rows, G * H, D, dtype=torch.bfloat16, device="cuda")
        sda.sparse_decode_rope_append(q, k, v, pos[None], self.inv, slots, self.cache, out, workspace=self.ws, **self.scales)
        torch.cuda.synchronize()
        assert sda.read_errors(self.ws, clear=True) == flags
        assert self.lens.tolist() == want["seq_lens"] and self.state.tolist() == want["free_next"]
        assert slots.tolist() == want["slots"] and np.array_equal(self.table.cpu().numpy(), want["table"])
        self.plain = dict(context=want["seq_lens"], ring=want["free_pages"], state=want["free_next"], table=want["table"])
        # every new token's key and value lie in their slot
        live = torch.tensor(want["slots"]) >= 0
        at = torch.tensor(want["slots"])[live]
        kr, size = step_util.rotate(k.cpu(), torch.tensor(want["positions"])[None], self.inv.cpu(), None)
        got = self.cache.cpu()[at // B, :, at % B]
        if self.fp8:
            got = step_util.e4m3_values(got)
            for x, y, s in ((kr[live], got[..., :D], KS), (v.cpu().double()[live], got[..., D:], VS)):
                x = x / float(torch.tensor(s, dtype=torch.float32))
                assert ((y - x).abs() <= x.abs() * 2.0 ** -4 + 2.0 ** -10 + 2.0 ** -16 / s).all()
        else:
            assert ((got[..., :D].double() - kr[live]).abs() <= kr[live].abs() * 2.0 ** -8 + size[live] * 2.0 ** -21).all()
            assert torch.equal(got[..., D:], v.cpu()[live])
        return out

    def attend(self, q, query_len):
        rows = self.n * query_len * G
        query = q.view(rows, H, D)
        out, lse = torch.full_like(query, float("nan")), torch.empty(rows, H, device="cuda")
        sda.sparse_decode_paged_attention(query, self.cache, self.table, self.lens, out, scale=D ** -0.5, query_len=query_len,
                                          lse=lse, workspace=self.ws, **self.scales)
        torch.cuda.synchronize()
        assert sda.read_errors(self.ws) == 0
        f = (float(torch.tensor(KS)), float(torch.tensor(VS))) if self.fp8 else (1.0, 1.0)
        o, l, spread, slack = step_util.paged_attention(query.cpu(), self.cache.cpu(), self.table.cpu(),
                                                        self.plain["context"], scale=float(np.float32(D ** -0.5)),
                                                        query_len=query_len, k_scale=f[0], v_scale=f[1])
        got = out.cpu().double()
        assert torch.isfinite(got).all()
        assert ((got - o).abs() <= step_util.attention_bound(o, spread, slack, self.fp8)).all()
        live = torch.isfinite(l)
        assert ((lse.cpu().double() - l).abs() <= slack + l.abs() * 2.0 ** -22 + 2.0 ** -18)[live].all()


@pytest.mark.parametrize("fp8", [False, True])
def test_requests_come_and_go(fp8):
    gen = torch.Generator().manual_seed(11)
    s = Server(6, 40, 12, fp8)
    s.step([23, 0, 7, 100, 1, 0], 140, 0, gen)                         # prompts, packed
    for new in ([1, 0, 1, 1, 1, 0], [1, 0, 1, -1, 1, 0], [1, 0, 1, 0, 1, 0], [1, 1, 1, 1, 1, 1]):
        s.attend(s.step(new, 6, 1, gen), 1)                            # one token each; slot 3 is released on the way
    s.step([0, 60, 0, 33, 0, 17], 120, 0, gen)                         # prompts of new requests, pages used again
    for new in ([3, 3, 1, 2, 3, 3], [1, 3, 2, -1, 3, 1]):              # up to three draft tokens
        s.attend(s.step(new, 18, 3, gen), 3)
    s.step([0, 0, 0, 190, 0, 150], 400, 0, gen)                        # the pool runs out for one of them
    s.attend(s.step([1] * 6, 6, 1, gen), 1)


def test_a_whole_step_in_one_graph():
    """Plan, append and attention captured once, replayed while the state on the GPU moves on,
    against the same steps run eagerly."""
    def fresh():
        s = Server(8, 64, 16, True)
        s.step([5, 40, 1, 90, 16, 15, 33, 2], 210, 0, torch.Generator().manual_seed(5))
        return s

    gen = torch.Generator().manual_seed(6)
    qkv = torch.randn(8, (G * H + 2 * G) * D, generator=gen).bfloat16().cuda()
    q, k, v = (x.view(8, -1, D) for x in qkv.split([G * H * D, G * D, G * D], dim=1))
    new = i32([1] * 8)

    def buffers():
        return dict(slots=torch.empty(8, dtype=torch.int64, device="cuda"), pos=i32([0] * 8), req=i32([0] * 8),
                    starts=i32([0] * 9), rot=torch.empty(8, G * H, D, dtype=torch.bfloat16, device="cuda"),
                    out=torch.empty(8 * G, H, D, dtype=torch.bfloat16, device="cuda"))

    def step(s, b):
        sda.sparse_decode_plan_step(s.lens, new, s.ring, s.state, s.table, block_size=B, slots=b["slots"],
                                    rows_per_request=1, positions=b["pos"], requests=b["req"], seq_lens=s.lens,
                                    token_starts=b["starts"], free_next=s.state)
        sda.sparse_decode_rope_append(q, k, v, b["pos"][None], s.inv, b["slots"], s.cache, b["rot"], **s.scales)
        sda.sparse_decode_paged_attention(b["rot"].view(8 * G, H, D), s.cache, s.table, s.lens, b["out"], scale=D ** -0.5,
                                          **s.scales)

    eager, be = fresh(), buffers()
    graphed, bg = fresh(), buffers()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        step(graphed, bg)
    for _ in range(20):                                                # past page ends
        step(eager, be)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(be["out"], bg["out"]) and torch.equal(be["slots"], bg["slots"])
        assert torch.equal(eager.lens, graphed.lens) and torch.equal(eager.cache, graphed.cache)
    assert torch.isfinite(be["out"]).all()
    assert eager.lens.tolist() == [25, 60, 21, 110, 36, 35, 53, 22]


def test_the_sparse_paths_read_the_same_cache():
    """What append writes, the framework's window and region attention read as well: over a whole
    short cache all three agree."""
    s = Server(4, 40, 8, False)
    gen = torch.Generator().manual_seed(8)
    s.step([64, 100, 33, 128 - 1], 330, 0, gen)
    q = s.step([1] * 4, 4, 1, gen).view(4 * G, H, D)
    kw = dict(scale=D ** -0.5)
    whole, window, regions = (torch.empty_like(q) for _ in range(3))
    sda.sparse_decode_paged_attention(q, s.cache, s.table, s.lens, whole, **kw)
    sda.sparse_decode_swa_attention(q, s.cache, s.table, s.lens, window, window=4096, **kw)
    ids = i32([list(range(8))] * (4 * G))
    pos = (s.lens - 1).repeat_interleave(G).contiguous()
    ids = torch.where(ids * B <= pos[:, None], ids, -1).to(torch.int32)
    sda.sparse_decode_attention(q, s.cache, ids, s.table, pos, torch.ones(4 * G, dtype=torch.bool, device="cuda"), regions, **kw)
    torch.cuda.synchronize()
    # each rounds its weights to bf16 at worst (2^-8) over |v| below 6, and its output once
    for other in (window, regions):
        assert ((whole.float() - other.float()).abs() <= 2.0 ** -8 * (6 + whole.float().abs() * 2)).all()

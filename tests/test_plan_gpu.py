"""A step's tables built on the GPU, against the request-by-request plain form: everything is
whole numbers and has to be equal."""
import random

import numpy as np
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import step_util

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def run(context, new, block, ring, state, table, rows, *, in_place=False, offset=0, workspace=None, stream=None,
        per_request=0):
    ctx, ring_t, st, tab = i32(context), i32(ring), i32(state), i32(np.asarray(table).tolist()).view(np.shape(table))
    raw = torch.full((rows + offset,), -7, dtype=torch.int64, device="cuda")
    pos, own = i32([-7] * (rows + offset)), i32([-7] * (rows + offset))
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda") if workspace is None else workspace
    kw = dict(seq_lens=ctx, free_next=st) if in_place else {}
    lens, starts, slots, positions, owners, nxt = sda.sparse_decode_plan_step(
        ctx, i32(new), ring_t, st, tab, block_size=block, slots=raw[offset:], positions=pos[offset:],
        requests=own[offset:], workspace=ws, stream=stream, rows_per_request=per_request, **kw)
    torch.cuda.synchronize()
    got = dict(seq_lens=lens, token_starts=starts, slots=slots, positions=positions, requests=owners, free_next=nxt,
               free_pages=ring_t, table=tab)
    return {k: v.cpu().numpy() for k, v in got.items()}, sda.read_errors(ws)


def check(context, new, block, ring, state, table, rows, **kw):
    got, flags = run(context, new, block, ring, state, table, rows, **kw)
    want, want_flags = step_util.plan(context, new, block, ring, state, table, rows, kw.get("per_request", 0))
    for k, v in want.items():
        assert np.array_equal(got[k].astype(np.int64).reshape(-1), np.asarray(v, dtype=np.int64).reshape(-1)), k
    assert flags == want_flags
    return got


def problem(r, requests, block, context, low, high, *, released=0.1, idle=0.1, room=1.0, row_room=1.0, spare=0):
    ctx = [r.randint(0, context) for _ in range(requests)]
    new = [-1 if r.random() < released else 0 if r.random() < idle else r.randint(low, high) for _ in range(requests)]
    held = [-(-c // block) for c in ctx]
    want = sum(-(-(c + n) // block) - h for c, n, h in zip(ctx, new, held) if n > 0)
    free = int(want * room) + spare
    total = max(1, sum(held) + free)
    ids = list(range(total))
    r.shuffle(ids)
    W = max(1, max(-(-(c + max(n, 0)) // block) for c, n in zip(ctx, new)))
    table = np.full((requests, W), -1)
    at = 0
    for q, h in enumerate(held):
        table[q, :h] = ids[at:at + h]
        at += h
    start = r.randrange(total)
    ring = [-5] * total
    for i in range(free):
        ring[(start + i) % total] = ids[at + i]
    rows = max(1, int(sum(max(n, 0) for n in new) * row_room))
    return ctx, new, block, ring, [start, free], table, rows


CASES = [  # requests, block, context, new tokens, options
    (1, 16, 0, (1, 1), {}),
    (1, 8, 100, (1, 70), dict(spare=3)),
    (7, 16, 64, (0, 40), {}),
    (64, 64, 4000, (1, 1), dict(spare=9)),
    (256, 64, 3000, (1, 3), {}),
    (1000, 16, 900, (1, 17), dict(spare=100)),
    (1025, 8, 200, (0, 5), {}),
    (100, 32, 500, (200, 900), {}),                 # more than one CTA
    (3000, 24, 300, (1, 60), dict(spare=11)),
    (8192, 128, 700, (1, 9), {}),
    (5, 1, 20, (1, 9), {}),                         # a page a token
    (300, 16, 500, (1, 90), dict(room=0.6)),        # pages run out
    (300, 16, 500, (1, 90), dict(row_room=0.55)),   # rows run out
    (300, 16, 500, (1, 90), dict(room=0.8, row_room=0.7)),
    (40, 16, 500, (1, 90), dict(room=0.0)),         # no free page: only partly filled ones take tokens
]


@pytest.mark.parametrize("requests,block,context,new,options", CASES)
@pytest.mark.parametrize("in_place", [False, True])
def test_matches_plain(requests, block, context, new, options, in_place):
    r = random.Random(requests * 131 + block)
    check(*problem(r, requests, block, context, *new, **options), in_place=in_place)


@pytest.mark.parametrize("seed", range(12))
def test_drawn(seed):
    r = random.Random(9000 + seed)
    low = r.choice([0, 1])
    check(*problem(r, r.randint(1, 700), r.choice([1, 8, 16, 48, 64]), r.choice([0, 30, 3000]), low,
                   r.choice([1, 7, 200]), room=r.choice([0.5, 1.0]), row_room=r.choice([0.5, 1.0]),
                   spare=r.choice([0, 5])), in_place=bool(seed & 1), offset=seed % 3)


@pytest.mark.parametrize("requests,k,low", [(1, 1, 1), (9, 1, 0), (64, 2, 0), (700, 4, 1), (3000, 3, 0), (8192, 1, 1)])
def test_so_many_rows_for_each_request(requests, k, low):
    r = random.Random(requests + k)
    ctx, new, block, ring, state, table, rows = problem(r, requests, 16, 200, low, k, room=0.9)
    check(ctx, new, block, ring, state, table, requests * k, per_request=k)
    new[0] = k + 1                                                            # more tokens than rows: left out
    check(ctx, new, block, ring, state, table, requests * k, per_request=k, in_place=True)


def test_rows_past_the_last_token_and_the_smallest_outputs():
    got = check([3, 0], [2, 1], 4, [9, 8, 7], [1, 2], [[5, -1], [-1, -1]], 11)
    assert got["slots"].tolist() == [23, 32, 28] + [-1] * 8
    check([0], [0], 4, [1], [0, 1], [[-1]], 0)                                # no token rows at all
    got, flags = run([], [], 4, [1, 2], [1, 1], np.zeros((0, 1)), 3)          # no requests
    assert got["token_starts"].tolist() == [0] and got["slots"].tolist() == [-1] * 3 and flags == 0
    assert got["free_next"].tolist() == [1, 1]


@pytest.mark.parametrize("context,new,state", [
    ([-1, 4, 4], [1, 1, 1], [0, 4]),            # a negative context
    ([4, 4, 4], [1, -2, 1], [0, 4]),            # a new length below -1
    ([4, 4, 4], [1, 2 ** 31 - 1, 1], [0, 4]),   # more pages than the table is wide
    ([4, 99, 4], [1, -1, 1], [0, 4]),           # releases more than the table holds
    ([4, 4, 4], [1, 1, 1], [9, 4]),             # a ring state out of range
    ([4, 4, 4], [1, -1, 1], [0, -3]),
    ([4, 4, 4], [1, -1, 1], [0, 8]),            # no room for what comes back
])
def test_requests_outside_the_contract_are_left_out(context, new, state):
    table = [[0, 1, -1], [2, 3, -1], [4, 5, -1]]
    check(context, new, 4, [10, 11, 12, 13, 14, 15, 16, 17], state, table, 8)


def test_bad_table_entry_under_a_partly_filled_page():
    check([5, 6], [2, 2], 4, [10, 11], [0, 2], [[0, -1, -1], [2, 3, -1]], 6)


def test_positions_past_32_bits_of_slots():
    """A slot is 64 bits wide: page * block passes 2^31 in a large cache."""
    got = check([100], [3], 64, [2 ** 31 - 5], [0, 1], [[2 ** 31 - 2, 2 ** 31 - 9]], 3)
    assert got["slots"][0] == (2 ** 31 - 9) * 64 + 36


def test_two_steps_in_place_match_the_plain_form():
    """Lengths, table and ring carried over steps on the GPU; pages released in one step come
    back in the next."""
    r = random.Random(4)
    ctx, new, block, ring, state, table, rows = problem(r, 50, 16, 300, 1, 40, released=0.4, spare=2)
    c, st, tab, rg = i32(ctx), i32(state), i32(np.asarray(table).tolist()), i32(ring)
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    for step in range(6):
        want, _ = step_util.plan(ctx, new, block, ring, state, table, 400)
        slots = torch.empty(400, dtype=torch.int64, device="cuda")
        sda.sparse_decode_plan_step(c, i32(new), rg, st, tab, block_size=block, slots=slots, seq_lens=c, free_next=st,
                                    workspace=ws)
        ctx, state, table, ring = want["seq_lens"], want["free_next"], want["table"], want["free_pages"]
        assert c.tolist() == ctx and st.tolist() == state and rg.tolist() == ring
        assert np.array_equal(tab.cpu().numpy(), table) and slots.tolist() == want["slots"]
        new = [r.choice([0, 1, 1, 5, -1]) for _ in ctx]


def test_graph_replay_and_another_stream():
    r = random.Random(5)
    ctx, new, block, ring, state, table, rows = problem(r, 200, 16, 0, 90, 200, released=0.0, spare=600)
    side = torch.cuda.Stream()
    c, n, st, tab, rg = i32(ctx), i32(new), i32(state), i32(np.asarray(table).tolist()), i32(ring)
    tab = torch.nn.functional.pad(tab, (0, 3), value=-1).contiguous()
    table = np.pad(np.asarray(table), ((0, 0), (0, 3)), constant_values=-1)
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    first = (c.clone(), st.clone(), tab.clone(), rg.clone())
    call = lambda: sda.sparse_decode_plan_step(c, n, rg, st, tab, block_size=block, slots=slots, seq_lens=c, free_next=st)
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=side):
            call()
    torch.cuda.synchronize()
    for t, v in zip((c, st, tab, rg), first):
        t.copy_(v)
    n.fill_(3)
    for _ in range(3):                                   # the length of the second step is the first's output
        want, _f = step_util.plan(ctx, [3] * len(ctx), block, ring, state, table, rows)
        g.replay()
        torch.cuda.synchronize()
        ctx, state, table, ring = want["seq_lens"], want["free_next"], want["table"], want["free_pages"]
        assert c.tolist() == ctx and st.tolist() == state and slots.tolist() == want["slots"]
        assert np.array_equal(tab.cpu().numpy(), table)


def test_strided_tables_and_lengths():
    both = i32([[5, 2, 9], [0, 3, 9], [17, 1, 9]])          # context and new as columns of one tensor
    wide = i32([[1, -1, -1, 77]] * 3)
    wide[2, :2] = torch.tensor([3, 4], device="cuda")
    slots = torch.empty(8, dtype=torch.int64, device="cuda")
    lens = i32([[0, 0]] * 3)
    out = sda.sparse_decode_plan_step(both[:, 0], both[:, 1], i32([20, 21, 22]), i32([0, 3]), wide[:, :3], block_size=16,
                                      slots=slots, seq_lens=lens[:, 1])
    want, _ = step_util.plan([5, 0, 17], [2, 3, 1], 16, [20, 21, 22], [0, 3], [[1, -1, -1], [1, -1, -1], [3, 4, -1]], 8)
    assert lens.tolist() == [[0, x] for x in want["seq_lens"]] and slots.tolist() == want["slots"]
    assert np.array_equal(wide[:, :3].cpu().numpy(), want["table"]) and wide[:, 3].tolist() == [77] * 3
    assert out[0].data_ptr() == lens[:, 1].data_ptr()

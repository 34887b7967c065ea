"""How the whole-cache attention splits units ((request, KV group) pairs): a worker each, a CTA
each, or cut over CTAs.  Table widths and counts of requests on both sides of each rule, against
float64 attention; the same requests under a wider table, which cuts them."""
import random

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from test_paged_gpu import Problem, check

pytestmark = pytest.mark.gpu


def lengths(top, n, seed):
    r = random.Random(seed)
    return ([top, 0, 1, top - 1, top // 2 + 3] + [r.randint(0, top) for _ in range(n)])[:n]


# tokens of a tile where a CTA has the unit, and workers of a CTA
KINDS = [(64, True, 8, 1, 64, 4), (64, False, 8, 1, 32, 4), (128, True, 16, 1, 32, 4), (128, False, 5, 3, 16, 4),
         (192, True, 16, 1, 32, 4), (192, False, 16, 1, 16, 4), (256, True, 8, 2, 16, 4), (256, False, 16, 1, 8, 4),
         (64, True, 16, 2, 64, 2), (128, False, 10, 3, 16, 2), (192, True, 16, 2, 32, 2), (192, False, 8, 3, 32, 2),
         (256, True, 16, 2, 32, 2), (192, True, 16, 4, 32, 1)]


@pytest.mark.parametrize("D,fp8,H,ql,tile,workers", KINDS)
@pytest.mark.parametrize("tiles", [2, 3, 8, 9, "alone", "cut"])
def test_table_widths_around_the_rules(D, fp8, H, ql, tile, workers, tiles):
    tiles = 12 * workers if tiles == "alone" else 12 * workers + 1 if tiles == "cut" else tiles
    p = Problem(lengths(tiles * tile, 5, tiles + D), D=D, fp8=fp8, H=H, ql=ql, G=2, block=8 if tile == 8 else 16,
                gate=tiles % 2 == 1, seed=tiles)
    assert p.table.shape[1] * p.block == tiles * tile
    p.check(*p.run())


@pytest.mark.parametrize("n", [304, 305, 1216, 1217])
@pytest.mark.parametrize("tiles", [8, 9])
def test_counts_of_units_around_the_rules(n, tiles):
    """One unit a CTA in one round, in several, and more than are taken that way."""
    r = random.Random(n + tiles)
    lens = [r.choice([0, 1, 20, 40, 66, r.randint(1, tiles * 8)]) for _ in range(n - 1)] + [tiles * 8]
    check(lens, D=256, H=2, G=1, block=8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ql", [1, 2])
def test_the_same_requests_under_a_wider_table(fp8, ql):
    """What a CTA does alone and what CTAs join agree with the exact values, and hence with one another."""
    lens = lengths(500, 9, 5)
    for spare in (0, 2000):
        check(lens, D=192, fp8=fp8, H=16, ql=ql, G=2, block=16, spare=spare, seed=3, gate=True)


def test_a_cta_alone_repeats_its_bits_and_leaves_the_workspace():
    p = Problem(lengths(700, 40, 9), D=192, fp8=True, H=16, G=2, block=16)
    ws = p.workspace()
    first = p.run(workspace=ws)
    again = p.run(workspace=ws)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(first, again))
    assert not ws.any()


def test_no_lse_and_unaligned_outputs():
    p = Problem(lengths(600, 6, 2), D=128, H=8, G=2, block=16, gate=True)
    want, lse = p.run()
    p.check(want, lse)
    raw = torch.full((p.query.shape[0], 8 * 131 + 3), 9.0, dtype=torch.bfloat16, device="cuda")
    out = raw[:, 1:1 + 8 * 131].view(-1, 8, 131)[:, :, 1:129]
    sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, **p.kw())
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    out.fill_(9.0)
    assert (raw == 9.0).all()


@pytest.mark.parametrize("n", [303, 304])
@pytest.mark.parametrize("tiles", [12, 13, 24, 25])
@pytest.mark.parametrize("ql,workers", [(4, 1), (2, 2)])
def test_many_query_rows_around_the_rules(n, tiles, ql, workers):
    """Twice the tiles where there is a unit for every CTA."""
    r = random.Random(n + tiles)
    top = tiles * workers * 32
    lens = [r.choice([0, 1, 33, r.randint(1, 200)]) for _ in range(n - 2)] + [top, top - 1]
    check(lens, D=128, H=16, ql=ql, G=1, block=32)

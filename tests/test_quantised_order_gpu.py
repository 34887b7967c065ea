"""Rows of one block in two places of an append's slots: told by a flag wherever they are, and no harm to other blocks."""
import numpy as np
import pytest
import torch

import quant_util
import sparse_decode_attention_02_gb300 as sda
from test_quantised_cache_gpu import Cache, slots_of

pytestmark = pytest.mark.gpu


def apart(c, slots, blocks, gen):
    """Appends rows of which those in `blocks` are not next to each other; all other blocks have to be equal."""
    key, value = c.rows(len(slots), gen)
    alone = [-1 if s >= 0 and s // c.S in blocks else s for s in slots]
    assert quant_util.append(key, value, alone, c.elements, c.plain_scales, c.int8) == 0
    sda.sparse_decode_quantised_append(key.cuda(), value.cuda(), torch.tensor(slots, device="cuda"), c.cache, c.scales, workspace=c.ws)
    torch.cuda.synchronize()
    assert sda.read_errors(c.ws, clear=True) == sda.FLAG_BOUNDS
    others = np.ones(c.elements.shape[0] * c.B // c.S, bool)
    others[list(blocks)] = False
    by_block = lambda x: x.reshape(len(c.elements), c.G, c.B // c.S, -1).swapaxes(1, 2).reshape(len(others), -1)[others]  # noqa: E731
    assert np.array_equal(by_block(c.scales.cpu().numpy()), by_block(c.plain_scales))
    assert np.array_equal(by_block(quant_util.values(c.cache.cpu().contiguous(), c.int8)), by_block(c.elements))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("slots,blocks", [([3, -1, 4], {0}), ([4, -1, 3], {0}), ([3, 40, 4], {0}), ([0, -1, 1], {0}), ([1, -1, 0], {0}),
                                          ([5, 21, 45, 6, 22, 46], {0, 2, 5}), ([635, 1, 2, 636], {79}), ([8, 9, 3, 10], {1}),
                                          ([-1] * 300 + [3, -1, 4], {0}), ([3] + [-1] * 300 + [4], {0}), ([9, 17, 12], {1}),
                                          ([0, -1, 0], {0}), ([8, 9, 320, 8, 9], {1}), ([16, 24] * 3, {2, 3})])
def test_a_few_rows_apart(slots, blocks, int8):
    apart(Cache(B=16, S=8, int8=int8), slots, blocks, torch.Generator().manual_seed(len(slots)))


@pytest.mark.parametrize("G,D", [(1, 64), (2, 128), (8, 16)])
@pytest.mark.parametrize("place", [0, 3])
@pytest.mark.parametrize("at", [(0, 2999), (64, 65 + 64), (70, 2000), (255, 257), (1500, 1502), (2047, 2900), (2048, 2050)])
def test_rows_apart_in_a_prompt(at, place, G, D):
    """Two rows of one block, the same slot at its beginning or two behind it, somewhere between a prompt's."""
    c = Cache(pages=100, G=G, B=32, S=16, D=D)
    slots = slots_of(list(range(95)), 5, 3000, 32)
    for i, row in enumerate(at):
        slots[row] = 98 * 32 + 16 + (place + i if place else 0)
    # the prompt's rows go on in their blocks from the first that is left out on: not in order either
    blocks = {98 * 2 + 1} | {(5 + row) // 16 for row in at}
    apart(c, slots, blocks, torch.Generator().manual_seed(at[0] + place))


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("requests,new", [(1000, 4), (300, 1), (1500, 2), (5000, 1)])
def test_many_requests_in_order_raise_no_flag(requests, new, int8):
    """A block each, behind its first place or across its end; more of them than a table of what is looked for has, and
    some padding."""
    c = Cache(pages=requests, G=2, B=16, S=8, D=16, int8=int8)
    slots = []
    for q in range(requests):
        first = 1 + q % 11
        slots += list(range(q * 16 + first, q * 16 + first + new)) + [-1] * (q % 7 == 0)
    c.append(*c.rows(len(slots), torch.Generator().manual_seed(new)), slots, flags=0)


def test_without_a_workspace_nothing_is_looked_for():
    c = Cache(B=16, S=8)
    key, value = (x.cuda() for x in c.rows(3, torch.Generator().manual_seed(1)))
    before = c.scales.clone()
    at = torch.tensor([3, -1, 4], device="cuda")
    d = sda._binding
    with torch.cuda.device(key.device):
        memory, where, *_ = d.load_marshal().pack(key, value, at, c.cache, c.scales)
        assert d.load().sparse_decode_quantised_append(*where, None, 0, None) == d.SDA_OK
    torch.cuda.synchronize()
    assert torch.equal(c.scales.view(-1, 2, 2, 2)[1:], before.view(-1, 2, 2, 2)[1:])


@pytest.mark.parametrize("rows,at", [(16384, (5, 16000)), (16384, (2046, 2048)), (16384, (2100, 14336)), (16384, (14335, 16383)),
                                     (12289, (4097, 12288)), (16384, None), (40000, None)])
def test_rows_far_apart(rows, at):
    """As many rows as are looked at, in any two of their parts; in order, and more of them."""
    c = Cache(pages=85, G=1, B=512, S=512, D=16)
    slots = slots_of(list(range(80)), 5, rows, 512)
    gen = torch.Generator().manual_seed(7)
    if at is None:
        c.append(*c.rows(len(slots), gen), slots, flags=0)
        return
    slots[at[0]], slots[at[1]] = 82 * 512 + 7, 82 * 512 + 9
    apart(c, slots, {82} | {(5 + row) // 512 for row in at}, gen)

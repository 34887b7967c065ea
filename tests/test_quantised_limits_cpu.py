"""The sizes up to which the quantised cache's entry points go: one past each is refused, the last one is not (it gets
as far as a workspace that is refused; descriptors with made-up addresses, nothing is launched)."""
import pytest

import sparse_decode_attention_02_gb300 as sda
from test_quantised_abi_cpu import F32, U8, UNS, WS, append, lib, paged, read, regions, t  # noqa: F401

BAD = dict(ws=1 << 24, wsb=128)                # a workspace that is too small, looked at after the sizes


def both(G=2, pages=5, block=16, span=8, D=64):
    """A cache and its scales in which every head's pages lie in the same place: sizes without their bytes."""
    return dict(cache=t(U8, (pages, G, block, 2 * D), (16, 16, 16, 1)), scales=t(F32, (pages, G, block // span, 2), (2, 2, 2, 1)))


def test_rows_of_an_append(lib):  # noqa: F811
    for rows, status in ((1 << 28, WS), ((1 << 28) + 1, UNS)):
        assert append(lib, T=rows, **BAD) == status


def test_rows_requests_and_columns_of_a_read(lib):  # noqa: F811
    for n, status in ((1 << 30, WS), ((1 << 30) + 1, UNS)):
        assert read(lib, T=n, **BAD) == status
        assert read(lib, Q=n, **BAD) == status
    for width, status in (((1 << 31) - 1, WS), (1 << 31, UNS)):
        assert read(lib, W=width, **BAD) == status


@pytest.mark.parametrize("entry", [append, read, paged, regions])
def test_tokens_of_a_page(lib, entry):  # noqa: F811
    for block, status in ((1 << 24, WS), ((1 << 24) + 8, UNS)):
        assert entry(lib, **both(block=block), **BAD) == status


@pytest.mark.parametrize("entry", [append, read, paged, regions])
def test_groups(lib, entry):  # noqa: F811
    for groups, status in ((1 << 16, WS), ((1 << 16) + 1, UNS)):
        assert entry(lib, G=groups, **both(G=groups), **BAD) == status


@pytest.mark.parametrize("entry", [read, paged, regions])
def test_pages(lib, entry):  # noqa: F811
    for pages, status in (((1 << 31) - 1, WS), (1 << 31, UNS)):
        assert entry(lib, **both(pages=pages), **BAD) == status


def test_slots_of_a_cache(lib):  # noqa: F811
    """32 bits of them for an append (less the two values that are none); a read has no such limit."""
    for pages, block, status in (((1 << 29) - 1, 8, WS), (1 << 29, 8, UNS), ((1 << 32) // 24, 24, WS), ((1 << 32) // 24 + 1, 24, UNS)):
        assert append(lib, **both(pages=pages, block=block), **BAD) == status
        assert read(lib, **both(pages=pages, block=block), **BAD) == WS


def test_rows_and_columns_of_whole_caches(lib):  # noqa: F811
    for rows, status in (((1 << 25) - 1, WS), (1 << 25, UNS)):
        assert paged(lib, reqs=rows, ql=1, G=1, **BAD) == status
    for width, status in (((1 << 31) - 1, WS), (1 << 31, UNS)):
        assert paged(lib, W=width, **BAD) == status


def test_rows_and_lists_of_regions(lib):  # noqa: F811
    for rows, status in (((1 << 25) - 1, WS), (1 << 25, UNS)):
        assert regions(lib, toks=rows, ql=1, G=1, **BAD) == status
    for listed, status in ((1 << 20, WS), ((1 << 20) + 1, UNS)):
        assert regions(lib, R=listed, rt=8, **BAD) == status
    for tokens, status in ((1 << 24, WS), ((1 << 24) + 8, UNS)):
        assert regions(lib, R=1, rt=tokens, **BAD) == status
    for listed, status in ((127, WS), (128, UNS)):                           # times 2^24 tokens
        assert regions(lib, R=listed, rt=1 << 24, **BAD) == status
    assert regions(lib, W=1 << 31, **BAD) == UNS


@pytest.mark.parametrize("entry", [append, read, paged, regions])
def test_strides_of_nothing(lib, entry):  # noqa: F811
    """Blocks, heads and pages that share their bytes or scales are refused where they would be written, and where read."""
    for at in range(3):
        cache, scales = [16, 16, 16, 1], [2, 2, 2, 1]
        cache[at] = scales[at] = 0
        assert entry(lib, **(both() | dict(cache=t(U8, (5, 2, 16, 128), tuple(cache))))) == UNS
        assert entry(lib, **(both() | dict(scales=t(F32, (5, 2, 2, 2), tuple(scales))))) == UNS


def test_workspace_bytes_of_rows_past_64_bits(lib):  # noqa: F811
    for rows in (1 << 63, 1 << 64, (1 << 64) + 5, -(1 << 63) - 1):
        with pytest.raises(OverflowError):
            sda.quantised_workspace_bytes(rows, 8)
    assert sda.quantised_workspace_bytes((1 << 63) - 1, 8) == sda.quantised_workspace_bytes(-(1 << 63), 8) == 0

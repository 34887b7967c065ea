"""Host-side checks of the quantised cache's entry points: every contract violation is refused with its
status before any CUDA call (descriptors with made-up addresses; nothing is dereferenced)."""
import ctypes

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from sparse_decode_attention_02_gb300 import _binding as B
from sparse_decode_attention_02_gb300 import build as lib_build
from test_abi_cpu import FakeDev

OK, INV, UNS, WS = B.SDA_OK, B.SDA_ERR_INVALID, B.SDA_ERR_UNSUPPORTED, B.SDA_ERR_WORKSPACE
BF16, FP8, U8, I32, F32, I64, I8 = 1, 2, 3, 4, 6, 7, 8
t = FakeDev.t


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    lib_build.build_marshal()
    return sda.load()


def ref(d):
    return ctypes.addressof(d) if d is not None else None


def cache_and_scales(pages=5, G=2, block=16, span=8, D=64, kind=U8):
    return dict(cache=t(kind, (pages, G, block, 2 * D)), scales=t(F32, (pages, G, block // span, 2)))


def append(lib, T=8, G=2, D=64, ws=None, wsb=0, like=None, **change):
    d = dict(key=t(BF16, (T, G, D)), value=t(BF16, (T, G, D)), slots=t(I64, (T,))) | cache_and_scales(G=G, D=D, **(like or {})) | change
    return lib.sparse_decode_quantised_append(*(ref(x) for x in d.values()), ws, wsb, None)


# what is wrong with a cache or its scales, for every entry that takes them
CACHES = [
    (INV, dict(cache=t(BF16, (5, 2, 16, 128)))), (INV, dict(cache=t(F32, (5, 2, 16, 128)))), (INV, dict(cache=t(U8, (5, 2, 16, 64)))),
    (INV, dict(cache=t(U8, (5, 3, 16, 128)))), (INV, dict(cache=t(U8, (4, 2, 16, 128)))), (INV, dict(cache=t(U8, (2, 16, 128)))),
    (INV, dict(cache=t(U8, (5, 2, 16, 128), (8192, 4096, 256, 2)))), (INV, dict(cache=None)), (INV, dict(scales=None)),
    (INV, dict(scales=t(BF16, (5, 2, 2, 2)))), (INV, dict(scales=t(F32, (5, 2, 3, 2)))), (INV, dict(scales=t(F32, (5, 2, 0, 2)))),
    (INV, dict(scales=t(F32, (5, 2, 2)))), (INV, dict(scales=t(F32, (5, 2, 2, 1)))), (INV, dict(scales=t(F32, (6, 2, 2, 2)))),
    (INV, dict(scales=t(F32, (5, 2, 2, 2), (16, 8, 4, 2)))),
    (UNS, dict(scales=t(F32, (5, 2, 4, 2)))),                                # blocks of four places
    (UNS, dict(scales=t(F32, (5, 2, 2, 2), (8, 4, 3, 1)))), (UNS, dict(scales=t(F32, (5, 2, 2, 2), (0, 4, 2, 1)))),
    (UNS, dict(scales=t(F32, (5, 2, 2, 2), addr=(1 << 20) + 4))), (UNS, dict(cache=t(U8, (5, 2, 16, 128), addr=(1 << 20) + 8))),
    (UNS, dict(cache=t(U8, (5, 2, 16, 128), (4104, 2048, 128, 1)))), (UNS, dict(cache=t(U8, (5, 2, 16, 128), (0, 2048, 128, 1)))),
]


@pytest.mark.parametrize("which", range(len(CACHES)))
def test_cache_refusals(lib, which):
    status, change = CACHES[which]
    assert append(lib, **change) == status
    assert read(lib, **change) == status


def test_append_refusals(lib):
    for name, bad in dict(key=t(F32, (8, 2, 64)), value=t(BF16, (8, 3, 64)), slots=t(I32, (8,))).items():
        assert append(lib, **{name: bad}) == INV, name
    assert append(lib, key=None) == INV
    assert append(lib, value=None) == INV
    assert append(lib, slots=None) == INV
    assert append(lib, value=t(BF16, (7, 2, 64))) == INV
    assert append(lib, slots=t(I64, (7,))) == INV
    assert append(lib, slots=t(I64, (8,), (2,))) == INV
    assert append(lib, key=t(BF16, (8, 2, 64), (256, 128, 2))) == INV
    assert append(lib, key=t(BF16, (8, 2, 64), (132, 64, 1))) == UNS
    assert append(lib, value=t(BF16, (8, 2, 64), addr=(1 << 20) + 8)) == UNS
    assert append(lib, key=t(BF16, (8, 2, 64), addr=0)) == INV
    assert append(lib, D=40) == UNS
    assert append(lib, D=528) == UNS
    assert append(lib, ws=1 << 24, wsb=128) == WS
    assert append(lib, ws=(1 << 24) + 16, wsb=256) == WS
    assert append(lib, wsb=256) == WS
    assert append(lib, T=0) == OK
    assert append(lib, T=0, like=dict(kind=I8)) == append(lib, T=0, like=dict(kind=FP8)) == OK


def read(lib, T=8, G=2, D=64, Q=3, W=4, ws=None, wsb=0, **change):
    d = cache_and_scales(G=G, D=D) | dict(table=t(I32, (Q, W)), starts=t(I32, (Q + 1,)), first=t(I32, (Q,)),
                                          key=t(BF16, (T, G, D)), value=t(BF16, (T, G, D))) | change
    return lib.sparse_decode_quantised_read(*(ref(x) for x in d.values()), ws, wsb, None)


def test_read_refusals(lib):
    for name, bad in dict(table=t(I64, (3, 4)), starts=t(I64, (4,)), first=t(I64, (3,)), key=t(F32, (8, 2, 64)),
                          value=t(BF16, (8, 2, 32))).items():
        assert read(lib, **{name: bad}) == INV, name
    assert read(lib, key=None, value=None) == INV
    assert read(lib, table=None) == INV
    assert read(lib, starts=None) == INV
    assert read(lib, starts=t(I32, (0,))) == INV
    assert read(lib, starts=t(I32, (4,), (2,))) == INV
    assert read(lib, first=t(I32, (4,))) == INV
    assert read(lib, table=t(I32, (2, 4))) == INV
    assert read(lib, table=t(I32, (3, 4), (8, 2))) == INV
    assert read(lib, value=t(BF16, (7, 2, 64))) == INV
    assert read(lib, key=t(BF16, (8, 2, 64), (0, 64, 1))) == INV             # rows that are written lie apart
    assert read(lib, key=t(BF16, (8, 2, 64), (128, 0, 1))) == INV
    assert read(lib, key=t(BF16, (8, 2, 64), (132, 64, 1))) == UNS
    assert read(lib, D=24) == UNS
    assert read(lib, ws=1 << 24, wsb=0) == WS
    assert read(lib, T=0) == OK
    assert read(lib, Q=0) == OK
    assert read(lib, T=0, key=None) == OK


def paged(lib, reqs=3, ql=2, G=2, H=8, D=64, W=5, scale=0.1, ws=1 << 24, wsb=None, like=None, **change):
    rows = reqs * ql * G
    like = cache_and_scales(G=G, D=D, **(like or {}))
    d = dict(q=t(BF16, (rows, H, D))) | like | dict(table=t(I32, (reqs, W)), lens=t(I32, (reqs,)), out=t(BF16, (rows, H, D)),
                                                    lse=t(F32, (rows, H)), gate=None) | change
    a = [ref(x) for x in d.values()]
    need = lib.sparse_decode_paged_workspace_bytes(H, ql, D)
    return lib.sparse_decode_quantised_paged_attention(*a[:7], scale, ql, a[7], ws, need if wsb is None else wsb, None)


def regions(lib, toks=6, ql=2, G=2, H=8, D=64, R=4, W=5, rt=0, scale=0.1, ws=1 << 24, wsb=None, like=None, **change):
    rows = toks * G
    like = cache_and_scales(G=G, D=D, **(like or {}))
    d = dict(q=t(BF16, (rows, H, D))) | like | dict(ids=t(I32, (rows, R)), table=t(I32, (toks // ql, W)), pos=t(I32, (rows,)),
                                                    act=t(5, (rows,)), out=t(BF16, (rows, H, D)), lse=t(F32, (rows, H)),
                                                    gate=None) | change
    a = [ref(x) for x in d.values()]
    need = lib.sparse_decode_quantised_workspace_bytes(rows, H, D)
    return lib.sparse_decode_quantised_attention(*a[:9], scale, ql, a[9], 1, rt, ws, need if wsb is None else wsb, None)


@pytest.mark.parametrize("entry", [paged, regions])
@pytest.mark.parametrize("which", range(len(CACHES)))
def test_cache_refusals_of_attention(lib, entry, which):
    status, change = CACHES[which]
    assert entry(lib, **change) == status


@pytest.mark.parametrize("entry", [paged, regions])
def test_attention_refusals(lib, entry):
    for name, bad in dict(q=t(F32, (12, 8, 64)), table=t(I64, (3, 5)), out=t(BF16, (12, 8, 32)), lse=t(F32, (12, 7)),
                          gate=t(BF16, (6, 15))).items():
        assert entry(lib, **{name: bad}) == INV, name
    assert entry(lib, q=None) == entry(lib, table=None) == entry(lib, out=None) == INV
    assert entry(lib, table=t(I32, (2, 5))) == INV
    assert entry(lib, table=t(I32, (3, 5), (10, 2))) == INV
    assert entry(lib, q=t(BF16, (12, 8, 64), (1024, 128, 2))) == INV
    assert entry(lib, lse=t(F32, (12, 8), (0, 1))) == INV
    assert entry(lib, out=t(BF16, (12, 8, 64), (0, 64, 1))) == INV
    assert entry(lib, scale=float("inf")) == INV
    assert entry(lib, D=96) == UNS
    assert entry(lib, ws=None) == WS
    assert entry(lib, ws=(1 << 24) + 128) == WS
    assert entry(lib, wsb=255) == WS
    assert entry(lib, q=t(BF16, (12, 8, 64), addr=0)) == INV


def test_paged_refusals(lib):
    assert paged(lib, lens=t(F32, (3,))) == INV
    assert paged(lib, lens=t(I32, (4,))) == INV                              # rows are not 4 requests'
    assert paged(lib, lens=None) == INV
    assert paged(lib, ql=0) == INV
    assert paged(lib, H=33) == UNS                                           # more than 64 query rows
    assert paged(lib, reqs=0) == OK


def test_region_refusals(lib):
    for name, bad in dict(ids=t(I64, (12, 4)), pos=t(I64, (12,)), act=t(I32, (12,))).items():
        assert regions(lib, **{name: bad}) == INV, name
    assert regions(lib, ids=None) == regions(lib, pos=None) == regions(lib, act=None) == INV
    assert regions(lib, ids=t(I32, (11, 4))) == regions(lib, pos=t(I32, (11,))) == regions(lib, act=t(5, (11,))) == INV
    assert regions(lib, ids=t(I32, (12, 4), (8, 2))) == INV
    assert regions(lib, rt=-8) == INV
    assert regions(lib, toks=5, ql=5, q=t(BF16, (11, 8, 64)), out=t(BF16, (11, 8, 64)), lse=None) == INV
    assert regions(lib, H=17) == UNS
    assert regions(lib, rt=12) == UNS                                        # gcd with pages of 16 is 4
    assert regions(lib, rt=1 << 25) == UNS
    assert regions(lib, R=1 << 17, rt=1 << 15) == UNS                        # more tokens than 31 bits count
    assert regions(lib, R=(1 << 20) + 1) == UNS
    assert regions(lib, toks=0) == OK
    assert regions(lib, toks=0, rt=40) == regions(lib, toks=0, R=0) == OK    # gcd 8; nothing listed


def test_region_workspace_bytes(lib):
    f = sda.quantised_workspace_bytes
    assert f(10, 0) == f(10, 17) == f(10, 8, 96) == f(-1, 8) == f(1 << 40, 8) == 0
    for rows in (0, 1, 63, 64, 65, 1000):
        assert f(rows, 8, 128) == sda.paged_workspace_bytes(8, 1, 128) + -(-rows * 4 // 256) * 256
    assert regions(lib, wsb=f(12, 8, 64) - 1) == WS


def host_calls(ws=None):
    bf, i32 = torch.bfloat16, torch.int32
    cache, scales = torch.zeros(3, 1, 16, 128, dtype=torch.int8), torch.zeros(3, 1, 2, 2)
    x, n, table = torch.zeros(4, 1, 64, dtype=bf), torch.ones(4, dtype=i32), torch.zeros(4, 2, dtype=i32)
    slots = torch.zeros(4, dtype=torch.int64)
    q, on = torch.zeros(4, 8, 64, dtype=bf), torch.ones(4, dtype=torch.bool)
    return dict(paged=lambda: sda.sparse_decode_quantised_paged_attention(q, cache, scales, table, n, q.clone(), scale=0.1,
                                                                          workspace=ws),
                regions=lambda: sda.sparse_decode_quantised_attention(q, cache, scales, table, table, n, on, q.clone(), scale=0.1,
                                                                      workspace=ws),
                append=lambda: sda.sparse_decode_quantised_append(x, x, slots, cache, scales, workspace=ws),
                read=lambda: sda.sparse_decode_quantised_read(cache, scales, table, n, x, x, workspace=ws))


@pytest.mark.parametrize("name", sorted(host_calls()))
def test_host_tensors_are_refused(lib, name):
    """Host tensors never reach the library: the binding raises before it allocates or calls."""
    before = dict(B._step_workspaces)
    with pytest.raises(ValueError, match="CUDA tensor"):
        host_calls()[name]()
    assert B._step_workspaces == before


@pytest.mark.parametrize("name", sorted(host_calls()))
@pytest.mark.parametrize("which", range(3))
def test_workspaces_with_gaps_are_refused(lib, monkeypatch, name, which):
    ws = [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(64, 300, dtype=torch.uint8)[:, :256],
          torch.zeros(1 << 12, dtype=torch.uint8)[::2]][which]

    class Marshal:
        pack = staticmethod(lambda *t: (b"", [None] * len(t), 0, 1, 0, 0))

        def __getattr__(self, name):
            return lambda *a: None

    monkeypatch.setattr(B, "_marshal", Marshal())
    monkeypatch.setattr(type(ws), "get_device", lambda t: 0)
    with pytest.raises(ValueError, match="contiguous"):
        host_calls(ws)[name]()

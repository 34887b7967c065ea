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


def host_calls(ws=None):
    bf, i32 = torch.bfloat16, torch.int32
    cache, scales = torch.zeros(3, 1, 16, 128, dtype=torch.int8), torch.zeros(3, 1, 2, 2)
    x, n, table = torch.zeros(4, 1, 64, dtype=bf), torch.ones(4, dtype=i32), torch.zeros(4, 2, dtype=i32)
    slots = torch.zeros(4, dtype=torch.int64)
    return dict(append=lambda: sda.sparse_decode_quantised_append(x, x, slots, cache, scales, workspace=ws),
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

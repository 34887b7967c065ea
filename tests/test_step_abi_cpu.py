"""Host-side checks of the serving-step entry points: every contract violation is refused with its
status before any CUDA call (descriptors with made-up addresses; nothing is dereferenced)."""
import ctypes

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from sparse_decode_attention_02_gb300 import _binding as B
from sparse_decode_attention_02_gb300 import build as lib_build
from test_abi_cpu import FakeDev

OK, INV, UNS, WS = B.SDA_OK, B.SDA_ERR_INVALID, B.SDA_ERR_UNSUPPORTED, B.SDA_ERR_WORKSPACE
BF16, FP8, U8, I32, F32, I64 = 1, 2, 3, 4, 6, 7
t = FakeDev.t


@pytest.fixture(scope="module")
def lib():
    lib_build.build()
    return sda.load()


def ref(d):
    return ctypes.addressof(d) if d is not None else None


def plan(lib, Q=4, T=9, F=20, W=6, block=16, per=0, ws=1 << 24, wsb=256, **change):
    d = dict(context=t(I32, (Q,)), new=t(I32, (Q,)), free=t(I32, (F,)), state=t(I32, (2,)), next=t(I32, (2,)),
             table=t(I32, (Q, W)), lens=t(I32, (Q,)), starts=t(I32, (Q + 1,)), slots=t(I64, (T,)), pos=t(I32, (T,)),
             req=t(I32, (T,))) | change
    a = [ref(x) for x in d.values()]
    return lib.sparse_decode_plan_step(a[0], a[1], block, per, *a[2:], ws, wsb, None)


def test_plan_refusals(lib):
    for name, bad in dict(context=t(I64, (4,)), new=t(I32, (5,)), free=t(I32, (0,)), state=t(I32, (3,)), next=t(I32, (1,)),
                          table=t(I32, (3, 6)), lens=t(F32, (4,)), starts=t(I32, (4,)), slots=t(I32, (9,)),
                          pos=t(I32, (8,)), req=t(I32, (9, 1))).items():
        assert plan(lib, **{name: bad}) == INV, name
    assert plan(lib, block=0) == INV
    assert plan(lib, per=-1) == INV
    assert plan(lib, per=2) == INV                                           # T != Q * k
    assert plan(lib, table=t(I32, (4, 6), (12, 2))) == INV                  # inner stride
    assert plan(lib, table=t(I32, (4, 6), (3, 1))) == INV                   # rows overlap
    assert plan(lib, lens=t(I32, (4,), (0,))) == INV                        # broadcast output
    assert plan(lib, slots=t(I64, (9,), (2,))) == INV
    assert plan(lib, context=None) == INV
    assert plan(lib, slots=t(I64, (9,), addr=0)) == INV
    assert plan(lib, Q=8193) == UNS
    assert plan(lib, F=(1 << 30) + 1) == UNS
    assert plan(lib, ws=None) == WS
    assert plan(lib, ws=(1 << 24) + 8) == WS
    assert plan(lib, wsb=255) == WS


def rope(lib, T=8, Hq=6, G=2, D=64, half=32, axes=1, sections=None, inter=0, adj=0, amp=1.0, fp8=False, scales=True,
         ws=None, wsb=0, block=16, **change):
    d = dict(q=t(BF16, (T, Hq, D)), out=t(BF16, (T, Hq, D), addr=1 << 21), k=t(BF16, (T, G, D)), v=t(BF16, (T, G, D)),
             pos=t(I32, (axes, T)), inv=t(F32, (half,)), slots=t(I64, (T,)),
             cache=t(U8 if fp8 else BF16, (5, G, block, 2 * D))) | change
    a = {k: ref(x) for k, x in d.items()}
    parts = (ctypes.c_int32 * 4)(*sections) if sections else None
    ks = 1 << 12 if fp8 and scales else None
    return lib.sparse_decode_rope_append(a["q"], a["out"], a["k"], a["v"], a["pos"], a["inv"], parts, inter, adj, amp,
                                         a["slots"], a["cache"], ks, ks, ws, wsb, None)


def test_rope_refusals(lib):
    assert rope(lib, q=None) == INV                                          # query and its output come together
    assert rope(lib, v=None) == INV
    assert rope(lib, slots=None) == INV
    assert rope(lib, cache=None) == INV
    assert rope(lib, q=None, out=None, k=None, v=None) == INV
    assert rope(lib, out=t(BF16, (8, 5, 64))) == INV
    assert rope(lib, k=t(F32, (8, 2, 64))) == INV
    assert rope(lib, k=t(BF16, (7, 2, 64))) == INV
    assert rope(lib, v=t(BF16, (8, 3, 64))) == INV
    assert rope(lib, q=t(BF16, (8, 6, 64), (768, 128, 2))) == INV            # inner stride
    assert rope(lib, q=t(BF16, (8, 6, 64), (6 * 64 + 4, 64, 1))) == UNS      # row stride not 16 bytes
    assert rope(lib, q=t(BF16, (8, 6, 64), addr=(1 << 20) + 8)) == UNS       # base not 16 bytes
    assert rope(lib, out=t(BF16, (8, 6, 64), (0, 64, 1))) == INV             # output rows overlap
    assert rope(lib, out=t(BF16, (8, 6, 64), (6 * 128, 128, 1), addr=1 << 20)) == INV   # in place, other strides
    assert rope(lib, D=40, half=16) == UNS
    assert rope(lib, D=528, half=32) == UNS
    assert rope(lib, half=40) == INV                                         # more dims than the head has
    assert rope(lib, half=12) == UNS
    assert rope(lib, pos=t(I64, (1, 8))) == INV
    assert rope(lib, pos=t(I32, (1, 7))) == INV
    assert rope(lib, axes=2) == INV                                          # several axes need sections
    assert rope(lib, axes=5, sections=[8, 8, 8, 8]) == INV
    assert rope(lib, axes=2, sections=[16, 15, 0, 0]) == INV                 # do not add up
    assert rope(lib, axes=2, sections=[40, -8, 0, 0]) == INV
    assert rope(lib, axes=3, sections=[10, 12, 10, 0], inter=1) == INV       # axis 1 has 11 pairs in turn
    assert rope(lib, inv=None) == INV
    assert rope(lib, amp=float("inf")) == INV
    assert rope(lib, slots=t(I32, (8,))) == INV
    assert rope(lib, slots=t(I64, (8,), (2,))) == INV
    assert rope(lib, cache=t(F32, (5, 2, 16, 128))) == INV
    assert rope(lib, cache=t(BF16, (5, 3, 16, 128))) == INV
    assert rope(lib, cache=t(BF16, (5, 2, 16, 64))) == INV
    assert rope(lib, fp8=True, scales=False) == INV
    assert rope(lib, fp8=True, cache=t(U8, (5, 2, 16, 128), (2 * 16 * 128 + 8, 16 * 128, 128, 1))) == UNS
    assert rope(lib, ws=1 << 24, wsb=128) == WS
    assert rope(lib, ws=(1 << 24) + 16, wsb=256) == WS
    assert rope(lib, T=0) == OK                                              # nothing to do


def paged(lib, reqs=3, ql=2, G=2, H=8, D=128, W=5, block=16, fp8=False, scales=True, scale=0.1, ws=1 << 24, wsb=None,
          **change):
    rows = reqs * ql * G
    d = dict(q=t(BF16, (rows, H, D)), cache=t(U8 if fp8 else BF16, (9, G, block, 2 * D)), table=t(I32, (reqs, W)),
             lens=t(I32, (reqs,)), out=t(BF16, (rows, H, D)), lse=t(F32, (rows, H)), gate=None) | change
    a = {k: ref(x) for k, x in d.items()}
    ks = 1 << 12 if fp8 and scales else None
    need = lib.sparse_decode_paged_workspace_bytes(H, ql, D)
    return lib.sparse_decode_paged_attention(a["q"], a["cache"], a["table"], a["lens"], a["out"], a["lse"], scale, ql, ks,
                                             ks, a["gate"], ws, need if wsb is None else wsb, None)


def test_paged_refusals(lib):
    for name, bad in dict(q=t(F32, (12, 8, 128)), table=t(I64, (3, 5)), lens=t(F32, (3,)), out=t(BF16, (12, 8, 64)),
                          cache=t(BF16, (9, 2, 16, 192)), lse=t(F32, (12, 7)), gate=t(BF16, (6, 15))).items():
        assert paged(lib, **{name: bad}) == INV, name
    assert paged(lib, q=None) == INV
    assert paged(lib, lens=t(I32, (4,))) == INV                              # rows are not 4 requests'
    assert paged(lib, table=t(I32, (2, 5))) == INV
    assert paged(lib, G=3, q=t(BF16, (13, 8, 128)), out=t(BF16, (13, 8, 128)), lse=None) == INV
    assert paged(lib, q=t(BF16, (12, 8, 128), (2048, 256, 2))) == INV
    assert paged(lib, table=t(I32, (3, 5), (10, 2))) == INV
    assert paged(lib, lse=t(F32, (12, 8), (0, 1))) == INV
    assert paged(lib, out=t(BF16, (12, 8, 128), (0, 128, 1))) == INV
    assert paged(lib, ql=0) == INV
    assert paged(lib, scale=float("nan")) == INV
    assert paged(lib, fp8=True, scales=False) == INV
    assert paged(lib, D=96) == UNS
    assert paged(lib, H=65, ql=1) == UNS
    assert paged(lib, H=33, ql=2) == UNS                                     # more than 64 query rows
    assert paged(lib, block=12) == UNS
    assert paged(lib, cache=t(BF16, (9, 2, 16, 256), (2 * 16 * 256 + 4, 16 * 256, 256, 1))) == UNS
    assert paged(lib, cache=t(BF16, (9, 2, 16, 256), addr=(1 << 20) + 8)) == UNS
    assert paged(lib, ws=None) == WS
    assert paged(lib, ws=(1 << 24) + 128) == WS
    assert paged(lib, wsb=lib.sparse_decode_paged_workspace_bytes(8, 2, 128) - 1) == WS
    assert paged(lib, reqs=0) == OK


def test_paged_workspace_bytes(lib):
    f = sda.paged_workspace_bytes
    assert f(0) == f(65) == f(33, 2) == f(8, 1, 96) == f(8, 0) == 0
    items = 304 * 4 * 8 * 32                                                 # join list
    for heads, ql, dim, workers in ((16, 1, 192, 4), (8, 3, 128, 2), (64, 1, 64, 1), (1, 1, 256, 4), (16, 3, 192, 1)):
        ctas = 456 if dim == 64 and workers < 4 else 304                     # three to an SM, or two
        pieces = ctas * workers * 2 * heads * ql
        assert f(heads, ql, dim) == 256 + items + pieces * dim * 4 + -(-pieces * 4 // 256) * 256


def test_host_tensors_are_refused(lib):
    """Host tensors never reach the library: the binding raises before it allocates or calls."""
    lib_build.build_marshal()
    bf, i32 = torch.bfloat16, torch.int32
    q, cache = torch.zeros(4, 8, 64, dtype=bf), torch.zeros(3, 1, 16, 128, dtype=bf)
    n, slots = torch.ones(4, dtype=i32), torch.zeros(4, dtype=torch.int64)
    table = torch.zeros(4, 2, dtype=i32)
    before = dict(B._step_workspaces)
    for call in (lambda: sda.sparse_decode_plan_step(n, n, n, n[:2], table, block_size=16, slots=slots),
                 lambda: sda.sparse_decode_rope_append(q, q[:, :1], q[:, :1], n[None], torch.ones(32), slots, cache),
                 lambda: sda.sparse_decode_paged_attention(q, cache, table, n, q.clone(), scale=0.1)):
        with pytest.raises(ValueError, match="CUDA tensor"):
            call()
    assert B._step_workspaces == before


def test_marshalling_matches_the_header():
    """pack() skips what is not on a GPU, and names what it cannot describe."""
    lib_build.build_marshal()
    m = B.load_marshal()
    memory, where, device, current, stream, capturing = m.pack(None, None)
    assert where == (None, None) and device == -1 and len(memory) == 2 * ctypes.sizeof(B.SdaTensor)
    assert m.pack(torch.zeros(3), None)[2] == -2
    with pytest.raises(TypeError):
        m.pack(3)
    with pytest.raises(ValueError, match="one-element"):
        m.scalar(torch.zeros(1), 0)


def test_sections_go_with_axes():
    q = torch.zeros(2, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="axis"):
        sda.sparse_decode_rope_append(q, None, None, torch.zeros(2, 2, dtype=torch.int32), torch.ones(32), None, None,
                                      sections=[32])

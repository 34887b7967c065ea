"""A passed workspace counts for the memory that it has: tensors that are broadcast or have gaps are
refused, by every entry, before the library is called."""
import contextlib

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from sparse_decode_attention_02_gb300 import _binding as B
from sparse_decode_attention_02_gb300 import build as lib_build

WORKSPACES = [torch.zeros(1, dtype=torch.uint8).expand(1 << 20), torch.zeros(64, 300, dtype=torch.uint8)[:, :256],
              torch.zeros(1 << 12, dtype=torch.uint8)[::2]]


@pytest.fixture
def lib(monkeypatch):
    """The binding with host tensors let through to a library that fails the test."""
    lib_build.build()
    sda.load()

    class Lib:
        addresses = dict.fromkeys(("sparse_decode_plan_step", "sparse_decode_rope_append", "sparse_decode_paged_attention"), 1)

        def __getattr__(self, name):
            def entry(*a):
                raise AssertionError("reached the library")
            return entry if name in STEP + OLD else getattr(plain, name)

    class Marshal:
        pack = staticmethod(lambda *t: (b"", [None] * len(t), 0, 1, 0, 0))
        plan_step = rope_append = paged_attention = staticmethod(lambda *a: None)

    plain = B._lib
    monkeypatch.setattr(B, "_lib", Lib())
    monkeypatch.setattr(B, "_marshal", Marshal)
    monkeypatch.setattr(B, "_device_of", lambda *t, stream=None: torch.device("cpu"))
    monkeypatch.setattr(B, "_current", lambda dev: contextlib.nullcontext())


STEP = ("sparse_decode_plan_step", "sparse_decode_rope_append", "sparse_decode_paged_attention")
OLD = ("sparse_decode_attention", "sparse_decode_swa_attention", "sparse_decode_summary_scores")


def calls(ws):
    bf, i32 = torch.bfloat16, torch.int32
    q, out = torch.zeros(4, 16, 192, dtype=bf), torch.zeros(4, 16, 192, dtype=bf)
    cache, table = torch.zeros(8, 1, 16, 384, dtype=bf), torch.zeros(4, 2, dtype=i32)
    n, slots = torch.ones(4, dtype=i32), torch.zeros(4, dtype=torch.int64)
    return dict(
        sparse_decode_attention=lambda: sda.sparse_decode_attention(q, cache, table, table, n, n > 0, out, scale=0.1, splits=1,
                                                                    workspace=ws),
        sparse_decode_swa_attention=lambda: sda.sparse_decode_swa_attention(q, cache, table, n, out, scale=0.1, window=4,
                                                                            splits=1, workspace=ws),
        sparse_decode_summary_scores=lambda: sda.sparse_decode_summary_scores(
            torch.zeros(4, 1, 8, 256, dtype=torch.uint8), torch.zeros(4, 1, 8), torch.zeros(16, 1, 256, dtype=torch.uint8),
            table, n, block_size=16, workspace=ws),
        sparse_decode_plan_step=lambda: sda.sparse_decode_plan_step(n, n, n, n[:2], table, block_size=16, slots=slots,
                                                                    workspace=ws),
        sparse_decode_rope_append=lambda: sda.sparse_decode_rope_append(q, q[:, :1], q[:, :1], n[None], torch.ones(32), slots,
                                                                        cache, workspace=ws),
        sparse_decode_paged_attention=lambda: sda.sparse_decode_paged_attention(q, cache, table, n, out, scale=0.1,
                                                                                workspace=ws))


@pytest.mark.parametrize("name", STEP + OLD)
@pytest.mark.parametrize("which", range(len(WORKSPACES)))
def test_refused(lib, monkeypatch, name, which):
    ws = WORKSPACES[which]
    monkeypatch.setattr(torch.cuda, "current_stream", lambda dev=None: type("S", (), {"cuda_stream": 0}))
    monkeypatch.setattr(type(ws), "get_device", lambda t: 0)
    with pytest.raises(ValueError, match="contiguous"):
        calls(ws)[name]()

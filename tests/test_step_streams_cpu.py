"""What a call on a stream of its own allocates and fills belongs to that stream: shown without a
GPU, by where the binding makes its tensors."""
import contextlib

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from sparse_decode_attention_02_gb300 import _binding as B
from sparse_decode_attention_02_gb300 import build as lib_build


class Stream:
    cuda_stream = 77


@pytest.fixture
def made(monkeypatch):
    """(name, stream current there) of every tensor that torch makes meanwhile."""
    lib_build.build()
    sda.load()
    current, made = [None], []

    @contextlib.contextmanager
    def on(stream):
        current.append(stream)
        yield
        current.pop()

    def watched(name):
        plain = getattr(torch, name)

        def make(*a, **kw):
            made.append((name, current[-1]))
            return plain(*a, **kw)
        return make

    monkeypatch.setattr(torch.cuda, "stream", on)
    for name in ("zeros", "zeros_like", "empty", "empty_like", "full", "tensor"):
        monkeypatch.setattr(torch, name, watched(name))
    monkeypatch.setattr(B, "_call", lambda *a, **kw: 0)
    return made


@pytest.mark.parametrize("slots", [None, torch.zeros(2, dtype=torch.int64)])
def test_rotated_queries_are_made_on_the_calls_stream(made, slots):
    q, pos, inv = torch.ones(2, 1, 64, dtype=torch.bfloat16), torch.ones(1, 2, dtype=torch.int32), torch.ones(32)
    made.clear()
    stream = Stream()
    out = sda.sparse_decode_rope_append(q, None, None, pos, inv, slots, None, stream=stream)
    assert out.shape == q.shape and made and all(s is stream for _, s in made), made


def test_step_tables_are_made_on_the_calls_stream(made):
    n, slots = torch.ones(2, dtype=torch.int32), torch.zeros(3, dtype=torch.int64)
    made.clear()
    stream = Stream()
    sda.sparse_decode_plan_step(n, n, n, n, n[None], block_size=16, slots=slots, stream=stream)
    assert made and all(s is stream for _, s in made), made


def on_the_gpu(monkeypatch, lib_calls):
    """Lets host tensors through the older entries up to the library, whose entries `lib_calls` succeed."""
    class Lib:
        def __getattr__(self, name):
            return (lambda *a: 0) if name in lib_calls else getattr(B._lib, name)

    lib = Lib()
    monkeypatch.setattr(B, "load", lambda: lib)
    monkeypatch.setattr(B, "_device_of", lambda *t, stream=None: torch.device("cpu"))
    monkeypatch.setattr(B, "_current", lambda dev: contextlib.nullcontext())


def test_default_workspaces_are_made_on_their_stream(made, monkeypatch):
    monkeypatch.setattr(B, "_workspaces", {})
    made.clear()
    stream = Stream()
    ws = B.default_workspace("cpu", 300, stream)
    assert ws.numel() >= 300 and not ws.any() and made and all(s is stream for _, s in made), made


@pytest.mark.parametrize("name,call", [
    ("sparse_decode_select_regions", lambda s: sda.sparse_decode_select_regions(torch.ones(2, 9), torch.ones(2), 4, stream=s)),
    ("sparse_decode_summary_scores",
     lambda s: sda.sparse_decode_summary_scores(torch.ones(2, 1, 8, 256, dtype=torch.uint8), torch.ones(2, 1, 8),
                                                torch.ones(2, 1, 256, dtype=torch.uint8), torch.ones(2, 3, dtype=torch.int32),
                                                torch.ones(2, dtype=torch.int32), block_size=16, stream=s))])
def test_outputs_of_the_selection_are_made_on_the_calls_stream(made, monkeypatch, name, call):
    on_the_gpu(monkeypatch, {name})
    plain = torch.ones
    made.clear()
    stream = Stream()
    call(stream)
    assert plain is torch.ones and made and all(s is stream for _, s in made), made


def test_uploaded_scales_belong_to_the_calls_stream(made, monkeypatch):
    on_the_gpu(monkeypatch, {"sparse_decode_attention"})
    q, i32 = torch.ones(1, 1, 192, dtype=torch.bfloat16), torch.ones(1, 1, dtype=torch.int32)
    cache = torch.ones(1, 1, 16, 384, dtype=torch.uint8)
    ws = torch.ones(1 << 12, dtype=torch.uint8)
    made.clear()
    stream = Stream()
    sda.sparse_decode_attention(q, cache, i32, i32, i32[0], i32[0] > 0, q.clone(), scale=0.1, splits=1, k_scale=0.5,
                                v_scale=0.25, workspace=ws, stream=stream)
    assert len(made) == 2 and all(s is stream for _, s in made), made

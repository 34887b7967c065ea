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

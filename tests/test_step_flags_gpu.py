"""The flags of serving-step calls that pass no workspace can be read, and outlive its growth."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from test_paged_gpu import Problem

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda", 0)


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def out_of_pages(**kw):
    """Two prompts of two pages each, and three free pages."""
    tensors = i32(0, 0), i32(20, 20), i32(4, 5, 6), i32(0, 3), i32(-1, -1, -1, -1).view(2, 2)
    out = sda.sparse_decode_plan_step(*tensors, block_size=16, slots=torch.empty(40, dtype=torch.int64, device="cuda"), **kw)
    torch.cuda.synchronize()                                 # before the tensors go
    return out


def test_a_pool_that_ran_out_is_seen_without_a_workspace():
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        assert sda.read_errors(sda.step_workspace(DEV)) == 0
        lens = out_of_pages()[0]
        assert sda.read_errors(sda.step_workspace(DEV), clear=True) == sda.FLAG_FULL
        assert sda.read_errors(sda.step_workspace("cuda")) == 0
        assert lens.tolist() == [20, 0]


def test_flags_outlive_a_larger_call():
    """plan_step needs 256 bytes, attention some MB: the buffer is replaced between flag and reading."""
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    p = Problem([300, 7, 2000], D=64, G=2)
    torch.cuda.synchronize()
    out_of_pages(stream=s)
    small = sda.step_workspace(DEV, stream=s)
    out = torch.empty_like(p.query)
    torch.cuda.synchronize()
    sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, stream=s, **p.kw())
    s.synchronize()
    large = sda.step_workspace(DEV, stream=s)
    assert large.numel() > small.numel()
    assert sda.read_errors(large, clear=True, stream=s) == sda.FLAG_FULL
    p.check(out, p.run()[1])


def test_the_flags_of_another_stream_are_its_own():
    a, b = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    out_of_pages(stream=a)
    assert sda.read_errors(sda.step_workspace(DEV, stream=b), stream=b) == 0
    assert sda.read_errors(sda.step_workspace(DEV, stream=a), clear=True, stream=a) == sda.FLAG_FULL


def test_a_captured_step_shows_its_flags_in_the_workspace_it_was_given():
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    state = dict(context=i32(0, 0), new=i32(20, 20), ring=i32(4, 5, 6), free=i32(0, 3), table=i32(-1, -1, -1, -1).view(2, 2))
    slots = torch.empty(40, dtype=torch.int64, device="cuda")
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        sda.sparse_decode_plan_step(state["context"], state["new"], state["ring"], state["free"], state["table"],
                                    block_size=16, slots=slots, workspace=ws)
    assert sda.read_errors(ws) == 0
    g.replay()
    assert sda.read_errors(ws, clear=True) == sda.FLAG_FULL


def test_a_workspace_with_gaps_is_refused():
    for ws in (torch.zeros(1, dtype=torch.uint8, device="cuda").expand(256), torch.zeros(512, dtype=torch.uint8, device="cuda")[::2]):
        for kw in ({}, dict(stream=torch.cuda.current_stream())):
            with pytest.raises(ValueError, match="contiguous"):
                out_of_pages(workspace=ws, **kw)

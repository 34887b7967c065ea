"""The two ways a serving-step call is made: natively, and through ctypes where the binding has to
see to a stream, a workspace or a scale first.  They give the same bits, and refuse alike."""
import numpy as np
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import sparse_decode_attention_02_gb300._binding as B
from test_paged_gpu import KS, VS, Problem
from test_plan_gpu import problem, run
from test_rope_gpu import make, scales

pytestmark = pytest.mark.gpu


def ways():
    """Keyword arguments that choose either way."""
    return [{}, dict(stream=torch.cuda.current_stream())]


def test_plan_both_ways():
    import random
    a = problem(random.Random(4), 300, 16, 400, 0, 5, spare=4)
    got = [run(*a, workspace=None, **kw)[0] for kw in ways()]
    for k in got[0]:
        assert np.array_equal(got[0][k], got[1][k])


@pytest.mark.parametrize("fp8", [False, True])
def test_rope_both_ways(fp8):
    outs = []
    numbers = {name: x.item() for name, x in scales(fp8).items()}             # to be uploaded
    for kw in ways() + [numbers] * fp8:
        q, k, v, pos, inv, slots, cache = make(9, 4, 2, 64, 64, axes=3, fp8=fp8, seed=1)
        out = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, sections=np.array([10, 12, 10]),
                                            **{**scales(fp8), **kw})
        outs.append((out, cache))
    same = [torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for o in outs[1:] for a, b in zip(o, outs[0])]
    assert all(same)


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_both_ways(fp8):
    p = Problem([300, 7, 0, 90], D=128, fp8=fp8, ql=2, G=2)
    outs = []
    for kw in ways() + [dict(k_scale=float(np.float32(KS)), v_scale=float(np.float32(VS)))] * fp8:
        for ws in (p.workspace(), None):
            out = torch.empty_like(p.query)
            sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, workspace=ws,
                                              **{**p.kw(), **kw, "query_len": np.int64(2)})
            outs.append(out)
    same = [torch.equal(o, outs[0]) for o in outs]
    assert all(same)


def test_another_current_stream_gets_its_own_workspace():
    p = Problem([300, 7, 2000], D=64, G=2)
    want, _ = p.run()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        for _ in range(2):                                                    # the first makes it, the second finds it
            out = torch.empty_like(p.query)
            sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, out, **p.kw())
    s.synchronize()
    assert torch.equal(out, want) and (0, s.cuda_stream) in B._step_workspaces


@pytest.mark.parametrize("way", [0, 1])
def test_refusals_both_ways(way):
    kw = ways()[way]
    p = Problem([30, 7], D=64)
    call = lambda **change: sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, torch.empty_like(p.query),
                                                              **{**p.kw(), **kw, **change})
    for change in (dict(query_len=2 ** 32 + 1), dict(query_len=-2 ** 31 - 1)):
        with pytest.raises(OverflowError):
            call(**change)
    with pytest.raises(TypeError):
        call(query_len=1.5)
    with pytest.raises(sda.SdaError):
        call(query_len=0)
    with pytest.raises(sda.SdaError):
        call(workspace=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="CUDA"):
        call(workspace=torch.zeros(1 << 20, dtype=torch.uint8))
    with pytest.raises(ValueError, match="CUDA"):
        call(lse=torch.empty(2, 8))
    f = Problem([30, 7], D=64, fp8=True)
    for bad in (torch.tensor([KS]), torch.ones(2, device="cuda"), torch.ones(1, device="cuda").half()):
        with pytest.raises(ValueError, match="one-element"):
            sda.sparse_decode_paged_attention(f.query, f.cache, f.table, f.seq_lens, torch.empty_like(f.query),
                                              **{**f.kw(), **kw, "k_scale": bad})
    i32 = lambda n: torch.zeros(n, dtype=torch.int32, device="cuda")
    table, slots = i32(6).view(3, 2), torch.zeros(3, dtype=torch.int64, device="cuda")
    for change in (dict(block_size=2 ** 32 + 16), dict(block_size=16, rows_per_request=2 ** 40)):
        with pytest.raises(OverflowError):
            sda.sparse_decode_plan_step(i32(3), i32(3), i32(4), i32(2), table, slots=slots, **change, **kw)


@pytest.mark.parametrize("rows", [1, 1023, 1024, 1025, 4096, 4097])
def test_rows_around_one_a_thread(rows):
    """Packed token rows where a thread has one, and where warps take runs of them."""
    import random
    from test_plan_gpu import check
    r = random.Random(rows)
    a = list(problem(r, 200, 16, 100, 0, 2 * rows // 190 + 1, spare=7))
    a[-1] = rows
    check(*a, in_place=bool(rows & 1))

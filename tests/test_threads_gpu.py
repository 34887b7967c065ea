"""Host threads that call sparse and window attention with splits on one stream, each with its own
tensors: the same bits as the same calls in turn, whatever workspace they share."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from gpu_util import scales
from sparse_decode_attention_02_gb300 import inputs
from test_step_threads_gpu import in_threads

pytestmark = pytest.mark.gpu
CALLS = 150


def calls(share):
    """Calls of both kinds, as functions of the output; `share`: with one passed workspace, on the
    static scratch where there is one, or the default workspace."""
    work = [inputs.make_workload(inputs.scaled(name, requests=n, ctx=(4000, 9000)), "cuda:0", fill="all")
            for name, n in (("gqa", 3), ("swa", 2), ("gqa", 2), ("swa", 1))]
    ws = torch.zeros(max(sda.workspace_bytes(w.rows, w.heads, 4) for w in work), dtype=torch.uint8, device="cuda")
    out = []
    for w in work:
        ks, vs = scales(w)
        kw = dict(scale=w.scale, query_len=w.query_len, splits=4, k_scale=ks, v_scale=vs, gate=w.gate)
        if share == "passed":
            kw["workspace"] = ws
        if w.seq_lens is not None and getattr(w, "window", 0):
            out.append((w, lambda o, w=w, kw=kw: sda.sparse_decode_swa_attention(
                w.query, w.cache, w.block_table, w.seq_lens, o, window=w.window, **kw)))
        else:
            f = sda.sparse_decode_attention_no_alloc if share == "static" else sda.sparse_decode_attention
            out.append((w, lambda o, w=w, kw=kw, f=f: f(w.query, w.cache, w.regions, w.block_table, w.positions, w.active,
                                                        o, region_tokens=w.region_tokens, **kw)))
    return out


@pytest.mark.parametrize("share", ["default", "passed", "static"])
def test_split_calls(share):
    jobs, checks = [], []
    for w, call in calls(share):
        want = torch.full_like(w.query, float("nan"))
        call(want)
        mine = [torch.full_like(want, float("nan")) for _ in range(CALLS)]
        checks.append((want, mine))
        jobs.append(lambda call=call, mine=mine: [call(o) for o in mine])
    torch.cuda.synchronize()
    in_threads(jobs)
    torch.cuda.synchronize()
    for want, mine in checks:
        assert torch.isfinite(want).all() and all(torch.equal(o, want) for o in mine)

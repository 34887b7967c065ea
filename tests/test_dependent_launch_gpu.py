"""Split attention whose gate is written by the kernel right before it, one that lets its dependents
start early."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from gpu_util import scales
from sparse_decode_attention_02_gb300 import inputs

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["gqa", "swa"])
def test_a_gate_written_by_the_kernel_before(name):
    w = inputs.make_workload(inputs.scaled(name, requests=2, ctx=(4000, 9000)), "cuda:0", fill="all")
    tokens, width = w.gate.shape if w.gate is not None else (w.rows // w.config.groups, w.config.groups * w.heads)
    gate = torch.randn(tokens, width, device="cuda").mul_(2).bfloat16()
    ks, vs = scales(w)
    kw = dict(scale=w.scale, query_len=w.query_len, splits=8, k_scale=ks, v_scale=vs)

    def attend(gate, out):
        if name == "swa":
            sda.sparse_decode_swa_attention(w.query, w.cache, w.block_table, w.seq_lens, out, window=w.window, gate=gate, **kw)
        else:
            sda.sparse_decode_attention(w.query, w.cache, w.regions, w.block_table, w.positions, w.active, out, gate=gate,
                                        region_tokens=w.region_tokens, **kw)

    want = torch.zeros_like(w.query)
    attend(gate, want)
    # the gate is the end of a large copy: rotary positions are left out, so rows pass through
    rows = 1 << 21
    source = torch.zeros(rows, width // 16, 16, dtype=torch.bfloat16, device="cuda")
    source[-tokens:] = gate.view(tokens, -1, 16)
    copy = torch.empty_like(source)
    outs = [torch.zeros_like(want) for _ in range(30)]
    for out in outs:
        copy.fill_(-30.0)                                     # a gate of about 0
        sda.sparse_decode_rope_append(source, None, None, None, None, None, None, copy)
        attend(copy[-tokens:].view(tokens, width), out)
    torch.cuda.synchronize()
    assert torch.isfinite(want).all() and all(torch.equal(o, want) for o in outs)

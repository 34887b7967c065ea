"""A host thread whose first CUDA work is a call of this library, everything being passed to it."""
import threading

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from gpu_util import scales
from sparse_decode_attention_02_gb300 import inputs
from test_paged_gpu import Problem

pytestmark = pytest.mark.gpu


def in_a_new_thread(job):
    torch.cuda.synchronize()
    wrong = []

    def run():
        try:
            job()
        except BaseException as e:      # noqa: BLE001 - handed to the test
            wrong.append(e)

    t = threading.Thread(target=run)
    t.start()
    t.join()
    torch.cuda.synchronize()
    if wrong:
        raise wrong[0]


@pytest.mark.parametrize("spare", [0, 900])
def test_whole_cache_attention(spare):
    p = Problem([300, 7, 2000], D=64, G=2, spare=spare)
    want, want_lse = p.run()
    got, lse, ws, kw = torch.zeros_like(want), torch.zeros_like(want_lse), p.workspace(), p.kw()
    in_a_new_thread(lambda: sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, got, lse=lse,
                                                              workspace=ws, **kw))
    assert torch.equal(got, want) and torch.equal(lse, want_lse)


def test_sparse_and_window_attention():
    for name in ("gqa", "swa"):
        w = inputs.make_workload(inputs.scaled(name, requests=3, ctx=(4000, 9000)), "cuda:0", fill="all")
        ks, vs = scales(w)
        ws = torch.zeros(sda.workspace_bytes(w.rows, w.heads, 4), dtype=torch.uint8, device="cuda")

        def call(out):
            kw = dict(scale=w.scale, query_len=w.query_len, splits=4, k_scale=ks, v_scale=vs, gate=w.gate, workspace=ws)
            if name == "swa":
                sda.sparse_decode_swa_attention(w.query, w.cache, w.block_table, w.seq_lens, out, window=w.window, **kw)
            else:
                sda.sparse_decode_attention(w.query, w.cache, w.regions, w.block_table, w.positions, w.active, out,
                                            region_tokens=w.region_tokens, **kw)
        want, got = torch.zeros_like(w.query), torch.zeros_like(w.query)
        call(want)
        in_a_new_thread(lambda: call(got))
        assert torch.equal(got, want)


def test_indexer_scores():
    w = inputs.make_index_workload("cuda:0", requests=3, groups=4, query_len=1, block=64, ctx=(5000, 9000))
    want, got = (torch.zeros(w.rows, w.n_cols, device="cuda") for _ in range(2))
    kw = dict(block_size=w.block, query_len=w.query_len)
    sda.sparse_decode_summary_scores(w.query, w.weights, w.summaries, w.block_table, w.seq_lens, scores=want, **kw)
    in_a_new_thread(lambda: sda.sparse_decode_summary_scores(w.query, w.weights, w.summaries, w.block_table, w.seq_lens,
                                                             scores=got, **kw))
    assert torch.equal(got, want)

"""Host threads that call whole-cache attention on one stream, each with its own tensors: the same
bits as the same calls in turn, whether they share the default workspace or one that is passed."""
import threading

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from test_paged_gpu import Problem

pytestmark = pytest.mark.gpu
CALLS = 150


def in_threads(jobs):
    """Runs the jobs at once, all beginning together; raises what one of them raised."""
    start, wrong = threading.Barrier(len(jobs)), []

    def run(job):
        try:
            start.wait()
            job()
        except BaseException as e:      # noqa: BLE001 - handed to the test
            wrong.append(e)

    threads = [threading.Thread(target=run, args=(j,)) for j in jobs]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    if wrong:
        raise wrong[0]


@pytest.mark.parametrize("way", ["native", "ctypes", "passed"])
def test_requests_that_are_cut(way):
    # tables wide enough that every call cuts its units and joins the pieces
    problems = [Problem([5000, 77, 1200], G=2, H=16, D=128, seed=1, spare=300),
                Problem([9000], G=2, H=16, D=128, seed=2, spare=300),
                Problem([2000, 3100, 0, 40, 777, 2500], G=2, H=16, D=128, seed=3, spare=300),
                Problem([3000, 41], G=1, H=8, D=128, ql=2, seed=4, spare=300)]
    want = [p.run() for p in problems]
    ws = torch.zeros(max(p.workspace().numel() for p in problems), dtype=torch.uint8, device="cuda")
    kw = dict(native={}, ctypes=dict(stream=torch.cuda.current_stream()), passed=dict(workspace=ws))[way]
    outs = [[(torch.full_like(o, float("nan")), torch.full_like(l, float("nan"))) for _ in range(CALLS)] for o, l in want]
    keys = [p.kw() for p in problems]
    for p, k, (o, l) in zip(problems, keys, want):           # the default workspace has its size
        sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, o, lse=l, **k, **kw)
    torch.cuda.synchronize()

    def job(p, k, mine):
        def run():
            for o, l in mine:
                sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, o, lse=l, **k, **kw)
        return run

    in_threads([job(*x) for x in zip(problems, keys, outs)])
    torch.cuda.synchronize()
    for (o, l), mine in zip(want, outs):
        assert all(torch.equal(a, o) and torch.equal(b, l) for a, b in mine)


def test_whole_steps_and_growing_workspaces():
    """Threads on a stream whose default workspace is still to be made, and grows on the way: tables,
    rotated keys and attention, each thread's with the results that it has alone."""
    stream = torch.cuda.Stream()

    def job(seed, results):
        p = Problem([900 * seed, 30], G=2, H=4 * seed, D=64 * seed, seed=seed, spare=200)
        want = p.run()
        got = torch.empty_like(want[0]), torch.empty_like(want[1])
        i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")
        plan = i32(5, 16), i32(1, 2), i32(7, 8, 9, 10), i32(1, 3), i32(0, -1, 1, -1).view(2, 2)
        slots = torch.empty(4, dtype=torch.int64, device="cuda")
        k = p.kw()
        torch.cuda.synchronize()

        def run():
            with torch.cuda.stream(stream):
                for _ in range(40):
                    sda.sparse_decode_plan_step(*plan, block_size=16, slots=slots)
                    sda.sparse_decode_paged_attention(p.query, p.cache, p.table, p.seq_lens, got[0], lse=got[1], **k)
            results[seed] = (want, got, slots, plan)
        return run

    results = {}
    in_threads([job(seed, results) for seed in (1, 2, 3, 4)])
    torch.cuda.synchronize()
    for (o, l), (a, b), slots, plan in results.values():
        assert torch.equal(o, a) and torch.equal(l, b)
        assert slots.tolist() == [5, 8 * 16, 8 * 16 + 1, -1]

"""Block tables that are not as wide as the longest request: wider ones give the same values whatever
their width, and a length past a narrow one counts as what the table holds."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
from test_paged_gpu import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ql", [1, 3])
def test_a_length_past_the_table_counts_as_the_table(fp8, ql):
    for spare in (0, 400):                                    # (cut, not cut: the longest request sets the width)
        p = Problem([16 * 40, 90, 16 * 40, 0], D=128, H=8, G=2, block=16, fp8=fp8, ql=ql)
        p.table[:, 7:] = torch.where(p.table[:, 7:] < 0, p.table[:, :1], p.table[:, 7:])
        if spare:
            page = p.table[:1, :1].expand(4, spare)
            p.table = torch.cat([p.table, page], 1)
            p.lens[0] = p.lens[2] = 16 * (40 + spare)
        p.lens = [p.table.shape[1] * 16 if n > 90 else n for n in p.lens]
        p.seq_lens.copy_(torch.tensor([p.lens[0] + 1, 90, 2 ** 31 - 1, 0]))
        out, lse = p.run(flags=sda.FLAG_BOUNDS)
        p.check(out, lse)


@pytest.mark.parametrize("lens", [[40], [211] * 46, [5, 0, 700, -1, 33]])
@pytest.mark.parametrize("fp8", [False, True])
def test_a_narrow_view_of_a_wide_table(lens, fp8):
    p = Problem(lens, D=192, H=8, G=2, block=16, fp8=fp8, spare=4000)
    out, lse = torch.full_like(p.query, 5.0), torch.full(p.query.shape[:2], 6.0, device="cuda")
    p.run(out=out, lse=lse)
    p.check(out, lse)
    need = max(1, -(-max(lens) // 16))
    p.run(out=out, lse=lse, table=p.table[:, :need])
    p.check(out, lse)

"""What a later token's value scale is does not reach the rows that do not see it: draft tokens whose values are far larger than
the tokens' before them, in a block of their own."""
import pytest
import torch

from test_quantised_attention_gpu import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("power", [12, 40, 110])
@pytest.mark.parametrize("lens,G,H,D,block,span,spare", [
    ([17, 18, 0, 33, 34, 15], 2, 4, 128, 16, 16, 0),            # by workers and CTAs alone
    ([2001, 1602, 17], 2, 4, 192, 64, 16, 0),                   # by clusters
    ([700, 641, 1, 3], 1, 8, 64, 32, 32, 0),                    # two tiles of rows
    ([5009, 33, 290], 2, 16, 128, 48, 16, 0),                   # four
    ([30001, 402], 1, 5, 256, 24, 8, 0),                        # over the line
    ([513, 9, 26] * 30, 2, 4, 64, 16, 8, 100),
])
def test_later_value_scales(lens, G, H, D, block, span, spare, power, int8):
    ql = 4
    p = Problem(lens, G=G, H=H, D=D, block=block, span=span, ql=ql, int8=int8, spare=spare, gate=D == 192)
    want, want_l = p.run()
    unseen = torch.zeros(p.query.shape[0], dtype=torch.bool)
    for q, n in enumerate(lens):
        first = (n - 1) // span * span                          # of the newest token's block
        page, part = p.pages[q][first // block] if n else None, first % block // span
        for j in range(ql if n else 0):
            if n - ql + 1 + j <= first:
                unseen[(q * ql + j) * G:(q * ql + j + 1) * G] = True
        if n and first >= n - ql + 1:                           # some row does not see it
            p.scales[page, :, part, 1] *= 2.0 ** power
    out, lse = p.run()
    p.check(out, lse)
    assert torch.equal(lse, want_l)
    assert unseen.any() and torch.equal(out.cpu()[unseen], want.cpu()[unseen])
    assert not torch.equal(out.cpu()[~unseen], want.cpu()[~unseen])

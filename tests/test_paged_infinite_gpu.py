"""Whole-cache attention over a bf16 cache in which some values are infinite."""
import pytest
import torch

import step_util
from test_paged_gpu import Problem

pytestmark = pytest.mark.gpu
INF = float("inf")


# (lens, spare table columns): a CTA alone with a unit, and units that are cut and joined
FORMS = [([150, 33, 700], 0), ([150, 33, 5000], 900)]


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("H,ql", [(8, 1), (16, 2), (16, 4)])
@pytest.mark.parametrize("lens,spare", FORMS)
def test_an_infinite_value_gives_an_infinity(D, H, ql, lens, spare):
    """V of a few tokens holds +inf or -inf in some dims (both signs in one): the rows that see the token
    get that infinity there, NaN where both meet, as sum_t w_t v_t has it; the other dims are unharmed."""
    p = Problem(lens, G=2, H=H, D=D, block=16, ql=ql, spare=spare, q_std=1.0)
    plant = {3: INF, 7: -INF, 8: INF}                        # dim: value
    for q, n in enumerate(lens):
        for d, x in plant.items():
            at = (5 * d + 2) % (n - ql)                      # every query token sees it
            p.cache[p.table[q, at // 16], :, at % 16, D + d] = x
        at = n - ql - 1
        p.cache[p.table[q, at // 16], :, at % 16, D + 8] = -INF
    out, lse = p.run()
    got = out.cpu().float()
    assert (got[..., 3] == INF).all() and (got[..., 7] == -INF).all() and torch.isnan(got[..., 8]).all()
    o, l, spread, slack = p.exact()
    rest = [d for d in range(D) if d not in plant]
    bound = step_util.attention_bound(o, spread, slack, False)
    assert ((got.double() - o).abs() <= bound)[..., rest].all()
    assert ((lse.cpu().double() - l).abs() <= slack + l.abs() * 2.0 ** -22 + 2.0 ** -18).all()


def test_an_infinite_value_of_the_newest_tokens():
    """Only the query tokens from its own on see it."""
    p = Problem([130, 64, 333], G=2, H=4, D=128, ql=4, block=16, spare=60)
    for q, n in enumerate(p.lens):
        p.cache[p.table[q, (n - 2) // 16], :, (n - 2) % 16, 128 + 5] = -INF
    got = p.run()[0].cpu().float().view(3, 4, 2, 4, 128)
    assert (got[:, 2:, ..., 5] == -INF).all() and torch.isfinite(got[:, :2]).all()
    assert torch.isfinite(got[..., [d for d in range(128) if d != 5]]).all()

"""Whole-cache attention over an E4M3 cache where one token in 64 takes nearly all of the weight."""
import math

import pytest
import torch

import step_util
from test_paged_gpu import KS, VS, Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("D", [64, 128, 192, 256])
@pytest.mark.parametrize("H,ql", [(8, 1), (16, 2), (16, 4)])
@pytest.mark.parametrize("lens,spare", [([700, 1500], 0), ([700, 1500], 900)])
@pytest.mark.parametrize("gap", [8, 12, 14, 16, 17.5, 18, 24])
def test_weights_far_below_the_largest(D, H, ql, lens, spare, gap):
    """Every 64th token takes nearly all of the weight and has V = 0; the others, `gap` nats below, have
    V = 1 and are all of the output.  Their weights keep 11 bits down to 2^-27 of the largest (18.7
    nats), beyond it 2^-38 of the largest absolutely; lse counts them in fp32."""
    p = Problem(lens, G=2, H=H, D=D, block=16, ql=ql, spare=spare, fp8=True)
    page = torch.zeros(16, 2 * D)
    page[:, D:] = 64.0                                       # V of the others, exact in E4M3
    sink = page.clone()
    sink[0, :D], sink[0, D:] = 32.0, 0.0
    e4m3 = lambda x: x.to(torch.float8_e4m3fn).view(torch.uint8).cuda()
    for q, n in enumerate(lens):
        for c in range(-(-n // 16)):
            p.cache[p.table[q, c]] = e4m3(sink if c % 4 == 0 else page)
    p.query.zero_()
    p.query[..., 0] = 4.0
    p.scale = gap / (4.0 * 32.0 * float(torch.tensor(KS)))
    out, lse = p.run()
    o, l, spread, slack = p.exact()
    largest = torch.exp(gap - l)[..., None]                  # weight of a sink
    far = 2.0 ** -38 * largest * max(lens) * 64.0 * VS
    bound = step_util.attention_bound(o, spread, slack, True) + (far if gap > 27 * math.log(2.0) else 0.0)
    worst = ((out.cpu().double() - o).abs() / bound).max().item()
    assert worst <= 1.0, f"error {worst:.2f} times its bound"
    assert ((lse.cpu().double() - l).abs() <= slack + l.abs() * 2.0 ** -22 + 2.0 ** -18).all()

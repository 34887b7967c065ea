"""Queries and scales at the ends of fp32's exponents, whose logits and outputs are ordinary ones or fit: attention over a
quantised cache against float64, within the bounds of every other size."""
import pytest
import torch

from test_quantised_attention_gpu import Problem

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("power", [-118, -60, 60, 118, 120, 121, 122, 124])
@pytest.mark.parametrize("lens,ql,regions", [([301, 40], 1, None), ([5000], 2, None), ([700, 30], 1, (12, 8))])
def test_large_queries_beside_small_key_scales(lens, ql, regions, power, int8):
    p = Problem(lens, G=2, H=8, D=192, block=16, span=8, ql=ql, int8=int8, q_std=2.0 ** power, regions=regions)
    p.scales[..., 0] *= 2.0 ** -power
    assert p.query.isfinite().all() and (p.scales[..., 0].nan_to_num(1.0) > 0).all()
    p.check(*p.run(regions=regions is not None), regions=regions is not None)


@pytest.mark.parametrize("int8", [False, True])
@pytest.mark.parametrize("lens,ql,G,regions", [([301, 40], 1, 2, None), ([30, 20], 3, 2, None), ([5000], 2, 4, None), ([30000], 1, 2, None),
                                               ([700, 30], 1, 2, (12, 8))])
def test_the_largest_value_scales(lens, ql, G, regions, int8):
    """2^126 in every block, and in some beside 1: elements of at most 1, whose values fit in fp32."""
    p = Problem(lens, G=G, H=8, D=64, block=16, span=8, ql=ql, int8=int8, regions=regions, scale_std=0.0)
    gen = torch.Generator().manual_seed(5)
    ones = torch.randint(-1, 2, p.cache.shape[:3] + (64,), generator=gen).cuda()
    p.cache[..., 64:] = ones.to(torch.int8) if int8 else ones.float().to(torch.float8_e4m3fn).view(torch.uint8)
    for some in (False, True):
        held = ~p.scales[..., 1].isnan()
        large = torch.rand(p.scales.shape[:3], generator=gen).cuda() < (0.3 if some else 1.0)
        p.scales[..., 1] = torch.where(held, torch.where(large, 2.0 ** 126, 1.0), p.scales[..., 1])
        p.check(*p.run(regions=regions is not None), regions=regions is not None)

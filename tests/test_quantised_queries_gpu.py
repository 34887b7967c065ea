"""Queries and key scales at the two ends of fp32's exponents, whose logits are ordinary ones: attention over a quantised
cache against float64, within the bounds of every other size."""
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

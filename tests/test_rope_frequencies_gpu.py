"""Rotary angles of large frequencies at far positions.  Frequencies are multiples of 1/4 up to 1024
(12 bits) and positions have 31, so float64 holds the products exactly; the kernel's angle is off by
1024 * 2^-32 of a turn at most (2^-19.3 rad), its sine and cosine by 2^-24 * 2 pi (2^-21.3)."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import step_util
from test_rope_gpu import bf16_bound

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("far", [5, 1 << 20, 2 ** 31 - 1])
@pytest.mark.parametrize("sign", [1, -1])
def test_large_frequencies(far, sign):
    gen = torch.Generator().manual_seed(far % 1000)
    q = torch.randn(50, 3, 128, generator=gen).bfloat16().cuda()
    pos = torch.randint(-far, far, (1, 50), generator=gen).int().cuda()
    pos[0, 0], pos[0, 1] = far, -far
    inv = (sign * (1024.0 - 7.0 * torch.arange(64) / 4)).cuda()
    out = sda.sparse_decode_rope_append(q, None, None, pos, inv, None, None)
    want, size = step_util.rotate(q.cpu(), pos.cpu(), inv.cpu(), None)
    assert ((out.cpu().double() - want).abs() <= bf16_bound(want, size) + size * 2.0 ** -19).all()

"""A decode step over a quantised cache with queries turned into a buffer of their own and keys in place, as the README has
it: the same bits as with both turned in place and the queries copied."""
import pytest
import torch

import sparse_decode_attention_02_gb300 as sda

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("int8", [False, True])
def test_turned_into_a_buffer_or_in_place(int8):
    n, groups, heads, dim, B, S = 9, 2, 4, 128, 32, 16
    gen = torch.Generator().manual_seed(3)
    inv_freq = (10000.0 ** (-torch.arange(dim // 2).double() / (dim // 2))).float().cuda()
    context = torch.tensor([1, 40, 0, 64, 65, 17, 100, 33, 2], dtype=torch.int32, device="cuda")
    new = torch.tensor([1, 1, 1, 1, 0, 1, 1, 1, 1], dtype=torch.int32, device="cuda")
    start = torch.randn(40, groups, B, 2 * dim, generator=gen).mul(30).clamp(-100, 100)
    start = (start.round().to(torch.int8) if int8 else start.to(torch.float8_e4m3fn)).cuda()
    qkv0 = torch.randn(n, (heads + 2) * groups * dim, generator=gen).bfloat16().cuda()
    got = []
    for into_a_buffer in (False, True):
        cache, scales, qkv, lens = start.clone(), torch.full((40, groups, B // S, 2), 0.02, device="cuda"), qkv0.clone(), context.clone()
        table = torch.arange(36, dtype=torch.int32, device="cuda").view(9, 4).clone()
        ring, state = torch.arange(36, 40, dtype=torch.int32, device="cuda"), torch.tensor([0, 4], dtype=torch.int32, device="cuda")
        slots = torch.empty(n, dtype=torch.int64, device="cuda")
        _, _, _, positions, _, _ = sda.sparse_decode_plan_step(lens, new, ring, state, table, block_size=B, slots=slots,
                                                               rows_per_request=1, seq_lens=lens, free_next=state)
        output = torch.zeros(n * groups, heads, dim, dtype=torch.bfloat16, device="cuda")
        q, k, v = qkv.view(n, -1, dim).split([heads * groups, groups, groups], dim=1)
        if into_a_buffer:
            rotated = q.contiguous()                          # rows of requests that are idle are left as they were
            sda.sparse_decode_rope_append(q, None, None, positions[None], inv_freq, slots, None, rotated)
            sda.sparse_decode_rope_append(k, None, None, positions[None], inv_freq, slots, None, k)
            q = rotated.view(n * groups, heads, dim)
        else:
            qk = qkv.view(n, -1, dim)[:, :heads * groups + groups]
            sda.sparse_decode_rope_append(qk, None, None, positions[None], inv_freq, slots, None, qk)
            q = q.reshape(n * groups, heads, dim)
        sda.sparse_decode_quantised_append(k, v, slots, cache, scales)
        sda.sparse_decode_quantised_paged_attention(q, cache, scales, table, lens, output, scale=dim ** -0.5)
        got.append((q.clone(), cache.view(torch.uint8), scales, output, slots))
    assert all(torch.equal(a, b) for a, b in zip(*got))
    assert (got[0][4] >= 0).sum() == 8 and got[0][3].isfinite().all() and not torch.equal(got[0][1], start.view(torch.uint8))

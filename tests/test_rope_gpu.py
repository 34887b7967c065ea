"""Rotary positions and the paged cache write, against the float64 formula.

bf16 outputs are off by half a step (2^-8 of the value), E4M3 ones by 2^-4 of it (2^-10 below the
smallest normal value); cos, sin and the two products round in fp32: 2^-21 of |a| + |b| at most."""
import math

import pytest
import torch

import sparse_decode_attention_02_gb300 as sda
import step_util

pytestmark = pytest.mark.gpu
KS, VS = 8.0 / 448.0, 5.0 / 448.0


def make(T, Hq, G, D, rot, axes=1, block=16, fp8=False, seed=0, far=300000, fused=False):
    gen = torch.Generator().manual_seed(seed + 7919 * T + D)
    width = (Hq + 2 * G) * D
    qkv = torch.randn(T, width, generator=gen).bfloat16().cuda()
    parts = [x.view(T, -1, D) for x in qkv.split([Hq * D, G * D, G * D], dim=1)]
    q, k, v = parts if fused else [x.contiguous() for x in parts]
    pos = torch.randint(-5, far, (axes, T), generator=gen).int().cuda()
    inv = (10000.0 ** (-torch.arange(rot // 2).double() / (rot // 2))).float().cuda()
    pages = -(-T // block) + 2
    slots = torch.randperm(pages * block, generator=gen)[:T].cuda()
    shape = (pages, G, block, 2 * D)
    cache = (torch.randint(0, 120, shape, generator=gen).to(torch.uint8) if fp8
             else torch.randn(shape, generator=gen).bfloat16()).cuda()
    return q, k, v, pos, inv, slots, cache


def scales(fp8):
    return dict(k_scale=torch.tensor([KS], device="cuda"), v_scale=torch.tensor([VS], device="cuda")) if fp8 else {}


def bf16_bound(x, size):
    return x.abs() * 2.0 ** -8 + size * 2.0 ** -21 + 2.0 ** -130


def check(args, out, before, fp8, *, sections=None, interleaved=False, adjacent=False, amplitude=1.0):
    q, k, v, pos, inv, slots, cache = [None if x is None else x.cpu() for x in args]
    kw = dict(sections=sections, interleaved=interleaved, adjacent=adjacent, amplitude=amplitude)
    live = slots >= 0
    if q is not None:
        want, size = step_util.rotate(q, pos, inv, **kw)
        got = out.cpu().double()
        assert ((got - want).abs() <= bf16_bound(want, size))[live].all()
    if k is None:
        return
    want_k, size = step_util.rotate(k, pos, inv, **kw)
    got = cache.permute(0, 2, 1, 3).reshape(-1, cache.shape[1], cache.shape[3])   # [slot, G, 2D]
    old = before.cpu().permute(0, 2, 1, 3).reshape(got.shape)
    rest = torch.ones(got.shape[0], dtype=torch.bool)
    rest[slots[live]] = False
    assert torch.equal(got[rest], old[rest]), "a slot that was not named changed"
    D = k.shape[2]
    new = got[slots[live]]
    if fp8:
        val = step_util.e4m3_values(new)
        for x, sz, y, sc in ((want_k, size, val[..., :D], KS), (v.double(), v.double().abs(), val[..., D:], VS)):
            sc = float(torch.tensor(sc, dtype=torch.float32))
            x, sz = (x[live] / sc).clamp(-448, 448), sz[live] / sc
            assert ((y - x).abs() <= x.abs() * 2.0 ** -4 + 2.0 ** -10 + sz * 2.0 ** -20).all()
    else:
        assert ((new[..., :D].double() - want_k[live]).abs() <= bf16_bound(want_k, size)[live]).all()
        assert torch.equal(new[..., D:], v[live])


@pytest.mark.parametrize("T,Hq,G,D,rot", [(1, 8, 1, 192, 192), (1, 1, 1, 64, 16), (3, 16, 2, 128, 64), (33, 5, 1, 192, 128),
                                          (257, 24, 3, 256, 256), (1001, 8, 2, 64, 64), (2500, 4, 1, 192, 96),
                                          (5, 2, 1, 16, 16), (70, 40, 8, 512, 512), (12, 3, 2, 80, 48)])
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("adjacent", [False, True])
def test_one_axis(T, Hq, G, D, rot, fp8, adjacent):
    a = make(T, Hq, G, D, rot, fp8=fp8, fused=T % 2 == 1)
    before = a[6].clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    out = sda.sparse_decode_rope_append(*a, adjacent_pairs=adjacent, workspace=ws, **scales(fp8))
    assert sda.read_errors(ws) == 0
    check(a, out, before, fp8, adjacent=adjacent)


@pytest.mark.parametrize("sections,interleaved", [([16, 24, 24], False), ([22, 21, 21], True), ([64], True), ([0, 64], False),
                                                  ([40, 24], True), ([10, 20, 4, 30], False), ([28, 4, 16, 16], True),
                                                  ([64, 0, 0], True)])
@pytest.mark.parametrize("fp8,adjacent", [(False, False), (True, True)])
def test_several_axes(sections, interleaved, fp8, adjacent):
    a = make(77, 6, 2, 192, 128, axes=len(sections), fp8=fp8)
    before = a[6].clone()
    out = sda.sparse_decode_rope_append(*a, sections=sections, interleaved_axes=interleaved, adjacent_pairs=adjacent,
                                        amplitude=1.25, **scales(fp8))
    check(a, out, before, fp8, sections=sections, interleaved=interleaved, adjacent=adjacent, amplitude=1.25)


@pytest.mark.parametrize("far", [1, 1 << 20, 2 ** 31 - 1])
def test_far_positions_keep_their_angle(far):
    """Up to 2^31: an fp32 angle would be off by whole turns there; 2^-53 of f leaves 2^-22 turns."""
    a = make(40, 2, 1, 64, 64, far=far)
    out = sda.sparse_decode_rope_append(*a)
    want, size = step_util.rotate(a[0].cpu(), a[3].cpu(), a[4].cpu(), None)
    assert ((out.cpu().double() - want).abs() <= bf16_bound(want, size) + size * 2.0 ** -19).all()


def test_padding_rows_are_left_alone():
    for fp8 in (False, True):
        q, k, v, pos, inv, slots, cache = make(50, 8, 2, 128, 128, fp8=fp8)
        slots[[0, 7, 48, 49]] = -1
        for t in (q, k, v):
            t[slots < 0] = float("nan")
        out = torch.full_like(q, 3.0)
        before = cache.clone()
        sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, out, **scales(fp8))
        assert (out[slots < 0] == 3.0).all()
        check((q, k, v, pos, inv, slots, cache), out, before, fp8)


def test_slots_outside_the_cache_are_flagged_and_left_out():
    q, k, v, pos, inv, slots, cache = make(20, 4, 1, 64, 64)
    n = cache.shape[0] * cache.shape[2]
    slots[3], slots[11], slots[12] = n, -2, 2 ** 62
    out, before = torch.full_like(q, 3.0), cache.clone()
    ws = torch.zeros(256, dtype=torch.uint8, device="cuda")
    sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, out, workspace=ws)
    assert sda.read_errors(ws) == sda.FLAG_BOUNDS
    assert (out[[3, 11, 12]] == 3.0).all()
    slots[[3, 11, 12]] = -1
    check((q, k, v, pos, inv, slots, cache), out, before, False)


def test_parts_alone_and_in_place():
    q, k, v, pos, inv, slots, cache = make(31, 8, 2, 192, 192)
    before = cache.clone()
    whole = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache)
    after = cache.clone()
    cache.copy_(before)
    assert torch.equal(sda.sparse_decode_rope_append(q, None, None, pos, inv, None, None), whole)
    assert torch.equal(cache, before)
    assert sda.sparse_decode_rope_append(None, k, v, pos, inv, slots, cache) is None
    assert torch.equal(cache, after)
    mine = q.clone()
    assert sda.sparse_decode_rope_append(mine, None, None, pos, inv, None, None, mine) is mine
    assert torch.equal(mine, whole)
    # no positions: keys and values as they are
    sda.sparse_decode_rope_append(None, k, v, None, None, slots, cache)
    got = cache.permute(0, 2, 1, 3).reshape(-1, 2, 384)[slots]
    assert torch.equal(got, torch.cat([k, v], -1))
    # positions of stride 0: one for all tokens
    one = pos[:, :1].expand(1, 31)
    a = sda.sparse_decode_rope_append(q, None, None, one, inv, None, None)
    b = sda.sparse_decode_rope_append(q, None, None, one.contiguous(), inv, None, None)
    assert torch.equal(a, b)


def test_padded_page_stride_and_saturation():
    T, G, D, B = 24, 2, 64, 8
    q, k, v, pos, inv, slots, _ = make(T, 2, G, D, 64, block=B)
    pages = 5
    slots = torch.randperm(pages * B)[:T].cuda()
    k *= 100.0                                          # past 448 * KS: saturates
    k[0, 0, 0], v[1, 0, 3], v[2, 1, 4] = float("inf"), float("-inf"), float("nan")
    pos[:, 0] = 0
    raw = torch.zeros(pages, G * B * 2 * D + 64, dtype=torch.uint8, device="cuda")
    cache = raw[:, :G * B * 2 * D].view(pages, G, B, 2 * D)
    sda.sparse_decode_rope_append(None, k, v, pos, inv, slots, cache, **scales(True))
    assert (raw[:, G * B * 2 * D:] == 0).all()
    val = step_util.e4m3_values(cache.cpu().contiguous()).permute(0, 2, 1, 3).reshape(-1, G, 2 * D)[slots.cpu()]
    assert val[1, 0, D + 3] == -448 and torch.isnan(val[2, 1, D + 4])
    want, size = step_util.rotate(k.cpu(), pos.cpu(), inv.cpu(), None)
    x = (want / float(torch.tensor(KS))).clamp(-448, 448)
    fine = torch.isfinite(want)
    fine[0] = False
    bound = x.abs() * 2.0 ** -4 + 2.0 ** -10 + size / KS * 2.0 ** -20
    assert ((val[..., :D] - x).abs() <= bound)[fine].all() and (x[fine].abs() == 448).any()


def test_graph_replay_on_another_stream():
    q, k, v, pos, inv, slots, cache = make(64, 8, 2, 192, 192)
    eager_cache = cache.clone()
    side = torch.cuda.Stream()
    out = torch.zeros_like(q)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, cache, out)
    pos += 12345
    g.replay()
    torch.cuda.synchronize()
    want = sda.sparse_decode_rope_append(q, k, v, pos, inv, slots, eager_cache, stream=torch.cuda.current_stream())
    assert torch.equal(out, want) and torch.equal(cache, eager_cache)


def test_turning_back_returns_the_input():
    """Negative positions turn backwards: within two bf16 roundings of the start."""
    q, *_rest = make(9, 4, 1, 128, 128)
    pos, inv = _rest[2], _rest[3]
    there = sda.sparse_decode_rope_append(q, None, None, pos, inv, None, None)
    back = sda.sparse_decode_rope_append(there, None, None, -pos, inv, None, None)
    length = math.sqrt(2) * q.float().abs().amax(-1, keepdim=True)
    assert ((back.float() - q.float()).abs() <= 3 * 2.0 ** -8 * length).all()

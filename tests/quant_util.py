"""Plain forms of the quantised cache's operators: written from the formulas, on the CPU, a block after
another.  Where the contract fixes an fp32 rounding it is made here too, so that elements and scales
have to be equal."""
from __future__ import annotations

import numpy as np
import torch

SMALLEST = np.float32(2.0 ** -126)


def round_e4m3(v):
    """Float64 values to the nearest E4M3 value, ties to even, saturated at 448."""
    v = np.asarray(v, np.float64)
    e = np.frexp(np.where(np.isfinite(v), v, 0.0))[1] - 1
    step = 2.0 ** (np.maximum(e, -6) - 3)
    with np.errstate(invalid="ignore"):
        return np.clip(np.rint(v / step) * step, -448.0, 448.0)


def round_int8(v):
    v = np.asarray(v, np.float64)
    return np.clip(np.rint(np.where(np.isnan(v), 0.0, v)), -127.0, 127.0)


def values(cache, int8):
    """The cache's elements as float64 values."""
    return (cache.view(torch.int8) if int8 else cache.view(torch.float8_e4m3fn).float()).double().numpy()


def least_scale(amax, int8):
    if int8:
        return max(np.float32(amax) / np.float32(127), SMALLEST)
    s = 2.0 ** -126
    while 448.0 * s < float(amax):
        s *= 2.0
    return np.float32(s)


def append(key, value, slots, elements, scales, int8):
    """The contract of sparse_decode_quantised_append on float64 `elements` [pages, G, B, 2D] and fp32
    `scales` [pages, G, B / S, 2], both changed in place.  Returns the flags."""
    pages, G, B, _ = elements.shape
    S, D = B // scales.shape[2], key.shape[2]
    rounded = round_int8 if int8 else round_e4m3
    flags = 0
    runs, before, out_of_order = [], -1, False
    for r, slot in enumerate(slots):
        slot = int(slot)
        if not 0 <= slot < pages * B:
            flags |= 0 if slot == -1 else 1
            before = -1
            continue
        if before < 0 or before // S != slot // S:
            runs.append([(r, slot)])
            out_of_order = False
        elif slot == before + 1 and not out_of_order:
            runs[-1].append((r, slot))
        else:
            flags |= 1
            out_of_order = True
        before = slot
    for run in runs:
        page, off = divmod(run[0][1], B)
        part, place = divmod(off, S)
        for g in range(G):
            for kv, x in ((0, key), (1, value)):
                x = x[[r for r, _ in run], g].float().numpy()
                finite = np.isfinite(x)
                flags |= 0 if finite.all() else 8
                need = least_scale(np.abs(np.where(finite, x, 0)).max(), int8)
                had = scales[page, g, part, kv]
                scale = need if place == 0 else max(had, need)
                at = slice(kv * D, (kv + 1) * D)
                if place and scale > had:
                    old = elements[page, g, off - place:off, at]
                    elements[page, g, off - place:off, at] = rounded(old.astype(np.float32) * (had / scale))
                scales[page, g, part, kv] = scale
                with np.errstate(invalid="ignore"):
                    elements[page, g, off:off + len(run), at] = rounded(x / scale)
    return flags


def read(elements, scales, table, starts, first, rows):
    """[rows, G, 2D] bf16, NaN where nothing is written, and the flags."""
    pages, G, B, D2 = elements.shape
    S = B // scales.shape[2]
    out = torch.full((rows, G, D2), float("nan"), dtype=torch.bfloat16)
    flags = 0
    for q in range(len(starts) - 1):
        for r in range(max(0, starts[q]), min(rows, starts[q + 1])):
            t = r - starts[q] + (first[q] if first is not None else 0)
            page = int(table[q][t // B]) if 0 <= t and t // B < len(table[q]) else -1
            if not 0 <= page < pages:
                flags |= 1
                continue
            s = np.repeat(scales[page, :, t % B // S], D2 // 2, -1)
            out[r] = torch.from_numpy(elements[page, :, t % B].astype(np.float32) * s).bfloat16()
    return out, flags


def attend(x, k, v, scale):
    """Float64 attention of query rows x [H, D] over tokens: (output, lse, spread, slack) as step_util.paged_attention
    gives them.  k and v are decoded: 2^-22 more for the key scale's two roundings."""
    H, D = x.shape
    if not len(k):
        return torch.zeros(H, D, dtype=torch.float64), torch.full((H,), -np.inf, dtype=torch.float64), \
            torch.zeros(H, D, dtype=torch.float64), torch.zeros(H, dtype=torch.float64)
    s = x @ k.T * scale
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - lse[:, None])
    slack = (x.abs() @ k.abs().T * abs(scale)).amax(-1) * (D / 16 + 5) * 2.0 ** -22
    return w @ v, lse, w @ v.abs(), slack


def attention_bound(o, spread, slack, most, tokens, gated=False):
    """|kernel - exact| <= one bf16 rounding of the output (half a step: 2^-8), the weights' rounding to fp16
    (2^-11; twice, for the scale's product in fp32 and the exponential: 2^-20), the logits' error in numerator and
    sum; `most`: what an element of the largest value scale can stand for, whose weights below 2^-27 of the largest are
    off by 2^-38 of it; with a gate one bf16 step more where the two sigmoids round apart."""
    weights = 2.0 ** -11 + 2.0 ** -19 + 2 * slack[..., None]
    return o.abs() * (2.0 ** -8 + (2.0 ** -7 if gated else 0.0)) * 1.01 + spread * weights + most * tokens * 2.0 ** -38 + 1e-37

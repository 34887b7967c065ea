"""Plain 64-bit forms of the serving-step operators (page tables, rotary positions with the
cache write, attention over the whole paged cache), and the error bounds the GPU tests use.

They are written from the formulas, on the CPU, with loops where the kernels have none."""
from __future__ import annotations

import numpy as np
import torch

E4M3_MAX = 448.0


def plan(context, new, block, ring, state, table, rows, per_request=0):
    """The contract of sparse_decode_plan_step, one request after another.  Returns (seq_lens,
    token_starts, slots, positions, requests, free_next, ring, table, flags)."""
    context, new, ring = [int(x) for x in context], [int(x) for x in new], [int(x) for x in ring]
    table = np.array(table, dtype=np.int64).copy()
    F, W = len(ring), table.shape[1]
    start, count = (int(x) for x in state)
    flags = 0
    usable = 0 <= start < F and 0 <= count <= F
    if not usable:
        flags |= 1
        start = count = 0
    asked = back = taken = returned = 0
    out_of_rows = False
    lens, slots, positions, owners, starts = [], [], [], [], []
    wanted_rows = 0
    ring_out = list(ring)
    for q, (c, n) in enumerate(zip(context, new)):
        starts.append(len(slots))
        lens.append(c)
        have = -(-max(c, 0) // block)
        if n == 0 and c >= 0:
            continue
        if c < 0 or n < -1 or have > W:
            flags |= 1
            continue
        if n == -1:
            back += have
            if usable and count + back <= F:
                for i in range(have):
                    ring_out[(start + count + returned + i) % F] = int(table[q, i])
                returned += have
                lens[q] = 0
            else:
                flags |= 1
            continue
        need = -(-(c + n) // block) - have
        if have + need > W or c + n > 2 ** 31 - 1 or 0 < per_request < n:
            flags |= 1
            continue
        asked += need
        if need and asked > count:
            flags |= 4
            continue
        wanted_rows += n
        if wanted_rows > rows:
            flags |= 4
            continue
        for i in range(need):
            table[q, have + i] = ring[(start + taken + i) % F]
        taken += need
        for pos in range(c, c + n):
            page = int(table[q, pos // block])
            if page < 0:
                flags |= 1
            slots.append(page * block + pos % block if page >= 0 else -1)
            positions.append(pos)
            owners.append(q)
        lens[q] = c + n
    starts.append(len(slots))
    if per_request:                       # spread out: a request's tokens are the last of its rows
        flat = list(zip(slots, positions, owners))
        starts = [(q + 1) * per_request - owners.count(q) for q in range(len(context))] + [rows]
        out = [(-1, -1, -1)] * rows
        for q in range(len(context)):
            mine = [x for x in flat if x[2] == q]
            out[starts[q]:(q + 1) * per_request] = mine
        slots, positions, owners = (list(x) for x in zip(*out)) if rows else ([], [], [])
    free_next = [(start + taken) % F, count - taken + returned] if usable else [int(x) for x in state]
    pad = [-1] * (rows - len(slots))
    return dict(seq_lens=lens, token_starts=starts, slots=slots + pad, positions=positions + pad,
                requests=owners + pad, free_next=free_next, free_pages=ring_out, table=table), flags


def pair_axes(half, sections, interleaved):
    if not interleaved:
        return [a for a, n in enumerate(sections) for _ in range(n)]
    A = len(sections)
    return [i % A if i % A > 0 and i // A < sections[i % A] else 0 for i in range(half)]


def rotate(x, positions, inv_freq, sections, interleaved=False, adjacent=False, amplitude=1.0):
    """[T, heads, D] turned in float64; also the sum |a| + |b| behind each output (its rounding scale)."""
    y = x.double().clone()
    size = y.abs()
    if positions is None:
        return y, size
    half = inv_freq.numel()
    for i, a in enumerate(pair_axes(half, sections or [half], interleaved)):
        lo, hi = (2 * i, 2 * i + 1) if adjacent else (i, i + half)
        t = positions[a].double() * inv_freq[i].double()
        c, s = torch.cos(t)[:, None] * amplitude, torch.sin(t)[:, None] * amplitude
        u, v = x[..., lo].double(), x[..., hi].double()
        y[..., lo], y[..., hi] = u * c - v * s, v * c + u * s
        size[..., lo] = size[..., hi] = (u.abs() + v.abs()) * abs(amplitude)
    return y, size


def e4m3_values(x):
    return x.view(torch.float8_e4m3fn).float().double()


def paged_attention(query, cache, table, lens, *, scale, query_len=1, k_scale=1.0, v_scale=1.0, gate=None):
    """Float64 attention of each request's newest tokens over its cache.  Returns (output, lse,
    spread, slack): `spread` is the attention over |v| (what an error of the weights multiplies)
    and `slack` bounds the relative error that fp32 logits give the weights."""
    rows, H, D = query.shape
    G, B = cache.shape[1], cache.shape[2]
    kv_all = e4m3_values(cache) if cache.dtype == torch.uint8 else cache.double()
    o = torch.zeros(rows, H, D, dtype=torch.float64)
    lse = torch.full((rows, H), -np.inf, dtype=torch.float64)
    spread, slack = torch.zeros_like(o), torch.zeros(rows, H, dtype=torch.float64)
    for q, n in enumerate(int(x) for x in lens):
        if n <= 0:
            continue
        n_pages = -(-n // B)
        pages = table[q, :n_pages].long()
        for g in range(G):
            kv = kv_all[pages, g].reshape(n_pages * B, 2 * D)[:n]
            k, v = kv[:, :D] * k_scale, kv[:, D:] * v_scale
            for j in range(query_len):
                seen = n - query_len + 1 + j
                if seen <= 0:
                    continue
                r = (q * query_len + j) * G + g
                x = query[r].double()
                s = x @ k[:seen].T * scale
                lse[r] = torch.logsumexp(s, -1)
                w = torch.exp(s - lse[r][:, None])
                o[r], spread[r] = w @ v[:seen], w @ v[:seen].abs()
                # each of D / 16 accumulations, the scaling and the exponent round to 2^-22
                slack[r] = (x.abs() @ k[:seen].abs().T * abs(scale)).amax(-1) * (D / 16 + 4) * 2.0 ** -22
    if gate is not None:
        f = (1.0 / (1.0 + torch.exp(-gate.float()))).bfloat16().double().view(-1, G, H).reshape(rows, H, 1)
        o, spread = o * f, spread * f
    return o, lse, spread, slack


def attention_bound(o, spread, slack, fp8, gated=False):
    """|kernel - exact| <= one bf16 rounding of the output (half a step: 2^-8), the weights' rounding
    (fp16 next to an E4M3 cache: 2^-11; bf16 twice: 2^-16), the logits' error in numerator and sum,
    2^-20 for the exponentials and sums; with a gate one bf16 step more where the two sigmoids round
    apart."""
    weights = (2.0 ** -11 if fp8 else 2.0 ** -16) + 2.0 ** -20 + 2 * slack[..., None]
    return o.abs() * (2.0 ** -8 + (2.0 ** -7 if gated else 0.0)) * 1.01 + spread * weights + 1e-30

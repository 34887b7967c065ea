"""The serving step around the paged cache: its operators, the cases they are timed on, and their plain forms.

  plan       block tables, slot maps and positions of a step, from request lengths (sparse_decode_plan_step)
  append     rotary positions with one to three axes, keys and values written to their slots (sparse_decode_rope_append)
  attention  attention over each request's whole paged cache (sparse_decode_paged_attention)

A case is a dict of sizes; lengths come from its numbers alone, contents from the seed.
"""
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX = 448.0
FP8_SCALE = 8.0 / 448.0     # K and V of unit variance in E4M3


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _attention(name, requests, low, high, *, empty=0, query_len=1, groups=1, heads=16, dim=192, block=64, fp8=False,
               gate=False, spread=1):
    c = dict(op="attention", requests=requests, low=low, high=high, empty=empty, query_len=query_len, groups=groups,
             heads=heads, dim=dim, block=block, fp8=fp8, gate=gate, spread=spread)
    return dict(c, name=name) if name else c


def _append(name, tokens, *, padding=0, groups=1, heads=16, dim=192, rotary=192, axes=1, interleaved=False,
            adjacent=False, block=64, fp8=False, spread=1):
    c = dict(op="append", tokens=tokens, padding=padding, groups=groups, heads=heads, dim=dim, rotary=rotary, axes=axes,
             interleaved=interleaved, adjacent=adjacent, block=block, fp8=fp8, spread=spread)
    return dict(c, name=name) if name else c


def _plan(name, requests, *, context, new_low, new_high, released=0, idle=0, block=64, room=1.0, spread=1):
    c = dict(op="plan", requests=requests, context=context, new_low=new_low, new_high=new_high, released=released,
             idle=idle, block=block, room=room, spread=spread)
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user, a first short answer: nothing but latency
        _attention("attention: one short request", 1, 40, 40, heads=8, block=16),
        # a batch of chats in a bf16 cache, 8K to 32K tokens each
        _attention("attention: batch of chats", 64, 8192, 32768, groups=2),
        # one request with a very long document in an FP8 cache: all of the GPU on few rows
        _attention("attention: one long document", 1, 261001, 261001, groups=4, fp8=True),
        # many short requests of odd lengths, some slots of the batch empty, smaller heads and pages
        _attention("attention: ragged short requests", 197, 1, 2500, empty=9, groups=4, heads=8, dim=128, block=16, fp8=True),
        # speculative decoding: two tokens a request are verified, gated layers
        _attention("attention: two draft tokens", 12, 65536, 131072, query_len=2, groups=4, gate=True),
        # long documents served together from an FP8 cache
        _attention("attention: batch of documents", 16, 131072, 262144, groups=4, fp8=True),
        # a decode step of one user
        _append("append: one token", 1, groups=1, heads=8, block=16),
        # a decode step of a full batch, FP8 cache, the captured batch larger than the live one
        _append("append: decode batch", 256, padding=19, groups=4, fp8=True),
        # video and image tokens of a prompt (time, height, width), an odd number of them
        _append("append: video prompt", 16363, groups=4, rotary=128, axes=3, fp8=True),
        # a decode step: each request gets its next token, some cross into a new page
        _plan("plan: decode batch", 256, context=32768, new_low=1, new_high=1, released=3, idle=5),
        # steps of mixed prompts and answers with small pages
        _plan("plan: prompts and answers", 1021, context=4096, new_low=1, new_high=900, released=37, idle=50, block=16),
        # a node starts: every prompt of a large batch is placed
        _plan("plan: all prompts", 4096, context=0, new_low=1, new_high=2048, block=32),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    spread = rng.randrange(1, 1 << 30)
    op = rng.choice(("attention", "append", "plan"))
    block = rng.choice((8, 16, 24, 32, 48, 64, 128))
    groups = rng.choice((1, 2, 3, 4, 8))
    dim = rng.choice((64, 128, 192, 192, 256))
    fp8 = rng.random() < 0.5
    if op == "attention":
        query_len = rng.choice((1, 1, 1, 2, 3, 4))
        heads = rng.randint(1, 16)
        requests = _log_uniform(rng, 1, 256)
        row = 2 * dim * (1 if fp8 else 2) * groups
        # K|V of at most 1.2 GB, so that no drawn case is more than the largest listed one
        high = _log_uniform(rng, 1, max(2, min(262144, int(1.2e9) // (row * requests))))
        low = max(1, int(high * rng.choice((0.05, 0.5, 1.0))))
        return _attention(None, requests, low, high, empty=rng.choice((0, 0, requests // 10)), query_len=query_len,
                          groups=groups, heads=heads, dim=dim, block=block, fp8=fp8, gate=rng.random() < 0.4, spread=spread)
    if op == "append":
        tokens = _log_uniform(rng, 1, 16000 * 4 // groups if groups > 4 else 16000)
        axes = rng.choice((1, 1, 2, 3))
        rotary = rng.choice([r for r in (32, 64, 96, 128, 192, 256) if r <= dim])
        return _append(None, tokens, padding=rng.choice((0, 0, tokens // 7)), groups=groups, heads=rng.randint(1, 12),
                       dim=dim, rotary=rotary, axes=axes, interleaved=axes > 1 and rng.random() < 0.5,
                       adjacent=rng.random() < 0.4, block=block, fp8=fp8, spread=spread)
    requests = _log_uniform(rng, 1, 4000)
    new_high = _log_uniform(rng, 1, max(1, min(2000, 3_000_000 // requests)))
    return _plan(None, requests, context=_log_uniform(rng, 1, 40000), new_low=rng.choice((0, 1, new_high)), new_high=new_high,
                 released=rng.choice((0, requests // 9)), idle=rng.choice((0, requests // 11)), block=block,
                 room=rng.choice((1.0, 1.0, 0.7)), spread=spread)


def _lengths(case):
    r = random.Random(case["spread"])
    lens = [r.randint(case["low"], case["high"]) for _ in range(case["requests"])]
    for q in r.sample(range(case["requests"]), case["empty"]):
        lens[q] = 0
    return lens


def _plan_lengths(case):
    """Context and new lengths of each request; new is -1 for a finished request whose pages go back."""
    r = random.Random(case["spread"])
    n = case["requests"]
    context = [r.randint(0, case["context"]) for _ in range(n)]
    new = [r.randint(case["new_low"], case["new_high"]) for _ in range(n)]
    for k, q in enumerate(r.sample(range(n), case["released"] + case["idle"])):
        new[q] = -1 if k < case["released"] else 0
    return context, new


def _ceil(a, b):
    return -(-a // b)


def _plan_sizes(case):
    """(pages held, pages wanted, pages released, new tokens) over all requests."""
    context, new = _plan_lengths(case)
    b = case["block"]
    held = sum(_ceil(c, b) for c in context)
    wanted = sum(_ceil(c + n, b) - _ceil(c, b) for c, n in zip(context, new) if n > 0)
    back = sum(_ceil(c, b) for c, n in zip(context, new) if n < 0)
    return held, wanted, back, sum(max(n, 0) for n in new)


def _sections(case):
    """Frequency pairs of each axis: time gets a quarter, the others share the rest (one axis: all)."""
    half, axes = case["rotary"] // 2, case["axes"]
    rest = (half - half // 4) // (axes - 1) if axes > 1 else 0
    if case["interleaved"]:
        rest = half // axes
    return [half - rest * (axes - 1)] + [rest] * (axes - 1)


def work(case):
    if case["op"] == "attention":
        lens = _lengths(case)
        elt = 1 if case["fp8"] else 2
        g, h, d, ql = (case[k] for k in ("groups", "heads", "dim", "query_len"))
        tokens = sum(lens)
        rows = case["requests"] * ql * g
        pages = sum(_ceil(x, case["block"]) for x in lens)
        nbytes = tokens * g * 2 * d * elt + rows * h * (4 * d + 4 + (2 if case["gate"] else 0)) + 4 * (pages + len(lens))
        return {"bytes": nbytes, "flops": 4 * d * h * g * sum(max(0, x - ql + 1 + j) for x in lens for j in range(ql))}
    if case["op"] == "append":
        t, g, d = case["tokens"] - case["padding"], case["groups"], case["dim"]
        elt = 1 if case["fp8"] else 2
        nbytes = t * (4 * g * case["heads"] * d + 4 * g * d + 2 * g * d * elt + 4 * case["axes"]) + 8 * case["tokens"]
        return {"bytes": nbytes, "flops": 3 * t * g * (case["heads"] + 1) * case["rotary"]}
    held, wanted, back, tokens = _plan_sizes(case)
    return {"bytes": 16 * case["requests"] + 8 * (wanted + back) + 16 * tokens, "flops": 0}


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _normal(shape, gen, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _cache(pages, groups, block, dim, fp8, gen):
    """A cache whose every page holds K|V of unit variance (bf16, or E4M3 bytes in units of FP8_SCALE)."""
    cache = torch.empty((pages, groups, block, 2 * dim), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda")
    flat = cache.view(-1)
    piece = 1 << 27
    for a in range(0, flat.numel(), piece):
        part = flat[a:a + piece]
        x = _normal((part.numel(),), gen)
        part.copy_((x / FP8_SCALE).clamp_(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8) if fp8 else x)
    return cache


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    state = {"case": case}
    if case["op"] == "attention":
        _prepare_attention(case, gen, state)
    elif case["op"] == "append":
        _prepare_append(case, gen, state)
    else:
        _prepare_plan(case, gen, state)
    return state


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _scales(case, state):
    s = torch.full((1,), FP8_SCALE, dtype=torch.float32, device="cuda") if case["fp8"] else None
    state["k_scale"], state["v_scale"] = s, s


def _prepare_attention(case, gen, s):
    lens = _lengths(case)
    b, g, h, d = (case[k] for k in ("block", "groups", "heads", "dim"))
    need = torch.tensor([_ceil(x, b) for x in lens], device="cuda")
    pages = max(1, int(need.sum()))
    width = max(1, int(need.max()))
    column = torch.arange(width, device="cuda")
    used = column[None] < need[:, None]
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[used] = torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[:int(need.sum())]
    rows = case["requests"] * case["query_len"] * g
    s.update(table=table, lens=_int32(lens), scale=d ** -0.5, longest=max(1, max(lens)),
             cache=_cache(pages, g, b, d, case["fp8"], gen), query=_normal((rows, h, d), gen, 2.0),
             gate=_normal((rows // g, g * h), gen, 2.0) if case["gate"] else None,
             output=torch.zeros((rows, h, d), dtype=torch.bfloat16, device="cuda"),
             lse=torch.zeros((rows, h), dtype=torch.float32, device="cuda"))
    _scales(case, s)


def _prepare_append(case, gen, s):
    r = random.Random(case["spread"])
    t, live = case["tokens"], case["tokens"] - case["padding"]
    g, d, b = case["groups"], case["dim"], case["block"]
    width = g * (case["heads"] + 2) * d
    qkv = _normal((t, width), gen)                           # one projection's output: q, k and v are views of it
    hq = g * case["heads"]
    q, k, v = (x.view(t, -1, d) for x in qkv.split([hq * d, g * d, g * d], dim=1))
    pages = _ceil(live, b) + 3
    slots = torch.full((t,), -1, dtype=torch.int64, device="cuda")
    page = torch.randperm(pages, generator=gen, device="cuda")
    at = torch.arange(live, device="cuda")
    slots[:live] = page[at // b] * b + at % b
    # the tokens of a prompt after an earlier part: a time axis, and the rows and columns of frames of 14 x 18
    first = r.randrange(200000)
    place = torch.arange(t, device="cuda")
    if case["axes"] == 1:
        positions = (first + place)[None]
    else:
        frame = first + place // 252
        positions = torch.stack([frame, first + place % 252 // 18, first + place % 18][:case["axes"]])
    half = case["rotary"] // 2
    inv_freq = (10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)).float()
    s.update(query=q, key=k, value=v, slots=slots, positions=positions.to(torch.int32).contiguous(), inv_freq=inv_freq,
             sections=_sections(case), cache=_cache(pages, g, b, d, case["fp8"], gen),
             query_out=torch.zeros((t, hq, d), dtype=torch.bfloat16, device="cuda"))
    _scales(case, s)


def _prepare_plan(case, gen, s):
    context, new = _plan_lengths(case)
    b = case["block"]
    held, wanted, back, tokens = _plan_sizes(case)
    free = max(1, int(wanted * case["room"]))
    total = held + free
    ids = torch.randperm(total, generator=gen, device="cuda", dtype=torch.int32)
    need = torch.tensor([_ceil(c, b) for c in context], device="cuda")
    width = max(1, max(_ceil(c + max(n, 0), b) for c, n in zip(context, new)))
    column = torch.arange(width, device="cuda")
    table = torch.full((len(new), width), -1, dtype=torch.int32, device="cuda")
    table[column[None] < need[:, None]] = ids[:held]
    start = total // 3
    ring = torch.full((total,), -1, dtype=torch.int32, device="cuda")
    ring[(start + torch.arange(free, device="cuda")) % total] = ids[held:]
    n, t = len(new), max(1, tokens)
    empty = lambda *shape: torch.zeros(shape, dtype=torch.int32, device="cuda")  # noqa: E731
    s.update(context=_int32(context), new=_int32(new), table=table, free_pages=ring, free_state=_int32([start, free]),
             free_next=empty(2), seq_lens=empty(n), starts=empty(n + 1), positions=empty(t), requests=empty(t),
             slots=torch.zeros((t,), dtype=torch.int64, device="cuda"))


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def run(state):
    return {"attention": _run_attention, "append": _run_append, "plan": _run_plan}[state["case"]["op"]](state)


def _run_attention(s):
    case = s["case"]
    if own:
        import sparse_decode_attention_02_gb300 as sda
        sda.sparse_decode_paged_attention(s["query"], s["cache"], s["table"], s["lens"], s["output"], scale=s["scale"],
                                          query_len=case["query_len"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                                          gate=s["gate"], lse=s["lse"])
        return s["output"], s["lse"]
    b, g, h, d, ql = (case[k] for k in ("block", "groups", "heads", "dim", "query_len"))
    n = case["requests"]
    at = torch.arange(s["longest"], device="cuda")
    page = s["table"].long().clamp(min=0)[:, at // b]                       # [requests, longest]
    kv = s["cache"][page, :, at % b]                                         # [requests, longest, groups, 2 dim]
    kv = (kv.view(FP8) if case["fp8"] else kv).float()
    ks, vs = (s["k_scale"], s["v_scale"]) if case["fp8"] else (1.0, 1.0)
    q = s["query"].float().view(n, ql, g, h, d)
    logits = torch.einsum("qjghd,qngd->qjghn", q, kv[..., :d]) * (s["scale"] * ks)
    last = s["lens"].long()[:, None] - ql + torch.arange(ql, device="cuda")   # position of each query token
    logits.masked_fill_((at > last[..., None])[:, :, None, None], float("-inf"))
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("qjghn,qngd->qjghd", p, kv[..., d:]) * vs
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    if s["gate"] is not None:
        gate = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
        o = o * gate.to(torch.bfloat16).float().view(n, ql, g, h, 1)
    lse = (top + torch.log(total)).view(n * ql * g, h)
    return o.view(n * ql * g, h, d).to(torch.bfloat16), lse


def _axis_of_pair(case, sections, device):
    """The axis that turns each frequency pair: in runs, or (interleaved) in turn while an axis has pairs left."""
    pair = torch.arange(case["rotary"] // 2, device=device)
    sizes = torch.tensor(sections, device=device)
    if not case["interleaved"]:
        return torch.searchsorted(torch.cumsum(sizes, 0), pair, right=True)
    axis = pair % len(sections)
    return torch.where((axis > 0) & (pair // len(sections) < sizes[axis]), axis, torch.zeros_like(axis))


def _run_append(s):
    case = s["case"]
    if own:
        import sparse_decode_attention_02_gb300 as sda
        sda.sparse_decode_rope_append(s["query"], s["key"], s["value"], s["positions"], s["inv_freq"], s["slots"],
                                      s["cache"], s["query_out"], sections=s["sections"],
                                      interleaved_axes=case["interleaved"], adjacent_pairs=case["adjacent"],
                                      k_scale=s["k_scale"], v_scale=s["v_scale"])
    else:
        b, g, d, rot = (case[k] for k in ("block", "groups", "dim", "rotary"))
        axis = _axis_of_pair(case, s["sections"], "cuda")
        angle = s["positions"].double()[axis].T * s["inv_freq"].double()     # far positions need 64 bits
        cos, sin = torch.cos(angle).float()[:, None], torch.sin(angle).float()[:, None]

        def turn(x):
            x = x.float()
            r = x[..., :rot]
            a, c = (r[..., 0::2], r[..., 1::2]) if case["adjacent"] else (r[..., :rot // 2], r[..., rot // 2:])
            y = a * cos - c * sin, c * cos + a * sin
            y = torch.stack(y, -1).flatten(-2) if case["adjacent"] else torch.cat(y, -1)
            return torch.cat([y, x[..., rot:]], -1)

        live = s["slots"] >= 0
        s["query_out"][live] = turn(s["query"])[live].to(torch.bfloat16)
        k, v = turn(s["key"])[live], s["value"].float()[live]
        if case["fp8"]:
            k, v = ((x / sc).clamp(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8)
                    for x, sc in ((k, s["k_scale"]), (v, s["v_scale"])))
        at = s["slots"][live]
        s["cache"][at // b, :, at % b] = torch.cat([k, v], -1).to(s["cache"].dtype)
    return s["query_out"], s["cache"].view(FP8) if case["fp8"] else s["cache"]


def _run_plan(s):
    case = s["case"]
    if own:
        import sparse_decode_attention_02_gb300 as sda
        sda.sparse_decode_plan_step(s["context"], s["new"], s["free_pages"], s["free_state"], s["table"],
                                    block_size=case["block"], free_next=s["free_next"], seq_lens=s["seq_lens"],
                                    token_starts=s["starts"], slots=s["slots"], positions=s["positions"],
                                    requests=s["requests"])
    else:
        b = case["block"]
        n, width = s["table"].shape
        ring, rows = s["free_pages"].numel(), s["slots"].numel()
        c, new = s["context"].long(), s["new"].long()
        start, count = s["free_state"].long()
        have = (c + b - 1) // b
        end = (c + new.clamp(min=0) + b - 1) // b
        # pages first, then token rows, in the order of the requests; a request that does not fit waits
        need = torch.where((new > 0) & (end <= width), end - have, 0)
        pages = torch.cumsum(need, 0)
        takes = (new > 0) & (end <= width) & ((need == 0) | (pages <= count))
        tokens = torch.cumsum(torch.where(takes, new, 0), 0)
        takes = takes & (tokens <= rows)
        taken = torch.where(takes, need, 0)
        added = torch.where(takes, new, 0)
        first = pages - need
        back = torch.where((new < 0) & (have <= width), have, 0)
        returned = torch.cumsum(back, 0)
        back = torch.where(count + returned <= ring, back, 0)    # a full ring keeps a request's pages with it
        gone = (new < 0) & (have <= width) & (count + returned <= ring)
        # columns of new pages, and pages that go back to the ring
        column = torch.arange(width, device="cuda")[None]
        fresh = (column >= have[:, None]) & (column < (have + taken)[:, None])
        from_ring = s["free_pages"][(start + first[:, None] + column - have[:, None]) % ring]
        table = torch.where(fresh, from_ring, s["table"])
        leaves = column < back[:, None]
        to_ring = (start + count + (returned - torch.where(gone, have, 0))[:, None] + column) % ring
        s["free_pages"][to_ring[leaves]] = s["table"][leaves]
        s["table"].copy_(table)
        s["free_next"].copy_(torch.stack([(start + taken.sum()) % ring, count - taken.sum() + back.sum()]))
        s["seq_lens"].copy_(torch.where(gone, 0, c + added))
        total = torch.cumsum(added, 0)
        s["starts"].copy_(torch.cat([torch.zeros_like(total[:1]), total]))
        row = torch.arange(rows, device="cuda")
        q = torch.searchsorted(total, row, right=True)
        live = q < n
        q = q.clamp(max=n - 1)
        pos = c[q] + row - (total - added)[q]
        slot = table[q, (pos // b).clamp(0, width - 1)].long() * b + pos % b
        for out, x in ((s["slots"], slot), (s["positions"], pos), (s["requests"], q)):
            out.copy_(torch.where(live, x, -1))
    return {k: s[k] for k in ("table", "free_pages", "free_next", "seq_lens", "starts", "slots", "positions", "requests")}


# ---------------------------------------------------------------------------------------------------------------------
# in 64 bits, from the definitions


def exact(case, seed):
    if case["op"] == "plan":
        return None                     # whole numbers: nothing is rounded
    s = prepare(case, seed)
    return _exact_attention(s) if case["op"] == "attention" else _exact_append(s)


def _exact_attention(s):
    case = s["case"]
    b, g, h, d, ql = (case[k] for k in ("block", "groups", "heads", "dim", "query_len"))
    out = torch.zeros((case["requests"], ql, g, h, d), dtype=torch.float64, device="cuda")
    lse = torch.full((case["requests"], ql, g, h), float("-inf"), dtype=torch.float64, device="cuda")
    query = s["query"].double().view(case["requests"], ql, g, h, d)
    unit = float(s["k_scale"]) if case["fp8"] else 1.0
    for r, n in enumerate(_lengths(case)):
        if not n:
            continue
        rows = s["cache"][s["table"][r, :_ceil(n, b)].long()]
        for k in range(g):
            kv = rows[:, k].reshape(-1, 2 * d)[:n]
            kv = (kv.view(FP8).float() if case["fp8"] else kv).double() * unit
            for j in range(ql):
                seen = n - ql + 1 + j
                if seen > 0:
                    z = query[r, j, k] @ kv[:seen, :d].T * s["scale"]
                    out[r, j, k] = torch.softmax(z, -1) @ kv[:seen, d:]
                    lse[r, j, k] = torch.logsumexp(z, -1)
    if case["gate"]:                    # the gate factor is rounded to bf16 by definition
        out *= torch.sigmoid(s["gate"].float()).to(torch.bfloat16).double().view(case["requests"], ql, g, h, 1)
    return out.view(s["output"].shape), lse.view(s["lse"].shape)


def _exact_append(s):
    case = s["case"]
    rot, b, d = case["rotary"], case["block"], case["dim"]
    cache = (s["cache"].view(FP8).float() if case["fp8"] else s["cache"]).double()
    out = torch.zeros(s["query_out"].shape, dtype=torch.float64, device="cuda")
    sections, axes = s["sections"], case["axes"]
    if case["interleaved"]:
        owner = [i % axes if i % axes and i // axes < sections[i % axes] else 0 for i in range(rot // 2)]
    else:
        owner = [a for a in range(axes) for _ in range(sections[a])]
    live = case["tokens"] - case["padding"]
    phase = torch.stack([s["positions"][a, :live].double() * float(s["inv_freq"][i]) for i, a in enumerate(owner)], 1)
    wave = torch.polar(torch.ones_like(phase), phase)[:, None]
    lo = [2 * i for i in range(rot // 2)] if case["adjacent"] else list(range(rot // 2))
    hi = [i + 1 for i in lo] if case["adjacent"] else [i + rot // 2 for i in lo]

    def turned(x):
        y = x[:live].double()
        z = torch.complex(y[..., lo], y[..., hi]) * wave
        y[..., lo], y[..., hi] = z.real, z.imag
        return y

    out[:live] = turned(s["query"])
    new = torch.cat([turned(s["key"]), s["value"][:live].double()], -1)
    if case["fp8"]:
        new = (new / float(s["k_scale"])).clamp(-FP8_MAX, FP8_MAX)
    at = s["slots"][:live]
    cache[at // b, :, at % b] = new
    return out, cache

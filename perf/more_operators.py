"""A paged cache of 8-bit elements with a scale for each block of tokens and head: its operators, the cases they are timed on, and their plain forms.

  append     keys and values quantised into their slots, the scales following them (sparse_decode_quantised_append)
  read       contexts read back in bf16, request after request (sparse_decode_quantised_read)
  chunk      a prompt's next chunk: written, then its whole context read back (both)
  attention  attention over each request's whole cache (sparse_decode_quantised_paged_attention)
  regions    attention over the selected regions of each row (sparse_decode_quantised_attention)

The cache is [pages, groups, block, 2 dim], keys then values, in E4M3 or 8-bit integers; its scales are [pages, groups,
block / span, 2], of the keys and of the values of `span` tokens.  A case is a dict of sizes; lengths come from its numbers
alone, contents from the seed.
"""
import random

import torch

own = False

FP8 = torch.float8_e4m3fn
FP8_MAX, INT8_MAX = 448.0, 127.0
SMALLEST = 2.0 ** -126      # of a scale


# ---------------------------------------------------------------------------------------------------------------------
# cases


def _case(name, op, **sizes):
    c = dict(op=op, **(dict(requests=1, low=1, high=1, new=0, empty=0, first=0, query_len=1, groups=1, heads=16, dim=192, block=64,
                            span=64, int8=False, gate=False, selected=0, region=8, spread=1) | sizes))
    return dict(c, name=name) if name else c


def listed():
    return [
        # a decode step of one user: nothing but latency
        _case("append: one token", "append", low=40, high=40, new=1, block=16, span=16),
        # a decode step of a full batch; some requests of it are idle, and a few blocks' scales grow
        _case("append: decode batch", "append", requests=256, low=700, high=4000, new=1, empty=19, groups=4, span=32),
        # one long prompt, an odd number of tokens behind an earlier part
        _case("append: prompt", "append", low=1001, high=1001, new=16363, groups=4),
        # chunked prompts: each chunk of 2048 is written, then the context so far is read back for its attention
        _case("chunk: next of a prompt", "chunk", low=14001, high=14001, new=2048, groups=2, dim=128, block=32, span=16, int8=True),
        # contexts of a batch read back for prompts' attention, their shared beginnings left out
        _case("read: several contexts", "read", requests=12, low=2000, high=8000, first=500, groups=2, dim=128, block=32, span=16,
              int8=True),
        # one very long context read back
        _case("read: long context", "read", low=131003, high=131003, groups=4),
        # one user, a first short answer: nothing but latency
        _case("attention: one short request", "attention", low=40, high=40, heads=8, block=16, span=16),
        # many short requests of odd lengths, some slots of the batch empty, smaller heads and pages
        _case("attention: ragged short", "attention", requests=197, low=1, high=2500, empty=9, groups=4, heads=8, dim=128, block=16,
              span=16, int8=True),
        # speculative decoding: two tokens a request are verified, gated layers
        _case("attention: two draft tokens", "attention", requests=12, low=16384, high=65536, query_len=2, groups=4, span=32, int8=True,
              gate=True),
        # long documents served together
        _case("attention: batch of documents", "attention", requests=16, low=65536, high=131072, groups=4),
        # a few users of sparse layers, regions of whole pages
        _case("regions: few users", "regions", requests=3, low=2000, high=5000, groups=2, span=16, int8=True, selected=32, region=64),
        # a decode batch of sparse layers: 1024 regions of 8 tokens for each row
        _case("regions: decode batch", "regions", requests=256, low=16384, high=32768, groups=2, selected=1024),
    ]


def _log_uniform(rng, low, high):
    return min(high, max(low, round(low * (high / low) ** rng.random())))


def draw(rng):
    spread = rng.randrange(1, 1 << 30)
    op = rng.choice(("append", "read", "chunk", "attention", "attention", "regions", "regions"))
    block = rng.choice((8, 16, 24, 32, 48, 64, 128))
    span = rng.choice([s for s in range(8, block + 1, 8) if block % s == 0])
    groups = rng.choice((1, 2, 3, 4, 8))
    dim = rng.choice((64, 128, 192, 192, 256))
    same = dict(block=block, span=span, groups=groups, dim=dim, int8=rng.random() < 0.5, spread=spread)
    row = 2 * dim * groups
    if op in ("append", "chunk"):
        requests = _log_uniform(rng, 1, 400) if op == "append" else _log_uniform(rng, 1, 8)
        new = _log_uniform(rng, 1, max(1, min(8000, int(2.5e7) // (row * requests))))
        high = _log_uniform(rng, 1, max(2, int(1e8) // (row * requests)))
        # E4M3: the cache itself is what a pass returns; integers are read back
        return _case(None, op, requests=requests, low=max(1, high // 3), high=high, new=new, empty=rng.choice((0, requests // 7)),
                     **(same | dict(int8=same["int8"] and op == "chunk")))
    if op == "read":
        requests = _log_uniform(rng, 1, 60)
        high = _log_uniform(rng, 1, max(2, int(2e8) // (row * requests)))
        return _case(None, op, requests=requests, low=max(1, high // 4), high=high, empty=rng.choice((0, requests // 10)),
                     first=rng.choice((0, high // 9)), **same)
    if op == "attention":
        requests = _log_uniform(rng, 1, 256)
        high = _log_uniform(rng, 1, max(2, min(131072, int(1.2e9) // (row * requests))))
        query_len = rng.choice((1, 1, 1, 2, 3, 4))
        return _case(None, op, requests=requests, low=max(1, int(high * rng.choice((0.05, 0.5, 1.0)))), high=high,
                     empty=rng.choice((0, 0, requests // 10)), query_len=query_len, heads=rng.randint(1, 16),
                     gate=rng.random() < 0.25, **same)
    region = rng.choice([r for r in (8, 16, 24, 32, 48, 64, 128) if block % r == 0 or r % block == 0])
    requests, query_len = _log_uniform(rng, 1, 200), rng.choice((1, 1, 2, 3))
    selected = _log_uniform(rng, 1, max(1, min(1024, int(8e8) // (row * region * requests * query_len))))
    high = _log_uniform(rng, max(query_len, region), max(query_len, region) + 40000)
    return _case(None, op, requests=requests, low=max(query_len, high // 2), high=high, empty=rng.choice((0, requests // 10)),
                 query_len=query_len, heads=rng.randint(1, 16), gate=rng.random() < 0.25, selected=selected, region=region, **same)


def _ceil(a, b):
    return -(-a // b)


def _lengths(case):
    """Tokens of each request that are in the cache before the pass; -1: an idle or empty slot of the batch."""
    r = random.Random(case["spread"])
    lens = [r.randint(case["low"], case["high"]) for _ in range(case["requests"])]
    for q in r.sample(range(case["requests"]), case["empty"]):
        lens[q] = -1
    return lens


def _reads(case):
    """(first token, tokens) of each request that a reading pass reads."""
    lens = [n + case["new"] if n >= 0 else 0 for n in _lengths(case)]
    return [(min(case["first"], n), n - min(case["first"], n)) for n in lens]


def work(case):
    g, h, d, s, ql = (case[k] for k in ("groups", "heads", "dim", "span", "query_len"))
    lens = _lengths(case)
    live = [n for n in lens if n >= 0]
    nbytes = flops = 0
    if case["op"] in ("append", "chunk"):
        rows = len(live) * case["new"]
        blocks = sum(_ceil(n + case["new"], s) - n // s for n in live)
        nbytes += rows * g * 2 * d * 3 + 8 * len(lens) * case["new"] + 16 * g * blocks
        flops += 4 * rows * g * d
    if case["op"] in ("read", "chunk"):
        tokens = sum(n for _, n in _reads(case))
        blocks = sum(_ceil(a + n, s) - a // s for a, n in _reads(case) if n)
        nbytes += tokens * g * 2 * d * 3 + 8 * g * blocks + 4 * tokens // case["block"] + 8 * len(lens)
        flops += 2 * tokens * g * d
    rows = len(lens) * ql * g
    if case["op"] == "attention":
        nbytes += sum(live) * g * 2 * d + 8 * g * sum(_ceil(n, s) for n in live) + 4 * sum(_ceil(n, case["block"]) for n in live)
        nbytes += rows * h * (4 * d + 4 + (2 if case["gate"] else 0)) + 4 * len(lens)
        flops += 4 * d * h * g * sum(max(0, n - ql + 1 + j) for n in live for j in range(ql))
    if case["op"] == "regions":
        rt = case["region"]
        tokens = 0
        for n in live:
            for j in range(ql):
                pos = n - ql + j
                regions = min(case["selected"], pos // rt + 1)
                tokens += regions * rt - (rt - 1 - pos % rt)     # the row's own region ends at its position
        nbytes += tokens * g * 2 * d + 8 * tokens * g // s + 4 * rows * case["selected"]
        nbytes += rows * h * (4 * d + (2 if case["gate"] else 0)) + 5 * rows
        flops += 4 * d * h * g * tokens
    return {"bytes": nbytes, "flops": flops}


# ---------------------------------------------------------------------------------------------------------------------
# inputs


def _normal(shape, gen, std=1.0, dtype=torch.bfloat16):
    return torch.empty(shape, dtype=dtype, device="cuda").normal_(0.0, std, generator=gen)


def _int32(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _need(amax, int8):
    """The least scale that holds values of up to `amax`: any for integers, a power of two for E4M3."""
    if int8:
        return (amax / INT8_MAX).clamp(min=SMALLEST)
    m, e = torch.frexp(amax)                                 # amax = m 2^e, m in [0.5, 1): 448 s = 0.875 * 2^9 s
    return torch.ldexp(torch.ones_like(m), e - 9 + (m > 0.875).to(e.dtype)).clamp(min=SMALLEST)


def _elements(x, int8):
    """Quotients as the cache's elements, in its bytes."""
    return (x.round().clamp(-INT8_MAX, INT8_MAX).to(torch.int8).view(torch.uint8) if int8
            else x.clamp(-FP8_MAX, FP8_MAX).to(FP8).view(torch.uint8))


def _values(elements, int8):
    return (elements.view(torch.int8) if int8 else elements.view(FP8)).float()


def _cache(pages, c, gen):
    """A cache whose every block was quantised from values of a magnitude of its own: keys grow from head to head, values less."""
    g, b, d, s = c["groups"], c["block"], c["dim"], c["span"]
    cache = torch.empty((pages, g, b, 2 * d), dtype=torch.uint8, device="cuda")
    scales = torch.empty((pages, g, b // s, 2), device="cuda")
    size = torch.tensor([2.0, 1.0], device="cuda") * 1.5 ** (torch.arange(g, device="cuda") % 4)[:, None]     # [groups, K or V]
    step = max(1, (1 << 26) // (g * b * 2 * d))
    for a in range(0, pages, step):
        n = min(step, pages - a)
        of_block = torch.exp(0.5 * _normal((n, g, b // s, 2), gen, dtype=torch.float32)) * size[None, :, None]
        x = _normal((n, g, b // s, s, 2, d), gen, dtype=torch.float32) * of_block[:, :, :, None, :, None]
        need = _need(x.abs().amax((3, 5)), c["int8"])
        scales[a:a + n] = need
        cache[a:a + n] = _elements(x / need[:, :, :, None, :, None], c["int8"]).view(n, g, b, 2 * d)
    return cache.view(torch.int8) if c["int8"] else cache, scales


def _tables(c, lens, gen, state):
    """Pages in any order for each request's tokens, and a cache of them."""
    b = c["block"]
    need = torch.tensor([_ceil(max(n, 0), b) for n in lens], device="cuda")
    pages = max(1, int(need.sum()))
    width = max(1, int(need.max()))
    table = torch.full((len(lens), width), -1, dtype=torch.int32, device="cuda")
    table[torch.arange(width, device="cuda")[None] < need[:, None]] = \
        torch.randperm(pages, generator=gen, device="cuda", dtype=torch.int32)[:int(need.sum())]
    state["table"] = table
    state["cache"], state["scales"] = _cache(pages, c, gen)


def prepare(case, seed):
    c, gen = case, torch.Generator(device="cuda").manual_seed(seed)
    g, h, d, b, ql = (c[k] for k in ("groups", "heads", "dim", "block", "query_len"))
    lens = _lengths(c)
    s = {"case": c}
    after = [n + c["new"] if n >= 0 else -1 for n in lens]
    _tables(c, after, gen, s)
    if c["op"] in ("append", "chunk"):
        t = len(lens) * c["new"]
        owner = torch.arange(len(lens), device="cuda").repeat_interleave(c["new"])
        pos = _int32(lens).long()[owner] + torch.arange(c["new"], device="cuda").repeat(len(lens))
        page = s["table"].long()[owner, (pos // b).clamp(0, s["table"].shape[1] - 1)]
        s["slots"] = torch.where(_int32(lens)[owner] >= 0, page * b + pos % b, torch.full_like(pos, -1))
        # one projection's output: key and value are views of it; a few tokens are larger than what came before
        qkv = _normal((t, (h + 2) * g * d), gen) * torch.exp(0.5 * _normal((t, 1), gen))
        s["key"], s["value"] = (x.view(t, g, d) for x in qkv.split([g * d, g * d, h * g * d], dim=1)[:2])
    if c["op"] in ("read", "chunk"):
        reads = _reads(c)
        starts = [0]
        for _, n in reads:
            starts.append(starts[-1] + n)
        s["starts"], s["first"] = _int32(starts), _int32([a for a, _ in reads])
        s["key_out"] = torch.zeros((starts[-1], g, d), dtype=torch.bfloat16, device="cuda")
        s["value_out"] = torch.zeros_like(s["key_out"])
    if c["op"] in ("attention", "regions"):
        rows = len(lens) * ql * g
        s.update(lens=_int32(lens).clamp(min=0), scale=d ** -0.5, longest=max(1, max(lens)), query=_normal((rows, h, d), gen),
                 gate=_normal((rows // g, g * h), gen, 2.0) if c["gate"] else None,
                 output=torch.zeros((rows, h, d), dtype=torch.bfloat16, device="cuda"),
                 lse=torch.zeros((rows, h), device="cuda"))
    if c["op"] == "regions":
        _select(c, lens, gen, s)
    return s


def _select(c, lens, gen, s):
    """The row's own region and others of its request, in no order, -1 where there are no more; rows of empty slots are off."""
    ql, g, k, rt = (c[x] for x in ("query_len", "groups", "selected", "region"))
    pos = (_int32(lens).long()[:, None] - ql + torch.arange(ql, device="cuda")).repeat_interleave(g, 1).reshape(-1)
    active = _int32(lens).repeat_interleave(ql * g) >= 0
    own_region = (pos // rt).clamp(min=0)
    most = max(k, int(own_region.max()) + 1)
    key = torch.rand((len(pos), most), generator=gen, device="cuda")
    key[torch.arange(most, device="cuda")[None] > own_region[:, None]] = -1.0
    key[torch.arange(len(pos), device="cuda"), own_region] = 2.0
    best, ids = key.topk(k, dim=1)
    s["regions"] = torch.where(best >= 0, ids, torch.full_like(ids, -1)).to(torch.int32)
    s["positions"], s["active"] = pos.to(torch.int32), active


# ---------------------------------------------------------------------------------------------------------------------
# one pass


def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import sparse_decode_attention_02_gb300 as sda
    c = s["case"]
    if c["op"] in ("append", "chunk"):
        sda.sparse_decode_quantised_append(s["key"], s["value"], s["slots"], s["cache"], s["scales"])
    if c["op"] == "append":
        return s["cache"].view(FP8), s["scales"]
    if c["op"] in ("read", "chunk"):
        sda.sparse_decode_quantised_read(s["cache"], s["scales"], s["table"], s["starts"], s["key_out"], s["value_out"],
                                         first_tokens=s["first"])
        return s["key_out"], s["value_out"]
    if c["op"] == "attention":
        sda.sparse_decode_quantised_paged_attention(s["query"], s["cache"], s["scales"], s["table"], s["lens"], s["output"],
                                                    scale=s["scale"], query_len=c["query_len"], gate=s["gate"], lse=s["lse"])
        return s["output"], s["lse"]
    sda.sparse_decode_quantised_attention(s["query"], s["cache"], s["scales"], s["regions"], s["table"], s["positions"],
                                          s["active"], s["output"], scale=s["scale"], query_len=c["query_len"],
                                          region_tokens=c["region"], gate=s["gate"])
    return s["output"]


def _run_plain(s):
    op = s["case"]["op"]
    if op in ("append", "chunk"):
        _plain_append(s)
    if op == "append":
        return s["cache"].view(FP8), s["scales"]
    return _plain_read(s) if op in ("read", "chunk") else _plain_attention(s) if op == "attention" else _plain_regions(s)


def _plain_append(s):
    c = s["case"]
    g, d, span, int8 = (c[k] for k in ("groups", "dim", "span", "int8"))
    raw, scales = s["cache"].view(torch.uint8), s["scales"]
    n = raw.shape[2] // span
    blocks = raw.view(raw.shape[0], g, n, span, 2, d)
    live = s["slots"] >= 0
    slots = s["slots"][live]
    x = torch.stack([s["key"][live], s["value"][live]], 2).float()                        # [rows, groups, K or V, dim]
    touched, which = torch.unique(slots // span, return_inverse=True)
    place = slots % span
    count = touched.shape[0]
    first = torch.full((count,), span, device="cuda").scatter_reduce(0, which, place, "amin")
    amax = torch.zeros((count, g, 2), device="cuda")
    amax = amax.scatter_reduce(0, which[:, None, None].expand(-1, g, 2), x.abs().amax(-1), "amax")
    page, part = touched // n, touched % n
    had = scales[page, :, part]                                                           # [count, groups, K or V]
    need = _need(amax, int8)
    scale = torch.where((first == 0)[:, None, None], need, torch.maximum(had, need))
    scales[page, :, part] = scale
    held = blocks[page, :, part]                                                          # [count, groups, span, K or V, dim]
    again = _elements(_values(held, int8) * (had / scale)[:, :, None, :, None], int8)
    older = torch.arange(span, device="cuda")[None] < first[:, None]
    keep = older[:, None, :, None] & (scale > had)[:, :, None]
    blocks[page, :, part] = torch.where(keep[..., None], again, held)
    blocks[slots // span // n, :, slots // span % n, place] = _elements(x / scale[which][..., None], int8)


def _decoded(s, page, place):
    """Keys and values of places of the cache, [..., groups, 2 dim] in 32 bits."""
    c = s["case"]
    d = c["dim"]
    at = s["scales"][page, :, place // c["span"]]                                         # [..., groups, 2]
    return _values(s["cache"][page, :, place], c["int8"]) * at.repeat_interleave(d, -1)


def _plain_read(s):
    c = s["case"]
    d, b = c["dim"], c["block"]
    rows = torch.arange(s["key_out"].shape[0], device="cuda")
    owner = torch.searchsorted(s["starts"].long(), rows, right=True) - 1
    token = rows - s["starts"].long()[owner] + s["first"].long()[owner]
    x = _decoded(s, s["table"].long()[owner, token // b], token % b).to(torch.bfloat16)
    return x[..., :d].contiguous(), x[..., d:].contiguous()


def _gate_of(s, shape):
    gate = 1.0 / (1.0 + torch.exp(-s["gate"].float()))
    return gate.to(torch.bfloat16).float().view(shape)


def _plain_attention(s):
    c = s["case"]
    b, g, h, d, ql, n = (c[k] for k in ("block", "groups", "heads", "dim", "query_len", "requests"))
    at = torch.arange(s["longest"], device="cuda")
    kv = _decoded(s, s["table"].long().clamp(min=0)[:, at // b], at % b)                  # [requests, longest, groups, 2 dim]
    q = s["query"].float().view(n, ql, g, h, d)
    logits = torch.einsum("qjghd,qngd->qjghn", q, kv[..., :d]) * s["scale"]
    last = s["lens"].long()[:, None] - ql + torch.arange(ql, device="cuda")               # position of each query token
    logits.masked_fill_((at > last[..., None])[:, :, None, None], float("-inf"))
    top = logits.amax(-1, keepdim=True)
    top = torch.where(top == float("-inf"), torch.zeros_like(top), top)
    p = torch.exp(logits - top)
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("qjghn,qngd->qjghd", p, kv[..., d:])
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    if s["gate"] is not None:
        o = o * _gate_of(s, (n, ql, g, h, 1))
    return o.view(n * ql * g, h, d).to(torch.bfloat16), (top + torch.log(total)).view(n * ql * g, h)


def _plain_regions(s):
    c = s["case"]
    b, g, h, d, ql, rt = (c[k] for k in ("block", "groups", "heads", "dim", "query_len", "region"))
    rows = s["query"].shape[0]
    row = torch.arange(rows, device="cuda")[:, None]
    token = (s["regions"].long()[:, :, None] * rt + torch.arange(rt, device="cuda")).view(rows, -1)
    seen = (token >= 0) & (s["regions"] >= 0).repeat_interleave(rt, 1) & (token <= s["positions"].long()[:, None]) & s["active"][:, None]
    token = torch.where(seen, token, torch.zeros_like(token))
    page = s["table"].long().clamp(min=0)[row // (g * ql), token // b]
    place, group = token % b, row % g
    scale = s["scales"][page, group, place // c["span"]]                                  # [rows, tokens, K or V]
    kv = _values(s["cache"][page, group, place], c["int8"])
    logits = torch.einsum("rhd,rnd->rhn", s["query"].float(), kv[..., :d]) * (scale[:, None, :, 0] * s["scale"])
    logits.masked_fill_(~seen[:, None], float("-inf"))
    top = logits.amax(-1, keepdim=True)
    p = torch.exp(logits - torch.where(top == float("-inf"), torch.zeros_like(top), top))
    total = p.sum(-1, keepdim=True)
    o = torch.einsum("rhn,rnd->rhd", p * scale[:, None, :, 1], kv[..., d:])
    o = torch.where(total > 0, o / total, torch.zeros_like(o))
    if s["gate"] is not None:
        o = o * _gate_of(s, (rows // g, g, h)).reshape(rows, h, 1)
    return o.to(torch.bfloat16)


# ---------------------------------------------------------------------------------------------------------------------
# the definitions in 64 bits, apart from the plain forms


def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    with torch.no_grad():
        if op in ("append", "chunk"):
            cache, scales = _exact_append(s)
            if op == "append":
                return cache, scales
            return _exact_read(s, cache, scales)
        if op == "read":
            return _exact_read(s, _exact_values(s), s["scales"].double())
        return _exact_attention(s) if op == "attention" else _exact_regions(s)


def _exact_values(s):
    return (s["cache"] if s["case"]["int8"] else s["cache"].view(FP8).float()).double()


def _round_e4m3(v):
    """To three bits behind the first, ties to even, in steps of 2^-9 below 2^-6."""
    step = torch.exp2((torch.frexp(v)[1] - 1).clamp(min=-6).double() - 3)
    return (torch.round(v / step) * step).clamp(-448, 448)


def _exact_append(s):
    """One run of tokens of a block after another: the rows of a request that lie in it."""
    c = s["case"]
    d, b, span, int8 = (c[k] for k in ("dim", "block", "span", "int8"))
    cache, scales = _exact_values(s), s["scales"].double()
    lens, table, new = _lengths(c), s["table"].tolist(), c["new"]
    rounded = torch.round if int8 else _round_e4m3
    for q, n in enumerate(lens):
        at = n
        while 0 <= n and at < n + new:
            end = min(n + new, (at // span + 1) * span)
            rows = slice(q * new + at - n, q * new + end - n)
            page, place = table[q][at // b], at % b
            start = place // span * span
            x = torch.cat([s["key"][rows], s["value"][rows]], -1).double()                # [rows, groups, 2 dim]
            top = x.view(-1, c["groups"], 2, d).abs().amax((0, 3))
            if int8:
                need = top / 127
            else:
                need = torch.exp2(torch.floor(torch.log2(top / 448)) - 1)
                for _ in range(3):
                    need = torch.where(448 * need < top, 2 * need, need)
            had = scales[page, :, place // span].clone()
            scale = need if at % span == 0 else torch.maximum(had, need)
            scales[page, :, place // span] = scale
            wide = scale.repeat_interleave(d, -1)                                         # [groups, 2 dim]
            if at % span:
                factor = (had / scale).repeat_interleave(d, -1)[:, None]
                held = cache[page, :, start:place]
                cache[page, :, start:place] = torch.where(factor < 1, rounded(held * factor), held)
            cache[page, :, place:place + end - at] = rounded(x / wide).transpose(0, 1)
            at = end
    return cache, scales


def _exact_read(s, values, scales):
    c = s["case"]
    d, b = c["dim"], c["block"]
    keys, vals = [], []
    for q, (a, n) in enumerate(_reads(c)):
        if n:
            pages = s["table"][q, :_ceil(a + n, b)].long()
            wide = scales[pages].repeat_interleave(c["span"], 2)                          # [pages, groups, block, 2]
            x = values[pages].view(*wide.shape, d) * wide[..., None]
            x = x.transpose(1, 2).reshape(-1, c["groups"], 2, d)[a:a + n]
            keys.append(x[:, :, 0])
            vals.append(x[:, :, 1])
    if not keys:
        return s["key_out"].double(), s["value_out"].double()
    return torch.cat(keys), torch.cat(vals)


def _rows_exact(s, q, pages, group):
    """Keys and values of a request's pages for one group, [tokens, dim] each."""
    c = s["case"]
    d = c["dim"]
    raw = s["cache"][pages, group]
    x = (raw if c["int8"] else raw.view(FP8).float()).double().view(-1, c["span"], 2, d)
    x = (x * s["scales"][pages, group].double().view(-1, 1, 2, 1)).view(-1, 2, d)
    return x[:, 0], x[:, 1]


def _gated(s, o):
    if s["gate"] is not None:               # the gate factor is rounded to bf16 by definition
        o *= torch.sigmoid(s["gate"].float()).to(torch.bfloat16).double().view(*o.shape[:2], 1)
    return o


def _exact_attention(s):
    c = s["case"]
    g, ql = c["groups"], c["query_len"]
    query = s["query"].double()
    out, lse = torch.zeros_like(query), torch.full(query.shape[:2], float("-inf"), dtype=torch.float64, device="cuda")
    for q, n in enumerate(_lengths(c)):
        pages = s["table"][q, :_ceil(max(n, 0), c["block"])].long()
        for group in range(g if n > 0 else 0):
            k, v = _rows_exact(s, q, pages, group)
            for j in range(ql):
                seen, r = n - ql + 1 + j, (q * ql + j) * g + group
                if seen > 0:
                    z = query[r] @ k[:seen].T * s["scale"]
                    out[r] = torch.softmax(z, -1) @ v[:seen]
                    lse[r] = torch.logsumexp(z, -1)
    return _gated(s, out), lse


def _exact_regions(s):
    c = s["case"]
    g, ql, rt = c["groups"], c["query_len"], c["region"]
    query = s["query"].double()
    out = torch.zeros_like(query)
    positions = s["positions"].tolist()
    for q, n in enumerate(_lengths(c)):
        pages = s["table"][q, :_ceil(max(n, 0), c["block"])].long()
        for group in range(g if n > 0 else 0):
            k, v = _rows_exact(s, q, pages, group)
            for j in range(ql):
                r = (q * ql + j) * g + group
                ids = s["regions"][r].long()
                t = (ids[ids >= 0][:, None] * rt + torch.arange(rt, device="cuda")).view(-1)
                t = t[t <= positions[r]]
                if len(t):
                    out[r] = torch.softmax(query[r] @ k[t].T * s["scale"], -1) @ v[t]
    return _gated(s, out)

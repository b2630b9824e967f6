"""The cache operators of the library, measured: writing tokens into the paged
KV cache (with the position rotation), single-token attention over a cache held
in 4 bits, and the causal attention of whole prompts over a paged cache.

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes what a serving program holds before the call, and ``run()``
makes one pass: with ``own`` the library's calls, without it the same
mathematics in elementary torch operations (32-bit arithmetic, rounded once).
``exact()`` computes the outputs in 64 bits from the definitions.

A case is a dict of

  op        append   new tokens into the cache, rotated; then, for 4-bit pages,
                     the values that the cache now holds for them
            decode   one query token per sequence over every token of a 4-bit cache
            listed   one query token over listed pages and the open tail of a 4-bit cache
            prompt   causal attention of each sequence's newest tokens over the cache
  fmt       q4 or bf16: the format of the cache's pages
  page      tokens of a page;  batch, hq, hkv: sequences, query heads, KV heads
  ctx       tokens of the longest sequence, the new ones included
  ragged    how far below ctx the shortest sequence may lie
  new       new tokens of the longest sequence (append, prompt); the others have
            down to half as many where ``odd`` is set
  rot       rotated dimensions of a head, pairs: "half" (d, d + rot/2) or "next" (d, d + 1)
  budget    tokens of the page list (listed)

4-bit pages hold, for every 32 consecutive dimensions of a token's key (and of
its value), a half-precision scale s = max|x| / 7 and codes in [-7, 7]: x = s * code.
"""

import math

import torch

own = False

D = 128
TILE = 16  # tokens of a tile of a 4-bit page


def listed():
    return [
        # one decode step of a small batch: eight conversations, bf16 pages; the smallest call, where latency counts
        dict(name="append step bf16 b8", op="append", fmt="bf16", page=64, batch=8, hq=32, hkv=8, ctx=1000, ragged=700,
             new=1, odd=0, rot=128, pairs="half", seed=1),
        # prompts of four users admitted together, bf16 pages, ragged lengths
        dict(name="append prompts bf16", op="append", fmt="bf16", page=64, batch=4, hq=32, hkv=8, ctx=5003, ragged=900,
             new=4099, odd=1, rot=128, pairs="half", seed=2),
        # one decode step of the growing workload's batch, into 4-bit pages
        dict(name="append step 4-bit b32", op="append", fmt="q4", page=64, batch=32, hq=32, hkv=8, ctx=1100, ragged=1000,
             new=1, odd=0, rot=128, pairs="half", seed=3),
        # long prompts into 16-token 4-bit pages of a model with 2 KV heads that rotates half of each head, neighbours paired
        dict(name="append prompts 4-bit", op="append", fmt="q4", page=16, batch=3, hq=32, hkv=2, ctx=11003, ragged=0,
             new=11003, odd=1, rot=64, pairs="next", seed=4),
        # the tiny workload: one sequence, one head, 4K tokens
        dict(name="decode 4-bit tiny", op="decode", fmt="q4", page=64, batch=1, hq=1, hkv=1, ctx=4096, ragged=0, seed=5),
        # the 128K workload's heads, an odd length that ends inside a page
        dict(name="decode 4-bit 128K", op="decode", fmt="q4", page=64, batch=1, hq=32, hkv=8, ctx=131001, ragged=0, seed=6),
        # the growing workload's batch at ragged lengths, in 16-token pages
        dict(name="decode 4-bit b32 9K", op="decode", fmt="q4", page=16, batch=32, hq=32, hkv=8, ctx=9216, ragged=4000,
             seed=7),
        # the 1M workload: 16 query heads share each of 2 KV heads
        dict(name="decode 4-bit 1M", op="decode", fmt="q4", page=64, batch=1, hq=32, hkv=2, ctx=1048576, ragged=0, seed=8),
        # the attention of one page-selected decode step at 128K: 32 listed pages and an open tail
        dict(name="listed 4-bit 128K", op="listed", fmt="q4", page=64, batch=1, hq=32, hkv=8, ctx=131001, ragged=0,
             budget=2048, seed=9),
        # one long prompt, from its first token, in 4-bit pages
        dict(name="prompt 4-bit 8K", op="prompt", fmt="q4", page=64, batch=1, hq=32, hkv=8, ctx=8191, ragged=0, new=8191,
             odd=0, seed=10),
        # the next chunk of two long prompts over what the cache holds already, bf16 pages
        dict(name="prompt chunk bf16 30K", op="prompt", fmt="bf16", page=64, batch=2, hq=32, hkv=8, ctx=30011, ragged=9000,
             new=2048, odd=1, seed=11),
        # five draft tokens of each of eight sequences checked at once, 4-bit 16-token pages
        dict(name="prompt 4-bit 5 of 16K", op="prompt", fmt="q4", page=16, batch=8, hq=32, hkv=8, ctx=16411, ragged=9000,
             new=5, odd=1, seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "decode", "listed", "prompt"])
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 8, 16]) if hkv <= 2 else rng.choice([1, 3, 4, 4])
    c = dict(op=op, fmt="q4", page=rng.choice([16, 64]), batch=1, hq=hkv * group, hkv=hkv, seed=rng.randrange(1 << 20))
    if op == "append":
        c["fmt"] = rng.choice(["q4", "bf16"])
        c["batch"] = _log(rng, 1, 32)
        c["new"] = rng.choice([1, _log(rng, 2, max(2, 12000 // c["batch"]))])
        c["ctx"] = c["new"] + rng.choice([0, _log(rng, 1, 1500)])
        c["ragged"] = rng.randrange(0, c["ctx"] - c["new"] + 1)
        c["odd"], c["rot"], c["pairs"] = rng.randrange(2), rng.choice([32, 64, 96, 128]), rng.choice(["half", "next"])
    elif op == "decode":
        c["ctx"] = _log(rng, 1, 300000)
        c["batch"] = _log(rng, 1, max(1, min(32, 600000 // (c["ctx"] * hkv))))
        c["ragged"] = rng.randrange(0, c["ctx"])
    elif op == "listed":
        c["ctx"] = _log(rng, 300, 300000)
        c["batch"] = _log(rng, 1, max(1, min(16, 600000 // (c["ctx"] * hkv))))
        c["ragged"] = rng.randrange(0, c["ctx"] // 2)
        c["budget"] = _log(rng, 64, 4096)
    else:
        c["fmt"] = rng.choice(["q4", "q4", "bf16"])
        c["new"] = _log(rng, 2, 4096)
        c["batch"] = _log(rng, 1, max(1, min(8, 4096 // c["new"])))
        c["ctx"] = c["new"] + rng.choice([0, _log(rng, 1, max(2, min(30000, 40000000 // (c["new"] * c["batch"]))))])
        c["ragged"], c["odd"] = rng.randrange(0, c["ctx"] - c["new"] + 1), rng.randrange(2)
    return c


def _lengths(case):
    """Tokens of each sequence, and how many of them are new."""
    n = case["batch"]
    ctx = [case["ctx"] - (b * 2654435761 >> 7) % (case["ragged"] + 1) if b else case["ctx"] for b in range(n)]
    new = [0] * n
    if "new" in case:
        new = [case["new"] - ((b * 40503 + 77) % (case["new"] // 2 + 1) if b and case["odd"] else 0) for b in range(n)]
    return ctx, new


def work(case):
    ctx, new = _lengths(case)
    hq, hkv = case["hq"], case["hkv"]
    token = hkv * (144 if case["fmt"] == "q4" else 512)  # keys and values of one token
    if case["op"] == "append":
        t = sum(new)
        moved = t * (hkv * 512 + 2 * hq * 256 + case["rot"] * 4) + t * token
        if case["fmt"] == "q4":
            moved += t * token + t * hkv * 512  # read back, and the values
        return {"bytes": moved, "flops": t * (hq + hkv) * case["rot"] * 3}
    if case["op"] == "prompt":
        pairs = sum(n * (c - n) + n * (n + 1) // 2 for c, n in zip(ctx, new))
        rows = sum(new) * hq
    elif case["op"] == "decode":
        pairs, rows = sum(ctx), case["batch"] * hq
    else:
        full = [max(0, c // case["page"] - 1) for c in ctx]
        ctx = [min(case["budget"] // case["page"], f) * case["page"] + c - f * case["page"] for c, f in zip(ctx, full)]
        pairs, rows = sum(ctx), case["batch"] * hq
    return {"bytes": sum(ctx) * token + rows * (4 * D + 4), "flops": 4 * D * pairs * hq}


# ---- the 4-bit pages: [pages][hkv][page * 144] bytes --------------------------------
# 64 bytes a token of key codes, 8 of key scales, 64 of value codes, 8 of value
# scales, each kind together; the scales' and values' order repeats every 16 tokens.


def _parts(blocks, page):
    return blocks.split([page * 64, page * 8, page * 64, page * 8], dim=-1)


def _keys(codes, scales):
    """[..., page * 64] and [..., page * 8] bytes -> [..., page, 128] in 32 bits."""
    lead = codes.shape[:-1]
    x = codes.view(*lead, -1, 4, 4, 2, 2)  # token, c, j, byte / 2, byte % 2
    x = torch.stack([x & 15, x >> 4], dim=-1).to(torch.int8) - 8
    x = x.movedim((-4, -5, -2, -1, -3), (-5, -4, -3, -2, -1))  # j, c, byte % 2, nibble, byte / 2
    x = x.reshape(*lead, -1, 4, 32).float()
    return (x * scales.view(torch.float16).view(*lead, -1, 4, 1).float()).flatten(-2)


def _values(codes, scales):
    lead = codes.shape[:-1]
    x = codes.view(*lead, -1, 2, 8, 4, 4, 2, 2)  # tile, t / 8, g, c, j, t % 2, byte
    x = torch.stack([x & 15, x >> 4], dim=-1).to(torch.int8) - 8
    x = x.movedim((-7, -5, -3, -4, -6, -2, -1), (-7, -6, -5, -4, -3, -2, -1))  # t / 8, c, t % 2, j, g, byte, nibble
    x = x.reshape(*lead, -1, TILE, 4, 32).float()
    s = scales.view(torch.float16).view(*lead, -1, 4, 2, 4, 2).movedim((-3, -4, -1, -2), (-4, -3, -2, -1))
    x = x * s.reshape(*lead, -1, TILE, 4, 1).float()
    return x.reshape(*lead, -1, D)


def _pack_keys(q):
    """int8 codes [..., page, 128] -> bytes [..., page * 64]."""
    lead = q.shape[:-2]
    x = (q + 8).to(torch.uint8).view(*lead, -1, 4, 4, 2, 2, 2)  # token, j, c, byte % 2, nibble, byte / 2
    x = x.movedim((-4, -5, -1, -3, -2), (-5, -4, -3, -2, -1))
    return (x[..., 0] | x[..., 1] << 4).reshape(*lead, -1)


def _pack_values(q):
    lead = q.shape[:-2]
    x = (q + 8).to(torch.uint8).view(*lead, -1, 2, 4, 2, 4, 8, 2, 2)  # tile, t / 8, c, t % 2, j, g, byte, nibble
    x = x.movedim((-7, -3, -6, -4, -5, -2, -1), (-7, -6, -5, -4, -3, -2, -1))
    return (x[..., 0] | x[..., 1] << 4).reshape(*lead, -1)


def _pack_value_scales(s):
    """half scales [..., page, 4] -> bytes [..., page * 8]."""
    lead = s.shape[:-2]
    x = s.view(*lead, -1, 2, 4, 2, 4).movedim((-4, -3, -1, -2), (-3, -4, -2, -1))  # tile, c, t / 8, j, t % 2
    return x.contiguous().view(*lead, -1).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed((case["seed"] << 20) ^ seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    P, B, hq, hkv = case["page"], case["batch"], case["hq"], case["hkv"]
    ctx, new = _lengths(case)
    cols = max(-(-c // P) for c in ctx)
    pages = B * cols + 3
    s = {"case": case, "ctx": ctx, "new": new, "max_new": max(new)}
    s["table"] = torch.randperm(pages, generator=gen, device="cuda")[:B * cols].view(B, cols).int()
    s["lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
    if case["fmt"] == "q4":
        blocks = torch.empty(pages, hkv, P * 144, dtype=torch.uint8, device="cuda")
        kq, ks, vq, vs = _parts(blocks, P)
        for codes, pack in ((kq, _pack_keys), (vq, _pack_values)):
            codes.copy_(pack((normal(pages, hkv, P, D) * 2.6).round_().clamp_(-7, 7).to(torch.int8)))
        for scales, pack in ((ks, lambda x: x.view(pages, hkv, -1).view(torch.uint8)), (vs, _pack_value_scales)):
            scales.copy_(pack((0.3 * (0.25 * normal(pages, hkv, P, 4)).exp()).half()))
        s["k"], s["v"] = blocks, None
    else:
        s["k"] = normal(pages, hkv, P, D).bfloat16()
        s["v"] = normal(pages, hkv, P, D).bfloat16()
    if case["op"] in ("append", "prompt"):
        t = sum(new)
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        s["total"] = t
    if case["op"] == "append":
        # the projection's output: queries, keys and values of a token side by side
        s["qkv"] = (normal(t, hq + 2 * hkv, D) * torch.where(torch.arange(D, device="cuda") % 32 == 5, 6.0, 1.0)).bfloat16()
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        at = torch.arange(max(ctx), dtype=torch.float64, device="cuda")[:, None] * inv
        s["rope"] = torch.cat([at.cos(), at.sin()], dim=1).float()
    elif case["op"] == "prompt":
        s["q"] = (2 * normal(t, hq, D)).bfloat16()
    else:
        s["q"] = (2.5 * normal(B, hq, D)).bfloat16()
    # all but the last full page have summaries, so the tail of a page list is between one and two pages
    s["nsum"] = (s["lens"] // P - 1).clamp(min=0).int()
    if case["op"] == "listed":
        k = min(case["budget"] // P, cols)
        rank = torch.rand(B, hkv, cols, generator=gen, device="cuda")
        rank.masked_fill_(torch.arange(cols, device="cuda") >= s["nsum"][:, None, None], 2.0)
        s["count"] = s["nsum"].clamp(max=k)[:, None].repeat(1, hkv).contiguous()
        chosen = rank.argsort(dim=-1)[..., :k]
        past = torch.arange(k, device="cuda") >= s["count"][..., None]
        s["list"] = chosen.masked_fill(past, 1 << 30).sort(dim=-1).values.masked_fill(past, 0).int()
    return s


def _handle(s):
    """The runtime that a serving program keeps for its cache."""
    if "handle" not in s:
        from sparse_kv_page_rank_gb300.runtime import LocksRuntime

        case = s["case"]
        s["handle"] = LocksRuntime(s["k"], s["v"], s["table"], s["lens"], s["nsum"], case["hq"], 2, case.get("budget", 0))
        if "list" in s:
            s["handle"].sel_pages.copy_(s["list"])
            s["handle"].sel_count.copy_(s["count"])
    return s["handle"]


def _softmax(scores, seen):
    """Weights and log-sum-exp of the last axis over the places that are seen."""
    scores = scores.masked_fill(~seen, float("-inf"))
    top = scores.amax(dim=-1, keepdim=True)
    w = (scores - top).exp()
    total = w.sum(dim=-1, keepdim=True)
    return w / total, (top + total.log()).squeeze(-1)


def _rotate(x, cos, sin, rot, pairs):
    """x [t, h, 128] in 32 bits, cos and sin [t, 1, rot / 2]."""
    y = x.clone()
    if pairs == "half":
        a, b = x[..., :rot // 2], x[..., rot // 2:rot]
        y[..., :rot // 2], y[..., rot // 2:rot] = a * cos - b * sin, b * cos + a * sin
    else:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        y[..., 0:rot:2], y[..., 1:rot:2] = a * cos - b * sin, b * cos + a * sin
    return y


def _quantise(x):
    """[..., 128] in 32 bits -> (int8 codes, half scales [..., 4])."""
    g = x.view(*x.shape[:-1], 4, 32)
    s = (g.abs().amax(dim=-1) / 7).half()
    q = (g / s.float()[..., None]).round().clamp(-7, 7).nan_to_num(0.0)
    return q.view(x.shape).to(torch.int8), s


def _places(s):
    """Of each new token: its sequence and its position there."""
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new, output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - s["cu"][seq] + (s["lens"] - new)[seq]
    return seq, at


def _append(s):
    case = s["case"]
    hq, hkv, P, rot = case["hq"], case["hkv"], case["page"], case["rot"]
    seq, at = _places(s)
    q, k, v = s["qkv"].float().split([hq, hkv, hkv], dim=1)
    cos, sin = s["rope"][at].unsqueeze(1).split(rot // 2, dim=-1)
    q = _rotate(q, cos, sin, rot, case["pairs"]).bfloat16()
    k = _rotate(k, cos, sin, rot, case["pairs"]).bfloat16()
    page, slot = s["table"][seq, at // P].long(), at % P
    if case["fmt"] == "bf16":
        s["k"][page, :, slot], s["v"][page, :, slot] = k, v.bfloat16()
        return {"q": q, "k_pool": s["k"], "v_pool": s["v"]}
    codes = [_quantise(x.float()) for x in (k, v)]
    # the page's bytes are rewritten around the new tokens, page by page of the whole pool
    kq, ks, vq, vs = _parts(s["k"], P)
    lead = kq.shape[:-1]
    keys = kq.reshape(*lead, P, 64).clone()
    keys[page, :, slot] = _pack_keys(codes[0][0].unsqueeze(2))
    kq.copy_(keys.view(*lead, -1))
    scales = ks.reshape(*lead, -1).view(torch.float16).view(*lead, P, 4)
    scales[page, :, slot] = codes[0][1]
    ks.copy_(scales.view(*lead, -1).view(torch.uint8))
    # a token's value bytes: 32 places of two bytes in its tile
    d = torch.arange(0, D, 4, device="cuda")
    t = slot % TILE
    base = slot // TILE * 1024 + t // 8 * 512 + t % 8 // 2 * 16 + t % 2 * 2
    where = base[:, None, None] + (d % 32 // 4 * 64 + d // 32 * 4)[:, None] + torch.arange(2, device="cuda")
    u = (codes[1][0] + 8).to(torch.uint8).view(-1, hkv, D // 4, 2, 2)
    u = u[..., 0] | u[..., 1] << 4
    heads = torch.arange(hkv, device="cuda")
    vq[page[:, None, None, None], heads[None, :, None, None], where[:, None]] = u
    base = slot // TILE * 128 + t % 8 // 2 * 32 + t // 8 * 16 + t % 2 * 2
    where = base[:, None, None] + (torch.arange(4, device="cuda") * 4)[:, None] + torch.arange(2, device="cuda")
    u = codes[1][1].contiguous().view(torch.uint8).view(-1, hkv, 4, 2)
    vs[page[:, None, None, None], heads[None, :, None, None], where[:, None]] = u
    keys, values = _keys(kq[page], ks[page]), _values(vq[page], vs[page])
    row = torch.arange(s["total"], device="cuda")
    return {"q": q, "k": keys[row, :, slot].bfloat16(), "v": values[row, :, slot].bfloat16()}


def _gather(s, tables):
    """Keys and values in 32 bits, [batch, hkv, tokens, 128], of the physical pages [batch, hkv or 1, n]."""
    hkv, P = s["case"]["hkv"], s["case"]["page"]
    heads = torch.arange(hkv, device="cuda")[:, None]
    if s["v"] is None:
        kq, ks, vq, vs = _parts(s["k"][tables, heads], P)
        k, v = _keys(kq.contiguous(), ks.contiguous()), _values(vq.contiguous(), vs.contiguous())
    else:
        k, v = s["k"][tables, heads].float(), s["v"][tables, heads].float()
    return k.flatten(2, 3), v.flatten(2, 3)


def _decode(s):
    case = s["case"]
    B, hq, hkv, P = case["batch"], case["hq"], case["hkv"], case["page"]
    if case["op"] == "decode":
        pages = torch.arange(s["table"].shape[1], device="cuda")[None, None, :].expand(B, 1, -1)
        held = torch.ones_like(pages, dtype=torch.bool)
    else:
        tail = s["nsum"][:, None] + torch.arange(2, device="cuda")
        pages = torch.cat([s["list"], tail[:, None, :].expand(B, hkv, 2)], dim=2).long()
        last = s["lens"][:, None, None] > pages * P
        k = s["list"].shape[2]
        held = torch.cat([torch.arange(k, device="cuda") < s["count"][..., None], last[..., k:]], dim=2)
    tables = s["table"].gather(1, pages.clamp(max=s["table"].shape[1] - 1).flatten(1)).view_as(pages).long()
    k, v = _gather(s, tables)
    at = (pages[..., None] * P + torch.arange(P, device="cuda")).flatten(2)
    seen = held.repeat_interleave(P, dim=2) & (at < s["lens"][:, None, None])
    q = s["q"].float().view(B, hkv, hq // hkv, D)
    w, lse = _softmax(q @ k.transpose(2, 3) / math.sqrt(D), seen[:, :, None, :])
    # places that are not seen may hold anything, so their values are left out and not only weighted with 0
    out = w @ v.masked_fill(~seen[..., None], 0.0)
    return {"out": out.reshape(B, hq, D).bfloat16(), "lse": lse.reshape(B, hq)}


def _prompt(s):
    case = s["case"]
    B, hq, hkv, P = case["batch"], case["hq"], case["hkv"], case["page"]
    seq, at = _places(s)
    row = torch.arange(s["total"], device="cuda") - s["cu"][seq]
    n = s["max_new"]
    q = torch.zeros(B, n, hkv, hq // hkv, D, device="cuda")
    q[seq, row] = s["q"].float().view(-1, hkv, hq // hkv, D)
    pos = torch.zeros(B, n, dtype=torch.long, device="cuda")
    pos[seq, row] = at
    k, v = _gather(s, s["table"][:, None, :].long())
    keys = torch.arange(k.shape[2], device="cuda")
    seen = keys <= pos[:, None, :, None]
    # the group's heads share their keys; a sequence's rows go head by head
    q = q.permute(0, 2, 3, 1, 4).reshape(B, hkv, -1, D)
    scores = (q @ k.transpose(2, 3) / math.sqrt(D)).view(B, hkv, hq // hkv, n, -1)
    w, lse = _softmax(scores, seen[:, :, None])
    out = (w.view(B, hkv, -1, k.shape[2]) @ v.masked_fill(keys[:, None] >= s["lens"][:, None, None, None], 0.0))
    out = out.view(B, hkv, hq // hkv, n, D).permute(0, 3, 1, 2, 4).reshape(B, n, hq, D)
    return {"out": out[seq, row].bfloat16(), "lse": lse.permute(0, 3, 1, 2).reshape(B, n, hq)[seq, row]}


def run(state):
    s, op = state, state["case"]["op"]
    if not own:
        return {"append": _append, "decode": _decode, "listed": _decode, "prompt": _prompt}[op](s)
    rt = _handle(s)
    if op == "append":
        hq, hkv = s["case"]["hq"], s["case"]["hkv"]
        q, k, v = s["qkv"].split([hq, hkv, hkv], dim=1)
        q = rt.append(k, v, q, rope=s["rope"], rotary_dim=s["case"]["rot"], interleaved=s["case"]["pairs"] == "next",
                      cu_tokens=s["cu"], max_tokens=s["max_new"])
        if s["v"] is not None:
            return {"q": q, "k_pool": s["k"], "v_pool": s["v"]}
        k, v = rt.read_tokens(s["total"], cu_tokens=s["cu"], max_tokens=s["max_new"])
        return {"q": q, "k": k, "v": v}
    if op == "prompt":
        out, lse = rt.prompt_attend(s["q"], cu_tokens=s["cu"], max_tokens=s["max_new"])
    elif op == "decode":
        out, lse = rt.dense_decode(s["q"])
    else:
        out, lse = rt.sparse_attend(s["q"])
    return {"out": out, "lse": lse}


# ---- the definitions in 64 bits ------------------------------------------------------


def _held(s, blocks):
    """[n, page * 144] bytes -> keys and values [n, page, 128] in 64 bits, place by place."""
    P = s["case"]["page"]
    t, d = torch.meshgrid(torch.arange(P, device="cuda"), torch.arange(D, device="cuda"), indexing="ij")
    bit = 4 * (d % 8 // 2) + 16 * (d % 2)
    kb, kn = t * 64 + d % 32 // 8 * 16 + d // 32 * 4 + bit // 8, bit % 8
    ks = P * 64 + t * 8 + d // 32 * 2
    u = t % 16
    vb = P * 72 + t // 16 * 1024 + u // 8 * 512 + d % 32 // 4 * 64 + u % 8 // 2 * 16 + d // 32 * 4 + u % 2 * 2 + d % 4 // 2
    vn = d % 2 * 4
    vs = P * 136 + t // 16 * 128 + u % 8 // 2 * 32 + u // 8 * 16 + d // 32 * 4 + u % 2 * 2
    out = []
    for b, n, sc in ((kb, kn, ks), (vb, vn, vs)):
        code = (blocks[:, b].int() >> n & 15) - 8
        scale = blocks.contiguous().view(torch.float16)[:, sc // 2].double()
        out.append(code * scale)
    return out


def _sequence(s, b, h):
    """Keys and values of one head of one sequence, [tokens, 128] in 64 bits."""
    pages = s["table"][b].long()
    k, v = _held(s, s["k"][pages, h]) if s["v"] is None else (s["k"][pages, h].double(), s["v"][pages, h].double())
    return k.reshape(-1, D)[:s["ctx"][b]], v.reshape(-1, D)[:s["ctx"][b]]


def _attend(q, k, v, hidden):
    x = q @ k.T / math.sqrt(D)
    if hidden is not None:
        x = x.masked_fill(hidden, float("-inf"))
    lse = x.logsumexp(dim=-1)
    return (x - lse[:, None]).exp() @ v, lse


def exact(case, seed):
    s = prepare(case, seed)
    B, hq, hkv, P = case["batch"], case["hq"], case["hkv"], case["page"]
    if case["op"] != "append":
        rows = s["q"].double()
        out = torch.empty(rows.shape, dtype=torch.float64, device="cuda")
        lse = torch.empty(rows.shape[:2], dtype=torch.float64, device="cuda")
        first = 0
        for b in range(B):
            n = s["new"][b] if case["op"] == "prompt" else 1
            for h in range(hkv):
                k, v = _sequence(s, b, h)
                if case["op"] == "listed":
                    full = int(s["nsum"][b])
                    chosen = s["list"][b, h, :int(s["count"][b, h])].tolist()
                    keep = [t for p in chosen for t in range(p * P, p * P + P)] + list(range(full * P, s["ctx"][b]))
                    k, v = k[keep], v[keep]
                for g in range(h * hq // hkv, (h + 1) * hq // hkv):
                    hidden = None
                    if case["op"] == "prompt":
                        at = torch.arange(s["ctx"][b], device="cuda")
                        hidden = at[None, :] > at[s["ctx"][b] - n:, None]
                    out[first:first + n, g], lse[first:first + n, g] = _attend(rows[first:first + n, g], k, v, hidden)
            first += n
        return {"out": out, "lse": lse}
    x = s["qkv"].double()
    at = torch.cat([torch.arange(c - n, c, device="cuda") for c, n in zip(s["ctx"], s["new"])])
    half = case["rot"] // 2
    angle = s["rope"].double()[at]
    turn = torch.complex(angle[:, :half], angle[:, half:])[:, None]
    y = x[:, :hq + hkv].clone()
    z = y[..., :2 * half].reshape(*y.shape[:2], 2, half).transpose(-1, -2) if case["pairs"] == "half" else y[..., :2 * half].reshape(*y.shape[:2], half, 2)
    z = torch.view_as_real(torch.view_as_complex(z.contiguous()) * turn)
    y[..., :2 * half] = z.transpose(-1, -2).flatten(-2) if case["pairs"] == "half" else z.flatten(-2)
    k, v = y[:, hq:], x[:, hq + hkv:]
    if case["fmt"] == "q4":
        held = []
        for a in (k.bfloat16().double(), v):
            g = a.reshape(*a.shape[:2], 4, 32)
            scale = (g.abs().amax(dim=-1, keepdim=True) / 7).half().double()
            held.append((torch.where(scale > 0, (g / scale).round().clamp(-7, 7), 0.0) * scale).view(a.shape))
        return {"q": y[:, :hq], "k": held[0], "v": held[1]}
    pools = [s["k"].double(), s["v"].double()]
    first = 0
    for b in range(B):
        for i in range(s["new"][b]):
            t = s["ctx"][b] - s["new"][b] + i
            if t % P == 0 or i == 0:  # the tokens of one page together
                m = min(P - t % P, s["new"][b] - i)
                page = int(s["table"][b, t // P])
                for pool, rows in zip(pools, (k, v)):
                    pool[page, :, t % P:t % P + m] = rows[first + i:first + i + m].transpose(0, 1)
        first += s["new"][b]
    return {"q": y[:, :hq], "k_pool": pools[0], "v_pool": pools[1]}

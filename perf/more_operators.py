"""The generation operators of the library, measured: appending tokens whose
positions have several axes, and beam search over the paged cache (choosing the
beams, moving them in the cache, attending with them).

``listed()`` names the cases, ``draw()`` gives more of the same ranges,
``prepare()`` makes what a serving program holds before the call, and ``run()``
makes one pass: with ``own`` the library's calls, without it the same
mathematics in elementary torch operations (32-bit arithmetic, 64 bits where
candidates are compared, rounded once). ``exact()`` computes the outputs in 64
bits from the definitions.

A case is a dict of

  op        turn     new tokens into the cache, rotated by their positions along several
                     axes; then, for 4-bit pages, the values that the cache now holds for them
            choose   the best continuations of every request's beams
            move     the beams' block tables, lengths and open pages after a choice; then, for
                     4-bit pages, what the open pages now hold
            attend   one query token per beam over the cache, whose first pages a request's beams share
  fmt       q4 or bf16: the format of the cache's pages (choose: bf16 or f32 logits)
  page      tokens of a page;  hq, hkv: query heads, KV heads
  batch     sequences (turn) or requests, each with ``beams`` of them
  ctx       turn: tokens of the longest sequence, the new ones included; else of the longest prompt
  ragged    how far below ctx the shortest may lie
  new       new tokens of the longest sequence (turn); the others have down to half as many where ``odd`` is set
  rot       rotated dimensions of a head, pairs: "half" (d, d + rot/2) or "next" (d, d + 1)
  parts     pairs of each axis, as a text;  cyclic: axes take turns (1) or follow one another (0)
  vocab     tokens to choose from;  keep: continuations kept;  ended: whether hypotheses may have ended
  tail      tokens of the longest continuation (move, attend);  layers: caches that move together
"""

import math

import torch

own = False

D = 128


def listed():
    return [
        # one decode step of a small batch of conversations about images: three axes, bf16 pages; latency
        dict(name="turn step bf16 b8", op="turn", fmt="bf16", page=64, batch=8, hq=32, hkv=8, ctx=1000, ragged=700, new=1,
             odd=0, rot=128, pairs="half", parts="16 24 24", cyclic=0, seed=1),
        # prompts of four users, text around images, ragged lengths
        dict(name="turn prompts bf16", op="turn", fmt="bf16", page=64, batch=4, hq=32, hkv=8, ctx=5003, ragged=900, new=4099,
             odd=1, rot=128, pairs="half", parts="24 20 20", cyclic=1, seed=2),
        # long video prompts into 16-token 4-bit pages, half of each head rotated, neighbours paired, height and width only
        dict(name="turn prompts 4-bit", op="turn", fmt="q4", page=16, batch=3, hq=32, hkv=2, ctx=11003, ragged=0, new=11003,
             odd=1, rot=64, pairs="next", parts="17 15", cyclic=0, seed=3),
        # one request of four beams, a small vocabulary: the smallest choice
        dict(name="choose b1 x 4", op="choose", fmt="bf16", batch=1, beams=4, vocab=32000, keep=4, ended=0, seed=4),
        # the growing workload's batch, four beams each, the 128K workload's vocabulary
        dict(name="choose b32 x 4", op="choose", fmt="bf16", batch=32, beams=4, vocab=128256, keep=4, ended=1, seed=5),
        # twice as many continuations as beams, so that ended ones can be set aside; 32-bit logits, rows that do not align
        dict(name="choose b24 x 8 f32", op="choose", fmt="f32", batch=24, beams=8, vocab=100003, keep=16, ended=0, seed=6),
        # one request of four beams in one layer's cache, a table for 128K tokens
        dict(name="move b1 x 4", op="move", fmt="bf16", page=64, batch=1, beams=4, hq=32, hkv=8, ctx=4001, ragged=0, tail=100,
             cols=2048, layers=1, seed=7),
        # sixteen requests of eight beams, four layers at once
        dict(name="move b16 x 8", op="move", fmt="bf16", page=64, batch=16, beams=8, hq=32, hkv=8, ctx=1200, ragged=500,
             tail=90, cols=64, layers=4, seed=8),
        # 16-token 4-bit pages
        dict(name="move 4-bit b32 x 4", op="move", fmt="q4", page=16, batch=32, beams=4, hq=32, hkv=8, ctx=2100, ragged=900,
             tail=77, cols=200, layers=1, seed=9),
        # one request of four beams, a short prompt
        dict(name="attend b1 x 4 2K", op="attend", fmt="bf16", page=64, batch=1, beams=4, hq=32, hkv=8, ctx=2001, ragged=0,
             tail=60, seed=10),
        # eight beams that share a document of 32K tokens
        dict(name="attend b1 x 8 32K", op="attend", fmt="bf16", page=64, batch=1, beams=8, hq=32, hkv=8, ctx=32768 + 11,
             ragged=0, tail=300, seed=11),
        # four requests of eight beams over 4-bit 16-token pages
        dict(name="attend 4-bit b4 x 8 16K", op="attend", fmt="q4", page=16, batch=4, beams=8, hq=32, hkv=8, ctx=16411,
             ragged=9000, tail=200, seed=12),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["turn", "choose", "move", "attend"])
    c = dict(op=op, seed=rng.randrange(1 << 20))
    if op == "choose":
        c["fmt"] = rng.choice(["bf16", "f32"])
        c["beams"] = _log(rng, 1, 16)
        c["vocab"] = _log(rng, 300, 200000)
        c["batch"] = _log(rng, 1, max(1, min(64, 16000000 // (c["vocab"] * c["beams"]))))
        c["keep"] = rng.choice([c["beams"], 2 * c["beams"], _log(rng, 1, 32)])
        c["ended"] = rng.randrange(2)
        return c
    hkv = rng.choice([1, 2, 4, 8])
    group = rng.choice([1, 2, 3, 4, 4, 8, 16]) if hkv <= 2 else rng.choice([1, 3, 4, 4])
    c.update(fmt=rng.choice(["q4", "bf16"]), page=rng.choice([16, 64]), hq=hkv * group, hkv=hkv)
    if op == "turn":
        c["batch"] = _log(rng, 1, 32)
        c["new"] = rng.choice([1, _log(rng, 2, max(2, 12000 // c["batch"]))])
        c["ctx"] = c["new"] + rng.choice([0, _log(rng, 1, 1500)])
        c["ragged"] = rng.randrange(0, c["ctx"] - c["new"] + 1)
        c["odd"], c["rot"], c["pairs"] = rng.randrange(2), rng.choice([32, 64, 96, 128]), rng.choice(["half", "next"])
        cuts = sorted(rng.randrange(0, c["rot"] // 2 + 1) for _ in range(rng.choice([1, 2, 2, 3])))
        parts, c["cyclic"] = [b - a for a, b in zip([0] + cuts, cuts + [c["rot"] // 2])], 0
        if rng.randrange(2):  # the axes after the first take turns, as many each
            n = rng.choice([2, 3])
            other = rng.randrange(1, c["rot"] // 2 // n + 1)
            parts, c["cyclic"] = [c["rot"] // 2 - (n - 1) * other] + [other] * (n - 1), 1
        c["parts"] = " ".join(map(str, parts))
        return c
    c["beams"] = _log(rng, 1, 16)
    c["ctx"] = _log(rng, 20, 4000 if op == "move" else 60000)
    c["ragged"] = rng.randrange(0, c["ctx"] // 2)
    c["tail"] = _log(rng, 1, 200)
    if op == "move":
        c["batch"] = _log(rng, 1, max(1, 128 // c["beams"]))
        c["layers"] = rng.choice([1, 2, 3]) if c["fmt"] == "bf16" else 1
        c["cols"] = (c["ctx"] + c["tail"]) // c["page"] + 2 + rng.choice([0, rng.randrange(1000)])
    else:
        c["ctx"] = min(c["ctx"], 7000000 // (c["beams"] * c["hq"]))
        c["ragged"] = min(c["ragged"], c["ctx"] // 2)
        c["batch"] = _log(rng, 1, max(1, min(8, 200000 // (c["ctx"] * hkv), 7000000 // (c["ctx"] * c["beams"] * c["hq"]))))
    return c


def _spread(i, n):
    """A number in [0, n] that looks drawn."""
    return (i * 2654435761 >> 7) % (n + 1)


def _lengths(case):
    """turn: tokens of each sequence, and how many are new. Else: tokens of each
    request's prompt, and of each beam."""
    n = case["batch"]
    ctx = [case["ctx"] - _spread(b, case["ragged"]) if b else case["ctx"] for b in range(n)]
    if case["op"] == "turn":
        return ctx, [case["new"] - ((b * 40503 + 77) % (case["new"] // 2 + 1) if b and case["odd"] else 0) for b in range(n)]
    beams = []
    for b, c in enumerate(ctx):
        gone = case["tail"] - (_spread(b + 5, case["tail"] // 2) if b else 0)
        for w in range(case["beams"]):
            # a beam that has ended is shorter than the others
            early = _spread(b + 7 * w, gone) if case["op"] == "attend" and w and (b + w) % 5 == 4 else 0
            beams.append(c + gone - early)
    return ctx, beams


def _pages(case):
    """Shared pages of each request; pages of the pool."""
    P, W = case["page"], case["beams"]
    ctx, lens = _lengths(case)
    shared = [c // P for c in ctx]
    cols = case.get("cols") or max(-(-n // P) for n in lens) + 1
    # every beam holds pages of its own for the tokens to come
    each = [min(cols, -(-(max(lens[b * W:b * W + W])) // P) + 1) - s for b, s in enumerate(shared)]
    return shared, each, cols


def _parents(case):
    """The beams that the last choice continued: most of them some, a few many."""
    W, out = case["beams"], []
    for b in range(case["batch"]):
        out += [min(W - 1, (_spread(97 * b + 13 * w + case["seed"], 1000) ** 2) * W // 1000000) for w in range(W)]
    return out


def _axes(case):
    """The axis of each rotated pair."""
    half, parts = case["rot"] // 2, [int(n) for n in case["parts"].split()]
    if not case["cyclic"]:
        return [a for a, n in enumerate(parts) for _ in range(n)]
    axis = [0] * half
    for a in range(1, len(parts)):
        for i in range(parts[a]):
            axis[a + i * len(parts)] = a
    return axis


def work(case):
    if case["op"] == "choose":
        rows, size = case["batch"] * case["beams"], 2 if case["fmt"] == "bf16" else 4
        live = rows - (sum(_has_ended(b, w) for b in range(case["batch"]) for w in range(case["beams"])) if case["ended"] else 0)
        return {"bytes": live * case["vocab"] * size + rows * 8 + case["batch"] * case["keep"] * 16,
                "flops": 3 * live * case["vocab"]}
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    token = hkv * (144 if case["fmt"] == "q4" else 512)  # keys and values of one token
    ctx, lens = _lengths(case)
    if case["op"] == "turn":
        t = sum(lens)
        moved = t * (hkv * 512 + 2 * hq * 256 + case["rot"] * 4 + 4 * len(case["parts"].split())) + t * token
        if case["fmt"] == "q4":
            moved += t * token + t * hkv * 512  # read back, and the values
        return {"bytes": moved, "flops": t * (hq + hkv) * case["rot"] * 3}
    W = case["beams"]
    if case["op"] == "move":
        parents, moved = _parents(case), 0
        for b in range(case["batch"]):
            mine = parents[b * W:b * W + W]
            open_tokens = lens[b * W] % P
            moved += (W - len(set(mine))) * open_tokens * token * 2 * case["layers"]
            # table entries of the beams that are not their own parents' successors
            moved += sum(8 * (lens[b * W] // P + 1) for w in range(W) if mine[w] != w) + 12 * W
            if case["fmt"] == "q4":
                moved += W * open_tokens * (token + hkv * 512)
        return {"bytes": moved, "flops": 0}
    shared = _pages(case)[0]
    once = sum(s * P for s in shared)
    tails = sum(n - shared[i // W] * P for i, n in enumerate(lens))
    rows = len(lens) * hq
    return {"bytes": (once + tails) * token + rows * (4 * D + 4), "flops": 4 * D * hq * sum(lens)}


# ---- the 4-bit pages: [pages][hkv][page * 144] bytes --------------------------------
# A token has 64 bytes of key codes, 4 key scales, 64 bytes of value codes and 4
# value scales. _where gives each of those 144 bytes its place in the page, and
# _KEY, _VALUE the dimensions in the low and high half of each code byte.


def _word(i):
    c, j, byte = i // 16, i // 4 % 4, i % 4
    d = 32 * j + 8 * c + 4 * (byte % 2) + byte // 2
    return d, d + 2


_KEY = [_word(i) for i in range(64)]
_VALUE = [(32 * j + 4 * c + 2 * e, 32 * j + 4 * c + 2 * e + 1) for j in range(4) for c in range(8) for e in range(2)]
_maps = {}


def _where(P):
    if P not in _maps:
        rows = []
        for t in range(P):
            u, tile = t % 16, t // 16
            inner = 16 * (u % 8 // 2) + 2 * (u % 2)
            row = [64 * t + i for i in range(64)] + [64 * P + 8 * t + i for i in range(8)]
            row += [72 * P + 1024 * tile + 512 * (u // 8) + inner + 64 * c + 4 * j + e
                    for j in range(4) for c in range(8) for e in range(2)]
            row += [136 * P + 128 * tile + 2 * inner + 16 * (u // 8) - 2 * (u % 2) + 4 * j + e for j in range(4) for e in range(2)]
            rows.append(row)
        order = [torch.tensor(m, device="cuda").T for m in (_KEY, _VALUE)]
        _maps[P] = torch.tensor(rows, device="cuda"), order
    return _maps[P]


def _tokens(blocks, P):
    """[..., page * 144] bytes -> [..., page, 144], token by token."""
    return blocks[..., _where(P)[0].flatten()].unflatten(-1, (P, 144))


def _values_of(tokens, P):
    """[..., 144] bytes -> keys and values [..., 128] in 32 bits."""
    out = []
    for (lo, hi), first in zip(_where(P)[1], (0, 72)):
        b = tokens[..., first:first + 64]
        x = torch.empty(*tokens.shape[:-1], D, device=tokens.device)
        x[..., lo], x[..., hi] = (b & 15).float() - 8, (b >> 4).float() - 8
        s = tokens[..., first + 64:first + 72].contiguous().view(torch.float16).float()
        out.append((x.unflatten(-1, (4, 32)) * s[..., None]).flatten(-2))
    return out


def _bytes_of(codes, scales, P):
    """Keys' and values' int8 codes [..., 128] and half scales [..., 4] -> [..., 144] bytes."""
    out = []
    for (lo, hi), q, s in zip(_where(P)[1], codes, scales):
        q = (q + 8).to(torch.uint8)
        out += [q[..., lo] | q[..., hi] << 4, s.contiguous().view(torch.uint8)]
    return torch.cat(out, dim=-1)


def _random_pool(case, pages, normal):
    """A pool of pages full of tokens: (k, v), or (blocks, None)."""
    P, hkv = case["page"], case["hkv"]
    if case["fmt"] == "bf16":
        return normal(pages, hkv, P, D).bfloat16(), normal(pages, hkv, P, D).bfloat16()
    blocks = torch.empty(pages, hkv, P * 144, dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 22) // (hkv * P))
    for i in range(0, pages, step):
        n = min(step, pages - i)
        codes = [(normal(n, hkv, P, D) * 2.6).round_().clamp_(-7, 7).to(torch.int8) for _ in range(2)]
        scales = [(0.3 * (0.25 * normal(n, hkv, P, 4)).exp()).half() for _ in range(2)]
        blocks[i:i + n, :, _where(P)[0].flatten()] = _bytes_of(codes, scales, P).flatten(-2)
    return blocks, None


def _has_ended(b, w):
    return w > 0 and (b + 3 * w) % 7 == 5


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed((case["seed"] << 20) ^ seed)

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda")

    B, s = case["batch"], {"case": case}
    if case["op"] == "choose":
        W, V = case["beams"], case["vocab"]
        # a few likely tokens stand out; one in thirty is forbidden
        x = 2.5 * normal(B * W, V) + 6.0 * (normal(B * W, V) > 3.3)
        x.masked_fill_(torch.rand(B * W, V, generator=gen, device="cuda") < 1 / 30, float("-inf"))
        s["logits"] = x.bfloat16() if case["fmt"] == "bf16" else x
        s["scores"] = (-20 - 0.5 * normal(B, W).abs()).contiguous()
        s["end"] = V // 3
        ended = [[int(_has_ended(b, w)) if case["ended"] else 0 for w in range(W)] for b in range(B)]
        s["ended"] = torch.tensor(ended, dtype=torch.int32, device="cuda")
        return s
    P, hq, hkv = case["page"], case["hq"], case["hkv"]
    ctx, lens = _lengths(case)
    if case["op"] == "turn":
        new = lens
        cols = max(-(-c // P) for c in ctx)
        pages = B * cols + 3
        t = sum(new)
        s.update(ctx=ctx, new=new, max_new=max(new), total=t)
        s["table"] = torch.randperm(pages, generator=gen, device="cuda")[:B * cols].view(B, cols).int()
        s["lens"] = torch.tensor(ctx, dtype=torch.int32, device="cuda")
        s["cu"] = torch.tensor([0] + new, device="cuda").cumsum(0).int()
        s["pools"] = [_random_pool(case, pages, normal)]
        # the projection's output: queries, keys and values of a token side by side
        s["qkv"] = (normal(t, hq + 2 * hkv, D) * torch.where(torch.arange(D, device="cuda") % 32 == 5, 6.0, 1.0)).bfloat16()
        half = case["rot"] // 2
        inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device="cuda") / half)
        at = torch.arange(max(ctx), dtype=torch.float64, device="cuda")[:, None] * inv
        s["rope"] = torch.cat([at.cos(), at.sin()], dim=1).float()
        # images of 40 by 25 patches between pieces of text, whose axes all advance
        i = torch.cat([torch.arange(c - n, c, device="cuda") for c, n in zip(ctx, new)])
        in_image = i % 1200 < 1000
        start = i // 1200 * 240
        patch = i % 1200
        text = start + (patch - 1000).clamp(min=0) + 40
        rows = [torch.where(in_image, start + off, text) for off in (patch * 0, patch // 40, patch % 40)]
        n = len(case["parts"].split())
        rows = ((rows if n == 3 else rows[1:]) * 2)[:n]
        s["positions"] = torch.stack(rows).clamp(max=max(ctx) - 1).int()
        return s
    W = case["beams"]
    shared, each, cols = _pages(case)
    s.update(ctx=ctx, new=lens, shared=shared)
    pages = sum(shared) + W * sum(each) + 3
    order = torch.randperm(pages, generator=gen, device="cuda").int()
    table = torch.zeros(B * W, cols, dtype=torch.int32, device="cuda")
    at = 0
    for b in range(B):
        table[b * W:b * W + W, :shared[b]] = order[at:at + shared[b]]
        at += shared[b]
        table[b * W:b * W + W, shared[b]:shared[b] + each[b]] = order[at:at + W * each[b]].view(W, each[b])
        at += W * each[b]
    s["table"], s["lens"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
    s["pools"] = [_random_pool(case, pages, normal) for _ in range(case.get("layers", 1))]
    s["nsum"] = torch.tensor(shared, dtype=torch.int32, device="cuda").repeat_interleave(W).contiguous()
    if case["op"] == "move":
        s["parents"] = torch.tensor(_parents(case), dtype=torch.int32, device="cuda").view(B, W)
        n = [x % P for x in lens]
        s["total"], s["max_new"] = sum(n), max(max(n), 1)
        s["cu"] = torch.tensor([0] + n, device="cuda").cumsum(0).int()
    else:
        s["q"] = (2.5 * normal(B * W, hq, D)).bfloat16()
        s["shared_pages"] = torch.tensor(shared, dtype=torch.int32, device="cuda")
    return s


def _handle(s):
    """What a serving program keeps: the runtimes of its layers' caches, the beams over them, the axes."""
    if "handle" not in s:
        from sparse_kv_page_rank_gb300 import locks
        from sparse_kv_page_rank_gb300.beams import LocksBeams
        from sparse_kv_page_rank_gb300.runtime import LocksRuntime

        case = s["case"]
        if case["op"] == "choose":
            s["handle"] = LocksBeams(width=case["beams"], device="cuda", end_token=s["end"])
            return s["handle"]
        nsum = s.get("nsum")
        if nsum is None:
            nsum = torch.zeros_like(s["lens"])
        rts = [LocksRuntime(k, v, s["table"], s["lens"], nsum, case["hq"], 2, 0) for k, v in s["pools"]]
        if case["op"] == "turn":
            s["handle"], s["axes"] = rts[0], locks.make_axes(_axes(case))
        else:
            s["handle"] = LocksBeams(rts, width=case["beams"])
    return s["handle"]


# ---- the plain forms -----------------------------------------------------------------


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
    g = x.unflatten(-1, (4, 32))
    s = (g.abs().amax(dim=-1) / 7).half()
    q = (g / s.float()[..., None]).round().clamp(-7, 7).nan_to_num(0.0)
    return q.flatten(-2).to(torch.int8), s


def _places(s):
    """Of each new token: its sequence and its position there."""
    new = (s["cu"][1:] - s["cu"][:-1]).long()
    seq = torch.repeat_interleave(torch.arange(len(s["new"]), device="cuda"), new, output_size=s["total"])
    at = torch.arange(s["total"], device="cuda") - s["cu"][seq] + (s["lens"] - new)[seq]
    return seq, at


def _read(s, seq, at):
    """What the first pool holds for those tokens."""
    P = s["case"]["page"]
    page, slot = s["table"][seq, at // P].long(), at % P
    heads = torch.arange(s["case"]["hkv"], device="cuda")
    where = _where(P)[0][slot]
    k, v = _values_of(s["pools"][0][0][page[:, None, None], heads[None, :, None], where[:, None]], P)
    return k.bfloat16(), v.bfloat16()


def _turn(s):
    case = s["case"]
    hq, hkv, P, rot = case["hq"], case["hkv"], case["page"], case["rot"]
    seq, at = _places(s)
    q, k, v = s["qkv"].float().split([hq, hkv, hkv], dim=1)
    axis = torch.tensor(_axes(case), device="cuda")
    row, pair = s["positions"].long()[axis].T, torch.arange(rot // 2, device="cuda")
    cos, sin = s["rope"][row, pair][:, None], s["rope"][row, pair + rot // 2][:, None]
    q = _rotate(q, cos, sin, rot, case["pairs"]).bfloat16()
    k = _rotate(k, cos, sin, rot, case["pairs"]).bfloat16()
    page, slot = s["table"][seq, at // P].long(), at % P
    k_pool, v_pool = s["pools"][0]
    if case["fmt"] == "bf16":
        k_pool[page, :, slot], v_pool[page, :, slot] = k, v.bfloat16()
        return {"q": q, "k_pool": k_pool, "v_pool": v_pool}
    (kq, ks), (vq, vs) = _quantise(k.float()), _quantise(v)
    heads = torch.arange(hkv, device="cuda")
    k_pool[page[:, None, None], heads[None, :, None], _where(P)[0][slot][:, None]] = _bytes_of((kq, vq), (ks, vs), P)
    k, v = _read(s, seq, at)
    return {"q": q, "k": k, "v": v}


def _choose(s):
    case = s["case"]
    B, W, V, K = case["batch"], case["beams"], case["vocab"], case["keep"]
    x = s["logits"].float().view(B, W, V)
    top = x.amax(dim=-1, keepdim=True)
    lse = top.squeeze(-1).double() + (x - top).double().exp().sum(dim=-1).log()
    # the best of each beam: larger logits first, then lower tokens, as one number
    bits = torch.where(x == 0, 0.0, x).view(torch.int32)
    order = (torch.where(bits < 0, bits ^ 0x7fffffff, bits).long() << 32) - torch.arange(V, device="cuda")
    n = min(K, V)
    token = order.topk(n, dim=-1).indices
    logit = x.gather(-1, token)
    score = s["scores"][..., None].double() + (logit.double() - lse[..., None])
    score.masked_fill_(logit == float("-inf"), float("-inf"))
    over = s["ended"].bool()[..., None]
    score = torch.where(over, s["scores"][..., None].double(), score)
    score[..., 1:].masked_fill_(over, float("-inf"))
    token = torch.where(over, s["end"], token)
    flat = (token + torch.arange(W, device="cuda")[:, None] * V).flatten(1)
    score = score.flatten(1)
    by_index = flat.argsort(dim=1)
    flat, score = flat.gather(1, by_index), score.gather(1, by_index)
    best = score.sort(dim=1, descending=True, stable=True).indices[:, :K]
    flat, score = flat.gather(1, best), score.gather(1, best)
    none = score == float("-inf")
    parent, token = flat // V, flat % V
    ended = (s["ended"].gather(1, parent.clamp(max=W - 1)) != 0) | (token == s["end"])
    return {"scores": score.float(), "parents": parent.masked_fill(none, -1).int(), "tokens": token.masked_fill(none, -1).int(),
            "ended": (ended & ~none).int()}


def _move(s):
    case = s["case"]
    B, W, P, hkv = case["batch"], case["beams"], case["page"], case["hkv"]
    rows = B * W
    base = torch.arange(B, device="cuda")[:, None] * W
    child = torch.arange(W, device="cuda")
    parent = s["parents"].long()
    same = parent[:, :, None] == parent[:, None, :]
    first = ~(same & (child[None, :] < child[:, None])).any(dim=-1)  # the lowest child of its parent
    used = (parent[:, :, None] == child).any(dim=1)
    nth = (~first).cumsum(dim=1) - 1
    free = (used.long() * W + child).argsort(dim=1)  # rows without children first, in order
    owner = torch.where(first, parent, free.gather(1, nth.clamp(min=0)))
    parent, owner, copied = (parent + base).flatten(), (owner + base).flatten(), (~first).flatten()
    lens, nsum = s["lens"][parent], s["nsum"][parent]
    cols = s["table"].shape[1]
    split = lens // P
    column = torch.arange(cols, device="cuda")
    table = torch.where(column < split[:, None], s["table"][parent], s["table"][owner])
    n = lens % P
    copied &= n > 0
    src = s["table"][parent, split.clamp(max=cols - 1)].long()
    dst = s["table"][owner, split.clamp(max=cols - 1)].long()
    whole = -(-n // 16) * 16
    slot = torch.arange(P, device="cuda")
    take = (copied[:, None] & (slot < whole[:, None]))
    row, slot = take.nonzero(as_tuple=True)
    for k, v in s["pools"]:
        if v is None:
            heads, where = torch.arange(hkv, device="cuda")[None, :, None], _where(P)[0][slot][:, None]
            k[dst[row][:, None, None], heads, where] = k[src[row][:, None, None], heads, where]
        else:
            for pool in (k, v):
                pool[dst[row], :, slot] = pool[src[row], :, slot]
    s["table"].copy_(table)
    s["lens"].copy_(lens)
    s["nsum"].copy_(nsum)
    out = {"table": s["table"], "lens": s["lens"], "summarized": s["nsum"]}
    if s["pools"][0][1] is None:
        out["k"], out["v"] = _read(s, *_places(s))
    else:
        for i, (k, v) in enumerate(s["pools"]):
            out[f"k{i}"], out[f"v{i}"] = k, v
    return out


def _gather(s, tables):
    """Keys and values in 32 bits, [n, hkv, tokens, 128], of the physical pages [n, pages]."""
    P = s["case"]["page"]
    k, v = s["pools"][0]
    k, v = (k[tables].float(), v[tables].float()) if v is not None else _values_of(_tokens(k[tables], P), P)
    return k.transpose(1, 2).flatten(2, 3), v.transpose(1, 2).flatten(2, 3)


def _attend(s):
    case = s["case"]
    W, hq, hkv, P = case["beams"], case["hq"], case["hkv"], case["page"]
    g, table = hq // hkv, s["table"].long()
    out = torch.empty(len(s["new"]), hq, D, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(len(s["new"]), hq, device="cuda")
    for b, shared in enumerate(s["shared"]):
        mine = slice(b * W, b * W + W)
        q = s["q"][mine].float().view(W, hkv, g, D) / math.sqrt(D)
        last = max(-(-n // P) for n in s["new"][mine])
        k, v = _gather(s, table[b * W:b * W + 1, :shared])
        kt, vt = _gather(s, table[mine, shared:last])
        seen = torch.arange(shared * P, last * P, device="cuda") < s["lens"][mine][:, None]
        x = (q.transpose(0, 1).reshape(hkv, W * g, D) @ k[0].transpose(1, 2)).view(hkv, W, g, -1).transpose(0, 1)
        y = (q @ kt.transpose(2, 3)).masked_fill(~seen[:, None, None], float("-inf"))
        x = torch.cat([x, y], dim=-1)
        top = x.amax(dim=-1, keepdim=True)
        x = (x - top).exp()
        total = x.sum(dim=-1, keepdim=True)
        a, z = x.split([shared * P, x.shape[-1] - shared * P], dim=-1)
        o = (a.transpose(0, 1).reshape(hkv, W * g, -1) @ v[0]).view(hkv, W, g, D).transpose(0, 1)
        # places that are not seen may hold anything, so their values are left out and not only weighted with 0
        o = o + z @ vt.masked_fill(~seen[:, None, :, None], 0.0)
        out[mine] = (o / total).reshape(W, hq, D).bfloat16()
        lse[mine] = (top + total.log()).reshape(W, hq)
    return {"out": out, "lse": lse}


def run(state):
    s, case = state, state["case"]
    op = case["op"]
    if not own:
        return {"turn": _turn, "choose": _choose, "move": _move, "attend": _attend}[op](s)
    h = _handle(s)
    if op == "turn":
        hq, hkv = case["hq"], case["hkv"]
        q, k, v = s["qkv"].split([hq, hkv, hkv], dim=1)
        q = h.append(k, v, q, rope=s["rope"], interleaved=case["pairs"] == "next", positions=s["positions"], axes=s["axes"],
                     cu_tokens=s["cu"], max_tokens=s["max_new"])
        if case["fmt"] == "bf16":
            return {"q": q, "k_pool": s["pools"][0][0], "v_pool": s["pools"][0][1]}
        k, v = h.read_tokens(s["total"], cu_tokens=s["cu"], max_tokens=s["max_new"])
        return {"q": q, "k": k, "v": v}
    if op == "choose":
        scores, parents, tokens, ended = h.select(s["logits"], s["scores"], ended=s["ended"], keep=case["keep"])
        return {"scores": scores, "parents": parents, "tokens": tokens, "ended": ended}
    if op == "attend":
        out, lse = h.attend(s["q"], s["shared_pages"])
        return {"out": out, "lse": lse}
    h.reorder(s["parents"])
    out = {"table": s["table"], "lens": s["lens"], "summarized": h.runtimes[0].n_summarized}
    if s["pools"][0][1] is None:
        out["k"], out["v"] = h.runtimes[0].read_tokens(s["total"], cu_tokens=s["cu"], max_tokens=s["max_new"])
    else:
        for i, (k, v) in enumerate(s["pools"]):
            out[f"k{i}"], out[f"v{i}"] = k, v
    return out


# ---- the definitions in 64 bits ------------------------------------------------------


def _held(blocks, P):
    """[n, page * 144] bytes -> keys and values [n, page, 128] in 64 bits, place by place."""
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
        out.append(code * blocks.contiguous().view(torch.float16)[:, sc // 2].double())
    return out


def _sequence(s, pages, h, n):
    """Keys and values of one head in those pages, [n, 128] in 64 bits."""
    k, v = s["pools"][0]
    k, v = _held(k[pages, h], s["case"]["page"]) if v is None else (k[pages, h].double(), v[pages, h].double())
    return k.reshape(-1, D)[:n], v.reshape(-1, D)[:n]


def _exact_turn(case, s):
    hq, hkv, P, half = case["hq"], case["hkv"], case["page"], case["rot"] // 2
    x = s["qkv"].double()
    y = x[:, :hq + hkv].clone()
    for i, axis in enumerate(_axes(case)):
        a, b = (i, i + half) if case["pairs"] == "half" else (2 * i, 2 * i + 1)
        row = s["positions"][axis].long()
        turn = torch.complex(s["rope"][row, i].double(), s["rope"][row, i + half].double())[:, None]
        z = torch.complex(x[:, :hq + hkv, a], x[:, :hq + hkv, b]) * turn
        y[..., a], y[..., b] = z.real, z.imag
    k, v = y[:, hq:], x[:, hq + hkv:]
    if case["fmt"] == "q4":
        held = []
        for a in (k.bfloat16().double(), v):
            g = a.reshape(*a.shape[:2], 4, 32)
            scale = (g.abs().amax(dim=-1, keepdim=True) / 7).half().double()
            held.append((torch.where(scale > 0, (g / scale).round().clamp(-7, 7), 0.0) * scale).view(a.shape))
        return {"q": y[:, :hq], "k": held[0], "v": held[1]}
    pools = [x.double() for x in s["pools"][0]]
    first = 0
    for b, n in enumerate(s["new"]):
        i = 0
        while i < n:  # the tokens of one page together
            t = s["ctx"][b] - n + i
            m = min(P - t % P, n - i)
            page = int(s["table"][b, t // P])
            for pool, rows in zip(pools, (k, v)):
                pool[page, :, t % P:t % P + m] = rows[first + i:first + i + m].transpose(0, 1)
            i += m
        first += n
    return {"q": y[:, :hq], "k_pool": pools[0], "v_pool": pools[1]}


def _exact_choose(case, s):
    B, W, V, K = case["batch"], case["beams"], case["vocab"], case["keep"]
    out = {"scores": torch.full((B, K), float("-inf"), dtype=torch.float64, device="cuda")}
    for name in ("parents", "tokens"):
        out[name] = torch.full((B, K), -1, dtype=torch.int32, device="cuda")
    out["ended"] = torch.zeros(B, K, dtype=torch.int32, device="cuda")
    for b in range(B):
        x = s["logits"][b * W:b * W + W].double()
        logp = s["scores"][b].double()[:, None] + x.log_softmax(dim=-1)
        for w in range(W):
            if s["ended"][b, w]:
                logp[w] = float("-inf")
                logp[w, s["end"]] = s["scores"][b, w].double()
        value, index = logp.flatten().sort(descending=True, stable=True)
        n = min(K, int((value > float("-inf")).sum()))
        value, index = value[:n], index[:n]
        out["scores"][b, :n], out["parents"][b, :n], out["tokens"][b, :n] = value, (index // V).int(), (index % V).int()
        out["ended"][b, :n] = ((index % V == s["end"]) | (s["ended"][b][index // V] != 0)).int()
    return out


def _exact_move(case, s):
    W, P = case["beams"], case["page"]
    table, lens, nsum = s["table"].tolist(), s["lens"].tolist(), s["nsum"].tolist()
    if case["fmt"] == "q4":
        heads = [_held(s["pools"][0][0][:, h], P) for h in range(case["hkv"])]
        pools = [torch.stack([x[i] for x in heads], dim=1) for i in range(2)]
    else:
        pools = [x.double() for pair in s["pools"] for x in pair]
    new_table, new_lens, new_nsum = [], [], []
    for b in range(case["batch"]):
        mine = s["parents"][b].tolist()
        without = [w for w in range(W) if w not in mine]
        seen = set()
        for p in mine:
            row, n = list(table[b * W + p]), lens[b * W + p]
            if p in seen:
                j, other = n // P, table[b * W + without.pop(0)]
                if n % P:
                    m = (n % P + 15) // 16 * 16
                    for x in pools:
                        x[other[j], :, :m] = x[row[j], :, :m]
                row = row[:j] + other[j:]
            seen.add(p)
            new_table.append(row)
            new_lens.append(n)
            new_nsum.append(nsum[b * W + p])
    table, lens, nsum = (torch.tensor(x, dtype=torch.int32, device="cuda") for x in (new_table, new_lens, new_nsum))
    out = {"table": table, "lens": lens, "summarized": nsum}
    if case["fmt"] == "q4":
        rows = [[x[new_table[i][n // P], :, :n % P].transpose(0, 1) for i, n in enumerate(new_lens) if n % P] for x in pools]
        none = pools[0].new_zeros(0, case["hkv"], D)
        out["k"], out["v"] = (torch.cat([none] + r) for r in rows)
    else:
        for i in range(case["layers"]):
            out[f"k{i}"], out[f"v{i}"] = pools[2 * i], pools[2 * i + 1]
    return out


def _exact_attend(case, s):
    hq, hkv, P = case["hq"], case["hkv"], case["page"]
    q = s["q"].double()
    out = torch.empty(q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(q.shape[:2], dtype=torch.float64, device="cuda")
    g = hq // hkv
    for i, n in enumerate(s["new"]):
        pages = s["table"][i, :-(-n // P)].long()
        for h in range(hkv):
            k, v = _sequence(s, pages, h, n)
            x = q[i, h * g:(h + 1) * g] @ k.T / math.sqrt(D)
            lse[i, h * g:(h + 1) * g] = x.logsumexp(dim=-1)
            out[i, h * g:(h + 1) * g] = (x - x.logsumexp(dim=-1, keepdim=True)).exp() @ v
    return {"out": out, "lse": lse}


def exact(case, seed):
    s = prepare(case, seed)
    return {"turn": _exact_turn, "choose": _exact_choose, "move": _exact_move, "attend": _exact_attend}[case["op"]](case, s)

"""Cases and 64-bit references for the calls that write the cache, read 4-bit
pages and attend prompts.  The 4-bit layout is restated here place by place from
include/locks.h; nothing is shared with the library."""

from __future__ import annotations

import math

import torch

D = 128


def q4_places(P: int):
    """Byte and bit of every key and value code, and byte of every scale:
    (kb, kn, ks, vb, vn, vs), each [P][128]."""
    t = torch.arange(P)[:, None].expand(P, D)
    d = torch.arange(D)[None, :].expand(P, D)
    j, u = d // 32, t % 16
    bit = 4 * ((d % 8) // 2) + 16 * (d % 2)
    kb, kn = 64 * t + 16 * ((d % 32) // 8) + 4 * j + bit // 8, bit % 8
    ks = 64 * P + 8 * t + 2 * j
    vbit = 4 * (d % 4)
    vb = (72 * P + 1024 * (t // 16) + 512 * (u // 8) + 64 * ((d % 32) // 4) + 16 * ((u % 8) // 2) + 4 * j + 2 * (u % 2)
          + vbit // 8)
    vs = 136 * P + 128 * (t // 16) + 32 * ((u % 8) // 2) + 16 * (u // 8) + 4 * j + 2 * (u % 2)
    return kb, kn, ks, vb, vbit % 8, vs


def pack(kq, ks, vq, vs):
    """Codes int [..., P, 128] and half scales [..., P, 4] -> uint8 [..., 144 P] (CPU)."""
    P = kq.shape[-2]
    lead = kq.shape[:-2]
    n = math.prod(lead)
    out = torch.zeros(n, 144 * P, dtype=torch.int32)
    kb, kn, ksb, vb, vn, vsb = q4_places(P)
    for q, b, bits in ((kq, kb, kn), (vq, vb, vn)):
        v = (q.reshape(n, P * D).int() + 8) << bits.reshape(1, -1).int()
        out.scatter_add_(1, b.reshape(1, -1).expand(n, -1), v)
    for s, b in ((ks, ksb), (vs, vsb)):
        raw = s.half().reshape(n, P * 4).view(torch.int16).int() & 0xffff
        b = b[:, ::32].reshape(1, -1).expand(n, -1)
        out.scatter_add_(1, b, raw & 255)
        out.scatter_add_(1, b + 1, raw >> 8)
    return out.to(torch.uint8).reshape(*lead, 144 * P)


def unpack(blocks):
    """uint8 [..., 144 P] -> (kq, ks, vq, vs) as codes int32 [..., P, 128] and half scales [..., P, 4]."""
    lead, P = blocks.shape[:-1], blocks.shape[-1] // 144
    x = blocks.reshape(-1, 144 * P).to(torch.int32)
    kb, kn, ksb, vb, vn, vsb = (p.to(blocks.device) for p in q4_places(P))
    out = []
    for b, bits, sb in ((kb, kn, ksb), (vb, vn, vsb)):
        q = ((x[:, b.reshape(-1)] >> bits.reshape(1, -1).int()) & 15) - 8
        lo, hi = x[:, sb[:, ::32].reshape(-1)], x[:, sb[:, ::32].reshape(-1) + 1]
        s = (lo | hi << 8).to(torch.int16).view(torch.float16)
        out += [q.reshape(*lead, P, D), s.reshape(*lead, P, 4)]
    return out


def dequant64(blocks):
    kq, ks, vq, vs = unpack(blocks)
    return (kq.double() * ks.double().repeat_interleave(32, dim=-1),
            vq.double() * vs.double().repeat_interleave(32, dim=-1))


class Case:
    """A paged cache on the GPU with lengths `lens`, in either format, whose
    unwritten slots and unowned pages hold NaN (or codes with NaN scales)."""

    def __init__(self, lens, hq, hkv, P, fmt, seed, spare=2, extra_cols=1, spread=1.0, nsum=None):
        g = torch.Generator().manual_seed(seed)
        self.lens, self.hq, self.hkv, self.P, self.fmt = list(lens), hq, hkv, P, fmt
        B = len(lens)
        self.B = B
        cols = max(1, max(-(-n // P) for n in lens)) + extra_cols
        used = [-(-n // P) for n in lens]
        pages = sum(used) + spare
        perm = torch.randperm(pages, generator=g)
        table = torch.full((B, cols), -7, dtype=torch.int32)  # entries past a sequence are never read
        k = 0
        for b in range(B):
            table[b, :used[b]] = perm[k:k + used[b]].int()
            k += used[b]
        if fmt == "q4":
            codes = [(torch.randn(pages, hkv, P, D, generator=g) * 2.6).round().clamp(-7, 7) for _ in range(2)]
            scales = [(0.3 * spread * (0.5 * torch.randn(pages, hkv, P, 4, generator=g)).exp()).half() for _ in range(2)]
            free = self._unwritten(table, used, pages, P)
            for s in scales:
                s.masked_fill_(free[:, None, :, None], float("nan"))
            self.k = pack(codes[0], scales[0], codes[1], scales[1]).cuda()
            self.v = None
        else:
            k = torch.randn(pages, hkv, P, D, generator=g) * spread
            v = torch.randn(pages, hkv, P, D, generator=g) * spread
            free = self._unwritten(table, used, pages, P)
            for x in (k, v):
                x.masked_fill_(free[:, None, :, None], float("nan"))
            self.k, self.v = k.bfloat16().cuda(), v.bfloat16().cuda()
        self.table = table.cuda()
        self.seq = torch.tensor(self.lens, dtype=torch.int32).cuda()
        full = [n // P for n in lens] if nsum is None else list(nsum)
        self.nsum = torch.tensor(full, dtype=torch.int32).cuda()
        self.gen = g

    def _unwritten(self, table, used, pages, P):
        free = torch.ones(pages, P, dtype=torch.bool)
        for b, n in enumerate(self.lens):
            for j in range(used[b]):
                free[table[b, j].item(), :max(0, min(P, n - j * P))] = False
        return free

    def runtime(self, rank=2, budget=0):
        from sparse_kv_page_rank_gb300.runtime import LocksRuntime
        return LocksRuntime(self.k, self.v, self.table, self.seq, self.nsum, self.hq, rank, budget)

    def query(self, n, spread=2.0):
        return (torch.randn(n, self.hq, D, generator=self.gen) * spread).bfloat16().cuda()

    def kv64(self, b):
        """Keys and values [hkv][len][128] of sequence b in 64 bits."""
        n = self.lens[b]
        pages = self.table[b, :-(-n // self.P)].long()
        if self.fmt == "q4":
            k, v = dequant64(self.k[pages])
        else:
            k, v = self.k[pages].double(), self.v[pages].double()
        return [x.transpose(0, 1).reshape(self.hkv, -1, D)[:, :n] for x in (k, v)]

    def scale64(self, b):
        """Per key [hkv][len][128]: the scale of its group (4-bit pages), else 0."""
        k, _ = self.kv64(b)
        if self.fmt != "q4":
            return torch.zeros_like(k)
        n = self.lens[b]
        pages = self.table[b, :-(-n // self.P)].long()
        s = unpack(self.k[pages])[1].double().repeat_interleave(32, dim=-1)
        return s.transpose(0, 1).reshape(self.hkv, -1, D)[:, :n]


def attend64(q, k, v, hidden=None, ksc=None, scale=None):
    """One head in 64 bits: q [n][128], k, v [t][128], hidden [n][t] or None.
    Returns out, lse, and for the tolerances the mean |value| under the same
    weights and the sum of |q||k| (with 80 times the code's scale added, the
    offset that 4-bit codes carry through the product) per query, at its largest."""
    scale = 1 / math.sqrt(D) if scale is None else scale
    q = q.double()
    if k.shape[0] == 0:
        z = torch.zeros(q.shape[0], D, dtype=torch.float64, device=q.device)
        return z, torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device=q.device), z, z[:, 0], z[:, 0]
    x = q @ k.T * scale
    mag = q.abs() @ (k.abs() if ksc is None else k.abs() + 80 * ksc).T * scale
    plain = q.abs() @ k.abs().T * scale
    if hidden is not None:
        x = x.masked_fill(hidden, -math.inf)
        mag = mag.masked_fill(hidden, 0)
        plain = plain.masked_fill(hidden, 0)
        none = hidden.all(dim=1)
    else:
        none = torch.zeros(q.shape[0], dtype=torch.bool, device=q.device)
    lse = x.logsumexp(dim=1)
    w = (x - lse[:, None]).exp().masked_fill(none[:, None], 0)
    return w @ v, lse, w @ v.abs(), mag.amax(dim=1), plain.amax(dim=1)

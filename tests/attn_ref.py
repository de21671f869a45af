"""Plain 64-bit forms of the attention half's operators, for the tests."""
import math

import torch

EPS = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11, torch.float32: 2.0 ** -24}   # half a step, relative


def kv_offsets(d, n):
    """[n][5d/4] byte offsets in a page of one head: K codes, V codes (channel order, 2i in the low half of byte i),
    K (scale, minimum) pairs, V scales, V minima; written from the layout in include/maple_attn.h."""
    rows = []
    for p in range(n):
        r, blk = p % 16, n * d // 2 + (p // 16) * 8 * d
        u, z = (r % 8) // 2, r % 2 + 2 * (r // 8)
        o = []
        for w in range(d // 8):
            o += [p * d // 2 + ((w % 4) * (d // 32) + w // 4) * 4 + b for b in range(4)]
        for w in range(d // 8):
            at = (z // 2) * 512 + ((w // 2) * 4 + u) * 16 + (z % 2) * 8 + (w % 2) * 4 if d == 128 else (w * 4 + u) * 16 + z * 4
            o += [blk + at + b for b in range(4)]
        o += [n * d + p * (d // 32) * 4 + b for b in range(d // 32 * 4)]
        for plane in range(2):
            for g in range(d // 32):
                o += [n * d + n * (d // 32) * (4 + 2 * plane) + (g * n + p) * 2 + b for b in range(2)]
        rows.append(o)
    return torch.tensor(rows)


def quantise_kv(x):
    """The cache's bytes of K or V rows x [..., d], every step rounded as the cache's definition says (32 bits, fp16
    scale and minimum): codes [..., d], scale, minimum [..., d/32]."""
    g = x.float().clamp(-60000.0, 60000.0).unflatten(-1, (-1, 32))
    mn = g.amin(-1).half()
    span = g.amax(-1) - mn.float()
    sc = (span / torch.full_like(span, 15.0)).half()
    c = torch.round((g - mn.float()[..., None]) / sc.float()[..., None]).clamp(0, 15)
    c = torch.where(sc[..., None] > 0, c, torch.zeros_like(c))
    return c.flatten(-2).to(torch.uint8), sc, mn


def kv_record(k, v):
    """A token's bytes, in the order of kv_offsets' columns."""
    two = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731
    raw = lambda h: h.contiguous().view(torch.uint8)  # noqa: E731
    (kc, ks, km), (vc, vs, vm) = quantise_kv(k), quantise_kv(v)
    return torch.cat([two(kc), two(vc), raw(torch.stack([ks, km], -1).flatten(-2)), raw(vs), raw(vm)], -1)


def kv_values(rec, d):
    """The keys and values (float64) that token bytes stand for."""
    G = d // 32
    f = rec[..., d:].contiguous().view(torch.float16).double()
    out = []
    for c, s, m in ((rec[..., :d // 2], f[..., 0:2 * G:2], f[..., 1:2 * G:2]), (rec[..., d // 2:d], f[..., 2 * G:3 * G], f[..., 3 * G:])):
        code = torch.stack([c & 15, c >> 4], -1).flatten(-2).double()
        out.append(code * s.repeat_interleave(32, -1) + m.repeat_interleave(32, -1))
    return out


def fill_pages(pages, n, k, v, slots):
    """Write K and V rows [T][Hkv][d] to the slots of a cache tensor."""
    d, Hkv = k.shape[2], k.shape[1]
    at = kv_offsets(d, n).to(pages.device)[slots % n]
    pages[(slots // n)[:, None, None], torch.arange(Hkv, device=pages.device)[None, :, None], at[:, None, :]] = kv_record(k, v)


def read_pages(pages, n, slots, d):
    at = kv_offsets(d, n).to(pages.device)[slots % n]
    head = torch.arange(pages.shape[1], device=pages.device)[None, :, None]
    return kv_values(pages[(slots // n)[:, None, None], head, at[:, None, :]], d)


def attend(q, k, v, seen, scale):
    """One head in 64 bits: out, the sum of p |v| that bounds the roundings of p, lse; q [m][d], k, v [n][d], seen [m][n]."""
    q, k, v = q.double(), k.double(), v.double()
    v = torch.where(seen.any(0)[:, None], v, torch.zeros_like(v))   # (keys that nobody sees may hold anything)
    s = torch.where(seen, q @ torch.where(seen.any(0)[:, None], k, torch.zeros_like(k)).t() * scale, -math.inf)
    lse = torch.logsumexp(s, 1)
    p = torch.where(seen, torch.exp(s - torch.where(lse.isfinite(), lse, torch.zeros_like(lse))[:, None]), torch.zeros_like(s))
    return p @ v, p @ v.abs(), lse


def prompt(q, k, v, lq, lk, scale, window):
    """Packed sequences; returns out, bound, lse in 64 bits, rows of the sequences only."""
    H, Hkv = q.shape[1], k.shape[1]
    out, bound = (torch.zeros(q.shape, dtype=torch.float64, device=q.device) for _ in range(2))
    lse = torch.full(q.shape[:2], -math.inf, dtype=torch.float64, device=q.device)
    a = b = 0
    for m, n in zip(lq, lk):
        pos = torch.arange(m, device=q.device)[:, None] + n - m
        j = torch.arange(n, device=q.device)[None, :]
        seen = (j <= pos) & ((j > pos - window) if window else (j <= pos))
        for h in range(H):
            if m and n:
                g = h // (H // Hkv)
                out[a:a + m, h], bound[a:a + m, h], lse[a:a + m, h] = attend(q[a:a + m, h], k[b:b + n, g], v[b:b + n, g], seen, scale)
        a, b = a + m, b + n
    return out, bound, lse

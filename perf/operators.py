"""The attention half of a decoder layer: what its operators are measured on.

Operators (names as in the package):

  linear      y[t][n] = alpha[n] s[t] sum_k w[n][k] q[t][k]: rows quantised to int8 (absmax, one scale per token), times
              int8 weights with one scale per output channel, summed exactly in integers.
  norm_rope   RMS norm of every query and key head, the rotation by position in the same pass, and (with a cache) the
              4-bit codes of the new keys and values written to their pages; the cache is read back at the same slots.
  prompt      causal attention over whole prompts, packed sequences of different lengths, grouped heads, optional window.
  cached      attention of one new token per sequence over a paged cache of 4-bit keys and values.

The cache: pages uint8 [P][Hkv][page bytes].  A token and head holds, for K and for V, d codes of 4 bits and one (scale,
minimum) pair of fp16 per 32 channels; value = minimum + scale * code.  `layout` below is the byte map of a page.
"""
import math

import torch

own = False

BF16, FP16, FP32 = "bf16", "fp16", "fp32"
_T = {BF16: torch.bfloat16, FP16: torch.float16, FP32: torch.float32}


# ---------------------------------------------------------------- the cases
def listed():
    return [
        # the query/key/value projection (d_model 2048 -> 16 query and 2 key/value heads of 128) of one decode token
        dict(name="linear decode T1", op="linear", T=1, K=2048, N=2560, out=BF16, bias=False),
        # an output head over a 65536-word vocabulary, the largest decode batch
        dict(name="linear head T64", op="linear", T=64, K=2048, N=65536, out=FP32, bias=False),
        # the same projection over a prompt of 4096 tokens
        dict(name="linear prompt T4096", op="linear", T=4096, K=2048, N=2560, out=BF16, bias=False),
        # one decode token's heads, its key and value appended to the cache
        dict(name="norm_rope decode T1", op="norm_rope", T=1, H=16, Hkv=2, d=128, rot=128, type=BF16, inter=False, page=64, far=131072),
        # a prompt of 4096 tokens, appended
        dict(name="norm_rope prompt T4096", op="norm_rope", T=4096, H=16, Hkv=2, d=128, rot=128, type=BF16, inter=False, page=64, far=4096),
        # a long packed prompt without a cache: heads of 64, half of each rotated, neighbours as pairs
        dict(name="norm_rope packed T16384", op="norm_rope", T=16384, H=32, Hkv=4, d=64, rot=32, type=FP16, inter=True, page=0, far=1000000),
        # a few short prompts, one of a single token
        dict(name="prompt short", op="prompt", lens="37,1,90,64,13", prefix=0, H=16, Hkv=2, d=128, window=0, type=BF16),
        # a global layer's prompt
        dict(name="prompt causal 8192", op="prompt", lens="8192", prefix=0, H=16, Hkv=2, d=128, window=0, type=BF16),
        # a windowed layer (512 tokens) over packed prompts of different lengths
        dict(name="prompt window packed", op="prompt", lens="4096,1,777,2500,129,640", prefix=0, H=32, Hkv=4, d=64, window=512, type=FP16),
        # one sequence in a windowed layer: the latency of a decode step
        dict(name="cached window B1", op="cached", lens="1500", H=16, Hkv=2, d=128, window=512, page=64, type=BF16),
        # one long sequence in a global layer
        dict(name="cached long B1", op="cached", lens="131071", H=16, Hkv=2, d=128, window=0, page=64, type=BF16),
        # a batch of very different lengths in a global layer
        dict(name="cached ragged B64", op="cached", lens=",".join(str(1 + (i * 2654435761) % 32768) for i in range(64)),
             H=16, Hkv=2, d=128, window=0, page=16, type=BF16),
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _heads(rng):
    d = rng.choice([64, 128])
    Hkv = rng.choice([1, 2, 4])
    return Hkv * rng.choice([1, 4, 5, 8]), Hkv, d


def draw(rng):
    op = rng.choice(["linear", "norm_rope", "prompt", "cached"])
    if op == "linear":
        T = _log(rng, 1, 4096)
        K = 16 * _log(rng, 16, 256)
        N = _log(rng, 64, 65536 if T <= 64 else 5120)
        return dict(op=op, T=T, K=K, N=N, out=rng.choice([BF16, FP32]), bias=rng.random() < 0.5)
    H, Hkv, d = _heads(rng)
    ty = rng.choice([BF16, FP16])
    if op == "norm_rope":
        return dict(op=op, T=_log(rng, 1, 8192), H=H, Hkv=Hkv, d=d, rot=rng.choice([d // 2, d]), type=ty, inter=rng.random() < 0.5,
                    page=rng.choice([0, 16, 32, 64]), far=_log(rng, 10000, 1000000))
    window = rng.choice([0, 0, 512, 100])
    if op == "prompt":
        n = _log(rng, 1, 8)
        lens = [_log(rng, 1, 4096 if n <= 2 else 2048) for _ in range(n)]
        return dict(op=op, lens=",".join(map(str, lens)), prefix=rng.choice([0, 0, 333]), H=H, Hkv=Hkv, d=d, window=window, type=ty)
    n = _log(rng, 1, 64)
    lens = [_log(rng, 1, 16384 if n > 4 else 131072) for _ in range(n)]
    return dict(op=op, lens=",".join(map(str, lens)), H=H, Hkv=Hkv, d=d, window=window, page=rng.choice([16, 32, 64]), type=ty)


def _lens(case):
    return [int(v) for v in case["lens"].split(",")]


def _pairs(case):
    """Key/query pairs that are not masked, of one query head."""
    w, n = case["window"], 0
    for m in _lens(case):
        p = case["prefix"]
        if not w:
            n += m * p + m * (m + 1) // 2
        else:
            full = max(0, m - max(0, w - 1 - p))        # queries that see a whole window
            rest = m - full                             # query i of the others sees p + i + 1 keys
            n += full * w + rest * p + rest * (rest + 1) // 2
    return n


def work(case):
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        return {"bytes": 2 * T * K + N * K + 4 * N * (2 if case["bias"] else 1) + T * N * (4 if case["out"] == FP32 else 2),
                "flops": 2 * T * N * K}
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if op == "norm_rope":
        T = case["T"]
        b = 4 * T * (H + Hkv) * d + 8 * T + 8 * d + 4 * case["rot"]
        if case["page"]:
            b += 2 * T * Hkv * d + 8 * T + 2 * T * Hkv * (5 * d // 4) + 4 * T * Hkv * d   # values in, codes out, read back
        return {"bytes": b, "flops": 10 * T * (H + Hkv) * d}
    if op == "prompt":
        n = sum(_lens(case))
        keys = n + case["prefix"] * len(_lens(case))
        return {"bytes": 2 * d * (2 * n * H + 2 * keys * Hkv) + 4 * n * H, "flops": 4 * d * H * _pairs(case)}
    w = case["window"]
    keys = sum(min(m, w) if w else m for m in _lens(case))
    return {"bytes": keys * Hkv * (5 * d // 4) + 4 * len(_lens(case)) * H * d, "flops": 4 * d * H * keys}


# ---------------------------------------------------------------- the cache's layout
def layout(d, page):
    """[page][5d/4] byte offsets in a page of one head, in a token's own order: K codes (d/2 bytes, channels 2i and 2i+1 in
    byte i), V codes, the K groups' (scale, minimum) fp16 pairs, the V groups' scales, the V groups' minima."""
    G, half = d // 32, d // 2
    p = torch.arange(page)[:, None]
    w = torch.arange(d // 8)[None, :]                               # 4-byte words of 8 channels
    kw = p * half + ((w % 4) * G + w // 4) * 4
    r = p % 16
    t, slot = (r % 8) // 2, r % 2 + 2 * (r // 8)
    if d == 128:
        vw = (p // 16) * 1024 + (slot // 2) * 512 + ((w // 2) * 4 + t) * 16 + (slot % 2) * 8 + (w % 2) * 4
    else:
        vw = (p // 16) * 512 + (w * 4 + t) * 16 + slot * 4
    vw = vw + page * half
    byte = torch.arange(4)
    g = torch.arange(G)[None, :]
    two = torch.arange(2)
    ks = page * d + p * G * 4 + torch.arange(G * 4)[None, :]
    vs = page * d + page * G * 4 + (g * page + p) * 2
    vm = vs + page * G * 2
    return torch.cat([(kw[:, :, None] + byte).reshape(page, -1), (vw[:, :, None] + byte).reshape(page, -1), ks,
                      (vs[:, :, None] + two).reshape(page, -1), (vm[:, :, None] + two).reshape(page, -1)], 1)


def _quantise(x):
    """x [..., d] in fp32 -> codes uint8 [..., d], scale and minimum fp16 [..., d/32]."""
    g = x.clamp(-60000.0, 60000.0).unflatten(-1, (-1, 32))
    lo = g.amin(-1).half()
    span = g.amax(-1) - lo.float()
    s = (span / torch.full_like(span, 15.0)).half()
    c = torch.round((g - lo.float()[..., None]) / s.float()[..., None]).clamp(0.0, 15.0)
    c = torch.where(s[..., None] > 0, c, torch.zeros_like(c))
    return c.flatten(-2).to(torch.uint8), s, lo


def _record(kc, ks, km, vc, vs, vm):
    """A token's bytes in its own order, from codes and fp16 pairs."""
    two = lambda c: c[..., 0::2] | (c[..., 1::2] << 4)  # noqa: E731
    raw = lambda h: h.contiguous().view(torch.uint8)  # noqa: E731
    return torch.cat([two(kc), two(vc), raw(torch.stack([ks, km], -1).flatten(-2)), raw(vs), raw(vm)], -1)


def _values(rec, d):
    """The fp32 keys and values that a token's bytes stand for."""
    G, half = d // 32, d // 2
    kc, vc, sc = rec[..., :half], rec[..., half:d], rec[..., d:].contiguous().view(torch.float16).float()
    codes = lambda c: torch.stack([c & 15, c >> 4], -1).flatten(-2).float().unflatten(-1, (G, 32))  # noqa: E731
    k = codes(kc) * sc[..., 0:2 * G:2, None] + sc[..., 1:2 * G:2, None]
    v = codes(vc) * sc[..., 2 * G:3 * G, None] + sc[..., 3 * G:, None]
    return k.flatten(-2), v.flatten(-2)


# ---------------------------------------------------------------- inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    randn = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    op = case["op"]
    if op == "linear":
        T, K, N = case["T"], case["K"], case["N"]
        # int8 absmax codes of normal weights, as a converter leaves them: 127 is each row's largest
        w = randn(N, K)
        amax = w.abs().amax(1, keepdim=True)
        return dict(case=case, x=randn(T, K).bfloat16(), w=torch.round(w * (127.0 / amax)).to(torch.int8),
                    alpha=(amax[:, 0] / 127.0) * K ** -0.5, bias=randn(N) if case["bias"] else None)
    H, Hkv, d, ty = case["H"], case["Hkv"], case["d"], _T[case["type"]]
    dev = dict(device="cuda")
    if op == "norm_rope":
        T, page = case["T"], case["page"]
        st = dict(case=case, qkv=(2.0 * randn(T, (H + 2 * Hkv) * d)).to(ty), qw=1.0 + 0.1 * randn(d), kw=1.0 + 0.1 * randn(d),
                  inv_freq=10000.0 ** (-torch.arange(0, case["rot"], 2, dtype=torch.float64, **dev) / case["rot"]))
        first = torch.randint(0, max(1, case["far"] - T), (1,), generator=g, device="cuda")
        st["positions"] = first + torch.arange(T, **dev)
        if page:
            pages = (T + page - 1) // page + 3
            order = torch.randperm(pages, generator=g, device="cuda")
            at = torch.arange(T, **dev) + (5 if T + 5 <= pages * page else 0)
            st["slots"] = order[at // page] * page + at % page
            st["pages"] = torch.zeros(pages, Hkv, page * (5 * d // 4), dtype=torch.uint8, device="cuda")
            st["at"] = layout(d, page).cuda()
        return st
    lens = _lens(case)
    if op == "prompt":
        n, keys = sum(lens), [m + case["prefix"] for m in lens]
        cu = lambda v: torch.tensor([0] + v, **dev).cumsum(0).int()  # noqa: E731
        q, k, v = (randn(n, H, d).to(ty), randn(sum(keys), Hkv, d).to(ty), randn(sum(keys), Hkv, d).to(ty))
        return dict(case=case, q=q, k=k, v=v, cu_q=cu(lens), cu_k=cu(keys), max_q=max(lens), max_k=max(keys))
    page, B = case["page"], len(lens)
    per = [(m + page - 1) // page for m in lens]
    P = sum(per)
    at = layout(d, page).cuda()
    pages = torch.empty(P, Hkv, page * (5 * d // 4), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 24) // (page * Hkv * d))
    for a in range(0, P, step):
        n = min(step, P - a)
        k, v = _quantise(randn(n, Hkv, page, d)), _quantise(randn(n, Hkv, page, d))
        pages[a:a + n].view(n, Hkv, -1)[:, :, at.flatten()] = _record(*k, *v).flatten(2)
    order = torch.randperm(P, generator=g, device="cuda").int()
    table = torch.zeros(B, max(per), dtype=torch.int32, device="cuda")
    rows = torch.repeat_interleave(torch.arange(B), torch.tensor(per))
    cols = torch.cat([torch.arange(m) for m in per])
    table[rows.cuda(), cols.cuda()] = order
    return dict(case=case, q=randn(B, H, d).to(ty), pages=pages, table=table, lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), at=at)


# ---------------------------------------------------------------- one pass
def run(state):
    case = state["case"]
    op = case["op"]
    if own:
        import ternary_weight_moe_forward_b200 as tw
        if op == "linear":
            return tw.int8_linear(state["x"], state["w"], state["alpha"], bias=state["bias"], out_dtype=_T[case["out"]])
        if op == "norm_rope":
            H, Hkv, d = case["H"], case["Hkv"], case["d"]
            q, k, v = state["qkv"].view(-1, H + 2 * Hkv, d).split([H, Hkv, Hkv], 1)
            args = dict(q_weight=state["qw"], k_weight=state["kw"], interleaved=case["inter"])
            if not case["page"]:
                return tw.qk_norm_rope(q, k, state["positions"], state["inv_freq"], **args)
            qo, ko = tw.qk_norm_rope(q, k, state["positions"], state["inv_freq"], v=v, pages=state["pages"], slots=state["slots"], **args)
            return (qo, ko) + tw.kv_read(state["pages"], state["slots"], d, dtype=_T[case["type"]])
        if op == "prompt":
            return tw.prompt_attention(state["q"], state["k"], state["v"], state["cu_q"], state["cu_k"], state["max_q"],
                                       window=case["window"], return_lse=True)
        return tw.cached_attention(state["q"], state["pages"], state["table"], state["lens"], window=case["window"])
    return {"linear": _linear, "norm_rope": _norm_rope, "prompt": _prompt, "cached": _cached}[op](state, case)


def _linear(s, case):
    x, K = s["x"].float(), case["K"]
    amax = x.abs().amax(1, keepdim=True)
    q = torch.round(x * (torch.full_like(amax, 127.0) / amax)).clamp(-127.0, 127.0)
    q = torch.where(amax > 0, q, torch.zeros_like(q))
    w = s["w"].float()
    # sums of 1024 products of int8 values are exact in fp32; longer ones are joined in 64 bits
    if K <= 1024:
        acc = q @ w.t()
    else:
        pad = -K % 1024
        q, w = torch.nn.functional.pad(q, (0, pad)), torch.nn.functional.pad(w, (0, pad))
        blocks = torch.bmm(q.unflatten(1, (-1, 1024)).transpose(0, 1), w.unflatten(1, (-1, 1024)).permute(1, 2, 0))
        acc = blocks.sum(0, dtype=torch.float64).float()
    y = acc * (s["alpha"] * (amax / 127.0))
    if s["bias"] is not None:
        y = y + s["bias"]
    return y.to(_T[case["out"]])


def _rotate(x, cos, sin, inter):
    """x [T][h][rot] by the angles [T][rot/2]."""
    cos, sin = cos[:, None], sin[:, None]
    a, b = (x[..., 0::2], x[..., 1::2]) if inter else x.chunk(2, -1)
    a, b = a * cos - b * sin, b * cos + a * sin
    return torch.stack([a, b], -1).flatten(-2) if inter else torch.cat([a, b], -1)


def _norm_rope(s, case):
    H, Hkv, d, rot, ty = case["H"], case["Hkv"], case["d"], case["rot"], _T[case["type"]]
    q, k, v = s["qkv"].view(-1, H + 2 * Hkv, d).float().split([H, Hkv, Hkv], 1)
    ang = s["positions"].double()[:, None] * s["inv_freq"]       # far positions: 64 bits
    cos, sin = ang.cos().float(), ang.sin().float()
    out = []
    for x, w in ((q, s["qw"]), (k, s["kw"])):
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + 1e-6) * w
        out.append(torch.cat([_rotate(x[..., :rot], cos, sin, case["inter"]), x[..., rot:]], -1).to(ty))
    if not case["page"]:
        return tuple(out)
    page, at = s["slots"] // case["page"], s["at"][s["slots"] % case["page"]]                 # [T], [T][bytes]
    rec = _record(*_quantise(out[1].float()), *_quantise(v))                                  # [T][Hkv][bytes]
    head = torch.arange(Hkv, device="cuda")[None, :, None]
    s["pages"][page[:, None, None], head, at[:, None, :]] = rec
    kr, vr = _values(s["pages"][page[:, None, None], head, at[:, None, :]], d)
    return (*out, kr.to(ty), vr.to(ty))


def _prompt(s, case):
    H, Hkv, d, w, P = case["H"], case["Hkv"], case["d"], case["window"], case["prefix"]
    G, n, m = H // Hkv, s["max_q"], s["max_k"]
    cq, ck = s["cu_q"].long(), s["cu_k"].long()
    lq = cq[1:] - cq[:-1]
    i, j = torch.arange(n, device="cuda"), torch.arange(m, device="cuda")
    # the packed rows, padded to the longest sequence
    q = s["q"][(cq[:-1, None] + i).clamp(max=len(s["q"]) - 1)].float().unflatten(2, (Hkv, G))           # [B][n][Hkv][G][d]
    k = s["k"][(ck[:-1, None] + j).clamp(max=len(s["k"]) - 1)].float()                                   # [B][m][Hkv][d]
    v = s["v"][(ck[:-1, None] + j).clamp(max=len(s["k"]) - 1)].float()
    B = len(lq)
    q = q.permute(0, 2, 3, 1, 4).reshape(B, Hkv, G * n, d)
    scores = (q @ k.permute(0, 2, 3, 1)).view(B, Hkv, G, n, m).mul_(d ** -0.5)
    far = j[None, :] - (i[:, None] + P)                          # key position minus query position
    hide = (far > 0) | (far <= -w) if w else far > 0
    scores.masked_fill_(hide, -math.inf)                         # (keys of another sequence lie past the diagonal)
    top = scores.amax(-1, keepdim=True)
    p = scores.sub_(top).exp_()
    total = p.sum(-1, keepdim=True)
    out = (p.view(B, Hkv, G * n, m) @ v.permute(0, 2, 1, 3)).view(B, Hkv, G, n, d) / total
    lse = (top + total.log()).squeeze(-1)
    keep = i[None, :] < lq[:, None]                              # rows of the sequences themselves
    return out.permute(0, 3, 1, 2, 4).flatten(2, 3)[keep].to(_T[case["type"]]), lse.permute(0, 3, 1, 2).flatten(2, 3)[keep]


def _cached(s, case):
    H, Hkv, d, w = case["H"], case["Hkv"], case["d"], case["window"]
    rec = s["pages"][:, :, s["at"]]                              # [P][Hkv][page][bytes], each token in its own order
    k, v = _values(rec, d)
    B, n = s["table"].shape
    seq = lambda x: x[s["table"].long()].permute(0, 2, 1, 3, 4).flatten(2, 3)  # noqa: E731  [B][Hkv][positions][d]
    k, v = seq(k), seq(v)
    q = s["q"].float().view(B, Hkv, H // Hkv, d)
    scores = (q @ k.transpose(-1, -2)) * d ** -0.5
    j, m = torch.arange(k.shape[2], device="cuda"), s["lens"].long()[:, None]
    hide = j >= m
    if w:
        hide = hide | (j < m - w)
    scores.masked_fill_(hide[:, None, None], -math.inf)
    p = torch.exp(scores - scores.amax(-1, keepdim=True))
    out = (p @ v) / p.sum(-1, keepdim=True)
    return out.view(B, H, d).to(_T[case["type"]])


# ---------------------------------------------------------------- in 64 bits, from the definitions
def exact(case, seed):
    s = prepare(case, seed)
    op = case["op"]
    if op == "linear":
        x = s["x"].double()
        amax = x.abs().amax(1, keepdim=True)
        # the codes are whole numbers by definition: 127/amax and its product with x are each rounded once to 32 bits
        q = torch.round((x * (torch.full_like(amax, 127.0) / amax).float().double()).float().double())
        y = (q @ s["w"].double().t()) * s["alpha"].double() * (amax / 127.0)
        return y if s["bias"] is None else y + s["bias"].double()
    H, Hkv, d = case["H"], case["Hkv"], case["d"]
    if op == "norm_rope":
        x = s["qkv"].double().view(-1, H + 2 * Hkv, d)
        rot, half = case["rot"], case["rot"] // 2
        e = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * s["inv_freq"])[:, None]
        res = []
        for part, w in ((x[:, :H], s["qw"]), (x[:, H:H + Hkv], s["kw"])):
            part = part / (part.pow(2).sum(-1, keepdim=True) / d + 1e-6).sqrt() * w.double()
            first = torch.arange(0, rot, 2, device="cuda") if case["inter"] else torch.arange(half, device="cuda")
            second = first + (1 if case["inter"] else half)
            z = torch.complex(part[..., first], part[..., second]) * e
            part[..., first], part[..., second] = z.real, z.imag
            res.append(part)
        if not case["page"]:
            return tuple(res)
        for kv in (res[1].to(_T[case["type"]]).double(), x[:, H + Hkv:]):      # the cache holds the rounded keys
            grp = kv.reshape(len(kv), Hkv, d // 32, 32)
            lo = grp.amin(-1, keepdim=True).half().double()
            sc = ((grp.amax(-1, keepdim=True) - lo) / 15).half().double()
            res.append((lo + sc * torch.round((grp - lo) / sc).clamp(0, 15)).reshape(len(kv), Hkv, d))
        return tuple(res)
    G, w = H // Hkv, case["window"]
    lens = _lens(case)
    if op == "prompt":
        out, lse = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda"), torch.empty(s["q"].shape[:2], dtype=torch.float64, device="cuda")
        a = b = 0
        for m in lens:
            mk = m + case["prefix"]
            at = torch.arange(m, device="cuda")[:, None] + case["prefix"] - torch.arange(mk, device="cuda")[None, :]
            seen = (at >= 0) & ((at < w) if w else (at >= 0))
            for h in range(H):
                sc = s["q"][a:a + m, h].double() @ s["k"][b:b + mk, h // G].double().t() / math.sqrt(d)
                sc[~seen] = -math.inf
                lse[a:a + m, h] = sc.logsumexp(1)
                out[a:a + m, h] = torch.softmax(sc, 1) @ s["v"][b:b + mk, h // G].double()
            a, b = a + m, b + mk
        return out, lse
    out = torch.empty(s["q"].shape, dtype=torch.float64, device="cuda")
    page, half, G32 = case["page"], d // 2, d // 32
    at = s["at"]
    for b, m in enumerate(lens):
        lo = max(0, m - w) if w else 0
        first = lo // page
        pg = s["pages"][s["table"][b, first:(m + page - 1) // page].long()]
        for h in range(Hkv):
            by = pg[:, h][:, at].reshape(-1, 5 * d // 4)[lo - first * page:m - first * page]
            f = by[:, d:].contiguous().view(torch.float16).double()
            val = []
            for c, sc, mn in ((by[:, :half], f[:, 0:2 * G32:2], f[:, 1:2 * G32:2]), (by[:, half:d], f[:, 2 * G32:3 * G32], f[:, 3 * G32:])):
                code = torch.empty(len(by), d, dtype=torch.float64, device="cuda")
                code[:, 0::2], code[:, 1::2] = (c % 16).double(), (c // 16).double()
                val.append(code * sc.repeat_interleave(32, 1) + mn.repeat_interleave(32, 1))
            sc = s["q"][b, h * G:(h + 1) * G].double() @ val[0].t() / math.sqrt(d)
            out[b, h * G:(h + 1) * G] = torch.softmax(sc, 1) @ val[1]
    return out

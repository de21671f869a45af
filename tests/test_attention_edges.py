"""Calls of the attention half at the edges of what they document: tiles that follow one another in a CTA, values that are
not finite, batches without a token, weights far below the largest, memory that overlaps.  64-bit forms: attn_ref."""
import math

import pytest
import torch

import attn_ref as ref
import ternary_weight_moe_forward_b200 as tw

pytestmark = pytest.mark.gpu
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return lambda *s: torch.randn(*s, generator=g, device="cuda")


def ints(r, n, k):
    return torch.clamp(torch.round(r(n, k) * 40), -127, 127).to(torch.int8)


def linear_ref(x, w, alpha, bias=None, resid=None):
    """Codes, exact sums, and the roundings in the documented order: the result to the bit."""
    amax = x.float().abs().amax(1, keepdim=True)
    q = torch.round(x.float() * (torch.full_like(amax, 127.0) / amax)).clamp(-127, 127)
    q = torch.where(amax > 0, q, torch.zeros_like(q))
    acc = (q.double() @ w.double().t()).float()
    y = acc * (alpha * (amax / torch.full_like(amax, 127.0)))
    if bias is not None:
        y = y + bias
    return y if resid is None else resid + y


# Sizes that lead to tiles of 160, 192 and 224 columns, more of them than SMs: some or all warps of a CTA store an odd number
# of pieces of 32 columns per tile
@pytest.mark.parametrize("T,N", [(2048, 2560), (3431, 1288), (2000, 5120), (3431, 1648), (4096, 2560), (2000, 8192)])
@pytest.mark.parametrize("K", [16, 128, 256])
def test_linear_tiles_that_follow_one_another(T, N, K):
    r = gen(T + N + K)
    x, w, al = r(T, K).to(BF16), ints(r, N, K), r(N).abs() * 0.01
    want = linear_ref(x, w, al).to(BF16)
    for _ in range(20):
        assert torch.equal(tw.int8_linear(x, w, al, out_dtype=BF16), want)


@pytest.mark.parametrize("T", [1, 3, 8, 9, 16, 17, 100, 130, 300])
@pytest.mark.parametrize("K,N", [(256, 64), (2048, 40), (8192, 24)])
@pytest.mark.parametrize("normalise", [False, True])
def test_linear_rows_that_are_not_finite(T, K, N, normalise):
    """A NaN or an infinity anywhere in a row makes that row's outputs NaN, and no other row's."""
    r = gen(T + K + N)
    x, w, al, bias = 3 * r(T, K), ints(r, N, K), r(N), r(N)
    x = x if normalise else x.to(BF16)
    resid = r(T, N)
    want = tw.int8_linear(x, w, al, bias, resid, normalise=normalise)
    assert want.isfinite().all()
    for n, bad in enumerate((math.nan, -math.nan, math.inf, -math.inf)):
        for at in (0, 31, 255, K - 1):
            row = (3 * n + at) % T
            y = x.clone()
            y[row, at] = bad
            got = tw.int8_linear(y, w, al, bias, resid, normalise=normalise)
            assert got[row].isnan().all()
            keep = torch.arange(T, device="cuda") != row
            assert torch.equal(got[keep], want[keep])
    y = x.clone()
    y[:, 1], y[:, 2] = math.nan, math.inf
    assert tw.int8_linear(y, w, al, normalise=normalise, out_dtype=BF16).isnan().all()


@pytest.mark.parametrize("T", [2, 40])
def test_linear_norm_beyond_fp32(T):
    """A row whose squares do not fit fp32 has no norm; rows of zeros, and of values whose squares vanish, have one."""
    r = gen(T)
    x, w, al = r(T, 512), ints(r, 33, 512), r(33)
    x[0] = 1e30
    x[1] = 0
    got = tw.int8_linear(x, w, al, normalise=True)
    assert got[0].isnan().all() and (got[1] == 0).all() and got[2:].isfinite().all()
    x[1] = 1e-30
    assert (tw.int8_linear(x, w, al, normalise=True)[1].abs() <= 1e-20).all()


def test_a_token_that_is_not_finite_stays_so_in_the_layer():
    """A NaN in one token's residual: its own row, and the later rows of its sequence, are NaN; another sequence is not."""
    from ternary_weight_moe_forward_b200 import synth
    attn = tw.AttentionLayer(256, 4, 2, 64, synth.attention_weights(256, 4, 2, 64, 5), 4, page_size=16)
    lens, s = [12, 9], torch.arange(21, device="cuda") + torch.cat([torch.zeros(12), torch.full((9,), 4.0)]).long().cuda()
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    c = torch.tensor([0, 12, 21], dtype=torch.int32, device="cuda")
    base = gen(8)(21, 256)
    want = attn.prompt(base.clone(), pos, s, c, 12)
    base[5, 17] = math.nan
    got = attn.prompt(base.clone(), pos, s, c, 12)
    assert torch.equal(got[:5], want[:5]) and torch.equal(got[12:], want[12:]) and got[5:12].isnan().all()


@pytest.mark.parametrize("H,Hkv,d,n", [(16, 2, 128, 64), (5, 1, 64, 16)])
def test_cached_batch_without_a_token(H, Hkv, d, n):
    """No sequence has a token, on a block table wide enough for two kernels: zeros, and the next kernel sees them."""
    pages = tw.kv_pages(4, Hkv, d, n)
    pages.fill_(0xFF)
    for B in (1, 3, 200, 2000):
        table = torch.zeros(B, 4096, dtype=torch.int32, device="cuda")
        q = gen(B)(B, H, d).to(BF16)
        for lens in (torch.zeros(B, dtype=torch.int32, device="cuda"), torch.full((B,), -5, dtype=torch.int32, device="cuda")):
            for _ in range(10):
                junk = torch.full((B, H, d), 7.0, dtype=BF16, device="cuda")   # (its memory is the next output's)
                del junk
                assert torch.count_nonzero(tw.cached_attention(q, pages, table, lens) * 1.0).item() == 0


@pytest.mark.parametrize("dt", [FP16, BF16])
@pytest.mark.parametrize("n", [300, 4096, 65536])
@pytest.mark.parametrize("gap", [14.3, 19.7, 23.4])
@pytest.mark.parametrize("peak", [0, -1])
def test_prompt_weights_far_below_the_largest(dt, n, gap, peak):
    """One key 2^gap above all others, with a value of zero: the output is the others' share.  A weight is off by half a step
    of its type, relative; of fp16 at least by half of the smallest step, 2^-25, where the largest weight is 2^7 or more:
    2^-32 of the sum for each of n keys, times the values (1 here)."""
    d, H = 64, 2
    q, k, v = torch.zeros(3, H, d, device="cuda"), torch.zeros(n, 1, d, device="cuda"), torch.ones(n, 1, d, device="cuda")
    q[..., 0] = 1
    q[:, 1, 0] = 0.5
    at = n - 3 if peak < 0 else 0                     # (the last of the keys that all three queries see)
    k[at, 0, 0], v[at] = gap * math.log(2), 0
    q, k, v = q.to(dt), k.to(dt), v.to(dt)
    cu = lambda m: torch.tensor([0, m], dtype=torch.int32, device="cuda")  # noqa: E731
    out, lse = tw.prompt_attention(q, k, v, cu(3), cu(n), 3, scale=1.0, return_lse=True)
    want, bound, wlse = ref.prompt(q, k, v, [3], [n], 1.0, 0)
    tol = ref.EPS[dt] * (1 + 2.0 ** -6) * (want.abs() + bound) + 2.0 ** -13 * bound + n * 2.0 ** -32
    assert ((out.double() - want).abs() <= tol).all()
    assert ((lse.double() - wlse).abs() <= 2.0 ** -13 + 2.0 ** -22 * wlse.abs()).all()


@pytest.mark.parametrize("Hkv,d,n", [(1, 64, 16), (2, 128, 64), (1, 128, 32)])
def test_cached_scores_keep_32_bits(Hkv, d, n):
    """Queries of 1 in the even channels, 2^-4 or 2^-4 + 2^-14 in the odd ones; keys of codes 0..15 in steps of 1/8 (minimum
    0), the even channels alike in all keys, the odd ones permuted: the scores, sums of at most 2^7 in steps of 2^-17,
    have an exact value in 32 bits.  They are scaled far up, so that the weights show their last bits: scale |q.k| is
    rounded twice on its way into the exponential (2^-24 of it each), and a weight counts twice (numerator and sum)."""
    r, scale, H = gen(d + n), 8192.0, 8 * Hkv
    lens = [2 + b % 4 for b in range(64)]
    pages, table = tw.kv_pages(64, Hkv, d, n), torch.arange(64, dtype=torch.int32, device="cuda")[:, None]
    codes = torch.arange(16, device="cuda") / 8
    kv = []
    for b, m in enumerate(lens):
        odd = torch.stack([codes[torch.argsort(r(16))] for _ in range(m * Hkv * d // 32)]).view(m, Hkv, d // 2)
        k = torch.stack([codes.repeat(d // 32).expand(m, Hkv, d // 2), odd], -1).flatten(-2)
        slots = b * n + torch.arange(m, device="cuda")
        ref.fill_pages(pages, n, k, r(m, Hkv, d), slots)
        kv.append(ref.read_pages(pages, n, slots, d))
        assert torch.equal(kv[b][0], k.double())
    q = torch.ones(64, H, d)
    q[..., 1::2] = 2.0 ** -4 + 2.0 ** -14 * torch.randint(0, 2, (64, H, d // 2), generator=torch.Generator().manual_seed(d))
    q = q.cuda().to(FP16)
    out = tw.cached_attention(q, pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), scale=scale)
    for b, m in enumerate(lens):
        k, v = kv[b]
        for h in range(H):
            want, bound, _ = ref.attend(q[b, h:h + 1], k[:, h // 8], v[:, h // 8], torch.ones(1, m, dtype=torch.bool, device="cuda"), scale)
            top = (k[:, h // 8] @ q[b, h].double()).max() * scale
            tol = ref.EPS[FP16] * (1 + 2.0 ** -6) * want.abs() + (2.0 ** -11 + 2.0 ** -13 + 4 * 2.0 ** -24 * top) * bound + 2.0 ** -24
            err = (out[b, h].double() - want[0]).abs()
            assert (err <= tol[0]).all(), (b, h, (err / tol[0]).max().item())


def test_parameters_serve_without_gradients():
    """Tensors that require a gradient: refused, unless gradients are off; a layer takes its weights without."""
    x, w = torch.ones(2, 256, dtype=BF16, device="cuda"), torch.ones(8, 256, dtype=torch.int8, device="cuda")
    al = torch.nn.Parameter(torch.ones(8, device="cuda"))
    with pytest.raises(ValueError, match="no gradients"):
        tw.int8_linear(x, w, al)
    for off in (torch.no_grad, torch.inference_mode):
        with off():
            assert (tw.int8_linear(x, w, al) == 256).all()
    from ternary_weight_moe_forward_b200 import synth
    weights = synth.attention_weights(256, 4, 2, 64, 5)
    weights["q_norm"] = torch.nn.Parameter(torch.from_numpy(weights["q_norm"]))
    attn = tw.AttentionLayer(256, 4, 2, 64, weights, 4, page_size=16)
    i = torch.arange(4, device="cuda")
    r = attn.prompt(gen(1)(4, 256), i, i, torch.tensor([0, 4], dtype=torch.int32, device="cuda"), 4)
    assert r.isfinite().all() and not r.requires_grad


def test_out_that_reaches_into_what_is_read():
    """An output anywhere in memory that the call reads is refused; the residual itself and neighbours are not."""
    mem = torch.ones(40, 256, device="cuda")
    w, al = torch.ones(256, 256, dtype=torch.int8, device="cuda"), torch.ones(256, device="cuda")
    x = mem[:8]
    with pytest.raises(ValueError, match="x must not be out"):
        tw.int8_linear(x, w, al, normalise=True, out=mem[7:15])
    with pytest.raises(ValueError, match="resid must be out"):
        tw.int8_linear(x, w, al, normalise=True, resid=mem[8:16], out=mem[15:23])
    with pytest.raises(ValueError, match="resid must be out"):
        tw.int8_linear(x, w, al, normalise=True, resid=mem[8:16], out=mem[8:12].view(BF16).view(8, 256))
    with pytest.raises(ValueError, match="weight, alpha or bias"):
        tw.int8_linear(x, w, mem[20], normalise=True, out=mem[16:24])
    want = tw.int8_linear(x, w, al, normalise=True, resid=mem[8:16])
    assert torch.equal(tw.int8_linear(x, w, al, normalise=True, resid=mem[8:16], out=mem[8:16]), want)
    assert torch.equal(tw.int8_linear(x, w, al, normalise=True, resid=mem[24:32], out=mem[16:24]), want)
    mem = torch.ones(60, 2, 64, dtype=FP16, device="cuda")
    q, k, v = mem[:10], mem[10:20], mem[20:30]
    c = torch.tensor([0, 10], dtype=torch.int32, device="cuda")
    for a in (1, 9, 11, 19, 29):
        with pytest.raises(ValueError, match="out must not be"):
            tw.prompt_attention(q, k, v, c, c, 10, out=mem[a:a + 10])
    assert (tw.prompt_attention(q, k, v, c, c, 10, out=mem[30:40]) == 1).all()


def test_numbers_that_do_not_fit():
    """Numbers beyond the fields of the C arguments are refused like other wrong arguments."""
    h = torch.ones(2, 1, 64, dtype=FP16, device="cuda")
    c, pages = torch.tensor([0, 2], dtype=torch.int32, device="cuda"), tw.kv_pages(1, 1, 64, 16)
    pos, f = torch.arange(2, device="cuda"), torch.zeros(0, dtype=torch.float64, device="cuda")
    for call in (lambda: tw.prompt_attention(h, h, h, c, c, 2, window=1 << 31), lambda: tw.prompt_attention(h, h, h, c, c, 1 << 40),
                 lambda: tw.prompt_attention(h, h, h, c, c, 2, scale=1e39), lambda: tw.prompt_attention(h, h, h, c, c, 2.0),
                 lambda: tw.cached_attention(h, pages, c[:, None], c, window=1 << 32),
                 lambda: tw.cached_attention(h, pages, c[:, None], c, scale=-1e300),
                 lambda: tw.qk_norm_rope(h, h, pos, f, eps=1e200)):
        with pytest.raises(ValueError, match="does not fit"):
            call()
    for scale in (math.inf, math.nan):
        with pytest.raises(tw.MapleError):
            tw.prompt_attention(h, h, h, c, c, 2, scale=scale)
    # the widest window is no window
    assert torch.equal(tw.prompt_attention(h, h, h, c, c, 2, window=(1 << 31) - 1), tw.prompt_attention(h, h, h, c, c, 2))
    assert torch.equal(tw.cached_attention(h, pages, c[:, None] * 0, c, window=(1 << 31) - 1),
                       tw.cached_attention(h, pages, c[:, None] * 0, c))


def test_linear_without_scales_is_refused():
    x, w = torch.ones(2, 64, dtype=BF16, device="cuda"), torch.ones(8, 64, dtype=torch.int8, device="cuda")
    with pytest.raises(tw.MapleError):
        tw.int8_linear(x, w, None)

"""The attention half's operators on the GPU against plain 64-bit forms (attn_ref).

Tolerances.  h(T) is half a step of type T relative to the value (attn_ref.EPS).  An output rounded once is off by
h |value|.  Attention: the weights p are rounded to the inputs' type (h(T)) before they meet the values (prompt), or to
fp16 and the values too (cached), which the sum A = sum p |v| / sum p bounds; a score sums d products in 32 bits, off by at
most d 2^-24 sum |q_i k_i| scale, below 2^-14 here (d = 128, |scaled sum| < 8), and enters p twice (numerator and sum) with
the 32-bit exponential (2^-22): 2^-13 A in all, with room for the accumulation of the products in 32 bits.
"""
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


def flag():
    return torch.zeros(1, dtype=torch.int32, device="cuda")


# ---------------------------------------------------------------- int8 linear
def linear_ref(x, w, alpha, bias=None, resid=None):
    """Codes, exact sums, and the roundings in the documented order: the result to the bit."""
    amax = x.float().abs().amax(1, keepdim=True)
    q = torch.round(x.float() * (torch.full_like(amax, 127.0) / amax)).clamp(-127, 127)
    q = torch.where(amax > 0, q, torch.zeros_like(q))
    acc = (q.double() @ w.double().t()).float()      # (an integer below 2^53: one rounding)
    y = acc * (alpha * (amax / torch.full_like(amax, 127.0)))
    if bias is not None:
        y = y + bias
    return y if resid is None else resid + y


@pytest.mark.parametrize("T,K,N", [(1, 16, 1), (1, 2048, 2560), (2, 48, 7), (3, 272, 130), (8, 2048, 257), (16, 1040, 64), (17, 256, 333),
                                   (33, 4096, 40), (64, 512, 1000), (65, 128, 128), (130, 2048, 515), (257, 1040, 2560), (1000, 336, 96),
                                   (5, 32768, 24), (300, 32768, 20), (2000, 1040, 4100), (4096, 512, 2560)])
@pytest.mark.parametrize("dt", [BF16, FP32])
def test_linear(T, K, N, dt):
    r = gen(T * 7 + K + N)
    x, w = r(T, K).to(BF16), torch.clamp(torch.round(r(N, K) * 40), -128, 127).to(torch.int8)
    alpha, bias, resid = r(N).abs() * 0.01, r(N), r(T, N)
    if T > 2:
        x[1] = 0
    for b, s in ((None, None), (bias, None), (bias, resid)):
        want = linear_ref(x, w, alpha, b, s).to(dt)
        assert torch.equal(tw.int8_linear(x, w, alpha, b, s, out_dtype=dt), want)


def test_linear_extreme_codes_strided_rows_and_in_place():
    # every product at its largest: 127 * 128 * 32768 does not fit fp32's integers, the sums must be exact
    x = torch.ones(70, 32768, device="cuda").to(BF16)
    w = torch.full((33, 32768), -128, dtype=torch.int8, device="cuda")
    al = torch.full((33,), 0.5, device="cuda")
    for T in (1, 9, 70):
        assert torch.equal(tw.int8_linear(x[:T], w, al), linear_ref(x[:T], w, al))
    r = gen(3)
    wide = r(40, 1024).to(BF16)
    x = wide[:, 512:768]
    w = torch.clamp(torch.round(r(64, 256) * 40), -127, 127).to(torch.int8)
    al, resid = r(64), r(40, 64)
    want = linear_ref(x, w, al, None, resid)
    got = tw.int8_linear(x, w, al, resid=resid, out=resid)
    assert got.data_ptr() == resid.data_ptr() and torch.equal(got, want)
    assert tw.int8_linear(x[:0], w, al).shape == (0, 64)


@pytest.mark.parametrize("T,K", [(1, 2048), (9, 256), (100, 2048), (3, 8192), (2, 32768), (16, 2048), (17, 2048)])
def test_linear_normalise(T, K):
    """The normed form quantises bf16(x / rms): off by one rounding of the norm at most, so one code in a while."""
    r = gen(T + K)
    x, w = 3 * r(T, K), torch.clamp(torch.round(r(96, K) * 40), -127, 127).to(torch.int8)
    al = r(96).abs()
    xn = (x.double() / (x.double().square().mean(1, keepdim=True) + 1e-6).sqrt()).to(BF16)
    got, want = tw.int8_linear(x, w, al, normalise=True), linear_ref(xn, w, al)
    # a bf16 value next to a rounding border may fall the other way (a step of 2^-8 of it, at most 1 code and its
    # neighbour): under 2^-12 of the values, each moving a sum by at most 2 codes of 127 * 127 per product
    amax = xn.float().abs().amax(1, keepdim=True)
    most = 2.0 * 127 * max(1.0, K * 2.0 ** -12) * al * (amax / 127)
    assert ((got - want).abs() <= most).all()
    assert (got == want).float().mean() > 0.5 or K > 8192


def test_linear_normalise_is_the_same_for_few_and_many_tokens():
    """The norm inside the kernel for few tokens and the one of its own for many give the same codes, so the same bits."""
    r = gen(77)
    x, w, al = 3 * r(40, 2048), torch.clamp(torch.round(r(200, 2048) * 40), -127, 127).to(torch.int8), r(200)
    x[5] = 0
    many = tw.int8_linear(x, w, al, normalise=True)
    for a, b in ((0, 1), (3, 11), (0, 16), (24, 40)):
        assert torch.equal(tw.int8_linear(x[a:b], w, al, normalise=True), many[a:b])
    x, w = x[:, :1024].contiguous(), w[:, :1024].contiguous()       # narrow enough for 16 rows in one kernel
    many = tw.int8_linear(x, w, al, normalise=True)
    for a, b in ((0, 1), (3, 11), (0, 16), (24, 40)):
        assert torch.equal(tw.int8_linear(x[a:b], w, al, normalise=True), many[a:b])


def test_prompt_refuses_to_write_over_its_input():
    q, k, v = (torch.ones(4, 2, 64, dtype=torch.float16, device="cuda") for _ in range(3))
    for x in (q, k, v):
        with pytest.raises(ValueError, match="out must not be"):
            tw.prompt_attention(q, k, v, cu([4]), cu([4]), 4, out=x)


def test_linear_refuses_to_write_over_its_input():
    x = torch.ones(2, 256, device="cuda")
    w, al = torch.ones(256, 256, dtype=torch.int8, device="cuda"), torch.ones(256, device="cuda")
    with pytest.raises(ValueError, match="x must not be out"):
        tw.int8_linear(x, w, al, normalise=True, out=x)
    y = tw.int8_linear(x, w, al, resid=x, normalise=True)           # x may be read twice
    torch.testing.assert_close(y, x + tw.int8_linear(x, w, al, normalise=True), rtol=2.0 ** -23, atol=0)


# ---------------------------------------------------------------- norm, rotation, cache
def rope_ref(x, w, pos, inv_freq, inter, eps=1e-6):
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if w is not None:
        x = x * w.double()
    rot = 2 * len(inv_freq)
    z = pos.double()[:, None] * inv_freq
    i = torch.arange(0, rot, 2, device="cuda") if inter else torch.arange(rot // 2, device="cuda")
    j = i + (1 if inter else rot // 2)
    a, b = x[..., i].clone(), x[..., j].clone()
    c, s = z.cos()[:, None], z.sin()[:, None]
    x[..., i], x[..., j] = a * c - b * s, b * c + a * s
    size = x.abs()
    size[..., i] = size[..., j] = (a.abs() + b.abs())
    return x, size


def freqs(rot, base=10000.0):
    return base ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / max(rot, 1))


@pytest.mark.parametrize("d,rot,H,Hkv,T", [(128, 128, 16, 2, 1), (128, 64, 5, 1, 7), (64, 64, 8, 4, 33), (64, 32, 32, 4, 257),
                                           (128, 0, 3, 3, 2), (64, 16, 1, 1, 5), (128, 112, 40, 8, 19)])
@pytest.mark.parametrize("dt,inter", [(BF16, False), (FP16, True)])
def test_norm_rope_and_append(d, rot, H, Hkv, T, dt, inter):
    r = gen(d + T)
    qkv = (2 * r(T, H + 2 * Hkv, d)).to(dt)
    q, k, v = qkv.split([H, Hkv, Hkv], 1)
    pos = 1000003 * torch.arange(T, device="cuda") % 1048576
    inv, qw, kw = freqs(rot), 1 + 0.1 * r(d), (None if T == 7 else 1 + 0.1 * r(d))
    pages_n, n = T // 16 + 2, (16, 32, 64)[T % 3]
    pages = tw.kv_pages(pages_n, Hkv, d, n)
    pages.fill_(0xAB)
    before = pages.clone()
    slots = torch.randperm(pages_n * n, device="cuda")[:T]
    if T > 3:
        slots[2] = -1
    f = flag()
    qo, ko = tw.qk_norm_rope(q, k, pos, inv, qw, kw, interleaved=inter, v=v, pages=pages, slots=slots, flags=f)
    for x, w, got in ((q, qw, qo), (k, kw, ko)):
        want, size = rope_ref(x, w, pos, inv, inter)
        # norm: 12 additions, a square root, a division and two products (2^-20 in all); sine and cosine 2^-22 of the
        # pair; then one rounding to dt (fp16: half of its smallest step, 2^-25, at the least)
        tol = ref.EPS[dt] * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -19 * size + 2.0 ** -25
        assert ((got.double() - want).abs() <= tol).all()
    # the cache: to the bit what its definition gives for the rounded keys and the values; nothing else is touched
    ref.fill_pages(before, n, ko[slots >= 0], v[slots >= 0], slots[slots >= 0])
    assert torch.equal(pages, before)
    kr, vr = tw.kv_read(pages, slots, d, dtype=dt, flags=f)
    ke, ve = ref.read_pages(pages, n, slots.clamp(min=0), d)
    for got, want in ((kr, ke), (vr, ve)):
        want[slots < 0] = 0
        # minimum + scale * code: one rounding to 32 bits, one to dt
        assert ((got.double() - want).abs() <= (ref.EPS[dt] * (1 + 2.0 ** -6) + 2.0 ** -24) * want.abs() + 2.0 ** -25).all()
    assert f.item() == 0
    # without a cache the same heads come out
    q2, k2 = tw.qk_norm_rope(q, k, pos, inv, qw, kw, interleaved=inter)
    assert torch.equal(q2, qo) and torch.equal(k2, ko)


def test_far_positions_keep_their_angle():
    """Angles near 2^31 radians: the rotation is taken from 64 bits."""
    r = gen(5)
    q = r(64, 2, 128).to(FP16)
    pos = (torch.arange(64, device="cuda") * 33554393) % (1 << 31)
    qo, _ = tw.qk_norm_rope(q, q, pos, freqs(128))
    want, size = rope_ref(q, None, pos, freqs(128), False)
    # (the angle itself: 2^31 * 2^-52 in either form)
    assert ((qo.double() - want).abs() <= ref.EPS[FP16] * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -18 * size + 2.0 ** -25).all()
    neg, _ = tw.qk_norm_rope(q, q, -pos, freqs(128))
    want, size = rope_ref(q, None, -pos, freqs(128), False)
    assert ((neg.double() - want).abs() <= ref.EPS[FP16] * want.abs() * (1 + 2.0 ** -6) + 2.0 ** -18 * size + 2.0 ** -25).all()


def test_cache_of_special_values():
    """Constant groups, infinities (clamped), NaN (their 32 channels only), zeros, huge values."""
    d, n = 64, 16
    v = torch.zeros(6, 1, d, device="cuda")
    v[1] = 3.25
    v[2, 0, 5], v[2, 0, 6] = math.inf, -math.inf
    v[3, 0, 40] = math.nan
    v[4] = torch.linspace(-2, 2, d)
    v[5, 0, 0], v[5, 0, 33] = 3.0e38, 1e-7
    v = v.to(BF16)
    pages, slots = tw.kv_pages(1, 1, d, n), torch.arange(6, device="cuda")
    k = torch.ones_like(v)
    tw.qk_norm_rope(k, k, slots, freqs(0), v=v, pages=pages, slots=slots)
    _, got = tw.kv_read(pages, slots, d, dtype=FP16)
    got = got[:, 0].double()
    assert (got[0] == 0).all() and (got[1] == 3.25).all()
    assert got[2].isfinite().all() and got[2, 5] > 59000 and got[2, 6] < -59000 and (got[2, 32:] == 0).all()
    assert got[3, 32:].isnan().all() and (got[3, :32] == 0).all()
    step = (v[4, 0, 31].double() - v[4, 0, 0].double()) / 15
    assert ((got[4] - v[4, 0].double()).abs() <= step * 0.51).all()
    assert got[5].isfinite().all()


def test_bad_slots_are_skipped_and_flagged():
    r = gen(9)
    d, n = 128, 16
    x = r(4, 1, d).to(BF16)
    pages = tw.kv_pages(2, 1, d, n)
    f = flag()
    slots = torch.tensor([0, 32, -1, 1 << 40], device="cuda")
    tw.qk_norm_rope(x, x, slots * 0, freqs(d), v=x, pages=pages, slots=slots, flags=f)
    assert f.item() == tw.MAPLE_FLAG_BAD_INDEX
    want = torch.zeros_like(pages)
    ko = tw.qk_norm_rope(x, x, slots * 0, freqs(d))[1]
    ref.fill_pages(want, n, ko[:1], x[:1], slots[:1])
    assert torch.equal(pages, want)
    f.zero_()
    k, v = tw.kv_read(pages, slots, d, flags=f)
    assert f.item() == tw.MAPLE_FLAG_BAD_INDEX and (k[1:] == 0).all() and (v[1:] == 0).all()


# ---------------------------------------------------------------- prompt attention
def cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def check_prompt(got, lse, want, bound, wlse, dt):
    tol = ref.EPS[dt] * (1 + 2.0 ** -6) * (want.abs() + bound) + 2.0 ** -13 * bound + 2.0 ** -24
    assert ((got.double() - want).abs() <= tol).all()
    seen = wlse.isfinite()
    assert torch.equal(lse.isfinite(), seen) and (lse[~seen] == -math.inf).all() and (got[~seen] == 0).all()
    assert ((lse.double() - wlse)[seen].abs() <= 2.0 ** -13 + 2.0 ** -22 * wlse[seen].abs()).all()


CASES = [  # query rows, key rows per sequence, window
    ([1], [1], 0), ([1], [300], 0), ([2, 1, 3], [2, 1, 3], 0), ([128], [128], 0), ([129], [129], 0), ([37, 1, 90, 0, 64, 13], None, 0),
    ([300], [700], 0), ([5, 130, 1], [900, 130, 257], 100), ([600], [600], 1), ([513, 40], None, 512), ([260], [260], 7),
    ([50, 20], [10, 20], 0), ([40, 3], [0, 3], 0), ([1000], [1000], 0), ([33] * 40, None, 0), ([900, 400], [1100, 400], 129)]


@pytest.mark.parametrize("lq,lk,window", CASES)
@pytest.mark.parametrize("H,Hkv,d,dt", [(16, 2, 128, BF16), (4, 4, 64, FP16), (5, 1, 128, FP16), (12, 2, 64, BF16)])
def test_prompt(lq, lk, window, H, Hkv, d, dt):
    lk = lk or lq
    r = gen(sum(lq) + window + H)
    q, k, v = r(sum(lq), H, d).to(dt), r(sum(lk), Hkv, d).to(dt), r(sum(lk), Hkv, d).to(dt)
    f = flag()
    out, lse = tw.prompt_attention(q, k, v, cu(lq), cu(lk), max(lq), window=window, return_lse=True, flags=f)
    check_prompt(out, lse, *ref.prompt(q, k, v, lq, lk, d ** -0.5, window), dt)
    assert f.item() == 0


@pytest.mark.parametrize("G", [1, 2, 3, 7, 16, 24, 64])
def test_prompt_group_sizes(G):
    r = gen(G)
    lq, d, dt = [70, 9, 141], 64, BF16
    q, k, v = r(220, 2 * G, d).to(dt), r(220, 2, d).to(dt), r(220, 2, d).to(dt)
    out, lse = tw.prompt_attention(q, k, v, cu(lq), cu(lq), 141, return_lse=True)
    check_prompt(out, lse, *ref.prompt(q, k, v, lq, lq, d ** -0.5, 0), dt)


def test_prompt_views_scale_and_large_scores():
    """Heads taken out of one fused projection; scores far apart (the running maximum moves all the way)."""
    r = gen(11)
    H, Hkv, d, lens = 8, 2, 128, [333, 200]
    qkv = r(533, H + 2 * Hkv, d)
    qkv[:, H:H + Hkv] *= torch.linspace(0.1, 12, 533, device="cuda")[:, None, None]
    qkv = qkv.to(BF16)
    q, k, v = qkv.split([H, Hkv, Hkv], 1)
    for scale in (0.25, 0.01, -0.1):
        out, lse = tw.prompt_attention(q, k, v, cu(lens), cu(lens), 333, scale=scale, return_lse=True)
        want, bound, wlse = ref.prompt(q, k, v, lens, lens, scale, 0)
        # scores here reach |scale| d 12 in absolute sum: their 32-bit sums are off by 2^-24 d of that, twice
        extra = 2 * 128 * 2.0 ** -24 * abs(scale) * 128 * 12
        tol = ref.EPS[BF16] * (1 + 2.0 ** -6) * (want.abs() + bound) + (2.0 ** -13 + extra) * bound
        assert ((out.double() - want).abs() <= tol).all()
        assert ((lse.double() - wlse).abs() <= 2.0 ** -13 + extra + 2.0 ** -22 * wlse.abs()).all()


@pytest.mark.parametrize("window", [0, 60])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_prompt_what_is_masked_does_not_reach(window, dt):
    """NaN and infinities in rows behind the last sequence, in another sequence and at later positions of the same one."""
    r = gen(13)
    H, Hkv, d, lens = 4, 2, 64, [150, 75]
    n = sum(lens) + 40
    q, k, v = r(n, H, d).to(dt), r(n, Hkv, d).to(dt), r(n, Hkv, d).to(dt)
    k[225:], v[225:] = math.nan, math.inf
    q[225:] = math.nan
    out = torch.full((n, H, d), 7.0, device="cuda", dtype=dt)
    base = tw.prompt_attention(q, k, v, cu(lens), cu(lens), 150, window=window, out=out)
    want, bound, wlse = ref.prompt(q[:225], k[:225], v[:225], lens, lens, d ** -0.5, window)
    assert ((base[:225].double() - want).abs() <= (ref.EPS[dt] * (1 + 2.0 ** -6) * (want.abs() + bound) + 2.0 ** -13 * bound) + 2.0 ** -24).all()
    assert (out[225:] == 7.0).all()                     # rows behind the last sequence
    k2, v2 = k.clone(), v.clone()
    k2[100, 0], v2[100, 0], v2[120, 1, 3], v2[130, 1, 5] = math.nan, math.nan, math.inf, math.nan
    got = tw.prompt_attention(q, k2, v2, cu(lens), cu(lens), 150, window=window)
    G = H // Hkv
    last = 100 + window if window else 150
    sees = torch.zeros(n, dtype=torch.bool, device="cuda")
    sees[100:min(last, 150)] = True
    assert torch.equal(got[:225, :G][~sees[:225]], base[:225, :G][~sees[:225]])
    assert got[:225, :G][sees[:225]].isnan().all()
    g1, b1 = got[:225, G:], base[:225, G:]
    at = torch.arange(225, device="cuda")
    s3, s5 = (at >= 120) & (at < min(150, 120 + (window or 150))), (at >= 130) & (at < min(150, 130 + (window or 150)))
    assert (g1[s3][..., 3] == math.inf).all() and g1[s5][..., 5].isnan().all()
    rest = torch.ones(d, dtype=torch.bool, device="cuda")
    rest[3] = rest[5] = False
    assert torch.equal(g1[..., rest], b1[..., rest])
    assert torch.equal(g1[~s3][..., 3], b1[~s3][..., 3]) and torch.equal(g1[~s5][..., 5], b1[~s5][..., 5])


def test_prompt_many_short_sequences_and_none():
    """700 sequences of 0 to 5 tokens (more than one round of the search for a block's sequence); no keys at all."""
    lens = [(i * 7) % 6 for i in range(700)]
    r = gen(17)
    H, Hkv, d, n = 4, 2, 64, sum(lens)
    q, k, v = r(n, H, d).to(FP16), r(n, Hkv, d).to(FP16), r(n, Hkv, d).to(FP16)
    out, lse = tw.prompt_attention(q, k, v, cu(lens), cu(lens), 5, return_lse=True)
    check_prompt(out, lse, *ref.prompt(q, k, v, lens, lens, d ** -0.5, 0), FP16)
    out, lse = tw.prompt_attention(q[:40], k[:0], v[:0], cu([40]), cu([0]), 40, return_lse=True)
    assert (out == 0).all() and (lse == -math.inf).all()
    assert tw.prompt_attention(q[:0], k, v, cu([0]), cu([n]), 0).shape == (0, H, d)


def test_prompt_nan_among_the_keys_that_are_seen():
    """A NaN key makes the rows that see it NaN, an infinite one too, wherever it stands in a tile of 128 keys."""
    r = gen(19)
    d, n = 128, 300
    q, k, v = r(n, 2, d).to(BF16), r(n, 1, d).to(BF16), r(n, 1, d).to(BF16)
    base = tw.prompt_attention(q, k, v, cu([n]), cu([n]), n)
    for j in (0, 5, 64, 127, 128, 299):
        for bad in (math.nan, math.inf):
            k2 = k.clone()
            k2[j, 0, 7] = bad
            got = tw.prompt_attention(q, k2, v, cu([n]), cu([n]), n)
            assert torch.equal(got[:j], base[:j])
            hit = q[j:, :, 7].float() * bad
            gone = hit.isnan() | (hit == math.inf)           # (a score of -inf is a weight of 0)
            assert got[j:][gone].isnan().all()


def test_prompt_bad_offsets_are_cut_and_flagged():
    r = gen(15)
    d = 64
    q, k, v = r(100, 2, d).to(BF16), r(100, 1, d).to(BF16), r(100, 1, d).to(BF16)
    for cq, ck, mq in (([0, 50, 130], [0, 50, 130], 100), ([0, 60, 40], [0, 60, 40], 100), ([-5, 50, 100], [0, 50, 100], 100),
                       ([0, 50, 100], [0, 50, 100], 20)):
        f = flag()
        cqt, ckt = torch.tensor(cq, dtype=torch.int32, device="cuda"), torch.tensor(ck, dtype=torch.int32, device="cuda")
        out = tw.prompt_attention(q, k, v, cqt, ckt, mq, flags=f, out=torch.zeros(100, 2, d, device="cuda", dtype=BF16))
        torch.cuda.synchronize()
        assert f.item() == tw.MAPLE_FLAG_BAD_INDEX and out.isfinite().all()


# ---------------------------------------------------------------- cached attention
def make_cache(r, lens, Hkv, d, n, spare=3):
    per = [(m + n - 1) // n for m in lens]
    P = sum(per) + spare
    order = torch.randperm(P, device="cuda")[:sum(per)].int()
    table = torch.full((len(lens), max(per + [1])), -1, dtype=torch.int32, device="cuda")
    pages = tw.kv_pages(P, Hkv, d, n)
    pages.fill_(0xFF)                                  # fp16 0xFFFF is a NaN: rows that hold no token
    a, kv = 0, []
    for b, m in enumerate(lens):
        table[b, :per[b]] = order[a:a + per[b]]
        a += per[b]
        if m:
            j = torch.arange(m, device="cuda")
            slots = table[b].long()[j // n] * n + j % n
            ref.fill_pages(pages, n, r(m, Hkv, d), r(m, Hkv, d) + 0.5, slots)
            kv.append(ref.read_pages(pages, n, slots, d))
        else:
            kv.append((torch.zeros(0, Hkv, d, device="cuda"),) * 2)
    return pages, table, kv


def check_cached(out, q, kv, lens, scale, window, dt):
    B, H, d = q.shape
    for b, m in enumerate(lens):
        k, v = kv[b]
        Hkv = k.shape[1]
        seen = torch.ones(1, max(m, 0), dtype=torch.bool, device="cuda")
        if window:
            seen[:, :max(0, m - window)] = False
        for h in range(H):
            if m <= 0:
                assert (out[b, h] == 0).all()
                continue
            g = h // (H // Hkv)
            want, bound, _ = ref.attend(q[b, h:h + 1], k[:, g], v[:, g], seen, scale)
            tol = ref.EPS[dt] * (1 + 2.0 ** -6) * want.abs() + (2.0 ** -11 + 2.0 ** -13) * bound + 2.0 ** -24
            assert ((out[b, h].double() - want[0]).abs() <= tol[0]).all(), (b, h, m)


@pytest.mark.parametrize("lens,window", [([1], 0), ([64], 0), ([65, 0, 1, 63, 129], 0), ([1500], 512), ([511, 512, 513, 7], 512), ([3000, 17, 16], 1),
                                         ([20000, 5, 700], 0), ([255] * 40, 100), ([9000], 0)])
@pytest.mark.parametrize("H,Hkv,d,n,dt", [(16, 2, 128, 64, BF16), (16, 2, 128, 16, FP16), (4, 4, 64, 32, BF16), (5, 1, 64, 16, FP16),
                                          (24, 2, 128, 32, BF16)])
def test_cached(lens, window, H, Hkv, d, n, dt):
    r = gen(sum(lens) + H)
    pages, table, kv = make_cache(r, lens, Hkv, d, n)
    q = r(len(lens), H, d).to(dt)
    f = flag()
    out = tw.cached_attention(q, pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"), window=window, flags=f)
    check_cached(out, q, kv, lens, d ** -0.5, window, dt)
    assert f.item() == 0


def test_cached_many_short_and_some_long_sequences():
    """Shares of the line that hold many short segments, empty ones and cuts of long ones; the same bits every time."""
    lens = [[1, 70, 0, 200, 1, 3000, 64, 65][i % 8] + i % 3 for i in range(200)] + [15000, 1, 1, 1]
    r = gen(41)
    d, n = 64, 16
    pages, table, kv = make_cache(r, lens, 2, d, n)
    q, ln = r(len(lens), 8, d).to(BF16), torch.tensor(lens, dtype=torch.int32, device="cuda")
    out = tw.cached_attention(q, pages, table, ln)
    check_cached(out, q, kv, lens, d ** -0.5, 0, BF16)
    for _ in range(20):
        assert torch.equal(tw.cached_attention(q, pages, table, ln), out)


@pytest.mark.parametrize("G", [1, 3, 8, 9, 17, 40])
def test_cached_group_sizes(G):
    r = gen(G)
    lens, d, n = [300, 70], 128, 64
    pages, table, kv = make_cache(r, lens, 2, d, n)
    q = r(2, 2 * G, d).to(FP16)
    out = tw.cached_attention(q, pages, table, torch.tensor(lens, dtype=torch.int32, device="cuda"))
    check_cached(out, q, kv, lens, d ** -0.5, 0, FP16)


def test_cached_query_magnitudes():
    """Queries from 2^-20 to 2^12 in one head: the products keep 32-bit accuracy whatever the query's size."""
    r = gen(21)
    lens, d, n = [200], 128, 64
    pages, table, kv = make_cache(r, lens, 1, d, n)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for size in (2.0 ** -20, 2.0 ** -6, 1.0, 2.0 ** 12):
        q = (r(1, 8, d) * size).to(BF16)
        out = tw.cached_attention(q, pages, table, ln, scale=0.09 / size)
        check_cached(out, q, kv, lens, 0.09 / size, 0, BF16)
    out = tw.cached_attention(torch.zeros_like(q), pages, table, ln)
    check_cached(out, torch.zeros_like(q), kv, lens, d ** -0.5, 0, BF16)


def test_cached_nan_values_stay_in_their_channels():
    """A NaN key's token makes its sequence's rows NaN; a NaN value its own 32 channels; other sequences are untouched."""
    r = gen(29)
    d, n, lens = 128, 16, [50, 90]
    pages, table, kv = make_cache(r, lens, 1, d, n)
    q, ln = r(2, 4, d).to(BF16), torch.tensor(lens, dtype=torch.int32, device="cuda")
    base = tw.cached_attention(q, pages, table, ln)
    k = kv[0][0][20:21].float().to(BF16)
    vbad = kv[0][1][20:21].float().to(BF16)
    vbad[0, 0, 70] = math.nan
    slot = (table[0, 1].long() * n + 4)[None]
    ref.fill_pages(pages, n, k, torch.nan_to_num(vbad), slot)
    tw.qk_norm_rope(k, k, slot * 0, freqs(0), v=vbad, pages=pages, slots=slot)
    got = tw.cached_attention(q, pages, table, ln)
    assert torch.equal(got[1], base[1])
    assert got[0, :, 64:96].isnan().all() and got[0, :, :64].isfinite().all() and got[0, :, 96:].isfinite().all()
    window = tw.cached_attention(q, pages, table, ln, window=25)       # the NaN row is masked, in a tile that is read
    assert window.isfinite().all()


def test_cached_bad_pages_and_lengths():
    r = gen(23)
    d, n = 64, 16
    pages, table, kv = make_cache(r, [40, 40], 1, d, n)
    q = r(2, 2, d).to(BF16)
    f = flag()
    bad = table.clone()
    bad[0, 1] = 1 << 30
    out = tw.cached_attention(q, pages, bad, torch.tensor([40, 4000], dtype=torch.int32, device="cuda"), flags=f)
    # (sequence 1 is cut to the 48 rows of its table, of which the last 8 hold NaN: only that it is cut can be seen)
    assert f.item() == tw.MAPLE_FLAG_BAD_INDEX and out[0].isfinite().all()
    # sequence 0 without its rows 16..31
    keep = torch.ones(40, dtype=torch.bool, device="cuda")
    keep[16:32] = False
    check_cached(out[:1], q[:1], [(kv[0][0][keep], kv[0][1][keep])], [24], d ** -0.5, 0, BF16)
    f.zero_()
    tw.cached_attention(q, pages, table, torch.tensor([-3, 40], dtype=torch.int32, device="cuda"), flags=f)
    assert f.item() == 0


# ---------------------------------------------------------------- streams, graphs, determinism
def test_captured_and_on_another_stream():
    r = gen(31)
    lens, H, Hkv, d, n = [700, 90], 16, 2, 128, 64
    pages, table, kv = make_cache(r, lens, Hkv, d, n)
    ln = torch.tensor(lens, dtype=torch.int32, device="cuda")
    q, k, v = r(200, H, d).to(BF16), r(200, Hkv, d).to(BF16), r(200, Hkv, d).to(BF16)
    c = cu([120, 80])
    w, al = torch.clamp(torch.round(r(256, 2048) * 40), -127, 127).to(torch.int8), r(256)
    x = r(150, 2048).to(BF16)
    pos = torch.arange(200, device="cuda")
    inv = freqs(d)

    def once():
        return [tw.int8_linear(x, w, al), tw.int8_linear(x[:3], w, al), *tw.qk_norm_rope(q, k, pos, inv),
                *tw.prompt_attention(q, k, v, c, c, 120, return_lse=True), tw.cached_attention(q[:2], pages, table, ln)]
    want = once()
    again = once()
    assert all(torch.equal(a, b) for a, b in zip(want, again))       # the same bits every time
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = once()
    torch.cuda.current_stream().wait_stream(side)
    assert all(torch.equal(a, b) for a, b in zip(want, other))
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got = once()
        graphs.append((g, got))
    for g, got in graphs:
        for t in got:
            t.zero_()
    for g, _ in graphs:
        g.replay()
    torch.cuda.synchronize()
    for _, got in graphs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))

"""The decoder stack: the attention operators run together with the MoE layer, prompt and decode, as a user runs them.

The operators' accuracy is tested one by one elsewhere; here the sublayer is compared with a plain 64-bit form whose int8
codes are taken at the same places.  Bound of that comparison: a code may fall on the other side of a rounding border
where a bf16 value does, which moves it by one step of amax/127; if every code of the two quantised rows did, a row's
relative error were 3/127 each (amax is near 3 of its rms), 5 % in all, far above the bf16 roundings (2^-8 each).
"""
import numpy as np
import pytest
import torch

import attn_ref as ref
import ternary_weight_moe_forward_b200 as tw
from ternary_weight_moe_forward_b200 import synth
from ternary_weight_moe_forward_b200.layer import Layer

pytestmark = pytest.mark.gpu
TINY = synth.CONFIGS["tiny"]["shape"]
H, HKV, D, PAGE, PAGES = 8, 2, 64, 16, 40
WINDOWS = (24, 24, 24, 0)


@pytest.fixture(scope="module")
def layers():
    made = []
    for l, window in enumerate(WINDOWS):
        attn = tw.AttentionLayer(TINY.d_model, H, HKV, D, synth.attention_weights(TINY.d_model, H, HKV, D, 5, l), PAGES,
                                 window=window, page_size=PAGE)
        made.append((attn, Layer(TINY, synth.layer_weights(TINY, 5, l), max_tokens=256)))
    yield made
    for _, moe in made:
        moe.close()


def place(lens, extra):
    """Pages for sequences of lens + extra tokens: block table, and the slot of every position."""
    order = torch.randperm(PAGES, generator=torch.Generator().manual_seed(3))
    per = [(m + extra + PAGE - 1) // PAGE for m in lens]
    table = torch.zeros(len(lens), max(per), dtype=torch.int32)
    a = 0
    for b, p in enumerate(per):
        table[b, :p] = order[a:a + p].int()
        a += p
    slots = [table[b].long()[torch.arange(m + extra) // PAGE] * PAGE + torch.arange(m + extra) % PAGE for b, m in enumerate(lens)]
    return table.cuda(), [s.cuda() for s in slots]


def cu(lens):
    return torch.tensor([0] + lens, device="cuda").cumsum(0).int()


def residual(T, seed):
    return torch.from_numpy(synth.residual(T, TINY.d_model, seed)).cuda()


def fake_quant(x):
    amax = x.abs().amax(1, keepdim=True)
    return torch.round(x * (127.0 / amax)).clamp(-127, 127) * (amax / 127.0)


def plain_sublayer(attn, resid, pos, seqs):
    """seqs: per sequence (rows of its new tokens, cached keys, cached values in 64 bits of all of its tokens)."""
    x = resid.double()
    x = (x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()).bfloat16().double()
    qkv = (fake_quant(x) @ attn.qkv.double().t() * attn.alpha_qkv.double()).bfloat16().double()
    q = qkv.view(-1, H + 2 * HKV, D)[:, :H]
    q = q / (q.square().mean(-1, keepdim=True) + 1e-6).sqrt() * attn.q_norm.double()
    ang = (pos.double()[:, None] * attn.inv_freq)[:, None]
    a, b = q.chunk(2, -1)
    q = torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).bfloat16()
    out = torch.zeros(len(x), H, D, dtype=torch.float64, device="cuda")
    for rows, k, v in seqs:
        at = pos[rows][:, None] - torch.arange(len(k), device="cuda")[None, :]
        seen = (at >= 0) & (at < attn.window if attn.window else at >= 0)
        for h in range(H):
            out[rows, h] = ref.attend(q[rows, h], k[:, h // (H // HKV)], v[:, h // (H // HKV)], seen, D ** -0.5)[0]
    return resid.double() + fake_quant(out.flatten(1).bfloat16().double()) @ attn.out.double().t() * attn.alpha_out.double()


def rel(a, b):
    return float((a.double() - b.double()).norm() / b.double().norm())


def test_prompt_then_decode(layers):
    lens, steps = [50, 1, 33], 5
    table, slots = place(lens, steps)
    stack = tw.DecoderStack(layers)
    T = sum(lens)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    flat = torch.cat([s[:m] for s, m in zip(slots, lens)])
    r0 = residual(T, 1)
    # layer by layer: the attention sublayer against the plain form, the MoE layer as it is
    r = r0.clone()
    for attn, moe in layers:
        before = r.clone()
        attn.prompt(r, pos, flat, cu(lens), max(lens))
        rows, seqs = 0, []
        for m, s in zip(lens, slots):
            # the prompt attends over its own bf16 keys and values; the cache holds them to 4 bits, so compare with those
            seqs.append((torch.arange(rows, rows + m, device="cuda"), *prompt_kv(attn, before, pos, rows, m)))
            rows += m
        want = plain_sublayer(attn, before, pos, seqs)
        assert rel(r - before, want - before.double()) < 0.05
        tw.maple_moe_stack_forward([moe.handle], r, T, torch.cuda.current_stream().cuda_stream)
    got = stack.prompt(r0.clone(), pos, flat, cu(lens), max(lens))
    assert torch.equal(got, r)
    # decode steps over the cache
    for i in range(steps):
        x0 = residual(len(lens), 10 + i)
        now = [m + i for m in lens]
        p, s = torch.tensor(now, device="cuda"), torch.stack([s[m] for s, m in zip(slots, now)])
        ln = torch.tensor([m + 1 for m in now], dtype=torch.int32, device="cuda")
        r = x0.clone()
        for attn, moe in layers:
            before = r.clone()
            attn.decode(r, p, s, table, ln)
            seqs = []
            for b, m in enumerate(now):
                k, v = ref.read_pages(attn.pages, PAGE, slots[b][:m + 1], D)
                seqs.append((torch.tensor([b], device="cuda"), k, v))
            want = plain_sublayer(attn, before, p, seqs)
            assert rel(r - before, want - before.double()) < 0.05
            tw.maple_moe_stack_forward([moe.handle], r, len(lens), torch.cuda.current_stream().cuda_stream)
        # the stack's own call writes the same cache rows again and gives the same bits
        assert torch.equal(stack.decode(x0.clone(), p, s, table, ln), r)
    assert stack.device_flags() == 0


def prompt_kv(attn, resid, pos, first, m):
    x = resid[first:first + m].double()
    x = (x / (x.square().mean(1, keepdim=True) + 1e-6).sqrt()).bfloat16().double()
    qkv = (fake_quant(x) @ attn.qkv.double().t() * attn.alpha_qkv.double()).bfloat16().double().view(m, H + 2 * HKV, D)
    k, v = qkv[:, H:H + HKV], qkv[:, H + HKV:]
    k = k / (k.square().mean(-1, keepdim=True) + 1e-6).sqrt() * attn.k_norm.double()
    ang = (pos[first:first + m].double()[:, None] * attn.inv_freq)[:, None]
    a, b = k.chunk(2, -1)
    return torch.cat([a * ang.cos() - b * ang.sin(), b * ang.cos() + a * ang.sin()], -1).bfloat16(), v


def test_prompt_in_chunks_reads_the_cache(layers):
    """A prompt's second part over the first part's cached keys: equal to the sublayer over the values that are read back."""
    attn, _ = layers[3]
    n1, n2 = 40, 23
    _, slots = place([n1 + n2], 0)
    s = slots[0]
    r1, r2 = residual(n1, 21), residual(n2, 22)
    attn.prompt(r1, torch.arange(n1, device="cuda"), s[:n1], cu([n1]), n1)
    before, pos = r2.clone(), torch.arange(n1, n1 + n2, device="cuda")
    attn.prompt(r2, pos, s[n1:], cu([n2]), n2, context=(s, cu([n1 + n2])))
    k, v = ref.read_pages(attn.pages, PAGE, s, D)
    want = plain_sublayer(attn, before, pos, [(torch.arange(n2, device="cuda"), k, v)])
    assert rel(r2 - before, want - before.double()) < 0.05
    assert attn.flags.item() == 0


def test_captured_decode_step(layers):
    """A decode step captured into a graph and replayed with other inputs in the same buffers."""
    lens = [30, 17, 64, 3]
    table, slots = place(lens, 2)
    stack = tw.DecoderStack(layers)
    pos = torch.cat([torch.arange(m, device="cuda") for m in lens])
    stack.prompt(residual(sum(lens), 31), pos, torch.cat([s[:m] for s, m in zip(slots, lens)]), cu(lens), max(lens))
    r, p = residual(4, 32), torch.tensor(lens, device="cuda")
    s, ln = torch.stack([s[m] for s, m in zip(slots, lens)]), torch.tensor([m + 1 for m in lens], dtype=torch.int32, device="cuda")
    x0, x1 = r.clone(), residual(4, 33)
    want = [stack.decode(x.clone(), p, s, table, ln) for x in (x0, x1)]
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        stack.decode(r, p, s, table, ln)
    for x, w in zip((x0, x1), want):
        r.copy_(x)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, w)


def test_refusals(layers):
    stack = tw.DecoderStack(layers)
    with pytest.raises(ValueError):
        stack.decode(torch.zeros(1, TINY.d_model, dtype=torch.bfloat16, device="cuda"), None, None, None, None)
    w = synth.attention_weights(TINY.d_model, H, HKV, D, 5)
    w["out"] = w["out"][:, :-1]
    with pytest.raises(ValueError):
        tw.AttentionLayer(TINY.d_model, H, HKV, D, w, PAGES)
    with pytest.raises(ValueError):
        tw.DecoderStack([(tw.AttentionLayer(512, H, HKV, D, synth.attention_weights(512, H, HKV, D, 5), 2), layers[0][1])])


def test_model_sizes():
    """d_model 2048 with 16 query and 2 key/value heads of 128: one layer, a prompt of 300 tokens and a decode step."""
    big = synth.CONFIGS["decode"]["shape"]
    attn = tw.AttentionLayer(big.d_model, 16, 2, 128, synth.attention_weights(big.d_model, 16, 2, 128, 7), 8, window=512)
    r = torch.from_numpy(synth.residual(300, big.d_model, 3)).cuda()
    before = r.clone()
    s = (torch.arange(301, device="cuda") // 64) * 64 + torch.arange(301, device="cuda") % 64
    attn.prompt(r, torch.arange(300, device="cuda"), s[:300], cu([300]), 300)
    table = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    one = torch.from_numpy(synth.residual(1, big.d_model, 4)).cuda()
    attn.decode(one, torch.tensor([300], device="cuda"), s[300:], table, torch.tensor([301], dtype=torch.int32, device="cuda"))
    torch.cuda.synchronize()
    assert attn.flags.item() == 0
    for t in (r - before, one):
        v = t.cpu().numpy()
        assert np.isfinite(v).all() and np.abs(v).max() > 0

"""Calls of the attention half that are refused before anything is launched or changed, without a GPU."""
import pytest
import torch

import ternary_weight_moe_forward_b200 as tw
from ternary_weight_moe_forward_b200 import synth


class Recorder:
    """Stands for both halves of a layer: records that it was called."""

    def __init__(self, d_model, max_tokens):
        self.d_model, self.max_tokens, self.shape, self.handle, self.calls = d_model, max_tokens, self, 0, 0

    def decode(self, *args):
        self.calls += 1

    prompt = decode


def test_stack_refuses_more_tokens_than_its_layers_take_before_it_starts():
    first, second = Recorder(64, 100), Recorder(64, 8)
    stack = tw.DecoderStack([(first, first), (second, second)])
    resid = torch.zeros(9, 64)
    with pytest.raises(ValueError, match="9 tokens"):
        stack.decode(resid, None, None, None, None)
    with pytest.raises(ValueError, match="9 tokens"):
        stack.prompt(resid, None, None, None, 9)
    assert first.calls == 0 and second.calls == 0


# a page of 64 tokens of 64 channels has as many bytes as one of 32 tokens of 128 channels
@pytest.mark.parametrize("made,other", [((64, 64), (128, 32)), ((64, 32), (128, 16)), ((128, 32), (64, 64)), ((128, 16), (64, 32))])
def test_a_cache_of_another_head_dim_is_refused(made, other):
    (d, n), (d2, n2) = made, other
    pages = tw.kv_pages(2, 1, d, n, device="cpu")
    assert pages.shape == tw.kv_pages(2, 1, d2, n2, device="cpu").shape
    x, i64, i32 = torch.zeros(1, 1, d2, dtype=torch.bfloat16), torch.zeros(1, dtype=torch.int64), torch.zeros(1, dtype=torch.int32)
    for call in (lambda h, **kw: tw.kv_read(pages, i64, h.shape[2], **kw),
                 lambda h, **kw: tw.qk_norm_rope(h, h, i64, torch.zeros(0, dtype=torch.float64), v=h, pages=pages, slots=i64, **kw),
                 lambda h, **kw: tw.cached_attention(h, pages, i32[None], i32, **kw)):
        with pytest.raises(ValueError, match="do not fit this head_dim and page_size"):
            call(x, page_size=n)
        with pytest.raises(ValueError, match="CUDA device"):        # (past that check: the bytes alone fit)
            call(x)
        with pytest.raises(ValueError, match="CUDA device"):
            call(torch.zeros(1, 1, d, dtype=torch.bfloat16), page_size=n)


@pytest.mark.parametrize("which", ["x", "alpha", "bias", "resid", "out"])
def test_linear_refuses_to_lose_a_gradient(which):
    t = dict(x=torch.zeros(2, 64, dtype=torch.bfloat16), alpha=torch.zeros(8), bias=torch.zeros(8), resid=torch.zeros(2, 8),
             out=torch.zeros(2, 8))
    w = torch.zeros(8, 64, dtype=torch.int8)
    t[which].requires_grad_()
    with pytest.raises(ValueError, match="no gradients"):
        tw.int8_linear(t.pop("x"), w, t.pop("alpha"), **t)


@pytest.mark.parametrize("which", range(4))
def test_attention_refuses_to_lose_a_gradient(which):
    h = [torch.zeros(2, 1, 64, dtype=torch.bfloat16) for _ in range(4)]
    h[which].requires_grad_()
    q, k, v, out = h
    i64, i32, f64 = torch.zeros(2, dtype=torch.int64), torch.zeros(2, dtype=torch.int32), torch.zeros(0, dtype=torch.float64)
    pages = tw.kv_pages(1, 1, 64, 16, device="cpu")
    with pytest.raises(ValueError, match="no gradients"):
        tw.prompt_attention(q, k, v, i32, i32, 2, out=out)
    if which < 3:
        with pytest.raises(ValueError, match="no gradients"):
            tw.qk_norm_rope(q, k, i64, f64, v=v, pages=pages, slots=i64)
    if which == 0:
        with pytest.raises(ValueError, match="no gradients"):
            tw.cached_attention(q, pages, i32[:, None], i32)
        with pytest.raises(ValueError, match="no gradients"):
            tw.qk_norm_rope(k, k, i64, f64, torch.ones(64, requires_grad=True))
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA device"):        # (past that check)
            tw.cached_attention(q, pages, i32[:, None], i32)




def test_the_memory_of_out():
    from ternary_weight_moe_forward_b200.attention import _overlap
    buf = torch.zeros(100)
    at = lambda a, n, *s: buf[a:a + n].view(*s)  # noqa: E731
    out = at(20, 12, 3, 4)
    for t, hit in ((None, False), (at(0, 20, 20), False), (at(0, 21, 21), True), (at(31, 1, 1), True), (at(32, 8, 8), False),
                   (buf.as_strided((2, 4), (50, 1), 0), True), (buf.as_strided((2, 4), (16, 1), 0), False),
                   (buf.as_strided((2, 4), (17, 1), 0), True), (buf.as_strided((3, 4), (0, 1), 16), False),
                   (buf.as_strided((3, 5), (0, 1), 16), True), (buf[25:25], False), (out.view(torch.int32), True)):
        assert _overlap(out, t) is hit
    assert not _overlap(buf[20:20], buf)


@pytest.mark.parametrize("name", ["qkv", "alpha_qkv", "out", "alpha_out", "q_norm", "k_norm"])
def test_a_layer_needs_its_weights(name):
    weights = synth.attention_weights(256, 4, 2, 64, 5)
    weights[name] = None
    if name.endswith("norm"):
        assert getattr(tw.AttentionLayer(256, 4, 2, 64, weights, 1, device="cpu"), name) is None
        return
    for w in (weights, {k: v for k, v in weights.items() if k != name}):
        with pytest.raises(ValueError, match=f"{name} is missing"):
            tw.AttentionLayer(256, 4, 2, 64, w, 1, device="cpu")

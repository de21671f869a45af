"""The attention half's C ABI without a GPU: the argument structs as Python packs them, and calls that are refused
before anything is launched."""
import ctypes as C
import os
import re
import subprocess

import pytest
import torch

import ternary_weight_moe_forward_b200 as tw
from ternary_weight_moe_forward_b200 import attention as at
from ternary_weight_moe_forward_b200 import build_lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "maple_attn.h")
STRUCTS = {"linear": at._LINEAR, "rope": at._ROPE, "read": at._READ, "prompt": at._PROMPT, "cached": at._CACHED}
P = 1 << 20   # an aligned address that is never followed


@pytest.fixture(scope="module")
def lib():
    build_lib.build()
    return at._lib()


def test_header_symbols_are_exported(lib):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER, encoding="utf-8").read(), flags=re.S)
    names = set(re.findall(r"^(?:int|int64_t)\s+(maple_attn_\w+)\s*\(", text, flags=re.M))
    assert {"maple_attn_linear", "maple_attn_qk_norm_rope", "maple_attn_kv_read", "maple_attn_prompt", "maple_attn_cached",
            "maple_attn_page_bytes", "maple_attn_linear_workspace", "maple_attn_cached_workspace"} == names
    out = subprocess.run(["nm", "-D", "--defined-only", tw.LIB_PATH], capture_output=True, text=True, check=True).stdout
    assert names <= set(re.findall(r" T (\w+)$", out, flags=re.M))


def test_struct_sizes_match_the_header(tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "maple_attn.h"\nint main(void){' + "".join(
        f'printf("%zu\\n", sizeof(maple_attn_{n}_args));' for n in STRUCTS) + "return 0;}\n")
    subprocess.run(["gcc", "-I", os.path.join(ROOT, "include"), str(src), "-o", str(tmp_path / "s")], check=True)
    sizes = subprocess.run([str(tmp_path / "s")], capture_output=True, text=True, check=True).stdout.split()
    assert [int(s) for s in sizes] == [s.size for s in STRUCTS.values()]


def test_page_bytes(lib):
    assert lib.maple_attn_page_bytes(128, 64) == 64 * 160
    assert lib.maple_attn_page_bytes(64, 16) == 16 * 80
    for d, n in ((96, 64), (128, 48), (128, 0), (0, 16), (128, 128)):
        assert lib.maple_attn_page_bytes(d, n) == tw.MAPLE_ERR_UNSUPPORTED_SHAPE


def call(lib, name, fields, **change):
    fields = {**fields, **change}
    return getattr(lib, "maple_attn_" + {"rope": "qk_norm_rope", "read": "kv_read"}.get(name, name))(
        STRUCTS[name].pack(*fields.values()), None)


LINEAR = dict(x=P, w=P, alpha=P, bias=0, resid=0, y=P, ws=P, wsb=1 << 20, flags=0, xs=64, T=20, K=64, N=8, dt=2, norm=0)
ROPE = dict(q=P, k=P, v=P, qo=P, ko=P, qw=0, kw=0, pos=P, inv=P, pages=P, slots=P, flags=0, qs=512, ks=512, vs=512, T=2, NP=4,
            H=4, Hkv=2, d=128, rd=128, n=16, dt=0, inter=0, eps=1e-6)
READ = dict(pages=P, slots=P, k=P, v=P, flags=0, n=2, NP=4, Hkv=2, d=128, ps=16, dt=0)
PROMPT = dict(q=P, k=P, v=P, out=P, lse=0, cq=P, ck=P, flags=0, qs=512, ks=256, vs=256, Tq=4, Tk=4, B=1, mq=4, H=4, Hkv=2, d=128,
              win=0, dt=0, scale=0.1)
CACHED = dict(q=P, out=P, pages=P, bt=P, lens=P, ws=P, wsb=1 << 30, flags=0, qs=512, ts=4, NP=4, B=2, mp=4, H=4, Hkv=2, d=128, n=16,
              win=0, dt=0, scale=0.1)


def test_null_and_empty(lib):
    for f in ("linear", "qk_norm_rope", "kv_read", "prompt", "cached"):
        assert getattr(lib, "maple_attn_" + f)(None, None) == tw.MAPLE_ERR_INVALID_ARG
    # no rows: nothing to do, nothing is read
    assert call(lib, "linear", LINEAR, T=0, x=0, y=0, ws=0, wsb=0) == tw.MAPLE_OK
    assert call(lib, "rope", ROPE, T=0) == tw.MAPLE_OK
    assert call(lib, "read", READ, n=0) == tw.MAPLE_OK
    assert call(lib, "prompt", PROMPT, B=0) == tw.MAPLE_OK
    assert call(lib, "prompt", PROMPT, Tq=0) == tw.MAPLE_OK
    assert call(lib, "cached", CACHED, B=0) == tw.MAPLE_OK


BAD, SHAPE = tw.MAPLE_ERR_INVALID_ARG, tw.MAPLE_ERR_UNSUPPORTED_SHAPE


@pytest.mark.parametrize("name,base,change,code", [
    *[("linear", LINEAR, c, BAD) for c in (dict(x=0), dict(w=0), dict(alpha=0), dict(y=0), dict(ws=0), dict(wsb=16), dict(x=P + 2),
                                          dict(w=P + 8), dict(y=P + 4), dict(xs=66), dict(dt=1), dict(dt=7), dict(resid=P + 4))],
    *[("linear", LINEAR, c, SHAPE) for c in (dict(K=24), dict(K=0), dict(K=32784), dict(N=0), dict(T=-1), dict(T=1 << 31),
                                            dict(N=1 << 36), dict(norm=1))],
    *[("rope", ROPE, c, BAD) for c in (dict(q=0), dict(k=0), dict(v=0), dict(qo=0), dict(ko=0, pages=0), dict(pos=0), dict(inv=0),
                                       dict(slots=0), dict(NP=0), dict(q=P + 8), dict(pages=P + 8), dict(qs=500), dict(vs=4), dict(T=-1),
                                       dict(dt=2), dict(eps=-1.0), dict(eps=float("nan")), dict(pos=P + 4))],
    *[("rope", ROPE, c, SHAPE) for c in (dict(d=96), dict(H=3), dict(H=0), dict(Hkv=0), dict(rd=130), dict(rd=8), dict(rd=-16),
                                         dict(n=48))],
    *[("read", READ, c, BAD) for c in (dict(pages=0), dict(slots=0), dict(k=0), dict(v=0), dict(n=-1), dict(NP=0), dict(dt=2),
                                       dict(k=P + 8))],
    *[("read", READ, c, SHAPE) for c in (dict(d=32), dict(ps=8), dict(Hkv=0))],
    *[("prompt", PROMPT, c, BAD) for c in (dict(q=0), dict(k=0), dict(v=0), dict(out=0), dict(cq=0), dict(ck=0), dict(B=-1), dict(mq=-1),
                                           dict(win=-1), dict(Tq=-1), dict(dt=2), dict(scale=float("inf")), dict(qs=513),
                                           dict(out=P + 8), dict(cq=P + 2), dict(B=1 << 17), dict(ks=0), dict(vs=-256),
                                           dict(Tk=1 << 31))],
    *[("prompt", PROMPT, c, SHAPE) for c in (dict(d=256), dict(H=5), dict(H=0), dict(Hkv=0), dict(H=256, Hkv=2))],
    *[("cached", CACHED, c, BAD) for c in (dict(q=0), dict(out=0), dict(pages=0), dict(bt=0), dict(lens=0), dict(NP=0), dict(B=-1),
                                           dict(mp=-1), dict(win=-1), dict(dt=2), dict(scale=float("nan")), dict(q=P + 8),
                                           dict(qs=7), dict(B=1 << 17), dict(pages=P + 8))],
    *[("cached", CACHED, c, SHAPE) for c in (dict(d=32), dict(n=24), dict(H=5), dict(H=0), dict(Hkv=0))],
])
def test_refused_before_any_launch(lib, name, base, change, code):
    assert call(lib, name, base, **change) == code


def test_python_refuses_wrong_tensors():
    x, w, al = torch.zeros(2, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.int8), torch.zeros(8)
    with pytest.raises(ValueError):
        tw.int8_linear(x, w, al)                      # not on a GPU
    with pytest.raises(ValueError):
        tw.int8_linear(x, w[:, :32], al)              # K does not match
    q = torch.zeros(2, 4, 128, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        tw.qk_norm_rope(q.float(), q, torch.zeros(2, dtype=torch.int64), torch.zeros(64, dtype=torch.float64))
    with pytest.raises(ValueError):
        tw.prompt_attention(q.transpose(0, 1), q, q, torch.zeros(2, dtype=torch.int32), torch.zeros(2, dtype=torch.int32), 2)
    with pytest.raises(ValueError):
        tw.cached_attention(q, torch.zeros(1, 2, 2560, dtype=torch.uint8), torch.zeros(2, 1, dtype=torch.int32),
                            torch.zeros(2, dtype=torch.int32))
    with pytest.raises(tw.MapleError):
        tw.kv_pages(1, 1, 96)


@pytest.mark.parametrize("head_dim", [0, -128, 32, 96, 256])
def test_python_refuses_a_head_dim_that_the_pages_do_not_have(head_dim):
    with pytest.raises(ValueError):
        tw.kv_read(torch.zeros(1, 2, 2560, dtype=torch.uint8), torch.zeros(2, dtype=torch.int64), head_dim)

"""Host-side tests of the trunk operators that need no GPU: descriptors, refusals with their status codes, empty
calls, and the plain forms' gradients against differences.  Pointers are fake addresses: nothing gets as
far as a launch."""
import ctypes
import math
import os
import re
import subprocess

import pytest
import torch

import trunk_reference as ref
from conv_batchnorm_relu_gb300 import attention, build, cbr, gradients, group_norm

P = 0x10000
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")
FAR = 1 << 40


@pytest.fixture(scope="module")
def lib():
    build.build()
    attention._load(), group_norm._load(), gradients._load()
    return cbr.load()


def att_desc(batch=2, tq=5, tk=7, q=(640, 128, 64), k=(448, 64, 64), v=None, o=None, do=None, dq=None, dk=None, dv=None, hq=2, hk=1, d=64,
             causal=0, dtype=0, scale=0.125):
    return attention._DESC.pack(batch, tq, tk, *q, *k, *(v or k), *(o or q), *(do or q), *(dq or q), *(dk or k), *(dv or k), hq, hk, d, causal,
                                dtype, scale)


def af(lib, desc, q=P, k=P + 4096, v=P + 8192, n=None, s=None, o=P + 16384, lse=P, ws=P, size=FAR):
    return lib.cbr_attention_forward(desc, q, k, v, n, s, o, lse, ws, size, None)


def ab(lib, desc, do=P, q=P + 4096, k=P + 8192, v=P + 12288, o=P + 16384, lse=P, n=None, s=None, dq=P + (1 << 20), dk=P + (2 << 20),
       dv=P + (3 << 20), ws=P, size=FAR):
    return lib.cbr_attention_backward(desc, do, q, k, v, o, lse, n, s, dq, dk, dv, ws, size, None)


def gn_desc(images=2, pixels=9, x=(144, 16), y=None, dy=None, dx=None, c=16, groups=4, act=1, dtype=0, eps=1e-5):
    return group_norm._DESC.pack(images, pixels, *x, *(y or x), *(dy or x), *(dx or x), c, groups, act, dtype, eps)


def gf(lib, desc, x=P, g=P, b=P, y=P + 4096, m=P, r=P, ws=P, size=FAR):
    return lib.cbr_group_norm_forward(desc, x, g, b, y, m, r, ws, size, None)


def gb(lib, desc, dy=P, x=P + 4096, g=P, b=P, m=P, r=P, dx=P + 8192, dg=P, db=P, ws=P, size=FAR):
    return lib.cbr_group_norm_backward(desc, dy, x, g, b, m, r, dx, dg, db, ws, size, None)


def clip(lib, grads=(P, P + 4096), sizes=(5, 7), types=(2, 0), outs=None, top=1.0, unscale=1.0, norm=P, scale=P + 4, ws=P, size=FAR, count=None):
    n = len(grads)
    vp = ctypes.c_void_p * max(n, 1)
    return lib.cbr_clip_gradients(n if count is None else count, vp(*grads), (ctypes.c_int64 * max(n, 1))(*sizes), (ctypes.c_int32 * max(n, 1))(*types),
                                  None if outs is None else vp(*outs), top, unscale, norm, scale, ws, size, None)


def test_descriptor_sizes_match_the_header(lib, tmp_path):
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "cbr.h"\nint main(void){printf("%zu %zu",sizeof(cbr_attention_desc_t),'
                   'sizeof(cbr_group_norm_desc_t));return 0;}\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I", os.path.dirname(cbr.HEADER_PATH), str(src), "-o", exe], check=True)
    sizes = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert sizes == [attention._DESC.size, group_norm._DESC.size]


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(tq=-1), 1), (dict(tk=-2), 1), (dict(hq=0), 1), (dict(hk=0), 1), (dict(hq=3, hk=2), 1), (dict(d=0), 1),
    (dict(scale=-1.0), 1), (dict(scale=math.nan), 1), (dict(scale=math.inf), 1), (dict(dtype=2), 3), (dict(dtype=9), 3), (dict(d=60), 3),
    (dict(d=136, q=(6400, 1280, 136), k=(6400, 640, 136)), 3), (dict(tq=(1 << 30) + 1), 3), (dict(tk=(1 << 30) + 1), 3), (dict(batch=1 << 39), 3),
    (dict(hq=65538, hk=1), 3), (dict(q=(640, 129, 64)), 2), (dict(q=(644, 128, 64)), 2), (dict(k=(448, 0, 64)), 1), (dict(k=(448, 56, 64)), 1),
    (dict(v=(-8, 64, 64)), 1), (dict(q=(1 << 39, 128, 64)), 1), (dict(o=(640, 64, 64)), 1), (dict(o=(0, 128, 64)), 1), (dict(o=(640, 128, 0)), 1),
    (dict(o=(320, 128, 64)), 1)])
def test_attention_descriptor_refusals(lib, kw, status):
    assert af(lib, att_desc(**kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(do=(640, 127, 64)), 2), (dict(dq=(640, 64, 64)), 1), (dict(dk=(0, 64, 64)), 1), (dict(dv=(440, 64, 64)), 1), (dict(dq=(0, 128, 64)), 1)])
def test_attention_backward_stride_refusals(lib, kw, status):
    assert ab(lib, att_desc(**kw)) == status


def test_attention_pointer_refusals(lib):
    d = att_desc()
    for k in ("q", "k", "v", "o"):
        assert af(lib, d, **{k: None}) == 1, k
    for k in ("q", "k", "v", "o"):
        assert af(lib, d, **{k: P + 40}) == 2, k
    assert af(lib, d, lse=P + 2) == 2 and af(lib, d, n=P + 2) == 2 and af(lib, d, s=P + 1) == 2
    for k in ("q", "k", "v"):
        assert af(lib, d, **{k: P + 16384}) == 1, k     # o in an input's place
    for k in ("do", "q", "k", "v", "o", "lse", "dq", "dk", "dv", "ws"):
        assert ab(lib, d, **{k: None}) == 1, k
    for k in ("do", "q", "k", "v", "o", "dq", "dk", "dv", "ws"):
        assert ab(lib, d, **{k: P + 8}) == 2, k
    for k in ("do", "q", "k", "v", "o"):
        assert ab(lib, d, **{k: P + (2 << 20)}) == 1, k
    assert ab(lib, d, dq=P + (2 << 20)) == 1 and ab(lib, d, dv=P + (1 << 20)) == 1
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.cbr_attention_workspace_size(d, ctypes.byref(f), ctypes.byref(b)) == 0 and b.value > 0
    assert ab(lib, d, size=b.value - 1) == 4
    assert lib.cbr_attention_workspace_size(None, ctypes.byref(f), None) == 1
    assert lib.cbr_attention_workspace_size(att_desc(d=12), ctypes.byref(f), None) == 3


def test_empty_calls_do_nothing(lib):
    assert af(lib, att_desc(batch=0)) == 0 and af(lib, att_desc(tq=0)) == 0
    assert ab(lib, att_desc(batch=0)) == 0 and ab(lib, att_desc(tq=0, tk=0)) == 0
    assert gf(lib, gn_desc(images=0)) == 0 and gf(lib, gn_desc(pixels=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(images=-1), 1), (dict(pixels=-1), 1), (dict(c=0), 1), (dict(groups=0), 1), (dict(groups=3), 1), (dict(act=3), 1), (dict(act=-1), 1),
    (dict(eps=0.0), 1), (dict(eps=math.nan), 1), (dict(eps=math.inf), 1), (dict(dtype=3), 3), (dict(c=16388, x=(160000, 16388)), 3),
    (dict(images=1 << 31), 3), (dict(pixels=1 << 31), 3), (dict(x=(144, 15)), 1), (dict(x=(140, 16)), 1), (dict(y=(0, 16)), 1), (dict(x=(-144, 16)), 1),
    (dict(y=(FAR + 1, 16)), 1), (dict(c=8192, groups=8192, x=(80000, 8192)), 3)])
def test_group_norm_descriptor_refusals(lib, kw, status):
    assert gf(lib, gn_desc(**kw)) == status


def test_group_norm_pointer_refusals(lib):
    d = gn_desc()
    for k in ("x", "y", "m", "r", "g", "b"):
        assert gf(lib, d, **{k: None}) == 1, k
    assert gf(lib, d, x=P + 1) == 2 and gf(lib, d, g=P + 2) == 2 and gf(lib, d, m=P + 1) == 2
    assert gf(lib, gn_desc(y=(160, 16)), y=P) == 1                              # in place, other strides
    for k in ("dy", "x", "m", "r", "dx", "g", "b", "dg", "db", "ws"):
        assert gb(lib, d, **{k: None}) == 1, k
    assert gb(lib, d, dx=P + 4096) == 1 and gb(lib, d, dx=P + 1) == 2 and gb(lib, d, ws=P + 8) == 2
    assert gb(lib, gn_desc(dx=(160, 16)), dx=P) == 1
    f, b = ctypes.c_size_t(), ctypes.c_size_t()
    assert lib.cbr_group_norm_workspace_size(d, ctypes.byref(f), ctypes.byref(b)) == 0 and b.value > 0
    assert gb(lib, d, size=b.value - 1) == 4 and gf(lib, d, ws=P + 8) == 2
    assert lib.cbr_group_norm_workspace_size(d, None, None) == 0
    # one image that no cluster holds: moments of its runs
    big = gn_desc(images=1, pixels=1 << 20, c=64, x=(64 << 20, 64), groups=8)
    assert lib.cbr_group_norm_workspace_size(big, ctypes.byref(f), ctypes.byref(b)) == 0 and f.value > 0
    assert gf(lib, big, size=f.value - 1) == 4 and gf(lib, big, ws=None) == 1


def test_clip_refusals(lib):
    for kw in (dict(top=-1.0), dict(top=math.nan), dict(unscale=0.0), dict(unscale=math.nan), dict(unscale=math.inf), dict(norm=None), dict(scale=None),
               dict(scale=P), dict(ws=None), dict(count=-1), dict(grads=(None, P)), dict(sizes=(-1, 3)), dict(outs=(P, None))):
        assert clip(lib, **kw) == 1, kw
    assert clip(lib, types=(3, 0)) == 3 and clip(lib, count=(1 << 20) + 1) == 3
    assert clip(lib, grads=(P + 2, P)) == 2 and clip(lib, grads=(P, P + 1)) == 2 and clip(lib, ws=P + 8) == 2 and clip(lib, norm=P + 2) == 2
    n = ctypes.c_size_t()
    assert lib.cbr_clip_workspace_size(2, ctypes.byref(n)) == 0 and clip(lib, size=n.value - 1) == 4
    assert lib.cbr_clip_workspace_size(-1, ctypes.byref(n)) == 1 and lib.cbr_clip_workspace_size(2, None) == 1


def test_clip_refuses_outs_that_share_memory(lib):
    a, b, c = P, P + 4096, P + 8192
    ok, no = (5, 1) if not torch.cuda.is_available() else (None, 1)
    for grads, outs, want in [((a, b), (a, b), ok), ((a, b), (c, c + 10), no), ((a, b), (c, c + 20), ok), ((a, a), (a, a), no), ((a, a), (b, c), ok),
                              ((a, b), (b, a), no), ((a, b), (c, a + 16), no), ((a, b), (a + 4, b), no), ((a, b), (a, b + 4), no)]:
        if want is not None:
            assert clip(lib, grads=grads, outs=outs) == want, (grads, outs)      # 5 values of 2 bytes, 7 of 4
    if ok is not None:
        assert clip(lib, grads=(a, a), sizes=(0, 7), outs=(a, a)) == ok


@NO_DEVICE
def test_valid_calls_reach_the_device_check(lib):
    assert af(lib, att_desc()) == 5 and ab(lib, att_desc()) == 5
    assert af(lib, att_desc(q=(640, 128, 0), k=(0, 64, 64), o=(640, 128, 64))) == 5      # inputs that repeat
    assert af(lib, att_desc(batch=1, q=(7, 128, 64), k=(3, 64, 1))) == 5                 # axes of one step
    assert af(lib, att_desc(tk=0), k=None, v=None) == 5
    assert gf(lib, gn_desc()) == 5 and gb(lib, gn_desc()) == 5
    assert gf(lib, gn_desc(), g=None, b=None) == 5 and gf(lib, gn_desc(), y=P) == 5
    assert gb(lib, gn_desc(), g=None, b=None, dg=None, db=None, ws=None) == 5
    assert clip(lib) == 5 and clip(lib, top=math.inf) == 5 and clip(lib, grads=(None, P), sizes=(0, 3)) == 5


def test_no_exception_leaves_an_entry():
    text = open(os.path.join(build.CSRC, "trunk_api.cu")).read()
    entries = re.findall(r"^cbr_status_t cbr_\w+\([^)]*\) \{\n(.*)$", text, re.M)
    assert len(entries) == 8 and all(e.strip().startswith("return guarded(") for e in entries)


def test_binding_wants_cuda_tensors():
    x = torch.zeros(1, 4, 2, 64, dtype=torch.float16)
    with pytest.raises(cbr.CBRError):
        attention.attention_forward(x, x, x)
    with pytest.raises(cbr.CBRError):
        group_norm.group_norm_forward(x, None, None, 4)
    for grads in ([], [torch.zeros(3)]):
        with pytest.raises(cbr.CBRError):
            gradients.clip_gradients(grads, 1.0)


# ---------------------------------------------------------------- the plain forms against differences

@pytest.mark.parametrize("causal", [False, True])
def test_attention_gradient_against_differences(causal):
    g = torch.Generator().manual_seed(1)
    q, do = (torch.randn(2, 4, 4, 8, generator=g, dtype=torch.float64) for _ in range(2))
    k, v = (torch.randn(2, 5, 2, 8, generator=g, dtype=torch.float64) for _ in range(2))
    lengths = torch.tensor([5, 3])
    # (the bounds go by the storage type; differences need 64 bits)
    ref.U[torch.float64] = 2.0 ** -53
    kw = dict(scale=0.3, causal=causal, lengths=lengths)
    f = ref.attention(q, k, v, **kw)
    got = ref.attention_backward(do, q, k, v, f["o"], f["lse"], **kw)
    h = 1e-5
    for name, t in (("dq", q), ("dk", k), ("dv", v)):
        for at in ((0, 1, 1, 3), (1, 2, 0, 7), (1, 3, 1, 0)):
            up, down = t.clone(), t.clone()
            up[at] += h
            down[at] -= h
            ops = {"dq": (q, k, v), "dk": (q, k, v), "dv": (q, k, v)}[name]
            i = ("dq", "dk", "dv").index(name)
            a, b = list(ops), list(ops)
            a[i], b[i] = up, down
            d = float(((ref.attention(*a, **kw)["o"] - ref.attention(*b, **kw)["o"]) * do).sum() / (2 * h))
            assert abs(d - float(got[name][at])) < 1e-8, (name, at)


@pytest.mark.parametrize("act", ["none", "relu", "silu"])
def test_group_norm_gradient_against_differences(act):
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(2, 3, 4, 6, generator=g, dtype=torch.float64) for _ in range(2))
    gamma, beta = 1 + 0.2 * torch.randn(6, generator=g, dtype=torch.float64), torch.randn(6, generator=g, dtype=torch.float64)
    f = ref.group_norm(x, gamma, beta, 3, 1e-5, act)
    got = ref.group_norm_backward(dy, x, gamma, beta, f["mean"], f["rstd"], 3, act)
    h = 1e-6

    def loss(x, gamma, beta):
        return float((ref.group_norm(x, gamma, beta, 3, 1e-5, act)["y"] * dy).sum())

    for i, (name, t, places) in enumerate((("dx", x, [(0, 1, 2, 3), (1, 2, 0, 5)]), ("dgamma", gamma, [(0,), (4,)]), ("dbeta", beta, [(1,), (5,)]))):
        for at in places:
            ops = [x, gamma, beta]
            up, down = t.clone(), t.clone()
            up[at] += h
            down[at] -= h
            d = (loss(*ops[:i], up, *ops[i + 1:]) - loss(*ops[:i], down, *ops[i + 1:])) / (2 * h)
            assert abs(d - float(got[name][at])) < 1e-6 * max(1.0, abs(d)), (name, at)

"""Host-side tests of the token operators that need no GPU: descriptors, refusals with their status codes,
empty calls, and the rotary table.  Pointers are fake addresses: nothing gets as far as a launch."""
import ctypes
import math

import pytest
import torch

from conv_batchnorm_relu_gb300 import build, cbr, tokens

P = 0x10000
NO_DEVICE = pytest.mark.skipif(torch.cuda.is_available(), reason="checks the no-device path")


@pytest.fixture(scope="module")
def lib():
    build.build()
    return tokens._load()


def distill_desc(rows=4, vocab=100, topk=3, ls=100, ds=100, ids=3, tops=3, dtype=0, top=0, id_bytes=4, temp=1.0):
    return tokens._DISTILL.pack(rows, vocab, topk, ls, ds, ids, tops, dtype, top, id_bytes, temp)


def fb(lib, desc, logits=P, ids=P, top=P, lse=None, w=None, loss=P, stats=None, d=P + (1 << 20)):
    return lib.cbr_distill_forward_backward(desc, logits, ids, top, lse, w, loss, stats, d, None)


def norm_desc(rows=4, dim=64, gate_rows=4, strides=(64,) * 8, dtype=0, kind=0, eps=1e-6, rho=1.0, beta=1.0):
    return tokens._NORM.pack(rows, dim, gate_rows, *strides, dtype, kind, eps, rho, beta)


def nf(lib, desc, x=P, f=P + 1024, w1=P, gate=P, w2=P, xo=P + 2048, h=P + 4096, stats=P):
    return lib.cbr_block_norm_forward(desc, x, f, w1, gate, w2, xo, h, stats, None)


def nb(lib, desc, dxo=P, dh=P + 64, xo=P + 128, f=P + 256, w1=P, gate=P, w2=P, stats=P, dx=P + 512, df=P + 1024, dw1=P,
       dg=P, dw2=P, ws=P, n=1 << 40):
    return lib.cbr_block_norm_backward(desc, dxo, dh, xo, f, w1, gate, w2, stats, dx, df, dw1, dg, dw2, ws, n, None)


def rotary_desc(batch=2, n=5, q=(640, 128, 64), k=(320, 64, 64), qo=None, ko=None, pos=(15, 3, 1), hq=2, hk=1, d=64,
                rot=64, axes=3, layout=0, dtype=0):
    return tokens._ROTARY.pack(batch, n, *q, *k, *(qo or q), *(ko or k), *pos, hq, hk, d, rot, axes, layout, dtype)


def rot(lib, desc, q=P, k=P + 1024, pos=P, f=P, a=P, qo=P + 8192, ko=P + 16384):
    return lib.cbr_rotary_forward(desc, q, k, pos, f, a, qo, ko, None)


def test_descriptor_sizes_match_the_header(lib, tmp_path):
    """The packed descriptors have the C structures' sizes (gcc on the header)."""
    import os
    import subprocess
    src = tmp_path / "s.c"
    src.write_text('#include <stdio.h>\n#include "cbr.h"\nint main(void){printf("%zu %zu %zu",sizeof(cbr_distill_desc_t),'
                   'sizeof(cbr_block_norm_desc_t),sizeof(cbr_rotary_desc_t));return 0;}\n')
    exe = str(tmp_path / "s")
    subprocess.run(["gcc", "-I", os.path.dirname(cbr.HEADER_PATH), str(src), "-o", exe], check=True)
    sizes = [int(v) for v in subprocess.run([exe], check=True, capture_output=True, text=True).stdout.split()]
    assert sizes == [tokens._DISTILL.size, tokens._NORM.size, tokens._ROTARY.size]


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-1), 1), (dict(vocab=0), 1), (dict(topk=-1), 1), (dict(ls=99), 1), (dict(ds=50), 1), (dict(ids=2), 1),
    (dict(tops=2), 1), (dict(temp=0.0), 1), (dict(temp=-1.0), 1), (dict(temp=math.nan), 1), (dict(temp=math.inf), 1),
    (dict(temp=1e-45), 1), (dict(id_bytes=2), 1), (dict(dtype=3), 3), (dict(top=7), 3), (dict(rows=1 << 41), 1),
    (dict(vocab=393217, ls=393217, ds=393217), 3), (dict(topk=1025, ids=1025, tops=1025), 3)])
def test_distill_descriptor_refusals(lib, kw, status):
    assert fb(lib, distill_desc(**kw)) == status


def test_distill_pointer_refusals(lib):
    d = distill_desc()
    for k in ("logits", "ids", "top", "loss", "d"):
        assert fb(lib, d, **{k: None}) == 1, k
    assert lib.cbr_distill_forward_backward(None, P, P, P, None, None, P, None, P, None) == 1
    assert lib.cbr_distill_forward(d, P, P, P, None, None, P, None, None) == 1          # the loss's stats are needed
    assert lib.cbr_distill_backward(d, None, P, P, P, None, None, None, P + 4096, None) == 1
    assert fb(lib, d, logits=P + 1) == 2 and fb(lib, d, ids=P + 2) == 2 and fb(lib, d, top=P + 1) == 2
    assert fb(lib, d, loss=P + 2) == 2 and fb(lib, d, lse=P + 2) == 2 and fb(lib, d, d=P + 1) == 2
    assert fb(lib, distill_desc(ds=128), d=P) == 1                                      # in place, another stride


def test_empty_calls_do_nothing(lib):
    assert lib.cbr_distill_forward_backward(distill_desc(rows=0), *([None] * 9)) == 0
    assert lib.cbr_block_norm_forward(norm_desc(rows=0, gate_rows=1), P, P, P, P, P, P, P, P, None) == 0
    assert rot(lib, rotary_desc(n=0)) == 0 and rot(lib, rotary_desc(batch=0)) == 0


@pytest.mark.parametrize("kw,status", [
    (dict(rows=-2), 1), (dict(dim=0), 1), (dict(gate_rows=0), 1), (dict(gate_rows=3), 1), (dict(strides=(63,) + (64,) * 7), 1),
    (dict(strides=(64, 10) + (64,) * 6), 1), (dict(strides=(64, 64, 1) + (64,) * 5), 1), (dict(kind=2), 1),
    (dict(eps=0.0), 1), (dict(eps=math.nan), 1), (dict(rho=math.inf), 1), (dict(beta=math.nan), 1), (dict(dtype=5), 3),
    (dict(dim=16385, strides=(16385,) * 8), 3)])
def test_norm_descriptor_refusals(lib, kw, status):
    assert nf(lib, norm_desc(**kw)) == status


def test_norm_pointer_refusals(lib):
    d = norm_desc()
    assert nf(lib, d, f=None, w2=None) == 1
    for k in ("x", "w1", "xo", "h"):
        assert nf(lib, d, **{k: None}) == 1, k
    assert nf(lib, d, x=P + 1) == 2 and nf(lib, d, w2=P + 2) == 2 and nf(lib, d, stats=P + 2) == 2
    assert nf(lib, d, h=P + 2048) == 1 and nf(lib, d, h=P) == 1                         # h on x_out, on x
    assert nf(lib, norm_desc(strides=(64, 64, 72, 64, 64, 64, 64, 64)), xo=P) == 1      # in place, another stride
    for k in ("dh", "xo", "w1", "stats", "dx", "df", "dw1", "dg", "dw2", "ws"):
        assert nb(lib, d, **{k: None}) == 1, k
    assert nb(lib, d, w2=None, dxo=None) == 1
    assert nb(lib, d, dx=P + 128) == 1 and nb(lib, d, df=P + 512) == 1
    assert nb(lib, d, ws=P + 8) == 2
    n = ctypes.c_size_t()
    assert lib.cbr_block_norm_workspace_size(d, ctypes.byref(n)) == 0 and n.value > 0
    assert nb(lib, d, n=n.value - 1) == 4
    assert lib.cbr_block_norm_workspace_size(d, None) == 1
    assert tokens.block_norm_workspace_size(4, 64) == n.value


@pytest.mark.parametrize("kw,status", [
    (dict(batch=-1), 1), (dict(n=-1), 1), (dict(d=0), 1), (dict(rot=3), 1), (dict(rot=0), 1), (dict(rot=66), 1),
    (dict(axes=0), 1), (dict(layout=2), 1), (dict(hq=-1), 1), (dict(q=(640, -1, 64)), 1), (dict(qo=(640, 0, 64)), 1),
    (dict(ko=(320, 32, 64)), 1), (dict(dtype=4), 3), (dict(d=1026, q=(6400, 3000, 1026), k=(6400, 3000, 1026)), 3),
    (dict(axes=9), 3), (dict(pos=(15, 1 << 41, 1)), 1)])
def test_rotary_descriptor_refusals(lib, kw, status):
    assert rot(lib, rotary_desc(**kw)) == status


def test_rotary_pointer_refusals(lib):
    d = rotary_desc()
    for k in ("q", "k", "pos", "f", "a", "qo", "ko"):
        assert rot(lib, d, **{k: None}) == 1, k
    assert rot(lib, d, q=P + 1) == 2 and rot(lib, d, f=P + 4) == 2 and rot(lib, d, pos=P + 2) == 2
    assert rot(lib, rotary_desc(qo=(1280, 256, 64)), qo=P) == 1                         # in place, other strides


@NO_DEVICE
def test_valid_calls_reach_the_device_check(lib):
    assert fb(lib, distill_desc()) == 5
    assert lib.cbr_distill_backward(distill_desc(), None, P, P, P, None, None, P, P, None) == 5
    assert nf(lib, norm_desc()) == 5 and nb(lib, norm_desc()) == 5
    assert rot(lib, rotary_desc()) == 5


def test_binding_wants_cuda_tensors():
    with pytest.raises(tokens.CBRError):
        tokens.distill_forward(torch.zeros(2, 3), torch.zeros(2, 1, dtype=torch.int32), torch.zeros(2, 1))
    with pytest.raises(tokens.CBRError):
        tokens.block_norm_forward(torch.zeros(2, 3), pre_weight=torch.ones(3))


def test_rotary_table_values():
    freq, axis = tokens.rotary_table((2, 3), theta=100.0, device="cpu")
    assert axis.tolist() == [0, 0, 1, 1, 1]
    for i, f in enumerate(freq.tolist()):
        assert abs(f / 2.0 ** 64 * 2 * math.pi - 100.0 ** (-i / 5)) < 1e-15
    freq, axis = tokens.rotary_table((1, 3), theta=100.0, order="cycled", spectrum="own", device="cpu")
    assert axis.tolist() == [0, 1, 1, 1]
    want = [1.0] + [100.0 ** (-j / 3) for j in range(3)]
    assert all(abs(f / 2.0 ** 64 * 2 * math.pi - w) < 1e-15 for f, w in zip(freq.tolist(), want))
    # frequencies of more than half a turn a step wrap, as the angles do
    assert tokens.rotary_table((2,), theta=0.01, device="cpu")[0].shape == (2,)
    for bad in ((), (0, 0), (-1, 4), (1,) * 9):
        with pytest.raises(tokens.CBRError):
            tokens.rotary_table(bad, device="cpu")
    with pytest.raises(tokens.CBRError):
        tokens.rotary_table((4,), order="shuffled", device="cpu")
    assert tokens.grid_positions(2, 2, device="cpu").tolist() == [[0, 0], [0, 1], [1, 0], [1, 1]]

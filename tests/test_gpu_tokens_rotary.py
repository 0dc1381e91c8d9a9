"""Rotary positions over several axes against whole-number angles in 64 bits: types, layouts, head counts
and widths, strides, far and negative positions, the backward as the transpose."""
import pytest
import torch

import token_reference as ref
from conv_batchnorm_relu_gb300 import tokens

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GUARD = 7.0


def sections(pairs):
    t = pairs // 4
    h = (pairs - t) // 2
    return (t, h, pairs - t - h)


def table(pairs, **kw):
    return tokens.rotary_table(sections(pairs), **kw)


def randn(*shape, dtype="f32", seed=0):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(DT[dtype]).cuda()


def positions(batch, n, seed=0, far=1000):
    g = torch.Generator().manual_seed(seed)
    return torch.randint(0, far, (batch, n, 3), generator=g, dtype=torch.int32).cuda()


def check(q, k, pos, freq, axis, layout, **kw):
    for back, f in ((False, tokens.rotary_forward), (True, tokens.rotary_backward)):
        got = f(q, k, pos, freq, axis, layout=layout, **kw)
        torch.cuda.synchronize()
        for name, a, o in (("q", q, got[0]), ("k", k, got[1])):
            if a is None:
                assert o is None
                continue
            want, bound = ref.rotary(a, pos, freq, axis, layout, back)
            ref.close(o, want, bound, name, a.dtype)
    return got


@pytest.mark.parametrize("layout", ["halves", "neighbours"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("batch,n,hq,hk,d,rot", [(1, 1, 1, 1, 2, 2), (1, 1, 16, 4, 128, 128), (2, 5, 3, 1, 6, 4),
                                                 (1, 37, 4, 4, 64, 64), (2, 19, 12, 12, 80, 72), (1, 9, 8, 2, 96, 96),
                                                 (1, 3, 1, 1, 1024, 1024), (3, 33, 5, 1, 40, 34), (1, 65, 2, 1, 256, 128),
                                                 (1, 300, 1, 1, 7, 6), (1, 700, 7, 1, 72, 72)])
def test_matches_plain_form(batch, n, hq, hk, d, rot, dtype, layout):
    q, k = randn(batch, n, hq, d, dtype=dtype, seed=1), randn(batch, n, hk, d, dtype=dtype, seed=2)
    freq, axis = table(rot // 2)
    check(q, k, positions(batch, n), freq, axis, layout)


@pytest.mark.parametrize("order", ["blocks", "cycled"])
@pytest.mark.parametrize("spectrum", ["shared", "own"])
def test_tables(order, spectrum):
    freq, axis = tokens.rotary_table((8, 12, 12), theta=500.0, order=order, spectrum=spectrum)
    counts = [int((axis == a).sum()) for a in range(3)]
    assert counts == [8, 12, 12]
    q = randn(1, 24, 2, 64, seed=3)
    check(q, None, positions(1, 24), freq, axis, "halves")
    check(None, q, positions(1, 24), freq, axis, "neighbours")


@pytest.mark.parametrize("axes", [1, 2, 4, 8])
def test_other_numbers_of_axes(axes):
    freq, axis = tokens.rotary_table([4] * axes)
    g = torch.Generator().manual_seed(4)
    pos = torch.randint(-500, 500, (2, 11, axes), generator=g, dtype=torch.int32).cuda()
    q = randn(2, 11, 3, 8 * axes, dtype="f16", seed=5)
    check(q, q, pos, freq, axis, "halves")


def test_far_and_negative_positions_lose_nothing():
    freq, axis = table(64)
    far = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 24 + 1, -1, 0, 123456789], dtype=torch.int32)
    pos = far[:, None].expand(6, 3)[None].contiguous().cuda()
    q = randn(1, 6, 2, 128, seed=6)
    check(q, q, pos, freq, axis, "halves")


def test_positions_repeated_over_the_batch():
    freq, axis = table(16)
    q = randn(3, 12, 2, 32, seed=7)
    pos = tokens.grid_positions(2, 3, 2)
    assert pos.tolist() == [[t, y, x] for t in range(2) for y in range(3) for x in range(2)]
    a = check(q, q, pos, freq, axis, "halves")
    b = check(q, q, pos[None].expand(3, -1, -1), freq, axis, "halves")
    c = check(q, q, pos[None], freq, axis, "halves")
    assert torch.equal(a[0], b[0]) and torch.equal(a[0], c[0])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("layout", ["halves", "neighbours"])
def test_views_of_a_fused_product_and_head_major_order(dtype, layout):
    freq, axis = table(20)
    pos = positions(2, 21)
    qkv = randn(2, 21, 6 + 2 * 3, 40, dtype=dtype, seed=8)
    check(qkv[:, :, :6], qkv[:, :, 6:9], pos, freq, axis, layout)
    major = randn(2, 5, 21, 40, dtype=dtype, seed=9).transpose(1, 2)      # [batch][heads][tokens] in memory
    check(major, major, pos, freq, axis, layout)
    odd = randn(2, 21, 5, 43, dtype=dtype, seed=10)[..., 1:41]           # odd strides, off the alignment
    check(odd, odd, pos, freq, axis, layout)
    # into views of another buffer, whose other elements stay as they were
    buf = torch.full((2, 21, 5, 47), GUARD, dtype=DT[dtype], device="cuda")
    out = (buf[..., 1:41], torch.empty_like(odd, memory_format=torch.contiguous_format))
    tokens.rotary_forward(odd, odd, pos, freq, axis, layout=layout, out=out)
    want = tokens.rotary_forward(odd, odd, pos, freq, axis, layout=layout)
    assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])
    out[0].fill_(GUARD)
    assert bool((buf == GUARD).all())


@pytest.mark.parametrize("layout", ["halves", "neighbours"])
@pytest.mark.parametrize("rot", [64, 48, 6])
def test_in_place(layout, rot):
    freq, axis = tokens.rotary_table((rot // 2,))
    pos = positions(2, 17)[..., :1]
    qkv = randn(2, 17, 8, 64, dtype="bf16", seed=11)
    want = tokens.rotary_forward(qkv[:, :, :4], qkv[:, :, 4:6], pos, freq, axis, layout=layout)
    rest = qkv[:, :, 6:].clone()
    q, k = qkv[:, :, :4], qkv[:, :, 4:6]
    tokens.rotary_forward(q, k, pos, freq, axis, layout=layout, out=(q, k))
    assert torch.equal(q, want[0]) and torch.equal(k, want[1]) and torch.equal(qkv[:, :, 6:], rest)


def test_backward_is_the_transpose():
    """<forward(a), b> = <a, backward(b)>, in 32 bits: a sum of n products good to its roundings."""
    freq, axis = table(32)
    pos = positions(2, 50)
    a, b = randn(2, 50, 3, 64, seed=12), randn(2, 50, 3, 64, seed=13)
    fa, _ = tokens.rotary_forward(a, None, pos, freq, axis)
    bb, _ = tokens.rotary_backward(b, None, pos, freq, axis)
    left, right = float((fa.double() * b).sum()), float((a.double() * bb).sum())
    assert abs(left - right) <= 16 * 2.0 ** -24 * float((a.double().abs() * b.abs()).sum() * 2)
    # and undoes the rotation
    back, _ = tokens.rotary_backward(fa, None, pos, freq, axis)
    assert float((back - a).abs().max()) <= 32 * 2.0 ** -24 * float(a.abs().max()) * 2


def test_nan_and_infinity_stay_in_their_pair():
    freq, axis = table(16)
    pos = positions(1, 4)
    q = randn(1, 4, 2, 40, seed=14)
    want = tokens.rotary_forward(q, None, pos, freq, axis)[0]
    q[0, 1, 0, 3] = float("nan")
    q[0, 2, 1, 39] = float("inf")          # past the rotated part: copied
    got = tokens.rotary_forward(q, None, pos, freq, axis)[0]
    touched = torch.zeros_like(q, dtype=torch.bool)
    touched[0, 1, 0, 3] = touched[0, 1, 0, 19] = True
    touched[0, 2, 1, 39] = True
    assert torch.equal(got[~touched], want[~touched])
    assert bool(torch.isnan(got[0, 1, 0, [3, 19]]).all()) and float(got[0, 2, 1, 39]) == float("inf")


def test_an_axis_outside_the_positions_is_the_last():
    freq, axis = table(8)
    pos = positions(1, 5)
    q = randn(1, 5, 1, 16, seed=15)
    wild = axis.clone()
    wild[wild == 2] = 200
    a, b = (tokens.rotary_forward(q, None, pos, freq, x)[0] for x in (axis, wild))
    assert torch.equal(a, b)


def test_other_stream():
    freq, axis = table(64)
    q, k, pos = randn(1, 500, 8, 128, seed=16), randn(1, 500, 2, 128, seed=17), positions(1, 500)
    first = tokens.rotary_forward(q, k, pos, freq, axis)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = tokens.rotary_forward(q, k, pos, freq, axis)
    side.synchronize()
    assert torch.equal(first[0], second[0]) and torch.equal(first[1], second[1])


def test_no_tokens():
    freq, axis = table(8)
    q = torch.empty(2, 0, 3, 16, device="cuda")
    out = tokens.rotary_forward(q, q, torch.empty(0, 3, dtype=torch.int32, device="cuda"), freq, axis)
    assert out[0].shape == q.shape


def test_refusals():
    freq, axis = table(8)
    q, pos = randn(1, 4, 2, 16), positions(1, 4)
    bad = pytest.raises(tokens.CBRError)
    with bad:
        tokens.rotary_forward(None, None, pos, freq, axis)
    with bad:
        tokens.rotary_forward(q[..., :12], None, pos, freq, axis)          # fewer elements than pairs
    with bad:
        tokens.rotary_forward(q.double(), None, pos, freq, axis)
    with bad:
        tokens.rotary_forward(q, q[:, :3], pos, freq, axis)
    with bad:
        tokens.rotary_forward(q, q.half(), pos, freq, axis)
    with bad:
        tokens.rotary_forward(q, None, pos.long(), freq, axis)
    with bad:
        tokens.rotary_forward(q, None, pos[:, :3], freq, axis)
    with bad:
        tokens.rotary_forward(q, None, pos, freq[:4], axis)
    with bad:
        tokens.rotary_forward(q, None, pos, freq, axis, layout="quarters")
    with bad:
        tokens.rotary_forward(q.transpose(2, 3), None, pos, freq, axis)
    with bad:
        tokens.rotary_forward(q, None, pos, freq, axis, out=(torch.zeros(1, 4, 1, 16, device="cuda").expand(1, 4, 2, 16), None))
    with bad:
        tokens.rotary_forward(q.cpu(), None, pos, freq, axis)

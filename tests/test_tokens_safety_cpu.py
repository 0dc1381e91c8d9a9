"""Refusals that keep the token operators' kernels inside their buffers and apart from one another, on fake
addresses: nothing gets as far as a launch."""
import pytest

from test_tokens_cpu import P, distill_desc, fb, lib, nb, nf, norm_desc, rot, rotary_desc  # noqa: F401

DEVICE_OR_OK = (0, 5)   # refused for want of a device only
FAR = 1 << 40


def test_rows_times_strides_stay_in_64_bits(lib):  # noqa: F811
    """Each size passes its own limit; their product, in bytes, does not fit an address."""
    for kw in (dict(rows=FAR, ls=FAR), dict(rows=FAR, ds=FAR), dict(rows=FAR, ids=FAR), dict(rows=FAR, tops=FAR),
               dict(rows=1 << 22, ls=FAR)):
        assert fb(lib, distill_desc(**kw)) == 1, kw
    assert fb(lib, distill_desc(rows=1 << 18, ls=FAR)) in DEVICE_OR_OK
    assert fb(lib, distill_desc(rows=1, ls=FAR)) in DEVICE_OR_OK
    for i in range(4):
        strides = [64] * 8
        strides[i] = FAR
        assert nf(lib, norm_desc(rows=FAR, gate_rows=1, strides=strides)) == 1, i
    for i in (1, 2, 4, 5, 6, 7):
        strides = [64] * 8
        strides[i] = FAR
        assert nb(lib, norm_desc(rows=FAR, gate_rows=1, strides=strides)) == 1, i
    for kw in (dict(q=(FAR, 128, 64)), dict(k=(FAR, 64, 64)), dict(qo=(FAR, 128, 64)), dict(ko=(FAR, 64, 64)),
               dict(pos=(FAR, 3, 1))):
        assert rot(lib, rotary_desc(batch=FAR, n=1, **kw)) == 1, kw
    assert rot(lib, rotary_desc(n=1 << 19, q=(640, FAR, 64))) == 1
    assert rot(lib, rotary_desc(hq=65536, q=(FAR, 128, FAR))) in DEVICE_OR_OK

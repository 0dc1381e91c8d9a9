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
    assert rot(lib, rotary_desc(batch=1, hq=65536, q=(FAR, 128, FAR))) in DEVICE_OR_OK


# batch 2, 5 tokens, 2 heads of q and 1 of k, 64 wide
@pytest.mark.parametrize("strides", [
    (640, 64, 64),          # a token's second head is the next token's first
    (640, 64, 320 - 64),    # the second head of the first token is the fifth token's first
    (320, 128, 64),         # the second batch begins in the first one's third token
    (192, 128, 64), (128, 128, 64), (640, 128, 128), (640, 96, 64)])
def test_rotary_outputs_that_overlap_are_refused(lib, strides):  # noqa: F811
    assert rot(lib, rotary_desc(qo=strides)) == 1


@pytest.mark.parametrize("strides", [
    (640, 128, 64), (640, 64, 320), (128, 256, 64), (64, 256, 128), (64, 128, 640), (1000, 200, 100), (10240, 1024, 512)])
def test_rotary_outputs_in_any_order_of_axes_are_taken(lib, strides):  # noqa: F811
    assert rot(lib, rotary_desc(qo=strides)) in DEVICE_OR_OK


def test_axes_of_one_step_may_have_any_stride(lib):  # noqa: F811
    assert rot(lib, rotary_desc(batch=1, n=1, hq=1, qo=(0, 0, 0), ko=(0, 1, 2))) in DEVICE_OR_OK
    assert rot(lib, rotary_desc(batch=1, qo=(7, 128, 64))) in DEVICE_OR_OK


def test_temperatures_at_the_end_of_the_range(lib):  # noqa: F811
    """The kernels' exponents have the factor log2(e) / T; where it is infinite a difference of 0 would be NaN."""
    assert fb(lib, distill_desc(temp=4e-39)) == 1      # 1 / T is finite yet
    assert fb(lib, distill_desc(temp=5e-39)) in DEVICE_OR_OK
    assert fb(lib, distill_desc(temp=3e38)) in DEVICE_OR_OK


def test_no_exception_leaves_an_entry(tmp_path):
    """The guard around every entry's body: a status for what it returns, CBR_ERR_CUDA for what it throws."""
    import os
    import re
    import shutil
    import subprocess

    from conv_batchnorm_relu_gb300 import build
    src = tmp_path / "g.cpp"
    src.write_text('#include <new>\n#include "token_ops.h"\nint main() {\n'
                   '  if (cbr::guarded([] { return 3; }) != CBR_ERR_UNSUPPORTED) return 1;\n'
                   '  if (cbr::guarded([]() -> int { throw std::bad_alloc(); }) != CBR_ERR_CUDA) return 2;\n'
                   '  return 0;\n}\n')
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(shutil.which("nvcc") or build._nvcc()))), "include")
    exe = str(tmp_path / "g")
    subprocess.run(["g++", "-std=c++17", "-I", build.CSRC, "-I", cuda, str(src), "-o", exe], check=True)
    assert subprocess.run([exe]).returncode == 0
    text = open(os.path.join(build.CSRC, "tokens_api.cu")).read()
    entries = re.findall(r"^cbr_status_t cbr_\w+\([^)]*\) \{\n(.*)$", text, re.M)
    assert len(entries) == 8 and all(e.strip().startswith("return guarded(") for e in entries)

"""Attention's scale over its whole range, 0 among it, with scores near the end of fp32's."""
import ctypes

import pytest

from test_gpu_attention import check, make

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("scale", [0.0, 1e-43, 1e-40, 2e-37, 1e-36, 1e-34])
@pytest.mark.parametrize("tq,tk,hq,dim,causal", [(140, 270, 2, 64, False), (300, 300, 1, 128, True), (1, 3000, 4, 128, False)])
def test_small_scales_of_large_scores(tq, tk, hq, dim, causal, scale):
    """Products up to 1e37: a scale below 1e-35 is taken as it is, and 0 makes every key alike."""
    # (the argument is an fp32 number: 1e-43 is 71.4 steps of 2^-149, and the call's scale 71 of them)
    check(make(2, tq, tk, hq, 1, dim, "bf16", seed=41, size=4e17), causal, ctypes.c_float(scale).value)

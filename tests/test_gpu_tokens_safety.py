"""What the token operators' binding must not hand to a kernel: memory of another device, workspaces that
are shorter than they look, numbers that a descriptor cannot hold."""
import pytest
import torch

from conv_batchnorm_relu_gb300 import tokens

pytestmark = pytest.mark.gpu


def test_a_workspace_elsewhere_or_shorter_than_it_looks_is_refused():
    x, w = torch.randn(12, 64, device="cuda"), torch.ones(64, device="cuda")
    stats = tokens.block_norm_forward(x, pre_weight=w)["stats"]
    n = tokens.block_norm_workspace_size(12, 64, torch.float32)
    want = tokens.block_norm_backward(None, x, x, pre_weight=w, stats=stats)

    def call(ws):
        return tokens.block_norm_backward(None, x, x, pre_weight=w, stats=stats, ws=ws)

    for ws in (torch.zeros(n, dtype=torch.uint8), torch.zeros(16, dtype=torch.uint8, device="cuda").repeat(1, 1).expand(n, 16),
               torch.zeros(1, dtype=torch.uint8, device="cuda").expand(n),
               torch.zeros(2 * n, dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(tokens.CBRError):
            call(ws)
    for dtype, size in ((torch.uint8, 1), (torch.float32, 4)):
        got = call(torch.zeros(n // size, dtype=dtype, device="cuda"))
        assert torch.equal(got["dx"], want["dx"]) and torch.equal(got["dpre_weight"], want["dpre_weight"])


@pytest.mark.parametrize("value", [1e39, -1e39, float("inf"), float("nan")])
def test_numbers_that_32_bits_cannot_hold_are_refused(value):
    x, w = torch.randn(3, 64, device="cuda"), torch.ones(64, device="cuda")
    ids = torch.zeros(3, 1, dtype=torch.int32, device="cuda")
    stats = torch.zeros(3, 4, device="cuda")
    with pytest.raises(tokens.CBRError):
        tokens.distill_forward(x, ids, x[:, :1], temperature=value)
    with pytest.raises(tokens.CBRError):
        tokens.block_norm_forward(x, pre_weight=w, eps=value)
    for name in ("residual_scale", "branch_scale"):
        with pytest.raises(tokens.CBRError):
            tokens.block_norm_forward(x, x, w, None, w, **{name: value})
        with pytest.raises(tokens.CBRError):
            tokens.block_norm_backward(x, x, x, x, w, None, w, stats, **{name: value})

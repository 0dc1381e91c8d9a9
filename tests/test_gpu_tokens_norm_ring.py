"""The norms' backward with many rows a block: its ring of rows in shared memory filled again and again, runs
of whole gates, gates that end inside a run, beside the forms without a ring at the same sizes."""
import pytest
import torch

from test_gpu_tokens_norm import check_backward, forward, make

pytestmark = pytest.mark.gpu


# on 152 SMs: 12000x512 about 10 rows a block and 6 of the ring, 6000x1024 10 and 6, 3001x4096 20 and 6, 2400x8192 16 and 3
@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("rows,dim,groups", [
    (12000, 512, 0), (12000, 512, 1), (12000, 512, 12000), (12000, 512, 3000), (6000, 1024, 24), (6000, 1024, 3000),
    (3001, 4096, 1), (3000, 4096, 8), (3000, 4096, 1500), (2400, 8192, 5)], ids=lambda v: str(v))
def test_more_rows_a_block_than_the_ring_holds(rows, dim, groups, dtype, kind):
    s, g = make(rows, dim, dtype, 4000 + rows + groups, "both", groups)
    check_backward(s, forward(s, kind), kind, g)


@pytest.mark.parametrize("form", ["pre", "post"])
@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_halves_of_the_operator_through_the_ring(kind, form):
    s, g = make(9000, 768, "bf16", 4100, form, 9)
    check_backward(s, forward(s, kind), kind, g)


@pytest.mark.parametrize("dtype,dim", [("f32", 512), ("bf16", 515), ("f16", 64), ("f32", 1024)])
def test_many_rows_without_a_ring(dtype, dim):
    for groups in (0, 40, 6000):
        s, g = make(12000, dim, dtype, 4200 + groups, "both", groups)
        check_backward(s, forward(s, "layer"), "layer", g)


def test_rows_apart_through_the_ring():
    """Rows with a stride of their own, still whole 16-byte vectors."""
    s, g = make(7000, 640, "bf16", 4300, "both", 7, stride=656)
    check_backward(s, forward(s, "rms"), "rms", g, stride=656)


def test_repeats_bit_for_bit_while_the_ring_goes_round():
    s, g = make(8192, 2048, "f16", 4400, "both", 8)
    _, _, first = check_backward(s, forward(s, "rms"), "rms", g)
    assert all(bool(torch.isfinite(t).all()) for t in first.values())

"""The distillation's numbers at the ends of their range: logits of any magnitude."""
import math

import pytest
import torch

import token_reference as ref
from test_gpu_tokens_distill import DT, compare, make

pytestmark = pytest.mark.gpu

LOG2E = 1.4426950408889634


# ------------------------------------------------------------------------------- large magnitudes

@pytest.mark.parametrize("rows", [1, 9])
@pytest.mark.parametrize("value", [-1e9, -1e10, -3e12, -1e20, -1e30, -3e37, 1e10, 1e20, 1e30])
def test_rows_of_one_large_value_are_uniform(value, rows):
    """A mask need not be the type's lowest value: a softmax of equal logits is uniform, whatever they are."""
    _, ids, top, lse = make(rows, 777, 4, "f32", 31, True)
    logits = torch.full((rows, 777), value, device="cuda")
    compare(logits, ids, top)
    compare(logits, ids, top, lse, temperature=2.0)


@pytest.mark.parametrize("rows", [2, 9])
@pytest.mark.parametrize("mask", [-1e9, -1e12, -1e30, -3e38])
def test_masked_words_beside_ordinary_ones(mask, rows):
    """Ordinary logits after, before and between words masked with a large negative number."""
    logits, ids, top, lse = make(rows, 5003, 6, "f32", 32, True)
    logits[0, :4000] = mask
    logits[1, 1000:] = mask
    logits[-1, ::2] = mask
    ids[:] = torch.tensor([4001, 4501, 5002, 1, 999, 3], device="cuda")
    ids[0] = torch.tensor([4001, 4501, 5002, 4444, 4203, 4701], device="cuda")
    ids[1] = torch.tensor([1, 3, 5, 998, 500, 2], device="cuda")
    ids[-1] = torch.tensor([1, 3, 5, 997, 501, 5001], device="cuda")
    compare(logits, ids, top)
    compare(logits, ids, top, lse)


@pytest.mark.parametrize("temperature", [2.0 ** -7, 1.0, 20.0])
@pytest.mark.parametrize("sign", [-1, 1])
def test_logits_about_every_power_of_two(sign, temperature):
    """Differences of a few units of the last place of a large common value: exact in 32 bits, so the
    probabilities are good to their roundings at any magnitude."""
    g = torch.Generator().manual_seed(33)
    powers = list(range(4, 40, 3)) + [20, 21, 22, 23]
    _, ids, top, _ = make(len(powers), 1201, 5, "f32", 34)
    lse = torch.logsumexp(top / temperature, 1) + 0.25
    logits = torch.empty(len(powers), 1201)
    for i, e in enumerate(powers):
        # a step that is a whole number of units, about a temperature wide
        unit = max(2.0 ** (e - 22), 2.0 ** math.floor(math.log2(temperature)))
        steps = torch.randint(-6, 7, (1201,), generator=g)
        logits[i] = sign * temperature / LOG2E * 2.0 ** e
        logits[i] = (logits[i] / unit).round() * unit + steps * unit
    compare(logits.cuda(), ids, top, lse, temperature=temperature)
    compare(logits.flip(1).cuda(), ids, top, temperature=temperature)

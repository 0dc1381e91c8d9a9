"""The distillation's numbers at the ends of their range: logits of any magnitude, teachers whose
logits have a common offset."""
import math

import pytest
import torch

import token_reference as ref
from conv_batchnorm_relu_gb300 import tokens
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


# ------------------------------------------------------------------------------- the teacher's offset

@pytest.mark.parametrize("temperature", [1.0, 2.0, 3.0])
def test_an_offset_of_the_teachers_logits_changes_nothing(temperature):
    """Over its entries alone a teacher is a softmax: logits and offset on a grid whose sums are exact give
    the same differences, and so the same results bit for bit."""
    logits, ids, _, _ = make(6, 1000, 10, "f32", 35)
    top = torch.randint(-160, 160, (6, 10), generator=torch.Generator().manual_seed(36)).float().cuda() / 32
    want = tokens.distill_forward_backward(logits, ids, top, temperature=temperature)
    for offset in (30.0, 300.0, -300.0, 3000.0, 65536.0):
        got = tokens.distill_forward_backward(logits, ids, top + offset, temperature=temperature)
        assert torch.equal(got["loss"], want["loss"]) and torch.equal(got["dlogits"], want["dlogits"]), offset


@pytest.mark.parametrize("temperature", [1.0, 2.0, 3.0])
def test_far_teachers_keep_their_bits(temperature):
    """Bounds that know differences of the teacher's logits only: with d = (t - largest) / T,
    a log p is off by 3 |d| w (a difference, 1 / T, a product) and by the logarithm of a sum of k terms,
    whose exponentials are off by as much and 2 roundings, (k / 32 + 16) w with their sum's; a log q by the same
    with v terms and a factor log2(e) / T of 3 roundings; the loss is their sum's, weighted with p, and the
    product's and the sum's roundings on top."""
    v, k = 64, 8
    logits, ids, top, _ = make(7, v, k, "f32", 37)
    top = top + 3000.0
    want = ref.distill(logits, ids, top, temperature)
    t = top.cpu().double() / temperature
    d = t - t.max(1, keepdim=True).values
    p = torch.softmax(t, 1)
    x = logits.cpu().double() / temperature
    dx = (x - x.max(1, keepdim=True).values).gather(1, ids.cpu().long())
    log_p, log_q = torch.log_softmax(t, 1), torch.log_softmax(x, 1).gather(1, ids.cpu().long())
    each_p = (3 * d.abs() + 3 * d.abs().max(1, keepdim=True).values) * ref.W + ref.rounds(k) + 4 * ref.W
    each_q = (6 * dx.abs() + 6 * x.abs().max()) * ref.W + ref.rounds(v) + 4 * ref.W
    mag = (p * (log_p.abs() + log_q.abs()))
    want["loss_bound"] = (p * (each_p * (1 + (log_p - log_q).abs()) + each_q) + mag * ref.rounds(k)).sum(1) * temperature ** 2
    got = tokens.distill_forward_backward(logits, ids, top, temperature=temperature)
    ref.close(got["loss"], want["loss"], want["loss_bound"], "loss")

"""The distillation's numbers at the ends of their range: logits of any magnitude, teachers whose
logits have a common offset, unlisted words that hold next to nothing of the student's mass."""
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


# ------------------------------------------------------------------------------- hardly any unlisted mass

def faint(rows, vocab, k, dtype, seed, gap, temperature, pad):
    """Students whose listed words stand gap * temperature above all others; the last columns are padding."""
    logits, ids, top, lse = make(rows, vocab, k, dtype, seed, True)
    lse = torch.logsumexp(top.float() / temperature, 1) + 0.1 + torch.rand(
        rows, generator=torch.Generator().manual_seed(seed + 1)).cuda()
    ids = (ids.long() % (vocab - pad)).to(ids.dtype)
    logits.scatter_(1, ids.long(), (logits.float().gather(1, ids.long()) + gap * temperature).to(logits.dtype))
    if pad:
        logits[:, vocab - pad:] = -math.inf
    return logits, ids, top, lse


def faint_reference(logits, ids, top, lse, weight, temperature):
    """The plain form, with bounds for a tail that is computed relative to its own largest word: an unlisted
    word's share of the unlisted mass is off by the roundings of sums and by w for each unit of the exponents
    that enter, and by an exponential lost below the normal range (2^-126 of the largest)."""
    want = ref.distill(logits, ids, top, temperature, lse, weight)
    z = logits.cpu().double() / temperature
    r, v = z.shape
    per = ref.rounds(v) + ref.rounds(ids.shape[1]) + 16 * ref.W
    listed = torch.zeros(r, v, dtype=torch.bool).scatter_(1, ids.cpu().long(), True)
    t = top.cpu().double() / temperature
    p = torch.exp(t - lse.cpu().double()[:, None])
    full = torch.zeros(r, v, dtype=torch.float64).scatter_add_(1, ids.cpu().long(), p)
    log_q = torch.log_softmax(z, 1)
    own = torch.softmax(z.masked_fill(listed, -math.inf), 1)
    spread = (z.max(1, keepdim=True).values - z.masked_fill(listed, -math.inf).max(1, keepdim=True).values).abs()
    size = (1 + log_q.abs().nan_to_num(0, 0, 0)) * per
    bound = torch.exp(log_q) * size * (p.sum(1, keepdim=True) + 1) + full * (1 + t.abs().max(1, keepdim=True).values) * per
    bound = bound + torch.where(listed, 0.0, own * (p.sum(1, keepdim=True) + 1) * (2 + spread) * (size + per)) + 2.0 ** -126
    w = torch.ones(r, dtype=torch.float64) if weight is None else weight.cpu().double()
    want["grad_bound"] = bound * w.abs()[:, None] * temperature
    u = want["stats"][:, 2]
    tail = u < 2.0 ** -64
    want["stats"][:, 2] = torch.where(tail & (u > 0), torch.log2(u.clamp(min=1e-320)), u)
    return want


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("gap", [20, 40, 60, 80, 90, 100, 130, 400, 700])
@pytest.mark.parametrize("rows,vocab,k,pad", [(2, 4099, 20, 7), (6, 1000, 10, 100), (5, 300, 6, 0)], ids=lambda v: str(v))
def test_a_tail_of_hardly_any_mass(rows, vocab, k, pad, gap, dtype):
    """The loss has its logarithm and the unlisted words share its gradient, however small it is."""
    temperature = 2.5
    logits, ids, top, lse = faint(rows, vocab, k, dtype, 38 + gap, gap, temperature, pad)
    for weight in (None, torch.full((rows,), 4096.0 / 3, device="cuda")):
        want = faint_reference(logits, ids, top, lse, weight, temperature)
        compare(logits, ids, top, lse, weight, temperature, want)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("scale", [1e9, 1e15, 1e22])
def test_large_scales_of_a_faint_tail(scale, dtype):
    """The factor of an unlisted word's exponential passes the range of 32 bits long before its gradient."""
    logits, ids, top, lse = faint(6, 515, 8, dtype, 39, 35, 4.0, 15)
    w = torch.full((6,), scale, device="cuda")
    if dtype == "f16":
        w.fill_(1024.0)
    want = faint_reference(logits, ids, top, lse, w, 4.0)
    compare(logits, ids, top, lse, w, 4.0, want)


def test_no_tail_below_the_range():
    """Words masked with a large negative number are as good as not there, as those at -infinity are."""
    for dtype in DT:
        logits, ids, top, lse = faint(6, 515, 8, dtype, 40, 10, 1.0, 15)
        low, none = logits.clone(), logits.clone()
        listed = torch.zeros_like(logits, dtype=torch.bool).scatter_(1, ids.long(), True)
        low[~listed], none[~listed] = torch.finfo(DT[dtype]).min, -math.inf
        a = tokens.distill_forward_backward(low, ids, top, teacher_lse=lse)
        b = tokens.distill_forward_backward(none, ids, top, teacher_lse=lse)
        assert torch.equal(a["loss"], b["loss"]) and torch.equal(a["dlogits"], b["dlogits"])
        compare(low, ids, top, lse)

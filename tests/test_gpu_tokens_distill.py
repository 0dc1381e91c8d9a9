"""Distillation from a teacher's top logits against its plain 64-bit form: types, odd vocabularies,
strides and alignments, masked and empty rows, infinities and NaN, gradients against differences."""
import math

import pytest
import torch

import token_reference as ref
from conv_batchnorm_relu_gb300 import tokens

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
GUARD = 7.0


def make(rows, vocab, k, dtype, seed, tail=False, stride=None, shift=0, id_dtype=torch.int32, top_dtype=None):
    """Inputs on the GPU; logits as a view with a row stride, `shift` elements off the allocation's start."""
    g = torch.Generator().manual_seed(seed)
    stride = stride or vocab
    buf = torch.randn(rows * stride + shift, generator=g).mul_(2).to(DT[dtype]).cuda()
    logits = torch.as_strided(buf, (rows, vocab), (stride, 1), shift)
    ids = torch.stack([torch.randperm(vocab, generator=g)[:k] for _ in range(rows)]) if rows else torch.zeros(0, k)
    ids = ids.reshape(rows, k).to(id_dtype).cuda()
    top = (torch.randn(rows, k, generator=g) * 2 + 3).to(top_dtype or DT[dtype]).cuda()
    lse = None
    if tail:
        lse = torch.logsumexp(top.float(), 1) + torch.rand(rows, generator=g).cuda() if k else torch.zeros(rows).cuda()
    return logits, ids, top, lse


def compare(logits, ids, top, lse=None, weight=None, temperature=1.0, want=None):
    """All three calls against the plain form, and against one another."""
    want = want or ref.distill(logits, ids, top, temperature, lse, weight)
    kw = dict(temperature=temperature, teacher_lse=lse, row_weight=weight)
    both = tokens.distill_forward_backward(logits, ids, top, **kw)
    fwd = tokens.distill_forward(logits, ids, top, **kw)
    grad = tokens.distill_backward(None, logits, ids, top, fwd["stats"], **kw)
    torch.cuda.synchronize()
    for name, loss in (("loss (one call)", both["loss"]), ("loss", fwd["loss"])):
        ref.close(loss, want["loss"], want["loss_bound"], name)
    for name, d in (("dlogits (one call)", both["dlogits"]), ("dlogits", grad)):
        ref.close(d, want["dlogits"], want["grad_bound"], name, logits.dtype)
    ref.close(fwd["stats"], want["stats"], want["stats"].abs().nan_to_num(0, 0, 0) * 2 * ref.rounds(logits.shape[1]), "stats")
    return want, both, fwd, grad


SHAPES = [(1, 1, 1), (3, 2, 2), (5, 7, 3), (2, 8, 8), (4, 64, 5), (9, 257, 33), (16, 1000, 10), (3, 2049, 128),
          (2, 4096, 64), (2, 50257, 33), (1, 65536, 1), (2, 100003, 300), (1, 131072, 128), (3, 8191, 1024)]


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("tail", [False, True], ids=["renormalised", "tail"])
@pytest.mark.parametrize("rows,vocab,k", SHAPES, ids=lambda v: str(v))
def test_matches_plain_form(rows, vocab, k, dtype, tail):
    logits, ids, top, lse = make(rows, vocab, k, dtype, 100 + vocab, tail)
    compare(logits, ids, top, lse, temperature=1.0 if vocab % 2 else 2.5)


@pytest.mark.parametrize("dtype", list(DT))
def test_many_rows(dtype):
    """More rows than blocks, so that each block works through several."""
    logits, ids, top, lse = make(2500, 515, 9, dtype, 7, True)
    w = torch.rand(2500, generator=torch.Generator().manual_seed(1)).cuda()
    w[::5] = 0
    compare(logits, ids, top, lse, w, 2.0)


@pytest.mark.parametrize("vocab", [333, 40960, 50257])
def test_more_rows_than_fit_at_once_on_wide_vocabularies(vocab):
    logits, ids, top, lse = make(330, vocab, 17, "bf16", 8, True)
    want, both, fwd, grad = compare(logits[:6], ids[:6], top[:6], lse[:6])
    all_rows = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)
    # a row's result does not depend on which rows are beside it
    assert torch.equal(all_rows["dlogits"][:6], both["dlogits"]) and torch.equal(all_rows["loss"][:6], both["loss"])
    last = tokens.distill_forward_backward(logits[-5:], ids[-5:], top[-5:], teacher_lse=lse[-5:])
    assert torch.equal(all_rows["dlogits"][-5:], last["dlogits"]) and torch.equal(all_rows["loss"][-5:], last["loss"])


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("vocab,stride,shift", [(1000, 1003, 1), (517, 520, 3), (2048, 2049, 0), (40001, 40016, 5)])
def test_strides_and_alignment(dtype, vocab, stride, shift):
    logits, ids, top, lse = make(5, vocab, 12, dtype, 3, True, stride=stride, shift=shift)
    compare(logits, ids, top, lse)
    # an output with its own stride and phase, whose gaps stay as they were
    for out_stride, out_shift in ((stride, shift), (vocab + 6, 2)):
        buf = torch.full((5 * out_stride + out_shift + 8,), GUARD, dtype=DT[dtype], device="cuda")
        out = torch.as_strided(buf, (5, vocab), (out_stride, 1), out_shift)
        tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse, out={"dlogits": out})
        expected = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)["dlogits"]
        assert torch.equal(out, expected)
        out.fill_(GUARD)
        assert bool((buf == GUARD).all())


def test_other_types_of_entries():
    for id_dtype in (torch.int32, torch.int64):
        for top_dtype in DT.values():
            logits, ids, top, lse = make(4, 700, 20, "bf16", 5, True, id_dtype=id_dtype, top_dtype=top_dtype)
            compare(logits, ids, top, lse, temperature=3.0)
    # entries as columns of a wider tensor
    logits, ids, top, lse = make(4, 700, 20, "f16", 6)
    compare(logits, ids[:, 3:11], top[:, 3:11])


def test_absent_entries_and_empty_rows():
    logits, ids, top, lse = make(8, 300, 6, "f32", 9, True)
    ids[0] = -1                                        # nothing listed
    ids[1, 3:] = -5
    ids[2, 0], ids[2, 1] = 300, 2 ** 31 - 1            # outside the vocabulary
    top[0], top[1, 3:], top[2, :2] = math.nan, math.nan, math.inf
    top[3] = -math.inf                                 # no mass (renormalised: an empty row)
    top[4, 2] = -math.inf
    for l in (None, lse):
        want, both, fwd, grad = compare(logits, ids, top, l)
        assert float(both["loss"][0]) == 0 and not bool(both["dlogits"][0].any()) and not bool(fwd["stats"][0].any())
        if l is None:
            assert float(both["loss"][3]) == 0 and not bool(both["dlogits"][3].any())


def test_no_entries_at_all():
    logits, ids, top, _ = make(3, 50, 0, "bf16", 2)
    for lse in (None, torch.zeros(3, device="cuda")):
        both = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)
        assert not bool(both["loss"].any()) and not bool(both["dlogits"].any())


def test_every_word_listed():
    logits, ids, top, lse = make(4, 40, 40, "f32", 12, True)
    compare(logits, ids, top, lse)      # no tail class: no mass outside the listed words
    compare(logits, ids, top)


def test_repeated_ids_add_up():
    logits, ids, top, lse = make(3, 500, 10, "f32", 13, True)
    ids[0, 4], ids[1, :] = ids[0, 2], ids[1, 0]
    compare(logits, ids, top, lse)
    compare(logits, ids, top)


@pytest.mark.parametrize("dtype", list(DT))
def test_masked_rows_are_zero_whatever_they_hold(dtype):
    logits, ids, top, lse = make(6, 1025, 8, dtype, 14, True)
    logits[1], logits[3] = math.nan, math.inf
    top[1] = math.nan
    lse[3] = math.nan
    w = torch.tensor([1.0, 0.0, 0.5, 0.0, 2.0, 0.0], device="cuda")
    want, both, fwd, grad = compare(logits, ids, top, lse, w)
    for i in (1, 3, 5):
        assert float(both["loss"][i]) == 0 and not bool(both["dlogits"][i].any()) and not bool(fwd["stats"][i].any())


@pytest.mark.parametrize("dtype", list(DT))
def test_infinities_and_lowest_values(dtype):
    logits, ids, top, lse = make(9, 777, 4, dtype, 15)
    logits[0, 300:] = -math.inf                        # padding columns
    ids[0] = torch.tensor([0, 5, 299, 17])
    logits[1] = -math.inf                              # nothing left: an empty row
    logits[2, 1:] = torch.finfo(DT[dtype]).min         # masked with the type's lowest value
    logits[3] = torch.finfo(DT[dtype]).min             # all of it: uniform
    logits[4, int(ids[4, 0])] = -math.inf              # the teacher wants a word that the mask forbids
    logits[5, 9] = math.inf
    logits[6, 9] = math.nan
    logits[7] = math.nan
    logits[8, :] = 0                                   # all equal
    want, both, fwd, grad = compare(logits, ids, top)
    assert float(both["loss"][1]) == 0 and not bool(both["dlogits"][1].any())
    assert math.isinf(float(want["loss"][4])) and math.isnan(float(want["loss"][6]))


def test_far_logits():
    """Differences of hundreds: every exponential but a few underflows."""
    g = torch.Generator().manual_seed(16)
    logits = (torch.randn(4, 3001, generator=g) * 300).cuda()
    _, ids, top, lse = make(4, 3001, 16, "f32", 17, True)
    compare(logits, ids, top)
    compare(logits, ids, top, lse, temperature=20.0)


def test_logits_overwritten_in_place():
    for vocab in (1000, 50257):
        logits, ids, top, lse = make(7, vocab, 11, "bf16", 18, True)
        want = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)["dlogits"]
        fwd = tokens.distill_forward(logits, ids, top, teacher_lse=lse)
        one, two = logits.clone(), logits.clone()
        tokens.distill_forward_backward(one, ids, top, teacher_lse=lse, out={"dlogits": one})
        tokens.distill_backward(None, two, ids, top, fwd["stats"], teacher_lse=lse, out=two)
        assert torch.equal(one, want) and torch.equal(two, want)


def test_upstream_gradient_scales_rows():
    logits, ids, top, lse = make(5, 999, 7, "f32", 19, True)
    fwd = tokens.distill_forward(logits, ids, top, teacher_lse=lse)
    up = torch.tensor([0.5, -2.0, 0.0, 4.0, 1.0], device="cuda")
    got = tokens.distill_backward(up, logits, ids, top, fwd["stats"], teacher_lse=lse)
    one = tokens.distill_backward(None, logits, ids, top, fwd["stats"], teacher_lse=lse)
    # powers of two scale exactly
    assert torch.equal(got, one * up[:, None])


@pytest.mark.parametrize("tail", [False, True])
def test_gradient_against_differences(tail):
    """Central differences of the kernel's own loss.  With a step of 2^-5 the difference quotient is
    off by h^2 / 6 of a third derivative (at most 1 / T^3 in size, times T^2) and by the loss's rounding
    over the step: 2 * 2^-24 * 20 (a loss of at most 20) * 2^5."""
    logits, ids, top, lse = make(1, 23, 5, "f32", 20, tail)
    h = 2.0 ** -5
    n = logits.shape[1]
    grad = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse, temperature=2.0)["dlogits"][0].cpu()
    shifted = torch.cat([logits + h * torch.eye(n, device="cuda"), logits - h * torch.eye(n, device="cuda")])
    many = lambda t: None if t is None else t.expand(2 * n, *t.shape[1:]).contiguous()  # noqa: E731
    loss = tokens.distill_forward(shifted, many(ids), many(top), teacher_lse=many(lse), temperature=2.0)["loss"].cpu()
    diff = (loss[:n] - loss[n:]) / (2 * h)
    # with a tail class the curvature also has 1 / q_rest's terms: a bound of 16 on the third derivative
    assert float((diff - grad).abs().max()) <= h * h / 6 * (16 if tail else 1) + 2 * 2.0 ** -24 * 20 / h


def test_other_stream_and_repeats():
    logits, ids, top, lse = make(64, 5000, 40, "bf16", 21, True)
    first = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)
    side.synchronize()
    assert torch.equal(first["dlogits"], second["dlogits"]) and torch.equal(first["loss"], second["loss"])


def test_captured_in_a_graph():
    logits, ids, top, lse = make(16, 33000, 40, "bf16", 22, True)
    want = tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse)
    out = {"loss": torch.zeros(16, device="cuda"), "dlogits": torch.zeros_like(logits)}
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        tokens.distill_forward_backward(logits, ids, top, teacher_lse=lse, out=out)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out["loss"], want["loss"]) and torch.equal(out["dlogits"], want["dlogits"])


def test_no_rows():
    logits, ids, top, _ = make(0, 100, 3, "f32", 23)
    both = tokens.distill_forward_backward(logits, ids, top)
    assert both["loss"].shape == (0,) and both["dlogits"].shape == (0, 100)


def test_refusals():
    logits, ids, top, lse = make(4, 100, 3, "f32", 24)
    bad = pytest.raises(tokens.CBRError)
    with bad:
        tokens.distill_forward(logits.double(), ids, top)
    with bad:
        tokens.distill_forward(logits, ids.float(), top)
    with bad:
        tokens.distill_forward(logits, ids[:3], top)
    with bad:
        tokens.distill_forward(logits, ids, top[:, :2])
    with bad:
        tokens.distill_forward(logits.t().contiguous().t(), ids, top)     # a row is not contiguous
    with bad:
        tokens.distill_forward(logits, ids, top, temperature=0.0)
    with bad:
        tokens.distill_forward(logits, ids, top, row_weight=torch.ones(3, device="cuda"))
    with bad:
        tokens.distill_forward(logits.cpu(), ids, top)
    with bad:
        tokens.distill_forward(logits[:1].expand(4, 100), ids, top, out={"stats": torch.zeros(4, 2, device="cuda")})
    with bad:
        tokens.distill_forward_backward(logits, ids, top, out={"dlogits": torch.zeros(4, 99, device="cuda")})

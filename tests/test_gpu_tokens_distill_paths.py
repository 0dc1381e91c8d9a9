"""The distillation's less travelled ways, for every type: ids listed several times, among few entries and
among hundreds of one warp's part, in one block's row and in a cluster's; gradients over the logits themselves."""
import pytest
import torch

from conv_batchnorm_relu_gb300 import tokens
from test_gpu_tokens_distill import DT, compare, make

pytestmark = pytest.mark.gpu


def listed_twice(rows, vocab, k, dtype, seed, start, width, id_dtype=torch.int32):
    """Ids drawn with replacement from a stretch of the vocabulary."""
    logits, _, _, _ = make(rows, vocab, 1, dtype, seed)
    g = torch.Generator().manual_seed(seed + 1)
    top = (torch.randn(rows, k, generator=g) * 2 + 3).to(DT[dtype]).cuda()
    ids = (start + torch.randint(0, width, (rows, k), generator=g)).to(id_dtype).cuda()
    lse = torch.logsumexp(top.float(), 1) + torch.rand(rows, generator=g).cuda()
    return logits, ids, top, lse


# rows of up to four are shared by a cluster; the stretch lies in one warp's part of a chunk, or in several
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [3, 6])
@pytest.mark.parametrize("vocab,k,start,width", [
    (300, 9, 40, 5), (300, 200, 0, 300), (515, 96, 100, 40), (1000, 1024, 7, 300), (40000, 64, 20000, 3),
    (40000, 600, 16380, 50), (50257, 257, 0, 50257), (131072, 400, 65000, 1000)], ids=lambda v: str(v))
def test_repeated_ids(vocab, k, start, width, rows, dtype):
    logits, ids, top, lse = listed_twice(rows, vocab, k, dtype, 50 + k, start, width)
    compare(logits, ids, top, lse)
    compare(logits, ids, top, None, None, 2.0)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [2, 5])
def test_one_id_in_every_entry(rows, dtype):
    logits, ids, top, lse = listed_twice(rows, 2000, 300, dtype, 51, 1234, 1, torch.int64)
    compare(logits, ids, top, lse)


@pytest.mark.parametrize("dtype", list(DT))
def test_repeats_among_absent_entries(dtype):
    logits, ids, top, lse = listed_twice(6, 700, 150, dtype, 52, 300, 20)
    ids[:, ::3] = -1
    ids[0, 40:], ids[1, :110] = -1, 700
    compare(logits, ids, top)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows", [2, 6])
def test_a_listed_nan_of_all_ones(rows, dtype):
    """The mark that an entry leaves in the row while it is read is itself a NaN that a row may hold."""
    logits, ids, top, lse = make(rows, 900, 40, dtype, 53, True)
    bits = logits.view(torch.int32 if dtype == "f32" else torch.int16)
    bits[0, int(ids[0, 3])] = -1
    bits[1, int(ids[1, 39])] = -1
    ids[1, 38] = ids[1, 39]
    want, both, _, _ = compare(logits, ids, top, lse)
    assert bool(both["loss"][:2].isnan().all()) and not bool(both["loss"][2:].isnan().any())


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,vocab", [(1, 131072), (2, 50257), (4, 4099), (4, 20000)])
def test_logits_overwritten_in_place_by_a_cluster(rows, vocab, dtype):
    logits, ids, top, lse = make(rows, vocab, 33, dtype, 54, True)
    weight = torch.ones(rows, device="cuda")
    weight[-1] = 0 if rows > 2 else 1
    kw = dict(teacher_lse=lse, row_weight=weight)
    want = tokens.distill_forward_backward(logits, ids, top, **kw)["dlogits"]
    fwd = tokens.distill_forward(logits, ids, top, **kw)
    apart = tokens.distill_backward(None, logits, ids, top, fwd["stats"], **kw)
    one, two = logits.clone(), logits.clone()
    tokens.distill_forward_backward(one, ids, top, out={"dlogits": one}, **kw)
    tokens.distill_backward(None, two, ids, top, fwd["stats"], out=two, **kw)
    assert torch.equal(one, want) and torch.equal(two, apart)

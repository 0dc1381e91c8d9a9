"""The norms around a gated residual block against their plain 64-bit form: types, widths, gates shared
by rows, strides and alignments, flat rows, gradients against differences."""
import pytest
import torch

import token_reference as ref
from conv_batchnorm_relu_gb300 import tokens

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS, RHO, BETA = 1e-6, 0.9, 0.7
GUARD = 7.0


def rows_of(rows, dim, dtype, g, scale=1.0, offset=0.0, stride=None, shift=0):
    stride = stride or dim
    buf = (torch.randn(rows * stride + shift, generator=g) * scale + offset).to(DT[dtype]).cuda()
    return torch.as_strided(buf, (rows, dim), (stride, 1), shift)


def make(rows, dim, dtype, seed, form="both", groups=1, stride=None, shift=0, offset=0.0):
    g = torch.Generator().manual_seed(seed)
    s = dict(x=rows_of(rows, dim, dtype, g, 2.0, offset, stride, shift), branch=None, w1=None, gate=None, w2=None)
    if form != "pre":
        s["branch"] = rows_of(rows, dim, dtype, g, 3.0, offset, stride, shift)
        s["w1"] = (1 + 0.2 * torch.randn(dim, generator=g)).cuda()
        if groups:
            s["gate"] = (0.5 * torch.randn(groups, dim, generator=g)).cuda()
    if form != "post":
        s["w2"] = (1 + 0.2 * torch.randn(dim, generator=g)).cuda()
    return s, g


def forward(s, kind, **kw):
    return tokens.block_norm_forward(s["x"], s["branch"], s["w1"], s["gate"], s["w2"], kind=kind, eps=EPS,
                                     residual_scale=RHO, branch_scale=BETA, **kw)


def check_forward(s, kind):
    want = ref.norm_forward(s["x"], s["branch"], s["w1"], s["gate"], s["w2"], kind, EPS, RHO, BETA)
    got = forward(s, kind)
    torch.cuda.synchronize()
    dt = s["x"].dtype
    if s["branch"] is not None:
        ref.close(got["x_out"], want["x_out"], want["x_bound"], "x_out", dt)
    else:
        assert got["x_out"] is None
    if s["w2"] is not None:
        ref.close(got["h"], want["h"], want["h_bound"], "h", dt)
    else:
        assert got["h"] is None
    return got, want


def check_backward(s, got, kind, g, with_dx_out=True, stride=None, shift=0):
    rows, dim = s["x"].shape
    name = {v: k for k, v in DT.items()}[s["x"].dtype]
    dx_out = rows_of(rows, dim, name, g, 1.0, 0.0, stride, shift) if with_dx_out else None
    dh = rows_of(rows, dim, name, g, 1.0, 0.0, stride, shift) if s["w2"] is not None else None
    x_out = got["x_out"] if s["branch"] is not None else s["x"]
    args = (dx_out, dh, x_out, s["branch"], s["w1"], s["gate"], s["w2"], got["stats"])
    kw = dict(kind=kind, residual_scale=RHO, branch_scale=BETA)
    back = tokens.block_norm_backward(*args, **kw)
    again = tokens.block_norm_backward(*args, **kw)
    torch.cuda.synchronize()
    want = ref.norm_backward(*args, kind, RHO, BETA)
    dt = s["x"].dtype
    for n, bound, t in (("dx", "dx_bound", dt), ("dbranch", "dbranch_bound", dt),
                        ("dpost_weight", "dpost_bound", torch.float32), ("dgate", "dgate_bound", torch.float32),
                        ("dpre_weight", "dpre_bound", torch.float32)):
        if want[n] is None:
            assert back[n] is None
            continue
        ref.close(back[n], want[n], want[bound], n, t)
        assert torch.equal(back[n], again[n]), f"{n}: another run gives another result"
    return args, kw, back


@pytest.mark.parametrize("kind", ["rms", "layer"])
@pytest.mark.parametrize("form", ["both", "pre", "post"])
@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,dim", [(1, 1), (3, 7), (1, 2048), (5, 64), (37, 96), (130, 257), (9, 1001), (4, 4096),
                                      (3, 5120), (2, 16384), (2, 9999)], ids=lambda v: str(v))
def test_matches_plain_form(rows, dim, dtype, form, kind):
    s, g = make(rows, dim, dtype, 1000 + dim, form)
    got, _ = check_forward(s, kind)
    check_backward(s, got, kind, g)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("rows,dim,groups", [(2400, 64, 0), (2400, 64, 1), (2400, 40, 3), (2400, 129, 800),
                                             (2400, 256, 2400), (1500, 1024, 5), (3001, 72, 1), (700, 2560, 7)])
def test_gates_shared_by_rows(rows, dim, groups, dtype):
    """More rows than blocks; gates that begin and end inside a block's rows, cover several, or one each."""
    s, g = make(rows, dim, dtype, 2000 + rows + dim, "both", groups)
    got, _ = check_forward(s, "layer")
    check_backward(s, got, "layer", g)


@pytest.mark.parametrize("dtype", list(DT))
@pytest.mark.parametrize("dim,stride,shift", [(64, 65, 1), (512, 520, 0), (1000, 1003, 5), (4096, 4100, 4)])
def test_strides_and_alignment(dim, stride, shift, dtype):
    s, g = make(11, dim, dtype, 3000 + dim, "both", 1, stride, shift)
    got, _ = check_forward(s, "rms")
    args, kw, back = check_backward(s, got, "rms", g, stride=stride, shift=shift)
    # outputs with strides of their own: the same values, the gaps untouched
    plan = [("x_out", "h"), ("dx", "dbranch")]
    for names, run in zip(plan, (lambda o: forward(s, "rms", out=o),
                                 lambda o: tokens.block_norm_backward(*args, **kw, out=o))):
        bufs = [torch.full((11 * stride + shift + 9,), GUARD, dtype=DT[dtype], device="cuda") for _ in names]
        out = {n: torch.as_strided(b, (11, dim), (stride, 1), shift) for n, b in zip(names, bufs)}
        plain = run(None)
        run(out)
        for n, b in zip(names, bufs):
            assert torch.equal(out[n], plain[n]), n
            out[n].fill_(GUARD)
            assert bool((b == GUARD).all()), f"{n}: wrote outside its rows"


def test_a_single_gate_vector_and_its_gradient():
    s, g = make(50, 128, "bf16", 4, "both", 1)
    s["gate"] = s["gate"][0].contiguous()
    got, _ = check_forward(s, "rms")
    _, _, back = check_backward(s, got, "rms", g)
    assert back["dgate"].shape == (128,)


def test_without_gradient_from_the_stream():
    for form in ("both", "pre"):
        s, g = make(33, 200, "f16", 5, form)
        got, _ = check_forward(s, "layer")
        check_backward(s, got, "layer", g, with_dx_out=False)


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_flat_rows(kind):
    """Zero and constant rows: the norm divides by sqrt(eps) and stays finite."""
    s, g = make(4, 300, "f32", 6)
    s["x"][0], s["branch"][0] = 0, 0
    s["x"][1], s["branch"][1] = 3.0, 0
    got, _ = check_forward(s, kind)
    assert bool(torch.isfinite(got["h"]).all())


def test_large_means_do_not_cancel():
    """A mean of a hundred deviations: variances come from differences from the mean."""
    s, g = make(9, 777, "f32", 7, "both", 1, offset=200.0)
    got, want = check_forward(s, "layer")
    check_backward(s, got, "layer", g)
    rel = ((got["stats"].cpu().double() - want["stats"]) / want["stats"]).abs().max()
    assert float(rel) <= 2 * 200 * ref.rounds(777)


def test_in_place_outputs():
    s, g = make(40, 96, "bf16", 8)
    got = forward(s, "rms")
    x, f = s["x"].clone(), s["branch"].clone()
    t = dict(s, x=x, branch=f)
    forward(t, "rms", out={"x_out": x, "h": f})
    assert torch.equal(x, got["x_out"]) and torch.equal(f, got["h"])
    args, kw, back = check_backward(s, got, "rms", g)
    dx, dh = args[0].clone(), args[1].clone()
    tokens.block_norm_backward(dx, dh, *args[2:], **kw, out={"dx": dx, "dbranch": dh})
    assert torch.equal(dx, back["dx"]) and torch.equal(dh, back["dbranch"])


def test_a_bad_row_stays_alone():
    s, g = make(20, 130, "f32", 9)
    clean = forward(s, "layer")
    s["x"][3, 5], s["branch"][7, 0] = float("nan"), float("inf")
    got = forward(s, "layer")
    keep = [i for i in range(20) if i not in (3, 7)]
    assert torch.equal(got["h"][keep], clean["h"][keep]) and torch.equal(got["x_out"][keep], clean["x_out"][keep])
    assert bool(torch.isnan(got["h"][3]).all()) and bool(torch.isnan(got["h"][7]).all())


@pytest.mark.parametrize("form", ["pre", "both"])
@pytest.mark.parametrize("dim", [130, 1001, 2048])
def test_an_infinite_rms_scales_a_row_to_nothing(dim, form):
    """1 / sqrt(infinity) is 0: the other elements of such a row become exact zeros (in x_out: the rest of
    the sum), the infinity itself times 0 is NaN; so does a row whose squares pass the range of 32 bits."""
    s, _ = make(6, dim, "f32", 12, form)
    f = s["x"] if form == "pre" else s["branch"]
    f[2, 7] = float("inf")
    f[4] = 1e25
    got = forward(s, "rms")
    out, rest = (got["h"], 0 * s["x"]) if form == "pre" else (got["x_out"], RHO * s["x"])
    others = [c for c in range(dim) if c != 7]
    assert torch.equal(out[2][others], rest[2][others]) and bool(torch.isnan(out[2, 7]))
    assert torch.equal(out[4], rest[4])


@pytest.mark.parametrize("kind", ["rms", "layer"])
def test_gradients_against_differences(kind):
    """A loss of fixed random weights on x_out and h, in the kernel's 32 bits: the central difference
    along a random direction is good to its rounding (the loss's terms times 2^-24, over the step) and
    h^2 times a third derivative; the step of 2^-6 leaves 2e-3 of the gradient's size for both."""
    s, g = make(6, 50, "f32", 10, "both", 2)
    s = {k: v.contiguous() for k, v in s.items()}
    a, b = torch.randn(6, 50, generator=g).cuda(), torch.randn(6, 50, generator=g).cuda()

    def loss(t):
        o = forward(t, kind)
        return float((o["x_out"].double() * a).sum() + (o["h"].double() * b).sum())

    got = forward(s, kind)
    back = tokens.block_norm_backward(a, b, got["x_out"], s["branch"], s["w1"], s["gate"], s["w2"], got["stats"],
                                      kind=kind, residual_scale=RHO, branch_scale=BETA)
    step = 2.0 ** -6
    for name, grad in (("x", "dx"), ("branch", "dbranch"), ("w1", "dpost_weight"), ("gate", "dgate"),
                       ("w2", "dpre_weight")):
        v = torch.randn(s[name].shape, generator=g).cuda()
        diff = (loss(dict(s, **{name: s[name] + step * v})) - loss(dict(s, **{name: s[name] - step * v}))) / (2 * step)
        along = float((back[grad].double() * v).sum())
        scale = float(back[grad].double().norm() * v.double().norm())
        assert abs(diff - along) <= 2e-3 * scale, (name, diff, along)


def test_other_stream():
    s, g = make(300, 1024, "bf16", 11)
    first = forward(s, "rms")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = forward(s, "rms")
    side.synchronize()
    assert torch.equal(first["h"], second["h"])


def test_no_rows():
    s, g = make(0, 32, "f32", 12)
    got = forward(s, "rms")
    assert got["h"].shape == (0, 32)
    e = torch.empty(0, 32, device="cuda")
    for name in ("dpre_weight", "dpost_weight", "dgate"):
        back = tokens.block_norm_backward(e, e, e, s["branch"], s["w1"], s["gate"], s["w2"], got["stats"])
        assert not bool(back[name].any())


def test_refusals():
    s, g = make(12, 64, "f32", 13)
    bad = pytest.raises(tokens.CBRError)
    with bad:
        tokens.block_norm_forward(s["x"])
    with bad:
        tokens.block_norm_forward(s["x"], s["branch"], None, None, s["w2"])
    with bad:
        tokens.block_norm_forward(s["x"], None, None, s["gate"], s["w2"])
    with bad:
        tokens.block_norm_forward(s["x"], s["branch"], s["w1"], torch.ones(5, 64, device="cuda"), s["w2"])
    with bad:
        tokens.block_norm_forward(s["x"], s["branch"].half(), s["w1"], None, s["w2"])
    with bad:
        tokens.block_norm_forward(s["x"], None, None, None, s["w2"], kind="batch")
    with bad:
        tokens.block_norm_forward(s["x"], None, None, None, s["w2"], eps=0.0)
    with bad:
        tokens.block_norm_forward(s["x"].cpu(), None, None, None, s["w2"])
    with bad:
        tokens.block_norm_forward(torch.zeros(2, 16385, device="cuda"), None, None, None, torch.ones(16385, device="cuda"))
    with bad:
        tokens.block_norm_backward(s["x"], None, s["x"], s["branch"], s["w1"], None, s["w2"], torch.zeros(12, 4, device="cuda"))
    with bad:
        tokens.block_norm_backward(s["x"], s["x"], s["x"], s["branch"], s["w1"], None, s["w2"], None)
    with bad:   # a workspace too small
        tokens.block_norm_backward(s["x"], s["x"], s["x"], s["branch"], s["w1"], None, s["w2"],
                                   torch.zeros(12, 4, device="cuda"), ws=torch.zeros(16, device="cuda"))

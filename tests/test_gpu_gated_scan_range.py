"""The gated scan at the ends of f32's range: gates that are the type's lowest value, with large values beside them; input gates far
below 0 with inputs that make up for it; rates next to 0; infinities. Bounds where there are some: gated_ref.GatedCase."""
import pytest
import torch

import gated_ref as G
import seq_ref as R
from test_gpu_gated_scan import Inputs, check_forward, check_gradient

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
F64 = torch.float64
SHAPES = [(2, 70, 66), (1, 700, 64)]  # one CTA a sequence and slab and rows that are not aligned; clusters


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def lowest(dtype, shape):
    """Values whose logistic function is below 4e-44, the type's lowest among them."""
    low = torch.tensor([torch.finfo(dtype).min, -100.0, -1e4, torch.finfo(dtype).min / 3]).to(dtype)
    return low[torch.arange(shape[0] * shape[1] * shape[2]) % 4].view(shape).contiguous()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rate", [True, False])
def test_output_gates_that_are_shut(mt, dtype, shape, rate):
    """z sigma(z) and its derivative are below 1e-41 in size there, so what is let through, and every gradient, is 0 but for
    that: values are below 100, a sum has a few thousand terms."""
    p = Inputs(dtype, *shape, rate, True, True)
    p.z = lowest(dtype, shape)
    out, _ = p.forward(mt)
    assert out.float().abs().max() < 1e-30
    for name, g in p.gradient(mt, dfinal=False).items():
        assert g.float().abs().max() < 1e-30, name


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rate", [0.3, 2.0 ** 100, None])
def test_shut_gates_pass_nothing_however_large(mt, dtype, shape, rate):
    """r at the type's lowest value: nothing is let in and nothing forgotten, bit for bit, and no gradient passes but the state's."""
    p = Inputs(dtype, *shape, rate is not None, False, False)
    p.r.fill_(torch.finfo(dtype).min)
    p.r[:, ::3] = -1e4
    p.x = (torch.finfo(dtype).max / 4 * torch.sign(p.x.float())).to(dtype)
    if rate is not None:
        p.rate.fill_(rate)
    out, state = p.forward(mt)
    assert torch.equal(state.cpu(), p.h0) and torch.equal(out.cpu(), p.h0[:, None].expand(shape).to(dtype))
    step = p.h0.cuda()
    one = torch.empty(shape[0], shape[2], dtype=dtype, device="cuda")
    mt.mt_gated_scan_step(p.x[:, 0].cuda(), p.r[:, 0].cuda(), step, one, rate=p.gates()["rate"])
    assert torch.equal(step.cpu(), p.h0) and torch.equal(one, out[:, 0])
    got = p.gradient(mt)
    assert (got["dx"] == 0).all() and (got["dr"] == 0).all()
    if rate is not None:
        assert (got["drate"] == 0).all()
    total = p.dout.to(F64)
    R.assert_within("dinit", got["dinit"], total.sum(1) + p.dfinal.to(F64), (shape[1] + 4) * 2 * R.U * (total.abs().sum(1) + p.dfinal.abs()))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("rate", [True, False])
def test_input_gates_far_below_zero(mt, monkeypatch, dtype, shape, rate):
    """Gates of 1e-17 to 1e-35, and inputs of 1e25. As the calls' documentation says, a logistic function below 2^-102 has an error of up to 2^-126
    beside the relative ones (1 / (1 + e) less 2^-126, rounded once), and an input gate below 2^-63 may count as 0 in a prompt with rate; these
    go into the bounds as the others do."""
    plain = G.sigmoid

    def allow(error):
        def sigmoid(x):
            s, c = plain(x)
            return G.Ball(s.v, s.e + error), c
        monkeypatch.setattr(G, "sigmoid", sigmoid)

    p = Inputs(dtype, *shape, rate, True, False)
    g = torch.Generator().manual_seed(11)
    p.i = (-40 - 40 * torch.rand(shape, generator=g)).to(dtype)
    p.x = (p.x.float() * 1e25).to(dtype)
    allow(2.0 ** -63 if rate else 2.0 ** -126)
    check_forward(mt, p)
    check_gradient(mt, p)
    allow(2.0 ** -126)
    want, final = G.GatedCase(p.x[:, :1], p.r[:, :1], p.i[:, :1], None, p.rate, p.h0).forward()
    state, out = p.h0.cuda(), torch.empty(shape[0], shape[2], dtype=dtype, device="cuda")
    gates = p.gates()
    mt.mt_gated_scan_step(p.x[:, 0].cuda(), p.r[:, 0].cuda(), state, out, i=gates["i"][:, 0], rate=gates["rate"])
    G.check("out", out, G.Ball(want.v[:, 0], want.e[:, 0]))
    G.check("state", state, final)


NEXT_TO_ZERO = [0.0, 1e-45, 1e-40, 5e-39, 1e-37, 1e-36, 1e-30, 1e-20]  # of which the first four let nothing in, with gates near 1/2


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
def test_rates_next_to_zero(mt, dtype, shape):
    """Where 1 - a^2 is below f32's normal numbers, the input's weight is 0, and so is its derivative; elsewhere both are as the definition
    has them. The sum for a rate of 0 is over the state's part alone: its terms are off by 8 U (products of four factors and their
    states and gradients, sums of up to the length) of their size."""
    p = Inputs(dtype, *shape, True, False, False)
    b, length, d = shape
    g = torch.Generator().manual_seed(12)
    p.r = (torch.rand(shape, generator=g) - 0.5).to(dtype)
    p.rate = torch.tensor(NEXT_TO_ZERO)[torch.arange(d) % 8].clone()
    dead = p.rate < 1e-38
    out, state = p.forward(mt)
    got = p.gradient(mt)
    assert torch.equal(state.cpu()[:, dead], p.h0[:, dead])
    assert torch.equal(out.cpu()[..., dead], p.h0[:, None, dead].expand(b, length, -1).to(dtype))
    assert (got["dx"][..., dead.cuda()] == 0).all() and (got["dr"].float().abs()[..., dead.cuda()] < 1e-30).all()
    after = p.dout.to(F64).flip(1).cumsum(1).flip(1) + p.dfinal.to(F64)[:, None]
    size = p.dout.to(F64).abs().flip(1).cumsum(1).flip(1) + p.dfinal.to(F64).abs()[:, None]
    s, h = torch.sigmoid(p.r.to(F64)), p.h0.to(F64)[:, None]
    R.assert_within("drate", got["drate"].cpu()[dead], (-after * h * s).sum((0, 1))[dead],
                    (2 * length + 40) * R.U * (size * h.abs() * s).sum((0, 1))[dead])
    live = ~dead
    cut = lambda t: t[..., live].contiguous()  # noqa: E731
    case = G.GatedCase(cut(p.x), cut(p.r), None, None, p.rate[live], p.h0[:, live])
    want, final = case.forward()
    G.check("out", out.cpu()[..., live], want)
    G.check("state", state.cpu()[:, live], final)
    want = case.gradient(cut(p.dout), p.dfinal[:, live])
    for name in want:
        G.check(name, got[name].cpu()[..., live], want[name])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("where", ["x", "h0"])
def test_infinities_stay_in_their_channel_and_after_their_token(mt, dtype, shape, where):
    p = Inputs(dtype, *shape, True, True, False)
    clean, last = p.forward(mt)
    at = shape[1] // 3 if where == "x" else 0
    if where == "x":
        p.x[0, at, 5] = float("inf")
    else:
        p.h0[0, 5] = -float("inf")
    out, state = p.forward(mt)
    assert not out[0, at:, 5].isfinite().any() and not state[0, 5].isfinite()
    out[0, at:, 5], state[0, 5] = clean[0, at:, 5], last[0, 5]
    assert torch.equal(out, clean) and torch.equal(state, last)


@pytest.mark.parametrize("shape", SHAPES)
def test_rates_below_zero_count_as_zero(mt, shape):
    p = Inputs(torch.float32, *shape, True, True, True)
    got = []
    for below in (0.0, -3.0):
        p.rate[::2] = below
        state, out = p.h0.cuda(), torch.empty(shape[0], shape[2], device="cuda")
        g = p.gates()
        mt.mt_gated_scan_step(p.x[:, 0].cuda(), p.r[:, 0].cuda(), state, out, i=g["i"][:, 0], z=g["z"][:, 0], rate=g["rate"])
        got.append((*p.forward(mt), *p.gradient(mt).values(), state, out))
    assert all(torch.equal(a, b) for a, b in zip(*got))

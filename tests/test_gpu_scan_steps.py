"""Step sizes of the selective scan that leave the softplus out but not the bias: Delta = delta + delta_bias, and 0 (not the bias)
from a sequence's end on, whatever part of a tile or a segment that end falls into. Bounds: seq_ref.ScanCase."""
import pytest
import torch

import seq_ref as R
from test_gpu_selective_scan import DTYPES, Inputs, check_forward, check_gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def biased(dtype, b, length, d, n, **kw):
    """Steps of 0.05 and more, most of them the bias: a token too many takes 5 % and more of a state with it."""
    x = Inputs(dtype, b, length, d, n, softplus=False, **kw)
    x.bias = torch.rand(d, generator=torch.Generator().manual_seed(d + n)) * 0.3 + 0.05
    return x


def ends(b, length):
    """Sequences that end at every place of a tile, in the first, a middle and the last segment."""
    some = [length, 1, length - 3, 5, length // 2 + 1, 0, length // 3]
    return torch.tensor([max(0, some[i % len(some)]) for i in range(b)], dtype=torch.int32)


@pytest.mark.parametrize("length", range(1, 18))
def test_every_length_of_a_tile(mt, length):
    x = biased(torch.float32, 2, length, 12, 4)
    check_forward(x, *x.forward(mt))
    check_gradient(x, x.gradient(mt))


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", [dict(b=2, length=13, d=32, n=16), dict(b=2, length=13, d=33, n=5, pad=1), dict(b=7, length=300, d=40, n=16, ragged=True),
                                dict(b=7, length=131, d=9, n=21, pad=3, ragged=True), dict(b=7, length=43, d=24, n=64, ragged=True),
                                dict(b=3, length=27, d=6, n=100, ragged=True), dict(b=7, length=70, d=20, n=16, groups=2, gate=False, skip=False, ragged=True)],
                         ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_ragged_and_cut(mt, dtype, kw):
    kw = dict(kw)
    if kw.pop("ragged", False):
        kw["lens"] = ends(kw["b"], kw["length"])
    x = biased(dtype, **kw)
    check_forward(x, *x.forward(mt))
    check_gradient(x, x.gradient(mt))


@pytest.mark.parametrize("head", [37, 5])
def test_steps_continue_a_prompt(mt, head):
    length = head + 4
    x = biased(torch.float32, 2, length, 20, 16)
    c = lambda t: t.cuda()  # noqa: E731
    state, outs = c(x.h0), [torch.empty(2, head, 20, device="cuda")]
    slots = mt.mt_selective_scan_scratch_slots(2, head, 20, 16)
    scratch = torch.empty(slots, dtype=torch.int64, device="cuda") if slots else None
    cut = lambda t: c(t)[:, :head]  # noqa: E731
    kw = dict(D=c(x.D), delta_bias=c(x.bias), softplus=False)
    mt.mt_selective_scan(cut(x.u), cut(x.delta), c(x.A), cut(x.B), cut(x.C), outs[0], scratch, z=cut(x.z), state=state, carry_in=True, **kw)
    for t in range(head, length):
        o, at = torch.empty(2, 20, device="cuda"), lambda v: c(v)[:, t]  # noqa: E731,B023
        mt.mt_selective_scan_step(at(x.u), at(x.delta), c(x.A), at(x.B), at(x.C), state, o, z=at(x.z), **kw)
        outs.append(o[:, None])
    check_forward(x, torch.cat(outs, 1), state)


@pytest.mark.parametrize("length", [3, 13, 200])
def test_a_sequence_does_not_see_how_far_the_others_go(mt, length):
    """The same tokens alone and in a batch of longer rows: the same state, outputs and gradients within the bounds of either."""
    n = max(1, length - 2)
    x = biased(torch.float32, 1, length, 16, 8, lens=torch.tensor([n], dtype=torch.int32))
    out, state = x.forward(mt)
    got = x.gradient(mt)
    short = biased(torch.float32, 1, length, 16, 8)
    for k in ("u", "delta", "B", "C", "z", "dout"):
        setattr(short, k, getattr(x, k)[:, :n].contiguous())
    short.A, short.D, short.bias, short.h0, short.dfinal = x.A, x.D, x.bias, x.h0, x.dfinal
    check_forward(short, out[:, :n], state)
    check_gradient(short, {k: v[:, :n] if v.dim() > 2 and k != "dinit" else v for k, v in got.items()})


def no_steps(n, softplus, length, lens):
    """Every step 0: exactly, by a softplus that underflows or by zeros."""
    x = Inputs(torch.float32, 3, length, 12, n, softplus=softplus, bias=False, lens=lens)
    x.delta[x.mask] = -200.0 if softplus else 0.0
    return x


@pytest.mark.parametrize("softplus", [True, False])
@pytest.mark.parametrize("n", [5, 16, 40])
@pytest.mark.parametrize("length,lens", [(1, None), (13, None), (200, None), (200, [200, 21, 0])], ids=str)
def test_a_step_of_zero_leaves_the_state_as_it_was(mt, n, softplus, length, lens):
    """Bit for bit, forward, one token at a time and (without dout) back."""
    x = no_steps(n, softplus, length, None if lens is None else torch.tensor(lens, dtype=torch.int32))
    _, state = x.forward(mt)
    assert torch.equal(state.cpu(), x.h0)
    x.dout = torch.where(x.mask[..., None], torch.zeros(()), x.dout)
    got = x.gradient(mt)
    assert torch.equal(got["dinit"].cpu(), x.dfinal)
    assert (got["dA"] == 0).all()
    if length == 1:
        one, state = torch.empty(3, 12, device="cuda"), x.h0.cuda()
        at = lambda v: v.cuda()[:, 0]  # noqa: E731
        mt.mt_selective_scan_step(at(x.u), at(x.delta), x.A.cuda(), at(x.B), at(x.C), state, one, softplus=softplus)
        assert torch.equal(state.cpu(), x.h0)

"""The selective scan where a warp goes over many tiles of tokens, which batches of real sizes make it do: tokens that are not cut at all,
segments long enough that every stage of the ring is refilled several times, and groups of several channel tiles, whose sums for dB and dC
meet in another kernel. The sizes are small ones for which the plan is the same (a group of channels is a warp's work, however few they
are); each test asks the plan's scratch sizes whether it is. Bounds: seq_ref.ScanCase."""
import pytest
import torch

import seq_ref as R
from test_gpu_selective_scan import Inputs, check_forward, check_gradient

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def lanes_of(n):
    p = 2
    while 4 * p < n:
        p *= 2
    return p


def grad_segments(mt, b, length, d, n, groups):
    """Segments of the gradient's plan, from its scratch: rows of dB and dC per channel tile, then parameter sums, carries and
    step sums a segment (the last two only where there are several)."""
    tiles = -(-(d // groups) // (128 // lanes_of(n) * 4))
    slots = mt.mt_selective_scan_scratch_slots(b, length, d, n, groups, grad=True)
    up = lambda x: (x + 3) // 4 * 2  # noqa: E731
    rows = groups * tiles * b * length * 4 * lanes_of(n)
    fits = [s for s in range(1, length + 1)
            if rows + up(b * s * d * (n + 2)) + (up(b * s * d * n) + up(b * s * d) if s > 1 else 0) == slots]
    assert len(fits) == 1, fits
    return fits[0], tiles


def check_all(x, got):
    """check_gradient, but for dz: the slope of silu, s (1 + z (1 - s)), crosses 0 at z = -1.2785, and near it its two terms cancel, in any f32
    evaluation. So they count with their absolute values, as the terms of every other result do. With a few hundred thousand
    gates some lie within 1e-4 of that place."""
    check_gradient(x, {k: v for k, v in got.items() if k != "dz"})
    case = x.case()
    m, z = case.magnitude(), R.zeroed(x.z, case.mask)
    s = R.sigmoid(z)
    m.dgate = s * (1 + z.abs() * (1 - s))
    R.assert_within("dz", got["dz"], case.grad(x.dout, x.dfinal)["dz"], 2 * case.rel() * m.grad(x.dout.abs(), x.dfinal.abs())["dz"])


# channels in groups of 8 (16-byte rows) and of 5 and 37 (odd rows); the last two have several channel tiles a group too
UNCUT = [dict(b=4, length=44, d=1520, n=16, groups=190), dict(b=4, length=43, d=950, n=7, groups=190, pad=1),
         dict(b=4, length=41, d=2560, n=36, groups=64), dict(b=4, length=42, d=2368, n=33, groups=64, pad=3)]


@pytest.mark.parametrize("ragged", [False, True])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", UNCUT, ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_tokens_that_are_not_cut(mt, kw, dtype, ragged):
    b, length, d, n, groups = (kw[k] for k in ("b", "length", "d", "n", "groups"))
    assert mt.mt_selective_scan_scratch_slots(b, length, d, n, groups) == 0
    assert grad_segments(mt, b, length, d, n, groups)[0] == 1
    x = Inputs(dtype, **kw, lens=torch.tensor([length, 33, 0, 21], dtype=torch.int32) if ragged else None)
    check_forward(x, *x.forward(mt))
    check_all(x, x.gradient(mt))


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16])
@pytest.mark.parametrize("kw", [dict(b=2, length=4090, d=128, n=4, groups=16), dict(b=2, length=4090, d=48, n=3, groups=16, pad=1)],
                         ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_segments_of_many_tiles(mt, kw, dtype):
    """Segments of 72 tokens forward, nine stages of 8; of 216 in the gradient."""
    assert 10 <= grad_segments(mt, *(kw[k] for k in ("b", "length", "d", "n", "groups")))[0] <= 60
    x = Inputs(dtype, **kw)
    check_forward(x, *x.forward(mt))
    check_all(x, x.gradient(mt))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kw", [dict(b=2, length=60, d=136, n=16), dict(b=2, length=60, d=131, n=16, pad=1), dict(b=2, length=40, d=600, n=8),
                                dict(b=1, length=33, d=144, n=64, groups=2), dict(b=2, length=37, d=90, n=21, groups=1, pad=2),
                                dict(b=1, length=33, d=40, n=128)], ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_groups_of_several_channel_tiles(mt, kw, dtype):
    assert grad_segments(mt, kw["b"], kw["length"], kw["d"], kw["n"], kw.get("groups", 1))[1] > 1
    x = Inputs(dtype, **kw)
    check_all(x, x.gradient(mt))


def test_slow_decays_keep_their_precision(mt):
    """States that remember about 110 tokens, over 1024 that are not cut, with terms of one sign, so that no sum hides a lean.
    The unit's exponential with the constant added to its argument leans by at most 1.3e-8 of a decay between 0.7 and 1 (measured), and a
    state sees a lean once for every token that it remembers. The rest is a random walk over half of them: 3.2e-8 rms of the unit
    (measured) and 2.5e-8 of the multiply-add's rounding a token. Without the constant the unit leans by 2.4e-8 at these decays, half as
    much again as the limit. dA meets states and adjoints: twice. ddelta is left out: its two sums nearly cancel here."""
    b, length, d, n, groups = 4, 1024, 760, 4, 190
    assert mt.mt_selective_scan_scratch_slots(b, length, d, n, groups) == 0
    x = Inputs(torch.float32, b, length, d, n, groups=groups, gate=False, skip=False, bias=False, seed=1)
    x.u, x.B, x.C, x.dout, x.dfinal, x.h0 = (v.abs() for v in (x.u, x.B, x.C, x.dout, x.dfinal, x.h0))
    x.delta = x.delta * 0.2 - 3.98  # steps near 0.0185
    x.A = -(torch.rand(d, n, generator=torch.Generator().manual_seed(1)) * 0.1 + 0.45)  # decays near 0.991
    case = x.case()
    memory = float((1 / (case.step.mean() * case.A.abs())).mean())
    limit = 1.3e-8 * memory + 4.1e-8 * (memory / 2) ** 0.5
    out, state = x.forward(mt)
    got, (want_out, want_state), want = x.gradient(mt), case.forward(), case.grad(x.dout, x.dfinal)
    off = lambda a, w: float((a.double().cpu() - w).norm() / w.norm())  # noqa: E731
    errors = dict(out=off(out, want_out), state=off(state, want_state), **{k: off(got[k], want[k]) for k in ("du", "dB", "dC", "dinit", "dA")})
    assert all(v <= limit * (2 if k == "dA" else 1) for k, v in errors.items()), (errors, limit)

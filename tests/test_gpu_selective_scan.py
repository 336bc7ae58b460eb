"""mt_selective_scan, its single-token form and its gradient against the
recurrence in 64 bits (seq_ref.ScanCase, which states the bounds)."""
import pytest
import torch

import seq_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN = float("nan")


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def wide(x, pad):
    """x on the GPU as a part of wider rows."""
    if x is None:
        return None
    if pad == 0:
        return x.cuda()
    flat = x.flatten(2)
    buf = torch.full((*flat.shape[:2], flat.shape[2] + 2 * pad), NAN, dtype=x.dtype, device="cuda")
    view = buf[..., pad:pad + flat.shape[2]]
    view.copy_(flat)
    return view.unflatten(2, x.shape[2:]) if x.dim() == 4 else view


class Inputs:
    def __init__(self, dtype, b, length, d, n, groups=1, gate=True, skip=True, bias=True, softplus=True, h0=True, lens=None, seed=0,
                 pad=0):
        g = torch.Generator().manual_seed(1000 * n + 10 * length + d + seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.mask = R.live_mask(lens, b, length)

        def act(*s, by=1.0):
            x = (r(*s) * by).to(dtype)
            x[~self.mask] = NAN  # what lies past a sequence's end must not be read
            return x

        self.softplus, self.lens, self.pad = softplus, lens, pad
        self.u, self.B, self.C = act(b, length, d), act(b, length, groups, n), act(b, length, groups, n)
        self.delta = act(b, length, d, by=0.5)
        if not softplus:
            self.delta = self.delta.abs() * 0.1
        self.A = -(torch.rand(d, n, generator=g) * 2 + 0.1)
        self.D = r(d) if skip else None
        self.z = act(b, length, d) if gate else None
        self.bias = -torch.rand(d, generator=g) * 5 if bias and softplus else None  # steps from 0.005 to 0.7
        self.h0 = r(b, d, n) if h0 else None
        self.dout = act(b, length, d)
        self.dfinal = r(b, d, n)

    def case(self):
        return R.ScanCase(self.u, self.delta, self.A, self.B, self.C, self.D, self.z, self.bias, self.softplus, self.h0, self.lens)

    def forward(self, mt, checkpoints=None, state=None):
        b, length, d = self.u.shape
        n, groups = self.A.shape[1], self.B.shape[2]
        c = lambda x: None if x is None else x.cuda()  # noqa: E731
        out = wide(torch.full_like(self.u, 5.0), self.pad)
        carry = self.h0 is not None
        if state is None:
            state = c(self.h0) if carry else torch.full((b, d, n), 9.0, device="cuda")
        slots = mt.mt_selective_scan_scratch_slots(b, length, d, n, groups)
        scratch = torch.full((slots,), -1, dtype=torch.int64, device="cuda") if slots else None  # NaN patterns
        p = self.pad
        mt.mt_selective_scan(wide(self.u, p), wide(self.delta, p), c(self.A), wide(self.B, p), wide(self.C, p), out, scratch, D=c(self.D),
                             z=wide(self.z, p), delta_bias=c(self.bias), softplus=self.softplus, state=state, carry_in=carry,
                             lens=c(self.lens), checkpoints=checkpoints)
        return out, state

    def gradient(self, mt, dfinal=True):
        b, length, d = self.u.shape
        n, groups = self.A.shape[1], self.B.shape[2]
        c = lambda x: None if x is None else x.cuda()  # noqa: E731
        ck = torch.full((max(1, mt.mt_selective_scan_checkpoint_slots(b, length, d, n)),), -1, dtype=torch.int64, device="cuda")
        self.forward(mt, ck)
        p = self.pad
        like = lambda x: wide(torch.full_like(x, 5.0), p)  # noqa: E731
        got = dict(du=like(self.u), ddelta=like(self.u), dB=like(self.B), dC=like(self.C), dA=torch.empty(d, n, device="cuda"),
                   dD=torch.empty(d, device="cuda"), ddelta_bias=torch.empty(d, device="cuda"), dinit=torch.empty(b, d, n, device="cuda"))
        if self.z is not None:
            got["dz"] = like(self.u)
        scratch = torch.full((mt.mt_selective_scan_scratch_slots(b, length, d, n, groups, grad=True),), -1, dtype=torch.int64,
                             device="cuda")
        mt.mt_selective_scan_grad(wide(self.u, p), wide(self.delta, p), c(self.A), wide(self.B, p), wide(self.C, p), wide(self.dout, p), ck,
                                  got["du"], got["ddelta"], got["dA"], got["dB"], got["dC"], scratch, D=c(self.D), dD=got["dD"],
                                  z=wide(self.z, p), dz=got.get("dz"), delta_bias=c(self.bias), ddelta_bias=got["ddelta_bias"],
                                  softplus=self.softplus, dfinal=c(self.dfinal) if dfinal else None, dinit=got["dinit"],
                                  lens=c(self.lens))
        return got


def lens_of(b, length):
    """Full, empty, one, and lengths around a tile's ends."""
    some = [length, 0, 1, min(length, 16), min(length, 17), max(0, length - 1), -4]
    return torch.tensor([some[i % len(some)] for i in range(b)], dtype=torch.int32)


def check_forward(x, out, state):
    case = x.case()
    want, last = case.forward()
    mag, lmag = case.magnitude().forward()
    R.assert_within("out", out, want, case.rel() * mag)
    R.assert_within("state", state, last, case.rel() * lmag)


CASES = [
    dict(b=1, length=1, d=1, n=1),
    dict(b=2, length=2, d=5, n=4, pad=1),
    dict(b=3, length=15, d=33, n=16, pad=4),
    dict(b=1, length=16, d=32, n=16),
    dict(b=7, length=17, d=36, n=16, groups=2, pad=8, ragged=True),
    dict(b=2, length=40, d=130, n=5, ragged=True),
    dict(b=2, length=33, d=12, n=21, groups=3, pad=2),
    dict(b=1, length=31, d=24, n=64, ragged=True),
    dict(b=2, length=18, d=9, n=100),
    dict(b=1, length=20, d=8, n=128, groups=2),
    dict(b=7, length=300, d=40, n=16, ragged=True),   # cut into segments, some without tokens
    dict(b=1, length=577, d=7, n=3, groups=7),
    dict(b=2, length=129, d=64, n=32, pad=4),
]


def build(dtype, kw, **more):
    kw = dict(kw)
    if kw.pop("ragged", False):
        kw["lens"] = lens_of(kw["b"], kw["length"])
    return Inputs(dtype, **kw, **more)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_prompt(mt, dtype, kw):
    x = build(dtype, kw)
    check_forward(x, *x.forward(mt))


@pytest.mark.parametrize("off", [dict(gate=False), dict(skip=False), dict(bias=False), dict(softplus=False), dict(h0=False),
                                 dict(gate=False, skip=False, bias=False, softplus=False, h0=False)], ids=lambda o: "-".join(o))
@pytest.mark.parametrize("length", [20, 200])
def test_without_optional_parts(mt, off, length):
    x = Inputs(torch.float32, 2, length, 20, 8, lens=lens_of(2, length), **off)
    check_forward(x, *x.forward(mt))
    check_gradient(x, x.gradient(mt))


def check_gradient(x, got, dfinal=True):
    case = x.case()
    final = x.dfinal if dfinal else None
    want = case.grad(x.dout, final)
    mag = case.magnitude().grad(x.dout.abs(), None if final is None else final.abs())
    b, length, d = x.u.shape
    tokens, per_group = b * length, d // case.groups
    for name in got:
        rel = 2 * case.rel()  # states from the left meet adjoints from the right
        if name in ("dA", "dD", "ddelta_bias"):
            rel += (tokens + 8) * R.U
        if name in ("dB", "dC"):
            rel += (per_group + 8) * R.U
        R.assert_within(name, got[name], want[name], rel * mag[name])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("kw", CASES, ids=lambda k: "-".join(f"{a}{v}" for a, v in k.items()))
def test_gradient(mt, dtype, kw):
    x = build(dtype, kw)
    check_gradient(x, x.gradient(mt))


def test_gradient_without_the_last_states(mt):
    x = Inputs(torch.float32, 2, 50, 20, 16)
    check_gradient(x, x.gradient(mt, dfinal=False), dfinal=False)


def test_gradient_against_differences(mt):
    """The kernels' own forward pass, moved along a direction, against the kernels' gradient. f32 rounding of a result of size s
    over a step of e leaves 2^-22 s / e, the third derivative e^2: e = 2^-7 leaves 3e-5 s and 6e-5, against directions of order 1."""
    e = 2.0 ** -7
    base = Inputs(torch.float32, 1, 9, 6, 4)
    got = base.gradient(mt)
    g = torch.Generator().manual_seed(4)

    def value(x):
        out, last = x.forward(mt)
        return float((out.double().cpu() * x.dout.double()).sum() + (last.double().cpu() * x.dfinal.double()).sum())

    for attr, name in (("u", "du"), ("delta", "ddelta"), ("A", "dA"), ("B", "dB"), ("C", "dC"), ("D", "dD"), ("z", "dz"),
                       ("bias", "ddelta_bias"), ("h0", "dinit")):
        x = getattr(base, attr)
        v = torch.randn(x.shape, generator=g)
        v /= v.norm()
        setattr(base, attr, x + e * v)
        up = value(base)
        setattr(base, attr, x - e * v)
        down = value(base)
        setattr(base, attr, x)
        want = float((got[name].double().cpu() * v.double()).sum())
        scale = float(got[name].double().norm().cpu()) + 1.0
        assert abs((up - down) / (2 * e) - want) <= 2e-3 * scale, (name, (up - down) / (2 * e), want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,d,n,groups", [(1, 1, 1, 1), (3, 7, 16, 1), (2, 40, 5, 2), (4, 24, 64, 1), (2, 6, 128, 3), (5, 33, 16, 1)])
def test_step(mt, dtype, b, d, n, groups):
    x = Inputs(dtype, b, 1, d, n, groups=groups)
    state = x.h0.cuda()
    out = torch.full((b, d), 5.0, dtype=dtype, device="cuda")
    one = lambda t: wide(t, 3)[:, 0]  # noqa: E731
    mt.mt_selective_scan_step(one(x.u), one(x.delta), x.A.cuda(), one(x.B), one(x.C), state, out, D=x.D.cuda(), z=one(x.z),
                              delta_bias=x.bias.cuda())
    check_forward(x, out[:, None], state)


def test_steps_continue_a_prompt(mt):
    """Prompt of 37 tokens, then 5 single tokens, against the prompt of 42."""
    x = Inputs(torch.float32, 2, 42, 20, 16)
    state = x.h0.cuda()
    c = lambda t: t.cuda()  # noqa: E731
    head = torch.empty(2, 37, 20, device="cuda")
    slots = mt.mt_selective_scan_scratch_slots(2, 37, 20, 16)
    scratch = torch.empty(slots, dtype=torch.int64, device="cuda") if slots else None
    cut = lambda t: c(t)[:, :37]  # noqa: E731
    mt.mt_selective_scan(cut(x.u), cut(x.delta), c(x.A), cut(x.B), cut(x.C), head, scratch, D=c(x.D), z=cut(x.z), delta_bias=c(x.bias),
                         state=state, carry_in=True)
    outs = [head]
    for t in range(37, 42):
        o = torch.empty(2, 20, device="cuda")
        at = lambda v: c(v)[:, t]  # noqa: E731,B023
        mt.mt_selective_scan_step(at(x.u), at(x.delta), c(x.A), at(x.B), at(x.C), state, o, D=c(x.D), z=at(x.z), delta_bias=c(x.bias))
        outs.append(o[:, None])
    check_forward(x, torch.cat(outs, 1), state)


@pytest.mark.parametrize("length", [1, 30, 400])
def test_slots_and_inactive_sequences(mt, length):
    b, d, n = 4, 12, 16
    x = Inputs(torch.float32, b, length, d, n, h0=False)
    pool = torch.randn(6, d, n, generator=torch.Generator().manual_seed(1))
    slots = torch.tensor([4, 6, 1, -1], dtype=torch.int32).cuda()
    c = lambda t: t.cuda()  # noqa: E731
    state, out = pool.cuda(), torch.full((b, length, d), 5.0, device="cuda")
    need = mt.mt_selective_scan_scratch_slots(b, length, d, n)
    scratch = torch.empty(need, dtype=torch.int64, device="cuda") if need else None
    kw = dict(D=c(x.D), delta_bias=c(x.bias), slots=slots)
    mt.mt_selective_scan(c(x.u), c(x.delta), c(x.A), c(x.B), c(x.C), out, scratch, z=c(x.z), state=state, carry_in=True, **kw)
    x.h0 = pool[[4, 0, 1, 0]]
    want, last = x.case().forward()
    mag, lmag = x.case().magnitude().forward()
    rel = x.case().rel()
    for i, s in ((0, 4), (2, 1)):
        R.assert_within("out", out[i], want[i], rel * mag[i])
        R.assert_within("state", state[s], last[i], rel * lmag[i])
    assert (out[[1, 3]] == 0).all()
    assert torch.equal(state.cpu()[[0, 2, 3, 5]], pool[[0, 2, 3, 5]])
    if length == 1:
        s2, o2 = pool.cuda(), torch.full((b, d), 5.0, device="cuda")
        at = lambda v: c(v)[:, 0]  # noqa: E731
        mt.mt_selective_scan_step(at(x.u), at(x.delta), c(x.A), at(x.B), at(x.C), s2, o2, z=at(x.z), **kw)
        assert (o2[[1, 3]] == 0).all() and torch.equal(s2.cpu()[[0, 2, 3, 5]], pool[[0, 2, 3, 5]])
        R.assert_within("out", o2[[0, 2]], want[[0, 2], 0], rel * mag[[0, 2], 0])


def test_nothing_to_do(mt):
    e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    A = -torch.ones(6, 4, device="cuda")
    state = torch.full((2, 6, 4), 3.0, device="cuda")
    none = (e(2, 0, 6), e(2, 0, 6), A, e(2, 0, 1, 4), e(2, 0, 1, 4), e(2, 0, 6))
    mt.mt_selective_scan(*none, state=state, carry_in=True)
    assert (state == 3).all()
    mt.mt_selective_scan(*none, state=state)
    assert (state == 0).all()
    for b, length in ((0, 5), (2, 0)):
        dA, dD = torch.full((6, 4), 3.0, device="cuda"), torch.full((6,), 3.0, device="cuda")
        dfinal, dinit = torch.randn(b, 6, 4, device="cuda"), e(b, 6, 4)
        a, s = (lambda: e(b, length, 6)), (lambda: e(b, length, 1, 4))
        scratch = torch.empty(max(1, mt.mt_selective_scan_scratch_slots(b, length, 6, 4, grad=True)), dtype=torch.int64, device="cuda")
        mt.mt_selective_scan_grad(a(), a(), A, s(), s(), a(), e(1), a(), a(), dA, s(), s(), scratch, dD=dD, dfinal=dfinal, dinit=dinit)
        assert (dA == 0).all() and (dD == 0).all() and torch.equal(dinit, dfinal)


def test_extreme_values(mt):
    """Steps that empty the state, steps of 0, gates that close: no NaN where the definition has none."""
    x = Inputs(torch.float32, 1, 40, 8, 16)
    x.delta[:, ::5] = 80.0   # a = exp(-160): the state is forgotten
    x.delta[:, 1::5] = -120.0  # a = 1, nothing enters
    x.z[:, ::3] = -200.0     # silu = -0
    x.z[:, 1::3] = 60.0
    out, state = x.forward(mt)
    check_forward(x, out, state)
    assert torch.isfinite(out).all() and torch.isfinite(state).all()
    for v in x.gradient(mt).values():
        assert torch.isfinite(v).all()


def test_same_bits_each_time_and_on_another_stream(mt):
    x = Inputs(torch.bfloat16, 2, 260, 72, 16)
    a, b = x.gradient(mt), x.gradient(mt)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c = x.gradient(mt)
    side.synchronize()
    for k in a:
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.parametrize("n", [3, 4])
@pytest.mark.parametrize("length,lens", [(140, None), (1040, None), (2064, [2064, 1041]), (4243, None), (4243, [2050, 4243])],
                         ids=lambda v: "full" if v is None else "ragged" if isinstance(v, list) else str(v))
def test_many_segments(mt, n, length, lens):
    """A token axis of 9 to 266 segments: the carries meet over more turns and more warps than one."""
    x = Inputs(torch.float32, 2, length, 6, n, lens=None if lens is None else torch.tensor(lens, dtype=torch.int32))
    check_forward(x, *x.forward(mt))
    check_gradient(x, x.gradient(mt))

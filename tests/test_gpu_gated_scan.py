"""mt_gated_scan, its single-token form and its gradient against the recurrence
in 64 bits (gated_ref.GatedCase, which carries the bounds)."""
import pytest
import torch

import gated_ref as G
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
    buf = torch.full((*x.shape[:-1], x.shape[-1] + 2 * pad), NAN, dtype=x.dtype, device="cuda")
    view = buf[..., pad:pad + x.shape[-1]]
    view.copy_(x)
    return view


class Inputs:
    """`memory` is how long the states last: the decays' distance from 1 (with rate)."""

    def __init__(self, dtype, b, length, d, rate=True, i=True, z=False, h0=True, lens=None, seed=0, pad=0, memory=0.1):
        g = torch.Generator().manual_seed(100 * length + d + seed)
        r = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
        self.lens, self.pad = lens, pad
        mask = R.live_mask(lens, b, length)

        def act(by=1.0):
            x = (r(b, length, d) * by).to(dtype)
            x[~mask] = NAN  # what lies past a sequence's end must not be read
            return x

        self.x, self.r = act(), act(1.5)
        self.i, self.z = act() if i else None, act() if z else None
        self.rate = torch.rand(d, generator=g) * 12 * memory if rate else None  # u on both sides of 1/2
        self.h0 = r(b, d) if h0 else None
        self.dout, self.dfinal = act(), r(b, d)

    def case(self):
        return G.GatedCase(self.x, self.r, self.i, self.z, self.rate, self.h0, self.lens)

    def gates(self):
        c = lambda t: None if t is None else t.cuda()  # noqa: E731
        return dict(i=wide(self.i, self.pad), z=wide(self.z, self.pad), rate=c(self.rate), lens=c(self.lens))

    def forward(self, mt, checkpoints=None):
        b, length, d = self.x.shape
        out = wide(torch.full_like(self.x, 5.0), self.pad)
        carry = self.h0 is not None
        state = self.h0.cuda() if carry else torch.full((b, d), 9.0, device="cuda")
        mt.mt_gated_scan(wide(self.x, self.pad), wide(self.r, self.pad), out, state=state, carry_in=carry,
                         checkpoints=checkpoints, **self.gates())
        return out, state

    def gradient(self, mt, dfinal=True):
        b, length, d = self.x.shape
        ck = torch.full((max(1, mt.mt_gated_scan_checkpoint_slots(b, length, d)),), -1, dtype=torch.int64, device="cuda")
        self.forward(mt, ck)
        like = lambda: wide(torch.full_like(self.x, 5.0), self.pad)  # noqa: E731
        got = dict(dx=like(), dr=like(), dinit=torch.full((b, d), 5.0, device="cuda"))
        if self.i is not None:
            got["di"] = like()
        if self.z is not None:
            got["dz"] = like()
        scratch = None
        if self.rate is not None:
            got["drate"] = torch.full((d,), 5.0, device="cuda")
            scratch = torch.full((max(1, mt.mt_gated_scan_scratch_slots(b, length, d)),), -1, dtype=torch.int64, device="cuda")
        mt.mt_gated_scan_grad(wide(self.x, self.pad), wide(self.r, self.pad), wide(self.dout, self.pad), ck, scratch=scratch,
                              dfinal=self.dfinal.cuda() if dfinal else None, **got, **self.gates())
        return got


def check_forward(mt, p):
    out, state = p.forward(mt)
    want, final = p.case().forward()
    G.check("out", out, want)
    G.check("state", state, final)


def check_gradient(mt, p, dfinal=True):
    got = p.gradient(mt, dfinal)
    want = p.case().gradient(p.dout, p.dfinal if dfinal else None)
    assert set(got) == set(want)
    for name in want:
        G.check(name, got[name], want[name])


SIZES = [(1, 1, 1), (2, 7, 3), (1, 8, 64), (2, 63, 65), (1, 64, 128), (2, 65, 40), (3, 130, 33), (1, 513, 66), (2, 1030, 72)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,length,d", SIZES)
@pytest.mark.parametrize("rate,i,z", [(True, True, True), (True, False, False), (False, False, True), (False, True, False)])
def test_scan_and_gradient(mt, dtype, b, length, d, rate, i, z):
    p = Inputs(dtype, b, length, d, rate, i, z, h0=length % 2 == 1)
    check_forward(mt, p)
    check_gradient(mt, p, dfinal=d % 2 == 0)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rate", [True, False])
@pytest.mark.parametrize("pad", [0, 1, 8])
def test_ragged_and_strided(mt, dtype, rate, pad):
    lens = torch.tensor([0, 300, 1, 64, 65, 299], dtype=torch.int32)
    p = Inputs(dtype, 6, 300, 72, rate, True, True, lens=lens, pad=pad)
    check_forward(mt, p)
    check_gradient(mt, p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [9, 16, 17, 25, 33, 96, 160, 200, 380, 448])
@pytest.mark.parametrize("d", [64, 65])
def test_warps_and_ctas_by_length(mt, dtype, length, d):
    """Lengths from two warps of one CTA to clusters of each size, one sequence ending early."""
    p = Inputs(dtype, 2, length, d, True, True, length % 2 == 0, lens=torch.tensor([length, length * 2 // 3], dtype=torch.int32))
    check_forward(mt, p)
    check_gradient(mt, p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [3, 16, 40])
def test_many_short_sequences(mt, dtype, length):
    lens = torch.tensor([(k * 7) % (length + 1) for k in range(70)], dtype=torch.int32)
    p = Inputs(dtype, 70, length, 576, length != 16, True, True, lens=lens)
    check_forward(mt, p)
    check_gradient(mt, p)


@pytest.mark.parametrize("length", [1, 9, 130])
def test_terms_that_cancel(mt, length):
    """First states and last gradients that all but cancel what the first and last tokens add."""
    p = Inputs(torch.float32, 4, length, 312, False, False, False)
    s = torch.sigmoid(p.r[:, 0])
    p.h0 = -s * p.x[:, 0] / (1 - s) * 1.001
    p.dfinal = p.dout[:, -1] * -1.001
    check_forward(mt, p)
    check_gradient(mt, p)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("length", [2048, 4099])
def test_long_memory(mt, dtype, length):
    """Decays of 0.999 and above: the states sum thousands of tokens."""
    p = Inputs(dtype, 1, length, 16, True, True, False, memory=1e-4)
    check_forward(mt, p)
    check_gradient(mt, p)


def test_lengths_outside_the_prompt_are_clamped(mt):
    p = Inputs(torch.float32, 2, 20, 8, lens=torch.tensor([20, 0], dtype=torch.int32))
    want = p.forward(mt)
    p.lens = torch.tensor([25, -3], dtype=torch.int32)
    for a, b in zip(want, p.forward(mt)):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", DTYPES)
def test_empty_prompt_leaves_states(mt, dtype):
    x = torch.empty(2, 0, 8, dtype=dtype, device="cuda")
    state = torch.randn(2, 8, device="cuda")
    keep = state.clone()
    mt.mt_gated_scan(x, x, x, state=state, carry_in=True)
    assert torch.equal(state, keep)
    mt.mt_gated_scan(x, x, x, state=state)
    assert (state == 0).all()
    one = torch.empty(1, dtype=torch.int64, device="cuda")
    rate, drate, dfinal, dinit = torch.ones(8, device="cuda"), torch.full((8,), 5.0, device="cuda"), keep, torch.empty(2, 8, device="cuda")
    mt.mt_gated_scan_grad(x, x, x, one, x, x, torch.empty(64, dtype=torch.int64, device="cuda"), rate=rate, drate=drate,
                          dfinal=dfinal, dinit=dinit)
    assert (drate == 0).all() and torch.equal(dinit, dfinal)
    none = torch.empty(0, 3, 8, dtype=dtype, device="cuda")
    drate.fill_(5.0)
    mt.mt_gated_scan_grad(none, none, none, one, none, none, torch.empty_like(one), rate=rate, drate=drate)
    assert (drate == 0).all()


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rate", [True, False])
def test_prompt_in_parts_and_tokens(mt, dtype, rate):
    """A prompt, its two parts with the state between them, and its tokens one by one."""
    p = Inputs(dtype, 3, 140, 66, rate, True, True)
    want, final = p.case().forward()
    state = p.h0.cuda()
    c = lambda t, lo, hi: t[:, lo:hi].cuda()  # noqa: E731
    outs = []
    for lo, hi in ((0, 77), (77, 131)):
        out = torch.empty(3, hi - lo, 66, dtype=dtype, device="cuda")
        mt.mt_gated_scan(c(p.x, lo, hi), c(p.r, lo, hi), out, i=c(p.i, lo, hi), z=c(p.z, lo, hi),
                         rate=None if p.rate is None else p.rate.cuda(), state=state, carry_in=True)
        outs.append(out)
    for t in range(131, 140):
        out = torch.empty(3, 66, dtype=dtype, device="cuda")
        row = lambda v: v[:, t].cuda()  # noqa: E731
        mt.mt_gated_scan_step(row(p.x), row(p.r), state, out, i=row(p.i), z=row(p.z), rate=None if p.rate is None else p.rate.cuda())
        outs.append(out[:, None])
    G.check("out", torch.cat(outs, 1), want)
    G.check("state", state, final)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("d,pad", [(1, 0), (65, 0), (128, 1), (4096, 8)])
@pytest.mark.parametrize("batch", [1, 5])
def test_step(mt, dtype, d, pad, batch):
    for rate, i, z in ((True, True, False), (False, False, True), (True, False, True)):
        p = Inputs(dtype, batch, 1, d, rate, i, z, pad=pad)
        want, final = p.case().forward()
        state = p.h0.cuda()
        g = p.gates()
        row = lambda t: None if t is None else t[:, 0]  # noqa: E731
        out = wide(torch.full_like(p.x, 5.0), pad)[:, 0]
        mt.mt_gated_scan_step(row(wide(p.x, pad)), row(wide(p.r, pad)), state, out, i=row(g["i"]), z=row(g["z"]), rate=g["rate"])
        G.check("out", out, Inputs_row(want))
        G.check("state", state, final)


def Inputs_row(ball):
    return G.Ball(ball.v[:, 0], ball.e[:, 0])


@pytest.mark.parametrize("step", [False, True])
def test_slots(mt, step):
    """Rows of a pool in any order; a sequence whose slot is outside it is inactive."""
    p = Inputs(torch.bfloat16, 5, 1 if step else 70, 40, True, True, True)
    slots = torch.tensor([6, -1, 0, 7, 3], dtype=torch.int32, device="cuda")
    pool = torch.full((7, 40), 4.5, device="cuda")
    live = [0, 2, 4]
    pool[slots[live].long()] = p.h0.cuda()[live]
    g = p.gates()
    out = torch.full_like(p.x, 5.0).cuda()
    if step:
        mt.mt_gated_scan_step(p.x.cuda()[:, 0], p.r.cuda()[:, 0], pool, out[:, 0], i=g["i"][:, 0], z=g["z"][:, 0], rate=g["rate"],
                              slots=slots)
    else:
        mt.mt_gated_scan(p.x.cuda(), p.r.cuda(), out, i=g["i"], z=g["z"], rate=g["rate"], state=pool, carry_in=True, slots=slots)
    want, final = p.case().forward()
    G.check("out", out[live], G.Ball(want.v[live], want.e[live]))
    G.check("state", pool[slots[live].long()], G.Ball(final.v[live], final.e[live]))
    assert (out[[1, 3]] == 0).all() and (pool[[1, 2, 4, 5]] == 4.5).all()


@pytest.mark.parametrize("rate", [True, False])
def test_extreme_gates(mt, rate):
    """Gates far outside the usual range: shut, a token passes nothing and leaves the state bit for bit; open, it replaces it
    as far as the decay goes. Every result and gradient is finite."""
    d, n = 32, 96
    g = torch.Generator().manual_seed(1)
    x = torch.randn(1, n, d, generator=g).cuda()
    r = torch.full((1, n, d), -1e4).cuda()
    i = torch.where(torch.arange(d) % 2 == 0, 1e4, -1e4).expand(1, n, d).contiguous().cuda()
    z = torch.where(torch.arange(d) % 3 == 0, 200.0, -200.0).expand(1, n, d).contiguous().cuda()
    rt = torch.full((d,), 0.3, device="cuda") if rate else None
    h0 = torch.randn(1, d, generator=g).cuda()
    state, out = h0.clone(), torch.empty_like(x)
    mt.mt_gated_scan(x, r, out, i=i, rate=rt, state=state, carry_in=True)
    assert torch.equal(state, h0) and torch.equal(out, h0[:, None].expand_as(out))
    big = torch.where(torch.arange(n) % 5 == 0, 1e4, -60.0)[None, :, None].expand(1, n, d).contiguous().cuda()
    ck = torch.empty(mt.mt_gated_scan_checkpoint_slots(1, n, d), dtype=torch.int64, device="cuda")
    scratch = torch.empty(mt.mt_gated_scan_scratch_slots(1, n, d), dtype=torch.int64, device="cuda")
    for gate in (r, big):
        mt.mt_gated_scan(x, gate, out, i=i, z=z, rate=rt, state=state, checkpoints=ck)
        got = [torch.empty_like(x) for _ in range(4)]
        drate = torch.empty(d, device="cuda") if rate else None
        dinit = torch.empty_like(h0)
        mt.mt_gated_scan_grad(x, gate, x, ck, got[0], got[1], scratch, i=i, di=got[2], z=z, dz=got[3], rate=rt, drate=drate, dinit=dinit)
        for t in (out, state, dinit, *got) + ((drate,) if rate else ()):
            assert torch.isfinite(t).all()
    if not rate:  # the state is the last input that was let in
        out2 = torch.empty_like(x)
        mt.mt_gated_scan(x, big, out2)
        assert torch.equal(out2[:, 95], x[:, 95])


def test_rate_of_zero(mt):
    """Nothing is forgotten and nothing let in; the derivative of the weight there counts as 0."""
    x = torch.randn(2, 70, 8, device="cuda")
    rate, h0 = torch.zeros(8, device="cuda"), torch.randn(2, 8, device="cuda")
    out, state = torch.empty_like(x), h0.clone()
    ck = torch.empty(mt.mt_gated_scan_checkpoint_slots(2, 70, 8), dtype=torch.int64, device="cuda")
    mt.mt_gated_scan(x, x, out, rate=rate, state=state, carry_in=True, checkpoints=ck)
    assert torch.equal(out, h0[:, None].expand_as(out)) and torch.equal(state, h0)
    dx, dr, drate, dinit = torch.empty_like(x), torch.empty_like(x), torch.empty_like(rate), torch.empty_like(h0)
    scratch = torch.empty(mt.mt_gated_scan_scratch_slots(2, 70, 8), dtype=torch.int64, device="cuda")
    mt.mt_gated_scan_grad(x, x, x, ck, dx, dr, scratch, rate=rate, drate=drate, dinit=dinit)
    assert (dx == 0).all() and (dr == 0).all() and torch.isfinite(drate).all()
    want = x.double().sum(1)
    R.assert_within("dinit", dinit, want, 70 * R.U * x.double().abs().sum(1).cpu())


def test_a_nan_stays_in_its_channel_and_after_it(mt):
    x = torch.randn(2, 200, 64, device="cuda")
    clean = torch.empty_like(x)
    mt.mt_gated_scan(x, x, clean)
    bad = x.clone()
    bad[1, 100, 5] = NAN
    out = torch.empty_like(x)
    mt.mt_gated_scan(bad, x, out)
    assert out[1, 100:, 5].isnan().all()
    out[1, 100:, 5] = clean[1, 100:, 5]
    assert torch.equal(out, clean)


def test_same_bits_every_time(mt):
    p = Inputs(torch.bfloat16, 3, 1100, 130, True, True, True)
    first = (*p.forward(mt), *p.gradient(mt).values())
    for a, b in zip(first, (*p.forward(mt), *p.gradient(mt).values())):
        assert torch.equal(a, b)

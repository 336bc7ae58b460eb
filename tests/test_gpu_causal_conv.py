"""mt_causal_conv, its single-token form and its gradient against 64 bits.

Bounds: p is width + 1 f32 terms: (width + 2) U sum|terms|; SiLU's slope is at
most 1.1 and its sigmoid is off by two evaluations (2 EX relative). The
gradient's g = dout * slope: the slope's own slope is at most 0.5, its evaluation 4 EX of at most 1.1.
Sums over n tokens are n f32 terms at most in a row: n U sum|terms|."""
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


def gen(seed):
    return torch.Generator().manual_seed(seed)


def wide(x, pad):
    """x on the GPU as a part of wider rows (pad channels before and after it)."""
    if pad == 0:
        return x.cuda()
    buf = torch.full((*x.shape[:-1], x.shape[-1] + 2 * pad), NAN, dtype=x.dtype, device="cuda")
    view = buf[..., pad:pad + x.shape[-1]]
    return view.copy_(x)


def make(seed, dtype, wdtype, b, length, d, width, lens):
    g = gen(seed)
    x = torch.randn(b, length, d, generator=g).to(dtype)
    mask = R.live_mask(lens, b, length)
    x[~mask] = NAN  # what lies past a sequence's end must not be read
    w = torch.randn(d, width, generator=g).mul_(0.5).to(wdtype)
    bias = torch.randn(d, generator=g).mul_(0.3).to(wdtype)
    state = torch.randn(b, width - 1, d, generator=g).to(dtype)
    return g, x, mask, w, bias, state


def bounds(x, w, bias, before, mask, silu):
    mag, _, pm = R.conv(x.abs(), w.abs(), None if bias is None else bias.abs(), False, before.abs(), mask)
    return pm


SHAPES = [(1, 1, 1, 1), (1, 1, 8, 4), (2, 2, 5, 4), (3, 5, 32, 3), (2, 33, 7, 4), (1, 100, 136, 2), (4, 64, 24, 4)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES)
@pytest.mark.parametrize("silu,with_bias,carry,ragged,pad", [(True, True, False, False, 0), (False, True, True, True, 8),
                                                            (True, False, True, False, 3), (True, True, True, True, 1)])
def test_prompt(mt, dtype, shape, silu, with_bias, carry, ragged, pad):
    b, length, d, width = shape
    lens = torch.arange(b, dtype=torch.int32) * 2 - 1 if ragged else None  # -1 (as 0), 1, 3, ...
    wdtype = torch.float32 if pad % 2 else dtype
    _, x, mask, w, bias, state = make(length + d, dtype, wdtype, b, length, d, width, lens)
    bias = bias if with_bias else None
    st, out = state.cuda(), wide(torch.full_like(x, 5.0), pad)
    mt.mt_causal_conv(wide(x, pad), w.cuda(), out, bias=None if bias is None else bias.cuda(), silu=silu, state=st, carry_in=carry,
                      lens=None if lens is None else lens.cuda())
    xz = R.zeroed(x, mask)
    before = state.double() if carry else torch.zeros_like(state, dtype=R.F64)
    bias64 = None if bias is None else bias.double()
    want, px, _ = R.conv(xz, w.double(), bias64, silu, before, mask)
    pm = bounds(xz, w.double(), bias64, before, mask, silu)
    slack = torch.where(mask[..., None], (1.1 * (width + 2) * R.U + (2 * R.EX + 2 * R.U if silu else 0)) * pm, 0.0)
    R.assert_within("out", out, want, slack)
    last = torch.stack([px[i, n:n + width - 1] for i, n in enumerate(mask.sum(1).tolist())])
    assert torch.equal(st.cpu().double(), last)  # inputs are copied


@pytest.mark.parametrize("dtype", DTYPES)
def test_slots_and_inactive_sequences(mt, dtype):
    b, length, d, width = 4, 6, 12, 4
    _, x, mask, w, bias, _ = make(2, dtype, dtype, b, length, d, width, None)
    pool = torch.randn(7, width - 1, d, generator=gen(4)).to(dtype)
    slots = torch.tensor([5, -1, 0, 7], dtype=torch.int32)
    st, out = pool.cuda(), torch.full((b, length, d), 5.0, dtype=dtype, device="cuda")
    args = dict(bias=bias.cuda(), slots=slots.cuda())
    mt.mt_causal_conv(x.cuda(), w.cuda(), out, state=st, carry_in=True, **args)
    for i, s in ((0, 5), (2, 0)):
        alone = pool[s:s + 1].cuda()
        o = torch.empty(1, length, d, dtype=dtype, device="cuda")
        mt.mt_causal_conv(x[i:i + 1].cuda(), w.cuda(), o, bias=bias.cuda(), state=alone, carry_in=True)
        assert torch.equal(o[0], out[i]) and torch.equal(alone[0], st[s])
    assert (out[[1, 3]] == 0).all()
    others = [1, 2, 3, 4, 6]
    assert torch.equal(st.cpu()[others], pool[others])
    st2, o2 = pool.cuda(), torch.full((b, d), 5.0, dtype=dtype, device="cuda")
    mt.mt_causal_conv_step(x[:, 0].cuda(), w.cuda(), st2, o2, **args)
    assert (o2[[1, 3]] == 0).all() and torch.equal(o2[[0, 2]], out[[0, 2], 0])
    assert torch.equal(st2.cpu()[others], pool[others])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,d,width,pad", [(1, 1, 2, 0), (3, 7, 4, 2), (5, 64, 3, 8), (2, 40, 1, 0)])
def test_token_by_token_is_the_prompt(mt, dtype, b, d, width, pad):
    """Steps from a zero state give the prompt's outputs and state, bit for bit (the same sums in the same order)."""
    length = 6
    _, x, _, w, bias, _ = make(d, dtype, torch.float32, b, length, d, width, None)
    whole = torch.empty(b, length, d, dtype=dtype, device="cuda")
    s1 = torch.full((b, width - 1, d), 9.0, dtype=dtype, device="cuda")
    mt.mt_causal_conv(x.cuda(), w.cuda(), whole, bias=bias.cuda(), state=s1)
    s2 = torch.zeros_like(s1)
    xg = wide(x, pad)
    for t in range(length):
        o = torch.empty(b, d, dtype=dtype, device="cuda")
        mt.mt_causal_conv_step(xg[:, t], w.cuda(), s2, o, bias=bias.cuda())
        assert torch.equal(o, whole[:, t])
    assert torch.equal(s1, s2)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("shape", SHAPES + [(2, 520, 9, 4), (1, 1100, 40, 4)])
@pytest.mark.parametrize("silu,with_bias,carry,ragged,pad", [(True, True, False, False, 0), (False, True, True, True, 8),
                                                            (True, False, True, True, 3)])
def test_gradient(mt, dtype, shape, silu, with_bias, carry, ragged, pad):
    b, length, d, width = shape
    lens = torch.arange(b, dtype=torch.int32) * 2 + length - 2 * b + 1 if ragged else None
    g, x, mask, w, bias, state = make(length + d, dtype, torch.float32, b, length, d, width, lens)
    bias = bias if with_bias else None
    dout = torch.randn(b, length, d, generator=g).to(dtype)
    dout[~mask] = NAN
    dx = wide(torch.full_like(x, 5.0), pad)
    dw, db = torch.empty(d, width, device="cuda"), torch.empty(d, device="cuda")
    ds = torch.empty(b, width - 1, d, dtype=dtype, device="cuda")
    scratch = torch.empty(mt.mt_causal_conv_grad_scratch_slots(b, length, d, width), dtype=torch.int64, device="cuda")
    mt.mt_causal_conv_grad(wide(x, pad), w.cuda(), wide(dout, pad), dx, dw, scratch, bias=None if bias is None else bias.cuda(),
                           dbias=db, silu=silu, state=state.cuda() if carry else None, dstate=ds,
                           lens=None if lens is None else lens.cuda())
    xz, gz = R.zeroed(x, mask), R.zeroed(dout, mask)
    before = state.double() if carry else torch.zeros_like(state, dtype=R.F64)
    b64, w64 = None if bias is None else bias.double(), w.double()
    want = R.conv_grad(xz, w64, b64, silu, before, mask, gz)
    pm = bounds(xz, w64, b64, before, mask, silu)
    # |g| <= 1.1 |dout|; its error: 0.5 dp |dout| + (4 EX + 4 U) 1.1 |dout|
    off = (0.5 * (width + 2) * R.U * pm + 1.1 * (4 * R.EX + 4 * R.U)) if silu else torch.full_like(pm, 2 * R.U)
    err = R.conv_grad(xz.abs(), w64.abs(), b64, silu, before.abs(), mask, gz.abs(), slope=off)
    top = R.conv_grad(xz.abs(), w64.abs(), b64, silu, before.abs(), mask, gz.abs(), slope=torch.full_like(pm, 1.1))
    n = b * length + 8
    for name, got, i, terms in (("dx", dx, 0, width + 1), ("dweight", dw, 1, n), ("dbias", db, 2, n), ("dstate", ds, 3, width + 1)):
        R.assert_within(name, got, want[i], err[i] + terms * R.U * top[i])


def test_gradient_of_nothing_is_zero(mt):
    for b, length in ((0, 5), (2, 0)):
        e = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
        dw, db, ds = torch.full((6, 4), 3.0, device="cuda"), torch.full((6,), 3.0, device="cuda"), torch.full((b, 3, 6), 3.0, device="cuda")
        scratch = torch.empty(max(1, mt.mt_causal_conv_grad_scratch_slots(b, length, 6, 4)), dtype=torch.int64, device="cuda")
        mt.mt_causal_conv_grad(e(b, length, 6), e(6, 4).zero_(), e(b, length, 6), e(b, length, 6), dw, scratch, dbias=db, dstate=ds)
        assert (dw == 0).all() and (db == 0).all() and (ds == 0).all()
    state = torch.full((2, 3, 6), 3.0, device="cuda")
    mt.mt_causal_conv(e(2, 0, 6), e(6, 4), e(2, 0, 6), state=state, carry_in=True)
    assert (state == 3).all()
    mt.mt_causal_conv(e(2, 0, 6), e(6, 4), e(2, 0, 6), state=state)
    assert (state == 0).all()


def test_same_bits_each_time(mt):
    _, x, _, w, bias, _ = make(1, torch.bfloat16, torch.float32, 3, 700, 264, 4, None)
    dout = torch.randn(x.shape, generator=gen(6)).to(x.dtype).cuda()
    got = []
    for fill in (0, -1):
        r = [torch.empty_like(dout), torch.empty(264, 4, device="cuda"), torch.empty(264, device="cuda")]
        scratch = torch.full((mt.mt_causal_conv_grad_scratch_slots(3, 700, 264, 4),), fill, dtype=torch.int64, device="cuda")
        mt.mt_causal_conv_grad(x.cuda(), w.cuda(), dout, r[0], r[1], scratch, bias=bias.cuda(), dbias=r[2])
        got.append(r)
    assert all(torch.equal(a, b) for a, b in zip(*got))

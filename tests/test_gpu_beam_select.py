"""mt_beam_select against all continuations sorted in 64 bits (gated_ref.beam_select). Tokens, parents, marks, slots and copies
must be equal. A score is off by the rounding to f32, and before it by that of its beam's sum: a sum of f32 terms in
spans of at most 64, (64 + 8) U, of exponentials good to 2^-21, which the logarithm passes on as an absolute error."""
import pytest
import torch

import gated_ref as G
import seq_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]
INF = float("inf")
SLACK = 72 * R.U + 2.0 ** -21


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def run(mt, logits, k_out, prior=None, finished=None, eos=-1, slots=None, in_place=False):
    b, k, v = logits.shape
    c = lambda t: None if t is None else t.cuda()  # noqa: E731
    prior, finished, slots = c(prior), c(finished), c(slots)
    new = lambda dtype: torch.full((b, k_out), 77, dtype=dtype, device="cuda")  # noqa: E731
    tokens, parents, src, dst = (new(torch.int32) for _ in range(4))
    scores = prior if in_place else new(torch.float32)
    marks = finished if in_place and finished is not None else new(torch.uint8)
    scratch = torch.full((mt.mt_beam_select_scratch_slots(b, k, k_out, v),), -1, dtype=torch.int64, device="cuda")
    mt.mt_beam_select(logits, tokens, parents, scores, scratch, prior=prior, finished=finished, finished_out=marks, eos=eos, slots=slots,
                      src=src if slots is not None else None, dst=dst if slots is not None else None)
    got = dict(tokens=tokens, parents=parents, scores=scores, finished=marks)
    if slots is not None:
        got.update(slots=slots, src=src, dst=dst)
    return got


def check(mt, logits, k_out, prior=None, finished=None, eos=-1, slots=None, in_place=False, view=None):
    want = G.beam_select(logits, k_out, prior, finished, eos, slots)
    got = run(mt, logits.cuda() if view is None else view, k_out, prior, finished, eos, slots, in_place)
    for name in want:
        if name != "scores":
            assert torch.equal(got[name].cpu().long(), want[name]), (name, got[name], want[name])
    w = want["scores"]
    hard = torch.isinf(w)
    assert torch.equal(torch.isinf(got["scores"]).cpu(), hard)
    R.assert_within("scores", torch.where(hard.cuda(), 0.0, got["scores"]), torch.where(hard, 0.0, w), torch.full_like(w, SLACK))


def rows(dtype, b, k, v, seed=0, by=2.0):
    g = torch.Generator().manual_seed(b * 1000 + k * 100 + v + seed)
    x = (torch.randn(b, k, v, generator=g) * by).to(dtype)
    prior = -torch.rand(b, k, generator=g) * 5 - 10
    slots = torch.randperm(3 * b * 32, generator=g).to(torch.int32)
    return x, prior, slots, g


SIZES = [(1, 1, 1, 1), (1, 1, 4, 5), (2, 4, 4, 1000), (3, 7, 7, 5003), (1, 32, 32, 777), (2, 3, 32, 20), (2, 2, 5, 3), (4, 8, 8, 8192),
         (2, 5, 3, 8193), (1, 2, 2, 32773), (1, 1, 32, 70001), (70, 3, 3, 65), (1, 4, 4, 131072), (1, 2, 16, 16384), (1, 9, 17, 24999)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,k,k_out,v", SIZES)
def test_selection(mt, dtype, b, k, k_out, v):
    x, prior, slots, g = rows(dtype, b, k, v)
    group = max(k, k_out)
    check(mt, x, k_out, prior, slots=slots[:b * group].view(b, group))
    check(mt, x, k_out)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,k,v", [(2, 4, 1000), (3, 8, 9001), (1, 16, 20000), (2, 32, 300)])
def test_finished_beams(mt, dtype, b, k, v):
    x, prior, slots, g = rows(dtype, b, k, v, 1)
    for ended in (torch.rand(b, k, generator=g) < 0.4, torch.ones(b, k, dtype=torch.bool)):
        x = x.clone()
        x[ended] = float("nan")  # not read
        for eos in (0, 7, v - 1):
            check(mt, x, k, prior, ended.to(torch.uint8) * 3, eos, slots[:b * k].view(b, k), in_place=eos == 7)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,k,v", [(2, 4, 1000), (2, 8, 9001), (1, 32, 40000), (3, 5, 64)])
def test_equal_logits(mt, dtype, b, k, v):
    """Ties by the hundred: within a beam the lowest token, between beams (with equal priors and rows) the lowest beam."""
    x, prior, _, g = rows(dtype, b, k, v, 2)
    x = torch.randint(-2, 3, (b, k, v), generator=g).to(dtype)
    check(mt, x, k, prior)
    same = x[:, :1].expand(b, k, v).contiguous()
    check(mt, same, k, torch.full((b, k), -1.5))
    check(mt, torch.zeros(b, k, v, dtype=dtype), k)
    check(mt, -torch.zeros(b, k, v, dtype=dtype) * (torch.arange(v) % 2), k)  # 0 and -0 are equal


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("up", [True, False])
def test_sorted_logits(mt, dtype, up):
    """The best tokens all in one place, at the start or at the end."""
    v = 30000
    x = torch.linspace(-3, 3, v)
    x = (x if up else x.flip(0)).to(dtype).expand(2, 32, v).contiguous()
    prior = -torch.arange(64, dtype=torch.float32).view(2, 32) * 0.037
    check(mt, x, 32, prior)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("v", [40, 9000])
def test_masked_tokens(mt, dtype, v):
    """Tokens that may not come next, rows with none, fewer than are asked for, and masks of the type's lowest value."""
    x, prior, slots, g = rows(dtype, 4, 6, v, 3)
    x[torch.rand(x.shape, generator=g) < 0.5] = -INF
    x[torch.rand(x.shape, generator=g) < 0.2] = float("nan")
    x[0, 1] = -INF
    x[0, 2] = float("nan")
    x[1] = -INF  # a sequence with no continuation at all
    x[2] = -INF
    x[2, 3, 5], x[2, 4, 17] = 1.0, 0.5  # two continuations for six places
    x[3, 0] = torch.finfo(dtype).min
    x[3, 1, 1:] = torch.finfo(dtype).min
    prior[0, 4], prior[3, 5] = -INF, float("nan")
    check(mt, x, 6, prior, slots=slots[:24].view(4, 6))
    check(mt, x, 9, prior)
    ended = torch.zeros(4, 6, dtype=torch.uint8)
    ended[1, 2] = ended[0, 4] = 1
    check(mt, x, 6, prior, ended, 3)


@pytest.mark.parametrize("dtype", DTYPES)
def test_infinite_logits(mt, dtype):
    """+inf counts as the largest finite value: it takes all of the probability, in equal shares."""
    x, prior, _, _ = rows(dtype, 2, 3, 500, 4)
    x[0, 1, 30] = INF
    x[1, 0, 5] = x[1, 0, 7] = INF
    check(mt, x, 3, prior)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("offset,width", [(0, 8200), (1, 8201), (3, 9000), (8, 8208)])
def test_rows_of_wider_tensors(mt, dtype, offset, width):
    v = 8190
    x, prior, _, _ = rows(dtype, 3, 4, v, 5)
    buf = torch.full((3, 5, width), INF, dtype=dtype, device="cuda")
    view = buf[:, 1:, offset:offset + v]
    view.copy_(x)
    check(mt, x, 4, prior, view=view)
    turned = torch.full((4, 3, width), INF, dtype=dtype, device="cuda")[:, :, offset:offset + v].transpose(0, 1)
    turned.copy_(x)
    check(mt, x, 4, prior, view=turned)


@pytest.mark.parametrize("dtype", DTYPES)
def test_wide_range_and_peaked(mt, dtype):
    x, prior, _, g = rows(dtype, 2, 4, 20000, 6, by=10.0)
    check(mt, x, 4, prior)
    x[:, :, 123] = 500.0  # one token has it all
    check(mt, x, 4, prior)
    check(mt, x, 4, prior - 1e6)


def test_same_bits_every_time(mt):
    x, prior, _, _ = rows(torch.bfloat16, 8, 16, 50001, 7)
    first = run(mt, x.cuda(), 16, prior)
    for _ in range(3):
        again = run(mt, x.cuda(), 16, prior)
        assert all(torch.equal(first[n], again[n]) for n in first)


def test_more_rows_than_a_grids_second_axis(mt):
    x, prior, _, _ = rows(torch.float32, 9000, 8, 9, 8)
    check(mt, x, 8, prior)

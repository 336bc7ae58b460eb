"""mt_embed and mt_embed_grad against plain forms: the lookup bit for bit (one
f32 product, rounded once), the gradient against sums in 64 bits.

Bound of the gradient: a run of k rows is summed in k f32 additions in some
fixed grouping, then scaled: (k + 2) U scale sum|dout|, plus one rounding to the
gradient's type."""
import pytest
import torch

import seq_ref as R

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def gen(seed):
    return torch.Generator().manual_seed(seed)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("tok", [torch.int32, torch.int64])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 1), (5, 3, 7), (33, 100, 64), (7, 50, 1001), (300, 17, 4096), (2, 9, 8), (64, 40, 130)])
def test_lookup(mt, dtype, tok, n, vocab, dim):
    g = gen(n + dim)
    table = torch.randn(vocab, dim, generator=g).to(dtype)
    tokens = torch.randint(-1, vocab + 1, (n,), generator=g).to(tok)  # -1 and vocab name no row
    for scale in (1.0, 0.37):
        out = torch.full((n, dim), 9.0, dtype=dtype, device="cuda")
        mt.mt_embed(tokens.cuda(), table.cuda(), out, scale=scale)
        has = (tokens >= 0) & (tokens < vocab)
        rows = (table[tokens.long().clamp(0, vocab - 1)].float() * torch.tensor(scale)).to(dtype)
        want = torch.where(has[:, None], rows, torch.zeros((), dtype=dtype))
        assert torch.equal(out.cpu(), want)


def test_lookup_of_unaligned_rows_and_shapes(mt):
    table = torch.randn(20, 24, generator=gen(1)).to(torch.bfloat16).cuda()
    odd = torch.empty(20 * 24 + 1, dtype=torch.bfloat16, device="cuda")[1:].view(20, 24).copy_(table)
    tokens = torch.arange(12, dtype=torch.int32, device="cuda").view(3, 4)
    a, b = (torch.empty(3, 4, 24, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    mt.mt_embed(tokens, table, a)
    mt.mt_embed(tokens, odd, b)
    assert torch.equal(a, b) and torch.equal(a.view(12, 24), table[:12])
    mt.mt_embed(tokens[:0], table, a[:0])  # nothing to do


def tokens_of(kind, n, vocab, g):
    if kind == "one":
        return torch.full((n,), vocab // 2)
    if kind == "none":
        return torch.full((n,), -1)
    if kind == "each":
        return torch.randperm(max(n, vocab), generator=g)[:n] % vocab
    if kind == "edges":  # long runs of the first and the last row, holes and strangers between
        t = torch.randint(-3, vocab + 3, (n,), generator=g)
        t[: n // 3] = 0
        t[n // 2:] = vocab - 1
        return t
    return torch.exp(torch.rand(n, generator=g) * torch.log(torch.tensor(vocab + 1.0))).long() - 1


def check_grad(got, tokens, dout, scale, base=None):
    vocab, dim = got.shape
    t = tokens.long()
    has = (t >= 0) & (t < vocab)
    sums = torch.zeros(vocab, dim, dtype=R.F64).index_add_(0, t[has], dout[has].double())
    mags = torch.zeros(vocab, dim, dtype=R.F64).index_add_(0, t[has], dout[has].double().abs())
    runs = torch.bincount(t[has], minlength=vocab).double()
    want = scale * sums
    slack = (runs[:, None] + 2) * R.U * scale * mags
    if base is not None:
        want = want + base.double()
        slack = slack + 2 * R.U * base.double().abs()
        assert torch.equal(got.cpu()[runs == 0], base[runs == 0])
    else:
        assert (got.cpu()[runs == 0] == 0).all()
    R.assert_within("dtable", got, want, slack)


@pytest.mark.parametrize("dtype,grad", [(torch.float32, torch.float32), (torch.bfloat16, torch.float32), (torch.float16, torch.float32),
                                        (torch.bfloat16, torch.bfloat16), (torch.float16, torch.float16)])
@pytest.mark.parametrize("kind", ["zipf", "one", "none", "each", "edges"])
@pytest.mark.parametrize("n,vocab,dim", [(1, 1, 8), (31, 40, 16), (33, 7, 33), (1000, 5000, 130), (5000, 3, 24)])
def test_gradient(mt, dtype, grad, kind, n, vocab, dim):
    g = gen(n)
    tokens = tokens_of(kind, n, vocab, g).to(torch.int32)
    dout = torch.randn(n, dim, generator=g).to(dtype)
    scratch = torch.empty(mt.mt_embed_grad_scratch_slots(n, vocab, dim), dtype=torch.int64, device="cuda")
    got = torch.full((vocab, dim), 7.0, dtype=grad, device="cuda")
    mt.mt_embed_grad(tokens.cuda(), dout.cuda(), got, scratch, scale=1.5)
    check_grad(got, tokens, dout, 1.5)
    base = torch.randn(vocab, dim, generator=g).to(grad)
    more = base.cuda()
    mt.mt_embed_grad(tokens.cuda(), dout.cuda(), more, scratch, scale=1.5, accumulate=True)
    check_grad(more, tokens, dout, 1.5, base)


@pytest.mark.parametrize("tok", [torch.int32, torch.int64])
def test_gradient_of_many_tokens_is_the_same_bits_each_time(mt, tok):
    """Long runs over many pieces, a vocabulary of many ranges; twice the same bits, whatever the scratch held."""
    g = gen(3)
    n, vocab, dim = 40_000, 200_000, 40
    tokens = tokens_of("zipf", n, vocab, g).to(tok)
    tokens[::3] = 77
    dout = torch.randn(n, dim, generator=g).to(torch.bfloat16)
    scratch = torch.full((mt.mt_embed_grad_scratch_slots(n, vocab, dim),), -1, dtype=torch.int64, device="cuda")
    got = [torch.empty(vocab, dim, device="cuda") for _ in range(2)]
    for t in got:
        mt.mt_embed_grad(tokens.cuda(), dout.cuda(), t, scratch)
    check_grad(got[0], tokens, dout, 1.0)
    assert torch.equal(got[0], got[1])


def test_gradient_of_no_tokens(mt):
    empty = torch.empty(0, dtype=torch.int32, device="cuda")
    dout = torch.empty(0, 8, device="cuda")
    scratch = torch.empty(mt.mt_embed_grad_scratch_slots(0, 5, 8), dtype=torch.int64, device="cuda")
    got = torch.full((5, 8), 3.0, device="cuda")
    mt.mt_embed_grad(empty, dout, got, scratch, accumulate=True)
    assert (got == 3).all()
    mt.mt_embed_grad(empty, dout, got, scratch)
    assert (got == 0).all()


def test_gradient_is_the_lookups_adjoint(mt):
    """<lookup(table), dout> = <table, gradient(dout)> on small integers, where every sum is exact."""
    g = gen(8)
    n, vocab, dim = 700, 90, 48
    tokens = torch.randint(-1, vocab, (n,), generator=g).to(torch.int32).cuda()
    table = torch.randint(-8, 9, (vocab, dim), generator=g).float().cuda()
    dout = torch.randint(-8, 9, (n, dim), generator=g).float().cuda()
    out, got = torch.empty(n, dim, device="cuda"), torch.empty(vocab, dim, device="cuda")
    mt.mt_embed(tokens, table, out, scale=2.0)
    scratch = torch.empty(mt.mt_embed_grad_scratch_slots(n, vocab, dim), dtype=torch.int64, device="cuda")
    mt.mt_embed_grad(tokens, dout, got, scratch, scale=2.0)
    assert (out.double() * dout.double()).sum() == (table.double() * got.double()).sum()

"""The gated scan where CTAs of a cluster share a sequence's tokens and tell one another their elements at every tile; and where one of
them does not (by the host's test hook), so that the others' waits run out: the call ends, says so, and leaves other sequences and channels
and later calls alone."""
import pytest
import torch

from test_gpu_gated_scan import Inputs, check_forward, check_gradient

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,d", [(1, 200), (9, 257), (11, 448)])  # clusters of 8, of 5 and of 3
def test_many_exchanges(mt, dtype, b, d):
    """Each side of the exchange used many times, beside other clusters on the same SMs; the same bits in every call."""
    lens = torch.tensor([1500 - 97 * n for n in range(b)], dtype=torch.int32)
    p = Inputs(dtype, b, 1500, d, True, True, True, lens=lens)
    check_forward(mt, p)
    check_gradient(mt, p)
    first = (*p.forward(mt), *p.gradient(mt).values())
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(first, (*p.forward(mt), *p.gradient(mt).values())))
    assert mt.mt_scan_status() == 0


class Withheld:
    """`silent` is the CTA that stops before its first tile (-1: none), `polls` the limit of each wait."""

    def __init__(self, mt, silent, polls):
        self.mt, self.silent, self.polls = mt, silent, polls

    def __enter__(self):
        self.mt.mt_scan_debug_lookback(skip_publish_tile=self.silent, spin_limit=self.polls)

    def __exit__(self, *_):
        self.mt.mt_scan_debug_lookback(-1, 0)


def calls(mt, p):
    """The forward call, and the gradient with the checkpoints of an undisturbed one, each with fresh outputs."""
    b, length, d = p.x.shape
    x, r, dout, h0 = p.x.cuda(), p.r.cuda(), p.dout.cuda(), p.h0.cuda()
    g = p.gates()
    ck = torch.zeros(mt.mt_gated_scan_checkpoint_slots(b, length, d), dtype=torch.int64, device="cuda")
    scratch = torch.zeros(mt.mt_gated_scan_scratch_slots(b, length, d), dtype=torch.int64, device="cuda")

    def forward(checkpoints=None):
        out, state = torch.full_like(x, 5.0), h0.clone()
        mt.mt_gated_scan(x, r, out, state=state, carry_in=True, checkpoints=checkpoints, **g)
        return dict(out=out, state=state)

    forward(ck)

    def gradient():
        got = {n: torch.full_like(x, 5.0) for n in ("dx", "dr", "di", "dz")}
        got.update(dinit=torch.full_like(h0, 5.0), drate=torch.full((d,), 5.0, device="cuda"))
        mt.mt_gated_scan_grad(x, r, dout, ck, scratch=scratch, **got, **g)
        return got

    return forward, gradient


# sequences, tokens, channels, CTAs of a cluster forward and backward, for 16-bit types; two slabs of channels each, so that block n + c
# is CTA c of a cluster of n for the first sequence's second slab
WITHHELD = [(2, 1500, 128, 8, 8), (2, 500, 128, 8, 8), (2, 160, 128, 3, 5), (2, 64, 128, 1, 2), (3, 128, 128, 2, 4)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("b,length,d,fwd,bwd", WITHHELD)
@pytest.mark.parametrize("last", [False, True])
def test_waits_that_run_out(mt, dtype, b, length, d, fwd, bwd, last):
    p = Inputs(dtype, b, length, d, True, True, True)
    for call, ctas in zip(calls(mt, p), (fwd, bwd)):
        if ctas == 1:
            continue
        want = call()
        assert mt.mt_scan_status() == 0
        with Withheld(mt, ctas + (ctas - 1 if last else 0), 4096):  # of the first sequence's second slab
            got = call()
            assert mt.mt_scan_status() == mt.MT_ERR_LOOKBACK_TIMEOUT
        for name in want:
            w, g = want[name], got[name]
            if name == "drate":  # summed over sequences
                assert torch.equal(w[:64], g[:64])
            else:
                assert torch.equal(w[0, ..., :64], g[0, ..., :64]) and torch.equal(w[1:], g[1:]), name
        again = call()
        assert mt.mt_scan_status() == 0
        assert all(torch.equal(want[n], again[n]) for n in want)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("b,d", [(1, 200), (9, 257)])
@pytest.mark.parametrize("polls", [1, 2, 5])
def test_waits_too_short_to_be_kept(mt, dtype, b, d, polls):
    """Waits of a poll or a few, which give up at any tile of any CTA, or not."""
    p = Inputs(dtype, b, 1500, d, True, True, True)
    for call in calls(mt, p):
        want = call()
        assert mt.mt_scan_status() == 0
        with Withheld(mt, -1, polls):
            for _ in range(5):
                got = call()
                status = mt.mt_scan_status()
                assert status == mt.MT_ERR_LOOKBACK_TIMEOUT or (status == 0 and all(torch.equal(want[n], got[n]) for n in want))
        again = call()
        assert mt.mt_scan_status() == 0
        assert all(torch.equal(want[n], again[n]) for n in want)

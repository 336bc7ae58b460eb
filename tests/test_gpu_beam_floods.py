"""mt_beam_select where more logits reach the last chosen one's score than the kernel has places for, so that it chooses again among the
groups' vectors and then among their logits: many sequences side by side, which reach that at different times, and calls one
after the other. Tokens, parents, marks, slots and copies are the lowest places of the highest value, which needs no sum; scores
and all else are the same bits in every sequence and call."""
import math

import pytest
import torch

from test_gpu_beam_select import SLACK, check, run

pytestmark = pytest.mark.gpu
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def first_places(k, k_out, v, start):
    """Parents and tokens of the first k_out places at or behind `start` in each row, rows in order."""
    places = [(j, t) for j in range(k) for t in range(start, min(v, start + k_out))][:k_out]
    return torch.tensor([p for p, _ in places]), torch.tensor([t for _, t in places])


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("k,k_out,v", [(1, 2, 16384), (4, 4, 9001), (2, 32, 2500), (16, 16, 5000), (8, 3, 1600)])
@pytest.mark.parametrize("start", [0, 77])
def test_floods_in_many_sequences(mt, dtype, k, k_out, v, start):
    """Every logit from `start` on the row's largest; 400 CTAs, so that an SM holds several, at different places in their work."""
    b = 400
    x = torch.full((1, k, v), -3.0, dtype=dtype)
    x[..., start:] = 1.0
    x = x.cuda().expand(b, k, v).contiguous()
    parents, tokens = first_places(k, k_out, v, start)
    group = max(k, k_out)
    slots = torch.arange(b * group, dtype=torch.int32).view(b, group)
    first = None
    for _ in range(5):
        got = run(mt, x, k_out, slots=slots)
        assert torch.equal(got["parents"].cpu().long(), parents.expand(b, k_out))
        assert torch.equal(got["tokens"].cpu().long(), tokens.expand(b, k_out))
        assert torch.equal(got["scores"], got["scores"][:1].expand(b, k_out))
        first = first or got
        assert all(torch.equal(first[n], got[n]) for n in got)


@pytest.mark.parametrize("dtype", DTYPES)
def test_floods_beside_ordinary_rows_and_finished_beams(mt, dtype):
    """Against the selection in 64 bits: sequences of one value, of few values and of ordinary ones in one call; some beams at their end."""
    g = torch.Generator().manual_seed(6)
    b, k, v = 24, 8, 3001
    x = torch.randn(b, k, v, generator=g).to(dtype)
    x[::3] = 0.5
    x[1::3] = torch.randint(0, 2, (b // 3, k, v), generator=g).to(dtype)
    prior = -torch.rand(b, k, generator=g)
    prior[::3] = -1.0
    ended = (torch.rand(b, k, generator=g) < 0.2).to(torch.uint8)
    slots = torch.randperm(b * k, generator=g).to(torch.int32).view(b, k)
    check(mt, x, k, prior, ended, 5, slots)


@pytest.mark.parametrize("at", [0, 5, (1 << 31) - 9])
def test_the_largest_vocabulary(mt, at):
    """2^31 - 1 logits, all but three of them equal: a few tokens stand out, at the row's ends or near its last vectors, and the flood's lowest follow.
    Score: 5 less the logarithm of 2^31 - 4 + 3 exp(5)."""
    v = (1 << 31) - 1
    x = torch.zeros(v, dtype=torch.bfloat16, device="cuda")
    top = sorted({at, 1 << 30, v - 1})
    x[torch.tensor(top, device="cuda")] = 5.0
    got = run(mt, x.view(1, 1, v), 5)
    others = [t for t in range(6) if t not in top]
    assert got["tokens"][0].tolist() == (top + others)[:5] and got["parents"][0].tolist() == [0] * 5
    log_sum = math.log(v - 3 + 3 * math.exp(5.0))
    want = torch.tensor([5.0 - log_sum] * 3 + [-log_sum] * 2)
    assert (got["scores"][0].cpu() - want).abs().max() <= SLACK + 2.0 ** -24 * 32

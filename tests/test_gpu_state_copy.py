"""mt_state_copy: rows of pools bit for bit, every other row left as it was."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def mt():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import prefix_scan_row_gb300 as m
    return m


def pool(*shape, dtype=torch.uint8, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = torch.empty(shape, dtype=dtype).element_size()
    last = torch.randint(0, 256, (*shape[:-1], shape[-1] * n), generator=g, dtype=torch.uint8)
    return last.view(dtype).cuda()


def bits(t):
    return t.contiguous().view(torch.uint8).cpu()


def check(mt, src, dst, pools, axis):
    want = []
    for p in pools:
        w = p.clone()
        for s, d in zip(src, dst):
            if 0 <= s < p.shape[axis] and 0 <= d < p.shape[axis]:
                w.select(axis, d).copy_(p.select(axis, s))
        want.append(bits(w))
    dev = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mt.mt_state_copy(dev(src), dev(dst), pools, axis=axis)
    for p, w in zip(pools, want):
        assert torch.equal(bits(p), w)


SRC, DST = [3, 3, -1, 0, 9, 5, 2, 6, 3, 1 << 30], [1, 4, 2, -1, 7, 5, 12, 1 << 30, 10, 8]  # some outside, one onto itself


@pytest.mark.parametrize("row", [1, 2, 3, 4, 7, 8, 16, 24, 4095, 4096, 16384, 16385, 16400, 50000])
def test_rows_of_any_size(mt, row):
    check(mt, SRC, DST, [pool(9, row)], 0)
    check(mt, SRC, DST, [pool(3, 9, row)], 1)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16, torch.int64])
@pytest.mark.parametrize("shape", [(9, 3, 40), (9, 33, 16), (11, 1, 5), (9, 64, 128)])
def test_pools_of_a_model(mt, dtype, shape):
    check(mt, SRC, DST, [pool(*shape, dtype=dtype), pool(9, 77, seed=1), pool(12, 256, dtype=torch.float32, seed=2)], 0)
    check(mt, SRC, DST, [pool(2, *shape, dtype=dtype), pool(5, 9, 77, seed=1)], 1)


@pytest.mark.parametrize("offset", [0, 1, 2, 4, 8])
def test_rows_of_wider_pools(mt, offset):
    wide = pool(9, 8192)
    keep = bits(wide)
    view = wide[:, offset:offset + 5000]
    check(mt, [3, 0], [1, 8], [view], 0)
    new = bits(wide)
    assert torch.equal(new[:, :offset], keep[:, :offset]) and torch.equal(new[:, offset + 5000:], keep[:, offset + 5000:])
    layers = pool(9, 3, 2048).transpose(0, 1)  # the layers of a slot beside each other
    check(mt, [3, 0], [1, 8], [layers], 1)


def test_many_pools(mt):
    check(mt, [0, 1], [3, 2], [pool(4, 100 + n, seed=n) for n in range(16)], 0)


def test_many_pairs(mt):
    n = 140001
    check_src = torch.randperm(2 * n, generator=torch.Generator().manual_seed(1)).to(torch.int32)
    src, dst = check_src[:n], check_src[n:]
    p = pool(2 * n, 3)
    want = p.cpu()
    want[dst.long()] = want[src.long()]
    mt.mt_state_copy(src.cuda(), dst.cuda(), p)
    assert torch.equal(p.cpu(), want)


def test_nothing_to_do(mt):
    none = torch.empty(0, dtype=torch.int32, device="cuda")
    p = pool(4, 8)
    keep = bits(p)
    mt.mt_state_copy(none, none, p)
    one = torch.zeros(1, dtype=torch.int32, device="cuda")
    mt.mt_state_copy(one, one + 1, [p[:0], p[:, :0]])
    assert torch.equal(bits(p), keep)


def test_offsets_past_32_bits(mt):
    """A pool of more than 4 GB: the last row onto the first and back into the middle."""
    row = 1 << 28
    p = torch.zeros(18, row, dtype=torch.uint8, device="cuda")
    p[17, -1], p[17, 5], p[16, 9] = 7, 8, 9
    dev = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    mt.mt_state_copy(dev(17, 16), dev(0, 9), p)
    assert int(p[0, -1]) == 7 and int(p[0, 5]) == 8 and int(p[9, 9]) == 9 and int(p[9, 5]) == 0

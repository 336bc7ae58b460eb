"""The gated scan where CTAs of a cluster share a sequence's tokens and tell one another their elements at every tile."""
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

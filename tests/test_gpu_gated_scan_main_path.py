"""The gated scan in the kernels that batches of real sizes get, over several tiles of a CTA that has all of a sequence's tokens: the carry from tile to
tile, both sides of the exchange between warps, every stage of the copies, the checkpoints of later tiles. 153 pairs of a sequence and 64 channels or
more have a CTA each; up to 456 of them take 16-bit prompts by four warps of 16 tokens, more by four of 8; f32 prompts by eight of 8,
gradients by four of 8. Bounds: gated_ref.GatedCase."""
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
@pytest.mark.parametrize("b,length,d", [(3, 200, 3840), (3, 203, 3837), (8, 151, 4032)])
@pytest.mark.parametrize("rate,i,z", [(True, True, True), (True, True, False), (False, False, True)])
def test_several_tiles_of_a_cta(mt, dtype, b, length, d, rate, i, z):
    assert 153 <= b * -(-d // 64) and length > 2 * 64
    lens = torch.tensor([length - 37 * (n % 3) for n in range(b)], dtype=torch.int32)
    p = Inputs(dtype, b, length, d, rate, i, z, h0=z, lens=lens)
    check_forward(mt, p)
    check_gradient(mt, p, dfinal=i)

"""Pools with no elements, of any shape, have nothing that mt_state_copy could refuse. No kernel is launched."""
import pytest
import torch

import prefix_scan_row_gb300 as mt


@pytest.mark.parametrize("shape,axis", [((4, 3, 0), 0), ((0, 3, 5), 0), ((2, 4, 3, 0), 1), ((0, 4, 3), 1), ((2, 0, 3), 1), ((3, 0, 7), 0)])
def test_empty_pools(shape, axis):
    none = torch.empty(0, dtype=torch.int32)
    mt.mt_state_copy(none, none, torch.empty(shape), axis=axis, stream=0)
    mt.mt_state_copy(none, none, [torch.empty(shape), torch.empty(4, 4, 2)], axis=axis, stream=0)
    with pytest.raises(ValueError):  # the others are looked at as before
        mt.mt_state_copy(none, none, [torch.empty(shape), torch.empty(4, 4, 3, 2).transpose(2, 3)], axis=axis, stream=0)

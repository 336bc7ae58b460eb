"""Fields of the argument blocks that a call says it ignores: whatever they hold, the call gets past its checks of arguments. With fake
pointers, which the check of the device's memory then refuses, or, without a GPU, the query of the device before it."""
import pytest

import prefix_scan_row_gb300 as mt
from test_seq_abi import ALIGN, P, block
from test_serving_abi import GATED

PASSED = (mt.MT_ERR_CUDA, mt.MT_ERR_MEMORY)
ODD = 0x70001  # aligned to nothing
GATED_IGNORED = {
    "mt_gated_scan": ("scratch", "dout", "dx", "dr", "di", "dz", "drate", "dfinal", "dinit"),
    "mt_gated_scan_step": ("lens", "checkpoints", "scratch", "dout", "dx", "dr", "di", "dz", "drate", "dfinal", "dinit"),
    "mt_gated_scan_grad": ("state", "out"),
}


def assert_ignored(fn, name, good, ignored):
    call = getattr(mt.lib, fn)
    assert call(block(name, **good), None) in PASSED
    for field in ignored:
        assert call(block(name, **{**good, field: ODD}), None) in PASSED, field


@pytest.mark.parametrize("fn", GATED_IGNORED)
def test_gated_scan(fn):
    assert_ignored(fn, "mt_gated_args", GATED, GATED_IGNORED[fn])


def test_gated_gradient_without_some_of_its_results():
    """di without i, dz without z, scratch without drate."""
    call = mt.lib.mt_gated_scan_grad
    for off, field in (("i", "di"), ("z", "dz"), ("drate", "scratch")):
        assert call(block("mt_gated_args", **{**GATED, off: 0, field: ODD}), None) in PASSED


@pytest.mark.parametrize("fn", GATED_IGNORED)
def test_gated_fields_that_count_are_refused(fn):
    for field in ("x", "r", "i", "z", "rate", "state", "out", "lens", "checkpoints", "scratch", "dout", "dx", "dr", "di", "dz", "drate",
                  "dfinal", "dinit"):
        if field not in GATED_IGNORED[fn]:
            assert getattr(mt.lib, fn)(block("mt_gated_args", **{**GATED, field: ODD}), None) == ALIGN, field
    if fn != "mt_gated_scan_grad":
        assert getattr(mt.lib, fn)(block("mt_gated_args", **{**GATED, "checkpoints": 0, "slots": P[20] + 2}), None) == ALIGN

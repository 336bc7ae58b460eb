"""Fields of the argument blocks that a call says it ignores: whatever they hold, the call gets past its checks of arguments. With fake
pointers, which the check of the device's memory then refuses, or, without a GPU, the query of the device before it."""
import pytest

import prefix_scan_row_gb300 as mt
from test_seq_abi import ALIGN, CONV, P, SSM, block, fields
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


CONV_IGNORED = {
    "mt_causal_conv": ("dout", "dx", "dweight", "dbias", "dstate", "scratch"),
    "mt_causal_conv_step": ("lens", "dout", "dx", "dweight", "dbias", "dstate", "scratch"),
    "mt_causal_conv_grad": ("out",),
}
SSM_IGNORED = {
    "mt_selective_scan": ("dout", "du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dfinal", "dinit"),
    "mt_selective_scan_step": ("lens", "scratch", "dout", "du", "ddelta", "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dfinal", "dinit"),
    "mt_selective_scan_grad": ("state", "out"),
}


@pytest.mark.parametrize("fn", CONV_IGNORED)
def test_convolution(fn):
    good = {**CONV, "wdtype": 1}  # weights of 16 bits
    assert_ignored(fn, "mt_conv_args", good, CONV_IGNORED[fn])
    for field in ("x", "weight", "bias", "state", "out", "lens", "dout", "dx", "dweight", "dbias", "dstate", "scratch"):
        if field not in CONV_IGNORED[fn]:
            assert getattr(mt.lib, fn)(block("mt_conv_args", **{**good, field: ODD}), None) == ALIGN, field


@pytest.mark.parametrize("fn", SSM_IGNORED)
def test_selective_scan(fn):
    assert_ignored(fn, "mt_ssm_args", SSM, SSM_IGNORED[fn])
    for field in ("u", "delta", "z", "B", "C", "A", "D", "delta_bias", "state", "out", "lens", "checkpoints", "scratch", "dout", "du", "ddelta",
                  "dz", "dB", "dC", "dA", "dD", "ddelta_bias", "dfinal", "dinit"):
        if field not in SSM_IGNORED[fn] and not (fn == "mt_selective_scan_step" and field == "checkpoints"):
            assert getattr(mt.lib, fn)(block("mt_ssm_args", **{**SSM, field: ODD}), None) == ALIGN, field


@pytest.mark.parametrize("fn,name,good,counts", [("mt_gated_scan_grad", "mt_gated_args", GATED, "drate"), ("mt_causal_conv_grad", "mt_conv_args", CONV, "dweight"),
                                                 ("mt_selective_scan_grad", "mt_ssm_args", SSM, "dA")])
def test_gradients_of_no_sequences(fn, name, good, counts):
    """They write the parameters' zeros and look at nothing else."""
    call = getattr(mt.lib, fn)
    odd = {field: ODD + 0x100 * n for n, field in enumerate(("dout", "dx", "du", "lens", "scratch", "dinit", "dfinal", "checkpoints"))
           if field in fields(name)}
    assert call(block(name, **{**good, "batch": 0, **odd}), None) in PASSED
    assert call(block(name, **{**good, "batch": 0, counts: ODD}), None) == ALIGN

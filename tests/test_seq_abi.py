"""Refusals of the sequence-model calls, on the host and before any CUDA call:
the C ABI with fake pointers that are never dereferenced, and the Python binding
with tensors that it must not pass on. No kernel is launched."""
import ctypes
import re
import struct

import pytest
import torch

import prefix_scan_row_gb300 as mt
from test_abi import HEADER

F32, BF16, F16, I32, I64 = 0, 1, 2, 3, 4
OK, ARG, DTYPE, ALIAS, ALIGN = 0, -1, -2, -3, -6
P = [0x10000 * (i + 1) for i in range(40)]  # fake, 16-byte aligned


def fields(name):
    text = re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)
    body = re.search(r"typedef struct \{([^}]*)\} " + name, text)[1]
    return [re.sub(r".*[\s*]", "", v.strip()) for s in body.split(";") if s.strip() for v in s.split(",")]


def block(name, **over):
    order = fields(name)
    assert set(over) <= set(order), set(over) - set(order)
    return struct.pack(f"={len(order)}q", *(over.get(k, 0) for k in order))


CONV = dict(dtype=BF16, wdtype=F32, batch=2, len=5, dim=8, width=4, silu=1, nslots=2, x=P[0], x_batch=40, x_token=8,
            weight=P[1], bias=P[2], state=P[3], out=P[4], out_batch=40, out_token=8, dout=P[5], dout_batch=40, dout_token=8,
            dx=P[6], dx_batch=40, dx_token=8, dweight=P[7], dbias=P[8], scratch=P[9])
SSM = dict(dtype=BF16, batch=2, len=5, dim=8, nstate=4, groups=2, softplus=1, nslots=2, u=P[0], delta=P[1], z=P[2], B=P[3],
           C=P[4], A=P[5], D=P[6], delta_bias=P[7], state=P[8], out=P[9], checkpoints=P[10], scratch=P[11], dout=P[12], du=P[13],
           ddelta=P[14], dz=P[15], dB=P[16], dC=P[17], dA=P[18], dD=P[19], ddelta_bias=P[20])


def test_packed_blocks_have_the_headers_fields():
    assert mt._CONV_ARGS.size == 8 * len(fields("mt_conv_args"))
    assert mt._SSM_ARGS.size == 8 * len(fields("mt_ssm_args"))


CONV_BAD = [(dict(batch=-1), ARG), (dict(dim=-1), ARG), (dict(width=0), ARG), (dict(width=5), ARG), (dict(dtype=I32), DTYPE),
            (dict(wdtype=F16), DTYPE), (dict(x=0), ARG), (dict(weight=0), ARG), (dict(nslots=1), ARG), (dict(x=P[0] + 1), ALIGN),
            (dict(weight=P[1] + 2), ALIGN), (dict(batch=1 << 40, dim=1 << 40), ARG), (dict(carry_in=1, state=0), ARG)]


@pytest.mark.parametrize("over,code", CONV_BAD)
@pytest.mark.parametrize("fn", ["mt_causal_conv", "mt_causal_conv_step", "mt_causal_conv_grad"])
def test_conv_refusals(fn, over, code):
    assert getattr(mt.lib, fn)(block("mt_conv_args", **{**CONV, **over}), None) == code


def test_conv_refusals_of_each_call():
    b = lambda **over: block("mt_conv_args", **{**CONV, **over})  # noqa: E731
    assert mt.lib.mt_causal_conv(None, None) == ARG
    assert mt.lib.mt_causal_conv(b(len=-1), None) == ARG
    assert mt.lib.mt_causal_conv(b(out=0), None) == ARG
    assert mt.lib.mt_causal_conv(b(out=P[0]), None) == ALIAS
    assert mt.lib.mt_causal_conv(b(state=P[0]), None) == ALIAS
    assert mt.lib.mt_causal_conv(b(slots=P[20], state=0), None) == ARG
    assert mt.lib.mt_causal_conv(b(batch=0), None) == OK
    assert mt.lib.mt_causal_conv(b(dim=0), None) == OK
    assert mt.lib.mt_causal_conv_step(b(state=0), None) == ARG
    assert mt.lib.mt_causal_conv_grad(b(scratch=0), None) == ARG
    assert mt.lib.mt_causal_conv_grad(b(scratch=P[9] + 8), None) == ALIGN
    assert mt.lib.mt_causal_conv_grad(b(dweight=0), None) == ARG
    assert mt.lib.mt_causal_conv_grad(b(dx=P[5]), None) == ALIAS
    assert mt.lib.mt_causal_conv_grad(b(slots=P[20]), None) == ARG


SSM_BAD = [(dict(batch=-1), ARG), (dict(nstate=0), ARG), (dict(nstate=129), ARG), (dict(groups=0), ARG), (dict(groups=3), ARG),
           (dict(dtype=I32), DTYPE), (dict(u=0), ARG), (dict(A=0), ARG), (dict(B=P[3] + 1), ALIGN), (dict(A=P[5] + 2), ALIGN),
           (dict(batch=1 << 40, dim=1 << 40), ARG)]


@pytest.mark.parametrize("over,code", SSM_BAD)
@pytest.mark.parametrize("fn", ["mt_selective_scan", "mt_selective_scan_step", "mt_selective_scan_grad"])
def test_scan_refusals(fn, over, code):
    assert getattr(mt.lib, fn)(block("mt_ssm_args", **{**SSM, **over}), None) == code


def test_scan_refusals_of_each_call():
    b = lambda **over: block("mt_ssm_args", **{**SSM, **over})  # noqa: E731
    assert mt.lib.mt_selective_scan(None, None) == ARG
    assert mt.lib.mt_selective_scan(b(len=-1), None) == ARG
    assert mt.lib.mt_selective_scan(b(nslots=1), None) == ARG
    assert mt.lib.mt_selective_scan(b(carry_in=1, state=0), None) == ARG
    assert mt.lib.mt_selective_scan(b(slots=P[30]), None) == ARG  # with checkpoints
    assert mt.lib.mt_selective_scan(b(out=P[0]), None) == ALIAS
    assert mt.lib.mt_selective_scan(b(len=4096, scratch=0), None) == ARG  # cut into segments: scratch needed
    assert mt.lib.mt_selective_scan(b(scratch=P[11] + 8), None) == ALIGN
    assert mt.lib.mt_selective_scan(b(batch=0), None) == OK
    assert mt.lib.mt_selective_scan_step(b(state=0), None) == ARG
    assert mt.lib.mt_selective_scan_step(b(out=P[8]), None) == ALIAS
    assert mt.lib.mt_selective_scan_grad(b(dz=0), None) == ARG
    assert mt.lib.mt_selective_scan_grad(b(checkpoints=0), None) == ARG
    assert mt.lib.mt_selective_scan_grad(b(dA=0), None) == ARG
    assert mt.lib.mt_selective_scan_grad(b(du=P[0]), None) == ALIAS
    assert mt.lib.mt_selective_scan_grad(b(slots=P[30]), None) == ARG


def test_embed_refusals():
    f, g = mt.lib.mt_embed, mt.lib.mt_embed_grad
    assert f(P[0], -1, I32, P[1], 5, 8, BF16, 1.0, P[2], None) == ARG
    assert f(P[0], 3, F32, P[1], 5, 8, BF16, 1.0, P[2], None) == DTYPE
    assert f(P[0], 3, I32, P[1], 5, 8, I32, 1.0, P[2], None) == DTYPE
    assert f(0, 3, I32, P[1], 5, 8, BF16, 1.0, P[2], None) == ARG
    assert f(P[0], 3, I32, P[1], 5, 8, BF16, 1.0, P[1], None) == ALIAS
    assert f(P[0] + 4, 3, I64, P[1], 5, 8, BF16, 1.0, P[2], None) == ALIGN
    assert f(P[0], 3, I32, P[1] + 2, 5, 8, F32, 1.0, P[2], None) == ALIGN
    assert f(P[0], 1 << 40, I32, P[1], 5, 1 << 40, BF16, 1.0, P[2], None) == ARG
    assert f(P[0], 0, I32, P[1], 5, 8, BF16, 1.0, P[2], None) == OK
    assert g(P[0], 3, I32, P[1], BF16, 5, 8, 1.0, P[2], F16, 0, P[3], None) == DTYPE
    assert g(P[0], 3, I32, P[1], BF16, 5, 8, 1.0, P[2], F32, 0, 0, None) == ARG
    assert g(P[0], 3, I32, P[1], BF16, 5, 8, 1.0, P[1], F32, 0, P[3], None) == ALIAS
    assert g(P[0], 3, I32, P[1], BF16, 5, 8, 1.0, P[2], F32, 0, P[3] + 8, None) == ALIGN
    assert g(P[0], 3, I32, P[1], BF16, 5, 8, 1.0, P[2] + 2, F32, 0, P[3], None) == ALIGN
    assert g(P[0], 0, I32, P[1], BF16, 0, 8, 1.0, P[2], F32, 0, P[3], None) == OK
    assert mt.lib.mt_embed_grad_scratch_slots(1 << 31, 5, 8) == -1
    assert mt.lib.mt_embed_grad_scratch_slots(5, 1 << 31, 8) == -1


def test_scratch_sizes():
    assert mt.mt_selective_scan_scratch_slots(16, 2048, 4096, 16) == 0  # enough channels: the tokens are not cut
    assert mt.mt_selective_scan_scratch_slots(1, 2048, 64, 16) > 0
    assert mt.mt_selective_scan_checkpoint_slots(2, 33, 10, 5) == (2 * 5 * 10 * 5 + 1) // 2  # a state every 8 tokens
    for bad in ((-1, 1, 1, 1), (1, 1, 1, 129), (1, 1, 1, 0)):
        with pytest.raises(ValueError):
            mt.mt_selective_scan_checkpoint_slots(*bad)
    with pytest.raises(ValueError):
        mt.mt_selective_scan_scratch_slots(1, 1, 3, 4, groups=2)
    with pytest.raises(ValueError):
        mt.mt_causal_conv_grad_scratch_slots(1, 1, 1, 9)


def test_binding_refuses_what_the_calls_would_misread():
    z = lambda *s, dtype=torch.float32: torch.zeros(*s, dtype=dtype)  # noqa: E731
    i32 = torch.int32
    with pytest.raises(ValueError, match="out must have"):
        mt.mt_embed(z(3, dtype=i32), z(5, 8), z(3, 7))
    with pytest.raises(ValueError, match="contiguous"):
        mt.mt_embed(z(3, dtype=i32), z(5, 16)[:, ::2], z(3, 8))
    with pytest.raises(ValueError, match="scratch"):
        mt.mt_embed_grad(z(3, dtype=i32), z(3, 8), z(5, 8), z(1, dtype=torch.int64))
    x, w = z(2, 5, 8), z(8, 4)
    with pytest.raises(ValueError, match="innermost"):
        mt.mt_causal_conv(z(2, 5, 16)[..., ::2], w, z(2, 5, 8))
    with pytest.raises(ValueError, match="out must be"):
        mt.mt_causal_conv(x, w, z(2, 5, 8, dtype=torch.float16))
    with pytest.raises(ValueError, match="state must be"):
        mt.mt_causal_conv(x, w, z(2, 5, 8), state=z(2, 4, 8))
    with pytest.raises(ValueError, match="row for every"):
        mt.mt_causal_conv(x, w, z(2, 5, 8), state=z(1, 3, 8))
    with pytest.raises(ValueError, match="lens must be"):
        mt.mt_causal_conv(x, w, z(2, 5, 8), lens=z(2, dtype=torch.int64))
    A, B = z(8, 4), z(2, 5, 1, 4)
    with pytest.raises(ValueError, match="delta must be"):
        mt.mt_selective_scan(x, z(2, 5, 7), A, B, B, z(2, 5, 8))
    with pytest.raises(ValueError, match="A must be"):
        mt.mt_selective_scan(x, x, A.double(), B, B, z(2, 5, 8))
    with pytest.raises(ValueError, match="two innermost"):
        mt.mt_selective_scan(x, x, A, z(2, 5, 2, 8)[..., :4], z(2, 5, 2, 4), z(2, 5, 8))
    with pytest.raises(ValueError, match="scratch is needed"):
        long = z(1, 4096, 8)
        mt.mt_selective_scan(long, long, A, z(1, 4096, 1, 4), z(1, 4096, 1, 4), z(1, 4096, 8))
    with pytest.raises(ValueError, match="dz is needed"):
        mt.mt_selective_scan_grad(x, x, A, B, B, x, z(64), z(2, 5, 8), z(2, 5, 8), A, B, B, z(999), z=x)

"""Refusals of the gated scan, the beam selection and the state copies, on the host and before any CUDA
call: the C ABI with fake pointers that are never dereferenced, and the Python binding. No kernel is launched."""
import ctypes

import pytest
import torch

import prefix_scan_row_gb300 as mt
from test_seq_abi import ALIAS, ALIGN, ARG, BF16, DTYPE, I32, OK, P, block, fields

GATED = dict(dtype=BF16, batch=2, len=5, dim=8, nslots=2, x=P[0], r=P[1], i=P[2], z=P[3], rate=P[4], state=P[5], out=P[6],
             checkpoints=P[7], scratch=P[8], dout=P[9], dx=P[10], dr=P[11], di=P[12], dz=P[13], drate=P[14], dinit=P[15])
BEAM = dict(dtype=BF16, batch=2, beams=4, beams_out=4, vocab=100, eos=3, logits=P[0], logits_batch=400, logits_beam=100, prior=P[1],
            finished=P[2], tokens=P[3], parents=P[4], scores=P[5], finished_out=P[6], slots=P[7], src=P[8], dst=P[9], scratch=P[10])


def test_packed_blocks_have_the_headers_fields():
    assert mt._GATED_ARGS.size == 8 * len(fields("mt_gated_args"))
    assert mt._BEAM_ARGS.size == 8 * len(fields("mt_beam_args"))
    assert mt._POOL.size == 48


GATED_BAD = [(dict(batch=-1), ARG), (dict(dim=-1), ARG), (dict(dtype=I32), DTYPE), (dict(x=0), ARG), (dict(r=0), ARG),
             (dict(x=P[0] + 1), ALIGN), (dict(rate=P[4] + 2), ALIGN), (dict(batch=1 << 40, dim=1 << 40), ARG), (dict(nslots=-1), ARG)]


@pytest.mark.parametrize("over,code", GATED_BAD)
@pytest.mark.parametrize("fn", ["mt_gated_scan", "mt_gated_scan_step", "mt_gated_scan_grad"])
def test_gated_refusals(fn, over, code):
    assert getattr(mt.lib, fn)(block("mt_gated_args", **{**GATED, **over}), None) == code


def test_gated_refusals_of_each_call():
    b = lambda **over: block("mt_gated_args", **{**GATED, **over})  # noqa: E731
    scan, step, grad = mt.lib.mt_gated_scan, mt.lib.mt_gated_scan_step, mt.lib.mt_gated_scan_grad
    for fn in (scan, step, grad):
        assert fn(None, None) == ARG
        assert fn(b(dim=0), None) == OK
    assert scan(b(batch=0), None) == OK and step(b(batch=0), None) == OK
    assert scan(b(len=-1), None) == ARG and scan(b(len=1 << 31), None) == ARG and grad(b(len=1 << 31), None) == ARG
    assert scan(b(out=0), None) == ARG
    assert scan(b(nslots=1), None) == ARG
    assert scan(b(out=P[0]), None) == ALIAS
    assert scan(b(state=P[1]), None) == ALIAS
    assert scan(b(out=P[5]), None) == ALIAS
    assert scan(b(checkpoints=P[6]), None) == ALIAS
    assert scan(b(slots=P[20]), None) == ARG  # checkpoints go by sequence
    assert scan(b(slots=P[20], state=0, checkpoints=0), None) == ARG
    assert scan(b(carry_in=1, state=0), None) == ARG
    assert step(b(state=0), None) == ARG and step(b(out=0), None) == ARG
    assert step(b(out=P[5]), None) == ALIAS and step(b(state=P[4]), None) == ALIAS
    assert step(b(nslots=1), None) == ARG
    for name in ("dout", "dx", "dr", "di", "dz", "checkpoints", "scratch", "rate"):
        assert grad(b(**{name: 0}), None) == ARG, name
    assert grad(b(slots=P[20]), None) == ARG
    assert grad(b(dx=P[9]), None) == ALIAS and grad(b(dx=P[11]), None) == ALIAS and grad(b(drate=P[4]), None) == ALIAS
    assert grad(b(scratch=P[8] + 8), None) == ALIGN
    assert grad(b(batch=1 << 31, len=1 << 31, dim=1 << 20), None) == ARG


def test_gated_sizes():
    assert mt.lib.mt_gated_scan_scratch_slots(-1, 1, 1) == -1 and mt.lib.mt_gated_scan_checkpoint_slots(1, -1, 1) == -1
    assert mt.lib.mt_gated_scan_checkpoint_slots(1 << 31, 1 << 31, 4) == -1
    assert mt.mt_gated_scan_checkpoint_slots(2, 65, 3) >= 3 and mt.mt_gated_scan_checkpoint_slots(2, 0, 3) == 0
    assert mt.lib.mt_gated_scan_scratch_slots(1, 1 << 31, 1) == -1 and mt.lib.mt_gated_scan_checkpoint_slots(1, 1 << 31, 1) == -1
    with pytest.raises(ValueError):
        mt.mt_gated_scan_scratch_slots(1, 1, -1)


BEAM_BAD = [(dict(batch=-1), ARG), (dict(beams=0), ARG), (dict(beams=33), ARG), (dict(beams_out=0), ARG), (dict(beams_out=33), ARG),
            (dict(vocab=0), ARG), (dict(vocab=1 << 31), ARG), (dict(beams=1, beams_out=5, vocab=4, eos=-1, finished=0), ARG), (dict(eos=100), ARG),
            (dict(eos=-1), ARG), (dict(dtype=I32), DTYPE), (dict(logits=0), ARG), (dict(tokens=0), ARG), (dict(parents=0), ARG),
            (dict(scores=0), ARG), (dict(scratch=0), ARG), (dict(src=0), ARG), (dict(dst=0), ARG), (dict(scores=P[0]), ALIAS),
            (dict(tokens=P[4]), ALIAS), (dict(src=P[9]), ALIAS), (dict(slots=P[9]), ALIAS), (dict(scratch=P[1]), ALIAS),
            (dict(tokens=P[1]), ALIAS), (dict(finished_out=P[1]), ALIAS), (dict(beams_out=3, scores=P[1]), ALIAS),
            (dict(beams_out=3, finished_out=P[2]), ALIAS), (dict(logits=P[0] + 1), ALIGN), (dict(prior=P[1] + 2), ALIGN),
            (dict(scratch=P[10] + 8), ALIGN), (dict(batch=0), OK)]


@pytest.mark.parametrize("over,code", BEAM_BAD)
def test_beam_refusals(over, code):
    assert mt.lib.mt_beam_select(block("mt_beam_args", **{**BEAM, **over}), None) == code


def test_beam_sizes():
    assert mt.lib.mt_beam_select(None, None) == ARG
    for bad in ((-1, 1, 1, 1), (1, 0, 1, 1), (1, 33, 1, 1), (1, 1, 33, 1), (1, 1, 1, 0), (1, 1, 1, 1 << 31), (1 << 55, 32, 32, 1 << 20)):
        assert mt.lib.mt_beam_select_scratch_slots(*bad) == -1
        with pytest.raises(ValueError):
            mt.mt_beam_select_scratch_slots(*bad)


def pools(*over):
    one = dict(base=P[5], nslots=4, row_bytes=64, row_stride=64, planes=1, plane_stride=0)
    return b"".join(mt._POOL.pack(*{**one, **o}.values()) for o in over)


@pytest.mark.parametrize("over", [dict(nslots=-1), dict(row_bytes=-1), dict(row_stride=63), dict(planes=-1), dict(base=0), dict(nslots=1 << 31),
                                  dict(planes=2, plane_stride=63), dict(nslots=1 << 30, row_stride=1 << 40)])
def test_copy_refusals(over):
    assert mt.lib.mt_state_copy(P[0], P[1], 3, pools({}, over), 2, None) == ARG


def test_copy_refusals_of_the_call():
    f = mt.lib.mt_state_copy
    assert f(P[0], P[1], -1, pools({}), 1, None) == ARG
    assert f(P[0], P[1], 1 << 31, pools({}), 1, None) == ARG
    assert f(P[0], P[1], 3, pools({}), 0, None) == ARG
    assert f(P[0], P[1], 3, pools(*[{}] * 17), 17, None) == ARG
    assert f(P[0], P[1], 3, None, 1, None) == ARG
    assert f(0, P[1], 3, pools({}), 1, None) == ARG
    assert f(P[0], 0, 3, pools({}), 1, None) == ARG
    assert f(P[0] + 2, P[1], 3, pools({}), 1, None) == ALIGN
    assert f(P[5], P[1], 3, pools({}), 1, None) == ALIAS
    assert f(0, 0, 0, pools({}), 1, None) == OK


def meta(*shape, dtype=torch.float32):
    return torch.empty(*shape, dtype=dtype)


def test_binding_refusals():
    x = meta(2, 5, 8)
    i32 = lambda *s: meta(*s, dtype=torch.int32)  # noqa: E731
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, meta(2, 5, 9), x)
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x.half(), x)
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, rate=meta(7))
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, rate=meta(8).double())
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, state=meta(1, 8))
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, state=meta(2, 9))
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, lens=i32(3))
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x.transpose(1, 2), x.transpose(1, 2), x.transpose(1, 2))
    with pytest.raises(ValueError):
        mt.mt_gated_scan(x, x, x, checkpoints=meta(1, dtype=torch.int64))
    with pytest.raises(ValueError):
        mt.mt_gated_scan_step(x[:, 0], x[:, 0], None, x[:, 1, :7])
    ck = meta(64, dtype=torch.int64)
    with pytest.raises(ValueError):
        mt.mt_gated_scan_grad(x, x, x, ck, x, x, i=x)
    with pytest.raises(ValueError):
        mt.mt_gated_scan_grad(x, x, x, ck, x, x, dz=x)
    with pytest.raises(ValueError):
        mt.mt_gated_scan_grad(x, x, x, ck, x, x, drate=meta(8))
    with pytest.raises(ValueError):
        mt.mt_gated_scan_grad(x, x, x, ck, x, x, rate=meta(8), drate=meta(8))  # no scratch
    logits, t = meta(2, 4, 100), i32(2, 4)
    scratch = meta(mt.mt_beam_select_scratch_slots(2, 4, 4, 100), dtype=torch.int64)
    good = dict(prior=meta(2, 4))
    for bad in (dict(prior=meta(2, 5)), dict(finished=meta(2, 4)), dict(slots=t), dict(slots=i32(2, 3), src=t, dst=t),
                dict(finished_out=t), dict(prior=meta(2, 4).double())):
        with pytest.raises(ValueError):
            mt.mt_beam_select(logits, t, t, meta(2, 4), scratch, **{**good, **bad})
    with pytest.raises(ValueError):
        mt.mt_beam_select(logits, t.long(), t, meta(2, 4), scratch)
    with pytest.raises(ValueError):
        mt.mt_beam_select(logits, t, t, meta(2, 4), scratch[:-1])
    with pytest.raises(ValueError):
        mt.mt_beam_select(logits.transpose(1, 2), i32(2, 4), i32(2, 4), meta(2, 4), scratch)
    with pytest.raises(ValueError):
        mt.mt_beam_select(logits, i32(3, 4), t, meta(2, 4), scratch)
    with pytest.raises(ValueError):
        mt.mt_state_copy(t, i32(2, 5), meta(4, 8))
    with pytest.raises(ValueError):
        mt.mt_state_copy(t.long(), t.long(), meta(4, 8))
    with pytest.raises(ValueError):
        mt.mt_state_copy(t, t, meta(4, 8), axis=2)
    with pytest.raises(ValueError):
        mt.mt_state_copy(t, t, meta(4), axis=1)
    with pytest.raises(ValueError):
        mt.mt_state_copy(t, t, meta(4, 8, 3).transpose(1, 2))
    with pytest.raises(mt.ScanError):
        mt.mt_state_copy(t, t, meta(1, 8).expand(4, 8), stream=0)

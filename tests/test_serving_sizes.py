"""Scratch of the calls of a server, which is sized once for the largest call: no smaller call takes more. And what a call takes by its plan,
restated here, is within it. On the host."""
import itertools

import pytest

import prefix_scan_row_gb300 as mt

BATCHES = [0, 1, 2, 3, 4, 5, 7, 8, 16, 17, 18, 19, 20, 32, 33, 64, 200]


def assert_no_smaller_call_takes_more(size, axes):
    """Every axis by itself, at every combination of the others."""
    for n, axis in enumerate(axes):
        for rest in itertools.product(*(a for k, a in enumerate(axes) if k != n)):
            slots = [size(*rest[:n], v, *rest[n:]) for v in axis]
            assert slots == sorted(slots), (n, rest, list(zip(axis, slots)))


def beam_plan(rows, vocab, size):
    """Slots that a call takes: two for every span of a row, and half a one for every group of 128 16-byte vectors."""
    groups = 8
    while True:
        spans = -(-vocab * size // (groups * 128 * 16))
        if groups == 1 or rows * spans >= 152 * 32 * 2:
            return 2 * rows * spans + -(-rows * spans * groups // 2)
        groups //= 2


VOCABS = [1, 40, 500, 8192, 8193, 24576, 32768, 50000, 100003, 131072, 1 << 20, (1 << 31) - 1]


def test_beam_scratch_serves_smaller_calls():
    assert_no_smaller_call_takes_more(mt.mt_beam_select_scratch_slots, [BATCHES, [1, 2, 3, 4, 8, 16, 32], [1, 7, 32], VOCABS])


@pytest.mark.parametrize("vocab", VOCABS)
def test_beam_scratch_holds_what_a_call_takes(vocab):
    for batch, beams in itertools.product(BATCHES, [1, 3, 4, 16, 32]):
        slots = mt.mt_beam_select_scratch_slots(batch, beams, 4, vocab)
        need = max(beam_plan(batch * beams, vocab, size) for size in (2, 4))
        assert need <= slots <= max(need, 5 * 152 * 32 * 2 * 2), (batch, beams)  # and no more than a few MB beyond


LENGTHS = [0, 1, 16, 32, 33, 64, 65, 100, 257, 515, 1500, 2048, 16384]
DIMS = [1, 63, 64, 65, 128, 200, 1001, 2048, 2049, 4096, 9728, 9729, 20000]


def grad_plan(batch, length, dim):
    """Slots that a gradient takes: half a one for every channel, sequence and CTA of its cluster."""
    places = [0, 304, 304, 276, 276, 264, 264, 252, 264]
    units, tiles, n = batch * -(-dim // 64), -(-length // 32), 8
    while n > 1 and (units * n > places[n] or n > tiles):
        n -= 1
    rounds = -(-tiles // n)
    ctas = -(-tiles // rounds) if rounds else 1
    return -(-batch * ctas * dim // 2)


def test_gated_scratch_and_checkpoints_serve_smaller_calls():
    assert_no_smaller_call_takes_more(mt.mt_gated_scan_scratch_slots, [BATCHES, LENGTHS, DIMS])
    assert_no_smaller_call_takes_more(mt.mt_gated_scan_checkpoint_slots, [BATCHES, LENGTHS, DIMS])


@pytest.mark.parametrize("length", LENGTHS)
def test_gated_scratch_holds_what_a_call_takes(length):
    for batch, dim in itertools.product(BATCHES, DIMS):
        slots = mt.mt_gated_scan_scratch_slots(batch, length, dim)
        need = grad_plan(batch, length, dim)
        assert need <= slots <= max(need, 152 * 64), (batch, dim)

"""Host model of the staging of activation rows in csrc/w4_stream.cu."""
import random

import numpy as np
import pytest

from w4_stream_model import batches, expert_launches, leftovers, segments


def test_row_maxima_start_from_zero_in_every_staging():
    """Two buffers of row maxima take turns; whatever the segments' rows (up to 8: several warps a
    row, which meet in a buffer; more: a warp a row), each staging finds its buffer empty. Cleared
    only in the stagings that use one, a buffer keeps the maxima of two stagings before."""
    rng = random.Random(5)
    old = 0
    for _ in range(2000):
        chunks = rng.choice((1, 1, 2, 3))
        segs = [(i, i, rng.randint(1, 24)) for i in range(rng.randint(1, 8))]
        assert leftovers(segs, chunks, every_turn=True) == []
        old += bool(leftovers(segs, chunks, every_turn=False))
    assert old > 100


def skewed_ids(seed, T, E, k):
    """T x k distinct experts, some of them in far more demand than others."""
    rng = np.random.default_rng(seed)
    p = np.exp(-3.0 * rng.permutation(E) / E)
    return np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(T)]).astype(np.int32)


# (T, H, F, E, k, format, launch): layers in which a CTA stages few rows, many, then few again
ALTERNATING = [
    (64, 64, 14336, 128, 8, "nf4", "down"),
    (64, 4096, 128, 512, 16, "nf4", "gate_up"),
    (64, 5120, 64, 384, 16, "mxfp4", "gate_up"),
]


def alternating(T, H, F, E, k, fmt, launch, sms=148):
    """(ids, tokens whose maxima an uncleared buffer would hand on)"""
    tiles, _, chunks, xrows, split = expert_launches(T, H, F, fmt)[launch]
    for seed in range(60):
        ids = skewed_ids(seed, T, E, k)
        slots = batches(ids, E, 8)
        rows = [len(s) for s in slots]
        tokens = set()
        for segs in segments(rows, tiles, xrows, sms // chunks if split else sms):
            for (b0, b1, _), _ in leftovers(segs, 1 if split else chunks, every_turn=False):
                tokens |= {int(s) // k for b in range(b0, b1 + 1) for s in slots[b]}
        if tokens:
            return ids, sorted(tokens)
    raise AssertionError("no routing of this layer alternates")


@pytest.mark.parametrize("case", ALTERNATING)
def test_layers_that_alternate_between_few_rows_and_many(case):
    """The layers the GPU test runs reach the sequence the buffers have to survive."""
    ids, tokens = alternating(*case)
    assert tokens and ids.shape == (case[0], case[4])

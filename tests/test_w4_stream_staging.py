"""Host model of the staging of activation rows in csrc/w4_stream.cu."""
import random

import numpy as np
import pytest

from test_w4_stream_bookkeeping import FORMATS, RING, STAGE_K, WARPS, scale_layout, shares
from w4_stream_model import batches, expert_launches, gemv_launch, leftovers, segments


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


# What the GPU tests of chunks are about; the sizes follow from the room in shared memory, so they
# are asserted here. Layers: (T, H, F, E, k, format, scales, interleaved), chunks of H in turn in
# the gate_up launch, chunks of F in the down launch, whether those are shared out over CTAs.
LAYERS_IN_CHUNKS = [
    ((20, 6464, 128, 3, 2, "nf4", "f32", True), 2, 1, False),
    ((20, 6464, 128, 3, 2, "nf4", "bf16", False), 2, 1, False),
    ((9, 12352, 64, 3, 2, "nf4", "f32", False), 3, 1, False),
    ((9, 12352, 64, 3, 2, "nf4", "bf16", True), 3, 1, False),
    ((9, 14400, 64, 3, 2, "mxfp4", "e8m0", False), 3, 1, False),
    ((33, 6464, 14336, 2, 1, "nf4", "f32", False), 2, 3, True),
    ((9, 64, 65536, 2, 1, "nf4", "bf16", False), 1, 11, False),
    ((9, 128, 65536, 2, 1, "mxfp4", "e8m0", True), 1, 10, False),
]
# Vector products (M, N, K, format, group, scales, zeros), chunks, shared out
PRODUCTS_IN_CHUNKS = [
    ((32, 24, 65536, "nf4", 64, "bf16", False), 20, False),
    ((32, 24, 65536, "mxfp4", 32, "e8m0", False), 18, False),
    ((32, 24, 65536, "int4", 32, "bf16", True), 24, False),
    ((32, 24, 65536, "int4", 64, "f32", True), 18, False),
    ((32, 24, 65536, "int4", 128, "bf16", True), 16, False),
    ((8, 40, 65536, "nf4", 64, "f32", False), 10, False),
    ((7, 40, 65536, "int4", 32, "f32", True), 10, False),
    ((8, 32800, 9280, "mxfp4", 32, "e8m0", False), 2, False),
    ((8, 32800, 9344, "int4", 128, "f32", True), 2, False),
    ((16, 2500, 8192, "nf4", 64, "f32", False), 4, True),
]


def test_cases_in_chunks_are_in_chunks():
    for (T, H, F, _, _, fmt, _, _), up, down, shared in LAYERS_IN_CHUNKS:
        got = expert_launches(T, H, F, fmt)
        assert got["gate_up"][2] == up and (got["down"][2], got["down"][4]) == (down, shared), got
    for (M, N, K, fmt, group, _, _), chunks, shared in PRODUCTS_IN_CHUNKS:
        assert gemv_launch(M, N, K, fmt, group)[1:] == (chunks, shared), (M, N, K, fmt, group)


class Ring:
    """A warp's ring: what its copies and its multiplication do, in the kernel's order."""

    def __init__(self):
        self.slot = self.phase = self.flying = 0
        self.filled = [[] for _ in range(RING)]     # per slot: the stages copied there so far
        self.waited = [0] * RING

    def start(self, left, kb, tile, nblk, per):
        self.a = [left, kb, tile, 0, 0]             # units left, unit, tile, units of the piece, its unit
        self.nblk, self.per = nblk, per
        at = self.slot
        for _ in range(RING):
            self.flying += 1
            self.refill(at)
            at = (at + 1) % RING

    def refill(self, slot):
        left, kb, tile, run, at = self.a
        if run <= 0:
            if left == 0:
                self.flying -= 1
                return
            run = min(left, self.nblk - kb)
            at, kb, left, tile = kb, 0, left - run, tile + 1
        # (a copy into a slot whose last one was read)
        assert len(self.filled[slot]) == self.waited[slot]
        self.filled[slot].append((tile - 1, at))
        self.a = [left, kb, tile, run - self.per, at + self.per]

    def next(self):
        """Waits for the stage to multiply: (tile, first unit)."""
        s = self.slot
        assert self.waited[s] & 1 == self.phase     # the parity waited for is that of the stage's copy
        assert len(self.filled[s]) == self.waited[s] + 1
        stage = self.filled[s][-1]
        self.waited[s] += 1
        return stage

    def advance(self):
        self.slot += 1
        if self.slot == RING:
            self.slot, self.phase = 0, self.phase ^ 1


@pytest.mark.parametrize("per", [2, 4])
def test_every_wait_is_for_the_stage_it_multiplies(per):
    """Segment after segment, with shares of no, one, two and many stages, and a warp that stops in
    the middle: what is left to drain are the copies under way, no more and no fewer."""
    rng = random.Random(per)
    stages = [0] * 4
    for _ in range(400):
        ring = Ring()
        for _ in range(rng.randint(1, 6)):
            ntile, nblk = rng.choice((1, 1, 2, 3, 7)), rng.choice((1, 2, 3, 4, 5, 16, 45))
            units = ntile * nblk
            cuts, w = shares(units), rng.randrange(WARPS)
            left, kb, tile = cuts[w + 1] - cuts[w], cuts[w] % nblk, cuts[w] // nblk
            ring.start(left, kb, tile, nblk, per)
            done, gives_up = 0, rng.random() < 0.1
            while left:
                piece, at = min(left, nblk - kb), kb
                left, kb = left - piece, 0
                while piece > 0 and not (gives_up and rng.random() < 0.3):
                    n = min(piece, per)
                    assert ring.next() == (tile, at)
                    ring.refill(ring.slot)
                    ring.advance()
                    piece, at, done = piece - n, at + n, done + 1
                if piece > 0:
                    break
                tile += 1
            else:
                gives_up = False
            stages[min(done, 3)] += 1
            while ring.flying:          # (none, unless the warp gave up)
                assert gives_up
                ring.next()
                ring.flying -= 1
                ring.advance()
            assert all(len(f) == n for f, n in zip(ring.filled, ring.waited))
            if gives_up:
                break
    assert min(stages) > 20


@pytest.mark.parametrize("fmt,group,size", FORMATS)
def test_activation_reads_stay_inside_the_staged_row(fmt, group, size):
    """The last byte any lane reads of a row lies in the last staged piece of 8 activations."""
    unit_k = scale_layout(fmt, group)[0]
    for K in (64, 128, 192, 320, 2880, 6144, 16384):
        if K % group or K % unit_k:
            continue
        for chunk in {min(-(-K // STAGE_K) * STAGE_K, 4096), STAGE_K}:
            for c in range(-(-K // chunk)):
                codes = min(chunk, K - c * chunk)
                units, words = codes // unit_k, unit_k // 32
                last = max(q * 16 + u * unit_k * 2 + w * 64 + 16
                           for u in (0, units - 1) for w in range(words) for q in range(4))
                assert units * unit_k == codes and last == codes * 2 <= chunk * 2 + 64

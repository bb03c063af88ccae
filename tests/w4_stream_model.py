"""Host model of how csrc/w4_stream.cu cuts an expert layer or a vector product
into chunks, batches and segments (index arithmetic only)."""
import numpy as np

from test_w4_stream_bookkeeping import SMEM_MAX, WARPS, choose_split, chunk_of, offsets

MAX_ROWS, MAX_SPLIT = 128, 8


def expert_launches(T, H, F, fmt):
    """{launch: (tiles per batch, chunk, chunks, rows staged at once, chunks shared out)}"""
    area = SMEM_MAX - 1024 - offsets(fmt, 32 if fmt == "mxfp4" else 64, False)
    cap, out = min(T, 8), {}
    for name, K, tiles in (("gate_up", H, F // 8), ("down", F, H // 16)):
        chunk = chunk_of(K, cap, area)
        n = -(-K // chunk)
        out[name] = (tiles, chunk, n, min(MAX_ROWS, area // (chunk * 2 + 64)),
                     name == "down" and 1 < n <= MAX_SPLIT)
    return out


def gemv_launch(M, N, K, fmt, group):
    """(chunk, chunks, shared out)"""
    area = SMEM_MAX - 1024 - offsets(fmt, group, True)
    split = choose_split(M, N, K, area)
    if split:
        return (*split, True)
    chunk = chunk_of(K, M if M <= 16 else (M + 1) // 2, area)
    return chunk, -(-K // chunk), False


def batches(ids, E, cap):
    """The slots of every batch: by expert, in slot order, `cap` at a time."""
    flat = np.asarray(ids).ravel()
    out = []
    for e in range(E):
        slots = np.flatnonzero(flat == e)
        out += [slots[r:r + cap] for r in range(0, len(slots), cap)]
    return out


def segments(rows, tiles, xrows, ctas):
    """Per CTA the (first batch, last batch, rows) of its segments; rows: of every batch."""
    total = len(rows) * tiles
    for c in range(ctas):
        lo, hi = total * c // ctas, total * (c + 1) // ctas
        out, at = [], lo
        while at < hi:
            first = last = at // tiles
            n, end = rows[first], (first + 1) * tiles
            while end < hi and n + rows[last + 1] <= xrows:
                last += 1
                n += rows[last]
                end += tiles
            at = min(end, hi)
            out.append((first, last, n))
        yield out


def leftovers(segs, chunks, every_turn):
    """The pairs (segment whose maxima are still in a buffer, segment that starts from them): rows
    that several warps stage meet their maxima in buffer turn % 2, and a turn clears the other one,
    every time or only when it uses its own."""
    holds, turn, out = [None, None], 0, []
    for s in segs:
        for _ in range(chunks):
            shared = WARPS // s[2] > 1
            if shared or every_turn:
                holds[turn % 2 ^ 1] = None
            if shared:
                if holds[turn % 2] is not None:
                    out.append((holds[turn % 2], s))
                holds[turn % 2] = s
            turn += 1
    return out

"""Calls of attention over pages that reach every way the work is shared out:
(dtype, block_tokens, key heads, query heads per key head, lengths, queries,
positions of their own, expected share).  A share is ("rows", ranges, lane
groups of the join) or ("chunk", cuts).
"""

CASES = [
    # few rows: whole items; ranges whose results 1, 2 .. 16 lane groups join
    ("bf16", 64, 8, 4, [900, 1] * 8, [1, 2] * 8, False, ("rows", 0, 1)),
    ("f16", 16, 8, 4, [600], [1], False, ("rows", 5, 4)),
    ("f32", 7, 4, 7, [600, 0, 900], [5, 5, 5], False, ("rows", 48, 4)),
    ("bf16", 64, 1, 8, [4000], [1], False, ("rows", 32, 16)),
    ("f16", 16, 2, 3, [2000] * 7, [1] * 7, False, ("rows", 112, 8)),
    ("bf16", 32, 64, 1, [700] * 9, [1] * 9, False, ("rows", 0, 1)),
    # up to 256 rows a request, a small step
    ("f16", 16, 2, 4, [500, 90, 700], [40, 60, 30], False, ("rows", 128, 4)),
    # many rows: whole items
    ("bf16", 16, 2, 4, [500, 90], [100, 60], False, ("chunk", 1)),
    ("f32", 5, 1, 4, [300], [140], False, ("chunk", 1)),
    # even cuts
    ("bf16", 64, 2, 4, [2100, 700], [40, 60], False, ("chunk", 4)),
    ("f16", 48, 1, 2, [1500, 0, 1600], [90, 0, 100], False, ("chunk", 3)),
    ("f32", 16, 2, 8, [1200, 1100], [9, 8], False, ("chunk", 2)),
    ("bf16", 7, 2, 8, [3000], [20], True, ("chunk", 1)),
    # cuts where rows see very different numbers of tokens
    ("f16", 16, 1, 4, [4300], [100], True, ("chunk", 2)),
    ("bf16", 64, 2, 4, [6300, 100], [70, 40], True, ("chunk", 3)),
    ("f32", 7, 1, 3, [4500, 10], [60, 30], True, ("chunk", 2)),
]


def blocks_of(lens, tb):
    """Table width: one more block than the longest request holds."""
    return -(-max(lens) // tb) + 1


def ident(c):
    return f"{c[0]}-T{c[1]}-H{c[2]}x{c[3]}-{sum(c[5])}q-{max(c[4])}"

"""Attention calls that reach every way the work is shared out.

cases(): the rows kernel's,
(name, format, dtype, block_tokens, key heads, query heads per key head,
lengths, queries, moved, expected share).  A share is (heads per score tile,
tiles of 16 rows, heads of different waves of a workgroup, cut into ranges).

PROMPTS: the prompt kernel's, (format, dtype, block_tokens, key heads, query
heads per key head, lengths, queries, tokens cut).  Many query heads per key
head make the rows that it needs out of few queries.
"""

LONG = [1100, 40, 0, 700]          # more than 32 tiles of 32 tokens
MANY = [int(x) for x in range(0, 36 * 26, 26)]      # 36 requests of at most 32 tiles
TOKENS = (64, 16, 7)               # a tile in one block, runs of 8 tokens in one, any


def cases():
    out = []
    for dtype in ("bf16", "f16", "f32"):
        for moved in (False, True):
            for tb in TOKENS:
                for fmt in ("int4", "fp8"):
                    # up to 8 rows of a head: two heads share a score tile
                    out.append(("pair", fmt, dtype, tb, 8, 4, LONG, [2, 1, 2, 1], moved, (2, 1, 1, True)))
                # more rows: two INT4 heads side by side, 16 or 32 rows at a time
                out.append(("sides 16", "int4", dtype, tb, 8, 5, LONG, [3, 1, 2, 3], moved, (1, 1, 2, True)))
                nt = 1 if moved or dtype == "f32" else 2
                out.append(("sides 32", "int4", dtype, tb, 8, 5, LONG, [7, 1, 0, 4], moved, (1, nt, 2, True)))
        # requests of few tiles: whole items, no ranges
        out.append(("pair whole", "int4", dtype, 16, 8, 2, MANY, [1] * 36, False, (2, 1, 1, False)))
        out.append(("pair whole", "fp8", dtype, 32, 8, 2, MANY, [1] * 36, True, (2, 1, 1, False)))
        out.append(("sides whole", "int4", dtype, 64, 8, 9, MANY, [1] * 36, False, (1, 1, 2, False)))
        # one head at a time: odd heads, FP8 of more rows, little work
        out.append(("alone", "fp8", dtype, 64, 8, 5, LONG, [3, 1, 2, 3], False, (1, 1, 1, True)))
        out.append(("alone odd", "int4", dtype, 16, 3, 4, [1100] * 2 + LONG, [1] * 6, True, (1, 1, 1, True)))
        out.append(("alone short", "int4", dtype, 64, 2, 8, [300, 64], [1, 1], False, (1, 1, 1, False)))
    # decodes beside a prompt: most requests have fewer rows than a workgroup of the prompt kernel
    steps = [int(x) for x in range(3, 1203, 75)]
    for fmt, dtype, tb, moved in (("int4", "bf16", 64, False), ("fp8", "f16", 16, True), ("int4", "f32", 7, False)):
        share = (1, 1 if moved or dtype == "f32" else 2, 2 if fmt == "int4" else 1, True)
        out.append(("step", fmt, dtype, tb, 2, 4, steps, [1] * 15 + [110], moved, share))
        out.append(("step first", fmt, dtype, tb, 4, 2, steps, [1] * 8 + [230] + [1] * 7, moved, share))
    return out


PROMPTS = [
    ("int4", "bf16", 64, 1, 128, [1100, 300], [37, 20], True),
    ("int4", "f16", 16, 2, 75, [200], [64], False),
    ("int4", "f32", 64, 1, 96, [130], [50], False),
    ("fp8", "bf16", 7, 1, 128, [90, 60, 77], [38, 0, 40], False),
    ("fp8", "f16", 64, 1, 64, [1300], [75], True),
    ("fp8", "f32", 32, 2, 128, [600], [37], False),
    ("int4", "bf16", 16, 4, 160, [150, 64, 100], [30, 20, 30], False),
]


def blocks_of(lens, tb):
    """Table width: one more block than the longest request holds."""
    return -(-max(lens) // tb) + 1


def name_of(c):
    return f"{c[0]}-{c[1]}-{c[2]}-T{c[3]}-H{c[4]}x{c[5]}" + ("-moved" if c[8] else "")

"""Ragged expert products on shared tiles past one round of the units, for every such form that the plan chooses there and for
every way in which the tiles of the last part round are dealt: cut into 4 or 2 parts of their tokens, or whole.

Keys: (gated, form, parts).  Values: t, rows asked for, seed of the counts, n, k, experts, codes given or not.
"""
import random

UNITS = 256
TILES = {9: (128, 128), 10: (256, 128), 11: (256, 192), 12: (256, 256)}   # packed rows x tokens
TAILS = {
    (0, 9, 1): (467, 16673, 1702, 281, 2064, 3, 1), (0, 9, 2): (70, 13816, 4510, 263, 784, 2, 0),
    (0, 9, 4): (179, 9160, 6476, 275, 528, 30, 0), (0, 10, 4): (551, 1864, 2320, 3211, 528, 8, 1),
    (0, 11, 1): (446, 2115, 9279, 6437, 1552, 7, 1), (0, 11, 2): (381, 1537, 6865, 7611, 656, 4, 1),
    (0, 11, 4): (30, 1133, 8632, 6527, 528, 5, 0), (0, 12, 1): (571, 8623, 3612, 4779, 1552, 2, 1),
    (0, 12, 2): (154, 3776, 1738, 4691, 1040, 3, 1), (0, 12, 4): (203, 1986, 3070, 6235, 528, 4, 1),
    (1, 9, 1): (395, 16785, 3140, 129, 1552, 6, 0), (1, 9, 2): (489, 13856, 6991, 147, 2064, 21, 0),
    (1, 9, 4): (179, 6152, 5583, 319, 656, 6, 0), (1, 10, 4): (370, 413, 3198, 6657, 528, 2, 0),
    (1, 11, 1): (562, 858, 3901, 7043, 1552, 3, 0), (1, 11, 2): (512, 827, 8679, 7353, 784, 2, 1),
    (1, 11, 4): (32, 405, 4495, 8691, 528, 2, 1), (1, 12, 1): (359, 7478, 239, 2719, 1552, 2, 0),
    (1, 12, 2): (281, 1177, 7754, 6089, 1552, 3, 0), (1, 12, 4): (235, 1176, 5902, 5641, 544, 2, 1),
}


def counts(experts, rows, seed):
    """Rows of every expert: none for some, the last one with the most on the mean."""
    rng = random.Random(seed)
    share = [0.0 if rng.random() < 0.2 else rng.random() ** 2 + 0.02 for _ in range(experts)]
    share[-1] += 0.3
    total = sum(share)
    return [int(rows * s / total) for s in share]


def tiles(key):
    """Rows of every tile in the order that the kernel deals them: four token tiles of an expert by its row tiles."""
    gated, form, _ = key
    _, rows, seed, n, _, experts, _ = TAILS[key]
    high, tokens = TILES[form]
    across = -(-((n + 15) // 16 * 16 * (gated + 1)) // high)
    out = []
    for c in counts(experts, rows, seed):
        each = -(-c // tokens)
        for first in range(0, each, 4):
            side = min(4, each - first)
            out += [min(tokens, c - (first + i % side) * tokens) for i in range(side * across)]
    return out

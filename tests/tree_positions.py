"""kv4_positions.py's caches, in which every position leaves its own mark, under
drafted trees: what lora_kv4_attend_tree then gives, with scale 0.  The
tolerance is kv4_positions.TOL: the same weights, codes and sums."""
import numpy as np

import draft_ref as R
import kv4_positions as P

CASES = [  # rows of each tree, positions with them, heads, kv, D, page, window; no class has more than 34 positions
    ([1], [1], 8, 2, 128, 64, 0),
    ([8], [1003], 32, 8, 128, 64, 0),                              # a cluster to a unit (loose bounds: ranges)
    ([5, 2, 6, 3] * 8, [97 * i + 40 for i in range(32)], 32, 8, 64, 16, 0),
    ([7, 0, 1, 3], [7, 40, 33, 99], 6, 2, 128, 16, 0),
    ([33], [70], 2, 1, 128, 16, 0),                                # bits in two words
    ([64, 20, 1], [700, 2100, 130], 32, 8, 128, 64, 0),            # tensor memory
    ([64, 31], [1500, 333], 16, 2, 128, 256, 0),                   # two blocks of 256 rows of a kv head
    ([100, 129], [100, 1000], 8, 1, 64, 16, 0),                    # trees past a tile of 128
    ([16] * 12, [2000 + 37 * i for i in range(12)], 16, 2, 128, 64, 0),
    ([12], [8000], 8, 2, 128, 128, 0),
    ([300], [2100], 4, 2, 128, 32, 0),
    ([9, 30], [700, 45], 4, 4, 64, 16, 3),                         # windows: narrower than the trees
    ([5, 2], [400, 90], 8, 2, 128, 16, 40),                        # inside a tile, across pages
    ([64, 50], [1500, 100], 32, 8, 128, 64, 200),
    ([64, 64], [3000, 300], 16, 2, 64, 128, 1),
    ([6], [3], 4, 2, 128, 16, 0),                                  # rows before the first position
    ([60, 70], [30, 0], 8, 1, 128, 16, 20),
]


def bits_of(case, kind):
    """Ancestors and the row itself, or any set of rows, rows without one among them."""
    q_lens = case[0]
    rng = np.random.default_rng(sum(q_lens) + sum(case[1]))
    if kind == "tree":
        return R.trees(rng, q_lens)
    return [[int.from_bytes(rng.bytes(-(-n // 8)), "little") & ((1 << n) - 1) if rng.random() < 0.8 else 0 for _ in range(n)] for n in q_lens]


def seen(case, bits):
    """The positions that each row sees."""
    out = []
    for mine, c in zip(bits, case[1]):
        n, window = len(mine), case[6]
        base = c - n
        for i, b in enumerate(mine):
            depth = max(1, bin(b).count("1")) - 1
            ctx = np.arange(max(0, base + depth - window + 1) if window else 0, max(0, base))
            own = base + np.array([j for j in range(n) if b >> j & 1], np.int64)
            out.append(np.concatenate([ctx, own[own >= 0]]).astype(np.int64) if base + i >= 0 else np.zeros(0, np.int64))
    return out


def want(case, positions, twice=()):
    """The results [rows][heads][D] over these positions of each row; `twice`: positions counted again."""
    H, KV, D = case[2:5]
    out = np.zeros((len(positions), H, D))
    for t, j in enumerate(positions):
        if len(j) == 0:
            continue
        j = np.concatenate([j, np.intersect1d(j, twice)]).astype(np.int64)
        sums = np.bincount(j // D % KV * D + j % D, weights=P.code(j), minlength=KV * D) / len(j)
        out[t] = np.repeat(sums.reshape(KV, D), H // KV, 0)
    return out

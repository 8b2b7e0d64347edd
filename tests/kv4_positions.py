"""Caches in which every position leaves its own mark on the attention's
result, and what the result then is.

With scale 0 every position that a row sees weighs the same.  V of position j
is code(j) in one dim of one kv head, j's class, and 0 elsewhere, so that a
row's result in a class is the sum of the codes of its positions there over
the number of positions that the row sees.  Codes are 8 to 15 (step 1, low 0:
exact), and no class of the cases has more than 34 positions, so that one
position lost, added or counted twice moves its class by at least
8 / (34 * 15) of its value, four times what the roundings can."""
import numpy as np

import kv4_ref as R

# Weights, codes and their sums are whole numbers below 2^26 with seven trailing
# zeros here, exact in fp16 and fp32 (2^7 a position, times 15); the quotient
# costs two fp32 roundings and the result one in bf16, of 8 significant bits.
TOL = 2.0 ** -8 + 2.0 ** -21

CASES = [  # q_lens, ctx_lens, heads, kv, D, page, window
    ([1], [1], 8, 2, 128, 64, 0),
    ([1], [4099], 8, 2, 128, 64, 0),
    ([1], [20000], 16, 8, 128, 128, 0),                            # a cluster to a unit, then ranges (loose bounds)
    ([1], [34000], 32, 8, 128, 32, 0),
    ([1] * 30, [97 * i + 1 for i in range(30)], 24, 8, 128, 64, 0),
    ([1] * 6, [31, 32, 33, 4095, 4096, 4097], 8, 4, 64, 16, 0),
    ([1, 5, 3, 0, 2], [700, 2049, 33, 90, 4000], 16, 4, 64, 16, 0),
    ([1, 1], [3000, 1025], 32, 2, 128, 256, 0),                    # 16 heads to a kv head
    ([1, 4, 1], [600, 3333, 20], 8, 2, 128, 32, 64),               # windows
    ([1, 2, 7], [16000, 4100, 9000], 32, 8, 128, 16, 4096),
    ([5, 1], [3, 1000], 8, 2, 128, 64, 100),                       # rows before the first position
    ([129], [129], 8, 2, 128, 64, 0),                              # prompts, chunks
    ([40, 100, 30], [40, 2000, 4100], 8, 2, 128, 32, 0),
    ([256], [4000], 8, 2, 128, 128, 0),
    ([64], [2100], 4, 1, 64, 16, 0),
    ([70, 33], [3000, 128], 16, 2, 64, 256, 1000),
    ([300], [300], 12, 4, 128, 16, 37),
    ([90, 65], [64, 500], 3, 1, 128, 64, 0),
]


def code(j):
    """8 to 15, without a pattern that tiles or pages share."""
    return 8 + (j * 2654435761 % 4294967296 >> 20) % 8


def rows(case):
    """(sequence, first position seen, last position) of every row; last < first: it sees nothing."""
    q_lens, ctx, *_, window = case
    return [(s, max(0, p - window + 1) if window else 0, p) for s, p in R.places(q_lens, ctx)]


def want(case, lost=(), only=None):
    """The results [rows][heads][D], of the rows `only`; `lost`: positions left out of every sequence, to show that they
    would be missed."""
    _, _, H, KV, D, _, _ = case
    here = rows(case) if only is None else [rows(case)[t] for t in only]
    out = np.zeros((len(here), H, D))
    for t, (_, j0, p) in enumerate(here):
        if p < 0:
            continue
        j = np.arange(j0, p + 1, dtype=np.int64)
        j = j[~np.isin(j, lost)]
        sums = np.bincount(j // D % KV * D + j % D, weights=code(j), minlength=KV * D) / max(1, len(j))
        out[t] = np.repeat(sums.reshape(KV, D), H // KV, 0)
    return out


def off_by(got, ref):
    """Largest error in units of the tolerance."""
    return float((np.abs(got - ref) / (TOL * np.abs(ref) + 1e-30)).max())


def pack_v(codes):
    """Codes [..., page][D] as the cache's bytes [..., page * D / 2]."""
    *lead, page, D = codes.shape
    c = codes.reshape(*lead, page // 2, 2, D // 4, 4).astype(np.uint32)
    words = np.zeros((*lead, page // 2, D // 4), np.uint32)
    for odd in (0, 1):
        for j in range(4):
            words |= c[..., odd, :, j] << np.uint32(16 * odd + 4 * j)
    return words.view(np.uint8).reshape(*lead, page * D // 2)


def pages_of(case, rng, table, n_pages):
    """A cache for the case's sequences: keys at random, values as above, 15 wherever no position lies."""
    _, ctx, _, KV, D, page, _ = case
    pages = R.random_pages(rng, n_pages, KV, page, D)
    codes = np.full((n_pages, KV, page, D), 15, np.uint8)
    for s, c in enumerate(ctx):
        j = np.arange(c, dtype=np.int64)
        at = np.asarray(table[s])[j // page]
        codes[at, :, j % page] = 0
        codes[at, j // D % KV, j % page, j % D] = code(j)
    G = D // R.GROUP
    pages[..., page * D // 2:page * D] = pack_v(codes)
    vp = np.zeros((n_pages, KV, page // 2, G, 2, 2), "<f2")
    vp[..., 0, :] = 1
    pages[..., page * (D + 4 * G):] = vp.reshape(n_pages, KV, -1).view(np.uint8)
    return pages

"""The oracle of the trees' positions, on the host: what it would show."""
import numpy as np
import pytest

import kv4_positions as P
import tree_positions as T


@pytest.mark.parametrize("kind", ["tree", "any"])
@pytest.mark.parametrize("case", T.CASES, ids=range(len(T.CASES)))
def test_a_lost_or_repeated_position_or_tile_shows(case, kind):
    """In the first and the last row that see anything: a position lost or counted twice by four times the tolerance, at the
    ends, at base and at edges of tiles; a tile lost or counted twice, and a page of the tree, by twice."""
    sees = T.seen(case, T.bits_of(case, kind))
    starts = np.repeat([c - n for n, c in zip(*case[:2])], case[0])
    some = [t for t, j in enumerate(sees) if len(j)]
    for t in {some[0], some[-1]} if some else ():
        j, base = sees[t], max(0, starts[t])
        ref = T.want(case, [j])
        edges = [e + d for tile in (32, 128) for e in range(0, int(j[-1]) + 1, max(tile, int(j[-1]) // 8 // tile * tile)) for d in (-1, 0)]
        for p in np.intersect1d(j, [j[0], j[-1], j[len(j) // 2], base - 1, base, base + 1, *edges]):
            assert P.off_by(T.want(case, [j[j != p]]), ref) > 4
            assert len(j) == 1 or P.off_by(T.want(case, [j], [p]), ref) > 4
        for tile in (case[5], 32, 128):
            for first in {int(p) // tile * tile for p in (j[0], j[-1], j[len(j) // 2], base)}:
                part = np.arange(first, first + tile)
                if 0 < np.isin(j, part).sum() < len(j):
                    assert P.off_by(T.want(case, [j[~np.isin(j, part)]]), ref) > 2
                    assert P.off_by(T.want(case, [j], part), ref) > 2


def test_no_class_has_more_positions_than_the_tolerance_counts_on():
    for case in T.CASES:
        assert max(case[1]) <= 34 * case[3] * case[4]

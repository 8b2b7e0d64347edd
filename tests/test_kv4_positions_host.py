"""The attention tests' oracles, on the host: that the packed caches hold what
they should, and that a position or tile left out of a reference shows."""
import numpy as np
import pytest

import kv4_positions as P
import kv4_ref as R


@pytest.mark.parametrize("case", P.CASES, ids=range(len(P.CASES)))
def test_the_cache_holds_the_marks(case):
    q_lens, ctx, H, KV, D, page, _ = case
    n = [-(-c // page) for c in ctx]
    table = [np.arange(sum(n[:s]), sum(n[:s + 1])) for s in range(len(n))]
    _, V = R.unpack(P.pages_of(case, np.random.default_rng(0), table, sum(n)), page, D)
    for s, c in enumerate(ctx):
        j = np.arange(c)
        v = V[table[s][j // page], :, j % page] if c else np.zeros((0, KV, D))
        assert (v.sum((1, 2)) == P.code(j)).all() and (v[j, j // D % KV, j % D] == P.code(j)).all()


@pytest.mark.parametrize("case", P.CASES, ids=range(len(P.CASES)))
def test_a_lost_position_or_tile_shows(case):
    """In the first and the last row that see anything: the ends and edges of tiles of what they see, by four times the
    tolerance, and whole tiles, which take from every class and from the number of positions alike, by twice."""
    rows = P.rows(case)
    seen = [t for t, r in enumerate(rows) if r[2] >= 0]
    for t in {seen[0], seen[-1]}:
        _, j0, p = rows[t]
        ref = P.want(case, only=[t])
        one = {j0, p, (j0 + p) // 2} | {j for tile in (32, 128) for e in range(-(-j0 // tile) * tile, p + 1, max(tile, (p - j0) // 8 // tile * tile))
                                        for j in (e - 1, e) if j >= j0}
        for j in sorted(one):
            assert P.off_by(P.want(case, [j], [t]), ref) > 4
        for tile in (32, 128):
            for first in {j // tile * tile for j in (j0, p, (j0 + p) // 2)}:
                assert P.off_by(P.want(case, np.arange(first, first + tile), [t]), ref) > 2


@pytest.mark.parametrize("case", [([1], [4099], 8, 1, 128, 64, 0), ([200], [1111], 4, 1, 64, 128, 0)], ids=range(2))
def test_a_lost_tile_shows_in_the_relative_error(case):
    """Of random caches, whose weights differ by powers of ten: nine in ten tiles of 32 positions, left out, move some
    head by more than the limit of 2^-7 that the GPU tests hold rows to.  The elementwise tolerance of kv4_ref, a
    bound for the worst case, lets many of them pass."""
    q_lens, ctx, H, KV, D, page, _ = case
    rng = np.random.default_rng(7 * H + D + 1)
    n = -(-ctx[0] // page)
    K, V = R.unpack(R.random_pages(rng, n, KV, page, D), page, D)
    q = 2 * rng.standard_normal((sum(q_lens), H, D))[-1:]
    ref, tol = R.attend(q, K, V, [1], ctx, [np.arange(n)], page, D ** -0.5)
    shown, let_pass, firsts = 0, 0, range(0, ctx[0], 32)
    for first in firsts:
        keep = np.ones(ctx[0], bool)
        keep[first:first + 32] = False
        k, v = (x.transpose(1, 0, 2, 3).reshape(KV, -1, D)[:, :ctx[0]][:, keep] for x in (K, V))
        w = np.exp(D ** -0.5 * q[0] @ k[0].T)
        out = w / w.sum(1, keepdims=True) @ v[0]
        rel = np.linalg.norm(out - ref[0], axis=1) / np.linalg.norm(ref[0], axis=1)
        shown += rel.max() > 2.0 ** -7
        let_pass += (np.abs(out - ref[0]) <= tol[0]).all()
    assert shown >= 0.9 * len(firsts) and let_pass > 0

"""Plain references of drafted decoding's operators, in whole numbers and 64
bits on the host, from the formulas that include/lora.h states."""
import numpy as np

import kv4_ref as R

BAD_SEGMENT, BAD_PAGE, NO_PAGES = 0x2, 0x8, 0x20


def plan(q_lens, lens, held, table, free, n_free, *, page, max_rows, max_q, max_ctx, depths=None):
    """Every output of lora_kv4_plan, and the status bits."""
    n, wide, n_pages = len(q_lens), table.shape[1], len(free)
    table, free, held = table.copy(), free.copy(), np.array(held, np.int64)
    faults = 0
    if not 0 <= n_free <= n_pages:
        faults, n_free = faults | BAD_PAGE, 0
    counts = (held >= 0) & (held <= wide)
    if not counts.all():
        faults |= BAD_SEGMENT
    for s in range(n):
        if q_lens[s] < 0:
            if counts[s]:
                for p in table[s, :held[s]]:
                    if n_free < n_pages:
                        free[n_free] = p
                        n_free += 1
                    else:
                        faults |= BAD_PAGE
            held[s] = 0
    top, asked, at = n_free, 0, 0
    starts, ctx = [0], np.zeros(n, np.int64)
    row_seq, pos, slots = (np.full(max_rows, -1, np.int64) for _ in range(3))
    for s in range(n):
        q = int(q_lens[s])
        m = max(0, q)
        if q >= 0:
            ok = bool(counts[s]) and m <= max_q and 0 <= lens[s] and lens[s] + m <= max_ctx
            if not ok:
                faults |= BAD_SEGMENT
            need = max(0, -(-(int(lens[s]) + m) // page) - int(held[s])) if ok and m else 0
            asked += need
            if ok and m and at + m > max_rows:
                ok, faults = False, faults | BAD_SEGMENT
            if ok and need and asked > top:
                ok, faults = False, faults | NO_PAGES
            if ok:
                ctx[s] = lens[s] + m
                for j in range(need):
                    table[s, held[s] + j] = free[top - 1 - (asked - need) - j]
                held[s] += need
                n_free -= need
                for i in range(m):
                    p, t = int(lens[s]) + i, at + i
                    d = i if depths is None else int(depths[t])
                    row_seq[t], pos[t] = s, lens[s] + d if 0 <= d < max_ctx else -1
                    slots[t] = int(table[s, p // page]) * page + p % page if 0 <= table[s, p // page] < n_pages else -1
        at += m
        starts.append(min(at, max_rows))
    return dict(q_starts=np.array(starts), ctx_lens=ctx, block_table=table, held=held, free_pages=free, n_free=n_free, row_seq=row_seq,
                positions=pos, slots=slots), faults


def trees(rng, q_lens, chain=False):
    """Bits of every row, as Python integers: ancestors and itself in random trees."""
    bits = []
    for n in q_lens:
        mine = []
        for i in range(n):
            up = i - 1 if chain else int(rng.integers(max(-1, i - 5), i)) if i else -1
            mine.append((mine[up] if up >= 0 else 0) | 1 << i)
        bits.append(mine)
    return bits


def words(bits, ld, noise=None):
    """int32 [rows][ld]; noise: an rng that fills the bits from n on."""
    rows = []
    for mine in bits:
        for b in mine:
            if noise is not None and len(mine) < 32 * ld:
                b |= int(noise.integers(0, 1 << 62)) << len(mine)
            rows.append([b >> 32 * w & 0xFFFFFFFF for w in range(ld)])
    return np.array(rows, np.uint32).reshape(-1, ld).view(np.int32)


def attend_tree(q, K, V, bits, ctx_lens, table, page, scale, window=0):
    """As kv4_ref.attend, whose bound on the error holds for any set of positions: (out, tol)."""
    T, H, D = q.shape
    n_kv = K.shape[1]
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    t = 0
    for s, (mine, c) in enumerate(zip(bits, ctx_lens)):
        n = len(mine)
        base = c - n
        pages = table[s][:-(-c // page)] if c else []
        for i in range(n):
            own = [base + j for j in range(n) if mine[i] >> j & 1 and base + j >= 0]
            depth = max(1, bin(mine[i] & ((1 << n) - 1)).count("1")) - 1
            seen = list(range(max(0, base + depth - window + 1) if window else 0, max(0, base))) + own
            if base + i >= 0 and seen:
                at = [(pages[j // page], j % page) for j in seen]
                ids, off = (np.array(x) for x in zip(*at))
                for h in range(n_kv):
                    kk, vv = K[ids, h, off], V[ids, h, off]
                    sl = slice(h * (H // n_kv), (h + 1) * (H // n_kv))
                    rows = q[t, sl]
                    sc = scale * rows @ kk.T
                    w = np.exp(sc - sc.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    E = 2.0 ** -10 * abs(scale) * np.max(np.abs(rows) @ np.abs(kk).T, axis=1, keepdims=True)
                    o, a = w @ vv, w @ np.abs(vv)
                    out[t, sl] = o
                    tol[t, sl] = 2.0 ** -8 * np.abs(o) + a * (2 * E + 2.0 ** -9) + 1e-30
            t += 1
    return out, tol


def place_bytes(page, D, o):
    """Indices, in a head's block, of the bytes of its position o: in the same order for every o."""
    G = D // R.GROUP
    k = np.arange(o * D // 2, (o + 1) * D // 2)
    v = page * D // 2 + o // 2 * D + 2 * (o % 2) + np.add.outer(4 * np.arange(D // 4), [0, 1]).ravel()
    kp = page * D + 4 * G * o + np.arange(4 * G)
    vp = page * (D + 4 * G) + 2 * (o % 2) + np.add.outer(8 * (o // 2 * G + np.arange(G)), [0, 1, 4, 5]).ravel()
    return np.concatenate([k, v, kp, vp])


def keep(pages, D, page, table, q_lens, ctx_lens, n_keep, path):
    """pages: uint8 [n_pages][n_kv][block] of one cache -> with the kept rows moved up."""
    out = pages.copy()
    for s, (n, c) in enumerate(zip(q_lens, ctx_lens)):
        for i in range(n_keep[s] if c >= n else 0):
            (sp, so), (dp, do) = divmod(c - n + int(path[s][i]), page), divmod(c - n + i, page)
            out[table[s][dp]][:, place_bytes(page, D, do)] = pages[table[s][sp]][:, place_bytes(page, D, so)]
    return out


def adjust(x, tokens, prompt, length, rep, freq, pres, biases, path=(), allowed=None):
    """One row of logits, float64 [vocab]; biases: pairs in their order; path: drafted tokens.  Returns (y, M): M is the
    sum of the magnitudes that its fp32 operations add up, each of which is off by 2^-24 of that at most."""
    V = len(x)
    inside = lambda a: np.asarray([v for v in a if 0 <= v < V], np.int64)  # noqa: E731
    made = np.bincount(np.concatenate([inside(tokens[prompt:length]), inside(path)]), minlength=V).astype(np.float64)
    seen = (made > 0) | (np.bincount(inside(tokens[:prompt]), minlength=V) > 0)
    with np.errstate(all="ignore"):
        y = np.where(seen, np.where(x > 0, x / rep, x * rep), x)
        M = np.abs(y) + np.where(made > 0, freq * made + pres, 0)
        y = np.where(made > 0, y - freq * made - pres, y)
    for v, b in dict((v, b) for v, b in biases if 0 <= v < V).items():
        y[v] += b
        M[v] += abs(b)
    if allowed is not None:
        y = np.where(allowed, y, -np.inf)
    return y, M

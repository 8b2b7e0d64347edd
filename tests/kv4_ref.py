"""Plain references of the norm and the 4-bit cache's operators, in 64 bits
on the host, from the formulas and the layout that include/lora.h states."""
import numpy as np

GROUP = 64
KMAX = 60000.0


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def block_bytes(page, D):
    return page * (D + 8 * (D // GROUP))


def _k_nibbles(D):
    """(word, nibble) of every K dim: word (t, w) holds dims 32w + 8t + n."""
    d = np.arange(D)
    return ((d % 32) // 8) * (D // 32) + d // 32, d % 8


def unpack(pages, page, D):
    """uint8 [n_pages][n_kv][block] -> K, V float64 [n_pages][n_kv][page][D]."""
    n, kv, _ = pages.shape
    G = D // GROUP
    raw = np.ascontiguousarray(pages)
    kw = raw[..., :page * D // 2].copy().view("<u4").reshape(n, kv, page, D // 8)
    w, nib = _k_nibbles(D)
    k = ((kw[..., w] >> (4 * nib).astype(np.uint32)) & 15).astype(np.float64)
    vw = raw[..., page * D // 2:page * D].copy().view("<u4").reshape(n, kv, page // 2, D // 4)
    v = np.empty((n, kv, page, D))
    for odd in (0, 1):
        for j in range(4):
            v[:, :, odd::2, j::4] = (vw >> np.uint32(16 * odd + 4 * j)) & 15
    with np.errstate(invalid="ignore"):   # what a page holds past its positions may be anything
        kp = raw[..., page * D:page * (D + 4 * G)].copy().view("<f2").reshape(n, kv, page, G, 2).astype(np.float64)
        vp = raw[..., page * (D + 4 * G):].copy().view("<f2").reshape(n, kv, page // 2, G, 2, 2).astype(np.float64)
    vp = np.moveaxis(vp, -1, 3).reshape(n, kv, page, G, 2)
    at = np.arange(D) // GROUP
    with np.errstate(invalid="ignore", over="ignore"):
        return k * kp[..., at, 0] + kp[..., at, 1], v * vp[..., at, 0] + vp[..., at, 1]


def random_pages(rng, n_pages, n_kv, page, D, k_scale=0.3, v_scale=0.3):
    """A cache of random codes and parameters: uint8 [n_pages][n_kv][block]."""
    G = D // GROUP
    codes = rng.integers(0, 256, (n_pages, n_kv, page * D), dtype=np.uint8)
    kp = np.empty((n_pages, n_kv, page, G, 2), "<f2")
    kp[..., 0] = k_scale * (0.5 + rng.random(kp.shape[:-1]))
    kp[..., 1] = -7.5 * k_scale + 0.3 * rng.standard_normal(kp.shape[:-1])
    vp = np.empty((n_pages, n_kv, page // 2, G, 2, 2), "<f2")
    vp[..., 0, :] = v_scale * (0.5 + rng.random(vp.shape[:-2] + (2,)))
    vp[..., 1, :] = -7.5 * v_scale + 0.3 * rng.standard_normal(vp.shape[:-2] + (2,))
    tail = [a.reshape(n_pages, n_kv, -1).view(np.uint8) for a in (kp, vp)]
    return np.concatenate([codes, *tail], 2)


def places(q_lens, ctx_lens):
    """(sequence, position) of every row."""
    return [(s, c - n + i) for s, (n, c) in enumerate(zip(q_lens, ctx_lens)) for i in range(n)]


def attend(q, K, V, q_lens, ctx_lens, table, page, scale, window=0):
    """q [T][H][D] float64; K, V from unpack().  Returns (out, tol): the
    attention and a bound on a kernel's error: the bf16 result (2^-8 of it),
    and, against sum p |v|, the softmax weights and values in fp16 (2^-11
    each, and as much again for the sum of the weights) and the scores'
    error E twice (numerator and denominator), where q, the cached keys in fp16
    and the fp32 sums cost at most 2^-10 of scale * sum |q| |k|."""
    T, H, D = q.shape
    n_kv = K.shape[1]
    out, tol = np.zeros((T, H, D)), np.zeros((T, H, D))
    t = 0
    for s, (n, c) in enumerate(zip(q_lens, ctx_lens)):
        pages = table[s][:-(-c // page)] if c else []
        k = np.concatenate([K[p] for p in pages], 1)[:, :c] if c else None    # [n_kv][c][D]
        v = np.concatenate([V[p] for p in pages], 1)[:, :c] if c else None
        for i in range(n):
            p = c - n + i
            if p >= 0:
                j0 = max(0, p - window + 1) if window else 0
                for h in range(n_kv):
                    kk, vv = k[h, j0:p + 1], v[h, j0:p + 1]
                    rows = q[t, h * (H // n_kv):(h + 1) * (H // n_kv)]
                    sc = scale * rows @ kk.T
                    w = np.exp(sc - sc.max(1, keepdims=True))
                    w /= w.sum(1, keepdims=True)
                    E = 2.0 ** -10 * abs(scale) * np.max(np.abs(rows) @ np.abs(kk).T, axis=1, keepdims=True)
                    o, a = w @ vv, w @ np.abs(vv)
                    sl = slice(h * (H // n_kv), (h + 1) * (H // n_kv))
                    out[t, sl] = o
                    tol[t, sl] = 2.0 ** -8 * np.abs(o) + a * (2 * E + 2.0 ** -9) + 1e-30
            t += 1
    return out, tol


def rotate(x, table, pos, pairs):
    """x [T][heads][D] float64, table [max_pos][half][2], pos [T][axes]."""
    x = x.copy()
    half = table.shape[1]
    first = 0
    for a, n in enumerate(pairs):
        i = np.arange(first, first + n)
        c, s = table[pos[:, a]][:, None, i, 0], table[pos[:, a]][:, None, i, 1]
        lo, hi = x[..., i].copy(), x[..., i + half].copy()
        x[..., i], x[..., i + half] = lo * c - hi * s, hi * c + lo * s
        first += n
    assert first == half
    return x


def quantise32(x):
    """The stored form of float32 values [..., D]: (codes, step, low), every
    operation rounded on its own as the append does it."""
    f = np.float32
    g = np.clip(x.astype(f), f(-KMAX), f(KMAX)).reshape(*x.shape[:-1], -1, GROUP)
    lo, hi = g.min(-1, keepdims=True), g.max(-1, keepdims=True)
    step = ((hi - lo) * f(1 / 15)).astype(np.float16).astype(f)
    low = lo.astype(np.float16).astype(f)
    with np.errstate(divide="ignore"):
        inv = np.where(step > 0, f(1) / step, f(0)).astype(f)
    codes = np.clip(np.rint((g - low) * inv), 0, 15)
    return codes, step, low


def norm(x, w, eps, res=None):
    """(h, n) in 64 bits; h rounded to bf16 where there is a residual."""
    import torch
    h = x if res is None else f64(torch.from_numpy((x + res).astype(np.float32)).to(torch.bfloat16))
    return h, h / np.sqrt((h * h).mean(1, keepdims=True) + eps) * w

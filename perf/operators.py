"""Cases and plain forms of the operators around a LoRA attention block.

Three operators, measured one pass at a time:

  norm    lora_rms_norm: h = bf16(x + residual), y = h / rms(h) * weight in
          bf16 (the input of the LoRA projections) and, from the same fp32
          values, in 8 bits with a scale per group of columns (the input of
          an 8-bit base product).
  append  lora_kv4_append + lora_kv4_read: rows [q|k|v] of the fused
          projection; q and k are rotated by tables of up to three position
          axes, k and v go to a paged cache in 4 bits; then the rows' cached
          values are read back (bf16).
  attend  lora_kv4_attend: causal attention of the batch's rows over the
          paged 4-bit cache, with grouped heads and an optional window; rows
          without a visible position give zeros.

The 4-bit cache: per page and kv head one block of bytes,
  K codes  [page][4][D/32] words; word (t, w) holds dims 32w + 8t + n at nibble n
  V codes  [page/2][D/4] words;   word i holds dims 4i + j, of the even token at
                                  nibble j, of the odd token at nibble 4 + j
  K params [page][D/64][2] fp16;  (step, lowest) of the token's group of 64 dims
  V params [page/2][D/64][4] fp16; (step even, step odd, lowest even, lowest odd)
and a value is code * step + lowest.
"""
import math
import random

import numpy as np
import torch

own = False

EPS = 1e-5
KMAX = 60000.0          # cached values saturate here, inside fp16's range


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token's norm before a projection group of a 70B-shaped layer
        {"name": "norm_token", "op": "norm", "rows": 1, "width": 8192, "group": 0, "eight": False, "res": True},
        # a decode batch's norm, bf16 for the adapters and 8 bits for the base product
        {"name": "norm_decode", "op": "norm", "rows": 64, "width": 4096, "group": 128, "eight": True, "res": True},
        # a Mistral-7B-shaped prefill batch (its 35,402 rows)
        {"name": "norm_prefill", "op": "norm", "rows": 35402, "width": 4096, "group": 0, "eight": True, "res": True},
        # decode: one new token in each of 256 requests
        {"name": "append_decode", "op": "append", "seqs": 256, "q_min": 1, "q_max": 1, "ctx_min": 1, "ctx_max": 4096,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "rot": 128, "axes": 1, "lens": 11},
        # prefill: ragged prompts with image tokens (time, height, width positions), and cached prefixes
        {"name": "append_prefill", "op": "append", "seqs": 16, "q_min": 64, "q_max": 2048, "ctx_min": 0, "ctx_max": 1000,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "rot": 128, "axes": 3, "lens": 12},
        # one request alone, one token: latency
        {"name": "attend_token", "op": "attend", "seqs": 1, "q_min": 1, "q_max": 1, "ctx_min": 1003, "ctx_max": 1003,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "window": 0, "lens": 21},
        # a ragged decode batch of 64 requests, heads of a 3B-shaped model (groups of 3)
        {"name": "attend_decode", "op": "attend", "seqs": 64, "q_min": 1, "q_max": 1, "ctx_min": 17, "ctx_max": 8192,
         "heads": 24, "kv": 8, "dim": 128, "page": 64, "window": 0, "lens": 22},
        # decode over long documents, 70B-shaped heads
        {"name": "attend_long", "op": "attend", "seqs": 8, "q_min": 1, "q_max": 1, "ctx_min": 131072, "ctx_max": 131072,
         "heads": 64, "kv": 8, "dim": 128, "page": 128, "window": 0, "lens": 23},
        # a few drafted tokens to a request, heads of 64, small pages
        {"name": "attend_draft", "op": "attend", "seqs": 32, "q_min": 2, "q_max": 5, "ctx_min": 100, "ctx_max": 4096,
         "heads": 32, "kv": 8, "dim": 64, "page": 16, "window": 0, "lens": 24},
        # decode and short chunks in a sliding window, Mistral-7B-shaped
        {"name": "attend_window", "op": "attend", "seqs": 24, "q_min": 1, "q_max": 64, "ctx_min": 512, "ctx_max": 12000,
         "heads": 32, "kv": 8, "dim": 128, "page": 32, "window": 4096, "lens": 25},
        # prompts of 64 to 2048 tokens from their first token on
        {"name": "attend_prefill", "op": "attend", "seqs": 16, "q_min": 64, "q_max": 2048, "ctx_min": 0, "ctx_max": 0,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "window": 0, "lens": 26},
        # one chunk of a long prompt over what is cached of it
        {"name": "attend_chunk", "op": "attend", "seqs": 1, "q_min": 1024, "q_max": 1024, "ctx_min": 31744, "ctx_max": 31744,
         "heads": 64, "kv": 8, "dim": 128, "page": 64, "window": 0, "lens": 27},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["norm", "append", "attend", "attend"])
    if op == "norm":
        width = 8 * _log(rng, 16, 2048)
        rows = _log(rng, 1, 35402)
        rows = max(1, min(rows, 35402 * 4096 // width))
        eight = rng.random() < 0.6
        return {"op": op, "rows": rows, "width": width, "group": rng.choice([0, 128]), "eight": eight,
                "res": rng.random() < 0.8}
    heads, kv = rng.choice([(24, 8), (32, 8), (64, 8), (8, 8), (28, 4), (16, 1), (40, 8)])
    c = {"op": op, "heads": heads, "kv": kv, "dim": rng.choice([64, 128, 128]), "page": rng.choice([16, 32, 64, 128]),
         "lens": rng.randrange(1 << 30)}
    if op == "append":
        seqs = _log(rng, 1, 256)
        q_max = _log(rng, 1, max(1, 16384 // seqs))
        c.update(seqs=seqs, q_min=rng.choice([1, q_max]), q_max=q_max, ctx_min=0, ctx_max=_log(rng, 1, 4096),
                 axes=rng.choice([1, 2, 3]), rot=rng.choice([c["dim"], c["dim"], c["dim"] // 2]))
        return c
    if rng.random() < 0.6:     # single tokens and drafts
        q_max = rng.choice([1, 1, 1, 2, 3, 7])
        seqs = _log(rng, 1, 128)
        ctx = _log(rng, 16, min(131072, 8 * 131072 * 8 // (seqs * kv)))
    else:                      # prompts and chunks
        q_max = _log(rng, 9, 2048)
        seqs = _log(rng, 1, max(1, 16384 // q_max))
        ctx = _log(rng, 16, 8192)
        while seqs > 1 and seqs * q_max * (q_max + ctx) * heads > 16 * 2048 * 2048 * 16:
            seqs = (seqs + 1) // 2
        ctx = max(16, min(ctx, 16 * 2048 * 2048 * 16 // (seqs * q_max * heads) - q_max))
    c.update(seqs=seqs, q_min=rng.choice([1, q_max]), q_max=q_max, ctx_min=rng.choice([0, ctx]), ctx_max=ctx,
             window=rng.choice([0, 0, 0, _log(rng, 16, 4096)]))
    return c


def _lens(c):
    """(query lengths, context lengths with the queries' own positions) of a case's requests."""
    r = random.Random(c["lens"])
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["seqs"])]
    lo, hi = c["ctx_min"], c["ctx_max"]
    ctx = [lo if lo == hi else min(hi, lo - 1 + int(round(math.exp(r.uniform(0, math.log(hi - lo + 2)))))) for _ in q]
    return q, [max(0, p) + n for p, n in zip(ctx, q)]


def _pairs(c):
    """Rotary pairs of each axis: a third each, the first axis takes the rest."""
    half, axes = c["rot"] // 2, c["axes"]
    each = half // axes
    return [half - each * (axes - 1)] + [each] * (axes - 1)


def block_bytes(page, dim):
    return page * (dim + dim // 64 * 8)


# ------------------------------------------------------------------- state ----

def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 17)
    bf = lambda *s, k=1.0: (torch.randn(*s, generator=g, device="cuda") * k).to(torch.bfloat16)  # noqa: E731
    s = {"c": c}
    if c["op"] == "norm":
        T, W = c["rows"], c["width"]
        s["x"] = bf(T, W)
        s["res"] = bf(T, W, k=4.0) if c["res"] else None
        s["w"] = (1 + 0.2 * torch.randn(W, generator=g, device="cuda")).to(torch.bfloat16)
        s["y"] = torch.empty_like(s["x"])
        s["h"] = torch.empty_like(s["x"]) if c["res"] else None
        n = -(-W // c["group"]) if c["group"] else 1
        s["y8"] = torch.empty(T, W, dtype=torch.float8_e4m3fn, device="cuda") if c["eight"] else None
        s["scales"] = torch.empty(T, n, dtype=torch.float32, device="cuda") if c["eight"] else None
        return s
    q, ctx = _lens(c)
    H, KV, D, page = c["heads"], c["kv"], c["dim"], c["page"]
    T, pages = sum(q), [-(-n // page) for n in ctx]
    r = random.Random(seed * 31 + c["lens"])
    ids = list(range(sum(pages) + 2))
    r.shuffle(ids)
    table = np.full((len(q), max(pages)), -1, np.int32)
    at = 0
    for i, n in enumerate(pages):
        table[i, :n] = ids[at:at + n]
        at += n
    s["table"] = torch.from_numpy(table).cuda()
    s["starts"] = torch.from_numpy(np.concatenate([[0], np.cumsum(q)]).astype(np.int32)).cuda()
    s["ctx"] = torch.from_numpy(np.asarray(ctx, np.int32)).cuda()
    s["max_q"], s["max_ctx"], s["rows"] = max(q), max(ctx), T
    s["page"], s["kv"], s["dim"] = page, KV, D
    if c["op"] == "append":
        s["pages"] = torch.zeros(len(ids), KV, block_bytes(page, D), dtype=torch.uint8, device="cuda")
        s["qkv"] = bf(T, (H + 2 * KV) * D)
        s["qkv"][:, H * D:(H + KV) * D].view(T, KV, D)[:, :, 5::32] *= 6      # keys have a few large channels
        s["q_out"] = torch.empty(T, H * D, dtype=torch.bfloat16, device="cuda")
        s["k_out"] = torch.empty(T, KV * D, dtype=torch.bfloat16, device="cuda")
        s["v_out"] = torch.empty(T, KV * D, dtype=torch.bfloat16, device="cuda")
        half = c["rot"] // 2
        f = 10000.0 ** (-torch.arange(half, device="cuda", dtype=torch.float64) / half)
        a = torch.arange(s["max_ctx"], device="cuda", dtype=torch.float64)[:, None] * f
        s["rope"] = torch.stack([a.cos(), a.sin()], -1).float()               # [max_pos][half][2]
        first = torch.cat([torch.arange(n - m, n, dtype=torch.int32) for m, n in zip(q, ctx)]).cuda()
        cols = [first] + [torch.randint(0, min(64, s["max_ctx"]), (T,), generator=g, device="cuda", dtype=torch.int32)
                          for _ in range(c["axes"] - 1)]
        s["pos"] = torch.stack(cols, 1).contiguous()
        s["seg"] = _pairs(c)
    else:
        # what an append leaves: codes that lie in a bell over 0..15, steps that vary by token and group
        nb, G = len(ids), D // 64
        code = torch.randint(0, 8, (nb, KV, page * D, 2), generator=g, device="cuda", dtype=torch.uint8)
        code += torch.randint(0, 9, code.shape, generator=g, device="cuda", dtype=torch.uint8)
        codes = code[..., 0] | (code[..., 1] << 4)
        del code
        step = 0.2 + 0.1 * torch.rand(nb, KV, 2, page, G, generator=g, device="cuda")
        low = -7.5 * step + 0.2 * torch.randn(step.shape, generator=g, device="cuda")
        kp = torch.stack([step[:, :, 0], low[:, :, 0]], -1).half()                                  # [..][page][G][2]
        vp = torch.stack([step[:, :, 1], low[:, :, 1]], 2).half()                                   # [..][2][page][G]
        vp = vp.view(nb, KV, 2, page // 2, 2, G).permute(0, 1, 3, 5, 2, 4).contiguous()             # [pair][G][2][2]
        s["pages"] = torch.cat([codes, kp.reshape(nb, KV, -1).view(torch.uint8), vp.reshape(nb, KV, -1).view(torch.uint8)], 2).contiguous()
        del codes, step, low, kp, vp
        s["q"] = bf(T, H * D, k=2.0)
        s["out"] = torch.empty_like(s["q"])
    if own:   # the handles that a serving program keeps: its cache, this step's batch, a workspace
        from lora_serving_gb300 import store
        s["cache"] = store.KV4Cache(nb if c["op"] == "attend" else len(ids), page, KV, D, pages=s["pages"])
        s["batch"] = store.KV4Batch(s["starts"], s["ctx"], s["table"], n_rows=T, max_q_len=s["max_q"], max_ctx_len=s["max_ctx"])
        if c["op"] == "attend":
            s["ws"] = store.kv4_workspace(s["cache"], H, s["batch"])
    return s


# --------------------------------------------------------------------- run ----

def run(s):
    c = s["c"]
    return (_own if own else _plain)[c["op"]](s, c)


def _own_norm(s, c):
    from lora_serving_gb300 import abi
    abi.lora_rms_norm(s["x"], s["w"], EPS, residual=s["res"], residual_out=s["h"], y=s["y"], y8=s["y8"],
                      scales=s["scales"], group=c["group"])
    return {k: s[k] for k in ("y", "h", "y8", "scales") if s[k] is not None}


def _own_append(s, c):
    from lora_serving_gb300 import abi
    H, KV, D = c["heads"], c["kv"], c["dim"]
    abi.lora_kv4_append(s["q_out"], s["qkv"], s["cache"], s["batch"], n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D,
                        rope=s["rope"], positions=s["pos"], axis_pairs=s["seg"])
    abi.lora_kv4_read(s["k_out"], s["v_out"], s["cache"], s["batch"])
    return {"q": s["q_out"], "k": s["k_out"], "v": s["v_out"]}


def _own_attend(s, c):
    from lora_serving_gb300 import abi
    abi.lora_kv4_attend(s["out"], s["q"], s["cache"], s["batch"], s["ws"], n_heads=c["heads"],
                        scale=1.0 / math.sqrt(c["dim"]), window=c["window"])
    return s["out"]


def _plain_norm(s, c):
    x = s["x"].float()
    out = {}
    if s["res"] is not None:
        out["h"] = (x + s["res"].float()).to(torch.bfloat16)
        x = out["h"].float()
    y = x * torch.rsqrt((x * x).mean(1, keepdim=True) + EPS) * s["w"].float()
    out["y"] = y.to(torch.bfloat16)
    if c["eight"]:
        T, W = y.shape
        n = s["scales"].shape[1]
        size = c["group"] or W
        grp = torch.nn.functional.pad(y, (0, n * size - W)).view(T, n, size)
        amax = grp.abs().amax(2)
        inv = torch.where(amax > 0, 448.0 / amax, torch.zeros_like(amax))
        out["scales"] = amax * (1.0 / 448.0)
        y8 = (grp * inv[..., None]).view(T, n * size)[:, :W]
        out["y8"] = y8.clamp(-448.0, 448.0).to(torch.float8_e4m3fn)
    return out


def _rows(s):
    """Of every row of the batch: its request, its place in the cache."""
    t = torch.arange(s["rows"], device="cuda")
    starts = s["starts"].long()
    b = torch.searchsorted(starts, t, right=True) - 1
    return b, s["ctx"].long()[b] - (starts[b + 1] - starts[b]) + t - starts[b]


def _quantise(x):
    """Values [.., D] in groups of 64: (codes, step, lowest), as the cache holds them."""
    x = x.clamp(-KMAX, KMAX).unflatten(-1, (-1, 64))
    lo, hi = x.amin(-1, keepdim=True), x.amax(-1, keepdim=True)
    step, low = ((hi - lo) * np.float32(1 / 15).item()).half().float(), lo.half().float()
    inv = torch.where(step > 0, torch.ones_like(step) / step, torch.zeros_like(step))
    return ((x - low) * inv).round().clamp(0, 15), step, low


def _plain_append(s, c):
    H, KV, D, page, half = c["heads"], c["kv"], c["dim"], c["page"], c["rot"] // 2
    T, G = s["rows"], D // 64
    x = s["qkv"].float().view(T, H + 2 * KV, D)
    b, p = _rows(s)
    axis = torch.repeat_interleave(torch.arange(c["axes"], device="cuda"), torch.tensor(s["seg"], device="cuda"), output_size=half)
    cs = s["rope"][s["pos"].long()[:, axis], torch.arange(half, device="cuda")]                     # [T][half][2]
    cos, sin = cs[:, None, :, 0], cs[:, None, :, 1]
    qk = x[:, :H + KV]
    lo, hi = qk[..., :half], qk[..., half:2 * half]
    qk = torch.cat([lo * cos - hi * sin, hi * cos + lo * sin, qk[..., 2 * half:]], -1)
    kc, ks, kl = _quantise(qk[:, H:])
    vc, vs, vl = _quantise(x[:, H + KV:])
    # into the cache: the bytes of one token of one head
    block = s["pages"]
    pg, off = s["table"].long()[b, p // page], p % page
    nib = kc.to(torch.uint8).view(T, KV, D // 32, 4, 4, 2).transpose(2, 3)                          # (t, w, byte, half)
    kbytes = (nib[..., 0] | (nib[..., 1] << 4)).reshape(T, KV, D // 2)
    nib = vc.to(torch.uint8).view(T, KV, D // 4, 2, 2)
    vbytes = (nib[..., 0] | (nib[..., 1] << 4)).reshape(T, KV, D // 4, 2)
    kp = torch.cat([ks, kl], -1).half().view(T, KV, G * 2).view(torch.uint8)
    vp = torch.cat([vs, vl], -1).half().view(torch.uint8).view(T, KV, G, 2, 2)
    r = lambda *n: torch.arange(math.prod(n), device="cuda").view(n)  # noqa: E731
    at_k = off[:, None] * (D // 2) + r(D // 2)
    at_v = page * D // 2 + (off // 2)[:, None, None] * D + (off % 2)[:, None, None] * 2 + 4 * r(D // 4)[:, None] + r(2)
    at_kp = page * D + off[:, None] * (G * 4) + r(G * 4)
    at_vp = (page * (D + G * 4) + (off // 2)[:, None, None, None] * (G * 8) + (off % 2)[:, None, None, None] * 2
             + 8 * r(G)[:, None, None] + 4 * r(2)[:, None] + r(2))
    for at, v in ((at_k, kbytes), (at_v, vbytes), (at_kp, kp), (at_vp, vp)):
        n = at.numel() // T
        block[pg[:, None, None], r(KV)[:, None], at.reshape(T, 1, n)] = v.reshape(T, KV, n)
    val = lambda code, step, low: (code * step + low).to(torch.bfloat16).reshape(T, KV * D)  # noqa: E731
    return {"q": qk[:, :H].to(torch.bfloat16).reshape(T, H * D), "k": val(kc, ks, kl), "v": val(vc, vs, vl)}


def _values(blocks, page, D):
    """The K and V that blocks [..][block_bytes] of a cache stand for: [..][page][D], 32 bits."""
    G, lead = D // 64, blocks.shape[:-1]
    nib = lambda b: torch.stack([b & 15, b >> 4], -1)  # noqa: E731
    kc = nib(blocks[..., :page * D // 2].reshape(*lead, page, 4, D // 32, 4)).transpose(-4, -3).reshape(*lead, page, G, 64)
    vc = nib(blocks[..., page * D // 2:page * D].reshape(*lead, page // 2, D // 4, 2, 2))
    vc = vc.movedim(-3, -4).reshape(*lead, page, G, 64)
    at = page * D
    kp = blocks[..., at:at + page * G * 4].contiguous().view(torch.float16).view(*lead, page, G, 2).float()
    vp = blocks[..., at + page * G * 4:].contiguous().view(torch.float16).view(*lead, page // 2, G, 2, 2).float()
    vp = vp.permute(*range(len(lead)), -4, -1, -3, -2).reshape(*lead, page, G, 2)
    out = [(code.float() * p[..., :1] + p[..., 1:]).reshape(*lead, page, D) for code, p in ((kc, kp), (vc, vp))]
    return out


def _plain_attend(s, c):
    H, KV, D, page, B = c["heads"], c["kv"], c["dim"], c["page"], c["seqs"]
    R, N, C = H // KV, s["max_q"], s["table"].shape[1] * page
    blocks = s["pages"][s["table"].long().clamp(min=0)].transpose(1, 2)                            # [B][KV][P][bytes]
    k, v = (x.reshape(B, KV, C, D) for x in _values(blocks, page, D))
    b, p = _rows(s)
    i = torch.arange(s["rows"], device="cuda") - s["starts"].long()[b]
    q = torch.zeros(B, N, H, D, device="cuda")
    q[b, i] = s["q"].float().view(-1, H, D) * (1.0 / math.sqrt(D))
    q = q.view(B, N, KV, R, D).permute(0, 2, 1, 3, 4).reshape(B, KV, N * R, D)
    last = torch.full((B, N), -1, device="cuda", dtype=torch.long)
    last[b, i] = p
    j = torch.arange(C, device="cuda")
    see = j <= last[..., None]
    if c["window"]:
        see &= j > last[..., None] - c["window"]
    see = see[:, None, :, None].expand(B, 1, N, R, C).reshape(B, 1, N * R, C)
    score = q @ k.transpose(-1, -2)
    score.masked_fill_(~see, -math.inf)
    top = score.amax(-1, keepdim=True)
    score.sub_(torch.where(top.isinf(), torch.zeros_like(top), top)).exp_()
    total = score.sum(-1, keepdim=True)
    o = (score @ v) / torch.where(total > 0, total, torch.ones_like(total))
    o = o.view(B, KV, N, R, D).permute(0, 2, 1, 3, 4).reshape(B, N, H * D)
    return o[b, i].to(torch.bfloat16)


_own = {"norm": _own_norm, "append": _own_append, "attend": _own_attend}
_plain = {"norm": _plain_norm, "append": _plain_append, "attend": _plain_attend}


# ------------------------------------------------------------------- exact ----

def exact(c, seed):
    s = prepare(c, seed)
    return {"norm": _exact_norm, "append": _exact_append, "attend": _exact_attend}[c["op"]](s, c)


def _exact_norm(s, c):
    out = {}
    h = s["x"].double()
    if c["res"]:
        h = (h + s["res"].double()).to(torch.bfloat16).double()
        out["h"] = h
    rms = ((h ** 2).sum(1) / c["width"] + EPS).sqrt()
    y = h / rms[:, None] * s["w"].double()
    out["y"] = y
    if c["eight"]:
        size = c["group"] or c["width"]
        parts = y.split(size, 1)
        out["scales"] = torch.stack([p.abs().max(1).values / 448 for p in parts], 1)
        out["y8"] = torch.cat([p / out["scales"][:, i:i + 1].clamp(min=1e-300) for i, p in enumerate(parts)], 1)
    return out


def _exact_append(s, c):
    H, KV, D, half = c["heads"], c["kv"], c["dim"], c["rot"] // 2
    T = s["rows"]
    x = s["qkv"].double().view(T, H + 2 * KV, D)
    rope = s["rope"].double()
    first = 0
    for a, n in enumerate(s["seg"]):             # every axis turns its own pairs
        i = torch.arange(first, first + n, device="cuda")
        z = torch.view_as_complex(rope[s["pos"][:, a].long()][:, first:first + n].contiguous())
        turned = torch.complex(x[:, :H + KV, i], x[:, :H + KV, i + half]) * z[:, None]
        x[:, :H + KV, i], x[:, :H + KV, i + half] = turned.real, turned.imag
        first += n
    out = {"q": x[:, :H].reshape(T, H * D)}
    for name, y in (("k", x[:, H:H + KV]), ("v", x[:, H + KV:])):
        y = y.reshape(T, -1, 64)
        low = y.min(2, keepdim=True).values
        step = ((y.max(2, keepdim=True).values - low) / 15).half().double()
        low = low.half().double()
        out[name] = (torch.round((y - low) / step.clamp(min=1e-30)).clamp(0, 15) * step + low).reshape(T, KV * D)
    return out


def _exact_attend(s, c):
    H, KV, D, page, W = c["heads"], c["kv"], c["dim"], c["page"], c["window"]
    q_lens, ctx = _lens(c)
    out = torch.zeros(s["rows"], KV, H // KV, D, device="cuda", dtype=torch.float64)
    shift = torch.arange(8, device="cuda", dtype=torch.int64) * 4
    t0 = 0
    for b, (n, m) in enumerate(zip(q_lens, ctx)):
        ids = s["table"][b, :-(-m // page)].long()
        j = torch.arange(m, device="cuda")
        i = torch.arange(n, device="cuda") + m - n
        hide = j[None] > i[:, None]
        if W:
            hide |= j[None] <= i[:, None] - W
        for h in range(KV):
            raw = s["pages"][ids, h].contiguous()
            words = raw[:, :page * D].contiguous().view(torch.int32).long() & 0xFFFFFFFF
            half16 = raw[:, page * D:].contiguous().view(torch.float16).double()
            kw = words[:, :page * D // 8].reshape(-1, 4, D // 32)
            k = torch.zeros(kw.shape[0], D, device="cuda", dtype=torch.float64)
            for t in range(4):
                for w in range(D // 32):
                    k[:, 32 * w + 8 * t:32 * w + 8 * t + 8] = ((kw[:, t, w, None] >> shift) & 15).double()
            vw = words[:, page * D // 8:].reshape(-1, D // 4)
            v = ((vw[..., None] >> shift) & 15).double()
            v = torch.stack([v[..., :4].flatten(1), v[..., 4:].flatten(1)], 1).reshape(-1, D)
            G = D // 64
            kp = half16[:, :page * G * 2].reshape(-1, G, 2).repeat_interleave(64, 1)
            vp = half16[:, page * G * 2:].reshape(-1, G, 2, 2).permute(0, 3, 1, 2).reshape(-1, G, 2).repeat_interleave(64, 1)
            k, v = (k * kp[..., 0] + kp[..., 1])[:m], (v * vp[..., 0] + vp[..., 1])[:m]
            q = s["q"][t0:t0 + n].double().view(n, KV, H // KV, D)[:, h].transpose(0, 1)             # [R][n][D]
            a = q @ k.T / math.sqrt(D)
            a.masked_fill_(hide, -math.inf)
            out[t0:t0 + n, h] = (torch.softmax(a, -1) @ v).transpose(0, 1)
            del a
        t0 += n
    return out.reshape(s["rows"], H * D)


# -------------------------------------------------------------------- work ----

def work(c):
    if c["op"] == "norm":
        T, W = c["rows"], c["width"]
        n = -(-W // c["group"]) if c["group"] else 1
        per = 2 + 2 + (4 if c["res"] else 0) + (1 if c["eight"] else 0)
        return {"bytes": T * W * per + 2 * W + (4 * T * n if c["eight"] else 0), "flops": 5 * T * W}
    H, KV, D = c["heads"], c["kv"], c["dim"]
    q, ctx = _lens(c)
    T = sum(q)
    token = KV * block_bytes(c["page"], D) // c["page"]
    if c["op"] == "append":
        # rows in, rotated q out, the cache's bytes, the values out; each row's table entries and positions
        return {"bytes": T * ((H + 2 * KV) * D * 2 + H * D * 2 + token + 2 * KV * D * 2 + c["rot"] * 4 + 4 * c["axes"]),
                "flops": T * ((H + KV) * c["rot"] * 3 + 2 * KV * D * 6)}
    pairs, seen = 0, 0
    for n, m in zip(q, ctx):
        w = c["window"] or m
        first = [max(0, m - n + i + 1 - w) for i in (0, n - 1)]
        seen += m - first[0]
        pairs += sum(min(w, m - n + i + 1) for i in range(n))
    return {"bytes": seen * token + 2 * T * H * D * 2, "flops": 4 * H * D * pairs}

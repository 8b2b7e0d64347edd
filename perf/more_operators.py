"""Cases and plain forms of the operators of drafted decoding over the 4-bit cache.

A serving step that verifies drafted tokens goes through four of them, measured one pass at a time:

  plan    lora_kv4_plan: from the rows that each request brings (none, a token, a
          tree of drafts, a prompt; -1: it has ended) the batch's row starts and
          lengths, pages for the new positions from a stack of free ones, pages of
          ended requests back to it, and for each row its request, rotary position
          and place in the cache.
  tree    lora_kv4_attend_tree: attention of the rows of a tree of drafted tokens:
          a row sees the cached context and those rows of its own request that its
          bits name (its ancestors and itself).
  logits  lora_logits_adjust: repetition, frequency and presence penalties by the
          request's tokens and the drafted ones on the row's path, biases, and a
          mask of the allowed tokens.
  keep    lora_kv4_keep: the cached positions of the accepted path of each tree move
          up to follow the context, in every layer's cache.

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


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # decode: one token in each of 64 requests, a page of 64 positions filled now and then
        {"name": "plan_decode", "op": "plan", "seqs": 64, "q_max": 1, "prompts": 0, "ended": 0.0, "ctx_max": 4096, "page": 64,
         "short": False, "lens": 11},
        # a mixed step: 16 prompts of up to 2048 tokens come in, some requests have ended, the others bring a token
        {"name": "plan_mixed", "op": "plan", "seqs": 256, "q_max": 1, "prompts": 16, "ended": 0.05, "ctx_max": 8192, "page": 64,
         "short": False, "lens": 12},
        # the most requests that a batch holds, a tree of up to 16 drafts each, small pages, too few of them left
        {"name": "plan_drafts", "op": "plan", "seqs": 4096, "q_max": 16, "prompts": 0, "ended": 0.02, "ctx_max": 2048, "page": 16,
         "short": True, "lens": 13},
        # one request alone, a small tree: latency
        {"name": "tree_one", "op": "tree", "seqs": 1, "q_min": 8, "q_max": 8, "ctx_min": 1003, "ctx_max": 1003,
         "heads": 32, "kv": 8, "dim": 128, "page": 64, "window": 0, "lens": 21},
        # a few drafts to a request, heads of 64, small pages
        {"name": "tree_few", "op": "tree", "seqs": 32, "q_min": 2, "q_max": 6, "ctx_min": 100, "ctx_max": 4096,
         "heads": 32, "kv": 8, "dim": 64, "page": 16, "window": 0, "lens": 22},
        # trees of 16 to 64 drafts in a sliding window, Mistral-7B-shaped heads
        {"name": "tree_window", "op": "tree", "seqs": 16, "q_min": 16, "q_max": 64, "ctx_min": 512, "ctx_max": 12000,
         "heads": 32, "kv": 8, "dim": 128, "page": 32, "window": 4096, "lens": 23},
        # full trees over long documents, 70B-shaped heads
        {"name": "tree_long", "op": "tree", "seqs": 8, "q_min": 64, "q_max": 64, "ctx_min": 32768, "ctx_max": 32768,
         "heads": 64, "kv": 8, "dim": 128, "page": 128, "window": 0, "lens": 24},
        # one token of one request, a small vocabulary, nothing masked
        {"name": "logits_token", "op": "logits", "seqs": 1, "q_min": 1, "q_max": 1, "vocab": 32000, "hist_max": 1000, "bias": 0,
         "masks": False, "drafts": False, "f32_in": False, "f32_out": False, "lens": 31},
        # a decode batch on its way to an fp32 sampler: penalties, biases, a grammar for most of the rows
        {"name": "logits_decode", "op": "logits", "seqs": 64, "q_min": 1, "q_max": 1, "vocab": 128256, "hist_max": 4096, "bias": 64,
         "masks": True, "drafts": False, "f32_in": False, "f32_out": True, "lens": 32},
        # trees of 32 drafts of 16 requests: each row's penalties by its own path
        {"name": "logits_tree", "op": "logits", "seqs": 16, "q_min": 32, "q_max": 32, "vocab": 128256, "hist_max": 8192, "bias": 16,
         "masks": True, "drafts": True, "f32_in": False, "f32_out": False, "lens": 33},
        # the accepted tokens of one request, 28 layers
        {"name": "keep_one", "op": "keep", "seqs": 1, "q_min": 16, "q_max": 16, "keep_max": 4, "ctx_max": 1000, "layers": 28,
         "kv": 8, "dim": 128, "page": 64, "lens": 41},
        # those of 64 requests, 32 layers
        {"name": "keep_batch", "op": "keep", "seqs": 64, "q_min": 16, "q_max": 64, "keep_max": 8, "ctx_max": 4096, "layers": 32,
         "kv": 8, "dim": 128, "page": 64, "lens": 42},
    ]


def _log(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["plan", "tree", "tree", "logits", "keep"])
    c = {"op": op, "lens": rng.randrange(1 << 30)}
    if op == "plan":
        seqs = _log(rng, 1, 4096)
        return c | {"seqs": seqs, "q_max": _log(rng, 1, max(1, min(64, 65536 // seqs))), "ctx_max": _log(rng, 1, 8192),
                    "prompts": rng.choice([0, 0, 1 + seqs // 20]) if seqs <= 256 else 0, "ended": rng.choice([0.0, 0.05, 0.5]),
                    "page": rng.choice([16, 32, 64, 128, 256]), "short": rng.random() < 0.25}
    if op == "keep":
        seqs, layers = _log(rng, 1, 64), rng.randint(1, 70)
        kv, dim = rng.choice([(8, 128), (8, 64), (4, 128), (2, 128), (1, 64)])
        return c | {"seqs": seqs, "layers": min(layers, max(1, 2048 // seqs)), "q_min": 1, "q_max": _log(rng, 1, 64), "keep_max": rng.randint(1, 8),
                    "ctx_max": _log(rng, 1, 8192), "kv": kv, "dim": dim, "page": rng.choice([16, 32, 64, 128, 256])}
    if op == "logits":
        vocab = _log(rng, 100, 262144)
        drafts = rng.random() < 0.4
        q_max = rng.randint(2, 64) if drafts else 1
        seqs = _log(rng, 1, max(1, min(256, 512 * 128256 // (vocab * q_max))))
        f32_in = rng.random() < 0.3
        return c | {"seqs": seqs, "q_min": rng.choice([1, q_max]), "q_max": q_max, "vocab": vocab, "hist_max": _log(rng, 1, 16384),
                    "bias": rng.choice([0, 3, 100, 300]), "masks": rng.random() < 0.6, "drafts": drafts, "f32_in": f32_in,
                    "f32_out": f32_in or rng.random() < 0.3}
    heads, kv, dim = rng.choice([(32, 8, 128), (24, 8, 128), (64, 8, 128), (32, 8, 64), (28, 4, 128), (16, 16, 64), (12, 1, 128)])
    seqs, q_max = _log(rng, 1, 64), _log(rng, 1, 64)
    most = 8 * 64 * 64 * 32768        # rows x heads x positions of the largest listed one
    ctx = _log(rng, 1, max(1, min(32768, most // (seqs * q_max * heads), 8 * 8 * 32768 // (seqs * kv))))
    return c | {"seqs": seqs, "q_min": rng.choice([1, q_max]), "q_max": q_max, "ctx_min": rng.choice([0, ctx]), "ctx_max": ctx,
                "heads": heads, "kv": kv, "dim": dim, "page": rng.choice([16, 32, 64, 128, 256]),
                "window": rng.choice([0, 0, 0, _log(rng, 16, 4096)])}


def _lens(c):
    """Of a case's requests: (rows that they bring, positions cached before, further number), by its kind."""
    r = random.Random(c["lens"])
    n, log = c["seqs"], lambda lo, hi: _log(r, lo, hi) if hi > 0 else 0  # noqa: E731
    if c["op"] == "plan":
        q = [-1 if r.random() < c["ended"] else c["q_max"] if c["q_max"] == 1 else r.randint(0, c["q_max"]) for _ in range(n)]
        ctx = [log(1, c["ctx_max"]) for _ in range(n)]
        for i in r.sample(range(n), c["prompts"]):
            q[i], ctx[i] = r.randint(64, 2048), 0
        return q, ctx, [r.randint(0, 1) for _ in range(n)]        # a page more than its positions need, as after rejected drafts
    if c["op"] == "logits":
        q = [r.randint(c["q_min"], c["q_max"]) for _ in range(n)]
        hist = [log(1, c["hist_max"]) for _ in range(n)]
        return q, hist, [r.randint(0, h) for h in hist]           # tokens, and of these the prompt's
    q = [r.randint(c["q_min"], c["q_max"]) for _ in range(n)]
    if c["op"] == "keep":
        return q, [log(1, c["ctx_max"]) for _ in range(n)], [r.randint(1, max(1, min(c["keep_max"], (m + 1) // 2))) for m in q]
    lo, hi = c["ctx_min"], c["ctx_max"]
    return q, [lo if lo == hi else min(hi, lo - 1 + log(1, hi - lo + 1)) for _ in range(n)], None


def block_bytes(page, dim):
    return page * (dim + dim // 64 * 8)


# ------------------------------------------------------------------- state ----

def _trees(r, q):
    """Parent of every row of each request's tree, in breadth-first order, a fifth of them chains."""
    all_parents = []
    for n in q:
        p = [-1] * n
        chain = r.random() < 0.2
        for i in range(1, n):
            p[i] = i - 1 if chain else min(i - 1, max(p[i - 1], 0) + (r.random() < 0.4 and i > 2))
        all_parents.append(p)
    return all_parents


def _tree_bits(parents, words):
    """int32 [rows][words]: bit j of a row: it sees row j of its request."""
    rows = []
    for p in parents:
        own_bits = []
        for i, up in enumerate(p):
            own_bits.append((own_bits[up] if up >= 0 else 0) | 1 << i)
        rows += own_bits
    full = np.array([[b >> 32 * w & 0xFFFFFFFF for w in range(words)] for b in rows], np.uint32).reshape(len(rows), words)
    return torch.from_numpy(full.view(np.int32)).cuda()


def _depths(parents):
    out = []
    for p in parents:
        d = []
        for up in p:
            d.append(d[up] + 1 if up >= 0 else 0)
        out += d
    return out


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def prepare(c, seed):
    g = torch.Generator(device="cuda").manual_seed(1000003 * seed + 29)
    r = random.Random(seed * 37 + c["lens"])
    s = {"c": c}
    q, ctx, more = _lens(c)
    if c["op"] == "plan":
        page, n = c["page"], len(q)
        held = [-(-m // page) + (e if m else 0) for m, e in zip(ctx, more)]
        total = [m + max(0, k) for m, k in zip(ctx, q)]
        need = sum(max(0, -(-t // page) - h) for t, h, k in zip(total, held, q) if k > 0)
        freed = sum(h for h, k in zip(held, q) if k < 0)
        spare = max(0, need // 2 - freed) if c["short"] else need + n // 4 + 3
        ids = list(range(sum(held) + spare))
        r.shuffle(ids)
        s["max_ctx"], s["max_q"], s["rows"] = max(max(total), 1), max(1, max(q)), max(1, sum(max(0, k) for k in q))
        wide = max(-(-s["max_ctx"] // page), max(held))
        table = np.full((n, wide), -1, np.int32)
        at = 0
        for i, h in enumerate(held):
            table[i, :h] = ids[at:at + h]
            at += h
        s |= {"table": _i32(table), "held": _i32(held), "free": _i32(ids[at:] + [-1] * at), "n_free": _i32([spare]), "q": _i32(q), "ctx": _i32(ctx)}
        rows = [max(0, k) for k in q]
        trees = _trees(r, rows) if 1 < c["q_max"] and not c["prompts"] else [range(-1, k - 1) for k in rows]
        s["depths"] = _i32(_depths(trees) or [0])
        if own:   # the plan that a serving program keeps; its counters' results go to arrays of their own
            from lora_serving_gb300 import store
            s["plan"] = store.KV4Plan(s["free"], s["n_free"], s["held"], s["table"], page_size=page, max_rows=s["rows"], max_q_len=s["max_q"],
                                      max_ctx_len=s["max_ctx"], n_free_out=torch.zeros_like(s["n_free"]), held_out=torch.zeros_like(s["held"]))
        return s
    T = sum(q)
    starts = np.concatenate([[0], np.cumsum(q)])
    s |= {"starts": _i32(starts), "rows": T, "max_q": max(q)}
    if c["op"] == "logits":
        V, n = c["vocab"], c["seqs"]
        kind = torch.float32 if c["f32_in"] else torch.bfloat16
        s["logits"] = (3 * torch.randn(T, -(-V // 8) * 8, generator=g, device="cuda")).to(kind)[:, :V]
        s["out"] = torch.empty(T, -(-V // 8) * 8, dtype=torch.float32 if c["f32_out"] else torch.bfloat16, device="cuda")[:, :V]
        often = lambda *size: (V * torch.rand(size, generator=g, device="cuda") ** 3).to(torch.int32).clamp(max=V - 1)  # noqa: E731
        s["tokens"] = often(n, max(ctx))                        # what stands past a request's tokens is not looked at
        s |= {"len": _i32(ctx), "prompt": _i32(more)}
        f = lambda lo, hi: (lo + (hi - lo) * torch.rand(n, generator=g, device="cuda")) * 1.0  # noqa: E731
        s |= {"rep": f(1.0, 1.3), "freq": f(0.0, 0.5), "pres": f(0.0, 0.5)}
        s["rep"][::4] = 1.0                                     # requests without penalties
        s["freq"][::4] = s["pres"][::4] = 0.0
        s["bias_ids"] = torch.randint(0, V, (n, c["bias"]), generator=g, device="cuda", dtype=torch.int32) if c["bias"] else None
        s["bias"] = 5 * torch.randn(n, c["bias"], generator=g, device="cuda") if c["bias"] else None
        s["n_bias"] = _i32([r.randint(0, c["bias"]) for _ in q]) if c["bias"] else None
        s["row_seq"] = _i32(np.repeat(np.arange(n), q))
        s["drafts"] = s["tree"] = None
        if c["drafts"]:
            parents = _trees(r, q)
            s["up"] = parents
            s["drafts"], s["tree"] = often(T), _tree_bits(parents, -(-max(q) // 32))
        s["allowed"] = s["allowed_rows"] = None
        if c["masks"]:    # grammars that leave a few tokens, about half, or nearly all, one set to a request; a quarter of the rows has none
            kinds = torch.randint(0, 3, (n, 1), generator=g, device="cuda")
            bits = [torch.randint(0, 256, (n, -(-V // 32) * 4), generator=g, device="cuda", dtype=torch.uint8) for _ in range(4)]
            few, most = bits[0] & bits[1] & bits[2] & bits[3], bits[0] | bits[1] | bits[2] | bits[3]
            s["allowed"] = torch.where(kinds == 0, few, torch.where(kinds == 1, bits[0], most)).view(torch.int32)
            s["allowed_rows"] = _i32([-1 if r.random() < 0.25 else i for i, k in enumerate(q) for _ in range(k)])
        if own:
            from lora_serving_gb300 import store
            s["rules"] = store.LogitsRules(s["tokens"], s["prompt"], s["len"], repetition=s["rep"], frequency=s["freq"], presence=s["pres"],
                                           bias_ids=s["bias_ids"], bias=s["bias"], n_bias=s["n_bias"])
        return s
    KV, D, page = c["kv"], c["dim"], c["page"]
    total = [a + b for a, b in zip(ctx, q)]
    first = [m // page if c["op"] == "keep" else 0 for m in ctx]     # a move touches the tree's own pages alone
    pages = [-(-t // page) - f for t, f in zip(total, first)]
    ids = list(range(sum(pages) + 2))
    r.shuffle(ids)
    table = np.full((len(q), max(f + n for f, n in zip(first, pages))), -1, np.int32)
    at = 0
    for i, (f, n) in enumerate(zip(first, pages)):
        table[i, f:f + n] = ids[at:at + n]
        at += n
    s |= {"table": _i32(table), "ctx": _i32(total), "max_ctx": max(total)}
    nb, G = len(ids), D // 64
    if c["op"] == "keep":
        s["pages"] = torch.randint(0, 256, (c["layers"], nb, KV, block_bytes(page, D)), generator=g, device="cuda", dtype=torch.uint8)
        path = np.full((len(q), c["keep_max"]), -1, np.int32)
        for i, (n, k) in enumerate(zip(q, more)):
            # the root, then rows that no kept one takes the place of (a pass over the same state then gives the same again)
            path[i, :k] = [0] + sorted(r.sample(range(k, n), k - 1))
        s |= {"path": _i32(path), "n_keep": _i32(more), "len": _i32(np.zeros(len(q)))}
    else:
        # what an append leaves: codes that lie in a bell over 0..15, steps that vary by token and group
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
        s["q"] = (2 * torch.randn(T, c["heads"] * D, generator=g, device="cuda")).to(torch.bfloat16)
        s["out"] = torch.empty_like(s["q"])
        s["up"] = _trees(r, q)
        s["tree"] = _tree_bits(s["up"], -(-max(q) // 32))
    if own:   # the handles that a serving program keeps: its caches, this step's batch, a workspace
        from lora_serving_gb300 import store
        s["batch"] = store.KV4Batch(s["starts"], s["ctx"], s["table"], n_rows=T, max_q_len=s["max_q"], max_ctx_len=s["max_ctx"])
        if c["op"] == "keep":
            s["layers"] = store.KV4Layers([store.KV4Cache(nb, page, KV, D, pages=p) for p in s["pages"]])
        else:
            s["cache"] = store.KV4Cache(nb, page, KV, D, pages=s["pages"])
            s["ws"] = store.kv4_workspace(s["cache"], c["heads"], s["batch"])
    return s


# --------------------------------------------------------------------- run ----

def run(s):
    c = s["c"]
    return (_own if own else _plain)[c["op"]](s, c)


def _own_plan(s, c):
    from lora_serving_gb300 import abi
    p = s["plan"]
    abi.lora_kv4_plan(p, s["q"], s["ctx"], depths=s["depths"])
    return {"starts": p.q_starts, "ctx": p.ctx_lens, "table": p.block_table, "held": p.held_out, "free": p.free_pages, "n_free": p.n_free_out,
            "row_seq": p.row_seq, "positions": p.positions, "slots": p.slots}


def _own_tree(s, c):
    from lora_serving_gb300 import abi
    abi.lora_kv4_attend_tree(s["out"], s["q"], s["cache"], s["batch"], s["tree"], s["ws"], n_heads=c["heads"], scale=1.0 / math.sqrt(c["dim"]),
                             window=c["window"])
    return s["out"]


def _own_logits(s, c):
    from lora_serving_gb300 import abi
    abi.lora_logits_adjust(s["out"], s["logits"], s["rules"], row_seq=s["row_seq"], drafts=s["drafts"], tree=s["tree"],
                           q_starts=s["starts"] if c["drafts"] else None, allowed=s["allowed"], allowed_rows=s["allowed_rows"])
    return s["out"]


def _own_keep(s, c):
    from lora_serving_gb300 import abi
    abi.lora_kv4_keep(s["layers"], s["batch"], s["n_keep"], s["path"], lens=s["len"])
    return {"pages": s["pages"], "lens": s["len"]}


def _plain_plan(s, c):
    q, ctx, held, table, page = s["q"].long(), s["ctx"].long(), s["held"].long(), s["table"], c["page"]
    n, wide = table.shape
    ended, rows = q < 0, q.clamp(min=0)
    ends = rows.cumsum(0)
    total = torch.where(ended, 0, ctx + rows)
    fits = ~ended & (rows <= s["max_q"]) & (total <= s["max_ctx"]) & (ends <= s["rows"])
    need = torch.where(fits & (rows > 0), ((total + page - 1) // page - held).clamp(min=0), 0)
    col = torch.arange(wide, device="cuda")
    # pages of ended requests onto the stack, in the order of the table
    back = torch.where(ended, held, 0)
    given = ended[:, None] & (col < held[:, None])
    place = s["n_free"] + (back.cumsum(0) - back)[:, None] + col
    free = s["free"].clone()
    free[place[given]] = table[given]
    there = s["n_free"] + back.sum()
    got = fits & ((need == 0) | (need.cumsum(0) <= there))
    take = torch.where(got, need, 0)
    new = (col >= held[:, None]) & (col < (held + take)[:, None])
    at = there - 1 - ((need.cumsum(0) - need)[:, None] + col - held[:, None])
    table = torch.where(new, free[at.clamp(0, free.numel() - 1)], table)
    # rows
    t = torch.arange(s["rows"], device="cuda")
    seq = torch.searchsorted(ends, t, right=True)
    live = seq < n
    seq = seq.clamp(max=n - 1)
    live = live & got[seq]
    i = t - (ends - rows)[seq]
    pos = ctx[seq] + i
    page_id = table[seq, (pos // page).clamp(max=wide - 1)].long()
    return {"starts": torch.cat([ends.new_zeros(1), ends]).clamp(max=s["rows"]).int(), "ctx": torch.where(got, total, 0).int(), "table": table,
            "held": torch.where(ended, 0, held + take).int(), "free": free, "n_free": (there - take.sum()).int(),
            "row_seq": torch.where(live, seq, -1).int(), "positions": torch.where(live, ctx[seq] + s["depths"], -1).int()[:, None],
            "slots": torch.where(live, page_id * page + pos % page, -1)}


def _bits(words, at):
    """Bit `at` (last dimension, 0 or more) of rows of 32-bit words, as truth values."""
    w = words.long()
    return torch.gather(w, -1, (at >> 5).clamp(max=w.shape[-1] - 1)) >> (at & 31) & 1 > 0


def _plain_tree(s, c):
    H, KV, D, page, W = c["heads"], c["kv"], c["dim"], c["page"], c["window"]
    R, G, n_seqs = H // KV, D // 64, c["seqs"]
    pages = s["pages"][s["table"].long().clamp(min=0)]                                                     # [seq][page][kv][block]
    shift = 4 * torch.arange(8, device="cuda", dtype=torch.int32)
    kw = pages[..., :page * D // 2].contiguous().view(torch.int32).view(*pages.shape[:3], page, 4, D // 32, 1)
    vw = pages[..., page * D // 2:page * D].contiguous().view(torch.int32).view(*pages.shape[:3], page // 2, D // 4, 1)
    kp = pages[..., page * D:page * (D + 4 * G)].contiguous().view(torch.float16).float().view(*pages.shape[:3], page, G, 1, 2)
    vp = pages[..., page * (D + 4 * G):].contiguous().view(torch.float16).float().view(*pages.shape[:3], page // 2, G, 2, 2)
    k = (kw >> shift & 15).transpose(-3, -2).reshape(*pages.shape[:3], page, G, 64).float()
    k = k * kp[..., 0] + kp[..., 1]
    v = (vw >> shift & 15).unflatten(-1, (2, 4)).permute(0, 1, 2, 3, 5, 4, 6).reshape(*pages.shape[:3], page // 2, 2, G, 64).float()
    v = v * vp[..., 0, :].transpose(-1, -2)[..., None] + vp[..., 1, :].transpose(-1, -2)[..., None]        # [pair][parity][G][64]
    k, v = (x.reshape(*pages.shape[:3], page, D).transpose(1, 2).reshape(n_seqs, KV, -1, D) for x in (k, v))
    n = (s["starts"][1:] - s["starts"][:-1]).long()
    base, i = s["ctx"].long() - n, torch.arange(s["max_q"], device="cuda")
    row = (s["starts"][:-1, None] + i).clamp(max=s["rows"] - 1)                                            # [seq][row]
    q = s["q"].float()[row].view(n_seqs, -1, KV, R, D).permute(0, 2, 1, 3, 4).reshape(n_seqs, KV, -1, D)
    j = torch.arange(k.shape[2], device="cuda") - base[:, None]                                            # places counted from the tree's first
    bits = s["tree"][row]
    tree = _bits(bits, (j[:, None] + 0 * i[:, None]).clamp(min=0)) & (j >= 0)[:, None] & (j < n[:, None])[:, None]
    sees = tree | (j < 0)[:, None]
    if W:
        depth = _bits(bits, i.expand(n_seqs, s["max_q"], -1).contiguous()).sum(-1).clamp(min=1) - 1
        sees &= tree | (j[:, None] > depth[..., None] - W)
    hide = ~sees[:, None, :, None, :].expand(-1, 1, -1, R, -1).reshape(n_seqs, 1, -1, j.shape[1])
    a = (q @ k.transpose(-1, -2)) * (1.0 / math.sqrt(D))
    a = a.masked_fill_(hide, -math.inf)
    a = torch.exp(a - a.amax(-1, keepdim=True))
    out = (a @ v) / a.sum(-1, keepdim=True)
    out = out.view(n_seqs, KV, -1, R, D).permute(0, 2, 1, 3, 4).reshape(n_seqs, s["max_q"], H * D)
    return out[i < n[:, None]].to(torch.bfloat16)


def _plain_logits(s, c):
    V, T, seq = c["vocab"], s["rows"], s["row_seq"].long()
    x = s["logits"].float()
    j = torch.arange(s["tokens"].shape[1], device="cuda")
    ids = torch.where(j < s["len"][:, None], s["tokens"], V).long()                 # column V: nothing
    ids_out = torch.where(j >= s["prompt"][:, None], ids, V)
    zeros = lambda n: torch.zeros(n, V + 1, dtype=torch.int32, device="cuda")  # noqa: E731
    every = zeros(c["seqs"]).scatter_add_(1, ids, torch.ones_like(ids, dtype=torch.int32))[seq]
    made = zeros(c["seqs"]).scatter_add_(1, ids_out, torch.ones_like(ids, dtype=torch.int32))[seq]
    if c["drafts"]:
        i = torch.arange(s["max_q"], device="cuda").expand(T, -1).contiguous()
        on = _bits(s["tree"], i)
        path = s["drafts"].long()[(s["starts"][:-1].long()[seq][:, None] + i).clamp(max=T - 1)]
        every.scatter_add_(1, path, on.int())
        made.scatter_add_(1, path, on.int())
    every, made = every[:, :V], made[:, :V].float()
    rep, freq, pres = (s[k][seq][:, None] for k in ("rep", "freq", "pres"))
    x = torch.where(every > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - freq * made - pres * (made > 0)
    if c["bias"]:
        e = torch.arange(c["bias"], device="cuda").expand(c["seqs"], -1)
        last = torch.full((c["seqs"], V + 1), -1, device="cuda", dtype=torch.int64)
        last.scatter_reduce_(1, torch.where(e < s["n_bias"][:, None], s["bias_ids"], V).long(), e, "amax")   # of a token's entries the last counts
        last = last[:, :V]
        x = x + torch.where(last >= 0, s["bias"].gather(1, last.clamp(min=0)), 0.0)[seq]
    if c["masks"]:
        m = s["allowed_rows"].long()
        v = torch.arange(V, device="cuda")
        x = x.masked_fill((s["allowed"].long()[:, v >> 5] >> (v & 31) & 1 == 0)[m.clamp(min=0)] & (m >= 0)[:, None], -math.inf)
    return x.to(s["out"].dtype)


def _plain_keep(s, c):
    KV, D, page = c["kv"], c["dim"], c["page"]
    G, pages = D // 64, s["pages"]
    n = s["starts"][1:] - s["starts"][:-1]
    base = (s["ctx"] - n).long()
    i = torch.arange(c["keep_max"], device="cuda")
    seq, i = torch.nonzero(i < s["n_keep"][:, None], as_tuple=True)
    src, dst = base[seq] + s["path"][seq, i], base[seq] + i
    sp, dp = s["table"][seq, src // page].long(), s["table"][seq, dst // page].long()
    so, do = src % page, dst % page
    cut = lambda a, b, *shape: pages[..., a:b].unflatten(-1, shape)  # noqa: E731
    k, kp = cut(0, page * D // 2, page, D // 2), cut(page * D, page * (D + 4 * G), page, 4 * G)
    v = cut(page * D // 2, page * D, page // 2, D // 4, 2, 2)                             # a word's halves: the even position, the odd one
    vp = cut(page * (D + 4 * G), page * (D + 8 * G), page // 2, G, 2, 2, 2)               # steps and lowest values, even and odd
    moved = [k[:, sp, :, so], kp[:, sp, :, so], v[:, sp, :, so // 2, :, so % 2], vp[:, sp, :, so // 2, :, :, so % 2]]
    k[:, dp, :, do], kp[:, dp, :, do], v[:, dp, :, do // 2, :, do % 2], vp[:, dp, :, do // 2, :, :, do % 2] = moved
    s["len"].copy_(base + s["n_keep"])
    return {"pages": pages, "lens": s["len"]}


_plain = {"plan": _plain_plan, "tree": _plain_tree, "logits": _plain_logits, "keep": _plain_keep}
_own = {"plan": _own_plan, "tree": _own_tree, "logits": _own_logits, "keep": _own_keep}


# ------------------------------------------------------------------- exact ----

def exact(c, seed):
    s = prepare(c, seed)
    return {"plan": _exact_plan, "tree": _exact_tree, "logits": _exact_logits, "keep": _exact_keep}[c["op"]](s, c)


def _exact_plan(s, c):
    h = lambda k: s[k].cpu().numpy().astype(np.int64)  # noqa: E731
    q, ctx, held, table, free, depths = h("q"), h("ctx"), h("held"), h("table"), h("free"), h("depths")
    n_free, page, n = int(h("n_free")[0]), c["page"], len(q)
    for i in np.flatnonzero(q < 0):
        free[n_free:n_free + held[i]] = table[i, :held[i]]
        n_free += int(held[i])
        held[i] = 0
    starts, out_ctx, at, asked, top = [0], [], 0, 0, n_free
    row_seq, pos, slots = (np.full(s["rows"], -1, np.int64) for _ in range(3))
    for i in range(n):
        m = max(0, int(q[i]))
        total = int(ctx[i]) + m
        ok = q[i] >= 0 and total <= s["max_ctx"] and m <= s["max_q"] and at + m <= s["rows"]
        need = max(0, -(-total // page) - int(held[i])) if ok and m else 0
        asked += need
        ok = ok and (need == 0 or asked <= top)
        if ok and need:
            table[i, held[i]:held[i] + need] = free[top - asked:top - asked + need][::-1]
            held[i] += need
            n_free -= need
        for j in range(m if ok else 0):
            p = int(ctx[i]) + j
            row_seq[at + j], pos[at + j], slots[at + j] = i, ctx[i] + depths[at + j], table[i, p // page] * page + p % page
        out_ctx.append(total if ok else 0)
        at += m
        starts.append(min(at, s["rows"]))
    up = lambda a: torch.from_numpy(np.asarray(a)).cuda()  # noqa: E731
    return {"starts": up(starts).int(), "ctx": up(out_ctx).int(), "table": up(table).int(), "held": up(held).int(), "free": up(free).int(),
            "n_free": up([n_free]).int(), "row_seq": up(row_seq).int(), "positions": up(pos).int()[:, None], "slots": up(slots)}


def _exact_tree(s, c):
    H, KV, D, page, W = c["heads"], c["kv"], c["dim"], c["page"], c["window"]
    q_lens, ctx, _ = _lens(c)
    out = torch.zeros(s["rows"], KV, H // KV, D, device="cuda", dtype=torch.float64)
    shift = torch.arange(8, device="cuda", dtype=torch.int64) * 4
    t0 = 0
    for b, (n, m) in enumerate(zip(q_lens, ctx)):
        ids = s["table"][b, :-(-(m + n) // page)].long()
        sees = np.zeros((n, m + n), bool)
        for i in range(n):              # up the tree from every row
            at, depth = i, 0
            while at >= 0:
                sees[i, m + at] = True
                at, depth = s["up"][b][at], depth + 1
            sees[i, max(0, m + depth - W) if W else 0:m] = True
        hide = torch.from_numpy(~sees).cuda()
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
            k, v = (k * kp[..., 0] + kp[..., 1])[:m + n], (v * vp[..., 0] + vp[..., 1])[:m + n]
            q = s["q"][t0:t0 + n].double().view(n, KV, H // KV, D)[:, h].transpose(0, 1)             # [R][n][D]
            a = (q @ k.T / math.sqrt(D)).masked_fill_(hide, -math.inf)
            out[t0:t0 + n, h] = (torch.softmax(a, -1) @ v).transpose(0, 1)
            del a
        t0 += n
    return out.reshape(s["rows"], H * D)


def _exact_logits(s, c):
    V, n = c["vocab"], c["seqs"]
    q, hist, prompt = _lens(c)
    x = s["logits"].double().clone()
    t = 0
    drafts = s["drafts"].tolist() if c["drafts"] else None
    rows = s["allowed_rows"].tolist() if c["masks"] else None
    rep, freq, pres = (s[k].double().tolist() for k in ("rep", "freq", "pres"))
    for b in range(n):
        tok = s["tokens"][b, :hist[b]].long()
        made0, all0 = torch.bincount(tok[prompt[b]:], minlength=V), torch.bincount(tok, minlength=V)
        bias = torch.zeros(V, device="cuda", dtype=torch.float64)
        if c["bias"]:
            k = int(s["n_bias"][b])
            table = dict(zip(s["bias_ids"][b, :k].tolist(), s["bias"][b, :k].double().tolist()))
            if table:
                bias[torch.tensor(list(table), device="cuda")] = torch.tensor(list(table.values()), device="cuda", dtype=torch.float64)
        for i in range(q[b]):
            made, seen = made0, all0
            if c["drafts"]:
                at, path = i, []
                while at >= 0:
                    path.append(drafts[t - i + at])
                    at = s["up"][b][at]
                extra = torch.bincount(torch.tensor(path, device="cuda"), minlength=V)
                made, seen = made0 + extra, all0 + extra
            y = x[t]
            hit = seen > 0
            y[hit] = torch.where(y[hit] < 0, y[hit] * rep[b], y[hit] / rep[b])
            y -= made * freq[b]
            y[made > 0] -= pres[b]
            y += bias
            if c["masks"] and rows[t] >= 0:
                word = s["allowed"][rows[t]].contiguous().view(torch.uint8)
                bit = (word[:, None] >> torch.arange(8, device="cuda", dtype=torch.uint8) & 1).flatten()[:V]
                y[bit == 0] = -math.inf
            t += 1
    return x


def _exact_keep(s, c):
    D, page, G = c["dim"], c["page"], c["dim"] // 64
    h = s["pages"].cpu().numpy().copy()
    table, path = s["table"].cpu().numpy(), s["path"].cpu().numpy()
    q, ctx, keep = _lens(c)
    for b in range(c["seqs"]):
        for i in range(keep[b]):
            (sp, so), (dp, do) = divmod(ctx[b] + int(path[b, i]), page), divmod(ctx[b] + i, page)
            of = [np.concatenate([np.arange(o * D // 2, (o + 1) * D // 2),
                                  page * D // 2 + o // 2 * D + 4 * np.arange(D // 4) + 2 * (o % 2),
                                  page * D // 2 + o // 2 * D + 4 * np.arange(D // 4) + 2 * (o % 2) + 1,
                                  np.arange(page * D + 4 * G * o, page * D + 4 * G * (o + 1)),
                                  *[page * (D + 4 * G) + (o // 2 * G + g) * 8 + 2 * (o % 2) + np.array([0, 1, 4, 5]) for g in range(G)]])
                  for o in (so, do)]
            h[:, table[b, dp], :, of[1]] = h[:, table[b, sp], :, of[0]]
    return {"pages": torch.from_numpy(h).cuda(), "lens": _i32([a + b for a, b in zip(ctx, keep)])}


# -------------------------------------------------------------------- work ----

def work(c):
    q, ctx, more = _lens(c)
    n, T = len(q), sum(max(0, k) for k in q)
    if c["op"] == "plan":
        page = c["page"]
        held = [-(-m // page) + (e if m else 0) for m, e in zip(ctx, more)]
        new = sum(max(0, -(-(m + k) // page) - h) for m, k, h in zip(ctx, q, held) if k > 0)
        back = sum(h for h, k in zip(held, q) if k < 0)
        # lengths in, starts and lengths out; a page's id from the stack to the table or back; a row's depth, and its request, position and place
        return {"bytes": 24 * n + 8 * (new + back) + 20 * T, "flops": 0}
    if c["op"] == "logits":
        V = c["vocab"]
        per = (4 if c["f32_in"] else 2) + (4 if c["f32_out"] else 2)
        return {"bytes": T * V * per + 4 * sum(ctx) + (n * V // 8 if c["masks"] else 0) + 8 * n * c["bias"] // 2 + 12 * n, "flops": 6 * T * V}
    KV, D = c["kv"], c["dim"]
    token = KV * block_bytes(c["page"], D) // c["page"]
    if c["op"] == "keep":
        return {"bytes": c["layers"] * 2 * token * sum(k - 1 for k in more) + 8 * n, "flops": 0} if sum(more) > n else {"bytes": 12 * n, "flops": 0}
    seen = sum(k + min(m, c["window"] or m) for k, m in zip(q, ctx))
    pairs = sum(k * (1 + min(m, c["window"] or m)) for k, m in zip(q, ctx))
    return {"bytes": seen * token + 2 * T * c["heads"] * D * 2, "flops": 4 * c["heads"] * D * pairs}

"""The attention half of a transformer layer for requests with LoRA adapters,
from the library's operators:

    h, x    = rms_norm(x + residual)            lora_rms_norm
    q, k, v = x W_qkv^T + B(A x)                lora_linear, each row its adapter
    q', k'  = rotary(q, k); cache += k', v      lora_kv4_append (4-bit pages)
    o       = attention(q', cache)              lora_kv4_attend
    y       = o W_o^T + B(A o)                  lora_linear

Prompts of several requests go through it in one batch, then tokens one at a
time, the cache growing page by page.  Run as a script it prints the time of
a step of each kind and how far the step-by-step outputs are from those of
one pass over the whole sequences.

    python examples/attention_block.py [--hidden 2048 --heads 16 --kv 4]
"""
from __future__ import annotations

import argparse
import math
import os
import sys

import numpy as np
import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

from lora_serving_gb300 import abi, build, store  # noqa: E402


class AttentionBlock:
    """One layer's weights, adapters and cache."""

    def __init__(self, hidden, heads, kv, dim, n_slots, rank, n_pages, page=64, max_pos=4096, seed=0, device="cuda"):
        g = torch.Generator().manual_seed(seed)
        rnd = lambda *s, k=1.0: (torch.randn(*s, generator=g) * k).to(torch.bfloat16)  # noqa: E731
        bits = lambda t: t.view(torch.int16).numpy().view(np.uint16)  # noqa: E731
        self.hidden, self.heads, self.kv, self.dim = hidden, heads, kv, dim
        self.norm_w = (1 + rnd(hidden, k=0.1)).to(device)
        wq, wk = heads * dim, kv * dim
        self.qkv = store.GroupStore(hidden, [("q", wq), ("k", wk), ("v", wk)], n_slots, rank, device)
        self.o = store.GroupStore(wq, [("o", hidden)], n_slots, rank, device)
        for st in (self.qkv, self.o):
            st.load_slots({k: [(bits(rnd(rank, st.h_in, k=0.02)), bits(rnd(w, rank, k=0.02)), 2.0 * rank, False)
                               for _, w in st.projs] for k in range(n_slots)})
        self.W_qkv = rnd(wq + 2 * wk, hidden, k=hidden ** -0.5).to(device)
        self.W_o = rnd(hidden, wq, k=wq ** -0.5).to(device)
        self.cache = store.KV4Cache(n_pages, page, kv, dim, device)
        self.rope = store.rope_table(max_pos, dim // 2, device=device)
        self.status = torch.zeros(1, dtype=torch.int32, device=device)

    def __call__(self, x, residual, ids, n_prefill, batch, base8=False):
        """x, residual [rows][hidden] bf16; ids: adapter slot of each row (-1:
        none), prefill rows first; batch: store.KV4Batch.  Returns (y, h) or,
        with base8, also the norm's 8-bit output and scales, what a base
        product in 8 bits would take."""
        T, D = x.shape[0], self.dim
        new = lambda cols, dtype=torch.bfloat16: torch.empty(T, cols, dtype=dtype, device=x.device)  # noqa: E731
        meta = store.BatchMeta(ids, n_prefill, self.qkv.n_slots, x.device)
        n, h = new(self.hidden), new(self.hidden)
        y8 = new(self.hidden, torch.float8_e4m3fn) if base8 else None
        scales = new(-(-self.hidden // 128), torch.float32) if base8 else None
        abi.lora_rms_norm(x, self.norm_w, 1e-5, residual=residual, residual_out=h, y=n, y8=y8, scales=scales,
                          group=128)
        qkv = new(self.qkv.ld_y)
        ws = store.workspace_for(T, 3, self.qkv.r_slot, x.device)
        store.linear(qkv, n, self.W_qkv, self.qkv, meta, ws, dev_status=self.status)
        wq, wk = self.heads * D, self.kv * D
        q = new(wq)
        abi.lora_kv4_append(q, qkv, self.cache, batch, n_heads=self.heads, q_off=0, k_off=wq, v_off=wq + wk,
                            rope=self.rope, dev_status=self.status)
        o = q   # attention may write over its queries
        abi.lora_kv4_attend(o, q, self.cache, batch, store.kv4_workspace(self.cache, self.heads, batch, x.device),
                            n_heads=self.heads, scale=1 / math.sqrt(D), dev_status=self.status)
        y = new(self.hidden)
        store.linear(y, o, self.W_o, self.o, meta, store.workspace_for(T, 1, self.o.r_slot, x.device),
                     dev_status=self.status)
        return (y, h, y8, scales) if base8 else (y, h)


def run(hidden=2048, heads=16, kv=4, dim=128, prompts=(700, 90, 333), steps=20, page=64, seed=0, say=print):
    """Prompts, then `steps` single tokens of each request; the same rows in
    one pass over a second cache.  Returns the relative difference of the
    single tokens' outputs."""
    dev = torch.device("cuda")
    rng = np.random.default_rng(seed)
    n = len(prompts)
    pages = [-(-(p + steps) // page) for p in prompts]
    order = rng.permutation(2 * sum(pages))
    table = np.full((2, n, max(pages)), -1, np.int32)                # one table for each of the two runs
    at = 0
    for run_i in range(2):
        for s in range(n):
            table[run_i, s, :pages[s]] = order[at:at + pages[s]]
            at += pages[s]
    block = AttentionBlock(hidden, heads, kv, dim, n_slots=4, rank=16, n_pages=2 * sum(pages), page=page, seed=seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    rows = [torch.randn(2, p + steps, hidden, generator=g, device=dev).to(torch.bfloat16) for p in prompts]   # x, residual
    slots = np.array([s % 4 - (s == 1) * 2 for s in range(n)], np.int32)                                       # the second request: base model
    cat = lambda parts: [torch.cat([r[i] for r in parts]) for i in (0, 1)]  # noqa: E731
    ev = lambda: torch.cuda.Event(enable_timing=True)  # noqa: E731

    # ---- prompts, then one token of every request at a time
    block(*cat([r[:, :p] for r, p in zip(rows, prompts)]), np.repeat(slots, prompts), sum(prompts),
          store.KV4Batch.from_lens(prompts, prompts, table[0]))
    outs, times = [], []
    for i in range(steps):
        x, res = cat([r[:, p + i:p + i + 1] for r, p in zip(rows, prompts)])
        batch = store.KV4Batch.from_lens([1] * n, [p + i + 1 for p in prompts], table[0])
        a, b = ev(), ev()
        a.record()
        y, h, y8, scales = block(x, res, slots, 0, batch, base8=True)
        b.record()
        outs.append(y)
        times.append((a, b))
    assert torch.equal(h, (x.float() + res.float()).bfloat16()) and scales.shape == (n, -(-hidden // 128))
    # ---- all of it in one pass
    total = [p + steps for p in prompts]
    a, b = ev(), ev()
    a.record()
    whole, _ = block(*cat(rows), np.repeat(slots, total), sum(total), store.KV4Batch.from_lens(total, total, table[1]))
    b.record()
    torch.cuda.synchronize()
    assert abi.lora_read_device_status(block.status) == 0
    last = torch.stack([w[-steps:] for w in whole.split(total)], 1).float()       # [steps][requests][hidden]
    off = float((torch.stack(outs).float() - last).norm() / last.norm())
    say(f"one pass over {sum(total)} rows: {a.elapsed_time(b):.3f} ms; a step of {n} single tokens: "
        f"{sorted(s.elapsed_time(e) for s, e in times)[steps // 2] * 1e3:.0f} us; outputs differ by {off:.2e} (relative)")
    return off


if __name__ == "__main__":
    ap = argparse.ArgumentParser()
    for name, v in (("hidden", 2048), ("heads", 16), ("kv", 4), ("dim", 128), ("steps", 20)):
        ap.add_argument("--" + name, type=int, default=v)
    build()
    run(**vars(ap.parse_args()))

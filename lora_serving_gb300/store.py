"""Device-resident adapter store and batch metadata (memory management only).

The store layout is the one the kernels read (peft orientation, K-major):
  A: bf16 [n_slots][r_slot][h_in]      per projection
  B: bf16 [n_slots][width][r_slot]     per projection, scale already folded
Slots are ``max_loras`` GPU slots and ``r_slot`` the slot rank
(``max_lora_rank``) of the vLLM offline LoRA page, step 2.  Folding and
padding happen in the C library (``lora_prepare_adapter``); this module only
allocates torch tensors, fills host staging buffers through the C call and
copies them to the device.
"""
from __future__ import annotations

import ctypes

import numpy as np
import torch

from . import abi


def _bits_to_device(a: np.ndarray, device) -> torch.Tensor:
    t = torch.from_numpy(np.ascontiguousarray(a).view(np.int16)).view(torch.bfloat16)
    return t.to(device, non_blocking=False)


class GroupStore:
    """Adapter store of one projection group (projections sharing x)."""

    def __init__(self, h_in: int, projs, n_slots: int, r_slot: int, device="cuda"):
        self.h_in, self.n_slots, self.r_slot = int(h_in), int(n_slots), int(r_slot)
        self.projs = [(str(n), int(w)) for n, w in projs]
        self.offsets = []
        o = 0
        for _, w in self.projs:
            self.offsets.append(o)
            o += w
        self.ld_y = o
        self.device = device
        self.A = [torch.zeros(n_slots, r_slot, h_in, dtype=torch.bfloat16, device=device) for _ in self.projs]
        self.B = [torch.zeros(n_slots, w, r_slot, dtype=torch.bfloat16, device=device) for _, w in self.projs]
        self._c = None

    def load_slots(self, adapters):
        """adapters: {slot: [(A_bits [r][h_in], B_bits [w][r], alpha, use_rslora) per projection]}."""
        for p, (_, w) in enumerate(self.projs):
            hA = np.zeros((self.n_slots, self.r_slot, self.h_in), np.uint16)
            hB = np.zeros((self.n_slots, w, self.r_slot), np.uint16)
            touched = []
            for k, per_proj in adapters.items():
                A, B, alpha, rs = per_proj[p]
                abi.lora_prepare_adapter(A, B, alpha, rs, self.r_slot, hA[k], hB[k])
                touched.append(k)
            if not touched:
                continue
            if len(touched) == self.n_slots:
                self.A[p].copy_(_bits_to_device(hA, "cpu"))
                self.B[p].copy_(_bits_to_device(hB, "cpu"))
            else:
                for k in touched:
                    self.A[p][k].copy_(_bits_to_device(hA[k], "cpu"))
                    self.B[p][k].copy_(_bits_to_device(hB[k], "cpu"))
        self._c = None
        return self

    @classmethod
    def from_workload(cls, wl, group_name: str, device="cuda"):
        g = next(g for g in wl.groups if g.name == group_name)
        st = cls(g.h_in, g.projs, wl.n_slots, wl.r_slot, device)
        adapters = {}
        for k in range(wl.n_slots):
            adapters[k] = [(wl.A[(g.name, pn, k)], wl.B[(g.name, pn, k)], float(wl.alphas[k]),
                            bool(wl.rslora[k])) for pn, _ in g.projs]
        return st.load_slots(adapters)

    def c_projs(self):
        """ctypes lora_proj_t array (kept alive by this object)."""
        if self._c is None:
            self._c = abi.make_projs([(self.A[p], self.B[p], self.offsets[p], w)
                                      for p, (_, w) in enumerate(self.projs)])
        return self._c

    def nbytes_slot(self) -> int:
        """Bytes of one slot across the group's projections."""
        return sum(self.r_slot * (self.h_in + w) * 2 for _, w in self.projs)


class BatchMeta:
    """Batch metadata from the C builder, copied to the device."""

    def __init__(self, ids, n_prefill: int, n_slots: int, device="cuda"):
        ids = np.ascontiguousarray(ids, np.int32)
        m = abi.lora_build_metadata(ids, n_prefill, n_slots)
        self.host = m
        self.host_ids = ids

        def up(a):
            a = np.ascontiguousarray(a, np.int32)
            if a.size == 0:
                a = np.zeros(1, np.int32)
            return torch.from_numpy(a).to(device)

        self.ids = up(ids)
        self.seg_starts = up(m["seg_starts"])
        self.seg_slot = up(m["seg_slot"])
        self.perm = up(m["perm"])
        self.gseg_starts = up(m["gseg_starts"])
        self.gseg_slot = up(m["gseg_slot"])
        self.n_rows, self.n_prefill = int(ids.size), int(n_prefill)
        c = abi.lora_meta_t()
        c.lora_ids = self.ids.data_ptr()
        c.n_rows, c.n_prefill = self.n_rows, self.n_prefill
        c.seg_starts, c.seg_slot = self.seg_starts.data_ptr(), self.seg_slot.data_ptr()
        c.n_segs, c.max_seg_len = m["n_segs"], m["max_seg_len"]
        c.perm, c.gseg_starts, c.gseg_slot = (self.perm.data_ptr(), self.gseg_starts.data_ptr(),
                                              self.gseg_slot.data_ptr())
        c.n_gsegs, c.max_gseg_len = m["n_gsegs"], m["max_gseg_len"]
        self.c = c


def workspace_for(n_rows: int, n_proj: int, r_slot: int, device="cuda") -> torch.Tensor:
    nbytes = max(abi.lora_apply_workspace_bytes(n_rows, n_proj, r_slot), 256)
    return torch.empty(nbytes, dtype=torch.uint8, device=device)


def apply(y: torch.Tensor, x: torch.Tensor, store: GroupStore, meta: BatchMeta,
          workspace: torch.Tensor, dev_status=None, stream=None, flags: int = 0):
    """One fused lora_apply call: y[:, slices] += delta of every projection."""
    abi.lora_apply(y, x, store.h_in, store.c_projs(), store.r_slot, store.n_slots, meta.c,
                   workspace, flags=flags, dev_status=dev_status, stream=stream)


def linear(y: torch.Tensor, x: torch.Tensor, W: torch.Tensor, store: GroupStore, meta: BatchMeta,
           workspace: torch.Tensor, dev_status=None, stream=None):
    """One lora_linear call: y[:, slices] = bf16(x W^T + delta) of every
    projection, W the group's stacked base weight [ld_y][h_in]."""
    abi.lora_linear(y, x, store.h_in, W, store.c_projs(), store.r_slot, store.n_slots, meta.c, workspace,
                    dev_status=dev_status, stream=stream)


class KV4Cache:
    """A paged 4-bit cache (layout: include/lora.h): device memory and the C
    struct that describes it.  pages: uint8 [n_pages][n_kv][block bytes], or
    a view of a larger buffer with another stride between pages (one page's
    blocks contiguous); allocated when None."""

    def __init__(self, n_pages: int, page_size: int, n_kv: int, head_dim: int, device="cuda", pages=None):
        block = abi.lora_kv4_block_bytes(page_size, head_dim)
        if not block:
            raise ValueError(f"no 4-bit cache with pages of {page_size} and heads of {head_dim}")
        if pages is None:
            pages = torch.zeros(n_pages, n_kv, block, dtype=torch.uint8, device=device)
        abi._dev(pages, "pages", "u8")
        if tuple(pages.shape) != (n_pages, n_kv, block) or pages.stride(2) != 1 or (n_kv > 1 and pages.stride(1) != block):
            raise ValueError(f"pages must be [{n_pages}][{n_kv}][{block}], contiguous within a page")
        self.pages = pages
        self.n_pages, self.page_size, self.n_kv, self.head_dim = n_pages, page_size, n_kv, head_dim
        stride = pages.stride(0) if n_pages > 1 else n_kv * block
        self.c = abi.lora_kv4_cache_t(pages.data_ptr(), stride, n_pages, page_size, n_kv, head_dim)
        self.addr = ctypes.addressof(self.c)


class KV4Batch:
    """Where a batch's rows stand in a cache: device int32 q_starts [n_seqs+1],
    ctx_lens [n_seqs] and block_table [n_seqs][pages], with the host's upper
    bounds.  The tensors may be refilled between calls (and replays of a
    captured graph) as long as the bounds hold.  held: device int32 [n_seqs],
    the pages of each sequence of a lora_kv4_plan's batch (its held_out)."""

    def __init__(self, q_starts, ctx_lens, block_table, *, n_rows: int, max_q_len: int, max_ctx_len: int, held=None):
        n_seqs = int(ctx_lens.numel())
        for name, t, n in (("q_starts", q_starts, n_seqs + 1), ("ctx_lens", ctx_lens, n_seqs)):
            if t.dim() != 1 or t.numel() != n or (n > 1 and t.stride(0) != 1):
                raise ValueError(f"{name} must hold {n} adjacent entries")
        if block_table.shape[0] != n_seqs:
            raise ValueError(f"block_table must have {n_seqs} rows")
        self.q_starts, self.ctx_lens, self.block_table, self.held = q_starts, ctx_lens, block_table, held
        # the C side checks ld_table against max_ctx_len: with a stride wider
        # than the row it would pass a table that is too narrow
        ld = int(block_table.shape[1])
        if n_seqs > 1 and int(block_table.stride(0)) != ld:
            raise ValueError("block_table must be contiguous")
        self.c = abi.lora_kv4_batch_t(abi._dev(q_starts, "q_starts", "i32"), abi._dev(ctx_lens, "ctx_lens", "i32"),
                                      abi._dev(block_table, "block_table", "i32", True), ld, n_seqs,
                                      int(n_rows), int(max_q_len), int(max_ctx_len), _vector(held, "held", "i32", n_seqs))
        self.addr = ctypes.addressof(self.c)

    @classmethod
    def from_lens(cls, q_lens, ctx_lens, block_table, device="cuda"):
        """From host lists: rows and positions (the rows' own included) of each sequence."""
        q, ctx = np.asarray(q_lens, np.int32), np.asarray(ctx_lens, np.int32)
        starts = np.concatenate([[0], np.cumsum(q)]).astype(np.int32)
        up = lambda a: torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(device)  # noqa: E731
        return cls(up(starts), up(ctx), up(np.asarray(block_table)), n_rows=int(starts[-1]),
                   max_q_len=int(q.max(initial=0)), max_ctx_len=int(ctx.max(initial=0)))


def kv4_workspace(cache: KV4Cache, n_heads: int, batch: KV4Batch, device="cuda") -> torch.Tensor:
    """A workspace for lora_kv4_attend over batches within this one's bounds."""
    nbytes = abi.lora_kv4_attend_workspace_bytes(n_heads, cache.n_kv, cache.head_dim, batch.c.max_q_len)
    return torch.empty(max(nbytes, 256), dtype=torch.uint8, device=device)


def _vector(t, name: str, dtype: str, n: int) -> int:
    """Pointer of a device tensor of n adjacent entries at least; 0 for None."""
    p = abi._dev(t, name, dtype)
    if t is not None and (t.dim() != 1 or t.numel() < n or (t.numel() > 1 and t.stride(0) != 1)):
        raise ValueError(f"{name} must hold {n} adjacent entries at least")
    return p


class KV4Plan:
    """The tables of a server's steps and the pages behind them, for
    abi.lora_kv4_plan.  Device int32 free_pages [n_pages] (a stack: the first
    n_free [1] entries), held [n_seqs] and block_table [n_seqs][columns] are the
    server's own; the counters' results go to them in place, or to n_free_out
    and held_out, with which a plan can be made again or dropped.  The call
    fills q_starts, ctx_lens, row_seq, positions [max_rows][1] (what
    lora_kv4_append takes) and slots, and `batch` is the store.KV4Batch of the
    step: rows from 0 to max_rows, of which those past the last are skipped."""

    def __init__(self, free_pages, n_free, held, block_table, *, page_size: int, max_rows: int, max_q_len: int,
                 max_ctx_len: int, n_free_out=None, held_out=None):
        n_seqs = int(held.numel())
        dev = held.device
        self.free_pages, self.n_free, self.held, self.block_table = free_pages, n_free, held, block_table
        self.n_free_out = n_free if n_free_out is None else n_free_out
        self.held_out = held if held_out is None else held_out
        if block_table.dim() != 2 or block_table.shape[0] != n_seqs:
            raise ValueError(f"block_table must have {n_seqs} rows")
        new = lambda n, dtype=torch.int32: torch.full((n,), -1, dtype=dtype, device=dev)  # noqa: E731
        self.q_starts, self.ctx_lens = torch.zeros(n_seqs + 1, dtype=torch.int32, device=dev), torch.zeros(n_seqs, dtype=torch.int32, device=dev)
        self.row_seq, self.positions, self.slots = new(max_rows), new(max_rows).view(-1, 1), new(max_rows, torch.int64)
        self.batch = KV4Batch(self.q_starts, self.ctx_lens, block_table, n_rows=max_rows, max_q_len=max_q_len, max_ctx_len=max_ctx_len,
                              held=self.held_out)
        pool = abi.lora_kv4_pool_t(_vector(free_pages, "free_pages", "i32", 1), _vector(n_free, "n_free", "i32", 1),
                                   _vector(held, "held", "i32", n_seqs), _vector(self.n_free_out, "n_free_out", "i32", 1),
                                   _vector(self.held_out, "held_out", "i32", n_seqs), self.batch.c.block_table,
                                   self.batch.c.ld_table, int(free_pages.numel()), int(page_size))
        self.c = abi.plan_args_t(self.q_starts.data_ptr(), self.ctx_lens.data_ptr(), self.row_seq.data_ptr(),
                                 self.positions.data_ptr(), self.slots.data_ptr(), n_seqs, int(max_rows), int(max_q_len),
                                 int(max_ctx_len), pool)
        self.addr = ctypes.addressof(self.c)

    @classmethod
    def empty(cls, n_seqs: int, n_pages: int, page_size: int, *, max_rows: int, max_q_len: int, max_ctx_len: int, device="cuda"):
        """Of a cache whose pages are all free and will be taken in their order."""
        i32 = lambda *a: torch.zeros(*a, dtype=torch.int32, device=device)  # noqa: E731
        return cls(torch.arange(n_pages - 1, -1, -1, dtype=torch.int32, device=device), i32(1) + n_pages, i32(n_seqs),
                   i32(n_seqs, -(-max_ctx_len // page_size)) - 1, page_size=page_size, max_rows=max_rows, max_q_len=max_q_len,
                   max_ctx_len=max_ctx_len)


class KV4Layers:
    """The caches of a model's layers, which one block table serves (abi.lora_kv4_keep)."""

    def __init__(self, caches):
        self.caches, self.n = list(caches), len(caches)
        self.c = (abi.lora_kv4_cache_t * max(self.n, 1))(*[c.c for c in self.caches])
        self.addr = ctypes.addressof(self.c)


class LogitsRules:
    """What requests ask of their logits (abi.lora_logits_adjust): int32 tokens
    [n_seqs][columns] with prompt_lens and token_lens [n_seqs]; fp32
    repetition, frequency and presence [n_seqs] or None; int32 bias_ids and fp32
    bias [n_seqs][columns] with n_bias [n_seqs], or None.  The tensors may be
    refilled between calls and replays."""

    def __init__(self, tokens, prompt_lens, token_lens, *, repetition=None, frequency=None, presence=None, bias_ids=None,
                 bias=None, n_bias=None):
        n = int(token_lens.numel())
        rows = lambda t, name, dtype: 0 if t is None else self._rows(t, name, dtype, n)  # noqa: E731
        if (bias_ids is None) != (bias is None) or (bias_ids is None) != (n_bias is None):
            raise ValueError("bias_ids, bias and n_bias come together")
        if bias is not None and tuple(bias.shape) != tuple(bias_ids.shape):
            raise ValueError("bias must have the shape of bias_ids")
        v = lambda t, name, dtype: _vector(t, name, dtype, n)  # noqa: E731
        self.keep = (tokens, prompt_lens, token_lens, repetition, frequency, presence, bias_ids, bias, n_bias)
        self.c = abi.lora_logits_rules_t(rows(tokens, "tokens", "i32"), v(prompt_lens, "prompt_lens", "i32"),
                                         v(token_lens, "token_lens", "i32"), v(repetition, "repetition", "f32"),
                                         v(frequency, "frequency", "f32"), v(presence, "presence", "f32"),
                                         rows(bias_ids, "bias_ids", "i32"), rows(bias, "bias", "f32"), v(n_bias, "n_bias", "i32"),
                                         int(tokens.shape[1]), 0 if bias is None else int(bias.shape[1]), n)
        self.addr = ctypes.addressof(self.c)

    @staticmethod
    def _rows(t, name, dtype, n):
        p = abi._dev(t, name, dtype, True)
        if t.shape[0] != n or not t.is_contiguous():
            raise ValueError(f"{name} must be contiguous, with {n} rows")
        return p


def rope_table(max_pos: int, pairs: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """fp32 [max_pos][pairs][2]: (cos, sin) of pos * base^(-i / pairs), angles in fp64."""
    f = base ** (-torch.arange(pairs, dtype=torch.float64) / pairs)
    a = torch.arange(max_pos, dtype=torch.float64)[:, None] * f
    return torch.stack([a.cos(), a.sin()], -1).to(torch.float32).to(device)

"""Drafted decoding as a server runs it: each step plans its tables on the GPU, appends the drafted rows to every layer's
cache, attends under the trees, adjusts the logits, and keeps the accepted paths; requests come in, end and give way to
others.  What is kept must be what the same tokens give one after another: the cached bytes and the adjusted logits
exactly, the attention within its tolerance (twice, for both are rounded)."""
import math

import numpy as np
import pytest
import torch

import draft_ref as R
import kv4_ref as K4
from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


class Server:
    """`slots` requests at a time; a step's kernels in one captured graph, keeping in another."""

    def __init__(self, slots, layers, H, KV, D, page, n_pages, vocab, max_rows, max_q, max_ctx, seed):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.H, self.KV, self.D, self.vocab, self.W, self.max_rows = H, KV, D, vocab, (H + 2 * KV) * D, max_rows
        self.embed = (torch.randn(layers, vocab, self.W, generator=g, device="cuda")).bfloat16()      # a token's q, k and v in each layer
        self.caches = [store.KV4Cache(n_pages, page, KV, D) for _ in range(layers)]
        self.plan = store.KV4Plan.empty(slots, n_pages, page, max_rows=max_rows, max_q_len=max_q, max_ctx_len=max_ctx)
        self.layers = store.KV4Layers(self.caches)
        self.rope = store.rope_table(max_ctx, D // 2)
        z = lambda *s: torch.zeros(*s, dtype=torch.int32, device="cuda")  # noqa: E731
        self.q_lens, self.lens, self.depths, self.drafts = z(slots), z(slots), z(max_rows), z(max_rows)
        self.tree, self.n_keep, self.path = z(max_rows, -(-max_q // 32)), z(slots), z(slots, max_q)
        self.tokens, self.prompts, self.token_lens = z(slots, max_ctx), z(slots), z(slots)
        f = lambda lo, hi: lo + (hi - lo) * torch.rand(slots, generator=g, device="cuda")  # noqa: E731
        self.rules = store.LogitsRules(self.tokens, self.prompts, self.token_lens, repetition=f(1, 1.5), frequency=f(0, 0.5), presence=f(0, 0.5))
        wide = -(-vocab // 8) * 8
        self.raw = (3 * torch.randn(max_ctx, wide, generator=g, device="cuda")).bfloat16()          # logits by position
        self.x = [torch.zeros(max_rows, self.W, dtype=torch.bfloat16, device="cuda") for _ in range(layers)]
        self.q = torch.zeros(max_rows, H * D, dtype=torch.bfloat16, device="cuda")
        self.o = [torch.zeros_like(self.q) for _ in range(layers)]
        self.logits = torch.zeros(max_rows, wide, dtype=torch.bfloat16, device="cuda")
        self.out = torch.zeros(max_rows, wide, dtype=torch.float32, device="cuda")[:, :vocab]
        self.ws = store.kv4_workspace(self.caches[0], H, self.plan.batch)
        self.status = z(1)
        self._step(), self._keep()
        torch.cuda.synchronize()
        self.graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
        for graph, work in zip(self.graphs, (self._step, self._keep)):
            with torch.cuda.graph(graph):
                work()

    def _step(self):
        p, H, KV, D = self.plan, self.H, self.KV, self.D
        abi.lora_kv4_plan(p, self.q_lens, self.lens, depths=self.depths, dev_status=self.status)
        for cache, x, o, e in zip(self.caches, self.x, self.o, self.embed):
            torch.index_select(e, 0, self.drafts, out=x)
            abi.lora_kv4_append(self.q, x, cache, p.batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, rope=self.rope,
                                positions=p.positions, dev_status=self.status)
            abi.lora_kv4_attend_tree(o, self.q, cache, p.batch, self.tree, self.ws, n_heads=H, scale=1 / math.sqrt(D), dev_status=self.status)
        torch.index_select(self.raw, 0, p.positions[:, 0].clamp(min=0), out=self.logits)
        abi.lora_logits_adjust(self.out, self.logits[:, :self.vocab], self.rules, row_seq=p.row_seq, drafts=self.drafts, tree=self.tree, q_starts=p.q_starts,
                               dev_status=self.status)

    def _keep(self):
        abi.lora_kv4_keep(self.layers, self.plan.batch, self.n_keep, self.path, lens=self.lens, dev_status=self.status)

    def step(self, jobs):
        """jobs: for each slot None (idle), "end", or (tokens, parents) of its rows."""
        rows, depth, bits, q = [], [], [], []
        for j in jobs:
            tokens, parents = j if isinstance(j, tuple) else ([], [])
            mine, d = [], []
            for i, up in enumerate(parents):
                mine.append((mine[up] if up >= 0 else 0) | 1 << i)
                d.append(d[up] + 1 if up >= 0 else 0)
            rows += tokens
            depth += d
            bits.append(mine)
            q.append(-1 if j == "end" else len(tokens))
        n = len(rows)
        self.q_lens.copy_(_i32(q))
        self.drafts[:n].copy_(_i32(rows))
        self.depths[:n].copy_(_i32(depth))
        self.tree[:n].copy_(torch.from_numpy(R.words(bits, self.tree.shape[1])))
        self.graphs[0].replay()

    def keep(self, paths):
        for s, p in enumerate(paths):
            self.path[s, :len(p)] = _i32(p)
        self.n_keep.copy_(_i32([len(p) for p in paths]))
        self.graphs[1].replay()


SHAPES = [dict(layers=3, H=8, KV=2, D=64, page=16, vocab=61), dict(layers=2, H=16, KV=2, D=128, page=32, vocab=200)]


@pytest.mark.parametrize("shape", SHAPES, ids=["small", "wide"])
def test_drafted_steps_give_what_the_tokens_give(shape):
    slots, steps, max_q, max_ctx = 5, 12, 40, 160
    rng = np.random.default_rng(shape["vocab"])
    sv = Server(slots, n_pages=5 * max_ctx // shape["page"] + 3, max_rows=slots * max_q, max_q=max_q, max_ctx=max_ctx, seed=1, **shape)
    V = shape["vocab"]
    running = [None] * slots          # [tokens kept so far, prompt's length, outputs of them by (layer) and logits]
    done = []
    for step in range(steps):
        jobs, follow = [], []
        for s in range(slots):
            r = running[s]
            if r is None:
                if step and rng.random() < 0.3:
                    jobs.append(None), follow.append(None)
                    continue
                tokens = rng.integers(0, V, rng.integers(1, max_q + 1)).tolist()      # a prompt: a chain, all of it kept
                running[s] = dict(tokens=[], prompt=len(tokens), out=[[] for _ in sv.caches], logits=[])
                jobs.append((tokens, [i - 1 for i in range(len(tokens))])), follow.append(list(range(len(tokens))))
            elif len(r["tokens"]) > 90 or (step > 3 and rng.random() < 0.15):
                done.append(r)
                running[s] = None
                jobs.append("end"), follow.append(None)
            else:
                n = int(rng.integers(1, 20))
                parents = [-1] + [int(rng.integers(max(0, i - 4), i)) for i in range(1, n)]
                path = [0]                                                            # the branch that is found right
                while rng.random() < 0.8:
                    kids = [i for i in range(n) if parents[i] == path[-1]]
                    if not kids:
                        break
                    path.append(int(rng.choice(kids)))
                jobs.append((rng.integers(0, V, n).tolist(), parents)), follow.append(path)
        sv.prompts.copy_(_i32([min(r["prompt"], len(r["tokens"])) if r else 0 for r in running]))
        sv.token_lens.copy_(_i32([len(r["tokens"]) if r else 0 for r in running]))
        for s, r in enumerate(running):
            if r and r["tokens"]:
                sv.tokens[s, :len(r["tokens"])] = _i32(r["tokens"])
        sv.step(jobs)
        sv.keep([f or [] for f in follow])
        torch.cuda.synchronize()
        assert abi.lora_read_device_status(sv.status) == 0
        starts = sv.plan.q_starts.tolist()
        for s, f in enumerate(follow):
            if f is None:
                continue
            r = running[s]
            at = [starts[s] + i for i in f]
            if r["tokens"]:
                r["logits"].append((len(r["tokens"]), sv.out[at].clone()))
            for out, o in zip(r["out"], sv.o):
                out.append(o[at].clone())
            r["tokens"] += [jobs[s][0][i] for i in f]
        assert sv.lens.tolist() == [len(r["tokens"]) if r else 0 for r in running]
        # the cached bytes are those of the tokens, one after another
        alive = [s for s in range(slots) if running[s]]
        lens = [len(running[s]["tokens"]) for s in alive]
        table = np.arange(len(alive) * 99).reshape(-1, 99)
        ref_batch = store.KV4Batch.from_lens(lens, lens, table)
        own = store.KV4Batch.from_lens(lens, lens, sv.plan.block_table.cpu().numpy()[alive])
        every = _i32(np.concatenate([running[s]["tokens"] for s in alive]))
        H, KV, D = sv.H, sv.KV, sv.D
        for layer, cache in enumerate(sv.caches):
            ref = store.KV4Cache(table.size, cache.page_size, KV, D)
            q = torch.empty(sum(lens), H * D, dtype=torch.bfloat16, device="cuda")
            abi.lora_kv4_append(q, sv.embed[layer][every.long()], ref, ref_batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, rope=sv.rope)
            got, want = ([torch.empty(sum(lens), KV * D, dtype=torch.bfloat16, device="cuda") for _ in range(2)] for _ in range(2))
            abi.lora_kv4_read(*got, cache, own)
            abi.lora_kv4_read(*want, ref, ref_batch)
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]), (step, layer)
            if step == steps - 1:     # and the attention that each kept row had, that of its place in the sequence
                o, tol = K4.attend(K4.f64(q).reshape(-1, H, D), *K4.unpack(ref.pages.cpu().numpy(), ref.page_size, D), lens, lens, table,
                                   ref.page_size, 1 / math.sqrt(D))
                had = torch.cat([torch.cat(running[s]["out"][layer]) for s in alive])
                assert (np.abs(K4.f64(had).reshape(o.shape) - o) <= tol).all(), layer
    # the logits of each kept row: those of a request that has its tokens behind it
    assert done and alive
    for s in alive:
        r = running[s]
        for first, rows in r["logits"]:
            n = rows.shape[0]
            part = lambda t: t[s:s + 1].expand(n).contiguous()  # noqa: E731
            rules = store.LogitsRules(_i32([r["tokens"]] * n), _i32([r["prompt"]] * n), _i32(range(first + 1, first + 1 + n)),
                                      repetition=part(sv.rules.keep[3]), frequency=part(sv.rules.keep[4]), presence=part(sv.rules.keep[5]))
            want = torch.empty(n, sv.raw.shape[1], dtype=torch.float32, device="cuda")[:, :V]
            abi.lora_logits_adjust(want, sv.raw[first:first + n, :V], rules)
            assert torch.equal(rows, want)


def test_a_request_without_pages_waits():
    """A sequence for which the pages have run out has no place: its rows come to nothing, its lengths stay, and it goes on once there are pages."""
    page, H, KV, D = 16, 4, 2, 64
    p = store.KV4Plan.empty(3, 4, page, max_rows=60, max_q_len=40, max_ctx_len=64)
    cache = store.KV4Cache(4, page, KV, D)
    lens, st = _i32([0, 0, 0]), _i32([0])
    x = torch.randn(60, (H + 2 * KV) * D, device="cuda").bfloat16()
    q, o = torch.zeros(60, H * D, dtype=torch.bfloat16, device="cuda"), torch.full((60, H * D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = store.kv4_workspace(cache, H, p.batch)
    tree = torch.full((60, 2), -1, dtype=torch.int32, device="cuda")

    def step(q_lens, keep):
        st.zero_()
        o.fill_(7)
        abi.lora_kv4_plan(p, _i32(q_lens), lens, dev_status=st)
        abi.lora_kv4_append(q, x, cache, p.batch, n_heads=H, q_off=0, k_off=H * D, v_off=(H + KV) * D, dev_status=st)
        abi.lora_kv4_attend_tree(o, q, cache, p.batch, tree, ws, n_heads=H, scale=0.1, dev_status=st)
        path = _i32([list(range(40))] * 3)
        abi.lora_kv4_keep(store.KV4Layers([cache]), p.batch, _i32(keep), path, lens=lens, dev_status=st)
        return abi.lora_read_device_status(st)

    assert step([16, 30, 12], [16, 30, 12]) == 0 and lens.tolist() == [16, 30, 12] and int(p.n_free) == 0
    assert step([1, 2, 4], [1, 2, 4]) == abi.LORA_DEV_NO_PAGES       # the first would need a page; the others fill their own
    assert lens.tolist() == [16, 32, 16] and (o[0] == 0).all() and (o[1:7].float().abs().sum(1) > 0).all() and (o[7:] == 7).all()
    assert p.ctx_lens.tolist() == [0, 32, 16] and p.row_seq.tolist()[:8] == [-1, 1, 1, 2, 2, 2, 2, -1] and p.slots.tolist()[0] == -1
    assert step([0, -1, 0], [0, 0, 0]) == 0 and int(p.n_free) == 2 and lens.tolist() == [16, 0, 16]
    assert step([1, 0, 1], [1, 0, 1]) == 0 and lens.tolist() == [17, 0, 17] and int(p.n_free) == 0

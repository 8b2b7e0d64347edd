"""lora_logits_adjust against tests/draft_ref.py in 64 bits.  Tolerance: half a
step of the output's type (2^-8 in bf16, 2^-24 in fp32, of the value), and for
each of the five fp32 operations before it 2^-24 of the magnitudes that they
add up."""
import numpy as np
import pytest
import torch

import draft_ref as R
from lora_serving_gb300 import abi, build, store

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    build()
    abi.load()
    assert torch.cuda.is_available()


def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).cuda()


def _f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).cuda()


def _case(seed, q_lens, V, hist, n_bias, drafts, masks, kinds=(BF, BF)):
    rng = np.random.default_rng(seed)
    n, T = len(q_lens), sum(q_lens)
    wide = -(-V // 8) * 8 + 8
    x = torch.from_numpy((3 * rng.standard_normal((T, wide))).astype(np.float32)).to(kinds[0]).cuda()
    tokens = (V * rng.random((n, max([1, *hist]))) ** 3).astype(np.int64)
    tokens[rng.random(tokens.shape) < 0.02] = rng.choice([-1, V, V + 7, 2 ** 31 - 1, -2 ** 31])   # count for nothing
    c = dict(x=x, wide=wide, tokens=tokens, length=np.array(hist), prompt=np.array([rng.integers(0, h + 1) for h in hist]),
             rep=1 + 0.3 * rng.random(n), freq=0.5 * rng.random(n), pres=0.5 * rng.random(n), q=q_lens, V=V, kinds=kinds)
    c["rep"][::3], c["freq"][::3], c["pres"][::3] = 1, 0, 0
    c = {k: v.astype(np.float32).astype(np.float64) if k in ("rep", "freq", "pres") else v for k, v in c.items()}
    if n_bias:
        c["bias_ids"] = rng.integers(0, V, (n, n_bias))
        c["bias_ids"][:, n_bias // 2] = c["bias_ids"][:, 0]                      # the same token twice
        c["bias_ids"][:, -1] = -1
        c["bias"] = (5 * rng.standard_normal((n, n_bias))).astype(np.float32).astype(np.float64)
        c["n_bias"] = rng.integers(0, n_bias + 1, n)
    if drafts:
        c["bits"], c["drafts"] = R.trees(rng, q_lens), (V * rng.random(T) ** 3).astype(np.int64)
        c["drafts"][rng.random(T) < 0.05] = -1
    if masks:
        c["sets"] = rng.random((n + 1, V)) < rng.random((n + 1, 1))
        c["sets"][0] = False                                                     # nothing allowed
        c["set_of"] = rng.integers(-1, n + 1, T)
    return c


def _words(sets, extra=1):
    n, V = sets.shape
    full = np.ones((n, (-(-V // 32) + extra) * 32), bool)                          # bits past the vocabulary do not matter
    full[:, :V] = sets
    return np.packbits(full, axis=1, bitorder="little").view("<i4")


def _args(c):
    rules = store.LogitsRules(_i32(c["tokens"]), _i32(c["prompt"]), _i32(c["length"]), repetition=_f32(c["rep"]), frequency=_f32(c["freq"]),
                              presence=_f32(c["pres"]), bias_ids=_i32(c["bias_ids"]) if "bias" in c else None,
                              bias=_f32(c["bias"]) if "bias" in c else None, n_bias=_i32(c["n_bias"]) if "bias" in c else None)
    kw = dict(row_seq=_i32(np.repeat(np.arange(len(c["q"])), c["q"])))
    if "drafts" in c:
        kw |= dict(drafts=_i32(c["drafts"]), tree=torch.from_numpy(R.words(c["bits"], -(-max(c["q"]) // 32), np.random.default_rng(1))).cuda(),
                   q_starts=_i32(np.concatenate([[0], np.cumsum(c["q"])])))
    if "sets" in c:
        kw |= dict(allowed=torch.from_numpy(_words(c["sets"])).cuda(), allowed_rows=_i32(c["set_of"]))
    return rules, kw


def _want(c):
    t, out = 0, []
    x = c["x"].double().cpu().numpy()[:, :c["V"]]
    for s, n in enumerate(c["q"]):
        biases = list(zip(c["bias_ids"][s, :c["n_bias"][s]].tolist(), c["bias"][s].tolist())) if "bias" in c else []
        for i in range(n):
            path = [c["drafts"][t - i + j] for j in range(n) if c["bits"][s][i] >> j & 1] if "drafts" in c else []
            allowed = c["sets"][c["set_of"][t]] if "sets" in c and c["set_of"][t] >= 0 else None
            out.append(R.adjust(x[t], c["tokens"][s], c["prompt"][s], c["length"][s], c["rep"][s], c["freq"][s], c["pres"][s], biases, path, allowed))
            t += 1
    return (np.array(a) for a in zip(*out))


def _check(got, want, M, kind):
    got = got.double().cpu().numpy()
    gone = np.isneginf(want)
    assert np.array_equal(np.isneginf(got), gone)
    half = 2.0 ** -8 if kind == BF else 2.0 ** -24
    g, w, m = got[~gone], want[~gone], M[~gone]
    tol = half * (np.abs(w) + 5 * 2.0 ** -24 * m) + 5 * 2.0 ** -24 * m + 1e-38
    assert (np.abs(g - w) <= tol).all(), float((np.abs(g - w) - tol).max())


CASES = [  # rows of each request, vocabulary, tokens of each, biases, drafts, masks
    ([1], 8, [0], 0, False, False),
    ([1], 32000, [700], 0, False, False),
    ([1, 1, 1], 1, [5, 0, 1], 2, False, True),
    ([1] * 9, 50257, [1000, 1, 0, 30, 4000, 7, 2, 90, 5000], 40, False, True),      # a vocabulary that no vector divides
    ([3, 1, 0, 17], 8193, [100, 3, 9, 2000], 5, True, True),
    ([40, 33], 4099, [50, 0], 0, True, False),
    ([64], 2047, [9000], 300, True, True),
    ([2, 2], 131072, [20000, 8], 2047, True, True),
    ([1] * 300, 1500, [20] * 300, 3, False, True),
]


@pytest.mark.parametrize("kinds", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
@pytest.mark.parametrize("rows,V", [(56, 100003), (66, 65537), (100, 50257), (16, 131071)])
def test_chunks_in_turns(rows, V, kinds):
    """Decode batches on either side of where the chunks change their length."""
    rng = np.random.default_rng(V)
    c = _case(V, [1] * rows, V, rng.integers(0, 400, rows).tolist(), 6, False, True, kinds)
    rules, kw = _args(c)
    out = torch.full((rows, c["wide"]), 9.0, dtype=kinds[1], device="cuda")
    abi.lora_logits_adjust(out[:, :V], c["x"][:, :V], rules, **kw)
    _check(out[:, :V], *_want(c), kinds[1])
    assert (out[:, V:] == 9).all()
    if kinds[0] == kinds[1]:     # in place
        x = c["x"][:, :V]
        abi.lora_logits_adjust(x, x, rules, **kw)
        assert torch.equal(x, out[:, :V])


@pytest.mark.parametrize("kinds", [(BF, BF), (F32, F32)], ids=["bb", "ff"])
@pytest.mark.parametrize("q,V", [([40] * 50, 300), ([40] * 50, 2048), ([130, 70, 1], 4099), ([200, 65], 150)], ids=lambda v: str(v) if isinstance(v, int) else f"{len(v)}x{max(v)}")
def test_rows_of_large_trees(q, V, kinds):
    """Rows that share a CTA in a vocabulary of one short chunk, and paths of more than two words."""
    c = _case(V, q, V, [30] * len(q), 4, True, True, kinds)
    rules, kw = _args(c)
    out = torch.full((sum(q), c["wide"]), 9.0, dtype=kinds[1], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_logits_adjust(out[:, :V], c["x"][:, :V], rules, dev_status=st, **kw)
    assert abi.lora_read_device_status(st) == 0
    _check(out[:, :V], *_want(c), kinds[1])
    assert (out[:, V:] == 9).all()


@pytest.mark.parametrize("case", CASES, ids=lambda c: f"{len(c[0])}x{max(c[0])}-{c[1]}")
@pytest.mark.parametrize("kinds", [(BF, BF), (BF, F32), (F32, F32), (F32, BF)], ids=["bb", "bf", "ff", "fb"])
def test_adjust(case, kinds):
    c = _case(case[1] + len(case[0]), *case, kinds)
    rules, kw = _args(c)
    out = torch.full((sum(c["q"]), c["wide"]), 9.0, dtype=kinds[1], device="cuda")
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    abi.lora_logits_adjust(out[:, :c["V"]], c["x"][:, :c["V"]], rules, dev_status=st, **kw)
    assert abi.lora_read_device_status(st) == 0
    _check(out[:, :c["V"]], *_want(c), kinds[1])
    assert (out[:, c["V"]:] == 9).all()
    if kinds[0] == kinds[1]:     # in place
        x = c["x"][:, :c["V"]]
        abi.lora_logits_adjust(x, x, rules, **kw)
        assert torch.equal(x, out[:, :c["V"]]) and torch.isfinite(c["x"][:, c["V"]:]).all()


def test_default_rows_masks_alone_and_rows_that_are_left():
    V, T = 1000, 6
    c = _case(3, [1] * T, V, [40] * T, 0, False, True)
    rules, kw = _args(c)
    every = torch.empty(T, V, dtype=BF, device="cuda")
    c["set_of"] = np.arange(T)
    abi.lora_logits_adjust(every, c["x"][:, :V], rules, allowed=kw["allowed"])     # row t: request t, set t
    _check(every, *_want(c), BF)
    only = torch.empty_like(every)
    abi.lora_logits_adjust(only, c["x"][:, :V], allowed=kw["allowed"])
    sets = torch.from_numpy(c["sets"][:T]).cuda()
    assert torch.equal(only, torch.where(sets, c["x"][:, :V], torch.tensor(-torch.inf, dtype=BF, device="cuda")))
    some = torch.full_like(every, 3.0)
    abi.lora_logits_adjust(some, c["x"][:, :V], rules, row_seq=_i32([0, -1, 2, 2, -1, 5]), allowed=kw["allowed"])
    assert (some[[1, 4]] == 3).all() and torch.equal(some[[0, 2, 5]], every[[0, 2, 5]]) and not (some[3] == 3).all()


def test_values_at_the_ends():
    """Infinities and NaN pass through their operations and no further; a masked token is -infinity whatever it was."""
    V = 64
    x = torch.zeros(2, V, dtype=F32, device="cuda")
    x[:, 0], x[:, 1], x[:, 2], x[:, 3], x[:, 4] = torch.inf, -torch.inf, torch.nan, 0.0, -0.0
    sets = np.ones((1, V), bool)
    sets[0, 40:44] = False
    x[1, 40:44] = torch.tensor([torch.nan, torch.inf, -torch.inf, 3e38], device="cuda")
    tokens = np.tile([0, 1, 2, 3, 4, 40], (2, 1))
    rules = store.LogitsRules(_i32(tokens), _i32([6, 0]), _i32([6, 6]), repetition=_f32([1.5, 2.0]), frequency=_f32([0.5, 0.25]), presence=_f32([9, 0.5]))
    out = torch.empty_like(x)
    abi.lora_logits_adjust(out, x, rules, allowed=torch.from_numpy(_words(sets)).cuda(), allowed_rows=_i32([-1, 0]))
    o = out.cpu()
    assert o[0, 0] == torch.inf and o[0, 1] == -torch.inf and o[0, 2].isnan() and (o[0, 3:] == 0).all()
    assert o[1, 0] == torch.inf and o[1, 1] == -torch.inf and o[1, 2].isnan() and (o[1, 3:5] == -0.75).all() and (o[1, 40:44] == -torch.inf).all()
    assert (o[1, 5:40] == 0).all() and (o[1, 44:] == 0).all()


def test_repeats_bit_for_bit():
    c = _case(8, [64, 3], 30000, [9000, 8000], 500, True, True)
    c["tokens"][:] = c["tokens"] % 11                          # thousands of counts on a few tokens
    rules, kw = _args(c)
    x = c["x"][:, :30000]
    first = torch.empty(67, 30000, dtype=BF, device="cuda")
    abi.lora_logits_adjust(first, x, rules, **kw)
    _check(first, *_want(c), BF)
    for _ in range(3):
        again = torch.empty_like(first)
        abi.lora_logits_adjust(again, x, rules, **kw)
        assert torch.equal(again, first)


def test_faults_leave_their_rows():
    V = 3000
    c = _case(5, [2, 2, 2, 2], V, [30] * 4, 6, True, True)
    rules, kw = _args(c)
    x, first = c["x"][:, :V], torch.full((8, V), 7.0, dtype=BF, device="cuda")
    abi.lora_logits_adjust(first, x, rules, **kw)

    def run(rows, bit, **change):
        out, st = torch.full_like(first, 7.0), torch.zeros(1, dtype=torch.int32, device="cuda")
        abi.lora_logits_adjust(out, x, rules, dev_status=st, **{**kw, **change})
        assert abi.lora_read_device_status(st) == bit
        keep = [t for t in range(8) if t not in rows]
        assert (out[rows] == 7).all() and torch.equal(out[keep], first[keep])

    seq = np.repeat(np.arange(4), 2)
    top = 2 ** 31 - 1
    for v in (4, -2, top):
        run([3], abi.LORA_DEV_BAD_SEGMENT, row_seq=_i32(np.where(np.arange(8) == 3, v, seq)))
    run([3], abi.LORA_DEV_BAD_SEGMENT, row_seq=_i32(np.where(np.arange(8) == 3, 2, seq)))     # not one of its request's rows
    for v in (5, -2, top):
        run([6], abi.LORA_DEV_SLOT_OUT_OF_RANGE, allowed_rows=_i32(np.where(np.arange(8) == 6, v, c["set_of"])))
    for t, v in ((rules.keep[2], 31), (rules.keep[2], -1), (rules.keep[1], 31), (rules.keep[1], -1), (rules.keep[8], 7), (rules.keep[8], -1)):
        old = int(t[1])
        t[1] = v
        run([2, 3], abi.LORA_DEV_BAD_SEGMENT)
        t[1] = old
    run([2, 3, 4, 5], abi.LORA_DEV_BAD_SEGMENT, q_starts=_i32([0, 2, 9, 6, 8]))
    run([0, 1], abi.LORA_DEV_BAD_SEGMENT, q_starts=_i32([-1, 2, 4, 6, 8]) + _i32([0, 0, 0, 0, 0]))


def test_replay_with_refilled_rules():
    V = 5000
    c = _case(6, [4, 4], V, [300, 200], 10, True, True)
    rules, kw = _args(c)
    x, out = c["x"][:, :V], torch.empty(8, V, dtype=F32, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    abi.lora_logits_adjust(out, x, rules, **kw, stream=side)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        abi.lora_logits_adjust(out, x, rules, **kw)
    for seed in (7, 8):
        d = _case(seed, [4, 4], V, [300, 200], 10, True, True)
        other, kd = _args(d)
        for a, b in zip(rules.keep, other.keep):
            a.copy_(b)
        for k in kw:
            kw[k].copy_(kd[k])
        c["x"].copy_(d["x"])
        g.replay()
        torch.cuda.synchronize()
        _check(out, *_want(d), F32)


def test_trees_past_a_thread_block_and_rows_between_others():
    """Paths of more rows than a block has threads; requests whose rows are not next to each other, some without rules."""
    V = 3000
    c = _case(12, [300, 1, 5], V, [200, 10, 50], 4, True, True)
    c["bits"][0] = [(1 << (i + 1)) - 1 for i in range(300)]        # a chain
    c["rep"][2], c["freq"][2], c["pres"][2] = 1, 0, 0
    c["n_bias"][2] = 0                                             # nothing to do for this one
    rules, kw = _args(c)
    out = torch.full((306, V), 9.0, dtype=F32, device="cuda")
    abi.lora_logits_adjust(out, c["x"][:, :V], rules, **kw)
    _check(out, *_want(c), F32)
    gaps = torch.full_like(out, 9.0)
    seq = np.repeat(np.arange(3), c["q"])
    seq[::2] = -1
    seq[100:200:3] = -1
    abi.lora_logits_adjust(gaps, c["x"][:, :V], rules, **{**kw, "row_seq": _i32(seq)})
    keep = torch.from_numpy(seq >= 0).cuda()
    assert torch.equal(gaps[keep], out[keep]) and (gaps[~keep] == 9).all()
    # rows of two requests in turn: each row's own, whatever went before in its block
    mix = np.arange(16) % 2
    d = _case(13, [1] * 2, V, [300, 40], 6, False, False)
    d["x"] = torch.from_numpy(np.random.default_rng(1).standard_normal((16, V)).astype(np.float32)).to(BF).cuda()
    rules, _ = _args(d)
    both = torch.empty(16, V, dtype=BF, device="cuda")
    abi.lora_logits_adjust(both, d["x"], rules, row_seq=_i32(mix))
    for t in range(16):
        one = torch.empty(1, V, dtype=BF, device="cuda")
        abi.lora_logits_adjust(one, d["x"][t:t + 1], rules, row_seq=_i32([mix[t]]))
        assert torch.equal(one[0], both[t])

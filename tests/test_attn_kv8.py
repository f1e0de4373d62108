"""pillar_attn_kv8: the draft/verify step over the 8-bit cache against the plain fp64 definition.

Tolerances, from the roundings (relative to what is stated):
  * logits: products of e4m3 and f16 values are exact in fp32 and D of them are summed in fp32 (2^-23 a step, of partial sums
    bounded by sum |q k|), then two fp32 multiplications: (D + 4) 2^-23 * scale * sum |q k| covers it.  A query element is an
    f16 value once its row's largest is brought to [2^14, 2^15), but for half of f16's smallest step (2^-25):
    2^-39 * scale * max |q| * sum |k| more.
  * LSE: the row's largest logit error, the base-2 exponential (2^-21 relative and the argument's rounding, 2^-23 |s|), the
    sum over n keys (n 2^-24 relative, in chains of at most n / 4) and a logarithm: 2^-18 + (1 + |lse|) 2^-20 covers
    contexts to 4096 keys.
  * out: a probability's weight is rounded to f16 (2^-11 at half a step), relative to sum p |v|, and the result to bf16 (2^-8 at
    half a step): |error| <= 2^-8 |out| + (2^-11 + 2^-16) sum p |v|, plus, for each of at most n keys whose weight is below
    f16's normal range, half of its smallest step (2^-25) against a weight of at least 2^7 for the row's largest probability at
    the largest value scale: n 2^-32 max |code| max vs.
A row's whole output is also held to the step's stated relative error of 1e-2.
"""
import ctypes
import math

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

torch = pytest.importorskip("torch")
SENTINEL = -12345.0


def test_host_checks():
    P.build()
    lib = P.load()
    kw = dict(B=2, Hq=4, Hkv=2, D=64, k=1, max_sparse=8, max_len=64, num_slots=128)
    s, a = P.make_shape(**kw), ctypes.c_void_p(256)
    n = P.pillar_attn_workspace_bytes(s)
    good = [a] * 6 + [4] + [a] * 8 + [n, None]

    def call(shape=s, fn=lib.pillar_attn_kv8, base=None, **over):
        args = list(base or good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return fn(ctypes.byref(shape), *args)

    null = [i for i in range(15) if i not in (6, 12, 14)]
    for i in null:
        assert call(**{f"a{i}": None}) == -1, i
    for i in (0, 1, 2, 11):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (3, 4, 5, 7, 8, 9, 10, 13):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    assert call(a12=ctypes.c_void_p(260)) == -1 and call(a6=0) == -1
    assert call(a14=None) == -2 and call(a14=ctypes.c_void_p(128)) == -2 and call(a15=n - 1) == -2
    for bad in (dict(num_slots=120), dict(schedule=3), dict(schedule=4), dict(D=96), dict(Hq=3)):
        assert call(shape=P.make_shape(**{**kw, **bad})) == -1
    assert call(shape=P.make_shape(**{**kw, "B": 0}), a14=None, a15=0) == 0  # nothing to do
    run = [a] * 6 + [4] + [a] * 5 + [n, None]
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 10):
        assert call(fn=lib.pillar_attn_run_kv8, base=run, **{f"a{i}": None}) == -1, i
    assert call(fn=lib.pillar_attn_run_kv8, base=run, a11=None) == -2


class Case:
    """One batch: a shuffled block pool with random codes and scales, queries, lists."""

    def __init__(self, seed, Hq, Hkv, D, k, lens, modes, lists=None, scale_spread=2, q_scale=1.0, pow2=True, **shape):
        g = np.random.default_rng(seed)
        self.g, self.Hq, self.Hkv, self.D, self.k = g, Hq, Hkv, D, k
        self.lens, self.modes, B = np.array(lens), np.array(modes), len(lens)
        nb = -(-self.lens // 16)
        self.blocks = int(nb.sum()) + 3
        perm = g.permutation(self.blocks)
        self.table = np.full((B, int(max(1, nb.max()))), self.blocks + 7)  # out of range where no block belongs
        at = 0
        for b in range(B):
            self.table[b, :nb[b]] = perm[at:at + nb[b]]
            at += nb[b]
        x = [g.standard_normal((self.blocks, Hkv, 16, D)) for _ in "kv"]
        self.k8, self.v8 = (C.e4m3_encode(y * 100) for y in x)
        if scale_spread is None:
            self.ks, self.vs = (np.full((self.blocks, Hkv), 0.01) for _ in "kv")
        else:
            self.ks, self.vs = (2.0 ** g.integers(-7 - scale_spread, scale_spread - 6, (self.blocks, Hkv)) for _ in "kv")
        if not pow2:
            self.ks, self.vs = (y * g.uniform(0.5, 1, y.shape) for y in (self.ks, self.vs))
        self.ks, self.vs = self.ks.astype(np.float32), self.vs.astype(np.float32)
        self.T = int(np.where(self.modes == 1, k + 1, 1).sum())
        self.q = f32_to_bf16_bits((g.standard_normal((self.T, Hq, D)) * q_scale).astype(np.float32))
        if lists is None:  # a few positions of each draft context, some repeated, one list empty
            ms = max(1, int(max(lens)) // 3)
            self.cnt = np.zeros((B, Hkv), np.int64)
            self.idx = np.zeros((B, Hkv, ms), np.int64)
            for b in range(B):
                for h in range(Hkv):
                    if modes[b] == 0 and lens[b]:
                        self.cnt[b, h] = g.integers(0, ms + 1)
                        self.idx[b, h] = g.integers(0, lens[b], ms)
        else:
            self.idx, self.cnt = lists
        self.V = int((self.modes == 1).sum())
        kw = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, k=k, row_lo=min(1, k), max_sparse=self.idx.shape[2],
                  max_len=int(max(1, max(lens))), num_slots=self.blocks * 16)
        self.shape = P.make_shape(**{**kw, **shape})
        self.scale = float(self.shape.sm_scale) or D ** -0.5

    def device(self, dump=True):
        dev = lambda x, t: torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")  # noqa: E731
        n_log = int(self.Hq * (self.k + 1) * self.lens[self.modes == 1].sum())
        d = dict(q=dev(self.q.view(np.int16), torch.int16), k8=dev(self.k8, torch.uint8), v8=dev(self.v8, torch.uint8),
                 ks=dev(self.ks, torch.float32), vs=dev(self.vs, torch.float32), table=dev(self.table, torch.int32),
                 mode=dev(self.modes, torch.int32), len=dev(self.lens, torch.int32), idx=dev(self.idx, torch.int32),
                 cnt=dev(self.cnt, torch.int32),
                 out=torch.full((self.T, self.Hq, self.D), 0x7fc0, dtype=torch.int16, device="cuda"),
                 logits=torch.full((n_log + 6,), SENTINEL, device="cuda") if dump else None,
                 lse=torch.full((max(1, self.V), self.Hq, self.k + 1), SENTINEL, device="cuda"),
                 ws=torch.empty(P.pillar_attn_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda"))
        return d

    def call(self, d, stream=None):
        P.pillar_attn_kv8(self.shape, d["q"], d["k8"], d["v8"], d["ks"], d["vs"], d["table"], d["mode"], d["len"], d["idx"],
                          d["cnt"], d["out"], d["logits"], d["lse"], d["ws"], stream=stream)

    def oracle(self):
        q = bf16_bits_to_f32(self.q).astype(np.float64)
        args = (self.table, self.modes, self.lens, self.idx, self.cnt, self.k, self.scale)
        out, logits, lse = C.attn_kv8(q, self.k8, self.v8, self.ks, self.vs, *args)
        # bounds: sums of magnitudes.  sum |q k| per logit; sum p |v| per output
        mag = lambda x: x & 0x7f  # noqa: E731
        top = np.broadcast_to(np.abs(q).max(-1, keepdims=True), q.shape)
        near = (self.D + 4) * 2.0 ** -23 * C.attn_kv8(np.abs(q), mag(self.k8), self.v8, self.ks, self.vs, *args)[1]
        reach = near + 2.0 ** -39 * C.attn_kv8(top, mag(self.k8), self.v8, self.ks, self.vs, *args)[1]
        spread = C.attn_kv8(q, self.k8, mag(self.v8), self.ks, np.abs(self.vs), *args)[0]
        return out, logits, lse, reach, spread

    def check(self, d, flags=0):
        assert P.pillar_get_error(d["ws"]) == flags
        out, logits, lse, reach, spread = self.oracle()
        got = bf16_bits_to_f32(d["out"].cpu().numpy().view(np.uint16)).astype(np.float64)
        vmax = float(np.abs(C.e4m3_decode(self.v8)).max() * np.abs(self.vs).max())
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -16) * spread + max(self.lens) * 2.0 ** -32 * vmax
        assert np.all(np.abs(got - out) <= tol), f"out: {np.max(np.abs(got - out) / tol):.2f} of the bound"
        norm = np.linalg.norm(out, axis=(1, 2))
        assert np.all(np.linalg.norm(got - out, axis=(1, 2)) <= 1e-2 * norm)
        z = d["lse"].cpu().numpy().astype(np.float64)[:self.V]
        fin = np.isfinite(lse)
        assert np.array_equal(np.isneginf(z), np.isneginf(lse))
        assert np.all(np.abs(z[fin] - lse[fin]) <= 2.0 ** -18 + (1 + np.abs(lse[fin])) * 2.0 ** -20 +
                      np.max(reach[np.isfinite(reach)], initial=0))
        if d["logits"] is not None:
            lg = d["logits"].cpu().numpy().astype(np.float64)
            assert np.all(lg[len(logits):] == SENTINEL)
            lg = lg[:len(logits)]
            seen = np.isfinite(logits)
            assert np.array_equal(np.isneginf(lg), ~seen)
            assert np.all(np.abs(lg[seen] - logits[seen]) <= reach[seen] + 1e-37)


def mixed(seed, B, lo, hi, k):
    g = np.random.default_rng(seed)
    modes = (np.arange(B) % 3 != 1).astype(int)
    return np.maximum(g.integers(lo, hi + 1, B), (k + 1) * modes), modes


CASES = [  # seed, Hq, Hkv, D, k, B, lo, hi: row tiles of 16 from one to four, every group size kind
    (0, 4, 1, 64, 4, 4, 1, 200), (1, 8, 8, 128, 0, 5, 1, 130), (2, 32, 8, 128, 8, 6, 20, 300), (3, 10, 2, 128, 8, 5, 60, 260),
    (4, 8, 1, 64, 7, 4, 8, 500), (5, 8, 2, 128, 3, 5, 1, 70), (6, 2, 2, 64, 15, 4, 16, 129), (7, 16, 2, 128, 1, 4, 2, 65),
    (8, 5, 1, 64, 2, 3, 1, 1100), (9, 12, 4, 128, 12, 3, 500, 1300), (10, 24, 8, 64, 1, 9, 1, 64),
]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,Hq,Hkv,D,k,B,lo,hi", CASES)
def test_matches_the_definition(seed, Hq, Hkv, D, k, B, lo, hi):
    c = Case(seed, Hq, Hkv, D, k, *mixed(seed, B, lo, hi, k))
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("vc,dc", [(64, 64), (128, 192), (2048, 2048)])
@pytest.mark.parametrize("Hq,k", [(4, 3), (8, 7)])
def test_split_contexts_and_lists(Hq, k, vc, dc):
    c = Case(20 + vc, Hq, 1, 128, k, [700, 1500, 64, 129], [1, 0, 0, 1], verify_chunk=vc, draft_chunk=dc)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,k", [(2, 0), (8, 3), (8, 7)])
@pytest.mark.parametrize("spread,pow2", [(None, True), (12, True), (3, False)])
def test_value_scales_far_apart(Hq, k, spread, pow2):
    """Blocks whose scales differ by up to 2^24: the accumulator follows the largest met so far."""
    c = Case(40 + k, Hq, 1, 64, k, [400, 333, 17], [1, 0, 1], scale_spread=spread, q_scale=0.02 if spread == 12 else 1.0,
             pow2=pow2)
    c.ks[:] = 2.0 ** -7
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_rows_whose_maximum_grows_along_the_context():
    c = Case(50, 8, 1, 128, 3, [900, 800], [1, 0], verify_chunk=1024)
    c.ks[:] = 2.0 ** -11
    for b in range(2):  # keys grow by 2 each block: the running maximum keeps moving
        for i in range(-(-int(c.lens[b]) // 16)):
            c.ks[c.table[b, i]] = 2.0 ** (-15 + i / 6)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_queries_of_every_magnitude():
    """Rows of tiny, huge, zero and mixed queries: each is brought to f16's range by a power of two of its own."""
    c = Case(51, 8, 2, 64, 2, [100, 64], [1, 0])
    q = bf16_bits_to_f32(c.q).copy()
    q[0, 0], q[0, 1], q[0, 2] = q[0, 0] * 1e-30, 0, q[0, 2] * 2.0 ** -20
    q[1, 0], q[1, 0, 3] = q[1, 0] * 2.0 ** -12, 1.0
    q[2, 1] *= 2.0 ** 14
    q[3, :, :] *= 2.0 ** -126
    c.q = f32_to_bf16_bits(q)
    c.ks[:] = 2.0 ** -14
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_edges_empty_lists_single_tokens_and_short_verifies():
    idx = np.zeros((6, 2, 4), np.int64)
    idx[1, 0] = [4, 4, 0, 4]           # the same position again counts again
    cnt = np.zeros((6, 2), np.int64)
    cnt[1], cnt[4] = [4, 1], [1, 0]
    c = Case(60, 4, 2, 128, 2, [1, 5, 3, 64, 1, 65], [0, 0, 1, 1, 0, 1], lists=(idx, cnt))
    d = c.device()
    c.call(d)
    c.check(d)
    c = Case(61, 8, 2, 64, 4, [2, 0, 5], [1, 1, 1])  # shorter than its k+1 rows: the first rows see nothing
    d = c.device()
    c.call(d)
    c.check(d, P.FLAG_REQUEST)


@pytest.mark.gpu
@pytest.mark.parametrize("schedule", [P.SCHEDULE_DRAFT_ONLY, P.SCHEDULE_VERIFY_ONLY])
def test_half_schedules_leave_the_other_mode_alone(schedule):
    c = Case(62, 8, 2, 64, 3, [100, 200, 90], [1, 0, 1])
    d = c.device()
    c.call(d)
    half = Case(62, 8, 2, 64, 3, [100, 200, 90], [1, 0, 1], schedule=schedule)
    e = half.device()
    half.call(e)
    draft_row = 4
    rows = np.arange(9) == draft_row
    if schedule == P.SCHEDULE_VERIFY_ONLY:
        rows = ~rows
        assert torch.equal(e["logits"], d["logits"]) and torch.equal(e["lse"], d["lse"])
    else:
        assert torch.all(e["logits"] == SENTINEL) and torch.all(e["lse"] == SENTINEL)
    a, b = e["out"].cpu().numpy(), d["out"].cpu().numpy()
    np.testing.assert_array_equal(a[rows], b[rows])
    assert np.all(a[~rows] == 0x7fc0)


@pytest.mark.gpu
def test_without_the_dump_and_from_a_plan():
    c = Case(63, 8, 2, 128, 2, [300, 77, 20, 1100], [1, 0, 1, 1], verify_chunk=256)
    d, e, f = c.device(), c.device(dump=False), c.device()
    c.call(d)
    c.call(e)
    assert torch.equal(d["out"], e["out"]) and torch.equal(d["lse"], e["lse"])
    P.pillar_attn_plan(c.shape, f["mode"], f["len"], f["cnt"], f["ws"])
    for _ in range(2):  # two layers on one plan
        f["out"].fill_(0x7fc0)
        P.pillar_attn_run_kv8(c.shape, f["q"], f["k8"], f["v8"], f["ks"], f["vs"], f["table"], f["idx"], f["out"],
                              f["logits"], f["lse"], f["ws"])
        assert torch.equal(d["out"], f["out"]) and torch.equal(d["logits"], f["logits"]) and torch.equal(d["lse"], f["lse"])
    assert P.pillar_get_error(f["ws"]) == 0


@pytest.mark.gpu
def test_bad_positions_blocks_and_modes_are_flagged_and_left_out():
    c = Case(64, 4, 1, 64, 2, [100, 60, 50], [1, 0, 0])
    c.idx[1, 0, :5], c.cnt[1, 0] = [3, -1, 60, 59, 1 << 30], 5
    d = c.device()
    c.call(d)
    c.check(d, P.FLAG_INDEX)
    c = Case(65, 4, 1, 64, 2, [100, 60, 50], [1, 0, 1])
    c.table[0, 2], c.table[2, 0], c.table[1, 1] = c.blocks, -1, 1 << 30
    d = c.device()
    c.call(d)
    c.check(d, P.FLAG_SLOT)
    c = Case(66, 4, 1, 64, 2, [100, 60, 50], [1, 0, 1])  # a table too narrow for the context
    c.table = np.ascontiguousarray(c.table[:, :4])
    full = np.full((3, 7), c.blocks + 7)
    full[:, :4] = c.table
    d = c.device()
    c.call(d)
    c.table = full
    c.check(d, P.FLAG_SLOT)
    c = Case(67, 4, 1, 64, 2, [64, 60], [0, 0])  # a mode that is none: a zero row
    d = c.device()
    d["mode"][1] = 5
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == P.FLAG_REQUEST and torch.all(d["out"][1] == 0)


@pytest.mark.gpu
def test_nothing_behind_a_context_is_read():
    """NaN codes and scales in every place that no position of the batch names: rows behind a context's end in its last
    block, blocks of nobody."""
    c = Case(68, 8, 2, 128, 2, [37, 100, 16], [1, 0, 1])
    used = np.zeros((c.blocks, 16), bool)
    for b, n in enumerate(c.lens):
        for t in range(n):
            used[c.table[b, t // 16], t % 16] = True
    d = c.device()
    free = torch.tensor(~used, device="cuda")[:, None, :, None]
    for x in ("k8", "v8"):
        d[x] = torch.where(free, torch.tensor(0x7f, dtype=torch.uint8, device="cuda"), d[x])
    unused = torch.tensor(~used.any(1), device="cuda")
    d["ks"][unused] = float("nan")
    d["vs"][unused] = float("inf")
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_captured_and_on_another_stream_and_two_at_once():
    c, e = Case(69, 8, 2, 128, 3, [600, 200, 90], [1, 0, 1]), Case(70, 4, 1, 64, 3, [300, 500], [1, 1])
    want, other = c.device(), e.device()
    c.call(want)
    e.call(other)
    torch.cuda.synchronize()
    d, f, s1, s2 = c.device(), e.device(), torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        c.call(d, s1)
        e.call(f, s2)
    torch.cuda.synchronize()
    g, h = c.device(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(h):
        c.call(g)
    h.replay()
    h.replay()
    torch.cuda.synchronize()
    for k in ("out", "logits", "lse"):
        assert torch.equal(want[k], d[k]) and torch.equal(want[k], g[k]) and torch.equal(other[k], f[k]), k


@pytest.mark.gpu
def test_batches_past_one_planner_chunk():
    c = Case(71, 8, 8, 64, 1, *mixed(71, 150, 2, 60, 1))
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    c = Case(72, 4, 2, 64, 1, [40, 20], [1, 0])
    d = c.device()
    names = ("q", "k8", "v8", "ks", "vs", "table", "mode", "len", "idx", "cnt", "out", "logits", "lse")
    good = [d[n] for n in names]
    P.pillar_attn_kv8(c.shape, *good, d["ws"])
    for i in range(len(good)):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i].unsqueeze(0)):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_attn_kv8(c.shape, *args, d["ws"])
    with pytest.raises(ValueError):
        P.pillar_attn_kv8(c.shape, *good, d["ws"].cpu())
    with pytest.raises(P.PillarError):
        P.pillar_attn_kv8(c.shape, *good, d["ws"][:512])


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [64, 2048])
@pytest.mark.parametrize("what", ["query", "infinite query", "key scale", "value scale"])
def test_a_nan_is_one_however_the_context_is_split(what, chunk):
    """A NaN in what a row reads makes the row NaN, and its LSE where the scores are; the other rows are as without it.  Split,
    some of a row's partial results (a scale) or all of them (its query) are NaN."""
    c = Case(73, 8, 2, 64, 2, [700, 600, 90], [1, 0, 1], verify_chunk=chunk, draft_chunk=chunk)
    c.cnt[1], c.idx[1, :, 7] = c.idx.shape[2], 40  # the lists name a position of the block that gets the scale
    d, e = c.device(), c.device()
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == 0
    rows, heads, lse = np.zeros((c.T, 8), bool), slice(4, 8), np.zeros((2, 8, 3), bool)
    if "query" in what:
        bad = 0x7f80 if what.startswith("inf") else 0x7fc0
        e["q"][1, 0] = e["q"][3, 5] = bad  # request 0's second row, head 0; the draft row, head 5
        rows[1, 0] = rows[3, 5] = lse[0, 0, 1] = True
    else:
        e["ks" if what == "key scale" else "vs"][int(c.table[0, 2]), 1] = float("nan")
        e["ks" if what == "key scale" else "vs"][int(c.table[1, 2]), 1] = float("nan")
        rows[:4, heads] = True
        lse[0, heads] = what == "key scale"
    c.call(e)
    assert P.pillar_get_error(e["ws"]) == 0
    value = lambda x: torch.from_numpy(bf16_bits_to_f32(x["out"].cpu().numpy().view(np.uint16)))  # noqa: E731
    got, want = value(e), value(d)
    at, z = torch.from_numpy(rows), torch.from_numpy(lse)
    assert torch.all(torch.isnan(got[at])) and torch.equal(got[~at], want[~at])
    got, want = e["lse"].cpu(), d["lse"].cpu()
    assert torch.all(torch.isnan(got[z])) and torch.equal(got[~z], want[~z])


@pytest.mark.gpu
@pytest.mark.parametrize("D,Hq,Hkv,k,lens,modes,chunks", [
    (128, 4, 1, 0, [2048, 1999, 1025, 3000, 129], [1, 1, 1, 0, 1], dict(verify_chunk=2048, draft_chunk=2048)),
    (128, 8, 2, 0, [2500, 1024, 1300, 3999, 64], [1, 1, 0, 1, 1], {}),
    (128, 4, 2, 3, [1500, 700, 257, 64], [1, 0, 1, 1], dict(verify_chunk=64, draft_chunk=64)),
    (128, 2, 2, 1, [2100, 1800, 333], [0, 1, 0], dict(verify_chunk=512, draft_chunk=128)),
    (128, 8, 1, 0, [640, 641, 639, 900], [1, 1, 1, 1], dict(verify_chunk=640)),
    (64, 8, 1, 0, [2500, 1300, 257], [1, 0, 1], dict(verify_chunk=256, draft_chunk=192)),
    (64, 2, 1, 3, [1700, 2048], [1, 1], dict(verify_chunk=2048)),
])
def test_items_of_at_most_eight_rows_over_long_contexts(D, Hq, Hkv, k, lens, modes, chunks):
    """Up to sixteen steps an item: the stages wrap, positions are resolved past the first steps, and split items join."""
    c = Case(80, Hq, Hkv, D, k, lens, modes, **chunks)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,k", [(8, 0), (16, 3), (24, 2)])
def test_more_items_than_ctas(Hq, k):
    """Every CTA goes through several items, long and short ones, some of one step: each takes the next from the queue while
    the present one runs."""
    g = np.random.default_rng(81)
    B = 90
    lens = np.where(np.arange(B) % 4 == 0, g.integers(600, 1100, B), g.integers(k + 1, 140, B))
    c = Case(81, Hq, 8, 128, k, lens, (np.arange(B) % 5 != 2).astype(int), verify_chunk=256)
    d = c.device()
    c.call(d)
    c.check(d)

"""pillar_attn_kv4: the draft/verify step over the 4-bit cache against the plain fp64 definition.

Tolerances, from the roundings (relative to what is stated):
  * logits: a key's values are exact in f16, a query's are once its row's largest is brought to [2^14, 2^15), but for half of
    f16's smallest step (2^-25): 2^-39 * scale * max |q| * sum |k|.  Their products are exact in fp32 and D of them are summed in
    fp32 (2^-23 a step, of partial sums bounded by sum |q k|), then at most two fp32 multiplications:
    (D + 4) 2^-23 * scale * sum |q k| covers it.
  * LSE: the row's largest logit error, the base-2 exponential (2^-21 relative and the argument's rounding, 2^-23 |s|), the
    sum over n keys (n 2^-24 relative, in chains of at most n / 4) and a logarithm: 2^-18 + (1 + |lse|) 2^-20 covers
    contexts to 4096 keys.
  * out: a probability is rounded to f16 (2^-11 at half a step), relative to sum p |v|, and the result to bf16 (2^-8 at half a
    step): |error| <= 2^-8 |out| + (2^-11 + 2^-16) sum p |v|, plus, for each of at most n keys whose weight is below f16's
    normal range, half of its smallest step (2^-25) against a weight of at least 2^6 for the row's largest probability:
    n 2^-31 max |v|; plus what the logits' own error does to a probability: 2 * max logit error * sum p |v|.
A row's whole output is also held to the step's stated relative error of 1e-2.
"""
import ctypes

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

    def call(shape=s, fn=lib.pillar_attn_kv4, base=None, **over):
        args = list(base or good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return fn(ctypes.byref(shape), *args)

    null = [i for i in range(15) if i not in (6, 12, 14)]
    for i in null:
        assert call(**{f"a{i}": None}) == -1, i
    for i in (0, 1, 2, 11):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (3, 4):
        assert call(**{f"a{i}": ctypes.c_void_p(260)}) == -1
    for i in (5, 7, 8, 9, 10, 13):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    assert call(a12=ctypes.c_void_p(260)) == -1 and call(a6=0) == -1
    assert call(a14=None) == -2 and call(a14=ctypes.c_void_p(128)) == -2 and call(a15=n - 1) == -2
    for bad in (dict(num_slots=120), dict(schedule=3), dict(schedule=4), dict(D=96), dict(Hq=3)):
        assert call(shape=P.make_shape(**{**kw, **bad})) == -1
    assert call(shape=P.make_shape(**{**kw, "B": 0}), a14=None, a15=0) == 0  # nothing to do
    run = [a] * 6 + [4] + [a] * 5 + [n, None]
    for i in (0, 1, 2, 3, 4, 5, 7, 8, 10):
        assert call(fn=lib.pillar_attn_run_kv4, base=run, **{f"a{i}": None}) == -1, i
    assert call(fn=lib.pillar_attn_run_kv4, base=run, a11=None) == -2


class Case:
    """One batch: a shuffled block pool with random codes and scales, queries, lists."""

    def __init__(self, seed, Hq, Hkv, D, k, lens, modes, lists=None, q_scale=1.0, spread=4, **shape):
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
        # codes as a normal distribution gives them under its group's largest, scales around 0.4 (byte 109 is 0.40625)
        self.k4, self.v4 = (C.kv4_codes(np.clip(g.standard_normal((self.blocks, Hkv, 16, D)) * 2.4, -6, 6)) for _ in "kv")
        self.ks, self.vs = (g.integers(109 - spread, 110 + spread, (self.blocks, Hkv, 16, D // 16)).astype(np.uint8)
                            for _ in "kv")
        self.T = int(np.where(self.modes == 1, k + 1, 1).sum())
        self.q = f32_to_bf16_bits((g.standard_normal((self.T, Hq, D)) * q_scale).astype(np.float32))
        if lists is None:  # a few positions of each draft context, some repeated, some lists empty
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
        return dict(q=dev(self.q.view(np.int16), torch.int16), k4=dev(C.kv4_pack(self.k4), torch.uint8),
                    v4=dev(C.kv4_pack(self.v4), torch.uint8), ks=dev(self.ks, torch.uint8), vs=dev(self.vs, torch.uint8),
                    table=dev(self.table, torch.int32), mode=dev(self.modes, torch.int32), len=dev(self.lens, torch.int32),
                    idx=dev(self.idx, torch.int32), cnt=dev(self.cnt, torch.int32),
                    out=torch.full((self.T, self.Hq, self.D), 0x7fc0, dtype=torch.int16, device="cuda"),
                    logits=torch.full((n_log + 6,), SENTINEL, device="cuda") if dump else None,
                    lse=torch.full((max(1, self.V), self.Hq, self.k + 1), SENTINEL, device="cuda"),
                    ws=torch.empty(P.pillar_attn_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda"))

    def call(self, d, stream=None):
        P.pillar_attn_kv4(self.shape, d["q"], d["k4"], d["v4"], d["ks"], d["vs"], d["table"], d["mode"], d["len"], d["idx"],
                          d["cnt"], d["out"], d["logits"], d["lse"], d["ws"], stream=stream)

    def oracle(self):
        q = bf16_bits_to_f32(self.q).astype(np.float64)
        k, v = C.kv4_decode(self.k4, self.ks), C.kv4_decode(self.v4, self.vs)
        args = (self.table, self.modes, self.lens, self.idx, self.cnt, self.k, self.scale)
        out, logits, lse = C.attn_cache(q, k, v, *args)
        # bounds: sums of magnitudes.  sum |q k| per logit; sum p |v| per output
        top = np.broadcast_to(np.abs(q).max(-1, keepdims=True), q.shape)
        reach = (self.D + 4) * 2.0 ** -23 * C.attn_cache(np.abs(q), np.abs(k), v, *args)[1]
        reach = reach + 2.0 ** -39 * C.attn_cache(top, np.abs(k), v, *args)[1]
        spread = C.attn_cache(q, k, np.abs(v), *args)[0]
        return out, logits, lse, reach, spread

    def check(self, d, flags=0):
        assert P.pillar_get_error(d["ws"]) == flags
        out, logits, lse, reach, spread = self.oracle()
        got = bf16_bits_to_f32(d["out"].cpu().numpy().view(np.uint16)).astype(np.float64)
        vmax = float(np.abs(C.kv4_decode(self.v4, self.vs)).max())
        # (draft rows have no logits to bound: |q . k| <= D |q| |k|, the same factors)
        q, k = np.abs(bf16_bits_to_f32(self.q)).max(), np.abs(C.kv4_decode(self.k4, self.ks)).max()
        off = min(2 * (self.D + 4) * 2.0 ** -23 * self.scale * self.D * float(q) * float(k), 2.0 ** -11)
        tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -11 + 2.0 ** -16 + off) * spread + max(self.lens) * 2.0 ** -31 * vmax
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


CASES = [  # seed, Hq, Hkv, D, k, B, lo, hi: one to 64 rows, every group size kind
    (0, 4, 1, 64, 4, 4, 1, 200), (1, 8, 8, 128, 0, 5, 1, 130), (2, 32, 8, 128, 8, 6, 20, 300), (3, 10, 2, 128, 8, 5, 60, 260),
    (4, 8, 1, 64, 7, 4, 8, 500), (5, 8, 2, 128, 3, 5, 1, 70), (6, 2, 2, 64, 15, 4, 16, 129), (7, 16, 2, 128, 1, 4, 2, 65),
    (8, 5, 1, 64, 2, 3, 1, 1100), (9, 12, 4, 128, 12, 3, 500, 1300), (10, 24, 8, 64, 1, 9, 1, 64), (11, 4, 4, 128, 62, 3, 70, 400),
    (12, 8, 1, 128, 7, 4, 8, 500),
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
@pytest.mark.parametrize("D", [64, 128])
def test_scales_over_their_whole_range(Hq, k, D):
    """Value scales of every byte that is written, key scales of every byte up to 0.5."""
    c = Case(40 + k, Hq, 1, D, k, [400, 333, 17], [1, 0, 1], q_scale=0.3)
    c.vs[:] = c.g.integers(0, C.TOP4 + 1, c.vs.shape)
    c.ks[:] = c.g.integers(0, 113, c.ks.shape)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,k", [(8, 3), (4, 0)])
def test_rows_whose_maximum_grows_along_the_context(Hq, k):
    c = Case(50, Hq, 1, 128, k, [900, 800], [1, 0], verify_chunk=1024)
    for b in range(2):  # keys grow from block to block: the running maximum keeps moving
        for i in range(-(-int(c.lens[b]) // 16)):
            c.ks[c.table[b, i]] = 40 + 90 * i // 57
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
    c.ks[:] = 8  # 2^-14
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
        P.pillar_attn_run_kv4(c.shape, f["q"], f["k4"], f["v4"], f["ks"], f["vs"], f["table"], f["idx"], f["out"],
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
@pytest.mark.parametrize("D", [64, 128])
def test_nothing_behind_a_context_is_read(D):
    """NaN scales in every place that no position of the batch names: rows behind a context's end in its last block, blocks
    of nobody."""
    c = Case(68, 8, 2, D, 2, [37, 100, 16], [1, 0, 1])
    used = np.zeros((c.blocks, 16), bool)
    for b, n in enumerate(c.lens):
        for t in range(n):
            used[c.table[b, t // 16], t % 16] = True
    d = c.device()
    free = torch.tensor(~used, device="cuda")[:, None, :, None]
    for x in ("ks", "vs"):
        d[x] = torch.where(free, torch.tensor(0xff, dtype=torch.uint8, device="cuda"), d[x])
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
    names = ("q", "k4", "v4", "ks", "vs", "table", "mode", "len", "idx", "cnt", "out", "logits", "lse")
    good = [d[n] for n in names]
    P.pillar_attn_kv4(c.shape, *good, d["ws"])
    for i in range(len(good)):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i].unsqueeze(0)):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_attn_kv4(c.shape, *args, d["ws"])
    with pytest.raises(ValueError):
        P.pillar_attn_kv4(c.shape, *good, d["ws"].cpu())
    with pytest.raises(P.PillarError):
        P.pillar_attn_kv4(c.shape, *good, d["ws"][:512])


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [64, 2048])
@pytest.mark.parametrize("what", ["query", "infinite query", "key scale", "value scale"])
def test_a_nan_is_one_however_the_context_is_split(what, chunk):
    """A NaN in what a row reads makes the row NaN (a value scale: in its sixteen dimensions), and its LSE where the scores
    are; the other rows are as without it.  Split, some of a row's partial results (a scale) or all of them (its query) are NaN."""
    c = Case(73, 8, 2, 64, 2, [700, 600, 90], [1, 0, 1], verify_chunk=chunk, draft_chunk=chunk)
    c.cnt[1], c.idx[1, :, 7] = c.idx.shape[2], 40  # the lists name a position of the block that gets the scale
    d, e = c.device(), c.device()
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == 0
    rows, heads, lse = np.zeros((c.T, 8, 64), bool), slice(4, 8), np.zeros((2, 8, 3), bool)
    if "query" in what:
        bad = 0x7f80 if what.startswith("inf") else 0x7fc0
        e["q"][1, 0] = e["q"][3, 5] = bad  # request 0's second row, head 0; the draft row, head 5
        rows[1, 0] = rows[3, 5] = lse[0, 0, 1] = True
    else:
        for b in (0, 1):
            e["ks" if what == "key scale" else "vs"][int(c.table[b, 2]), 1, 8, 1] = 0xff  # position 40
        if what == "key scale":
            rows[:4, heads], lse[0, heads] = True, True
        else:
            rows[:4, heads, 16:32] = True
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
    c = Case(80, Hq, Hkv, D, k, lens, modes, **chunks)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,k", [(8, 0), (16, 3), (24, 2), (32, 12)])
def test_more_items_than_ctas(Hq, k):
    """Every CTA goes through several items, long and short ones, of many rows and of few."""
    g = np.random.default_rng(81)
    B = 90
    lens = np.where(np.arange(B) % 4 == 0, g.integers(600, 1100, B), g.integers(k + 1, 140, B))
    c = Case(81, Hq, 8, 128, k, lens, (np.arange(B) % 5 != 2).astype(int), verify_chunk=256)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,k,B,lo,hi,shape", [
    (32, 8, 128, 8, 150, 9, 128, {}),                   # a tile an item, many items a CTA
    (24, 8, 64, 6, 170, 7, 300, {}),                    # one to three tiles
    (20, 4, 64, 4, 40, 5, 900, dict(verify_chunk=64)),  # pieces of half a tile
    (8, 2, 128, 2, 60, 3, 400, dict(verify_chunk=64, draft_chunk=64)),  # 12 rows, and lists
    (6, 1, 64, 2, 9, 1, 700, {}),                       # 18 rows: a group of eight with two in it
])
def test_short_items_in_numbers(Hq, Hkv, D, k, B, lo, hi, shape):
    c = Case(90, Hq, Hkv, D, k, *mixed(90, B, lo, hi, k), **shape)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_many_rows_from_a_plan_without_a_dump_and_captured(D):
    c = Case(91, 32, 4, D, 4, [300, 77, 20, 1100], [1, 0, 1, 1], verify_chunk=256)
    d, e, f = c.device(), c.device(dump=False), c.device()
    c.call(d)
    c.check(d)
    c.call(e)
    assert torch.equal(d["out"], e["out"]) and torch.equal(d["lse"], e["lse"])
    P.pillar_attn_plan(c.shape, f["mode"], f["len"], f["cnt"], f["ws"])
    run = lambda: P.pillar_attn_run_kv4(c.shape, f["q"], f["k4"], f["v4"], f["ks"], f["vs"], f["table"], f["idx"], f["out"],  # noqa: E731
                                        f["logits"], f["lse"], f["ws"])
    run()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        run()
    for _ in range(2):
        for name in ("out", "logits", "lse"):
            assert torch.equal(d[name], f[name]), name
            f[name].fill_(0x7fc0 if name == "out" else SENTINEL)
        g.replay()
    assert P.pillar_get_error(f["ws"]) == 0


@pytest.mark.gpu
def test_waits_that_run_out_anywhere_in_the_pipeline():
    """Bounds from one microsecond to more than the call takes, in items of more than sixteen rows: every CTA ends, the call says so
    and a whole one that follows at once on the stream, on a workspace of its own, is right; so is the next on the same workspace."""
    g = np.random.default_rng(92)
    big = dict(seed=92, Hq=32, Hkv=8, D=128, k=6, lens=g.integers(600, 1500, 24), modes=(np.arange(24) % 4 != 1).astype(int))
    short, full = Case(**big, wait_timeout_us=1), Case(**big)
    small = Case(93, 32, 8, 128, 4, [300, 90, 400], [1, 0, 1])
    want, d, after = small.device(), full.device(), small.device()
    small.call(want)
    small.check(want)
    seen = 0
    for bound in (1, 2, 3, 4, 6, 9, 13, 20, 30, 50, 5000):
        short.shape.wait_timeout_us = bound
        short.call(d)
        small.call(after)
        flags = P.pillar_get_error(d["ws"])
        assert flags & ~P.FLAG_TIMEOUT == 0 and P.pillar_get_error(after["ws"]) == 0, bound
        seen |= flags if bound == 1 else 0
        for name in ("out", "logits", "lse"):
            assert torch.equal(after[name], want[name]), (bound, name)
            after[name].fill_(0x7fc0 if name == "out" else SENTINEL)
    assert seen == P.FLAG_TIMEOUT, "no wait ran out"
    d["out"].fill_(0x7fc0)
    d["logits"].fill_(SENTINEL)
    d["lse"].fill_(SENTINEL)
    full.call(d)
    full.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,k,shape", [
    (8, 2, 128, 4, {}), (6, 1, 64, 2, dict(verify_chunk=64)), (8, 2, 64, 5, dict(verify_chunk=256)), (8, 1, 128, 2, {}), (10, 2, 128, 2, {}),
    (16, 2, 128, 2, dict(verify_chunk=2048)), (7, 1, 64, 3, {}),
])
def test_up_to_32_rows_without_a_dump(Hq, Hkv, D, k, shape):
    """15 to 28 rows a verify item; a first item of fewer keys than warps have, one of many pieces."""
    c = Case(94, Hq, Hkv, D, k, [k + 1, 40, 700, 2100, 129], [1, 0, 1, 1, 1], **shape)
    d = c.device(dump=False)
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("schedule", [P.SCHEDULE_UNIFIED, P.SCHEDULE_DRAFT_ONLY, P.SCHEDULE_VERIFY_ONLY])
@pytest.mark.parametrize("Hq,Hkv,k", [(8, 2, 0), (8, 2, 2), (32, 4, 4)])
def test_runs_on_one_plan_that_splits_nothing(Hq, Hkv, k, schedule):
    """Contexts of one item each, more items than CTAs: a run on the plan of an earlier one finds the whole queue again."""
    g = np.random.default_rng(95)
    B = 400
    c = Case(95, Hq, Hkv, 64, k, g.integers(k + 1, 100, B), g.integers(0, 2, B), schedule=schedule)
    full = Case(95, Hq, Hkv, 64, k, c.lens, c.modes)
    d, f = full.device(), c.device()
    full.call(d)
    assert P.pillar_get_error(d["ws"]) == 0
    off = np.concatenate([[0], np.cumsum(np.where(c.modes == 1, k + 1, 1))])
    rows = torch.zeros(c.T, dtype=torch.bool, device="cuda")
    for b in range(B):
        rows[off[b]:off[b + 1]] = bool(schedule == P.SCHEDULE_UNIFIED or (c.modes[b] == 1) == (schedule == P.SCHEDULE_VERIFY_ONLY))
    P.pillar_attn_plan(c.shape, f["mode"], f["len"], f["cnt"], f["ws"])
    for _ in range(3):
        f["out"].fill_(0x7fc0)
        f["logits"].fill_(SENTINEL)
        f["lse"].fill_(SENTINEL)
        P.pillar_attn_run_kv4(c.shape, f["q"], f["k4"], f["v4"], f["ks"], f["vs"], f["table"], f["idx"], f["out"], f["logits"],
                              f["lse"], f["ws"])
        assert torch.equal(f["out"][rows], d["out"][rows]) and torch.all(f["out"][~rows] == 0x7fc0)
        for name in ("logits", "lse"):
            assert torch.all(f[name] == SENTINEL) if schedule == P.SCHEDULE_DRAFT_ONLY else torch.equal(f[name], d[name]), name
    assert P.pillar_get_error(f["ws"]) == 0

"""pillar_prompt_attn: causal attention over packed prompts against the plain fp64 definition.

Tolerances, from the roundings:
  * lse: the scores are sums of D exact products in fp32 (2^-23 a step of partial sums bounded by sum |q k|) times the scale,
    the base-2 exponential 2^-21 relative with its argument rounded (2^-23 |s|), n terms summed in fp32 and a logarithm:
    (D + 4) 2^-23 scale max sum |q k| + 2^-18 + (1 + |lse|) 2^-20.
  * out: probabilities are rounded to bf16 (2^-8 at half a step), relative to sum p |v|, their sum is kept in fp32 of the
    unrounded ones, and the result is rounded to bf16: |error| <= 2^-8 |out| + (2^-8 + 2^-16 + 2 lse-error) sum p |v|.
A row's whole output is also held to a relative error of 1e-2.
"""
import ctypes

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

torch = pytest.importorskip("torch")
SENTINEL = -12345.0


def shape_of(B, Hq, Hkv, D, max_len, **kw):
    return P.make_shape(B=B, Hq=Hq, Hkv=Hkv, D=D, k=0, row_lo=0, max_sparse=0, max_len=max_len, num_slots=1, **kw)


def test_host_checks():
    P.build()
    lib = P.load()
    s, a = shape_of(2, 4, 2, 64, 100), ctypes.c_void_p(256)
    n = P.pillar_prompt_attn_workspace_bytes(s, 50)
    assert n > 0 and n % 256 == 0
    good = [a, 0, a, 0, a, 0, 50, a, a, a, a, n, None]

    def call(shape=s, **over):
        args = list(good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return lib.pillar_prompt_attn(ctypes.byref(shape), *args)

    for i in (0, 2, 4, 7, 8):
        assert call(**{f"a{i}": None}) == -1
    for i in (0, 2, 4, 8):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (7, 9):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    for i, short in ((1, 128), (3, 64), (5, 64)):
        for stride in (short, 260, -512):
            assert call(**{f"a{i}": stride}) == -1
    assert call(a6=-1) == -1
    assert call(a10=None) == -2 and call(a10=ctypes.c_void_p(128)) == -2 and call(a11=n - 1) == -2
    assert call(a6=0, a10=None, a11=0) == 0 and call(shape=shape_of(0, 4, 2, 64, 100), a10=None, a11=0) == 0
    for bad in (dict(D=96), dict(Hq=3), dict(Hq=18), dict(max_len=0)):
        assert call(shape=shape_of(**{**dict(B=2, Hq=4, Hkv=2, D=64, max_len=100), **bad})) == -1
    with pytest.raises(P.PillarError):
        P.pillar_prompt_attn_workspace_bytes(s, -1)


class Case:
    def __init__(self, seed, Hq, Hkv, D, lens, gap=0, tail=3, pad=0, scale=1.0, **shape):
        g = np.random.default_rng(seed)
        self.Hq, self.Hkv, self.D = Hq, Hkv, D
        self.off = gap + np.concatenate([[0], np.cumsum(lens)])  # `gap` rows before the first sequence, `tail` behind the last
        self.n = int(self.off[-1]) + tail
        draw = lambda h: f32_to_bf16_bits((g.standard_normal((self.n, h, D)) * scale).astype(np.float32))  # noqa: E731
        self.q, self.k, self.v = draw(Hq), draw(Hkv), draw(Hkv)
        self.pad = pad
        self.shape = shape_of(len(lens), Hq, Hkv, D, max(1, max(lens)), **shape)
        self.scale = float(self.shape.sm_scale) or D ** -0.5

    def device(self, lse=True, q=None, k=None, v=None):
        def dev(x):
            w = x.shape[1] * self.D
            wide = torch.full((self.n, w + self.pad), 0x7fc0, dtype=torch.int16)
            wide[:, :w] = torch.from_numpy(x.reshape(self.n, w).view(np.int16))
            return wide.cuda()[:, :w].unflatten(1, (x.shape[1], self.D))
        return dict(q=dev(self.q if q is None else q), k=dev(self.k if k is None else k), v=dev(self.v if v is None else v),
                    off=torch.tensor(self.off, dtype=torch.int32, device="cuda"),
                    out=torch.full((self.n, self.Hq, self.D), 0x7fc1, dtype=torch.int16, device="cuda"),
                    lse=torch.full((self.n, self.Hq), SENTINEL, device="cuda") if lse else None,
                    ws=torch.empty(P.pillar_prompt_attn_workspace_bytes(self.shape, self.n), dtype=torch.uint8, device="cuda"))

    def call(self, d, stream=None):
        P.pillar_prompt_attn(self.shape, d["q"], d["k"], d["v"], d["off"], d["out"], d["lse"], d["ws"], stream=stream)

    def check(self, d, flags=0, off=None):
        assert P.pillar_get_error(d["ws"]) == flags
        off = self.off if off is None else off
        q, k, v = (bf16_bits_to_f32(x).astype(np.float64) for x in (self.q, self.k, self.v))
        got = bf16_bits_to_f32(d["out"].cpu().numpy().view(np.uint16)).astype(np.float64)
        z = None if d["lse"] is None else d["lse"].cpu().numpy().astype(np.float64)
        G, seen = self.Hq // self.Hkv, np.zeros(self.n, bool)
        for a, e in zip(off[:-1], off[1:]):
            a, e = int(a), int(e)
            if a == e:
                continue
            seen[a:e] = True
            mask = np.tril(np.ones((e - a, e - a), bool))
            for h in range(self.Hq):
                s = self.scale * (q[a:e, h] @ k[a:e, h // G].T)
                reach = self.scale * np.where(mask, np.abs(q[a:e, h]) @ np.abs(k[a:e, h // G]).T, 0).max()
                s = np.where(mask, s, -np.inf)
                m = s.max(1, keepdims=True)
                p = np.exp(s - m)
                l = p.sum(1, keepdims=True)
                out, spread, lse = p @ v[a:e, h // G] / l, p @ np.abs(v[a:e, h // G]) / l, (m + np.log(l))[:, 0]
                slack = (self.D + 4) * 2.0 ** -23 * reach + 2.0 ** -18
                tol = 2.0 ** -8 * np.abs(out) + (2.0 ** -8 + 2.0 ** -16 + 2 * slack) * spread + 1e-30
                err = np.abs(got[a:e, h] - out)
                assert np.all(err <= tol), f"head {h} of rows {a}..{e}: {np.max(err / tol):.2f} of the bound"
                assert np.all(np.linalg.norm(got[a:e, h] - out, axis=1) <= 1e-2 * np.linalg.norm(out, axis=1) + 1e-30)
                if z is not None:
                    assert np.all(np.abs(z[a:e, h] - lse) <= slack + (1 + np.abs(lse)) * 2.0 ** -20)
        assert np.all(d["out"].cpu().numpy()[~seen] == 0x7fc1)  # rows of no sequence
        if z is not None:
            assert np.all(z[~seen] == SENTINEL)


def test_the_check_agrees_with_the_oracle():
    g = np.random.default_rng(1)
    q, k, v = g.standard_normal((9, 4, 8)), g.standard_normal((9, 2, 8)), g.standard_normal((9, 2, 8))
    out, lse = C.prompt_attn(q, k, v, [0, 6], 0.4)
    s = np.where(np.tril(np.ones((6, 6), bool)), 0.4 * (q[:6, 3] @ k[:6, 1].T), -np.inf)
    p = np.exp(s - s.max(1, keepdims=True))
    np.testing.assert_allclose(out[:6, 3], p @ v[:6, 1] / p.sum(1, keepdims=True), rtol=1e-12)
    np.testing.assert_allclose(lse[:6, 3], s.max(1) + np.log(p.sum(1)), rtol=1e-12)


CASES = [  # seed, Hq, Hkv, D, lengths, gap, token padding
    (0, 1, 1, 64, [1], 0, 0), (1, 4, 1, 64, [1, 2, 63, 64, 65, 127, 128, 129], 0, 0), (2, 8, 8, 128, [200], 5, 0),
    (3, 10, 2, 128, [255, 256, 257, 1], 0, 8), (4, 8, 1, 64, [0, 300, 0, 5, 0], 2, 24), (5, 16, 8, 128, [37], 0, 0),
    (6, 4, 2, 128, [1100, 3, 640], 0, 64), (7, 5, 1, 64, [513, 2, 1025], 1, 0), (8, 2, 2, 128, [384, 385, 383, 511], 0, 0),
    (9, 2, 1, 64, [17] * 40, 0, 0),
]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,Hq,Hkv,D,lens,gap,pad", CASES)
def test_matches_the_definition(seed, Hq, Hkv, D, lens, gap, pad):
    c = Case(seed, Hq, Hkv, D, lens, gap=gap, pad=pad)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_a_long_sequence_and_no_lse(D):
    c = Case(20, 2, 1, D, [2900], tail=0)
    d = c.device(lse=False)
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("scale", [0.02, 6.0])
def test_flat_and_peaked_rows(scale):
    """Nearly equal scores; and scores in the hundreds, whose running maximum moves by more than 2^8 between tiles."""
    c = Case(21, 2, 1, 128, [700], scale=scale)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_keys_that_grow_along_the_sequence():
    c = Case(22, 2, 2, 64, [900, 130])
    x = bf16_bits_to_f32(c.k)
    x *= np.linspace(0.2, 12, c.n)[:, None, None].astype(np.float32)
    c.k = f32_to_bf16_bits(x)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_a_given_scale():
    c = Case(23, 4, 4, 64, [150, 20], sm_scale=0.031)
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_sequences_do_not_meet():
    """NaN and infinities in the neighbours, before, between and behind: every other sequence is as without them."""
    lens = [100, 60, 300, 5]
    c = Case(24, 4, 2, 128, lens)
    d = c.device()
    c.call(d)
    bad = np.zeros(c.n, bool)
    bad[c.off[1]:c.off[2]] = bad[c.off[3]:c.off[4]] = bad[c.off[4]:] = True
    q, k, v = c.q.copy(), c.k.copy(), c.v.copy()
    q[bad], k[bad], v[bad] = 0x7fc0, 0x7f80, 0xffc0  # NaN, infinity, NaN
    e = c.device(q=q, k=k, v=v)
    c.call(e)
    torch.cuda.synchronize()
    keep = torch.tensor(~bad, device="cuda")
    assert torch.equal(d["out"][keep], e["out"][keep]) and torch.equal(d["lse"][keep], e["lse"][keep])


@pytest.mark.gpu
def test_bad_offsets_are_flagged_and_skipped():
    c = Case(25, 2, 1, 64, [50, 40, 30, 20])
    for i, value, kept in ((1, 200, [2, 3]), (2, 10, [0, 3]), (4, c.n + 1, [0, 1, 2]), (0, -1, [1, 2, 3])):
        off = c.off.copy()
        off[i] = value
        d = c.device()
        d["off"][i] = value
        c.call(d)
        torch.cuda.synchronize()
        assert P.pillar_get_error(d["ws"]) == P.FLAG_REQUEST
        w = c.device()
        c.call(w)
        for b in kept:
            a, e = int(c.off[b]), int(c.off[b + 1])
            assert torch.equal(d["out"][a:e], w["out"][a:e]), (i, b)
    c = Case(26, 2, 1, 64, [50, 40])
    c.shape.max_len = 45  # the first is longer
    d = c.device()
    c.call(d)
    c.check(d, P.FLAG_REQUEST, off=c.off[1:])


@pytest.mark.gpu
def test_captured_and_on_another_stream_and_two_at_once():
    c, e = Case(27, 8, 2, 128, [400, 37, 130]), Case(28, 4, 1, 64, [300, 260])
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
    for k in ("out", "lse"):
        assert torch.equal(want[k], d[k]) and torch.equal(want[k], g[k]) and torch.equal(other[k], f[k]), k


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    c = Case(29, 4, 2, 64, [20, 10])
    d = c.device()
    good = [d[x] for x in ("q", "k", "v", "off", "out", "lse")]
    P.pillar_prompt_attn(c.shape, *good, d["ws"])
    for i in range(6):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i].unsqueeze(0), good[i][:-1]):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_prompt_attn(c.shape, *args, d["ws"])
    with pytest.raises(ValueError):
        P.pillar_prompt_attn(c.shape, d["q"].transpose(1, 2).contiguous().transpose(1, 2), *good[1:], d["ws"])
    with pytest.raises(P.PillarError):
        P.pillar_prompt_attn(c.shape, *good, d["ws"][:256])


@pytest.mark.gpu
def test_a_wait_that_runs_out_is_flagged_and_the_next_call_is_right():
    """With a bound of a microsecond, less than any tile takes from memory, some wait of the pipeline gives up: the call
    returns with PILLAR_FLAG_TIMEOUT, and the next one on the same buffers, with the default bound, is whole."""
    c = Case(90, 8, 2, 128, [700, 300, 513])
    d = c.device()
    c.shape.wait_timeout_us = 1
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == P.FLAG_TIMEOUT
    c.shape.wait_timeout_us = 0
    d["out"].fill_(0x7fc1)
    d["lse"].fill_(SENTINEL)
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_a_largest_length_beyond_every_sequence():
    c = Case(91, 4, 1, 64, [700, 40, 1200])
    c.shape.max_len = 2 ** 31 - 1
    d = c.device()
    c.call(d)
    c.check(d)


@pytest.mark.gpu
def test_sequences_that_overlap_beyond_the_workspace_are_skipped():
    """Offsets up and down again: every other sequence is all of the rows, far more tiles than n rows can have."""
    c = Case(92, 2, 1, 64, [20] * 64)
    off = np.zeros(65, np.int64)
    off[1::2] = c.off[-1]
    d = c.device()
    d["off"].copy_(torch.tensor(off, dtype=torch.int32))
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == P.FLAG_REQUEST
    assert torch.all(d["out"] == 0x7fc1) and torch.all(d["lse"] == SENTINEL)
    d["off"].copy_(torch.tensor(c.off, dtype=torch.int32))
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("D,lens", [(128, [256, 130, 1, 200] * 40), (64, [384, 140, 257, 60] * 40), (128, [37])])
def test_calls_whose_last_copies_are_issued_before_a_wait_runs_out(D, lens):
    """Units of so few key tiles that the load thread never waits for a slot: it has issued everything when the products' or the
    softmax's wait gives up, and still sees its copies land before the CTA leaves its shared memory to the next one, here one
    of a whole call that follows on the stream at once."""
    c, e = Case(93, 4, 2, D, lens), Case(94, 4, 2, D, lens)
    d, f, want = c.device(), e.device(), e.device()
    e.call(want)
    for _ in range(4):
        c.shape.wait_timeout_us = 1
        c.call(d)
        e.call(f)
        assert P.pillar_get_error(d["ws"]) & ~P.FLAG_TIMEOUT == 0 and P.pillar_get_error(f["ws"]) == 0
        assert torch.equal(f["out"], want["out"]) and torch.equal(f["lse"], want["lse"])
        f["out"].fill_(0x7fc1)
        f["lse"].fill_(SENTINEL)
    c.shape.wait_timeout_us = 0
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128])
def test_waits_that_run_out_anywhere_in_the_pipeline(D):
    """Bounds from one microsecond to more than the whole call takes, so that waits give up at the start, in the middle and
    hardly at all: a warp goes on or gives up as one, and a whole call that follows at once is right."""
    c, e = Case(95, 4, 2, D, [700, 1300, 5, 900] * 20), Case(96, 4, 2, D, [300, 41] * 30)
    d, f, want = c.device(), e.device(), e.device()
    e.call(want)
    for bound in (1, 2, 3, 4, 6, 9, 13, 20, 30, 50, 400):
        c.shape.wait_timeout_us = bound
        c.call(d)
        e.call(f)
        assert P.pillar_get_error(d["ws"]) & ~P.FLAG_TIMEOUT == 0 and P.pillar_get_error(f["ws"]) == 0, bound
        assert torch.equal(f["out"], want["out"]) and torch.equal(f["lse"], want["lse"]), bound
        f["out"].fill_(0x7fc1)
        f["lse"].fill_(SENTINEL)


def test_token_counts_past_32_bits_are_refused():
    s = shape_of(2, 4, 2, 64, 100)
    for n in (2 ** 31, 2 ** 32 + 5, -2 ** 31 - 1):
        with pytest.raises(ValueError):
            P.pillar_prompt_attn_workspace_bytes(s, n)
    with pytest.raises(P.PillarError):
        P.pillar_prompt_attn_workspace_bytes(s, -2 ** 31)

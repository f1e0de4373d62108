"""pillar_kv4_read and pillar_kv8_read: positions of a cache as bf16 rows.  4-bit values are exact in bf16; 8-bit ones are one
fp32 product (exact: four significant bits times a power of two, or rounded by 2^-24) rounded to bf16."""
import ctypes

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from tests.test_kv4_append import cache, dev, shape_of
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

torch = pytest.importorskip("torch")
MARK = 0x1234  # bf16 bits of rows that are to stay


@pytest.mark.parametrize("fmt,align", [("kv4", 8), ("kv8", 4)])
def test_host_checks(fmt, align):
    P.build()
    fn = getattr(P.load(), f"pillar_{fmt}_read")
    s = shape_of(2, 2, 64, 8, 64)
    a = ctypes.c_void_p(256)
    good = [a] * 5 + [4, a, a, 3, a, 0, a, 0, None, None]

    def call(shape=s, **over):
        args = list(good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return fn(ctypes.byref(shape), *args)

    for i in (0, 1, 2, 3, 4, 6, 7, 9, 11):
        assert call(**{f"a{i}": None}) == -1, i
    for i in (0, 1, 9, 11):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (2, 3):
        assert call(**{f"a{i}": ctypes.c_void_p(256 + align // 2)}) == -1
    for i in (4, 6, 7, 13):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    for stride in (64, 132, -128):
        assert call(a10=stride) == -1 and call(a12=stride) == -1
    assert call(a8=-1) == -1 and call(a5=0) == -1
    assert call(a8=0) == 0 and call(shape=shape_of(0, 2, 64, 8, 64)) == 0  # nothing to do
    assert call(shape=P.make_shape(B=2, Hq=2, Hkv=2, D=64, k=0, row_lo=0, max_sparse=0, max_len=64, num_slots=40)) == -1


class Held:
    """A cache of either format: its device arrays and its values."""

    def __init__(self, fmt, seed, B, Hkv, D, lens, pow2=True):
        self.fmt, self.D, self.Hkv = fmt, D, Hkv
        self.g, self.table, pools, scales, self.total = cache(seed, B, Hkv, D, lens)
        if fmt == "kv4":
            self.arrays = [dev(C.kv4_pack(p), torch.uint8) for p in pools] + [dev(x, torch.uint8) for x in scales]
            self.values = [C.kv4_decode(p, x) for p, x in zip(pools, scales)]
            self.fn = P.pillar_kv4_read
        else:
            g = self.g
            codes = [(g.integers(0, 127, p.shape) | g.integers(0, 2, p.shape) << 7).astype(np.uint8) for p in pools]
            sc = [(2.0 ** g.integers(-12, 12, p.shape[:2]) * (1 if pow2 else g.uniform(0.5, 1, p.shape[:2]))).astype(np.float32)
                  for p in pools]
            self.arrays = [dev(c, torch.uint8) for c in codes] + [dev(x, torch.float32) for x in sc]
            prod = [C.e4m3_decode(c).astype(np.float32) * x[..., None, None] for c, x in zip(codes, sc)]  # one fp32 product
            self.values = [bf16_bits_to_f32(f32_to_bf16_bits(p)).astype(np.float64) for p in prod]
            self.fn = P.pillar_kv8_read

    def read(self, first, off, table=None, n=None, pad=0, flags=None, stream=None, shape=None):
        """The rows as bf16 bits, K and V, and whether the gaps between them are as they were."""
        n = int(off[-1]) if n is None else n
        B, row = len(first), self.Hkv * self.D
        s = shape or shape_of(B, self.Hkv, self.D, self.total, 16 * self.table.shape[1])
        wide = [torch.full((max(1, n), row + pad * (i + 1)), MARK, dtype=torch.int16, device="cuda") for i in range(2)]
        out = [w[:n].as_strided((n, self.Hkv, self.D), (w.shape[1], self.D, 1)) for w in wide]
        torch.cuda.synchronize()
        self.fn(s, *self.arrays, dev(self.table if table is None else table, torch.int32), dev(first, torch.int32),
                dev(off, torch.int32), *out, device_flags=flags, stream=stream)
        torch.cuda.synchronize()
        assert all(bool((w[:, row:] == MARK).all()) for w in wide)
        return [o.cpu().numpy().view(np.uint16) for o in out]


def same(got, want):
    """Equal values, by their bits but for the sign of zeros."""
    want = f32_to_bf16_bits(want.astype(np.float32))
    np.testing.assert_array_equal(np.where(got == 0x8000, 0, got), np.where(want == 0x8000, 0, want))


CASES = [  # seed, Hkv, D, first positions, rows
    (0, 1, 64, [0], [1]), (1, 8, 128, [0, 3, 16, 31], [5, 60, 16, 2]), (2, 3, 64, [7, 0, 0, 100], [100, 0, 17, 2]),
    (3, 5, 64, [i % 20 for i in range(40)], [1, 7, 0, 33] * 10), (4, 2, 128, [1, 0], [3000, 2500]), (5, 33, 128, [2], [11]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("fmt,pow2", [("kv4", True), ("kv8", True), ("kv8", False)])
@pytest.mark.parametrize("seed,Hkv,D,first,n", CASES)
def test_matches_the_definition(fmt, pow2, seed, Hkv, D, first, n):
    c = Held(fmt, seed, len(first), Hkv, D, [f + m for f, m in zip(first, n)], pow2)
    off = np.concatenate([[0], np.cumsum(n)])
    N = int(off[-1])
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    for pad in (0, 8):
        for got, v in zip(c.read(first, off, pad=pad, flags=flags), c.values):
            same(got, C.kv_read(v, c.table, first, off, np.zeros((N, Hkv, D))))
    assert int(flags.item()) == 0


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["kv4", "kv8"])
def test_bad_inputs_are_flagged_and_their_rows_stay(fmt):
    c = Held(fmt, 20, 4, 2, 64, [32, 48, 16, 16])
    first, off = [4, 20, 0, 3], [0, 6, 20, 21, 30]

    def one(first, off, flag, still, table=None, n=33, shape=None):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = c.read(first, off, table, n=n, flags=flags, shape=shape)
        assert int(flags.item()) == flag
        for x, v in zip(got, c.values):
            want = np.full((n, 2, 64), bf16_bits_to_f32(np.array([MARK], np.uint16))[0], np.float64)
            for b in still:
                want[off[b]:off[b + 1]] = C.kv_read(v, c.table[b:b + 1], [first[b]], [0, off[b + 1] - off[b]],
                                                    want[off[b]:off[b + 1]])
            same(x, want)

    one(first, off, 0, (0, 1, 2, 3))
    one([-1, 20, 0, 3], off, P.FLAG_REQUEST, (1, 2, 3))
    one([4, 2 ** 31 - 1, 0, 3], off, P.FLAG_REQUEST, (0, 2, 3))
    one(first, [0, 6, 20, 21, 40], P.FLAG_REQUEST, (0, 1, 2))
    bad = c.table.copy()
    bad[2, 0] = c.total
    one(first, off, P.FLAG_SLOT, (0, 1, 3), table=bad)
    one(first, off, P.FLAG_REQUEST, (0, 2, 3), shape=shape_of(4, 2, 64, c.total, 33))  # position 33 is past max_len


@pytest.mark.gpu
def test_other_stream_captured_and_scales_that_are_none():
    c = Held("kv4", 30, 2, 2, 128, [90, 40])
    first, off = [10, 0], [0, 80, 120]
    want = c.read(first, off)
    for a, b in zip(want, c.read(first, off, stream=torch.cuda.Stream())):
        np.testing.assert_array_equal(a, b)
    s = shape_of(2, 2, 128, c.total, 16 * c.table.shape[1])
    args = (dev(c.table, torch.int32), dev(first, torch.int32), dev(off, torch.int32))
    out = [torch.zeros((120, 2, 128), dtype=torch.int16, device="cuda") for _ in "kv"]
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.fn(s, *c.arrays, *args, *out)
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(want, out):
        np.testing.assert_array_equal(a, b.cpu().numpy().view(np.uint16))
    c.arrays[2][c.table[0, 1], 0, 3, 5] = 0xff  # position 19, head 0, dimensions 80 .. 95: no number
    got = bf16_bits_to_f32(c.read(first, off)[0])
    assert np.all(np.isnan(got[9, 0, 80:96])) and np.isfinite(got).sum() == got.size - 16


@pytest.mark.gpu
@pytest.mark.parametrize("fmt", ["kv4", "kv8"])
def test_the_binding_refuses_tensors_that_do_not_fit(fmt):
    c = Held(fmt, 40, 2, 2, 64, [20, 20])
    s = shape_of(2, 2, 64, c.total, 16 * c.table.shape[1])
    out = [torch.zeros((5, 2, 64), dtype=torch.bfloat16, device="cuda") for _ in "kv"]
    good = [*c.arrays, dev(c.table, torch.int32), dev([0, 1], torch.int32), dev([0, 2, 5], torch.int32), *out]
    c.fn(s, *good)
    for i in range(len(good)):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i].unsqueeze(0)):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                c.fn(s, *args)

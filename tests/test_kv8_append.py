"""pillar_kv8_append: codes and scales of the 8-bit cache, bit for bit against the plain definition (the scale is a power of
two, so every division is exact and each value is rounded once)."""
import ctypes

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

torch = pytest.importorskip("torch")


def shape_of(B, Hkv, D, num_blocks, max_len):
    return P.make_shape(B=B, Hq=Hkv, Hkv=Hkv, D=D, k=0, row_lo=0, max_sparse=0, max_len=max_len, num_slots=num_blocks * 16)


def test_host_checks():
    P.build()
    lib = P.load()
    s = shape_of(2, 2, 64, 8, 64)
    a = ctypes.c_void_p(256)
    good = [a, 0, a, 0, 3, a, a, a, 4, a, a, a, a, None, None]

    def call(shape=s, **over):
        args = list(good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return lib.pillar_kv8_append(ctypes.byref(shape), *args)

    for i in (0, 2, 5, 6, 7, 9, 10, 11, 12):
        assert call(**{f"a{i}": None}) == -1
    for i in (0, 2, 9, 10):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (5, 6, 7, 11, 12, 13):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    for stride in (64, 132, -128):  # shorter than a row, not a multiple of 8, negative
        assert call(a1=stride) == -1 and call(a3=stride) == -1
    assert call(a4=-1) == -1 and call(a8=0) == -1
    assert call(a4=0) == 0 and call(shape=shape_of(0, 2, 64, 8, 64)) == 0  # nothing to do
    assert call(shape=P.make_shape(B=2, Hq=2, Hkv=2, D=64, k=0, row_lo=0, max_sparse=0, max_len=64, num_slots=40)) == -1


def cache(seed, B, Hkv, D, lens, spread=0, spare=2):
    """A pool with random finite codes and power-of-two scales, and block tables for the lengths."""
    g = np.random.default_rng(seed)
    nb = -(-np.asarray(lens) // 16)
    total = int(nb.sum()) + spare
    perm = g.permutation(total)
    table = np.zeros((B, int(max(1, nb.max()))), np.int64)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    pools = [g.integers(0, 127, (total, Hkv, 16, D)).astype(np.uint8) | (g.integers(0, 2, (total, Hkv, 16, D)) << 7)
             .astype(np.uint8) for _ in "kv"]
    scales = [2.0 ** g.integers(-8 - spread, spread - 6, (total, Hkv)).astype(np.float64) for _ in "kv"]
    return g, table, pools, scales, total


def run(s, new, strides, lens, off, table, pools, scales, flags=None, stream=None):
    dev = lambda x, t: torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")  # noqa: E731
    k8, v8 = (dev(p, torch.uint8) for p in pools)
    ks, vs = (dev(x, torch.float32) for x in scales)
    t = []
    for x, st in zip(new, strides):
        bits = torch.from_numpy(f32_to_bf16_bits(x).view(np.int16))
        wide = torch.full((max(1, len(x)), st), 0x7fc0, dtype=torch.int16)  # NaN between the rows
        wide[:len(x), :bits[0].numel() if len(x) else 0] = bits.reshape(len(x), -1)
        t.append(wide.cuda()[:len(x)].as_strided((len(x),) + x.shape[1:], (st, x.shape[2], 1)))
    P.pillar_kv8_append(s, t[0], t[1], dev(lens, torch.int32), dev(off, torch.int32), dev(table, torch.int32), k8, v8, ks,
                        vs, device_flags=flags, stream=stream)
    torch.cuda.synchronize()
    return (k8.cpu().numpy(), ks.cpu().numpy()), (v8.cpu().numpy(), vs.cpu().numpy())


CASES = [  # seed, Hkv, D, lengths, new tokens per request
    (0, 1, 64, [1], [1]), (1, 8, 128, [16, 17, 32, 5], [16, 1, 9, 5]), (2, 3, 64, [100, 1, 48, 33], [100, 0, 17, 2]),
    (3, 2, 128, [15, 16, 31, 64, 200], [3, 1, 16, 40, 9]), (4, 5, 64, [7] * 40, [1, 7, 0, 3] * 10),
    (5, 8, 128, list(range(60, 190)), [1 + 8 * (i % 9 == 0) for i in range(130)]),
    (6, 2, 64, [4000, 3, 2777], [4000, 3, 2777]), (7, 1, 128, [3001], [2999]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,Hkv,D,lens,n", CASES)
@pytest.mark.parametrize("spread,pad", [(0, 0), (20, 24)])
def test_matches_the_definition(seed, Hkv, D, lens, n, spread, pad):
    g, table, pools, scales, total = cache(seed, len(lens), Hkv, D, lens, spread)
    off = np.concatenate([[0], np.cumsum(n)])
    N = int(off[-1])
    new = []
    for _ in "kv":
        x = g.standard_normal((N, Hkv, D)) * 2.0 ** g.integers(-spread - 2, spread + 3, (N, Hkv, 1))
        x[g.random((N, Hkv)) < 0.1] = 0  # rows of zeros
        new.append(bf16_bits_to_f32(f32_to_bf16_bits(x.astype(np.float32))))
    s = shape_of(len(lens), Hkv, D, total, max(lens))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(s, new, (Hkv * D + pad, Hkv * D + 2 * pad), lens, off, table, pools, scales, flags)
    assert int(flags.item()) == 0
    for x, p, sc, (codes, scale) in zip(new, pools, scales, got):
        want_c, want_s = C.kv8_append(p, sc, x.astype(np.float64), lens, off, table)
        np.testing.assert_array_equal(scale, want_s)
        np.testing.assert_array_equal(C.e4m3_decode(codes), C.e4m3_decode(want_c))


@pytest.mark.gpu
def test_extreme_magnitudes_and_empty_blocks():
    """The largest and smallest bf16 values, a zero row first and values later, a scale of zero before."""
    big, tiny = 3.3895313892515355e38, 2.0 ** -133
    new = np.zeros((5, 2, 64), np.float32)
    new[0, 0, 3], new[0, 1, 5] = big, tiny
    new[1, 0, 0], new[2, 0, 0] = -big, 1.0
    new[3, 0, 7] = 448 * 2.0 ** -126
    lens, off, table = [3, 34, 17], [0, 2, 4, 5], np.array([[0, 0, 0], [1, 2, 3], [4, 5, 0]])
    pools = [np.full((6, 2, 16, 64), 0x38, np.uint8)] * 2
    scales = [np.zeros((6, 2))] * 2
    scales[0][5] = 0.0
    s = shape_of(3, 2, 64, 6, 48)
    got = run(s, (new, new[:, ::-1].copy()), (128, 128), lens, off, table, pools, scales)
    for x, (codes, scale) in zip((new, new[:, ::-1]), got):
        want_c, want_s = C.kv8_append(pools[0], scales[0], x.astype(np.float64), lens, off, table)
        np.testing.assert_array_equal(scale, want_s)
        np.testing.assert_array_equal(C.e4m3_decode(codes), C.e4m3_decode(want_c))


@pytest.mark.gpu
def test_bad_inputs_are_flagged_and_skipped():
    D, Hkv = 64, 2
    lens, off = [20, 40, 5, 9], [0, 4, 6, 7, 9]
    g, table, pools, scales, total = cache(21, 4, Hkv, D, [32, 48, 16, 16])
    x = bf16_bits_to_f32(f32_to_bf16_bits(g.standard_normal((12, Hkv, D)).astype(np.float32)))
    s = shape_of(4, Hkv, D, total, 48)

    def check(lens, off, table, flag, still, new=x, n=12, scales=scales):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(s, (new[:n], new[:n]), (128, 128), lens, off, table, pools, scales, flags)
        assert int(flags.item()) == flag
        keep_off = np.concatenate([[0], np.cumsum([(off[b + 1] - off[b]) if b in still else 0 for b in range(4)])])
        rows = np.concatenate([np.arange(off[b], off[b + 1]) for b in still]).astype(int)
        for p, sc, (codes, scale) in zip(pools, scales, got):
            want_c, want_s = C.kv8_append(p, sc, new[rows].astype(np.float64), lens, keep_off, table)
            np.testing.assert_array_equal(scale, want_s)
            np.testing.assert_array_equal(C.e4m3_decode(codes), C.e4m3_decode(want_c))

    check(lens, off, table, 0, [0, 1, 2, 3])                                   # rows 9..11 lie behind the last request
    t = table.copy()
    t[1, 2] = total
    check(lens, off, t, P.FLAG_SLOT, [0, 2, 3])                                # request 1's rows are all in that block
    t[1, 2] = -1
    check(lens, off, t, P.FLAG_SLOT, [0, 2, 3])
    check([20, 1, 5, 9], off, table, P.FLAG_REQUEST, [0, 2, 3])                # fewer positions than new tokens
    check([20, 49, 5, 9], off, table, P.FLAG_REQUEST, [0, 2, 3])               # past max_len
    check(lens, [0, 4, 6, 7, 13], table, P.FLAG_REQUEST, [0, 1, 2])            # more rows than given


@pytest.mark.gpu
def test_values_that_are_not_finite():
    D, s = 128, shape_of(1, 1, 128, 1, 16)
    x = np.random.default_rng(5).standard_normal((16, 1, D)).astype(np.float32)
    x = bf16_bits_to_f32(f32_to_bf16_bits(x))
    y, z = x.copy(), x.copy()
    y[3, 0, 7], y[9, 0, 0], y[15, 0, 127] = np.nan, np.inf, -np.inf
    z[3, 0, 7], z[9, 0, 0], z[15, 0, 127] = 0, 0, 0
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    pools, scales = [np.zeros((1, 1, 16, D), np.uint8)] * 2, [np.ones((1, 1))] * 2
    got = run(s, (y, x), (D, D), [16], [0, 16], np.zeros((1, 1)), pools, scales, flags)
    assert int(flags.item()) == P.FLAG_VALUE
    want, want_s = C.kv8_append(pools[0], scales[0], z.astype(np.float64), [16], [0, 16], np.zeros((1, 1)))
    want[0, 0, 9, 0], want[0, 0, 15, 127] = 0x7e, 0xfe
    np.testing.assert_array_equal(C.e4m3_decode(got[0][0]), C.e4m3_decode(want))
    np.testing.assert_array_equal(got[0][1], want_s)
    # a scale of earlier rows that is no scale: the earlier rows become zero
    for before in (np.nan, np.inf, -1.0):
        flags.zero_()
        got = run(s, (x[:2], x[:2]), (D, D), [9], [0, 2], np.zeros((1, 1)), [np.full((1, 1, 16, D), 0x38, np.uint8)] * 2,
                  [np.full((1, 1), before)] * 2, flags)
        assert int(flags.item()) == P.FLAG_VALUE
        assert np.all(C.e4m3_decode(got[0][0][0, 0, :7]) == 0) and np.all(C.e4m3_decode(got[0][0][0, 0, 9:]) == 0)
        assert got[0][1][0, 0] == C.scale_of(np.abs(x[:2]).max())


@pytest.mark.gpu
def test_a_scale_from_elsewhere_divides():
    """Earlier rows under a scale that is no power of two: new rows are x / scale, rounded once from the fp32 quotient."""
    D, s = 64, shape_of(1, 1, 64, 1, 16)
    x = bf16_bits_to_f32(f32_to_bf16_bits(np.random.default_rng(6).standard_normal((4, 1, D)).astype(np.float32)))
    scale = np.float32(0.3)
    got = run(s, (x, x), (D, D), [8], [0, 4], np.zeros((1, 1)), [np.full((1, 1, 16, D), 0x41, np.uint8)] * 2,
              [np.full((1, 1), scale)] * 2)
    assert got[0][1][0, 0] == scale and np.all(got[0][0][0, 0, :4] == 0x41) and np.all(got[0][0][0, 0, 8:] == 0x41)
    np.testing.assert_array_equal(got[0][0][0, 0, 4:8], C.e4m3_encode((x[:, 0] / scale).astype(np.float64)))


@pytest.mark.gpu
def test_captured_calls_and_another_stream():
    g, table, pools, scales, total = cache(31, 3, 2, 64, [50, 20, 90])
    lens, off = [50, 20, 90], [0, 30, 31, 40]
    x = g.standard_normal((40, 2, 64)).astype(np.float32)
    s = shape_of(3, 2, 64, total, 90)
    want = run(s, (x, x), (128, 128), lens, off, table, pools, scales)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = run(s, (x, x), (128, 128), lens, off, table, pools, scales, stream=side)
    dev = lambda v, t: torch.tensor(np.ascontiguousarray(v), dtype=t, device="cuda")  # noqa: E731
    k8, v8 = (dev(p, torch.uint8) for p in pools)
    ks, vs = (dev(v, torch.float32) for v in scales)
    xb = torch.from_numpy(f32_to_bf16_bits(x).view(np.int16)).cuda()
    args = (dev(lens, torch.int32), dev(off, torch.int32), dev(table, torch.int32), k8, v8, ks, vs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        P.pillar_kv8_append(s, xb, xb, *args)
    graph.replay()
    graph.replay()  # the same rows again change nothing
    torch.cuda.synchronize()
    for a, b, c in zip(want, got, ((k8, ks), (v8, vs))):
        for u, v, w in zip(a, b, c):
            np.testing.assert_array_equal(u, v)
            np.testing.assert_array_equal(u, w.cpu().numpy())


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    s = shape_of(1, 2, 64, 2, 32)
    new = torch.zeros((3, 2, 64), dtype=torch.bfloat16, device="cuda")
    i32 = dict(dtype=torch.int32, device="cuda")
    good = [new, new, torch.tensor([3], **i32), torch.tensor([0, 3], **i32), torch.zeros((1, 2), **i32),
            torch.zeros((2, 2, 16, 64), dtype=torch.uint8, device="cuda"),
            torch.zeros((2, 2, 16, 64), dtype=torch.float8_e4m3fn, device="cuda"),
            torch.zeros((2, 2), device="cuda"), torch.zeros((2, 2), device="cuda")]
    P.pillar_kv8_append(s, *good)
    for i in range(9):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i][None]):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_kv8_append(s, *args)
    for wrong in (new[:2], new.transpose(1, 2), new[:, :, ::2], new[:, :1], torch.zeros((3, 64, 2), device="cuda").bfloat16()):
        with pytest.raises(ValueError):
            P.pillar_kv8_append(s, new, wrong, *good[2:])
    wide = torch.zeros((3, 132), dtype=torch.bfloat16, device="cuda")[:, :128].unflatten(1, (2, 64))
    with pytest.raises(P.PillarError):  # rows that do not start on 16 bytes
        P.pillar_kv8_append(s, wide, new, *good[2:])
    P.pillar_kv8_append(s, new[:0], new[:0], torch.tensor([0], **i32), torch.tensor([0, 0], **i32), *good[4:])


@pytest.mark.gpu
@pytest.mark.parametrize("bad", [-1, 0, 2, -2 ** 31, -2 ** 31 + 1, -2 ** 31 + 2, -2 ** 31 + 3, 2 ** 31 - 1])
def test_lengths_that_are_none(bad):
    """Request 1's three new tokens under every kind of wrong length, the lowest ones among them, whose difference to the new
    tokens passes 31 bits: flagged, its rows skipped, the others' as ever."""
    lens, off, keep = [20, bad, 9], [0, 4, 7, 9], [0, 4, 4, 6]
    g, table, pools, scales, total = cache(22, 3, 2, 64, [32, 48, 16])
    x = bf16_bits_to_f32(f32_to_bf16_bits(g.standard_normal((9, 2, 64)).astype(np.float32)))
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(shape_of(3, 2, 64, total, 48), (x, x), (128, 128), lens, off, table, pools, scales, flags)
    assert int(flags.item()) == P.FLAG_REQUEST
    rows = x[[0, 1, 2, 3, 7, 8]].astype(np.float64)
    for p, sc, (codes, scale) in zip(pools, scales, got):
        want_c, want_s = C.kv8_append(p, sc, rows, [20, 3, 9], keep, table)
        np.testing.assert_array_equal(scale, want_s)
        np.testing.assert_array_equal(C.e4m3_decode(codes), C.e4m3_decode(want_c))

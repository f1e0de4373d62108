"""pillar_kv4_append: codes and scale bytes of the 4-bit cache, bit for bit against the plain definition (a scale is the
smallest that fits, a code the nearest; no rounding comes before them)."""
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
        return lib.pillar_kv4_append(ctypes.byref(shape), *args)

    for i in (0, 2, 5, 6, 7, 9, 10, 11, 12):
        assert call(**{f"a{i}": None}) == -1
    for i in (0, 2, 9, 10):
        assert call(**{f"a{i}": ctypes.c_void_p(264)}) == -1
    for i in (11, 12):
        assert call(**{f"a{i}": ctypes.c_void_p(260)}) == -1
    for i in (5, 6, 7, 13):
        assert call(**{f"a{i}": ctypes.c_void_p(258)}) == -1
    for stride in (64, 132, -128):  # shorter than a row, not a multiple of 8, negative
        assert call(a1=stride) == -1 and call(a3=stride) == -1
    assert call(a4=-1) == -1 and call(a8=0) == -1
    assert call(a4=0) == 0 and call(shape=shape_of(0, 2, 64, 8, 64)) == 0  # nothing to do
    assert call(shape=P.make_shape(B=2, Hq=2, Hkv=2, D=64, k=0, row_lo=0, max_sparse=0, max_len=64, num_slots=40)) == -1
    wide = 1 << 21  # heads whose row is past 2^26 values
    assert call(shape=P.make_shape(B=1, Hq=wide, Hkv=wide, D=64, k=0, row_lo=0, max_sparse=0, max_len=16, num_slots=16)) == -1


def cache(seed, B, Hkv, D, lens, spare=2):
    """A pool with random codes and scales, and block tables for the lengths."""
    g = np.random.default_rng(seed)
    nb = -(-np.asarray(lens) // 16)
    total = int(nb.sum()) + spare
    perm = g.permutation(total)
    table = np.zeros((B, int(max(1, nb.max()))), np.int64)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    pools = [g.integers(0, 16, (total, Hkv, 16, D)).astype(np.uint8) for _ in "kv"]
    scales = [g.integers(0, C.TOP4 + 1, (total, Hkv, 16, D // 16)).astype(np.uint8) for _ in "kv"]
    return g, table, pools, scales, total


def dev(x, t):
    return torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")


def packed_rows(x, stride):
    """[n, Hkv, D] fp32 on the device as bf16 rows `stride` elements apart, NaN between them."""
    bits = torch.from_numpy(f32_to_bf16_bits(x).view(np.int16))
    wide = torch.full((max(1, len(x)), stride), 0x7fc0, dtype=torch.int16)
    wide[:len(x), :bits[0].numel() if len(x) else 0] = bits.reshape(len(x), -1)
    return wide.cuda()[:len(x)].as_strided((len(x),) + x.shape[1:], (stride, x.shape[2], 1))


def run(s, new, strides, lens, off, table, pools, scales, flags=None, stream=None):
    k4, v4 = (dev(C.kv4_pack(p), torch.uint8) for p in pools)
    ks, vs = (dev(x, torch.uint8) for x in scales)
    t = [packed_rows(x, st) for x, st in zip(new, strides)]
    torch.cuda.synchronize()
    P.pillar_kv4_append(s, t[0], t[1], dev(lens, torch.int32), dev(off, torch.int32), dev(table, torch.int32), k4, v4, ks,
                        vs, device_flags=flags, stream=stream)
    torch.cuda.synchronize()
    return (k4.cpu().numpy(), ks.cpu().numpy()), (v4.cpu().numpy(), vs.cpu().numpy())


def check(got, new, pools, scales, lens, off, table):
    for x, p, sc, (packed, byte) in zip(new, pools, scales, got):
        want_c, want_s = C.kv4_append(p, sc, x.astype(np.float64), lens, off, table)
        np.testing.assert_array_equal(byte, want_s)
        codes, zero = C.kv4_unpack(packed), want_c & 7 == 0  # (the sign of a zero has no meaning)
        np.testing.assert_array_equal(np.where(zero, codes & 7, codes), np.where(zero, 0, want_c))


CASES = [  # seed, Hkv, D, lengths, new tokens per request
    (0, 1, 64, [1], [1]), (1, 8, 128, [16, 17, 32, 5], [16, 1, 9, 5]), (2, 3, 64, [100, 1, 48, 33], [100, 0, 17, 2]),
    (3, 2, 128, [15, 16, 31, 64, 200], [3, 1, 16, 40, 9]), (4, 5, 64, [7] * 40, [1, 7, 0, 3] * 10),
    (5, 8, 128, list(range(60, 110)), [1 + 8 * (i % 9 == 0) for i in range(50)]),
    (6, 1, 64, [2000, 3, 1777], [2000, 3, 777]), (7, 1, 128, [3001], [2999]), (8, 33, 64, [9, 2], [5, 2]),
]


@pytest.mark.gpu
@pytest.mark.parametrize("seed,Hkv,D,lens,n", CASES)
@pytest.mark.parametrize("spread,pad", [(0, 0), (9, 24)])
def test_matches_the_definition(seed, Hkv, D, lens, n, spread, pad):
    g, table, pools, scales, total = cache(seed, len(lens), Hkv, D, lens)
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
    check(got, new, pools, scales, lens, off, table)


@pytest.mark.gpu
def test_every_magnitude_and_every_tie():
    """Each bf16 magnitude once as the largest of its group (the scale), and the seven ties of every scale."""
    mags = np.arange(1, 0x7f80, dtype=np.uint16)
    n = -(-len(mags) // 16)
    x = np.zeros((n, 4, 64), np.float32)  # 16 groups a row
    x.reshape(-1, 16)[:len(mags), 5] = bf16_bits_to_f32(mags) * np.where(np.arange(len(mags)) % 2, -1, 1)
    ties = np.zeros((226, 16))
    for b in range(1, 227):
        ties[b - 1, :8] = np.array([6, 0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5]) * C.SCALE4[b]
        ties[b - 1, 8:15] = -ties[b - 1, 1:8] * (1 + 2.0 ** -7)  # just past them
    y = np.zeros((n, 4, 64), np.float32)
    y.reshape(-1, 16)[:226] = ties
    y = bf16_bits_to_f32(f32_to_bf16_bits(y))
    lens, off = [n], [0, n]
    g, table, pools, scales, total = cache(9, 1, 4, 64, lens)
    flags = torch.zeros(1, dtype=torch.int32, device="cuda")
    got = run(shape_of(1, 4, 64, total, n), (x, y), (256, 256), lens, off, table, pools, scales, flags)
    assert int(flags.item()) == P.FLAG_VALUE  # (the magnitudes past 61440)
    check(got, (x, y), pools, scales, lens, off, table)


@pytest.mark.gpu
def test_values_that_are_none():
    """NaN is stored as 0, an infinity as the largest value of its sign; the scale goes by the finite values."""
    x = np.zeros((3, 1, 64), np.float32)
    x[0, 0, :4] = [np.nan, np.inf, 3.0, -np.inf]
    x[1, 0, 20] = -np.inf
    x[2, 0, 40:42] = [65000.0, np.nan]
    lens, off = [3], [0, 3]
    g, table, pools, scales, total = cache(10, 1, 1, 64, lens)
    for k in range(3):
        one = np.zeros_like(x)
        one[k] = x[k]
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(shape_of(1, 1, 64, total, 3), (one, one), (64, 64), lens, off, table, pools, scales, flags)
        assert int(flags.item()) == P.FLAG_VALUE
        for packed, byte in got:
            row = C.kv4_decode(C.kv4_unpack(packed), byte)[table[0, 0], 0]
            if k == 0:
                assert list(row[0, :5]) == [0, 3, 3, -3, 0]
            elif k == 1:
                assert row[1, 20] == -6 * 2.0 ** -17 and np.count_nonzero(row[1]) == 1
            else:
                assert row[2, 40] == 61440 and np.count_nonzero(row[2]) == 1


@pytest.mark.gpu
def test_bad_inputs_are_flagged_and_skipped():
    D, Hkv = 64, 2
    lens, off = [20, 40, 5, 9], [0, 4, 6, 7, 9]
    g, table, pools, scales, total = cache(21, 4, Hkv, D, [32, 48, 16, 16])
    x = bf16_bits_to_f32(f32_to_bf16_bits(g.standard_normal((12, Hkv, D)).astype(np.float32)))
    s = shape_of(4, Hkv, D, total, 48)

    def one(lens, off, table, flag, still, n=12):
        flags = torch.zeros(1, dtype=torch.int32, device="cuda")
        got = run(s, (x[:n], x[:n]), (128, 128), lens, off, table, pools, scales, flags)
        assert int(flags.item()) == flag
        keep = [b for b in range(4) if b in still]
        rows = np.concatenate([x[off[b]:off[b + 1]] for b in keep]) if keep else x[:0]
        koff = np.concatenate([[0], np.cumsum([off[b + 1] - off[b] for b in keep])])
        check(got, (rows, rows), pools, scales, [lens[b] for b in keep], koff, table[keep])

    one(lens, off, table, 0, (0, 1, 2, 3))                       # rows behind the last request are not read
    one([20, 49, 5, 9], off, table, P.FLAG_REQUEST, (0, 2, 3))   # past max_len
    one([20, 1, 5, 9], off, table, P.FLAG_REQUEST, (0, 2, 3))    # fewer positions than new tokens
    one([-2 ** 31, 40, 5, 9], off, table, P.FLAG_REQUEST, (1, 2, 3))
    one([2 ** 31 - 1, 40, 5, 9], off, table, P.FLAG_REQUEST, (1, 2, 3))
    one(lens, [0, 4, 6, 7, 13], table, P.FLAG_REQUEST, (0, 1, 2))  # offsets past n
    bad = table.copy()
    bad[0, 1], bad[3, 0] = total, -1
    one(lens, off, bad, P.FLAG_SLOT, (1, 2))
    narrow = np.ascontiguousarray(table[:, :2])
    one(lens, off, narrow, P.FLAG_REQUEST, (0, 2, 3))            # request 1's rows lie in block 2


@pytest.mark.gpu
def test_in_parts_again_and_on_another_stream():
    """Rows are independent: in two calls, or twice, on another stream, the same cache."""
    lens, n = [70, 33], [40, 33]
    g, table, pools, scales, total = cache(30, 2, 2, 128, lens)
    x = bf16_bits_to_f32(f32_to_bf16_bits(g.standard_normal((73, 2, 128)).astype(np.float32)))
    s = shape_of(2, 2, 128, total, 70)
    once = run(s, (x, x), (256, 256), lens, [0, 40, 73], table, pools, scales)
    check(once, (x, x), pools, scales, lens, [0, 40, 73], table)
    st = torch.cuda.Stream()
    some = run(s, (x[:30], x[:30]), (256, 256), [60, 0], [0, 30, 30], table, pools, scales, stream=st)
    pools2 = [C.kv4_unpack(p) for p, _ in some]
    rest = np.concatenate([x[30:40], x[40:]])
    both = run(s, (rest, rest), (256, 256), lens, [0, 10, 43], table, pools2, [b for _, b in some], stream=st)
    for a, b in zip(once, both):
        np.testing.assert_array_equal(a[0], b[0])
        np.testing.assert_array_equal(a[1], b[1])


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    s = shape_of(2, 2, 64, 4, 32)
    z = lambda sh, t: torch.zeros(sh, dtype=t, device="cuda")  # noqa: E731
    good = [z((3, 2, 64), torch.bfloat16), z((3, 2, 64), torch.bfloat16), z(2, torch.int32), z(3, torch.int32),
            z((2, 2), torch.int32), z((4, 2, 16, 32), torch.uint8), z((4, 2, 16, 32), torch.uint8),
            z((4, 2, 16, 4), torch.uint8), z((4, 2, 16, 4), torch.uint8)]
    P.pillar_kv4_append(s, *good)
    for i in range(len(good)):
        for wrong in (good[i].cpu(), good[i].to(torch.float64), good[i].unsqueeze(0)):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_kv4_append(s, *args)
    with pytest.raises(ValueError):
        P.pillar_kv4_append(s, *good, device_flags=z(2, torch.int32))

"""The 4-bit cache's plain definitions, pinned by closed forms and against the 8-bit step's definition."""
import math

import numpy as np

from oracle import cache as C


def test_formats():
    s = C.SCALE4
    as_f16 = (np.arange(256, dtype=np.uint16) << 7).view(np.float16).astype(np.float64)  # the same bits, as an f16 value
    np.testing.assert_array_equal(s, as_f16)
    assert s[1] == 2.0 ** -17 and s[C.TOP4] == 10240 and 6 * s[C.TOP4] < 65504 < 6 * s[C.TOP4 + 1]
    assert [C.E2M1[c] for c in (1, 2, 3, 7)] == [0.5, 1, 1.5, 6]


def test_encode_picks_the_smallest_scale_and_the_nearest_code():
    x = np.zeros(32)
    x[:4] = [6.0, -5.0, 2.5, 0.25]      # scale 1 exactly: ties go to the even code
    x[16:19] = [6.0001, -3.1, 0.4]      # just past it: the next scale
    code, byte = C.kv4_encode(x)
    assert C.SCALE4[byte[0]] == 1 and C.SCALE4[byte[1]] == 1.125
    assert list(code[:4]) == [7, 8 | 6, 4, 0] and list(code[16:19]) == [7, 8 | 5, 1]
    g = np.random.default_rng(0)
    x = g.standard_normal((40, 64)) * 2.0 ** g.integers(-16, 12, (40, 1))
    code, byte = C.kv4_encode(x)
    a = np.abs(x.reshape(40, 4, 16)).max(-1)
    assert np.all(a <= 6 * C.SCALE4[byte]) and np.all((a > 6 * C.SCALE4[byte - 1]) | (byte == 1))
    back = C.kv4_decode(code, byte)
    assert np.all(np.abs(back - x) <= np.repeat(C.SCALE4[byte], 16, -1))        # half the widest step (4 to 6)
    # what is held is held again, where neighbouring scales are at most 9/8 apart: the largest value is above 6 * 8/9 scales,
    # rounds to 6 and asks for the same scale (scales below 2^-14 are a fixed step apart)
    normal = np.repeat(byte >= 8, 16, -1)
    np.testing.assert_array_equal(C.kv4_decode(*C.kv4_encode(back))[normal], back[normal])
    assert normal.mean() > 0.5
    np.testing.assert_array_equal(C.kv4_unpack(C.kv4_pack(code)), code)


def test_extremes():
    for x, want in ((1e30, 61440.0), (-61440.0, -61440.0), (2.0 ** -18, 2.0 ** -18), (2.0 ** -20, 0.0), (0.0, 0.0)):
        code, byte = C.kv4_encode(np.r_[x, np.zeros(15)])
        assert C.kv4_decode(code, byte)[0] == want


def test_append_and_read_round_trip():
    g = np.random.default_rng(1)
    table = np.array([[3, 0, 5], [1, 4, 2]])
    codes, byte = np.zeros((6, 2, 16, 32), np.uint8), np.ones((6, 2, 16, 2), np.uint8)
    x = g.integers(-3, 4, (30, 2, 32)) * 1.0
    x[..., ::16] = 6.0                                                          # scale 1: small integers are exact
    codes, byte = C.kv4_append(codes, byte, x, [35, 20], [0, 17, 30], table)
    out = C.kv_read(C.kv4_decode(codes, byte), table, [18, 7], [0, 17, 30], np.full_like(x, 99))
    np.testing.assert_array_equal(out, x)
    assert np.count_nonzero(codes.any(-1)) == 30 * 2                            # and nothing else was written


def test_attention_agrees_with_the_8_bit_definition_on_shared_values():
    g = np.random.default_rng(2)
    k8, v8 = (g.integers(0, 100, (7, 2, 16, 32)).astype(np.uint8) for _ in "kv")
    sc = 2.0 ** g.integers(-9, -6, (7, 2)).astype(np.float64)
    table, q = np.array([[0, 2, 4], [6, 1, 9]]), g.standard_normal((4, 4, 32))
    idx = g.integers(0, 50, (2, 2, 9))
    args = (table, [1, 0], [40, 36], idx, np.array([[0, 0], [9, 4]]), 2, 0.2)
    want = C.attn_kv8(q, k8, v8, sc, sc, *args)
    got = C.attn_cache(q, C.e4m3_decode(k8) * sc[..., None, None], C.e4m3_decode(v8) * sc[..., None, None], *args)
    for a, b in zip(got, want):
        np.testing.assert_array_equal(a, b)
    assert math.isinf(want[1].min())

"""The numpy definitions of the cache operators, checked against closed forms and invariants."""
import numpy as np
import pytest

from oracle import cache as C


def test_e4m3_values_and_rounding():
    v = C.e4m3_table()
    assert v[0x00] == 0 and v[0x01] == 2.0 ** -9 and v[0x08] == 2.0 ** -6 and v[0x38] == 1.0 and v[0x7e] == 448.0
    assert np.isnan(v[0x7f]) and np.isnan(v[0xff]) and v[0xfe] == -448.0
    finite = np.array([c for c in range(256) if (c & 127) != 127])
    np.testing.assert_array_equal(C.e4m3_encode(v[finite]), finite)  # every value is its own code
    # half-way between 1 and 1.125 goes to the even code, just above it up
    assert C.e4m3_encode(1.0625) == 0x38 and C.e4m3_encode(1.0625 + 1e-9) == 0x39 and C.e4m3_encode(1.1875) == 0x3a
    assert C.e4m3_encode(1e9) == 0x7e and C.e4m3_encode(-1e9) == 0xfe and C.e4m3_encode(2.0 ** -10) == 0x00
    # relative error of normal values at most half a step, 2^-4
    x = np.random.default_rng(0).uniform(2.0 ** -6, 448, 10000)
    assert np.max(np.abs(C.e4m3_decode(C.e4m3_encode(x)) / x - 1)) <= 2.0 ** -4


@pytest.mark.parametrize("amax,e", [(448.0, 0), (449.0, 1), (1.75, -8), (1.7501, -7), (224.0, -1), (0.0, -126),
                                    (1e-40, -126), (3.3e38, 120)])
def test_scale_is_the_smallest_power_of_two(amax, e):
    s = C.scale_of(amax)
    assert s == 2.0 ** e and amax <= 448 * s and (e == -126 or amax > 448 * s / 2)


def test_append_again_changes_nothing_and_growth_keeps_values():
    rng = np.random.default_rng(3)
    codes, scale = np.zeros((4, 2, 16, 8), np.uint8), np.full((4, 2), 7.0)
    table = np.array([[2, 0], [3, 1]])
    x = rng.standard_normal((22, 2, 8))
    c1, s1 = C.kv8_append(codes, scale, x, [20, 2], [0, 20, 22], table)
    got = C.e4m3_decode(c1) * s1[..., None, None]
    np.testing.assert_allclose(got[2], x[:16].transpose(1, 0, 2), rtol=0, atol=np.abs(x).max() / 28)
    np.testing.assert_array_equal(c1[0, :, 4:], 0)
    c2, s2 = C.kv8_append(c1, s1, x, [20, 2], [0, 20, 22], table)
    np.testing.assert_array_equal(c1, c2)
    np.testing.assert_array_equal(s1, s2)
    # a row 64 times larger: the block's scale grows by 64, its earlier rows keep their values to the coarser step
    y = np.full((1, 2, 8), 64 * np.abs(x[16:20]).max())
    c3, s3 = C.kv8_append(c1, s1, y, [21, 2], [0, 1, 1], table)
    assert np.all(s3[0] >= 32 * s1[0]) and np.array_equal(s3[1:], s1[1:])
    old, new = got[0, :, :4], (C.e4m3_decode(c3) * s3[..., None, None])[0, :, :4]
    assert np.all(np.abs(new - old) <= np.maximum(np.abs(old) * 2.0 ** -4, s3[0][:, None, None] * 2.0 ** -10))


def test_block_map_grows_rolls_back_and_runs_short():
    ring = np.array([5, 1, 0, 3, 2, 4])
    r = C.block_map([17, 0, 5], [0, 0, 0], np.full((3, 4), 9), ring, [4, 3], 64, 6)
    # blocks 2 and 4 to request 0, 5 to request 2 (the ring wraps)
    assert r["table"][0, :2].tolist() == [2, 4] and r["table"][2, 0] == 5 and not r["bad"]
    assert r["kv_off"].tolist() == [0, 17, 17, 22] and r["new_off"].tolist() == [0, 17, 17, 22]
    assert r["slots"].tolist() == [32 + i for i in range(16)] + [64] + [80 + i for i in range(5)]
    assert r["state"].tolist() == [1, 0] and np.array_equal(r["slots"], r["new_slots"])
    back = C.block_map([16, 0, 0], r["granted"], r["table"], r["ring"], r["state"], 64, 6)
    assert back["state"].tolist() == [1, 2] and back["ring"][1:3].tolist() == [4, 5] and len(back["new_slots"]) == 0
    short = C.block_map([16, 33, 20, 4], [16, 0, 16, 3], np.arange(16).reshape(4, 4) % 6, ring, [0, 2], 64, 6)
    assert short["bad"] == {"block"} and short["granted"].tolist() == [16, 0, 16, 4]  # 33 does not fit, nor what follows
    assert short["state"].tolist() == [0, 2]


def test_attention_over_the_cache_agrees_with_the_bf16_oracle():
    """Codes under powers of two are bf16 values, so the step's own oracle, written apart, has to agree."""
    import oracle
    rng = np.random.default_rng(8)
    Hq, Hkv, D, k, lens, mode = 4, 2, 64, 2, [37, 20, 5], [1, 0, 1]
    k8, v8 = (rng.integers(0, 120, (9, Hkv, 16, D)).astype(np.uint8) for _ in "kv")
    ks, vs = (2.0 ** rng.integers(-9, -5, (9, Hkv)).astype(np.float64) for _ in "kv")
    table = np.array([[3, 0, 7], [5, 1, 0], [8, 0, 0]])
    idx, cnt = rng.integers(0, 20, (3, Hkv, 6)), np.array([[0, 0], [6, 0], [0, 0]])
    from workloads import bf16_bits_to_f32, f32_to_bf16_bits
    qb = f32_to_bf16_bits(rng.standard_normal((7, Hq, D)).astype(np.float32) * 0.3)
    out, logits, lse = C.attn_kv8(bf16_bits_to_f32(qb).astype(np.float64), k8, v8, ks, vs, table, mode, lens, idx, cnt, k,
                                  D ** -0.5)
    bits = [f32_to_bf16_bits((C.e4m3_decode(c) * s[..., None, None]).transpose(0, 2, 1, 3).reshape(-1, Hkv, D)
                             .astype(np.float32)) for c, s in ((k8, ks), (v8, vs))]
    slots = np.concatenate([[table[b, t // 16] * 16 + t % 16 for t in range(n)] for b, n in enumerate(lens)])
    r = oracle.attn_unified(Hq=Hq, Hkv=Hkv, D=D, k=k, scale=D ** -0.5, q=qb, k_pool=bits[0], v_pool=bits[1],
                            slot_table=slots.astype(np.int32), req_mode=np.array(mode, np.int32),
                            req_len=np.array(lens, np.int32), sparse_idx=idx.astype(np.int32),
                            sparse_cnt=cnt.astype(np.int32))
    np.testing.assert_allclose(out, r.out, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(logits, r.logits, rtol=1e-12, atol=1e-13)
    np.testing.assert_allclose(lse, oracle.verify_lse_of(r, np.array(mode), k, Hq), rtol=1e-12)


def test_prompt_attention_closed_forms():
    rng = np.random.default_rng(9)
    q, k, v = rng.standard_normal((6, 4, 8)), rng.standard_normal((6, 2, 8)), rng.standard_normal((6, 2, 8))
    out, lse = C.prompt_attn(q, k, v, [0, 1, 1, 5], 0.3)
    np.testing.assert_allclose(out[0], v[0].repeat(2, 0))                 # a row alone is its value
    np.testing.assert_allclose(lse[1], 0.3 * (q[1] * k[1].repeat(2, 0)).sum(-1))
    assert np.all(out[5] == 0)                                            # behind the last sequence
    same, _ = C.prompt_attn(q, np.ones_like(k), v, [0, 6], 0.3)
    np.testing.assert_allclose(same[3, 0], v[:4, 0].mean(0))              # equal keys: the mean of what is seen


def test_block_map_gives_nothing_back_that_the_ring_has_no_room_for():
    """Request 0's four blocks are in the ring already: 8 + 4 are more than the 10 there are, whatever request 1 takes."""
    table, ring = np.array([[4, 5, 6, 7, 0, 0], [0] * 6]), np.arange(10)
    r = C.block_map([0, 96], [64, 0], table, ring, [7, 8], 96, 10)
    assert r["bad"] == {"block"} and r["state"].tolist() == [3, 2] and np.array_equal(r["ring"], ring)
    assert r["table"][1].tolist() == [7, 8, 9, 0, 1, 2] and r["granted"].tolist() == [0, 96]
    r = C.block_map([0, 96], [64, 0], table, ring, [7, 6], 96, 10)
    assert not r["bad"] and r["state"].tolist() == [3, 4] and r["ring"].tolist() == [0, 1, 2, 4, 5, 6, 7, 7, 8, 9]

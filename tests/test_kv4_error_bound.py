"""How far a value of the 4-bit cache may be off, as the README states it, by the plain definition of its codes and scales."""
import numpy as np
import pytest

from oracle import cache as C
from workloads import bf16_bits_to_f32

LOW, TOP = 6 * 2.0 ** -14, 61440.0


def stored(x):
    return C.kv4_decode(*C.kv4_encode(x))


def groups(seed, lo, hi, n):
    """Sixteen bf16 values each: a largest from [lo, hi] (bits), values below it, those near the middle of the widest gap among them."""
    g = np.random.default_rng(seed)
    a = np.unique(np.concatenate([[lo, lo + 1, hi - 1, hi], g.integers(lo, hi + 1, n)]))
    bits = (a[:, None] * np.concatenate([[1.0], g.uniform(0, 1, 7), np.zeros(8)])).astype(np.int64)
    bits[:, 0] = a
    top = bf16_bits_to_f32(a.astype(np.uint16)).astype(np.float64)
    scale = np.array([C.SCALE4[C.kv4_encode(np.full(16, t))[1][0]] for t in top])
    five = (np.float32(5) * scale.astype(np.float32)).view(np.uint32) >> 16
    bits[:, 8:] = five[:, None] + np.arange(-4, 4)  # about 5 scales
    x = bf16_bits_to_f32(bits.astype(np.uint16)).astype(np.float64)
    return np.minimum(x, top[:, None]), top


@pytest.mark.parametrize("lo,hi", [(0x0001, 0x39bf), (0x3500, 0x39c0), (0x39c0, 0x4770), (0x39c0, 0x3a60), (0x4740, 0x4770)])
def test_the_stated_bounds(lo, hi):
    x, top = groups(lo + hi, lo, hi, 150)
    off = np.abs(stored(x) - x).max(-1)
    assert np.all(off <= np.where(top > LOW, top * 3 / 16, top / 6 + 2.0 ** -17))


def test_the_bound_of_large_groups_is_met_and_does_not_hold_for_small_ones():
    assert bf16_bits_to_f32(np.array([0x39c0, 0x4770], np.uint16)).tolist() == [LOW, TOP]
    x = np.zeros(16)
    x[0], x[1] = 2.0 ** -19, -2.0 ** -20
    assert np.all(stored(x) == 0)
    x[0], x[1] = 2 * TOP, TOP / 2
    assert stored(x)[0] == TOP
    x, top = groups(7, 0x3e00, 0x4600, 200)
    assert np.max(np.abs(stored(x) - x).max(-1) / top) > 0.18
    x, top = groups(8, 0x3600, 0x3780, 60)
    assert np.max(np.abs(stored(x) - x).max(-1) / top) > 0.2

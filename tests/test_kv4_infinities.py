"""Infinities in what the 4-bit attention reads: rows of every kind of item, whole and split contexts.

No tolerances: an infinity decides a row as a whole (NaN, or untouched), and the rows beside it are bit for bit those of the
call without it."""
import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from tests.test_attn_kv4 import Case
from workloads import bf16_bits_to_f32

torch = pytest.importorskip("torch")

# 8 rows a verify item, 16, 21 (with a dump of logits by the kernel of many rows, without one by that of few), 56, 63 tokens
KINDS = [(2, 1, 64, 3, True), (4, 1, 128, 3, True), (6, 2, 64, 6, True), (6, 2, 64, 6, False), (8, 1, 128, 6, True),
         (4, 1, 128, 0, False), (1, 1, 64, 62, True)]


def batch(Hq, Hkv, D, k, chunk, seed=100):
    """A context of one key for its first row, a longer one, and a request with lists."""
    c = Case(seed, Hq, Hkv, D, k, [k + 1, 300 + k, 140], [1, 1, 0], verify_chunk=chunk, draft_chunk=chunk)
    c.cnt[2] = c.idx.shape[2]
    return c


def values(d):
    return torch.from_numpy(bf16_bits_to_f32(d["out"].cpu().numpy().view(np.uint16)))


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [64, 2048])
@pytest.mark.parametrize("bits,codes", [(0x7f80, (9, 16)), (-0x80, (1, 8))])
@pytest.mark.parametrize("Hq,Hkv,D,k,dump", KINDS)
def test_an_infinite_query_whose_scores_are_all_minus_infinity_is_nan(Hq, Hkv, D, k, dump, bits, codes, chunk):
    """The element's sign is the opposite of every key's: no score is NaN, and none is there to subtract from."""
    c = batch(Hq, Hkv, D, k, chunk)
    c.k4[..., 5] = c.g.integers(*codes, c.k4.shape[:-1])
    d, e = c.device(dump), c.device(dump)
    rows, lse = np.zeros((c.T, Hq, D), bool), np.zeros((2, Hq, k + 1), bool)
    for b, j, h in ((0, 0, 0), (0, k, Hq - 1), (1, min(1, k), 0), (1, k, Hq - 1)):
        e["q"][b * (k + 1) + j, h, 5] = bits
        rows[b * (k + 1) + j, h] = lse[b, h, j] = True
    e["q"][2 * (k + 1), 0, 5] = bits
    rows[2 * (k + 1), 0] = True
    for x in (d, e):
        c.call(x)
        assert P.pillar_get_error(x["ws"]) == 0
    at, z = torch.from_numpy(rows), torch.from_numpy(lse)
    got, want = values(e), values(d)
    assert torch.all(torch.isnan(got[at])) and torch.equal(got[~at], want[~at])
    got, want = e["lse"].cpu(), d["lse"].cpu()
    assert torch.all(torch.isnan(got[z])) and torch.equal(got[~z], want[~z])
    if dump:  # the logits are the scores themselves
        off = 0
        for b in range(2):
            n = int(c.lens[b])
            got, want = (x["logits"][off:off + Hq * (k + 1) * n].view(Hq, k + 1, n).cpu() for x in (e, d))
            assert torch.all(torch.isneginf(got[z[b]])) and torch.equal(got[~z[b]], want[~z[b]])
            off += Hq * (k + 1) * n


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7f80, -0x80, 0x7fc0])
@pytest.mark.parametrize("Hq,k", [(2, 3), (4, 3), (8, 6)])
def test_a_row_that_sees_no_position_is_zero_whatever_its_query(Hq, k, bits):
    c = Case(101, Hq, 1, 64, k, [2, 20], [1, 1])  # the first k - 1 rows of the first request see nothing
    d = c.device()
    d["q"][:k + 1] = bits
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == P.FLAG_REQUEST
    out, z = values(d), d["lse"].cpu()
    assert torch.all(out[:k - 1] == 0) and torch.all(torch.isneginf(z[0, :, :k - 1]))
    assert torch.all(torch.isnan(out[k - 1:k + 1])) and torch.all(torch.isnan(z[0, :, k - 1:]))
    assert torch.all(torch.isfinite(out[k + 1:])) and torch.all(torch.isfinite(z[1]))


def with_a_bad_key(Hq, Hkv, D, k, chunk, what):
    """Position 40 of the second request and of the lists' has an infinite scale in its second group of the last KV head."""
    c = batch(Hq, Hkv, D, k, chunk, seed=102)
    c.idx[2, Hkv - 1, 0] = 40
    for b in (1, 2):
        at = (int(c.table[b, 2]), Hkv - 1, 8)
        codes, scales = (c.k4, c.ks) if what == "k" else (c.v4, c.vs)
        codes[at][16:32] = c.g.integers(1, 8, 16)
        scales[at][1] = 0xf8
    return c


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [64, 2048])
@pytest.mark.parametrize("Hq,Hkv,D,k,dump", KINDS)
def test_a_key_whose_score_is_minus_infinity_counts_as_one_that_is_not_there(Hq, Hkv, D, k, dump, chunk):
    """(The definition's weight of 0, within its usual tolerances.)"""
    c = with_a_bad_key(Hq, Hkv, D, k, chunk, "k")
    c.q[..., 16:32] |= 0x8000
    d = c.device(dump)
    c.call(d)
    c.check(d)


@pytest.mark.gpu
@pytest.mark.parametrize("chunk", [64, 2048])
@pytest.mark.parametrize("what", ["k", "v"])
@pytest.mark.parametrize("Hq,Hkv,D,k,dump", KINDS)
def test_an_infinite_value_reaches_the_rows_that_see_it(Hq, Hkv, D, k, dump, what, chunk):
    """A score of +inf: NaN.  An infinite value of V: its dimensions are not finite; they may be NaN in rows that do not see it, but
    all of these see it.  Everything else is bit for bit what it is with a scale of 1 there."""
    c = with_a_bad_key(Hq, Hkv, D, k, chunk, what)
    c.q[..., 16:32] &= 0x7fff
    e = c.device(dump)
    (c.ks if what == "k" else c.vs)[(c.ks if what == "k" else c.vs) == 0xf8] = 0x78
    d = c.device(dump)
    for x in (d, e):
        c.call(x)
        assert P.pillar_get_error(x["ws"]) == 0
    heads = slice(Hq - Hq // Hkv, Hq)
    rows, lse = np.zeros((c.T, Hq, D), bool), np.zeros((2, Hq, k + 1), bool)
    rows[k + 1:, heads, slice(None) if what == "k" else slice(16, 32)] = True
    lse[1, heads] = what == "k"
    at, z = torch.from_numpy(rows), torch.from_numpy(lse)
    got, want = values(e), values(d)
    assert torch.all(torch.isnan(got[at]) if what == "k" else ~torch.isfinite(got[at])) and torch.equal(got[~at], want[~at])
    got, want = e["lse"].cpu(), d["lse"].cpu()
    assert torch.all(torch.isnan(got[z])) and torch.equal(got[~z], want[~z])


@pytest.mark.gpu
@pytest.mark.parametrize("bits", [0x7f80, 0x7fc0])
@pytest.mark.parametrize("Hq,k", [(2, 3), (4, 3), (8, 6)])
def test_a_position_that_is_skipped_is_one_to_see(Hq, k, bits):
    c = Case(103, Hq, 1, 64, k, [20, 30, 30, 40], [1, 0, 0, 0])
    c.table[0] = c.blocks
    c.cnt[:, 0] = [0, 2, 0, 3]
    c.idx[1, 0, :2] = [-1, 30]
    d = c.device()
    d["q"][:k + 3] = bits
    c.call(d)
    assert P.pillar_get_error(d["ws"]) == P.FLAG_SLOT | P.FLAG_INDEX
    out = values(d)
    assert torch.all(torch.isnan(out[:k + 2])) and torch.all(torch.isnan(d["lse"]))
    assert torch.all(out[k + 2] == 0) and torch.all(torch.isfinite(out[k + 3]))  # an empty list; a sound one

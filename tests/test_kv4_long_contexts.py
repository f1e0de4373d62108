"""pillar_attn_kv4 over contexts from 8192 positions on, with the default item sizes: items of 2048 keys, or those that the call
cuts so that every CTA has one, and from a plan of pillar_attn_plan, which does not cut.

Tolerances: those of test_attn_kv4.py, whose LSE bound is stated for contexts to 4096 keys.  For 100001: an item has at most 2048
keys, whose weights a lane sums in at most 64 roundings, 3 exchanges and 4 warps; its record is one of at most 98, each a rounding
and an exponential (2^-21 relative, its argument 2^-23 |s|): (64 + 3 + 4 + 98) 2^-24 + 2^-20 + 8 * 2^-23 < 1.3e-5 relative, absolute
in the LSE.  The bound there, 2^-18 + (1 + |lse|) 2^-20, is 1.3e-5 from an LSE of 9 = log 8192 on, and these contexts' are above it:
about log n + 1/2, as the scores' deviation is 1.  (98 records come with an LSE of 12, where the bound is 1.6e-5; the 8 items of a
context of 8192 keys make 4e-6.)  What the merge adds to an output, 98 * 2^-24 sum p |v|, is within the 2^-16 there."""
import pytest

import sparse_self_speculative_pillar_gb300 as P
from tests.test_attn_kv4 import Case

torch = pytest.importorskip("torch")

CASES = [  # Hq, Hkv, D, k, lens, modes, dump: the item size on 152 SMs
    (8, 2, 64, 0, [100001, 9000, 8192, 700], [1, 1, 1, 0], False),  # cut to 1344 keys
    (8, 2, 64, 0, [100001, 8191], [1, 1], True),                    # cut to 1024 (152 pieces)
    (2, 1, 128, 2, [65537, 12000, 30], [1, 0, 1], True),            # 1024, and lists of more than one item
    (8, 2, 128, 3, [40000, 8191, 20001], [1, 1, 0], True),          # 16 rows: 1024
    (4, 1, 64, 5, [20000, 8192, 8193], [1, 1, 0], False),           # 24 rows: the planner's own
    (16, 2, 64, 3, [30000, 8200, 5000], [1, 0, 1], True),           # 32 rows: the planner's own
]


def guarded(c, dump):
    """The case's buffers, with a workspace of exactly the size asked for and bytes behind it that nobody may touch."""
    d, n = c.device(dump), P.pillar_attn_workspace_bytes(c.shape)
    d["room"] = torch.full((n + 4096,), 0xa5, dtype=torch.uint8, device="cuda")
    d["ws"] = d["room"][:n]
    return d


@pytest.mark.gpu
@pytest.mark.parametrize("Hq,Hkv,D,k,lens,modes,dump", CASES)
def test_long_contexts_in_one_call_and_from_a_plan(Hq, Hkv, D, k, lens, modes, dump):
    c = Case(110, Hq, Hkv, D, k, lens, modes)
    d, f = guarded(c, dump), guarded(c, dump)
    c.call(d)
    c.check(d)
    P.pillar_attn_plan(c.shape, f["mode"], f["len"], f["cnt"], f["ws"])
    for _ in range(2):
        f["out"].fill_(0x7fc0)
        P.pillar_attn_run_kv4(c.shape, f["q"], f["k4"], f["v4"], f["ks"], f["vs"], f["table"], f["idx"], f["out"], f["logits"],
                              f["lse"], f["ws"])
        c.check(f)
    if dump:  # a score does not go by the item it belongs to
        assert torch.equal(d["logits"], f["logits"])
    for x in (d, f):
        assert torch.all(x["room"][x["ws"].numel():] == 0xa5)


@pytest.mark.gpu
def test_a_plan_may_ask_for_the_size_that_the_call_would_take():
    """A plan whose shape has the call's cut as its verify_chunk gives the call's outputs bit for bit."""
    lens, modes = [50000, 9000, 20], [1, 1, 0]
    c, cut = Case(111, 8, 2, 64, 0, lens, modes), Case(111, 8, 2, 64, 0, lens, modes, verify_chunk=1024)
    d, e = c.device(), cut.device()
    c.call(d)
    P.pillar_attn_plan(cut.shape, e["mode"], e["len"], e["cnt"], e["ws"])
    P.pillar_attn_run_kv4(cut.shape, e["q"], e["k4"], e["v4"], e["ks"], e["vs"], e["table"], e["idx"], e["out"], e["logits"],
                          e["lse"], e["ws"])
    assert P.pillar_get_error(d["ws"]) == 0 and P.pillar_get_error(e["ws"]) == 0
    for name in ("out", "logits", "lse"):
        assert torch.equal(d[name], e[name]), name

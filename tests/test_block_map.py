"""pillar_block_map: block tables, slot tables and new tokens' slots from request lengths, bit for bit against the plain
definition; shortage, rollback, bad inputs, capacities; the slots serve the page-size-1 calls."""
import ctypes

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C

torch = pytest.importorskip("torch")
SENTINEL = -77


def shape_of(B, num_blocks, max_len):
    return P.make_shape(B=B, Hq=1, Hkv=1, D=64, k=0, row_lo=0, max_sparse=0, max_len=max_len, num_slots=num_blocks * 16)


def test_host_checks():
    P.build()
    lib = P.load()
    s = shape_of(2, 8, 64)
    n = P.pillar_block_map_workspace_bytes(s)
    assert n > 0 and n % 256 == 0
    a = ctypes.c_void_p(256)
    good = [a, a, a, 4, a, a, a, a, a, 64, a, a, 64, a, 1 << 20, None]

    def call(shape=s, **over):
        args = list(good)
        for i, v in over.items():
            args[int(i[1:])] = v
        return lib.pillar_block_map(ctypes.byref(shape), *args)

    for i in (0, 1, 2, 4, 5, 6, 7, 8, 10, 11):  # a null or misaligned array
        assert call(**{f"a{i}": None}) == -1
        assert call(**{f"a{i}": ctypes.c_void_p(257)}) == -1
    assert call(a7=ctypes.c_void_p(260)) == -1 and call(a8=ctypes.c_void_p(264)) == -1  # kv_off 8, slot_table 16
    assert call(a3=0) == -1 and call(a9=-1) == -1 and call(a12=-1) == -1
    assert call(a13=None) == -2 and call(a13=ctypes.c_void_p(128)) == -2 and call(a14=n - 1) == -2
    assert call(shape=P.make_shape(B=2, Hq=1, Hkv=1, D=64, k=0, row_lo=0, max_sparse=0, max_len=64, num_slots=24)) == -1
    with pytest.raises(P.PillarError):
        P.pillar_block_map_workspace_bytes(shape_of(-1, 8, 64))


def play(req_len, prev_len, table, ring, state, max_len, num_blocks, slot_cap=None, new_cap=None, stream=None):
    """One call on the GPU; returns its outputs on the host and its flags."""
    B = len(req_len)
    s = shape_of(B, num_blocks, max_len)
    dev = lambda x, t=torch.int32: torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")  # noqa: E731
    want = C.block_map(req_len, prev_len, table, ring, state, max_len, num_blocks)
    t, r, st = dev(table), dev(ring), dev(state)
    full = lambda n, dt=torch.int32: torch.full((n,), SENTINEL, dtype=dt, device="cuda")  # noqa: E731
    granted, kv_off, new_off = full(B), full(B + 1, torch.int64), full(B + 1)
    slots = full(len(want["slots"]) + 5 if slot_cap is None else slot_cap)
    new = full(len(want["new_slots"]) + 3 if new_cap is None else new_cap)
    ws = torch.empty(P.pillar_block_map_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    P.pillar_block_map(s, dev(req_len), dev(prev_len), t, r, st, granted, kv_off, slots, new_off, new, ws, stream=stream)
    flags = P.pillar_get_error(ws, stream=stream)
    got = dict(table=t, ring=r, state=st, granted=granted, kv_off=kv_off, new_off=new_off, slots=slots, new_slots=new)
    return {k: v.cpu().numpy() for k, v in got.items()}, want, flags


def check(got, want):
    for k in ("table", "ring", "state", "granted", "kv_off", "new_off"):
        np.testing.assert_array_equal(got[k], want[k], err_msg=k)
    for k in ("slots", "new_slots"):
        n = min(len(want[k]), len(got[k]))
        np.testing.assert_array_equal(got[k][:n], want[k][:n], err_msg=k)
        assert np.all(got[k][n:] == SENTINEL), k


def batch(seed, B, max_len, zero=0.2, spare=3):
    """Random previous and next lengths (some empty, some shrinking), tables over a shuffled pool, the rest free."""
    g = np.random.default_rng(seed)
    prev = g.integers(0, max_len + 1, B) * (g.random(B) >= zero)
    req = np.where(g.random(B) < 0.5, np.minimum(max_len, prev + g.integers(0, 20, B)), g.integers(0, max_len + 1, B))
    req = req * (g.random(B) >= zero)
    W = -(-max_len // 16) + 1
    nb = -(-prev // 16)
    need = int(np.maximum(-(-req // 16) - nb, 0).sum())
    total = int(nb.sum()) + need + spare
    perm = g.permutation(total)
    table = np.full((B, W), SENTINEL)
    at = 0
    for b in range(B):
        table[b, :nb[b]] = perm[at:at + nb[b]]
        at += nb[b]
    free = perm[at:]
    ring = np.full(total, SENTINEL)
    head = int(g.integers(0, total))
    ring[(head + np.arange(len(free))) % total] = free
    return req, prev, table, ring, [head, len(free)], total


@pytest.mark.gpu
@pytest.mark.parametrize("seed,B,max_len", [(0, 1, 1), (1, 1, 5000), (2, 7, 40), (3, 128, 700), (4, 1024, 33), (5, 1025, 90),
                                            (6, 2500, 20), (7, 33, 16), (8, 300, 4097)])
def test_matches_the_definition(seed, B, max_len):
    req, prev, table, ring, state, total = batch(seed, B, max_len)
    got, want, flags = play(req, prev, table, ring, state, max_len, total)
    assert flags == 0 and not want["bad"]
    check(got, want)


@pytest.mark.gpu
def test_many_empty_requests_between_long_ones():
    B = 3000
    prev = np.zeros(B, np.int64)
    req = np.zeros(B, np.int64)
    req[[0, 1500, 2999]] = [5000, 1, 9000]
    got, want, flags = play(req, prev, np.full((B, 563), SENTINEL), np.arange(900)[::-1], [899, 900], 9000, 900)
    assert flags == 0
    check(got, want)


@pytest.mark.gpu
def test_shortage_denies_the_first_that_does_not_fit_and_all_after_it():
    req, prev, table, ring, state, total = batch(11, 40, 300, spare=0)
    state = [state[0], state[1] // 2]
    got, want, flags = play(req, prev, table, ring, state, 300, total)
    assert flags == P.FLAG_BLOCK and want["bad"] == {"block"}
    check(got, want)
    got, want, flags = play(req, prev, table, ring, [state[0], 0], 300, total)
    assert flags == P.FLAG_BLOCK
    check(got, want)


@pytest.mark.gpu
def test_bad_lengths_blocks_and_ring_state_are_flagged():
    table = np.array([[0, 1, 9], [2, 3, 4], [5, 6, 7], [-1, 8, 0]])
    req, prev = [16, -1, 99, 20], [16, 33, -3, 18]
    got, want, flags = play(req, prev, table, np.arange(10), [3, 2], 48, 10)
    assert flags == P.FLAG_REQUEST | P.FLAG_SLOT and want["bad"] == {"request", "slot"}
    check(got, want)
    for state in ([-1, 2], [10, 0], [0, 11], [0, -5]):
        got, want, flags = play([20, 3], [16, 3], table[:2], np.arange(10), state, 48, 10)
        assert flags == P.FLAG_BLOCK
        check(got, want)


@pytest.mark.gpu
@pytest.mark.parametrize("slot_cap,new_cap", [(0, 0), (1, 2), (6, 1), (4097, 5)])
def test_entries_past_the_capacities_are_not_written(slot_cap, new_cap):
    req, prev, table, ring, state, total = batch(12, 30, 700, zero=0)
    got, want, flags = play(req, prev, table, ring, state, 700, total, slot_cap, new_cap)
    assert flags == P.FLAG_COUNT
    check(got, want)


@pytest.mark.gpu
def test_steps_in_a_row_captured_and_on_another_stream():
    """A batch that grows, rolls back and finishes, each step on what the one before left; the same steps replayed from a
    captured graph on fresh buffers write the same."""
    num, B, max_len = 64, 6, 200
    lens = [[0] * 6, [5, 40, 16, 0, 100, 17], [14, 49, 25, 9, 109, 26], [9, 41, 17, 1, 100, 18], [0, 42, 18, 2, 101, 0],
            [33, 43, 19, 3, 102, 200]]
    s = shape_of(B, num, max_len)

    def fresh():
        i32 = dict(dtype=torch.int32, device="cuda")
        return dict(table=torch.full((B, 13), SENTINEL, **i32), ring=torch.arange(num, **i32).flip(0).contiguous(),
                    state=torch.tensor([60, num], **i32), granted=torch.zeros(B, **i32),
                    kv_off=torch.zeros(B + 1, dtype=torch.int64, device="cuda"), slots=torch.full((1200,), SENTINEL, **i32),
                    new_off=torch.zeros(B + 1, **i32), new=torch.full((600,), SENTINEL, **i32),
                    ws=torch.empty(P.pillar_block_map_workspace_bytes(s), dtype=torch.uint8, device="cuda"),
                    lens=[torch.tensor(x, **i32) for x in lens])

    def steps(d, stream=None):
        for a, b in zip(d["lens"], d["lens"][1:]):
            P.pillar_block_map(s, b, a, d["table"], d["ring"], d["state"], d["granted"], d["kv_off"], d["slots"],
                               d["new_off"], d["new"], d["ws"], stream=stream)

    a = fresh()
    steps(a)
    table, ring, state = np.full((B, 13), SENTINEL), np.arange(num)[::-1], [60, num]
    for p, n in zip(lens, lens[1:]):
        w = C.block_map(n, p, table, ring, state, max_len, num)
        table, ring, state = w["table"], w["ring"], w["state"]
    for k, v in (("table", table), ("ring", ring), ("state", state), ("kv_off", w["kv_off"])):
        np.testing.assert_array_equal(a[k].cpu().numpy(), v, err_msg=k)
    np.testing.assert_array_equal(a["slots"].cpu().numpy()[:len(w["slots"])], w["slots"])
    b, g, side = fresh(), torch.cuda.CUDAGraph(), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.graph(g, stream=side):
        steps(b)
    g.replay()
    torch.cuda.synchronize()
    c = fresh()
    side.wait_stream(torch.cuda.current_stream())
    steps(c, stream=side)
    torch.cuda.synchronize()
    for k in ("table", "ring", "state", "granted", "kv_off", "slots", "new_off"):
        assert torch.equal(a[k], b[k]) and torch.equal(a[k], c[k]), k


@pytest.mark.gpu
def test_the_binding_refuses_tensors_that_do_not_fit():
    s = shape_of(2, 8, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = torch.empty(P.pillar_block_map_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    good = [torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros((2, 4), **i32), torch.zeros(8, **i32),
            torch.zeros(2, **i32), torch.zeros(2, **i32), torch.zeros(3, dtype=torch.int64, device="cuda"),
            torch.zeros(16, **i32), torch.zeros(3, **i32), torch.zeros(16, **i32), ws]
    P.pillar_block_map(s, *good)
    for i in range(10):
        for wrong in (good[i].cpu(), good[i].float(), good[i][:-1] if i in (0, 1, 3, 4, 5, 6, 8) else good[i].unsqueeze(0)):
            args = list(good)
            args[i] = wrong
            with pytest.raises(ValueError):
                P.pillar_block_map(s, *args)
    with pytest.raises(ValueError):
        P.pillar_block_map(s, *good[:2], torch.zeros((2, 8), **i32)[:, ::2], *good[3:])
    with pytest.raises(P.PillarError):
        P.pillar_block_map(s, *good[:10], ws[:256])


@pytest.mark.gpu
def test_lengths_up_to_the_largest_int():
    """A length whose rounding up to whole blocks passes 31 bits needs more blocks than any pool has: refused, nothing taken."""
    most, B = 2 ** 31 - 1, 2
    s = shape_of(B, 10, most)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    table = torch.zeros((B, 2 ** 27), dtype=torch.int32, device="cuda")
    ring, state, granted = i32(list(range(10))), i32([0, 10]), i32([SENTINEL] * B)
    kv_off, new_off = torch.zeros(B + 1, dtype=torch.int64, device="cuda"), i32([0] * (B + 1))
    slots, new = i32([SENTINEL] * 64), i32([SENTINEL] * 64)
    ws = torch.empty(P.pillar_block_map_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    P.pillar_block_map(s, i32([20, most]), i32([0, 0]), table, ring, state, granted, kv_off, slots, new_off, new, ws)
    assert P.pillar_get_error(ws) == P.FLAG_BLOCK
    assert granted.tolist() == [20, 0] and state.tolist() == [2, 8] and kv_off.tolist() == [0, 20, 20]
    assert slots.tolist()[:21] == list(range(20)) + [SENTINEL] and table[:, :3].tolist() == [[0, 1, 0], [0, 0, 0]]


def test_granted_lengths_in_the_place_of_the_lengths_read_are_refused():
    lib, s = P.load(), shape_of(2, 8, 64)
    at = [ctypes.c_void_p(256 * (i + 1)) for i in range(16)]
    args = [at[0], at[1], at[2], 4, at[3], at[4], at[5], at[6], at[7], 64, at[8], at[9], 64, at[10], 1 << 20, None]
    for other in (0, 1):
        wrong = list(args)
        wrong[6] = wrong[other]
        assert lib.pillar_block_map(ctypes.byref(s), *wrong) == -1


@pytest.mark.gpu
@pytest.mark.parametrize("count,took", [(8, 6), (7, 7), (10, 1), (6, 6), (9, 0)])
def test_more_given_back_than_the_ring_has_room_for(count, took):
    """Tables that hold blocks which the ring holds too: giving them back would write into places that the same call pops."""
    table = np.array([[4, 5, 6, 7] + [SENTINEL] * 4, [SENTINEL] * 8])
    for seed in range(3):
        ring = np.random.default_rng(seed).permutation(10)
        got, want, flags = play([0, 16 * took], [64, 0], table, ring, [7, count], 128, 10)
        over = count + 4 > 10
        assert flags == (P.FLAG_BLOCK if over else 0) and want["bad"] == ({"block"} if over else set())
        check(got, want)
        if over:
            assert list(got["state"]) == [(7 + took) % 10, count - took]
            np.testing.assert_array_equal(got["ring"], ring)


@pytest.mark.gpu
def test_many_more_given_back_than_the_ring_has_room_for():
    """The same with hundreds of requests that give and take in one call: the outcome does not depend on timing."""
    B, num = 600, 2000
    table = np.tile(np.arange(9), (B, 1)) + 3 * np.arange(B)[:, None]
    prev, req = np.where(np.arange(B) % 2, 0, 130), np.where(np.arange(B) % 2, 96, 0)
    ring = np.random.default_rng(5).permutation(num)
    for _ in range(3):
        got, want, flags = play(req, prev, table, ring, [1999, num], 144, num)
        assert flags == P.FLAG_BLOCK and want["bad"] == {"block"}
        check(got, want)


def test_extents_past_32_bits_are_refused():
    wide = lambda n: torch.empty((1, n), dtype=torch.int32, device="meta")  # noqa: E731
    assert P._dim32("block_table", wide(2 ** 31 - 1), 1, 2) == 2 ** 31 - 1
    for n in (2 ** 31, 2 ** 32 + 4):
        with pytest.raises(ValueError):
            P._dim32("block_table", wide(n), 1, 2)


@pytest.mark.gpu
def test_a_table_wider_than_32_bits_is_refused():
    """2^32 + 4 entries a row (17 GB, never touched): taken as four, most of the requests' blocks would have no place."""
    s = shape_of(1, 8, 64)
    i32 = dict(dtype=torch.int32, device="cuda")
    ws = torch.empty(P.pillar_block_map_workspace_bytes(s), dtype=torch.uint8, device="cuda")
    small = [torch.zeros(1, **i32), torch.zeros(1, **i32), torch.empty((1, 2 ** 32 + 4), **i32), torch.zeros(8, **i32),
             torch.zeros(2, **i32), torch.zeros(1, **i32), torch.zeros(2, dtype=torch.int64, device="cuda"),
             torch.zeros(16, **i32), torch.zeros(2, **i32), torch.zeros(16, **i32), ws]
    with pytest.raises(ValueError):
        P.pillar_block_map(s, *small)

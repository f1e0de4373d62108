"""The 4-bit cache's operators together, as a serving loop uses them: block map, append, prompt attention, verify and draft
attention, Top-K, the next draft step's lists, and the cache read back for a bf16 pool and for another prompt pass.

Beside the 4-bit cache the loop of test_cache_run.py keeps its 8-bit and bf16 ones through the same maps.  Values held are compared
exactly, the attention is held to the bounds of test_attn_kv4.py; the bf16 step on the values read back is held to its stated relative
error against the same definition."""
import types

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from tests import test_attn_kv4 as A4
from tests import test_cache_run as R
from workloads import f32_to_bf16_bits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
Hq, Hkv, D, K = R.Hq, R.Hkv, R.D, R.K
dev, bits, f64 = R.dev, R.bits, R.f64


class Loop(R.Loop):
    def __init__(self, B, seed):
        super().__init__(B, seed)
        z = lambda d: torch.zeros((R.BLOCKS, Hkv, 16, d), dtype=torch.uint8, device="cuda")  # noqa: E731
        self.cache4 = [z(D // 2), z(D // 2), z(D // 16), z(D // 16)]
        self.held = [[np.zeros((R.BLOCKS, Hkv, 16, d), np.uint8) for d in (D, D // 16)] for _ in "kv"]  # codes, scale bytes

    def grow(self, lens, k=None, v=None):
        super().grow(lens, k, v)
        if k is not None:
            P.pillar_kv4_append(self.shape, bits(k), bits(v), self.lens, self.new_off, self.table, *self.cache4, self.flags)

    def mirror(self, lens, k=None, v=None):
        super().mirror(lens, k, v)
        w = self.want
        for i, x in enumerate((k, v)):
            if x is not None:
                self.held[i] = C.kv4_append(*self.held[i], f64(x), w["lens"], self.new_off.cpu().numpy(), w["table"])
            codes, scales = (self.cache4[j].cpu().numpy() for j in (i, i + 2))
            np.testing.assert_array_equal(scales, self.held[i][1])
            np.testing.assert_array_equal(C.kv4_decode(C.kv4_unpack(codes), scales), C.kv4_decode(*self.held[i]))

    def attend(self, d, stream=None):
        P.pillar_attn_kv4(self.shape, d["q"], *self.cache4, self.table, d["mode"], self.lens, self.idx, self.cnt, d["out"],
                          d["logits"], d["lse"], self.ws, stream=stream)

    def check_attention(self, d, modes):
        w, c = self.want, object.__new__(A4.Case)
        c.Hq, c.Hkv, c.D, c.k, c.scale, c.modes, c.lens = Hq, Hkv, D, K, D ** -0.5, np.array(modes), w["lens"]
        c.V, c.q, c.table = int((c.modes == 1).sum()), d["q"].cpu().numpy().view(np.uint16), w["table"]
        (c.k4, c.ks), (c.v4, c.vs) = self.held
        c.idx, c.cnt = self.idx.cpu().numpy(), self.cnt.cpu().numpy()
        c.check(d)

    def read(self):
        """Every context out of the 4-bit cache, held to the definition: rows, and their offsets."""
        w, off = self.want, np.concatenate([[0], np.cumsum(self.want["lens"])])
        k, v = (torch.full((int(off[-1]), Hkv, D), 0x7fc1, dtype=torch.int16, device="cuda") for _ in "kv")
        P.pillar_kv4_read(self.shape, *self.cache4, self.table, dev(np.zeros(self.B), torch.int32), dev(off, torch.int32), k, v,
                          self.flags)
        assert int(self.flags) == 0
        for x, held in zip((k, v), self.held):
            want = C.kv_read(C.kv4_decode(*held), w["table"], np.zeros(self.B, int), off, np.zeros(tuple(x.shape)))
            np.testing.assert_array_equal(f64(x.cpu().numpy().view(np.uint16)), want)
        return k, v, off

    def check_moved(self, d, modes):
        """The contexts read back, stored into bf16 pools by their slots: the bf16 step on them."""
        k, v, off = self.read()
        kept = self.kb, self.vb, self.ctx_k, self.ctx_v
        self.kb, self.vb = (torch.zeros_like(self.kb) for _ in "kv")
        P.pillar_kv_append(self.shape, k, v, self.slots[:len(k)].contiguous(), self.kb, self.vb, self.flags)
        assert int(self.flags) == 0
        self.ctx_k, self.ctx_v = ([f64(x.cpu().numpy().view(np.uint16))[off[b]:off[b + 1]] for b in range(self.B)] for x in (k, v))
        self.check_bf16(d, modes)
        self.kb, self.vb, self.ctx_k, self.ctx_v = kept


def test_a_serving_loop():
    lens = np.array([37, 100, 16, 5])
    B = len(lens)
    loop = Loop(B, 11)

    def step(lens, with_rows=True):
        n = loop.new_rows(lens)
        kv = (R.rows(loop.g, n, Hkv), R.rows(loop.g, n, Hkv)) if with_rows else (None, None)
        loop.grow(lens, *kv)
        loop.mirror(lens, *kv)
        return kv

    R.prompts(loop, *step(lens), 0, B)
    lens = lens + K + 1
    step(lens)
    modes = [1] * B
    d = loop.outputs(modes)
    loop.attend(d)
    loop.select(d, B)
    loop.check_attention(d, modes)
    loop.check_select(d, B)
    loop.check_moved(d, modes)
    for _ in range(2):
        lens = lens + 1
        step(lens)
        loop.lists()
        d, modes = loop.outputs([0] * B), [0] * B
        loop.attend(d)
        assert int(loop.flags) == 0
        loop.check_attention(d, modes)
        loop.check_moved(d, modes)
    # tokens are taken back, request 2 is finished and its blocks serve a new prompt
    lens = np.array([lens[0] - 2, lens[1] - 20, 0, lens[3]])
    step(lens, with_rows=False)
    lens = np.array([lens[0] + K + 1, lens[1] + 1, 200, lens[3] + K + 1])
    R.prompts(loop, *step(lens), 2, 3)
    modes = [1, 0, 1, 1]
    loop.idx[1] = dev(loop.g.integers(0, lens[1], (Hkv, R.MAX_SPARSE)), torch.int32)
    loop.cnt[1] = dev([R.MAX_SPARSE, 17], torch.int32)
    d = loop.outputs(modes)
    loop.attend(d)
    loop.check_attention(d, modes)
    loop.check_moved(d, modes)
    # a prompt pass over the values that the cache holds
    k, v, off = loop.read()
    k, v = (x.cpu().numpy().view(np.uint16)[off[1]:off[3]] for x in (k, v))
    where = types.SimpleNamespace(g=loop.g, new_off=dev(off[1:4] - off[1], torch.int32))
    R.prompts(where, k, v, 0, 2)


def test_two_captured_steps_on_one_workspace():
    """A verify step (map, append, attention, Top-K, lists) and a draft step (map, append, lists, attention, read back of the new
    row) as two graphs that share the attention's workspace, replayed in turn on lengths and rows that change."""
    start, B = np.array([33, 70, 48]), 3
    eager, graph = Loop(B, 12), Loop(B, 12)
    g = eager.g
    first = (R.rows(g, int(start.sum()), Hkv), R.rows(g, int(start.sum()), Hkv))
    z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731

    def buffers(lp, nq):
        return dict(req=z(B), granted=z(B), new_slots=z(B * nq), mode=z(B) + (nq > 1), group=torch.arange(B, dtype=torch.int32, device="cuda"),
                    k=z(B * nq, Hkv, D).short(), v=z(B * nq, Hkv, D).short(), q=z(B * nq, Hq, D).short(),
                    out=z(B * nq, Hq, D).short(), logits=torch.zeros(Hq * (K + 1) * B * R.MAX_LEN, device="cuda"),
                    lse=torch.zeros((B, Hq, K + 1), device="cuda"), back=[z(B, Hkv, D).short() for _ in "kv"])

    def enqueue(lp, s, verify):
        P.pillar_block_map(lp.shape, s["req"], lp.lens, lp.table, lp.ring, lp.state, s["granted"], lp.kv_off, lp.slots, lp.new_off,
                           s["new_slots"], lp.map_ws)
        lp.lens.copy_(s["granted"])
        P.pillar_kv4_append(lp.shape, s["k"], s["v"], lp.lens, lp.new_off, lp.table, *lp.cache4, lp.flags)
        lists = lambda: P.pillar_draft_lists(lp.shape, B, lp.next_idx, lp.next_cnt, s["group"], lp.verify_len, lp.lens, lp.slots,  # noqa: E731
                                             lp.idx, lp.cnt, None, lp.flags)
        if verify:
            lp.verify_len.copy_(lp.lens)
        else:
            lists()
        P.pillar_attn_kv4(lp.shape, s["q"], *lp.cache4, lp.table, s["mode"], lp.lens, lp.idx, lp.cnt, s["out"], s["logits"], s["lse"],
                          lp.ws)
        if verify:
            P.pillar_topk_select(lp.shape, B, s["logits"], s["lse"], lp.lens, s["group"], lp.some, lp.next_idx, lp.next_cnt, lp.topk_ws)
        else:
            P.pillar_kv4_read(lp.shape, *lp.cache4, lp.table, lp.lens - 1, s["group4"], *s["back"], lp.flags)

    made = []
    for lp in (eager, graph):
        lp.grow(start, *first)
        lp.next_idx, lp.next_cnt, lp.verify_len, lp.some = z(B, Hkv, lp.shape.max_topk), z(B, Hkv), z(B), z(B) + 20
        lp.topk_ws = torch.empty(P.pillar_topk_workspace_bytes(lp.shape, B), dtype=torch.uint8, device="cuda")
        made.append([buffers(lp, K + 1), buffers(lp, 1)])
        made[-1][1]["group4"] = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    names = ("lens", "table", "ring", "state", "idx", "cnt", "next_idx", "next_cnt", "verify_len")
    saved = [getattr(graph, n).clone() for n in names] + [x.clone() for x in graph.cache4]
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()]
    for i, verify in enumerate((True, False)):
        with torch.cuda.graph(graphs[i]):
            enqueue(graph, made[1][i], verify)
    for x, y in zip([getattr(graph, n) for n in names] + graph.cache4, saved):
        x.copy_(y)
    lens = start
    for turn in range(6):
        verify = turn % 3 == 0
        i, nq = (0, K + 1) if verify else (1, 1)
        lens = lens + nq
        for name, heads in (("k", Hkv), ("v", Hkv), ("q", Hq)):
            x = bits(R.rows(g, B * nq, heads))
            for m in made:
                m[i][name].copy_(x)
        for m in made:
            m[i]["req"].copy_(dev(lens, torch.int32))
        enqueue(eager, made[0][i], verify)
        graphs[i].replay()
        torch.cuda.synchronize()
        for n in names:
            assert torch.equal(getattr(eager, n), getattr(graph, n)), (turn, n)
        for a, b in zip(eager.cache4 + made[0][i]["back"], graph.cache4 + made[1][i]["back"]):
            assert torch.equal(a, b), turn
        for n in ("out", "logits", "lse"):
            assert torch.equal(made[0][i][n], made[1][i][n]), (turn, n)
        for lp in (eager, graph):
            assert P.pillar_get_error(lp.map_ws) == 0 and P.pillar_get_error(lp.ws) == 0 and int(lp.flags) == 0


@pytest.mark.parametrize("heads,k", [(16, 3), (32, 6)])
def test_pools_past_32_bits(heads, k):
    """The same blocks at the start of small pools and at the end of pools of 4.9 GB; rows read back packed and 32 MB apart."""
    kv_heads, dim, lens, far = 8, 128, [300, 130, 77], 600000
    g = np.random.default_rng(13)
    n, nb = sum(lens), [-(-x // 16) for x in lens]
    near = sum(nb)
    rowset = lambda r, h: torch.from_numpy(f32_to_bf16_bits(g.standard_normal((r, h, dim)).astype(np.float32)).view(np.int16)).cuda()  # noqa: E731
    kn, vn, q = rowset(n, kv_heads), rowset(n, kv_heads), rowset(2 * (k + 1) + 1, heads)
    off, length = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32), dev(lens, torch.int32)
    mode, lists = dev([1, 0, 1], torch.int32), dev(g.integers(0, 130, (3, kv_heads, 40)), torch.int32)
    results = []
    for blocks in (near, far):
        table = np.full((3, max(nb)), -1)
        at = blocks - near
        for b in range(3):
            table[b, :nb[b]] = np.arange(at, at + nb[b])
            at += nb[b]
        s = P.make_shape(B=3, Hq=heads, Hkv=kv_heads, D=dim, k=k, max_sparse=40, max_len=300, num_slots=blocks * 16)
        cache = [torch.empty((blocks, kv_heads, 16, d), dtype=torch.uint8, device="cuda") for d in (64, 64, 8, 8)]
        t, flags = dev(table, torch.int32), dev([0], torch.int32)
        P.pillar_kv4_append(s, kn, vn, length, off, t, *cache, flags)
        out, lse = torch.zeros_like(q), torch.zeros((2, heads, k + 1), device="cuda")
        logits = torch.zeros(heads * (k + 1) * (lens[0] + lens[2]), device="cuda")
        ws = torch.empty(P.pillar_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        P.pillar_attn_kv4(s, q, *cache, t, mode, length, lists, dev(np.full((3, kv_heads), 40), torch.int32), out, logits, lse, ws)
        back = [torch.zeros((n, kv_heads, dim), dtype=torch.int16, device="cuda") for _ in "kv"]
        if blocks == far:
            stride = 1 << 24
            back = [torch.empty((n - 1) * stride + kv_heads * dim, dtype=torch.int16, device="cuda").as_strided(
                (n, kv_heads, dim), (stride, dim, 1)) for _ in "kv"]
        P.pillar_kv4_read(s, *cache, t, torch.zeros_like(length), off, *back, flags)
        assert int(flags) == 0 and P.pillar_get_error(ws) == 0
        # (the scales of the positions that there are: what lies behind a context's end in its last block nobody wrote)
        scales = [cache[2][table[b, i // 16], :, i % 16] for b in range(3) for i in range(lens[b])]
        results.append((torch.stack(scales), out, logits, lse, *(x.contiguous() for x in back)))
        del cache, back
    for a, b in zip(*results):
        assert torch.equal(a, b)

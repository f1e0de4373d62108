"""The cache operators together, as a serving loop uses them: block map, prompt attention, both caches' appends, verify and draft
attention over the 8-bit cache, Top-K and the next draft step's lists, with no host read between the calls of a step.

Each step's maps and cache are held to the plain definitions exactly, its attention to the bounds of test_attn_kv8.py; the bf16
cache, filled through the same maps, goes through pillar_attn_unified and is held to its stated relative error.
"""
import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from oracle import cache as C
from tests import test_attn_kv8 as A8
from tests import test_prompt_attn as PA
from workloads import bf16_bits_to_f32, f32_to_bf16_bits

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")

Hq, Hkv, D, K = 8, 2, 64, 3
BLOCKS, WIDTH, MAX_LEN, MAX_SPARSE = 40, 20, 320, 96


def dev(x, t):
    return torch.tensor(np.ascontiguousarray(x), dtype=t, device="cuda")


def rows(g, n, heads):
    return f32_to_bf16_bits(g.standard_normal((n, heads, D)).astype(np.float32))


def bits(x):
    return dev(x.view(np.int16), torch.int16)


def f64(x):
    return bf16_bits_to_f32(x).astype(np.float64)


class Loop:
    """The device's state and, beside it, what the definitions say it has to be."""

    def __init__(self, B, seed):
        self.B, self.g = B, np.random.default_rng(seed)
        i32 = lambda x: dev(x, torch.int32)  # noqa: E731
        ring = self.g.permutation(BLOCKS)
        self.shape = P.make_shape(B=B, Hq=Hq, Hkv=Hkv, D=D, k=K, max_sparse=MAX_SPARSE, max_len=MAX_LEN, num_slots=BLOCKS * 16,
                                  max_topk=MAX_SPARSE - K - 1)
        self.table, self.ring, self.state = i32(np.full((B, WIDTH), -1)), i32(ring), i32([0, BLOCKS])
        self.lens = i32(np.zeros(B))
        self.k8, self.v8 = (torch.zeros((BLOCKS, Hkv, 16, D), dtype=torch.uint8, device="cuda") for _ in "kv")
        self.ks, self.vs = (torch.zeros((BLOCKS, Hkv), device="cuda") for _ in "kv")
        self.kb, self.vb = (torch.zeros((BLOCKS * 16, Hkv, D), dtype=torch.int16, device="cuda") for _ in "kv")
        self.kv_off, self.new_off = torch.zeros(B + 1, dtype=torch.int64, device="cuda"), i32(np.zeros(B + 1))
        self.slots = i32(np.full(B * MAX_LEN, -7))
        self.map_ws = torch.empty(P.pillar_block_map_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda")
        self.ws = torch.empty(P.pillar_attn_workspace_bytes(self.shape), dtype=torch.uint8, device="cuda")
        self.flags = i32([0])
        self.idx, self.cnt = i32(np.zeros((B, Hkv, MAX_SPARSE))), i32(np.zeros((B, Hkv)))
        # the definitions' side
        self.want = dict(table=np.full((B, WIDTH), -1), ring=ring, state=[0, BLOCKS], lens=np.zeros(B, int),
                         k8=np.zeros((BLOCKS, Hkv, 16, D), np.uint8), v8=np.zeros((BLOCKS, Hkv, 16, D), np.uint8),
                         ks=np.zeros((BLOCKS, Hkv)), vs=np.zeros((BLOCKS, Hkv)))
        self.ctx_k, self.ctx_v = [np.zeros((0, Hkv, D))] * B, [np.zeros((0, Hkv, D))] * B  # the rows as bf16 values

    def new_rows(self, lens):
        return max(1, int(np.maximum(np.array(lens) - self.want["lens"], 0).sum()))

    def grow(self, lens, k=None, v=None):
        """One block map to these lengths and, with rows, both appends."""
        n = 1 if k is None else len(k)
        new_slots, granted = dev(np.full(n, -7), torch.int32), torch.zeros_like(self.lens)
        P.pillar_block_map(self.shape, dev(lens, torch.int32), self.lens, self.table, self.ring, self.state, granted, self.kv_off,
                           self.slots, self.new_off, new_slots, self.map_ws)
        self.lens = granted
        if k is not None:
            kd, vd = bits(k), bits(v)
            P.pillar_kv8_append(self.shape, kd, vd, granted, self.new_off, self.table, self.k8, self.v8, self.ks, self.vs, self.flags)
            P.pillar_kv_append(self.shape, kd, vd, new_slots, self.kb, self.vb, self.flags)

    def mirror(self, lens, k=None, v=None):
        """The same by the definitions, and the device's maps and caches against them."""
        w = self.want
        m = C.block_map(lens, w["lens"], w["table"], w["ring"], w["state"], MAX_LEN, BLOCKS)
        assert not m["bad"]
        for b in range(self.B):
            a, e = m["new_off"][b], m["new_off"][b + 1]
            for ctx, x in ((self.ctx_k, k), (self.ctx_v, v)):
                ctx[b] = ctx[b][:m["granted"][b]]
                if x is not None:
                    ctx[b] = np.concatenate([ctx[b], f64(x[a:e])])
        if k is not None:
            w["k8"], w["ks"] = C.kv8_append(w["k8"], w["ks"], f64(k), m["granted"], m["new_off"], m["table"])
            w["v8"], w["vs"] = C.kv8_append(w["v8"], w["vs"], f64(v), m["granted"], m["new_off"], m["table"])
        w.update(table=m["table"], ring=m["ring"], state=m["state"], lens=m["granted"])
        assert P.pillar_get_error(self.map_ws) == 0 and int(self.flags) == 0
        for name in ("table", "ring", "state", "lens", "k8", "v8", "ks", "vs"):
            np.testing.assert_array_equal(getattr(self, name).cpu().numpy(), w[name], err_msg=name)
        np.testing.assert_array_equal(self.slots.cpu().numpy()[:len(m["slots"])], m["slots"])
        np.testing.assert_array_equal(self.new_off.cpu().numpy(), m["new_off"])

    def outputs(self, modes):
        """Buffers of one attention step whose lengths are the present ones."""
        modes = np.array(modes)
        T, V = int(np.where(modes == 1, K + 1, 1).sum()), int((modes == 1).sum())
        n = int(Hq * (K + 1) * self.want["lens"][modes == 1].sum())
        return dict(q=bits(rows(self.g, T, Hq)), mode=dev(modes, torch.int32), out=torch.zeros((T, Hq, D), dtype=torch.int16, device="cuda"),
                    logits=torch.full((n + 6,), A8.SENTINEL, device="cuda"), lse=torch.zeros((max(1, V), Hq, K + 1), device="cuda"), ws=self.ws)

    def attend(self, d):
        P.pillar_attn_kv8(self.shape, d["q"], self.k8, self.v8, self.ks, self.vs, self.table, d["mode"], self.lens, self.idx, self.cnt,
                          d["out"], d["logits"], d["lse"], self.ws)

    def check_attention(self, d, modes):
        w, c = self.want, object.__new__(A8.Case)
        c.Hq, c.Hkv, c.D, c.k, c.scale, c.modes, c.lens = Hq, Hkv, D, K, D ** -0.5, np.array(modes), w["lens"]
        c.V, c.q = int((c.modes == 1).sum()), d["q"].cpu().numpy().view(np.uint16)
        c.table, c.k8, c.v8 = w["table"], w["k8"], w["v8"]
        c.ks, c.vs = w["ks"].astype(np.float32), w["vs"].astype(np.float32)
        c.idx, c.cnt = self.idx.cpu().numpy(), self.cnt.cpu().numpy()
        c.check(d)

    def check_bf16(self, d, modes):
        """The bf16 cache through the same maps: pillar_attn_unified on the slot table."""
        out, ws = torch.zeros_like(d["out"]), torch.empty_like(self.ws)
        logits, lse = torch.empty(max(1, len(d["logits"])), device="cuda"), torch.empty_like(d["lse"])
        P.pillar_attn_unified(self.shape, d["q"], self.kb, self.vb, self.slots, d["mode"], self.lens, self.idx, self.cnt, out, logits,
                              lse, ws)
        assert P.pillar_get_error(ws) == 0
        got, q = f64(out.cpu().numpy().view(np.uint16)), f64(d["q"].cpu().numpy().view(np.uint16))
        idx, cnt, r = self.idx.cpu().numpy(), self.cnt.cpu().numpy(), 0
        for b, mode in enumerate(modes):
            nq, L = (K + 1 if mode == 1 else 1), int(self.want["lens"][b])
            want = np.zeros((nq, Hq, D))
            for j in range(nq):
                for h in range(Hq):
                    g = h * Hkv // Hq
                    seen = np.arange(L - nq + j + 1) if mode == 1 else idx[b, g, :cnt[b, g]]
                    want[j, h] = C._attend(q[r + j, h], self.ctx_k[b][seen, g], self.ctx_v[b][seen, g], D ** -0.5)[0]
            assert np.linalg.norm(got[r:r + nq] - want) <= 1e-2 * np.linalg.norm(want) + 1e-30
            r += nq

    def select(self, d, V):
        """The Top-K of a step in which every request verified (a third of the context)."""
        s, lens = self.shape, self.want["lens"]
        self.next_idx, self.next_cnt = torch.zeros((V, Hkv, s.max_topk), dtype=torch.int32, device="cuda"), torch.zeros((V, Hkv), dtype=torch.int32, device="cuda")
        self.group, self.verify_len = torch.arange(V, dtype=torch.int32, device="cuda"), self.lens.clone()
        self.topk_ws = torch.empty(P.pillar_topk_workspace_bytes(s, V), dtype=torch.uint8, device="cuda")
        P.pillar_topk_select(s, V, d["logits"], d["lse"], self.lens, self.group, dev(np.maximum(1, lens // 3), torch.int32), self.next_idx,
                             self.next_cnt, self.topk_ws)

    def check_select(self, d, V):
        assert P.pillar_get_error(self.topk_ws) == 0
        idx, cnt, lens = self.next_idx.cpu().numpy(), self.next_cnt.cpu().numpy(), self.want["lens"]
        logits, lse, at = d["logits"].cpu().numpy().astype(np.float64), d["lse"].cpu().numpy().astype(np.float64), 0
        for v in range(V):
            L, n = int(lens[v]), max(1, int(lens[v]) // 3)
            p = np.exp(logits[at:at + Hq * (K + 1) * L].reshape(Hq, K + 1, L) - lse[v][:, :, None])[:, 1:]
            at += Hq * (K + 1) * L
            for h in range(Hkv):
                score = p[h * Hq // Hkv:(h + 1) * Hq // Hkv].mean((0, 1))
                chosen = idx[v, h, :n]
                assert cnt[v, h] == n and np.all(np.diff(chosen) > 0) and 0 <= chosen[0] and chosen[-1] < L
                rest = np.delete(score, chosen)  # none of the others is larger, but for fp32 (exp 2^-21, sums and difference 2^-19)
                assert len(rest) == 0 or score[chosen].min() >= rest.max() * (1 - 2.0 ** -18)

    def lists(self):
        P.pillar_draft_lists(self.shape, self.B, self.next_idx, self.next_cnt, self.group, self.verify_len, self.lens, self.slots, self.idx,
                             self.cnt, None, self.flags)


def prompts(loop, k, v, lo, hi):
    """Causal attention of the requests lo .. hi - 1, whose rows new_off places among k and v."""
    q, n = rows(loop.g, len(k), Hq), len(k)
    shape = PA.shape_of(hi - lo, Hq, Hkv, D, MAX_LEN)
    d = dict(q=bits(q), out=torch.full((n, Hq, D), 0x7fc1, dtype=torch.int16, device="cuda"),
             lse=torch.full((n, Hq), PA.SENTINEL, device="cuda"),
             ws=torch.empty(P.pillar_prompt_attn_workspace_bytes(shape, n), dtype=torch.uint8, device="cuda"))
    P.pillar_prompt_attn(shape, d["q"], bits(k), bits(v), loop.new_off[lo:hi + 1], d["out"], d["lse"], d["ws"])
    c = object.__new__(PA.Case)
    c.Hq, c.Hkv, c.D, c.n, c.scale, c.q, c.k, c.v = Hq, Hkv, D, n, D ** -0.5, q, k, v
    c.check(d, off=loop.new_off[lo:hi + 1].cpu().numpy())


def test_a_serving_loop():
    lens = np.array([37, 100, 16, 5])
    B = len(lens)
    loop = Loop(B, 1)

    def step(lens, with_rows=True):
        n = loop.new_rows(lens)
        kv = (rows(loop.g, n, Hkv), rows(loop.g, n, Hkv)) if with_rows else (None, None)
        loop.grow(lens, *kv)
        loop.mirror(lens, *kv)
        return kv

    kv = step(lens)  # the prompts
    prompts(loop, *kv, 0, B)
    lens = lens + K + 1  # every request verifies its first k + 1 tokens
    step(lens)
    modes = [1] * B
    d = loop.outputs(modes)
    loop.attend(d)
    loop.select(d, B)
    loop.check_attention(d, modes)
    loop.check_bf16(d, modes)
    loop.check_select(d, B)
    for _ in range(2):  # two draft steps on the lists of that verify step
        lens = lens + 1
        step(lens)
        loop.lists()
        d, modes = loop.outputs([0] * B), [0] * B
        loop.attend(d)
        assert int(loop.flags) == 0
        assert np.array_equal(loop.cnt.cpu().numpy(), loop.next_cnt.cpu().numpy() + (loop.lens - loop.verify_len).cpu().numpy()[:, None])
        loop.check_attention(d, modes)
        loop.check_bf16(d, modes)
    # two tokens of request 0 and twenty of request 1 are taken back, request 2 is finished; its blocks serve a new prompt
    lens = np.array([lens[0] - 2, lens[1] - 20, 0, lens[3]])
    step(lens, with_rows=False)
    lens = np.array([lens[0] + K + 1, lens[1] + 1, 200, lens[3] + K + 1])
    kv = step(lens)
    prompts(loop, *kv, 2, 3)
    modes = [1, 0, 1, 1]
    loop.idx[1] = dev(loop.g.integers(0, lens[1], (Hkv, MAX_SPARSE)), torch.int32)
    loop.cnt[1] = dev([MAX_SPARSE, 17], torch.int32)
    d = loop.outputs(modes)
    loop.attend(d)
    loop.check_attention(d, modes)
    loop.check_bf16(d, modes)


def test_a_step_captured_whole_and_replayed():
    """Map, append, attention, Top-K and lists as one graph, on lengths and rows that change between replays."""
    start = np.array([33, 70, 48])
    eager, graph = Loop(3, 2), Loop(3, 2)
    first = (rows(eager.g, int(start.sum()), Hkv), rows(eager.g, int(start.sum()), Hkv))
    kd, vd, q = ([rows(eager.g, 3 * (K + 1), h) for _ in range(2)] for h in (Hkv, Hkv, Hq))
    made = []

    def enqueue(lp, req_len, k, v, q, st):
        """From lp.lens to req_len, all on the device."""
        P.pillar_block_map(lp.shape, req_len, lp.lens, lp.table, lp.ring, lp.state, st["granted"], lp.kv_off, lp.slots, lp.new_off,
                           st["new_slots"], lp.map_ws)
        lp.lens.copy_(st["granted"])
        P.pillar_kv8_append(lp.shape, k, v, lp.lens, lp.new_off, lp.table, lp.k8, lp.v8, lp.ks, lp.vs, lp.flags)
        P.pillar_attn_kv8(lp.shape, q, lp.k8, lp.v8, lp.ks, lp.vs, lp.table, st["mode"], lp.lens, lp.idx, lp.cnt, st["out"], st["logits"],
                          st["lse"], lp.ws)
        P.pillar_topk_select(lp.shape, 3, st["logits"], st["lse"], lp.lens, st["group"], st["K"], st["next_idx"], st["next_cnt"], st["tws"])
        P.pillar_draft_lists(lp.shape, 3, st["next_idx"], st["next_cnt"], st["group"], lp.lens, lp.lens, lp.slots, lp.idx, lp.cnt, None,
                             lp.flags)

    def buffers(lp):
        z = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
        return dict(granted=z(3), new_slots=z(3 * (K + 1)), mode=z(3) + 1, group=torch.arange(3, dtype=torch.int32, device="cuda"), K=z(3) + 20,
                    next_idx=z(3, Hkv, lp.shape.max_topk), next_cnt=z(3, Hkv), out=torch.zeros((3 * (K + 1), Hq, D), dtype=torch.int16, device="cuda"),
                    logits=torch.zeros(Hq * (K + 1) * 3 * MAX_LEN, device="cuda"), lse=torch.zeros((3, Hq, K + 1), device="cuda"),
                    tws=torch.empty(P.pillar_topk_workspace_bytes(lp.shape, 3), dtype=torch.uint8, device="cuda"))

    for lp in (eager, graph):
        lp.grow(start, *first)
        made.append(buffers(lp))
    req, k, v, qd = dev(start, torch.int32), bits(kd[0]), bits(vd[0]), bits(q[0])
    saved = {n: getattr(graph, n).clone() for n in ("lens", "table", "ring", "state", "k8", "v8", "ks", "vs")}
    torch.cuda.synchronize()
    h = torch.cuda.CUDAGraph()
    with torch.cuda.graph(h):
        enqueue(graph, req, k, v, qd, made[1])
    for n, x in saved.items():  # (a capture runs nothing, but the state it starts from is made sure of)
        getattr(graph, n).copy_(x)
    for i in range(2):
        lens = start + (K + 1) * (i + 1)
        req.copy_(dev(lens, torch.int32))
        for dst, src in ((k, kd[i]), (v, vd[i]), (qd, q[i])):
            dst.copy_(bits(src))
        enqueue(eager, dev(lens, torch.int32), bits(kd[i]), bits(vd[i]), bits(q[i]), made[0])
        h.replay()
        torch.cuda.synchronize()
        for n in ("lens", "table", "ring", "state", "k8", "v8", "ks", "vs", "slots", "idx", "cnt", "kv_off", "new_off"):
            assert torch.equal(getattr(eager, n), getattr(graph, n)), n
        for n in ("out", "logits", "lse", "next_idx", "next_cnt"):
            assert torch.equal(made[0][n], made[1][n]), n
        for lp in (eager, graph):
            assert P.pillar_get_error(lp.map_ws) == 0 and P.pillar_get_error(lp.ws) == 0 and int(lp.flags) == 0


def test_pools_and_strides_past_32_bits():
    """The same blocks at the start of a small pool and at the end of one of 5 GB; the same prompt rows packed and 8 MB apart."""
    heads, dim, lens, far = 8, 128, [300, 130, 77], 300000
    g = np.random.default_rng(5)
    n, nb = sum(lens), [-(-x // 16) for x in lens]
    near = sum(nb)
    rowset = lambda h: torch.from_numpy(f32_to_bf16_bits(g.standard_normal((n, h, dim)).astype(np.float32)).view(np.int16)).cuda()  # noqa: E731
    k, v, q = rowset(heads), rowset(heads), rowset(16)
    off, length = dev(np.concatenate([[0], np.cumsum(lens)]), torch.int32), dev(lens, torch.int32)
    mode, lists = dev([1, 0, 1], torch.int32), dev(g.integers(0, 130, (3, heads, 40)), torch.int32)
    q8 = q[:2 * 4 + 1].contiguous()
    results = []
    for blocks in (near, far):
        table = np.full((3, max(nb)), -1)
        at = blocks - near
        for b in range(3):
            table[b, :nb[b]] = np.arange(at, at + nb[b])
            at += nb[b]
        s = P.make_shape(B=3, Hq=16, Hkv=heads, D=dim, k=3, max_sparse=40, max_len=300, num_slots=blocks * 16)
        k8, v8 = (torch.empty((blocks, heads, 16, dim), dtype=torch.uint8, device="cuda") for _ in "kv")
        ks, vs = (torch.empty((blocks, heads), device="cuda") for _ in "kv")
        t, flags = dev(table, torch.int32), dev([0], torch.int32)
        P.pillar_kv8_append(s, k, v, length, off, t, k8, v8, ks, vs, flags)
        out, lse = torch.zeros_like(q8), torch.zeros((2, 16, 4), device="cuda")
        logits = torch.zeros(16 * 4 * (lens[0] + lens[2]), device="cuda")
        ws = torch.empty(P.pillar_attn_workspace_bytes(s), dtype=torch.uint8, device="cuda")
        P.pillar_attn_kv8(s, q8, k8, v8, ks, vs, t, mode, length, lists, dev(np.full((3, heads), 40), torch.int32), out, logits, lse, ws)
        assert int(flags) == 0 and P.pillar_get_error(ws) == 0
        results.append((ks[blocks - near:].clone(), out, logits, lse))
        del k8, v8, ks, vs
    for a, b in zip(*results):
        assert torch.equal(a, b)
    s, stride = PA.shape_of(3, 16, heads, dim, 300), 1 << 22
    ws = torch.empty(P.pillar_prompt_attn_workspace_bytes(s, n), dtype=torch.uint8, device="cuda")
    outs = []
    for apart in (False, True):
        rows3 = []
        for x in (q, k, v):
            if apart:
                wide = torch.empty((n - 1) * stride + x.shape[1] * dim, dtype=torch.int16, device="cuda")
                y = wide.as_strided(x.shape, (stride, dim, 1))
                y.copy_(x)
                x = y
            rows3.append(x)
        out, lse = torch.zeros((n, 16, dim), dtype=torch.int16, device="cuda"), torch.zeros((n, 16), device="cuda")
        P.pillar_prompt_attn(s, *rows3, off, out, lse, ws)
        assert P.pillar_get_error(ws) == 0
        outs.append((out, lse))
        del rows3
    assert torch.equal(outs[0][0], outs[1][0]) and torch.equal(outs[0][1], outs[1][1])

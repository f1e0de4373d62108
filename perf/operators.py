"""Timed cases of the serving operators around the PillarAttn step, with their plain forms.

Four operators, used in this order when a model is served:

  block_map    block tables, the page-size-1 slot table and the new tokens' slots from request lengths
  prompt       causal attention over whole prompts, packed, grouped heads
  append       new K/V rows into the 8-bit cache: e4m3 codes, a power-of-two scale per block of 16 tokens and KV head
  attn8        the draft/verify attention step over the 8-bit cache

``run`` computes the plain form (elementary torch operations in fp32) where ``own`` is false and makes the
framework's calls where it is true.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False
BLOCK = 16          # tokens of a cache block
E4M3_MAX = 448.0


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # one speculative step of a small batch: room for the new tokens, then the rollback of the rejected ones
        dict(name="map_small", op="block_map", B=4, k=4, lo=256, hi=512),
        # a server with many requests and long contexts: 2048 requests, 17 million slots
        dict(name="map_large", op="block_map", B=2048, k=8, lo=1024, hi=16384),
        # one short prompt (Qwen3-1.7B-shaped heads): latency
        dict(name="prompt_short", op="prompt", B=1, lo=37, hi=37, Hq=16, Hkv=8, D=128),
        # a prefill batch of ragged prompts (Qwen3-8B-shaped heads)
        dict(name="prompt_ragged", op="prompt", B=24, lo=1, hi=2047, Hq=32, Hkv=8, D=128),
        # one long document (Qwen3-8B-shaped heads)
        dict(name="prompt_long", op="prompt", B=1, lo=16384, hi=16384, Hq=32, Hkv=8, D=128),
        # head dimension 64, four query heads on one KV head
        dict(name="prompt_d64", op="prompt", B=12, lo=300, hi=4100, Hq=4, Hkv=1, D=64),
        # the new tokens of a decode step: one per draft request, k+1 per verify request
        dict(name="append_step", op="append", B=128, k=8, prompt=0, lo=64, hi=1024, Hkv=8, D=128),
        # the K/V of a prefill batch
        dict(name="append_prompt", op="append", B=32, k=0, prompt=1, lo=100, hi=4000, Hkv=8, D=128),
        # the smallest step: two draft and two verify requests, head dimension 64
        dict(name="attn8_tiny", op="attn8", B=4, Hq=4, Hkv=1, D=64, k=4, mix="mixed", lo=256, hi=512, s=0.1, dump=1),
        # single tokens over their whole contexts, no dump: plain decoding
        dict(name="attn8_decode", op="attn8", B=64, Hq=32, Hkv=8, D=128, k=0, mix="full", lo=1000, hi=30000, s=0.05,
             dump=0),
        # the Qwen3-8B-shaped speculative step: 128 requests, one ninth verify
        dict(name="attn8_8b", op="attn8", B=128, Hq=32, Hkv=8, D=128, k=8, mix="mixed", lo=6144, hi=10240, s=0.05, dump=1),
        # the Qwen3-14B-shaped step: five query heads per KV head, contexts 4K to 24K
        dict(name="attn8_14b", op="attn8", B=128, Hq=40, Hkv=8, D=128, k=8, mix="mixed", lo=4096, hi=24576, s=0.05,
             dump=1),
    ]


def _span(rng, lo, hi):
    """An integer spread over [lo, hi] on a logarithmic scale."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("block_map", "prompt", "append", "attn8"))
    if op == "block_map":
        B = _span(rng, 1, 2048)
        hi = _span(rng, 64, 16384)
        return dict(op=op, B=B, k=rng.randint(0, 15), lo=_span(rng, 16, hi), hi=hi)
    D = rng.choice((64, 128))
    if op == "prompt":
        Hkv = rng.choice((1, 2, 8))
        G = rng.choice((1, 2, 4, 5, 8))
        # at most the long document's work: B * hi^2 * Hq * D bounded
        hi = _span(rng, 1, 16384)
        most = 16384 * 16384 * 32 * 128
        B = max(1, min(_span(rng, 1, 64), most // (hi * hi * G * Hkv * D), 262144 // hi))
        while hi * hi * G * Hkv * D > most:
            G = max(1, G // 2)
        return dict(op=op, B=B, lo=_span(rng, 1, hi), hi=hi, Hq=G * Hkv, Hkv=Hkv, D=D)
    if op == "append":
        Hkv = rng.choice((1, 2, 5, 8))
        prompt = rng.randint(0, 1)
        B = _span(rng, 1, 32 if prompt else 256)
        hi = _span(rng, 20, 4000 if prompt else 1024)
        return dict(op=op, B=B, k=rng.randint(0, 12), prompt=prompt, lo=_span(rng, 17, hi), hi=hi, Hkv=Hkv, D=D)
    G = rng.choice((1, 2, 4, 5, 8))
    Hkv = rng.choice((1, 2, 8))
    mix = rng.choice(("mixed", "mixed", "full", "draft"))
    k = rng.randint(1 if mix == "draft" else 0, min(12, 64 // G - 1))
    hi = _span(rng, 100, 24576)
    # at most the 14B-shaped step's keys and logits
    B = max(1, min(_span(rng, 1, 128), (128 * 9000) // hi))
    if mix == "full":
        B = max(1, min(B, 15 * 40 * 9 * 14000 // (hi * G * Hkv * (k + 1))))
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, k=k, mix=mix, lo=_span(rng, 32, hi), hi=hi,
                s=rng.choice((0.03, 0.05, 0.1)), dump=rng.randint(0, 1))


# ------------------------------------------------------------------------------------------------ inputs

def _lengths(case, seed):
    """The case's lengths (the same for every seed: a case is one amount of work)."""
    g = np.random.default_rng((case["B"], case["lo"], case["hi"]))
    return np.rint(np.exp(g.uniform(math.log(case["lo"]), math.log(case["hi"] + 0.49), case["B"]))).astype(np.int64)


def _mode(case):
    i = np.arange(case["B"])
    if case["mix"] == "full":
        return np.ones(case["B"], np.int64)
    if case["mix"] == "draft":
        return np.zeros(case["B"], np.int64)
    return (i % (case["k"] + 1) == 0).astype(np.int64)


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _tables(g, L, spare):
    """Block tables [B, max_blocks] over a shuffled pool and the blocks left free, in the order they are handed out."""
    nb = -(-L // BLOCK)
    total = int(nb.sum()) + spare
    perm = g.permutation(total)
    max_blocks = int(max(1, nb.max())) + 1
    t = np.zeros((len(L), max_blocks), np.int64)
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, perm[at:], total


def _quantise(x):
    """[..., BLOCK, D] fp32 -> e4m3 codes and a power-of-two scale per leading index."""
    scale = _pow2_scale(x.abs().amax(dim=(-1, -2)))
    return (x / scale[..., None, None]).to(torch.float8_e4m3fn), scale


def _pow2_scale(amax):
    """The smallest 2^e with amax <= 448 * 2^e, e >= -126."""
    m, x = torch.frexp(amax)
    e = torch.where(m <= 0.875, x - 9, x - 8)
    e = torch.where(amax > 0, e, torch.full_like(e, -126)).clamp(min=-126)
    return torch.ldexp(torch.ones_like(amax), e)


def prepare(case, seed):
    op = case["op"]
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    g = np.random.default_rng((int(seed), 99))
    s = dict(op=op, case=dict(case))
    if op == "block_map":
        _prepare_map(case, g, s)
    elif op == "prompt":
        L = _lengths(case, seed)
        T = int(L.sum())
        Hq, Hkv, D = case["Hq"], case["Hkv"], case["D"]
        off = _offsets(L)
        s["q"] = torch.randn((T, Hq, D), generator=gen, device="cuda").bfloat16()
        s["k"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").bfloat16()
        s["v"] = torch.randn((T, Hkv, D), generator=gen, device="cuda").bfloat16()
        s["seq_off"] = _dev(off, torch.int32)
        s["max_len"] = int(L.max())
        s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
        s["lse"] = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
        s["shape_of"] = dict(B=case["B"], Hq=Hq, Hkv=Hkv, D=D, k=0, row_lo=0, max_sparse=0, max_len=s["max_len"],
                             num_slots=1)
    elif op == "append":
        _prepare_append(case, g, gen, seed, s)
    else:
        _prepare_attn8(case, g, gen, seed, s)
    return s


def _prepare_map(case, g, s):
    """A running batch before a step, and the free blocks of its pool."""
    P0 = _lengths(case, 0)
    mode = np.arange(case["B"]) % (case["k"] + 1) == 0
    n = np.where(mode, case["k"] + 1, 1)
    L = P0 + n
    table, free, total = _tables(g, P0, spare=case["B"] + 64)
    ring = np.zeros(total, np.int64)
    head = int(g.integers(0, total))
    ring[(head + np.arange(len(free))) % total] = free
    hi = int(L.max())
    s["prev"], s["len"] = _dev(P0, torch.int32), _dev(L, torch.int32)
    width = -(-hi // BLOCK)
    t = np.zeros((case["B"], width), np.int64)
    t[:, :min(width, table.shape[1])] = table[:, :width]
    s["table"] = _dev(t, torch.int32)
    s["ring"], s["state"] = _dev(ring, torch.int32), _dev(np.array([head, len(free)]), torch.int32)
    i32, B = dict(dtype=torch.int32, device="cuda"), case["B"]
    # the step's outputs, and the rollback's
    for j, tot in ((0, int(L.sum())), (1, int(P0.sum()))):
        s["granted%d" % j] = torch.zeros(B, **i32)
        s["kv_off%d" % j] = torch.zeros(B + 1, dtype=torch.int64, device="cuda")
        s["slots%d" % j] = torch.zeros(tot, **i32)
        s["new_off%d" % j] = torch.zeros(B + 1, **i32)
        s["new_slots%d" % j] = torch.zeros(int(n.sum()), **i32)
    s["shape_of"] = dict(B=B, Hq=1, Hkv=1, D=64, k=0, row_lo=0, max_sparse=0, max_len=hi, num_slots=total * BLOCK)


def _prepare_append(case, g, gen, seed, s):
    """New K/V rows and a cache that holds what came before them."""
    B, Hkv, D = case["B"], case["Hkv"], case["D"]
    P0 = _lengths(case, seed)
    if case["prompt"]:
        n, P0 = P0, np.zeros_like(P0)
    else:
        n = np.where(np.arange(B) % (case["k"] + 1) == 0, case["k"] + 1, 1)
    L = P0 + n
    table, _, total = _tables(g, L, spare=8)
    N = int(n.sum())
    cache = torch.randn((total, Hkv, BLOCK, D), generator=gen, device="cuda")
    s["k8"], s["k_scale"] = _quantise(cache)
    s["v8"], s["v_scale"] = _quantise(cache.roll(1, 0))
    # one token in sixteen has large keys: the scale of its block grows and the older rows are rounded again
    x = torch.randn((N, Hkv, D), generator=gen, device="cuda")
    big = torch.rand((N, 1, 1), generator=gen, device="cuda") < 1 / 16
    s["k_new"] = torch.where(big, x * 6, x).bfloat16()
    s["v_new"] = torch.randn((N, Hkv, D), generator=gen, device="cuda").bfloat16()
    s["len"], s["new_off"] = _dev(L, torch.int32), _dev(_offsets(n), torch.int32)
    s["table"] = _dev(table, torch.int32)
    s["shape_of"] = dict(B=B, Hq=Hkv, Hkv=Hkv, D=D, k=0, row_lo=0, max_sparse=0, max_len=int(L.max()),
                         num_slots=total * BLOCK)


def _prepare_attn8(case, g, gen, seed, s):
    """A batch of draft and verify requests over a filled 8-bit cache."""
    B, Hq, Hkv, D, k = (case[x] for x in ("B", "Hq", "Hkv", "D", "k"))
    mode = _mode(case)
    L = np.maximum(_lengths(case, seed), k + 1)
    table, _, total = _tables(g, L, spare=8)
    # keys and queries with the pillar structure: one position in twenty carries the head's direction
    u = torch.randn((Hkv, D), generator=gen, device="cuda")
    u = u / u.norm(dim=-1, keepdim=True)
    k8 = torch.empty((total, Hkv, BLOCK, D), dtype=torch.float8_e4m3fn, device="cuda")
    v8 = torch.empty_like(k8)
    ks = torch.empty((total, Hkv), dtype=torch.float32, device="cuda")
    vs = torch.empty_like(ks)
    for at in range(0, total, 8192):
        n = min(8192, total - at)
        x = torch.randn((n, Hkv, BLOCK, D), generator=gen, device="cuda")
        x += 2 * u[None, :, None, :] * (torch.rand((n, Hkv, BLOCK, 1), generator=gen, device="cuda") < 0.05)
        k8[at:at + n], ks[at:at + n] = _quantise(x)
        v8[at:at + n], vs[at:at + n] = _quantise(torch.randn((n, Hkv, BLOCK, D), generator=gen, device="cuda"))
    rows = np.where(mode == 1, k + 1, 1)
    q_off = _offsets(rows)
    T = int(rows.sum())
    q = torch.randn((T, Hq, D), generator=gen, device="cuda") + 3 * u.repeat_interleave(Hq // Hkv, 0)
    s.update(k8=k8, v8=v8, k_scale=ks, v_scale=vs, q=q.bfloat16())
    s["len"], s["mode"], s["table"] = _dev(L, torch.int32), _dev(mode, torch.int32), _dev(table, torch.int32)
    # critical lists of the draft requests: ascending positions, ceil(s L) per KV head
    cnt = np.where(mode == 0, np.minimum(L, np.ceil(case["s"] * L)), 0).astype(np.int64)
    ms = int(max(1, cnt.max()))
    Lmax = int(L.max())
    idx = torch.zeros((B, Hkv, ms), dtype=torch.int32, device="cuda")
    Ld, cd = _dev(L, torch.int64), _dev(cnt, torch.int64)
    for at in range(0, B, 16):
        n = min(16, B - at)
        w = torch.rand((n, Hkv, Lmax), generator=gen, device="cuda")
        w = torch.where(torch.arange(Lmax, device="cuda") < Ld[at:at + n, None, None], w, -1.0)
        top = w.topk(ms, dim=-1).indices  # by weight: the first cnt are a random subset of the context
        top = torch.where(torch.arange(ms, device="cuda") < cd[at:at + n, None, None], top, Lmax)
        idx[at:at + n] = torch.where(top < Lmax, top, Lmax).sort(dim=-1).values.to(torch.int32)
    s["idx"] = torch.where(idx < Lmax, idx, 0)
    s["cnt"] = _dev(np.repeat(cnt[:, None], Hkv, 1), torch.int32)
    # where the plain form finds its rows: draft requests, verify requests, and the packed logits of the latter
    dr, ve = np.nonzero(mode == 0)[0], np.nonzero(mode == 1)[0]
    s["draft"], s["verify"] = _dev(dr, torch.int64), _dev(ve, torch.int64)
    s["draft_row"] = _dev(q_off[dr], torch.int64)
    s["verify_row"] = _dev(q_off[ve][:, None] + np.arange(k + 1)[None, :], torch.int64)
    V, Lv = len(ve), L[ve]
    n_log = int(Hq * (k + 1) * Lv.sum())
    s["V"], s["Lmax"] = V, int(Lv.max()) if V else 1
    s["logits"] = torch.zeros(max(2, n_log) if case["dump"] else 2, dtype=torch.float32, device="cuda")
    s["n_log"] = n_log if case["dump"] else 0
    s["lse"] = torch.zeros((max(1, V), Hq, k + 1), dtype=torch.float32, device="cuda")
    s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    s["shape_of"] = dict(B=B, Hq=Hq, Hkv=Hkv, D=D, k=k, row_lo=min(1, k), max_sparse=ms, max_len=Lmax,
                         num_slots=total * BLOCK)


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return {"block_map": _run_map, "prompt": _run_prompt, "append": _run_append, "attn8": _run_attn8}[s["op"]](s)


def _handle(s, workspace_bytes=None):
    """The binding, the shape record and the workspace that a program makes once and keeps."""
    import sparse_self_speculative_pillar_gb300 as P
    if "shape" not in s:
        s["shape"] = P.make_shape(**s["shape_of"])
        if workspace_bytes:
            s["ws"] = torch.empty(workspace_bytes(P, s["shape"]), dtype=torch.uint8, device="cuda")
    return P


def _run_map(s):
    """A step's blocks and slots, then the rollback to the lengths before it (every drafted token rejected)."""
    for j, (new, old) in enumerate((("len", "prev"), ("prev", "len"))):
        if own:
            P = _handle(s, lambda P, shape: P.pillar_block_map_workspace_bytes(shape))
            P.pillar_block_map(s["shape"], s[new], s[old], s["table"], s["ring"], s["state"], s["granted%d" % j],
                               s["kv_off%d" % j], s["slots%d" % j], s["new_off%d" % j], s["new_slots%d" % j], s["ws"])
        else:
            _plain_map(s[new].long(), s[old].long(), s["table"], s["ring"], s["state"], s["granted%d" % j],
                       s["kv_off%d" % j], s["slots%d" % j], s["new_off%d" % j], s["new_slots%d" % j])
    return {x: s[x] for x in ("table", "ring", "state", "granted0", "kv_off0", "slots0", "new_off0", "new_slots0",
                              "granted1", "kv_off1", "slots1", "new_off1")}


def _plain_map(L, P0, table, ring, state, granted, kv_off, slots, new_off, new_slots):
    dev, Q, (B, W) = L.device, ring.numel(), table.shape
    head, count = state[0].long(), state[1].long()
    nb, mb = (L + BLOCK - 1) // BLOCK, (P0 + BLOCK - 1) // BLOCK
    want = (nb - mb).clamp(min=0)
    have = want.cumsum(0)
    ok = (want == 0) | (have <= count)
    Lg = torch.where(ok, L, P0)
    ng = torch.where(ok, nb, mb)
    give = (mb - nb).clamp(min=0)
    first_in, first_out = have - want, give.cumsum(0) - give
    j = torch.arange(W, device=dev)[None, :]
    taken = ring[(head + first_in[:, None] + j - mb[:, None]) % Q]
    back = torch.where((j >= nb[:, None]) & (j < mb[:, None]), (head + count + first_out[:, None] + j - nb[:, None]) % Q, Q)
    more = torch.cat([ring, ring[:1]])
    more.scatter_(0, back.reshape(-1), table.reshape(-1))
    table.copy_(torch.where((j >= mb[:, None]) & (j < ng[:, None]), taken, table))
    ring.copy_(more[:Q])
    used = (want * ok).sum()
    state.copy_(torch.stack([(head + used) % Q, count - used + give.sum()]))
    granted.copy_(Lg)
    zero = torch.zeros(1, dtype=torch.int64, device=dev)
    ko = torch.cat([zero, Lg.cumsum(0)])
    no = torch.cat([zero, (Lg - P0).clamp(min=0).cumsum(0)])
    kv_off.copy_(ko)
    new_off.copy_(no)
    for off, dst, first in ((ko, slots, torch.zeros_like(P0)), (no, new_slots, P0)):
        i = torch.arange(dst.numel(), device=dev)
        b = torch.searchsorted(off[1:], i, right=True).clamp(max=B - 1)
        t = i - off[b] + first[b]
        value = table[b, (t // BLOCK).clamp(max=W - 1)] * BLOCK + t % BLOCK
        dst.copy_(torch.where(i < off[-1], value, dst))


def _run_prompt(s):
    if own:
        P = _handle(s, lambda P, shape: P.pillar_prompt_attn_workspace_bytes(shape, s["q"].shape[0]))
        P.pillar_prompt_attn(s["shape"], s["q"], s["k"], s["v"], s["seq_off"], s["out"], s["lse"], s["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    q, k, v, off, Lm = s["q"], s["k"], s["v"], s["seq_off"].long(), s["max_len"]
    (T, Hq, D), Hkv, B = q.shape, k.shape[1], off.numel() - 1
    i = torch.arange(Lm, device=q.device)
    at = (off[:-1, None] + i[None, :]).clamp(max=T - 1)                     # padded [B, Lm] -> packed rows
    qp = q[at].float().view(B, Lm, Hkv, Hq // Hkv, D).permute(0, 2, 3, 1, 4).reshape(B, Hkv, -1, D)
    kp, vp = k[at].float().transpose(1, 2), v[at].float().transpose(1, 2)   # [B, Hkv, Lm, D]
    sc = (qp @ kp.transpose(-1, -2)).view(B, Hkv, Hq // Hkv, Lm, Lm).mul_(1 / math.sqrt(D))
    sc.masked_fill_(i[None, :] > i[:, None], -math.inf)                     # (a row never sees past its own sequence)
    m = sc.amax(-1, keepdim=True)
    p = sc.sub_(m).exp_()
    den = p.sum(-1, keepdim=True)
    o = (p.view(B, Hkv, -1, Lm) @ vp).view(B, Hkv, Hq // Hkv, Lm, D) / den
    lse = (m + den.log())[..., 0]                                           # [B, Hkv, G, Lm]
    t = torch.arange(T, device=q.device)
    b = torch.searchsorted(off[1:], t, right=True)
    r = t - off[b]
    out = o.permute(0, 3, 1, 2, 4).reshape(B, Lm, Hq, D)[b, r].bfloat16()
    return {"out": out, "lse": lse.permute(0, 3, 1, 2).reshape(B, Lm, Hq)[b, r]}


def _run_append(s):
    if own:
        P = _handle(s)
        P.pillar_kv8_append(s["shape"], s["k_new"], s["v_new"], s["len"], s["new_off"], s["table"], s["k8"], s["v8"],
                            s["k_scale"], s["v_scale"])
    else:
        off, L = s["new_off"].long(), s["len"].long()
        i = torch.arange(s["k_new"].shape[0], device=L.device)
        b = torch.searchsorted(off[1:], i, right=True)
        pos = L[b] - off[b + 1] + i
        blk, row = s["table"][b, pos // BLOCK].long(), pos % BLOCK
        fresh = torch.zeros(s["k8"].shape[0], device=L.device)
        fresh = fresh.scatter_reduce(0, blk, (row == 0).float(), "amax")[:, None] > 0
        for x, pool, scale in ((s["k_new"], s["k8"], s["k_scale"]), (s["v_new"], s["v8"], s["v_scale"])):
            x = x.float()
            amax = torch.zeros_like(scale).index_reduce_(0, blk, x.abs().amax(-1), "amax")
            seen = torch.zeros_like(fresh[:, 0], dtype=torch.float32).index_fill(0, blk, 1.0)[:, None] > 0
            need = _pow2_scale(amax)
            new = torch.where(seen, torch.where(fresh, need, torch.maximum(scale, need)), scale)
            ratio = torch.where(seen & ~fresh, scale / new, torch.ones_like(scale))
            codes = (pool.float() * ratio[..., None, None]).to(torch.float8_e4m3fn)
            codes.view(torch.uint8)[blk, :, row] = (x / new[blk][..., None]).to(torch.float8_e4m3fn).view(torch.uint8)
            pool.copy_(codes)
            scale.copy_(new)
    return {x: s[x] for x in ("k8", "v8", "k_scale", "v_scale")}


def _run_attn8(s):
    c = s["case"]
    if own:
        P = _handle(s, lambda P, shape: P.pillar_attn_workspace_bytes(shape))
        P.pillar_attn_kv8(s["shape"], s["q"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["table"], s["mode"],
                          s["len"], s["idx"], s["cnt"], s["out"], s["logits"] if c["dump"] else None, s["lse"], s["ws"])
        return {"out": s["out"], "logits": s["logits"][:s["n_log"]], "lse": s["lse"][:s["V"]]}
    Hq, Hkv, D, k = c["Hq"], c["Hkv"], c["D"], c["k"]
    G, scale, q = Hq // Hkv, 1 / math.sqrt(D), s["q"].float().view(-1, Hkv, Hq // Hkv, D)
    L, table = s["len"].long(), s["table"].long()
    out, lse, logits = torch.zeros((q.shape[0], Hq, D), device=q.device), s["lse"][:s["V"]], s["logits"][:s["n_log"]]
    h = torch.arange(Hkv, device=q.device)

    def rows(pool, scales, blk, head, row):  # dequantised cache rows
        return pool.view(torch.uint8)[blk, head, row].view(torch.float8_e4m3fn).float() * scales[blk, head][..., None]

    if s["draft"].numel():  # one row per request over its lists
        d, pos = s["draft"], s["idx"][s["draft"]].long()                                   # [n, Hkv, ms]
        blk, row, head = table[d[:, None, None], pos // BLOCK], pos % BLOCK, h[None, :, None]
        kk, vv = rows(s["k8"], s["k_scale"], blk, head, row), rows(s["v8"], s["v_scale"], blk, head, row)
        sc = q[s["draft_row"]] @ kk.transpose(-1, -2) * scale                              # [n, Hkv, G, ms]
        seen = torch.arange(pos.shape[-1], device=q.device) < s["cnt"][d][..., None]
        p = _softmax(sc.masked_fill(~seen[:, :, None], -math.inf))[0]
        out[s["draft_row"]] = (p @ vv).view(-1, Hq, D)
    if s["V"]:  # k+1 causal rows per request over the whole context
        w, Lm = s["verify"], s["Lmax"]
        t = torch.arange(Lm, device=q.device)
        blk = table[w[:, None], (t // BLOCK)[None, :].clamp(max=table.shape[1] - 1)][:, None]  # [V, 1, Lm]
        head, row = h[None, :, None], (t % BLOCK)[None, None, :]
        kk, vv = rows(s["k8"], s["k_scale"], blk, head, row), rows(s["v8"], s["v_scale"], blk, head, row)
        qv = q[s["verify_row"]].permute(0, 2, 3, 1, 4).reshape(-1, Hkv, G * (k + 1), D)
        sc = (qv @ kk.transpose(-1, -2) * scale).view(-1, Hkv, G, k + 1, Lm)
        lim = L[w][:, None] - (k + 1) + torch.arange(k + 1, device=q.device)[None, :]       # [V, k+1]
        sc = sc.masked_fill((t > lim[..., None])[:, None, None], -math.inf)
        if c["dump"]:  # packed [V][Hq][k+1][L_v]
            n = Hq * (k + 1)
            off = torch.cat([torch.zeros_like(L[:1]), (n * L[w]).cumsum(0)])
            i = torch.arange(s["n_log"], device=q.device)
            v = torch.searchsorted(off[1:], i, right=True)
            r = i - off[v]
            Lv = L[w][v]
            logits.copy_(sc.reshape(-1)[(v * n + r // Lv) * Lm + r % Lv])
        p, z = _softmax(sc)
        lse.copy_(z.reshape(-1, Hq, k + 1))
        o = (p.view(-1, Hkv, G * (k + 1), Lm) @ vv).view(-1, Hq, k + 1, D)
        out[s["verify_row"]] = o.transpose(1, 2)
    return {"out": out.bfloat16(), "logits": logits, "lse": lse}


def _softmax(sc):
    m = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(m > -math.inf, m, 0.0)).exp()
    den = p.sum(-1, keepdim=True)
    return p / den.clamp(min=1e-30), (m + den.log())[..., 0]


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op = case["op"]
    L = _lengths(case, 0)
    if op == "block_map":
        P0 = L
        n = np.where(np.arange(case["B"]) % (case["k"] + 1) == 0, case["k"] + 1, 1)
        nb = -(-(P0 + n) // BLOCK)
        # two calls: lengths and blocks in; slots, new tokens' slots and offsets out
        byt = 2 * case["B"] * 8 + int(nb.sum() + (-(-P0 // BLOCK)).sum()) * 4
        byt += int((P0 + n).sum() + P0.sum() + n.sum()) * 4 + 2 * case["B"] * 16
        return {"bytes": byt, "flops": 0}
    D, Hkv = case["D"], case["Hkv"]
    if op == "prompt":
        T, Hq = int(L.sum()), case["Hq"]
        return {"bytes": T * D * 2 * (2 * Hq + 2 * Hkv) + T * Hq * 4, "flops": int((L * (L + 1) // 2).sum()) * Hq * D * 4}
    if op == "append":
        n = L if case["prompt"] else np.where(np.arange(case["B"]) % (case["k"] + 1) == 0, case["k"] + 1, 1)
        N = int(n.sum())
        blocks = int((-(-n // BLOCK)).sum())
        return {"bytes": N * Hkv * D * 2 * 3 + blocks * (Hkv * 8 + 4), "flops": 0}
    k, Hq, mode = case["k"], case["Hq"], _mode(case)
    L = np.maximum(L, k + 1)
    cnt = np.where(mode == 0, np.minimum(L, np.ceil(case["s"] * L)), 0).astype(np.int64)
    full = int(L[mode == 1].sum())
    T = int(np.where(mode == 1, k + 1, 1).sum())
    byt = full * Hkv * D * 2 + int(cnt.sum()) * Hkv * D * 2          # codes of K and V
    byt += int((-(-L[mode == 1] // BLOCK)).sum()) * (Hkv * 8 + 4)     # scales and table of whole contexts
    byt += int(cnt.sum()) * Hkv * 4                                   # lists
    byt += T * Hq * D * 4 + int((mode == 1).sum()) * Hq * (k + 1) * 4
    if case["dump"]:
        byt += full * Hq * (k + 1) * 4
    return {"bytes": byt, "flops": 4 * D * Hq * (full * (k + 1) + int(cnt.sum()))}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    op = case["op"]
    if op == "block_map":
        return None
    if op == "prompt" and work(case)["flops"] > 3e12:
        return None
    s = prepare(case, seed)
    if op == "prompt":
        return _exact_prompt(s)
    if op == "append":
        return _exact_append(s)
    return _exact_attn8(s)


def _attend(q, k, v, scale, visible):
    """q [..., r, D], k and v [n, D], visible [r, n]: output, log-sum-exp and scores in 64 bits."""
    sc = torch.matmul(q, k.T) * scale
    sc = torch.where(visible, sc, torch.full_like(sc, -math.inf))
    z = torch.logsumexp(sc, -1)
    p = torch.exp(sc - torch.where(torch.isfinite(z), z, torch.zeros_like(z))[..., None])
    return torch.matmul(p, v), z, sc


def _exact_prompt(s):
    q, k, v, off = s["q"], s["k"], s["v"], s["seq_off"].tolist()
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out = torch.zeros((T, Hq, D), dtype=torch.float64, device=q.device)
    lse = torch.zeros((T, Hq), dtype=torch.float64, device=q.device)
    for a, e in zip(off[:-1], off[1:]):
        for h in range(Hq):
            kk, vv = k[a:e, h // G].double(), v[a:e, h // G].double()
            for r in range(a, e, 4096):
                r1 = min(e, r + 4096)
                see = torch.arange(a, r1, device=q.device)[None, :] <= torch.arange(r, r1, device=q.device)[:, None]
                out[r:r1, h], lse[r:r1, h], _ = _attend(q[r:r1, h].double(), kk[:r1 - a], vv[:r1 - a], D ** -0.5, see)
    return {"out": out, "lse": lse}


def _e4m3_values():
    """Every finite value of the format: 4 exponent bits of bias 7, 3 fraction bits."""
    c = np.arange(128)
    e, m = c >> 3, c & 7
    v = np.where(e == 0, m * 2.0 ** -9, (8 + m) * 2.0 ** (e - 10.0))
    return v[:127]


def _nearest(x):
    """x (fp64) to the nearest e4m3 value, ties to the even code."""
    v = torch.from_numpy(_e4m3_values()).to(x.device)
    a = x.abs().clamp(max=E4M3_MAX)
    hi = torch.searchsorted(v, a.contiguous()).clamp(max=126)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - v[lo], v[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return torch.where(up, v[hi], v[lo]) * torch.sign(x)


def _exact_append(s):
    L, off, table = s["len"].tolist(), s["new_off"].tolist(), s["table"].tolist()
    got = {}
    for x, pool, scale in (("k_new", "k8", "k_scale"), ("v_new", "v8", "v_scale")):
        new, val, sc = s[x].double(), s[pool].double(), s[scale].double()
        for b in range(len(L)):
            n = off[b + 1] - off[b]
            t = L[b] - n
            while t < L[b]:
                i, r = t // BLOCK, t % BLOCK
                e = min(BLOCK, L[b] - i * BLOCK)
                j = table[b][i]
                rows = new[off[b] + t - (L[b] - n):][:e - r].transpose(0, 1)        # [Hkv, rows, D]
                a = rows.abs().amax((1, 2))
                two = torch.exp2(torch.ceil(torch.log2(a.clamp(min=1e-60) / E4M3_MAX)).clamp(min=-126))
                if r:
                    grown = torch.maximum(sc[j], two)
                    val[j] = torch.where((grown > sc[j])[:, None, None], _nearest(val[j] * (sc[j] / grown)[:, None, None]),
                                         val[j])
                    two = grown
                val[j, :, r:e] = _nearest(rows / two[:, None, None])
                sc[j] = two
                t = (i + 1) * BLOCK
        got[pool], got[scale] = val, sc
    return {x: got[x] for x in ("k8", "v8", "k_scale", "v_scale")}


def _exact_attn8(s):
    c = s["case"]
    Hq, Hkv, D, k = c["Hq"], c["Hkv"], c["D"], c["k"]
    G, dev = Hq // Hkv, s["q"].device
    L, mode, cnt = s["len"].tolist(), s["mode"].tolist(), s["cnt"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros((s["V"], Hq, k + 1), dtype=torch.float64, device=dev)
    logits, row, v = [], 0, 0
    for b in range(c["B"]):
        blocks = s["table"][b].long()
        t = torch.arange(L[b], device=dev)
        j, r = blocks[t // BLOCK], t % BLOCK
        nq = k + 1 if mode[b] else 1
        for g in range(Hkv):
            if mode[b]:
                jj, rr = j, r
                see = t[None, :] <= (L[b] - nq + torch.arange(nq, device=dev))[:, None]
            else:
                n = cnt[b][g]
                at = s["idx"][b, g, :n].long()
                jj, rr = j[at], r[at]
                see = torch.ones((1, n), dtype=torch.bool, device=dev)
            kk = s["k8"].view(torch.uint8)[jj, g, rr].view(torch.float8_e4m3fn).double() * s["k_scale"][jj, g].double()[:, None]
            vv = s["v8"].view(torch.uint8)[jj, g, rr].view(torch.float8_e4m3fn).double() * s["v_scale"][jj, g].double()[:, None]
            qq = s["q"][row:row + nq, g * G:(g + 1) * G].double().transpose(0, 1)        # [G, nq, D]
            o, z, sc = _attend(qq, kk, vv, D ** -0.5, see)
            out[row:row + nq, g * G:(g + 1) * G] = o.transpose(0, 1)
            if mode[b]:
                lse[v, g * G:(g + 1) * G] = z
                if c["dump"]:
                    logits.append(sc.reshape(-1))
        row += nq
        v += mode[b]
    flat = torch.cat(logits) if logits else torch.zeros(0, dtype=torch.float64, device=dev)
    return {"out": out, "logits": flat, "lse": lse}

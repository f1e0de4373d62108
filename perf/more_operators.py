"""Timed cases of the 4-bit cache's operators and of reading a cache back, with their plain forms.

  store     new K/V rows into the 4-bit cache (e2m1 codes, one scale byte per 16 values of a row), then read back: the
            values that later steps will attend to
  read4     a run of positions of each request, out of the 4-bit cache, as bf16 rows
  read8     the same out of the 8-bit cache
  attn4     the draft/verify attention step over the 4-bit cache

A value of the 4-bit cache is e2m1(code) * scale, with the codes' magnitudes 0, 0.5, 1, 1.5, 2, 3, 4, 6 and a scale byte of
five exponent bits (bias 15) and three fraction bits; an even dimension is the low half of its byte.

``run`` computes the plain form (elementary torch operations in fp32) where ``own`` is false and makes the framework's calls
where it is true.
"""
from __future__ import annotations

import math

import numpy as np
import torch

own = False
BLOCK = 16          # tokens of a cache block
GROUP = 16          # values that share a scale byte
MAGNITUDES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)
TOP_SCALE = 10240.0  # the largest scale that is written


# ------------------------------------------------------------------------------------------------ cases

def listed():
    return [
        # the new tokens of a decode step: one per draft request, k+1 per verify request
        dict(name="store_step", op="store", B=128, k=8, prompt=0, lo=64, hi=1024, Hkv=8, D=128),
        # the K/V of a prefill batch, stored and taken back rounded, so that the prompt attends to what is kept of it
        dict(name="store_prompt", op="store", B=32, k=0, prompt=1, lo=100, hi=4000, Hkv=8, D=128),
        # a few hundred positions of one short request, head dimension 64: latency
        dict(name="read4_short", op="read4", B=1, lo=333, hi=333, Hkv=1, D=64),
        # long contexts given back as bf16, e.g. to move them to the bf16 pools
        dict(name="read4_long", op="read4", B=16, lo=4096, hi=24576, Hkv=8, D=128),
        # the shared prefixes of a ragged batch, five KV heads of 64
        dict(name="read8_ragged", op="read8", B=24, lo=1, hi=2047, Hkv=5, D=64),
        # long contexts of the 8-bit cache
        dict(name="read8_long", op="read8", B=16, lo=4096, hi=24576, Hkv=8, D=128),
        # the smallest step: two draft and two verify requests, head dimension 64
        dict(name="attn4_tiny", op="attn4", B=4, Hq=4, Hkv=1, D=64, k=4, mix="mixed", lo=256, hi=512, s=0.1, dump=1),
        # one user with a long context, single tokens: the context is split over the whole GPU
        dict(name="attn4_one", op="attn4", B=1, Hq=32, Hkv=8, D=128, k=0, mix="full", lo=100001, hi=100001, s=0.05,
             dump=0),
        # single tokens over their whole contexts, no dump: plain decoding
        dict(name="attn4_decode", op="attn4", B=64, Hq=32, Hkv=8, D=128, k=0, mix="full", lo=1000, hi=30000, s=0.05,
             dump=0),
        # a step in which nobody verifies: every request attends to its list
        dict(name="attn4_drafts", op="attn4", B=128, Hq=32, Hkv=8, D=128, k=8, mix="draft", lo=6144, hi=10240, s=0.05,
             dump=0),
        # the Qwen3-8B-shaped speculative step: 128 requests, one ninth verify
        dict(name="attn4_8b", op="attn4", B=128, Hq=32, Hkv=8, D=128, k=8, mix="mixed", lo=6144, hi=10240, s=0.05, dump=1),
        # the Qwen3-14B-shaped step: five query heads per KV head, contexts 4K to 24K
        dict(name="attn4_14b", op="attn4", B=128, Hq=40, Hkv=8, D=128, k=8, mix="mixed", lo=4096, hi=24576, s=0.05,
             dump=1),
    ]


def _span(rng, lo, hi):
    """An integer spread over [lo, hi] on a logarithmic scale."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(("store", "read4", "read8", "attn4", "attn4"))
    D = rng.choice((64, 128))
    if op == "store":
        prompt = rng.randint(0, 1)
        hi = _span(rng, 20, 4000 if prompt else 1024)
        return dict(op=op, B=_span(rng, 1, 32 if prompt else 256), k=rng.randint(0, 12), prompt=prompt,
                    lo=_span(rng, 17, hi), hi=hi, Hkv=rng.choice((1, 2, 5, 8)), D=D)
    if op in ("read4", "read8"):
        hi = _span(rng, 1, 24576)
        return dict(op=op, B=max(1, min(_span(rng, 1, 128), 200000 // hi)), lo=_span(rng, 1, hi), hi=hi,
                    Hkv=rng.choice((1, 2, 5, 8)), D=D)
    G = rng.choice((1, 2, 4, 5, 8))
    Hkv = rng.choice((1, 2, 8))
    mix = rng.choice(("mixed", "mixed", "full", "draft"))
    k = rng.randint(1 if mix == "draft" else 0, min(12, 64 // G - 1))
    hi = _span(rng, 100, 100000)
    # at most the 14B-shaped step's keys and logits
    B = max(1, min(_span(rng, 1, 128), (128 * 9000) // hi))
    if mix == "full":
        B = max(1, min(B, 15 * 40 * 9 * 14000 // (hi * G * Hkv * (k + 1))))
    return dict(op=op, B=B, Hq=G * Hkv, Hkv=Hkv, D=D, k=k, mix=mix, lo=_span(rng, 32, hi), hi=hi,
                s=rng.choice((0.03, 0.05, 0.1)), dump=rng.randint(0, 1))


# ------------------------------------------------------------------------------------------------ inputs

def _lengths(case):
    """The case's lengths (the same for every seed: a case is one amount of work)."""
    g = np.random.default_rng((case["B"], case["lo"], case["hi"]))
    return np.rint(np.exp(g.uniform(math.log(case["lo"]), math.log(case["hi"] + 0.49), case["B"]))).astype(np.int64)


def _new_tokens(case):
    L = _lengths(case)
    return L if case["prompt"] else np.where(np.arange(case["B"]) % (case["k"] + 1) == 0, case["k"] + 1, 1)


def _mode(case):
    if case["mix"] == "full":
        return np.ones(case["B"], np.int64)
    if case["mix"] == "draft":
        return np.zeros(case["B"], np.int64)
    return (np.arange(case["B"]) % (case["k"] + 1) == 0).astype(np.int64)


def _dev(a, dtype):
    return torch.from_numpy(np.ascontiguousarray(a)).to("cuda").to(dtype)


def _offsets(n):
    return np.concatenate([[0], np.cumsum(n)]).astype(np.int64)


def _tables(g, L, spare):
    """Block tables [B, max_blocks] over a shuffled pool, and the blocks of the pool."""
    nb = -(-L // BLOCK)
    total = int(nb.sum()) + spare
    perm = g.permutation(total)
    t = np.zeros((len(L), int(max(1, nb.max())) + 1), np.int64)
    at = 0
    for b, n in enumerate(nb):
        t[b, :n] = perm[at:at + n]
        at += n
    return t, total


def _scales4(x):
    """x [..., D] fp32 -> scale bytes and scales [..., D / 16]: the smallest scale s with max |x| <= 6 s."""
    a = x.unflatten(-1, (-1, GROUP)).abs().amax(-1)
    f, e = torch.frexp((a / 6).clamp(min=2.0 ** -17, max=TOP_SCALE))          # f in [0.5, 1)
    e = e.clamp(min=-13)                                                       # (subnormal scales: a fixed step)
    s = torch.ldexp(torch.ceil(torch.ldexp((a / 6).clamp(min=2.0 ** -17, max=TOP_SCALE), 4 - e)), e - 4)
    return (s.half().view(torch.int16) >> 7).to(torch.uint8), s


def _quantise4(x):
    """[..., D] fp32 -> packed codes [..., D / 2] and scale bytes [..., D / 16]."""
    byte, s = _scales4(x)
    y = (x.unflatten(-1, (-1, GROUP)) / s[..., None]).flatten(-2)
    a = y.abs()
    # the nearest magnitude, ties to the even code
    c = (a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5) + (a >= 3.5) + (a > 5)
    c = c.to(torch.uint8) | (torch.signbit(x).to(torch.uint8) << 3)
    return c[..., 0::2] | (c[..., 1::2] << 4), byte


def _values4(codes, scale):
    """Packed codes [..., D / 2] and scale bytes [..., D / 16] -> fp32 values [..., D]."""
    table = torch.tensor(MAGNITUDES + tuple(-m for m in MAGNITUDES), device=codes.device)
    c = torch.stack((codes & 15, codes >> 4), -1).flatten(-2)
    s = (scale.to(torch.int16) << 7).view(torch.float16).float()
    return (table[c.int()].unflatten(-1, (-1, GROUP)) * s[..., None]).flatten(-2)


def _cache4(gen, total, Hkv, D, u=None):
    """A filled 4-bit pool; with u, one position in twenty carries the head's direction."""
    codes = torch.empty((total, Hkv, BLOCK, D // 2), dtype=torch.uint8, device="cuda")
    scale = torch.empty((total, Hkv, BLOCK, D // GROUP), dtype=torch.uint8, device="cuda")
    for at in range(0, total, 4096):
        n = min(4096, total - at)
        x = torch.randn((n, Hkv, BLOCK, D), generator=gen, device="cuda")
        if u is not None:
            x += 2 * u[None, :, None, :] * (torch.rand((n, Hkv, BLOCK, 1), generator=gen, device="cuda") < 0.05)
        codes[at:at + n], scale[at:at + n] = _quantise4(x)
    return codes, scale


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(int(seed) * 7919 + 13)
    g = np.random.default_rng((int(seed), 99))
    s = dict(op=case["op"], case=dict(case))
    {"store": _prepare_store, "read4": _prepare_read, "read8": _prepare_read, "attn4": _prepare_attn}[case["op"]](case, g, gen, s)
    return s


def _shape_of(case, L, total, **over):
    return dict(dict(B=case["B"], Hq=case["Hkv"], Hkv=case["Hkv"], D=case["D"], k=0, row_lo=0, max_sparse=0,
                     max_len=int(L.max()), num_slots=total * BLOCK), **over)


def _prepare_store(case, g, gen, s):
    """New K/V rows, and a cache that holds what came before them."""
    B, Hkv, D, n = case["B"], case["Hkv"], case["D"], _new_tokens(case)
    L = n if case["prompt"] else _lengths(case) + n
    table, total = _tables(g, L, spare=8)
    N = int(n.sum())
    s["k4"], s["k_scale"] = _cache4(gen, total, Hkv, D)
    s["v4"], s["v_scale"] = s["k4"].roll(1, 0), s["k_scale"].roll(1, 0)
    # keys with a few large dimensions, as rotary keys have; one token in sixteen is large as a whole
    wide = 1 + 9 * (torch.rand((1, Hkv, D), generator=gen, device="cuda") < 1 / 32)
    big = 1 + 5 * (torch.rand((N, 1, 1), generator=gen, device="cuda") < 1 / 16)
    s["k_new"] = (torch.randn((N, Hkv, D), generator=gen, device="cuda") * wide * big).bfloat16()
    s["v_new"] = torch.randn((N, Hkv, D), generator=gen, device="cuda").bfloat16()
    s["len"], s["new_off"], s["first"] = _dev(L, torch.int32), _dev(_offsets(n), torch.int32), _dev(L - n, torch.int32)
    s["table"] = _dev(table, torch.int32)
    s["k_out"], s["v_out"] = torch.zeros_like(s["k_new"]), torch.zeros_like(s["v_new"])
    s["shape_of"] = _shape_of(case, L, total)


def _prepare_read(case, g, gen, s):
    """A filled cache, and a run of positions of each request."""
    B, Hkv, D, n = case["B"], case["Hkv"], case["D"], _lengths(case)
    first = g.integers(0, 100, B)  # (behind a part that the reader has already)
    L = first + n
    table, total = _tables(g, L, spare=8)
    if case["op"] == "read4":
        s["k4"], s["k_scale"] = _cache4(gen, total, Hkv, D)
        s["v4"], s["v_scale"] = s["k4"].roll(1, 0), s["k_scale"].roll(1, 0)
    else:
        for x in "kv":
            c = torch.randint(0, 255, (total, Hkv, BLOCK, D), generator=gen, device="cuda", dtype=torch.uint8)
            s[x + "8"] = torch.where((c & 127) == 127, c - 1, c).view(torch.float8_e4m3fn)  # (every code but NaN)
            s[x + "_scale"] = torch.exp2(torch.randint(-9, -5, (total, Hkv), generator=gen, device="cuda").float())
    s["first"], s["out_off"], s["table"] = _dev(first, torch.int32), _dev(_offsets(n), torch.int32), _dev(table, torch.int32)
    N = int(n.sum())
    s["k_out"] = torch.zeros((N, Hkv, D), dtype=torch.bfloat16, device="cuda")
    s["v_out"] = torch.zeros_like(s["k_out"])
    s["shape_of"] = _shape_of(case, L, total)


def _prepare_attn(case, g, gen, s):
    """A batch of draft and verify requests over a filled 4-bit cache."""
    B, Hq, Hkv, D, k = (case[x] for x in ("B", "Hq", "Hkv", "D", "k"))
    mode = _mode(case)
    L = np.maximum(_lengths(case), k + 1)
    table, total = _tables(g, L, spare=8)
    # keys and queries with the pillar structure: one position in twenty carries the head's direction
    u = torch.randn((Hkv, D), generator=gen, device="cuda")
    u = u / u.norm(dim=-1, keepdim=True)
    s["k4"], s["k_scale"] = _cache4(gen, total, Hkv, D, u)
    s["v4"], s["v_scale"] = _cache4(gen, total, Hkv, D)
    rows = np.where(mode == 1, k + 1, 1)
    q_off = _offsets(rows)
    T = int(rows.sum())
    q = torch.randn((T, Hq, D), generator=gen, device="cuda") + 3 * u.repeat_interleave(Hq // Hkv, 0)
    s["q"] = q.bfloat16()
    s["len"], s["mode"], s["table"] = _dev(L, torch.int32), _dev(mode, torch.int32), _dev(table, torch.int32)
    # critical lists of the draft requests: ascending positions, ceil(s L) per KV head
    cnt = np.where(mode == 0, np.minimum(L, np.ceil(case["s"] * L)), 0).astype(np.int64)
    ms, Lmax = int(max(1, cnt.max())), int(L.max())
    idx = torch.zeros((B, Hkv, ms), dtype=torch.int32, device="cuda")
    Ld, cd = _dev(L, torch.int64), _dev(cnt, torch.int64)
    for at in range(0, B if cnt.max() else 0, 16):
        n = min(16, B - at)
        w = torch.rand((n, Hkv, Lmax), generator=gen, device="cuda")
        w = torch.where(torch.arange(Lmax, device="cuda") < Ld[at:at + n, None, None], w, -1.0)
        top = w.topk(ms, dim=-1).indices  # by weight: the first cnt are a random subset of the context
        top = torch.where(torch.arange(ms, device="cuda") < cd[at:at + n, None, None], top, Lmax)
        idx[at:at + n] = top.sort(dim=-1).values.to(torch.int32)
    s["idx"] = torch.where(idx < Lmax, idx, 0)
    s["cnt"] = _dev(np.repeat(cnt[:, None], Hkv, 1), torch.int32)
    # where the plain form finds its rows: draft requests, verify requests, and the packed logits of the latter
    dr, ve = np.nonzero(mode == 0)[0], np.nonzero(mode == 1)[0]
    s["draft"], s["verify"] = _dev(dr, torch.int64), _dev(ve, torch.int64)
    s["draft_row"] = _dev(q_off[dr], torch.int64)
    s["verify_row"] = _dev(q_off[ve][:, None] + np.arange(k + 1)[None, :], torch.int64)
    V, Lv = len(ve), L[ve]
    n_log = int(Hq * (k + 1) * Lv.sum())
    s["V"], s["Lv"] = V, Lv.tolist()
    s["logits"] = torch.zeros(max(2, n_log) if case["dump"] else 2, dtype=torch.float32, device="cuda")
    s["n_log"] = n_log if case["dump"] else 0
    s["lse"] = torch.zeros((max(1, V), Hq, k + 1), dtype=torch.float32, device="cuda")
    s["out"] = torch.zeros((T, Hq, D), dtype=torch.bfloat16, device="cuda")
    s["shape_of"] = _shape_of(case, L, total, Hq=Hq, k=k, row_lo=min(1, k), max_sparse=ms)


# ------------------------------------------------------------------------------------------------ one pass

def run(s):
    return {"store": _run_store, "read4": _run_read4, "read8": _run_read8, "attn4": _run_attn}[s["op"]](s)


def _handle(s, workspace_bytes=None):
    """The binding, the shape record and the workspace that a program makes once and keeps."""
    import sparse_self_speculative_pillar_gb300 as P
    if "shape" not in s:
        s["shape"] = P.make_shape(**s["shape_of"])
        if workspace_bytes:
            s["ws"] = torch.empty(workspace_bytes(P, s["shape"]), dtype=torch.uint8, device="cuda")
    return P


def _places(s, first, off, rows):
    """Block and row of the block of each packed row."""
    off = off.long()
    i = torch.arange(rows, device=off.device)
    b = torch.searchsorted(off[1:], i, right=True)
    pos = first[b].long() + i - off[b]
    return s["table"][b, pos // BLOCK].long(), pos % BLOCK


def _run_store(s):
    if own:
        P = _handle(s)
        P.pillar_kv4_append(s["shape"], s["k_new"], s["v_new"], s["len"], s["new_off"], s["table"], s["k4"], s["v4"],
                            s["k_scale"], s["v_scale"])
        P.pillar_kv4_read(s["shape"], s["k4"], s["v4"], s["k_scale"], s["v_scale"], s["table"], s["first"], s["new_off"],
                          s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    blk, row = _places(s, s["first"], s["new_off"], s["k_new"].shape[0])
    for x in "kv":
        codes, scale = _quantise4(s[x + "_new"].float())
        s[x + "4"][blk, :, row] = codes
        s[x + "_scale"][blk, :, row] = scale
        s[x + "_out"].copy_(_values4(s[x + "4"][blk, :, row], s[x + "_scale"][blk, :, row]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_read4(s):
    if own:
        P = _handle(s)
        P.pillar_kv4_read(s["shape"], s["k4"], s["v4"], s["k_scale"], s["v_scale"], s["table"], s["first"], s["out_off"],
                          s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    blk, row = _places(s, s["first"], s["out_off"], s["k_out"].shape[0])
    for x in "kv":
        s[x + "_out"].copy_(_values4(s[x + "4"][blk, :, row], s[x + "_scale"][blk, :, row]))
    return {"k": s["k_out"], "v": s["v_out"]}


def _run_read8(s):
    if own:
        P = _handle(s)
        P.pillar_kv8_read(s["shape"], s["k8"], s["v8"], s["k_scale"], s["v_scale"], s["table"], s["first"], s["out_off"],
                          s["k_out"], s["v_out"])
        return {"k": s["k_out"], "v": s["v_out"]}
    blk, row = _places(s, s["first"], s["out_off"], s["k_out"].shape[0])
    for x in "kv":
        codes = s[x + "8"].view(torch.uint8)[blk, :, row].view(torch.float8_e4m3fn)
        s[x + "_out"].copy_(codes.float() * s[x + "_scale"][blk][..., None])
    return {"k": s["k_out"], "v": s["v_out"]}


def _softmax(sc):
    m = sc.amax(-1, keepdim=True)
    p = (sc - torch.where(m > -math.inf, m, 0.0)).exp()
    den = p.sum(-1, keepdim=True)
    return p / den.clamp(min=1e-30), (m + den.log())[..., 0]


def _run_attn(s):
    c = s["case"]
    if own:
        P = _handle(s, lambda P, shape: P.pillar_attn_workspace_bytes(shape))
        P.pillar_attn_kv4(s["shape"], s["q"], s["k4"], s["v4"], s["k_scale"], s["v_scale"], s["table"], s["mode"],
                          s["len"], s["idx"], s["cnt"], s["out"], s["logits"] if c["dump"] else None, s["lse"], s["ws"])
        return {"out": s["out"], "logits": s["logits"][:s["n_log"]], "lse": s["lse"][:s["V"]]}
    Hq, Hkv, D, k = c["Hq"], c["Hkv"], c["D"], c["k"]
    G, scale, q = Hq // Hkv, 1 / math.sqrt(D), s["q"].float().view(-1, Hkv, Hq // Hkv, D)
    L, table = s["len"].long(), s["table"].long()
    out, lse, logits = torch.zeros((q.shape[0], Hq, D), device=q.device), s["lse"][:s["V"]], s["logits"][:s["n_log"]]
    h = torch.arange(Hkv, device=q.device)

    def rows(x, blk, head, row):  # values of cache rows
        return _values4(s[x + "4"][blk, head, row], s[x + "_scale"][blk, head, row])

    for at in range(0, s["draft"].numel(), 32):  # one row per request over its lists, 32 requests at a time
        d, into = s["draft"][at:at + 32], s["draft_row"][at:at + 32]
        pos = s["idx"][d].long()                                                           # [n, Hkv, ms]
        blk, row, head = table[d[:, None, None], pos // BLOCK], pos % BLOCK, h[None, :, None]
        kk, vv = rows("k", blk, head, row), rows("v", blk, head, row)
        sc = q[into] @ kk.transpose(-1, -2) * scale                                        # [n, Hkv, G, ms]
        seen = torch.arange(pos.shape[-1], device=q.device) < s["cnt"][d][..., None]
        p = _softmax(sc.masked_fill(~seen[:, :, None], -math.inf))[0]
        out[into] = (p @ vv).view(-1, Hq, D)
    end = 0
    for v, n in enumerate(s["Lv"]):  # k+1 causal rows over the whole context, a request at a time
        t = torch.arange(n, device=q.device)
        blk = table[s["verify"][v], t // BLOCK][None, :]
        kk, vv = rows("k", blk, h[:, None], (t % BLOCK)[None, :]), rows("v", blk, h[:, None], (t % BLOCK)[None, :])
        qv = q[s["verify_row"][v]].permute(1, 2, 0, 3).reshape(Hkv, G * (k + 1), D)
        sc = (qv @ kk.transpose(-1, -2) * scale).view(Hkv, G, k + 1, n)
        lim = n - (k + 1) + torch.arange(k + 1, device=q.device)
        sc = sc.masked_fill(t > lim[:, None], -math.inf)
        if c["dump"]:  # packed [V][Hq][k+1][L_v]
            logits[end:end + sc.numel()] = sc.reshape(-1)
            end += sc.numel()
        p, z = _softmax(sc)
        lse[v] = z.reshape(Hq, k + 1)
        o = (p.view(Hkv, G * (k + 1), n) @ vv).view(Hq, k + 1, D)
        out[s["verify_row"][v]] = o.transpose(0, 1)
    return {"out": out.bfloat16(), "logits": logits, "lse": lse}


# ------------------------------------------------------------------------------------------------ work

def work(case):
    op, D, Hkv = case["op"], case["D"], case["Hkv"]
    row4 = Hkv * 2 * (D // 2 + D // GROUP)  # a token's codes and scales, K and V
    row16 = Hkv * 2 * D * 2                 # its bf16 values
    if op == "store":
        n = _new_tokens(case)
        N = int(n.sum())
        return {"bytes": N * (2 * row16 + row4) + int((-(-n // BLOCK)).sum()) * 4 + case["B"] * 12, "flops": 0}
    L = _lengths(case)
    if op in ("read4", "read8"):
        N, blocks = int(L.sum()), int((-(-L // BLOCK)).sum())
        held = N * row4 if op == "read4" else N * Hkv * 2 * D + blocks * Hkv * 8
        return {"bytes": N * row16 + held + blocks * 4 + case["B"] * 8, "flops": 0}
    k, Hq, mode = case["k"], case["Hq"], _mode(case)
    L = np.maximum(L, k + 1)
    cnt = np.where(mode == 0, np.minimum(L, np.ceil(case["s"] * L)), 0).astype(np.int64)
    full, listed_keys = int(L[mode == 1].sum()), int(cnt.sum())
    T = int(np.where(mode == 1, k + 1, 1).sum())
    byt = (full + listed_keys) * row4                                 # codes and scales of K and V
    byt += int((-(-L[mode == 1] // BLOCK)).sum()) * 4                 # tables of whole contexts
    byt += listed_keys * Hkv * 4                                      # lists
    byt += T * Hq * D * 4 + int((mode == 1).sum()) * Hq * (k + 1) * 4
    if case["dump"]:
        byt += full * Hq * (k + 1) * 4
    return {"bytes": byt, "flops": 4 * D * Hq * (full * (k + 1) + listed_keys)}


# ------------------------------------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    return {"store": _exact_store, "read4": _exact_read, "read8": _exact_read, "attn4": _exact_attn}[case["op"]](s)


def _e2m1(code):
    """Sign, two exponent bits of bias 1, one fraction bit (int64 codes)."""
    e, m = (code >> 1) & 3, (code & 1).double()
    a = torch.where(e == 0, m / 2, torch.exp2((e - 1).double()) * (1 + m / 2))
    return torch.where(code & 8 > 0, -a, a)


def _scale_value(byte):
    """Five exponent bits of bias 15, three fraction bits (int64 bytes)."""
    e, m = byte >> 3, (byte & 7).double()
    return torch.where(e == 0, m * 2.0 ** -17, torch.exp2((e - 15).double()) * (1 + m / 8))


def _held(pool, scale, blk, head, row):
    """Values of 4-bit rows in 64 bits."""
    c = pool[blk, head, row].long()
    codes = torch.stack((c % 16, c // 16), -1).reshape(c.shape[:-1] + (-1,))
    return _e2m1(codes) * _scale_value(scale[blk, head, row].long()).repeat_interleave(GROUP, -1)


def _exact_store(s):
    """Of the definition alone: the scale out of all scales, then the nearest value out of all codes."""
    out = {}
    scales = _scale_value(torch.arange(1, 227, device="cuda"))  # 2^-17 .. 10240, ascending
    mags = torch.tensor(MAGNITUDES, dtype=torch.float64, device="cuda")
    for x in "kv":
        parts = []
        for new in s[x + "_new"].double().split(4096):
            gr = new.reshape(new.shape[:-1] + (-1, GROUP))
            sc = scales[torch.searchsorted(6 * scales, gr.abs().amax(-1).contiguous()).clamp(max=225)][..., None]
            a = (gr.abs() / sc).clamp(max=6.0)
            hi = torch.searchsorted(mags, a).clamp(max=7)
            lo = (hi - 1).clamp(min=0)
            dl, dh = a - mags[lo], mags[hi] - a
            n = torch.where((dh < dl) | ((dh == dl) & (hi % 2 == 0)), mags[hi], mags[lo])
            parts.append((n * torch.sign(gr) * sc).reshape(new.shape))
        out[x] = torch.cat(parts)
    return out


def _exact_read(s):
    first, off, table = s["first"].tolist(), s["out_off"].tolist(), s["table"].tolist()
    out, h = {}, torch.arange(s["k_out"].shape[1], device="cuda")[None, :]
    for x in "kv":
        parts = []
        for b in range(len(first)):
            t = np.arange(first[b], first[b] + off[b + 1] - off[b])
            blk = torch.tensor(np.asarray(table[b])[t // BLOCK], device="cuda")[:, None]
            row = torch.tensor(t % BLOCK, device="cuda")[:, None]
            if s["op"] == "read4":
                parts.append(_held(s[x + "4"], s[x + "_scale"], blk, h, row))
            else:
                c = s[x + "8"].view(torch.uint8)[blk, h, row].long()
                e, m = (c >> 3) & 15, (c & 7).double()
                a = torch.where(e == 0, m * 2.0 ** -9, (8 + m) * torch.exp2((e - 10).double()))
                parts.append(torch.where(c > 127, -a, a) * s[x + "_scale"][blk, h].double()[..., None])
        out[x] = torch.cat(parts)
    return out


def _exact_attn(s):
    c = s["case"]
    Hq, Hkv, D, k = c["Hq"], c["Hkv"], c["D"], c["k"]
    G, dev = Hq // Hkv, s["q"].device
    L, mode, cnt = s["len"].tolist(), s["mode"].tolist(), s["cnt"].tolist()
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device=dev)
    lse = torch.zeros((s["V"], Hq, k + 1), dtype=torch.float64, device=dev)
    logits, row, v = [], 0, 0
    for b in range(c["B"]):
        blocks = s["table"][b].long()
        nq = k + 1 if mode[b] else 1
        for g in range(Hkv):
            t = torch.arange(L[b], device=dev) if mode[b] else s["idx"][b, g, :cnt[b][g]].long()
            j, r = blocks[t // BLOCK], t % BLOCK
            kk, vv = (_held(s[x + "4"], s[x + "_scale"], j, g, r) for x in "kv")
            qq = s["q"][row:row + nq, g * G:(g + 1) * G].double().transpose(0, 1)          # [G, nq, D]
            sc = torch.matmul(qq, kk.T) * D ** -0.5
            if mode[b]:
                sc = torch.where(t[None, :] <= (L[b] - nq + torch.arange(nq, device=dev))[:, None], sc, -math.inf)
            z = torch.logsumexp(sc, -1)
            p = torch.exp(sc - torch.where(torch.isfinite(z), z, 0.0)[..., None])
            out[row:row + nq, g * G:(g + 1) * G] = torch.matmul(p, vv).transpose(0, 1)
            if mode[b]:
                lse[v, g * G:(g + 1) * G] = z
                if c["dump"]:
                    logits.append(sc.reshape(-1))
        row += nq
        v += mode[b]
    flat = torch.cat(logits) if logits else torch.zeros(0, dtype=torch.float64, device=dev)
    return {"out": out, "logits": flat, "lse": lse}

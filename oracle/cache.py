"""Plain numpy definitions of the cache operators, in integers and fp64 -- TEST INFRASTRUCTURE.

Element by element, with Python loops, sharing no code with the CUDA library:

  block_map     block tables and slot maps from request lengths
  kv8_append    new rows into the 8-bit cache (e4m3 codes, a power-of-two scale per block and KV head)
  attn_kv8      draft / verify attention over that cache
  prompt_attn   causal attention over packed prompts

Pinned by tests/test_cache_oracle_pins.py.
"""
from __future__ import annotations

import math

import numpy as np

BLOCK = 16


def block_map(req_len, prev_len, table, ring, state, max_len, num_blocks):
    """Returns a dict of the call's outputs (lists where lengths depend on the data) and the problems it meets
    ("request", "block", "slot").  table, ring and state are not modified."""
    table, ring, (head, count) = np.array(table), np.array(ring), [int(x) for x in state]
    before, B, W = ring.copy(), len(req_len), np.array(table).shape[1]
    most, bad = min(max_len, W * BLOCK), set()
    ring_ok = 0 <= head < num_blocks and 0 <= count <= num_blocks
    if not ring_ok:
        bad.add("block")
        head = count = 0
    asked = taken = given = 0
    granted, kv_off, new_off, slots, new_slots = [], [0], [0], [], []
    push = []
    for b in range(B):
        p, n = int(prev_len[b]), int(req_len[b])
        if not 0 <= p <= most:
            bad.add("request")
            p = n = 0
        if not 0 <= n <= most:
            bad.add("request")
            n = p
        have, want = -(-p // BLOCK), -(-n // BLOCK)
        asked += max(want - have, 0)
        if want > have and asked > count:
            bad.add("block")
            n, want = p, have
        for i in range(have, want):
            table[b, i] = before[(head + taken) % num_blocks]
            taken += 1
        for i in range(want, have):
            push.append(int(table[b, i]))
            given += 1

        def slot(t):
            blk = int(table[b, t // BLOCK])
            if not 0 <= blk < num_blocks:
                bad.add("slot")
                return -1
            return blk * BLOCK + t % BLOCK

        granted.append(n)
        slots += [slot(t) for t in range(n)]
        kv_off.append(len(slots))
        new_slots += [slot(t) for t in range(p, n)]
        new_off.append(len(new_slots))
    if ring_ok and count + given > num_blocks:  # the tables and the ring disagree: nothing is given back
        bad.add("block")
        push, given = [], 0
    if ring_ok:
        for i, blk in enumerate(push):
            if not 0 <= blk < num_blocks:
                bad.add("slot")
            ring[(head + count + i) % num_blocks] = blk
        state = [(head + taken) % num_blocks, count - taken + given]
    return dict(table=table, ring=ring, state=np.array(state), granted=np.array(granted), kv_off=np.array(kv_off),
                new_off=np.array(new_off), slots=np.array(slots, np.int64), new_slots=np.array(new_slots, np.int64),
                bad=bad)


# ---------------------------------------------------------------- e4m3

def e4m3_table():
    """Value of each of the 256 codes: sign, 4 exponent bits of bias 7, 3 fraction bits; 0x7f and 0xff are NaN."""
    v = np.empty(256)
    for c in range(256):
        e, m = (c >> 3) & 15, c & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        v[c] = math.nan if (c & 127) == 127 else (-x if c & 128 else x)
    return v


_VALUES = e4m3_table()


def e4m3_encode(x):
    """Codes of fp64 values: nearest, ties to the even code, magnitudes past 448 to 448; the sign of zero is kept."""
    x = np.asarray(x, np.float64)
    mag = _VALUES[:127]
    a = np.minimum(np.abs(x), 448.0)
    hi = np.minimum(np.searchsorted(mag, a), 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - mag[lo], mag[hi] - a
    up = (dh < dl) | ((dh == dl) & (hi % 2 == 0))
    return (np.where(up, hi, lo) | np.where(np.signbit(x), 128, 0)).astype(np.uint8)


def e4m3_decode(codes):
    return _VALUES[np.asarray(codes, np.uint8)]


def scale_of(amax):
    """2^e, e the smallest integer >= -126 with amax <= 448 * 2^e."""
    e = -126
    while amax > 448.0 * 2.0 ** e:
        e += 1
    return 2.0 ** e


def kv8_append(codes, scale, new, req_len, new_off, table):
    """codes [num_blocks, Hkv, 16, D] uint8 and scale [num_blocks, Hkv] after the new rows [n, Hkv, D] (fp64, finite)."""
    codes, scale = codes.copy(), scale.astype(np.float64)
    for b in range(len(req_len)):
        n = int(new_off[b + 1]) - int(new_off[b])
        first, last = int(req_len[b]) - n, int(req_len[b])
        for i in range(first // BLOCK, -(-last // BLOCK) if n else 0):
            lo, hi = max(first, i * BLOCK), min(last, (i + 1) * BLOCK)
            blk = int(table[b, i])
            for h in range(codes.shape[1]):
                x = new[int(new_off[b]) + lo - first:int(new_off[b]) + hi - first, h]
                s = scale_of(np.abs(x).max())
                r = lo % BLOCK
                if r:
                    s = max(s, scale[blk, h])
                    if s > scale[blk, h]:  # the block's other rows under the larger scale
                        codes[blk, h] = e4m3_encode(e4m3_decode(codes[blk, h]) * (scale[blk, h] / s))
                codes[blk, h, r:r + hi - lo] = e4m3_encode(x / s)
                scale[blk, h] = s
    return codes, scale


# ---------------------------------------------------------------- attention

def _attend(q, k, v, scale):
    """One query row over the keys it sees: output, log-sum-exp, scaled scores (all fp64)."""
    s = scale * (k @ q)
    if len(s) == 0:
        return np.zeros(v.shape[1]), -math.inf, s
    m = s.max()
    e = np.exp(s - m)
    return e @ v / e.sum(), m + math.log(e.sum()), s


def attn_kv8(q, k8, v8, k_scale, v_scale, table, req_mode, req_len, sparse_idx, sparse_cnt, k, scale):
    """q [T, Hq, D] fp64; the cache as codes [num_blocks, Hkv, 16, D] and scales.  Listed positions outside [0, L) and
    blocks outside the pool are left out.  Returns out [T, Hq, D], the packed logits and the LSEs [V, Hq, k+1]."""
    T, Hq, D = q.shape
    nblk, Hkv = k8.shape[:2]
    G, row = Hq // Hkv, 0
    out, logits, lse = np.zeros_like(q), [], []
    for b in range(len(req_len)):
        L, verify = int(req_len[b]), int(req_mode[b]) == 1
        nq = k + 1 if verify else 1
        dump, z = np.full((Hq, nq, L), -math.inf), np.full((Hq, nq), -math.inf)
        for g in range(Hkv):
            listed = range(L) if verify else [int(t) for t in sparse_idx[b, g, :int(sparse_cnt[b, g])]]
            t = np.array([x for x in listed if 0 <= x < L and 0 <= int(table[b, x // BLOCK]) < nblk], np.int64)
            blk = table[b, t // BLOCK].astype(np.int64) if len(t) else np.zeros(0, np.int64)
            kk = e4m3_decode(k8[blk, g, t % BLOCK]) * k_scale[blk, g].astype(np.float64)[:, None]
            vv = e4m3_decode(v8[blk, g, t % BLOCK]) * v_scale[blk, g].astype(np.float64)[:, None]
            for j in range(nq):
                n = int(np.searchsorted(t, L - nq + j, side="right")) if verify else len(t)
                for h in range(g * G, (g + 1) * G):
                    o, zz, s = _attend(q[row + j, h], kk[:n], vv[:n], scale)
                    out[row + j, h] = o
                    if verify:
                        dump[h, j, t[:n]] = s
                        z[h, j] = zz
        if verify:
            logits.append(dump.reshape(-1))
            lse.append(z)
        row += nq
    return (out, np.concatenate(logits) if logits else np.zeros(0),
            np.stack(lse) if lse else np.zeros((0, Hq, k + 1)))


def prompt_attn(q, k, v, seq_off, scale):
    """Causal attention of packed prompts, fp64 [T, heads, D]; rows outside the sequences are left at zero (LSE 0)."""
    T, Hq, D = q.shape
    G = Hq // k.shape[1]
    out, lse = np.zeros((T, Hq, D)), np.zeros((T, Hq))
    for a, e in zip(seq_off[:-1], seq_off[1:]):
        for h in range(Hq):
            for i in range(int(a), int(e)):
                out[i, h], lse[i, h], _ = _attend(q[i, h], k[int(a):i + 1, h // G], v[int(a):i + 1, h // G], scale)
    return out, lse

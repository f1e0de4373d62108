"""The 4-bit attention's item size for long contexts: the rule, and the calls that it decides."""
import ctypes
import os
import subprocess

import numpy as np
import pytest

import sparse_self_speculative_pillar_gb300 as P
from sparse_self_speculative_pillar_gb300 import _build

torch = pytest.importorskip("torch")

# the rule as the library's host code has it; a division by zero ends the program on every machine
PROGRAM = r"""
#include <cstdio>
#include "pillar_internal.h"
int main() {
    pillar_shape_t s = {};
    s.D = 128;
    int nsm;
    while (std::scanf("%d %d %d %d %d %d", &s.B, &s.Hq, &s.Hkv, &s.k, &s.max_len, &nsm) == 6)
        std::printf("%d\n", pillar::kv4_chunk(s, nsm));
}
"""


@pytest.fixture(scope="module")
def chunks(tmp_path_factory):
    d = tmp_path_factory.mktemp("rule")
    (d / "rule.cpp").write_text(PROGRAM)
    include = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_build.nvcc()))), "include")
    subprocess.run(["g++", "-std=c++17", "-O1", "-fsanitize=integer-divide-by-zero", "-fsanitize-undefined-trap-on-error",
                    "-I", _build.CSRC, "-I", include, str(d / "rule.cpp"), "-o", str(d / "rule")], check=True)

    def ask(rows):
        text = "\n".join(" ".join(str(int(x)) for x in r) for r in rows) + "\n"
        r = subprocess.run([str(d / "rule")], input=text, capture_output=True, text=True)
        assert r.returncode == 0, r.returncode
        return [int(x) for x in r.stdout.split()]

    return ask


def test_a_batch_of_no_requests_has_no_item_size(chunks):
    assert chunks([(0, 32, 8, 0, n, 152) for n in (1, 8191, 8192, 100001)]) == [0] * 4


def test_items_fit_the_planner_the_workspace_and_the_ctas(chunks):
    g = np.random.default_rng(5)
    rows = [(1, 32, 8, 0, 100001, 152), (4, 16, 2, 0, 100001, 152), (1, 8, 8, 0, 8191, 152), (1, 8, 1, 2, 100001, 152)]
    for _ in range(500):
        Hkv, G = int(g.integers(1, 9)), int(g.integers(1, 9))
        rows.append((g.integers(1, 700), G * Hkv, Hkv, g.integers(0, 64 // G), int(np.exp(g.uniform(8, 14))), 152))
        rows.append((g.integers(1, 12), G * Hkv, Hkv, g.integers(0, 16 // G), int(np.exp(g.uniform(9, 14))), 152))
    got = chunks(rows)
    assert got[:4] == [1344, 1344, 0, 0]  # 76 pieces a context; short contexts; 24 rows
    assert sum(1024 < c for c in got) > 10 and 1024 in got
    for (B, Hq, Hkv, k, L, nsm), c in zip(rows, got):
        assert c == 0 or (1024 <= c < 2048 and c % 64 == 0 and L >= 8192 and (k + 1) * (Hq // Hkv) <= 16)
        if c > 1024:
            assert B * Hkv * -(-L // c) <= 4 * nsm
        s = dict(B=int(B), Hq=Hq, Hkv=Hkv, D=128, k=int(k), max_sparse=8, max_len=int(L), num_slots=1 << 20, row_lo=0)
        assert P.pillar_attn_workspace_bytes(P.make_shape(verify_chunk=c, **s)) <= P.pillar_attn_workspace_bytes(P.make_shape(**s))


@pytest.mark.gpu
@pytest.mark.parametrize("max_len", [64, 8192, 1 << 20])
def test_a_call_with_no_requests(max_len):
    s, lib = P.make_shape(B=0, Hq=8, Hkv=2, D=64, k=0, row_lo=0, max_sparse=4, max_len=max_len, num_slots=1600), P.load()
    none = [None] * 6 + [4] + [None] * 7
    assert lib.pillar_attn_kv4(ctypes.byref(s), *none, None, 0, None) == 0
    assert lib.pillar_attn_run_kv4(ctypes.byref(s), *[None] * 6, 4, *[None] * 4, None, 0, None) == 0
    t = lambda *n, x=torch.int32: torch.zeros(n, dtype=x, device="cuda")  # noqa: E731
    ws = torch.full((P.pillar_attn_workspace_bytes(s),), 0xff, dtype=torch.uint8, device="cuda")
    pool, scales = t(100, 2, 16, 32, x=torch.uint8), t(100, 2, 16, 4, x=torch.uint8)
    P.pillar_attn_kv4(s, t(0, 8, 64, x=torch.bfloat16), pool, pool, scales, scales, t(0, 4), t(0), t(0), t(0, 2, 4), t(0, 2),
                      t(0, 8, 64, x=torch.bfloat16), None, t(1, 8, 1, x=torch.float32), ws)
    assert P.pillar_get_error(ws) == 0

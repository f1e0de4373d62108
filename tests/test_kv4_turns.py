"""How the 4-bit append and the reads deal a packed batch out to CTAs: the rule, and batches around its border."""
import subprocess

import pytest

import sparse_self_speculative_pillar_gb300 as P
from sparse_self_speculative_pillar_gb300 import _build

torch = pytest.importorskip("torch")

PROGRAM = r"""
#include <cstdio>
#include "pillar_rows.cuh"
int main() {
    int n, resident, nsm;
    while (std::scanf("%d %d %d", &n, &resident, &nsm) == 3) {
        const int rows = pillar::rows_of_turn(n, resident, nsm);
        std::printf("%d %u\n", rows, pillar::row_ctas(n, rows, resident, nsm));
    }
}
"""


def test_a_grid_is_never_more_ctas_than_are_resident(tmp_path):
    (tmp_path / "turns.cu").write_text(PROGRAM)
    subprocess.run([_build.nvcc(), *_build.ARCH, "-std=c++17", "-I", _build.CSRC, str(tmp_path / "turns.cu"), "-o",
                    str(tmp_path / "turns")], check=True)
    cases = [(n, res, nsm) for res in (4, 5) for nsm in (1, 132, 152)
             for n in sorted({1, 15, 16, 17, res * nsm - 1, res * nsm, res * nsm + 1, 6 * nsm, 12 * nsm, 16 * nsm, 16 * nsm + 1,
                              64 * nsm, 10 ** 6, 2 ** 31 - 1})]
    r = subprocess.run([str(tmp_path / "turns")], input="\n".join("%d %d %d" % c for c in cases), capture_output=True, text=True,
                       check=True)
    for (n, res, nsm), line in zip(cases, r.stdout.splitlines(), strict=True):
        rows, ctas = map(int, line.split())
        assert 1 <= ctas <= res * nsm and ctas <= n, (n, res, nsm)  # all of them run at once
        assert rows == (1 if n <= res * nsm else 16)                # a row each where that is enough CTAs


@pytest.mark.gpu
@pytest.mark.parametrize("n", [1, 607, 608, 609, 760, 761, 1216, 2432, 2433, 9729])
def test_one_call_does_what_calls_of_few_rows_do(n):
    """A row's codes depend on that row alone, and so does what is read."""
    g, Hkv, D = torch.Generator(device="cuda").manual_seed(n), 3, 64
    blocks = -(-n // 16) + 2
    s = P.make_shape(B=1, Hq=Hkv, Hkv=Hkv, D=D, k=0, row_lo=0, max_sparse=0, max_len=n, num_slots=blocks * 16)
    x, y = (torch.randn((n, Hkv, D), generator=g, device="cuda").bfloat16() for _ in "kv")
    table = torch.randperm(blocks, generator=g, device="cuda").int()[None, :].contiguous()
    i32 = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    new = lambda: [torch.zeros((blocks, Hkv, 16, w), dtype=torch.uint8, device="cuda")  # noqa: E731
                   for w in (D // 2, D // 2, D // 16, D // 16)]
    back = lambda: [torch.zeros_like(x) for _ in "kv"]  # noqa: E731
    one, few, got, want, flags = new(), new(), back(), back(), i32(0)
    P.pillar_kv4_append(s, x, y, i32(n), i32(0, n), table, *one, flags)
    P.pillar_kv4_read(s, *one, table, i32(0), i32(0, n), *got, flags)
    for a in range(0, n, 300):
        m = min(300, n - a)
        P.pillar_kv4_append(s, x[a:a + m], y[a:a + m], i32(a + m), i32(0, m), table, *few, flags)
        P.pillar_kv4_read(s, *one, table, i32(a), i32(0, m), *(w[a:a + m] for w in want), flags)
    codes, scale = (torch.randint(0, 0x7f, (blocks, Hkv, 16, D), generator=g, device="cuda", dtype=torch.uint8),
                    torch.rand((blocks, Hkv), generator=g, device="cuda"))
    got8, want8 = back(), back()
    P.pillar_kv8_read(s, codes, codes, scale, scale, table, i32(0), i32(0, n), *got8, flags)
    for a in range(0, n, 300):
        m = min(300, n - a)
        P.pillar_kv8_read(s, codes, codes, scale, scale, table, i32(a), i32(0, m), *(w[a:a + m] for w in want8), flags)
    assert flags.item() == 0
    for a, b in zip(one + got + got8, few + want + want8):
        assert torch.equal(a, b)
    assert torch.any(got[0] != 0)

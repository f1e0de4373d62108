"""A device wait that runs out, on the GPU.

With a wait bound of one microsecond -- far below the time the persistent
kernel's roles need to hand work to one another (every hand-off waits on a
global-memory round trip) -- some pipeline wait of every CTA gives up.  The
kernel must then record PILLAR_FLAG_TIMEOUT, let the copies and tensor-core
work already in flight finish (those drains keep their one-second bound),
free its tensor memory and return; the CUDA context stays usable, and the
next call on the same buffers with the default bound must be exact against
the oracle.  Nothing here faults, traps or hangs: every wait involved is
bounded."""
import math

import numpy as np
import pytest

import workloads as W

pytestmark = pytest.mark.gpu
torch = pytest.importorskip("torch")
import sparse_self_speculative_pillar_gb300 as P  # noqa: E402
from tests._gpu_common import Gpu, compare_attn, run_oracle  # noqa: E402


def test_short_wait_bound_reports_timeout_and_the_next_call_is_exact():
    w = W.generate(W.scaled("qwen3_8b", B=12, length_scale=0.05, seed_offset=9))
    g = Gpu(w, wait_timeout_us=1)
    g.attn()
    flags = g.attn_flags()
    assert flags & P.FLAG_TIMEOUT, f"device flags 0x{flags:x}: no wait ran out"
    assert flags & ~(P.FLAG_TIMEOUT) == 0, f"device flags 0x{flags:x}"
    # the same buffers, the default bound
    g.shape.wait_timeout_us = 0
    g.out.zero_()
    g.logits.fill_(math.nan)
    g.lse.fill_(math.nan)
    g.attn()
    assert g.attn_flags() == 0
    res = g.host()
    compare_attn(w, res, run_oracle(w))


def test_wait_bound_is_checked_on_the_host():
    w = W.generate(W.scaled("qwen3_8b", B=4, length_scale=0.02, seed_offset=10))
    g = Gpu(w)
    g.shape.wait_timeout_us = -5
    with pytest.raises(P.PillarError):
        g.attn()
    g.shape.wait_timeout_us = 50_000  # a 50 ms bound: ample for this step
    g.attn()
    assert g.attn_flags() == 0
    np.testing.assert_equal(np.isfinite(g.host()["out"]).all(), True)


def test_steps_whose_copies_are_all_issued_before_a_wait_runs_out():
    """Contexts of so few tiles that the loaders have issued everything when a wait of the other roles gives up: they still see
    their copies land before a CTA leaves its shared memory to the next one, here one of a whole step that follows on the stream
    at once."""
    w = W.generate(W.scaled("qwen3_8b", B=4, length_scale=0.02, seed_offset=11))
    g, h, want = Gpu(w), Gpu(w), Gpu(w)
    want.attn()
    assert want.attn_flags() == 0
    for _ in range(4):
        g.shape.wait_timeout_us = 1
        g.attn()
        h.attn()
        assert g.attn_flags() & ~P.FLAG_TIMEOUT == 0 and h.attn_flags() == 0
        for name in ("out", "logits", "lse"):
            assert torch.equal(getattr(h, name), getattr(want, name)), name
        h.out.zero_()
        h.logits.fill_(math.nan)
        h.lse.fill_(math.nan)
    g.shape.wait_timeout_us = 0
    g.attn()
    assert g.attn_flags() == 0
    compare_attn(w, g.host(), run_oracle(w))


def test_waits_that_run_out_anywhere_in_the_pipeline():
    """Bounds from one microsecond to more than the whole step takes: a warp goes on or gives up as one, and a whole step that
    follows at once is right."""
    w, v = W.generate(W.scaled("qwen3_8b", B=24, length_scale=0.2, seed_offset=12)), W.generate(W.scaled("qwen3_8b", B=6, length_scale=0.03, seed_offset=13))
    g, h, want = Gpu(w), Gpu(v), Gpu(v)
    want.attn()
    assert want.attn_flags() == 0
    for bound in (1, 2, 3, 4, 6, 9, 13, 20, 30, 50, 400):
        g.shape.wait_timeout_us = bound
        g.attn()
        h.attn()
        assert g.attn_flags() & ~P.FLAG_TIMEOUT == 0 and h.attn_flags() == 0, bound
        for name in ("out", "logits", "lse"):
            assert torch.equal(getattr(h, name), getattr(want, name)), (bound, name)
        h.out.zero_()

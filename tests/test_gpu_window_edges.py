"""GPU tests of what the attention over E4M3 caches and windows counts, clamps and makes of what is not finite, against the
plain 64-bit form.  Tolerances: tests/_parity.py."""
import numpy as np
import pytest
import torch

from _parity import check_attention
from _spec import cast
from _window import Blocks, attend
from paged_kv_cache_slot_gb300 import workloads as wl
from test_gpu_window import Call, _f64

pytestmark = pytest.mark.gpu

PATHS = [(False, 128), (True, 128), (False, 64), (True, 64)]


def _at_length(p, r, L):
    """Request r as if it had L cached positions (its window's last ones still there)."""
    return attend(wl.to_f32(p.q[r]).astype(np.float64), p.keys[r][:L], p.values[r][:L], L, True, p.window, p.sinks, None,
                  p.there[r][:L])


@pytest.mark.parametrize("fp8,d", PATHS)
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 9), (500, 9)])
def test_lengths_above_the_bound_are_clamped_and_counted_once(fp8, d, window, sinks):
    """Requests at, above and below the bound, and of a negative length (none): two errors, no more, and the longer ones'
    rows are those of requests of the bound's length."""
    p = Blocks([200, 201, 90, 333, 5], 2, 16, 4, d, 16, fp8=fp8)     # (all blocks are there)
    p.window, p.sinks = window, sinks
    c = Call(p, max_ctx=200)
    p.lens[4] = -3
    c.lens[4] = -3
    got = _f64(c.run())
    assert int(c.err) == 2
    for r, L in enumerate((200, 200, 90, 200)):
        check_attention(got[r], _at_length(p, r, L), "bf16", f"request {r}")
    assert (got[4] == 0).all()


@pytest.mark.parametrize("fp8,d", PATHS)
def test_bad_entries_are_counted_exactly(fp8, d):
    """An id past the cache in a block of first tokens, in the window's first block, between the two and in a block of a long
    request that columns share: once a KV head each, but for the one that nobody reads."""
    p = Blocks([3000, 700, 20000], 1, 16, 4, d, 16, fp8=fp8, window=600, sinks=20)
    for r, b, read in ((0, 1, True), (0, 150, True), (0, 100, False), (1, 6, True), (2, 1224, True)):
        p.table[r, b] = p.total + 7
        p.there[r][b * 16:(b + 1) * 16] = False
        assert ((b + 1) * 16 > p.lens[r] - 600 or b * 16 < 20) == read
    c = Call(p)
    got = _f64(c.run())
    assert int(c.err) == 4 * 4
    for r in range(3):
        check_attention(got[r], p.want(r), "bf16", f"request {r}")


@pytest.mark.parametrize("fp8,d", PATHS)
def test_queries_that_are_not_finite(fp8, d):
    """A query head with a NaN: its rows are NaN where they see a key and 0 where they see none, all others as ever."""
    p = Blocks([0, 1, 40, 600], 2, 8, 2, d, 16, fp8=fp8, window=100, sinks=3)
    want = [p.want(r) for r in range(4)]
    bad = cast(np.full(1, np.nan, np.float32), "bf16")[0]
    p.q[:, 0, 3, 5] = bad
    p.q[:, 1, 6, 0] = bad
    got = _f64(Call(p).run())
    for r in range(4):
        for t, h in ((0, 3), (1, 6)):
            sees = p.lens[r] - 2 + t >= 0
            assert np.isnan(got[r, t, h]).all() if sees else (got[r, t, h] == 0).all()
        keep = np.ones((2, 8), bool)
        keep[0, 3] = keep[1, 6] = False
        check_attention(got[r][keep], want[r][keep], "bf16", f"request {r}")


@pytest.mark.parametrize("d", [128, 64])
@pytest.mark.parametrize("e", [-60, -41, -40, 40, 41, 60])
def test_scales_of_values_at_the_ends_of_their_range(d, e):
    """V scales outside [2^-40, 2^40] count as the nearer end; all blocks of a request have them, or one of many does."""
    p = Blocks([300, 500], 1, 8, 2, d, 16, fp8=True, spread=0.0)
    clamped = 2.0 ** min(max(e, -40), 40)
    for r, blocks in ((0, range(19)), (1, [7])):
        for b in blocks:
            i = p.table[r, b]
            p.values[r][b * 16:(b + 1) * 16] *= clamped / p.vs[i][:, None]
            p.vs[i] = 2.0 ** e
    got = _f64(Call(p).run())
    for r in range(2):
        # outputs of a magnitude of about 1, for which the bars are made
        by = clamped if e > 0 or r == 0 else 1.0
        check_attention(got[r] / by, p.want(r) / by, "bf16", f"request {r}")


@pytest.mark.parametrize("fp8", [False, True])
def test_a_step_of_two_calls_on_one_workspace(fp8):
    """Two layers' calls, one behind the other on one stream, share a workspace and keep their results apart."""
    ps = [Blocks([3000, 33, 700], 1, 16, 4, 128, 16, fp8=fp8, seed=s, window=900, sinks=4) for s in range(2)]
    cs = [Call(p) for p in ps]
    cs[1].ws = cs[0].ws
    for _ in range(2):
        for c in cs:
            c.run()
    for p, c in zip(ps, cs):
        for r in range(3):
            check_attention(_f64(c.out)[r], p.want(r), "bf16", f"request {r}")

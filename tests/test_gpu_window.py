"""GPU tests of the attention over E4M3 caches with a scale a block and head, and
of windows whose first tokens stay visible, against the plain 64-bit form.

Tolerances: the bars of tests/_parity.py, which count the output's rounding and
that of the weights; over E4M3 caches the reference has the codes' own values, so
that the caches' rounding is on both sides."""
import numpy as np
import pytest
import torch

import oracle
from _parity import check_attention
from _spec import cast
from _window import Blocks, attend, build_step, write_blocks
from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
MODES = {True: bkv.BKV_MASK_CAUSAL, False: bkv.BKV_MASK_ALL}


def _d(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.uint16 and dtype is None:
        dtype = torch.bfloat16
    return (t.view(dtype) if dtype is not None else t).to(DEV)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


class Call:
    """A call's tensors on the GPU; the workspace holds NaN, so that a partial that nobody wrote would show."""

    def __init__(self, p, max_ctx=None):
        nr, t, hq, d = p.q.shape
        self.p, self.max_ctx = p, int(p.lens.max(initial=0)) if max_ctx is None else max_ctx
        self.q, self.k, self.v, self.table, self.lens = (_d(x) for x in (p.q, p.k, p.v, p.table, p.lens))
        self.scales = (_d(p.ks), _d(p.vs)) if p.fp8 else ()
        self.ws = bkv.alloc_window_workspace(nr, t, hq, p.k.shape[2], d, p.bs, self.max_ctx)
        self.ws.fill_(0xFF)
        self.out = torch.full_like(self.q, 9.0)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, causal=True, scale=0.0, stream=None, window=None, sinks=None, **kw):
        p = self.p
        w, s = p.window if window is None else window, p.sinks if sinks is None else sinks
        fn = bkv.bkv_paged_decode_fp8_blocks if p.fp8 else bkv.bkv_paged_decode_sink
        return fn(self.q, self.k, self.v, *self.scales, self.table, self.lens, self.max_ctx, self.out, self.ws,
                  sliding_window=w, num_sinks=s, softmax_scale=scale, mask_mode=MODES[causal], err_count=self.err,
                  stream=stream, **kw)


def _check(p, causal=True, scale=0.0, errors=0, rows=None):
    c = Call(p)
    got = _f64(c.run(causal, scale))
    assert int(c.err) == errors
    for r in range(len(p.lens)) if rows is None else rows:
        check_attention(got[r], p.want(r, causal, scale if scale > 0 else None), p.dtype, f"request {r}")
    return c


HEADS = [(32, 8), (4, 4), (8, 1), (15, 5), (7, 1), (24, 2)]


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv", HEADS)
@pytest.mark.parametrize("t", [1, 2, 5])
def test_full_attention(fp8, hq, hkv, t):
    """No window: lengths from one token, over block and tile borders, in every head layout."""
    lens = [max(t, n) for n in (1, 2, 15, 16, 17, 64, 100, 127, 128, 129, 300, 513, 1000)]
    _check(Blocks(lens, t, hq, hkv, 128, 16, fp8=fp8, seed=hq + t))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("bs", [8, 16, 32, 64, 128, 256, 24, 1])
@pytest.mark.parametrize("window,sinks", [(1, 0), (1, 1), (16, 4), (100, 4), (128, 64), (33, 130), (500, 7), (4000, 5)])
def test_window_and_sinks(fp8, bs, window, sinks):
    """Windows and first tokens that end inside and at the borders of blocks and tiles, overlap, meet, or leave blocks
    between them that are not there; requests shorter than both."""
    rng = np.random.default_rng(window)
    lens = [3, window, window + 3, sinks + window, sinks + window + 4, 129, 257, 640, 1000] + rng.integers(3, 1200, 4).tolist()
    lens = [max(3, n) for n in lens]
    _check(Blocks(lens, 3, 8, 2, 128, bs, fp8=fp8, seed=bs, window=window, sinks=sinks))


@pytest.mark.parametrize("dtype,fp8", [("bf16", False), ("f32", False), ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("d", [2, 18, 32, 64, 80, 100, 128, 192, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (70, 5)])
def test_types_and_head_dims(dtype, fp8, d, window, sinks):
    lens = [1, 2, 40, 64, 65, 200, 333]
    _check(Blocks(lens, 1, 6, 2, d, 16, dtype, fp8, seed=d, window=window, sinks=sinks))
    _check(Blocks([max(3, n) for n in lens], 3, 12, 3, d, 8, dtype, fp8, seed=d + 1, window=window, sinks=sinks))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window,sinks", [(0, 0), (50, 6)])
def test_masks_and_scales(fp8, causal, window, sinks):
    """Both mask modes, a softmax scale of the caller's, scales that are no powers of two, requests with fewer cached
    positions than query tokens (whose first tokens see nothing) and with none."""
    p = Blocks([0, 1, 3, 4, 5, 60, 200, 0], 4, 16, 4, 128, 16, fp8=fp8, window=window, sinks=sinks, pow2=False)
    c = _check(p, causal, scale=0.11)
    assert bool((c.out[0] == 0).all()) and bool((c.out[7] == 0).all())
    if causal:
        assert bool((c.out[1, :3] == 0).all()) and bool((c.out[2, :1] == 0).all())


@pytest.mark.parametrize("fp8,d", [(False, 128), (True, 128), (False, 64), (True, 64)])
@pytest.mark.parametrize("window", [300, 299, (1 << 31) - 1])
def test_windows_as_long_as_any_request(fp8, d, window):
    """A window that reaches every position is none: query tokens before the request's first position, whose window
    begins far below zero, see what the mask mode leaves."""
    _check(Blocks([1, 2, 8, 150, 300], 9, 4, 2, d, 16, fp8=fp8, window=window, sinks=0), causal=False)
    _check(Blocks([1, 2, 8, 150, 300], 9, 4, 2, d, 16, fp8=fp8, window=window, sinks=3))


@pytest.mark.parametrize("fp8", [False, True])
def test_null_entries_and_errors(fp8):
    """Null entries in the window and among the first tokens' blocks, whole requests of them; ids past the cache, tables
    too narrow, lengths above the bound: masked, and counted once a KV head (a length once)."""
    holes = [(0, 0), (1, 1), (1, 2), (2, 30), (3, 0), (3, 1), (3, 2), (3, 3)]
    p = Blocks([100, 90, 600, 64, 300], 1, 16, 4, 128, 16, fp8=fp8, window=150, sinks=20, holes=holes)
    c = _check(p)
    assert bool((c.out[3] == 0).all())
    p.table[4, 0] = p.total + 3
    p.table[2, 37] = 1 << 30
    p.there[4][:16] = False
    p.there[2][37 * 16:38 * 16] = False
    p.table[0, 3] = p.total
    p.there[0][48:64] = False
    p.table[2, 20] = p.total                                        # and one that nobody reads
    _check(p, errors=3 * 4)
    wide = p.table
    p.table = np.ascontiguousarray(wide[:, :20])                    # without the 10 blocks of request 2's window
    p.there[2][320:] = False
    _check(p, errors=(2 + 10) * 4)
    p.table = wide
    c = Call(p, max_ctx=200)
    c.run()
    assert int(c.err) >= 2


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hq,hkv,t", [(64, 4, 2), (40, 2, 7), (32, 1, 1), (8, 8, 40), (16, 4, 100)])
def test_many_query_rows(fp8, hq, hkv, t):
    """More query rows a KV head than one group holds."""
    lens = [t, t + 1, 130, 300, 777]
    _check(Blocks([max(t, n) for n in lens], t, hq, hkv, 128, 16, fp8=fp8, seed=t, window=90, sinks=5))
    _check(Blocks([max(t, n) for n in lens], t, hq, hkv, 128, 64, fp8=fp8, seed=t))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("hkv", [1, 3, 100, 160])
def test_kv_head_counts(fp8, hkv):
    """KV head counts that leave SMs over, and more of them than there are SMs."""
    _check(Blocks([1000, 3, 129, 700], 1, 2 * hkv, hkv, 128, 16, fp8=fp8, seed=hkv, window=300, sinks=9))


@pytest.mark.parametrize("fp8", [False, True])
def test_long_requests_beside_short_ones(fp8):
    """Streams that many columns share beside ones of a tile: 40000 positions, 1, and what is between."""
    _check(Blocks([40003, 1, 5, 128, 2000, 64, 9000], 1, 8, 2, 128, 64, fp8=fp8))
    _check(Blocks([40003, 1, 5, 128, 2000, 64, 9000], 1, 8, 2, 128, 64, fp8=fp8, window=20001, sinks=70))


@pytest.mark.parametrize("fp8", [False, True])
def test_more_requests_than_a_launch_takes(fp8):
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 60, 2500)
    lens[[0, 1023, 1024, 2047, 2048, 2499]] = 300
    p = Blocks(lens, 1, 4, 1, 128, 16, fp8=fp8, window=40, sinks=3)
    _check(p, rows=[0, 1023, 1024, 2047, 2048, 2499] + rng.integers(0, 2500, 80).tolist())


@pytest.mark.parametrize("fp8,d", [(False, 128), (True, 128), (False, 64), (True, 64)])
def test_many_short_requests_have_the_same_bits_in_every_run(fp8, d):
    rng = np.random.default_rng(4)
    lens = np.where(rng.random(900) < 0.8, rng.integers(4, 129, 900), rng.integers(129, 700, 900))
    p = Blocks(lens, 4, 16, 4, d, 16, fp8=fp8)
    c = _check(p, rows=rng.permutation(900)[:50])
    first = c.out.clone()
    for _ in range(10):
        c.out.fill_(3.0)
        c.run()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("t,bs", [(4, 16), (1, 16), (4, 64)])
def test_long_and_one_tile_requests_in_turn(fp8, t, bs):
    """Units of one tile before, between and behind units of many, whose tiles are then at different stages in the two
    softmax streams: every request's rows, and the same bits in every run."""
    rng = np.random.default_rng(t)
    lens = np.where(rng.random(160) < 0.5, rng.integers(t, 100, 160), rng.integers(600, 2600, 160))
    p = Blocks(lens, t, 32, 8, 128, bs, fp8=fp8, seed=t, window=2048, sinks=4)
    c = _check(p, rows=rng.permutation(160)[:60])
    first = c.out.clone()
    for _ in range(10):
        c.out.fill_(3.0)
        c.run()
        assert torch.equal(first, c.out)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("rising", [True, False])
def test_scores_that_rise_or_fall_along_the_cache(fp8, rising):
    """Scores from -60 to 60 in base e along a request, so that the softmax's reference moves again and again, or never
    behind the first tile."""
    p = Blocks([1500, 900, 130], 2, 8, 2, 128, 16, fp8=fp8)
    for r in range(3):
        L = int(p.lens[r])
        u = np.zeros(128, np.float32)
        u[:8] = 1.0
        p.q[r] = cast(np.broadcast_to(u, p.q[r].shape).copy(), "bf16")
        along = np.linspace(-1, 1, L) * (1 if rising else -1) * 60 * 128 ** 0.5 / 8
        for pos in range(L):
            b, i = p.table[r, pos // 16], pos % 16
            row = np.zeros((2, 128), np.float32)
            row[:, :8] = along[pos]
            if fp8:
                if i == 0:
                    p.ks[b] = 0.25
                p.k[b, i] = oracle.e4m3_encode(row / np.float32(0.25))
                p.keys[r][pos] = oracle.e4m3_decode(p.k[b, i]) * 0.25
            else:
                p.k[b, i] = cast(row, "bf16")
                p.keys[r][pos] = wl.to_f32(p.k[b, i])
    _check(p)


@pytest.mark.parametrize("fp8,d", [(False, 128), (True, 128), (False, 64), (True, 64)])
@pytest.mark.parametrize("bad", [np.nan, np.inf, -np.inf])
def test_values_that_are_not_finite_where_a_token_does_not_see_them(fp8, d, bad):
    """Keys and values of NaN and infinity in the caches at positions that a token does not see: those of later tokens of
    its step, before its window beside its first tokens in their own blocks, behind the request's end in its last block.
    The tokens that see them have NaN or their value, the others what the plain form says."""
    if fp8 and not np.isnan(bad):
        pytest.skip("E4M3 has no infinities")
    t, L = 3, 300
    p = Blocks([L, L, 70], t, 8, 2, d, 16, fp8=fp8, window=100, sinks=5)
    want = [p.want(r) for r in range(3)]
    put = (lambda c, i, j: c.__setitem__((i, j), 0x7F)) if fp8 else (
        lambda c, i, j: c.__setitem__((i, j), cast(np.full(c.shape[2:], bad, np.float32), "bf16")))
    seen = {}
    # request 0: the last token's value and key; a row before every window in a block that the window begins in; the
    # sinks' block behind the sinks; what the first token's window alone holds
    for r, pos, rows in ((0, L - 1, [2]), (0, 196, []), (0, 7, []), (1, L - t - 100 + 1, [0])):
        i, j = p.table[r, pos // 16], pos % 16
        put(p.v, i, j)
        if np.isnan(bad):
            put(p.k, i, j)
        for x in rows:
            seen.setdefault(r, set()).add(x)
    got = _f64(Call(p).run())
    for r in range(3):
        for x in range(t):
            if x in seen.get(r, ()):
                assert not np.isfinite(got[r, x]).any() if np.isnan(bad) else not np.isfinite(got[r, x]).all()
            else:
                check_attention(got[r, x], want[r][x], "bf16", f"request {r} token {x}")


def test_infinite_scores():
    """bf16 keys of infinity: a score of -inf weighs nothing, one of +inf makes the row NaN."""
    for d in (128, 64):
        p = Blocks([200], 1, 4, 1, d, 16, window=50, sinks=4)
        p.q[:] = cast(np.ones(p.q.shape, np.float32), "bf16")
        want_there = p.there[0].copy()
        i, j = p.table[0, 180 // 16], 180 % 16
        row = np.zeros(p.k.shape[2:], np.float32)
        row[:] = -1e38
        row[0, 0] = -np.inf
        p.k[i, j] = cast(row, "bf16")
        p.there[0][180] = False
        check_attention(_f64(Call(p).run())[0], p.want(0), "bf16")
        p.there[0][:] = want_there
        p.k[i, j] = cast(-row, "bf16")
        assert np.isnan(_f64(Call(p).run())).all()


def test_scales_far_apart():
    """Blocks whose values lie a factor of 2^40 apart, and first tokens with large scores and small values."""
    for d in (128, 64):
        p = Blocks([1000], 1, 8, 2, d, 16, fp8=True, spread=0.0)
        rng = np.random.default_rng(1)
        for b in range(63):
            f = 2.0 ** int(rng.integers(-20, 21))
            p.vs[p.table[0, b]] *= f
            p.values[0][b * 16:(b + 1) * 16] *= f
        got = _f64(Call(p).run())[0]
        check_attention(got, p.want(0), "bf16")
        p = Blocks([1000], 1, 8, 2, d, 16, fp8=True)
        i = p.table[0, 0]
        p.ks[i] *= 8
        p.keys[0][:16] *= 8
        p.vs[i] *= 2.0 ** -12
        p.values[0][:16] *= 2.0 ** -12
        check_attention(_f64(Call(p).run())[0], p.want(0), "bf16")


def test_sinks_of_zero_are_the_window_alone():
    """num_sinks 0 gives bkv_paged_decode_swa's result up to both kernels' rounding; window 0 ignores num_sinks."""
    p = Blocks([500, 3, 90, 1000], 2, 16, 4, 128, 32, window=130)
    c = Call(p)
    a = _f64(c.run())
    ws = bkv.alloc_workspace(4, 2, 16, 4, 128, 32, 1000)
    b = torch.full_like(c.q, 3.0)
    bkv.bkv_paged_decode_swa(c.q, c.k, c.v, c.table, c.lens, 1000, b, ws, 130)
    # each of the two is within half a bar of the exact row
    check_attention(a, _f64(b), "bf16")
    full = Blocks([500, 3, 90, 1000], 2, 16, 4, 128, 32)
    c = Call(full)
    x = c.run(window=0, sinks=0).clone()
    assert torch.equal(x, c.run(window=0, sinks=77))


@pytest.mark.parametrize("fp8", [False, True])
def test_strided_tables_streams_and_views(fp8):
    """A table that is a view of a wider one, inputs made on another stream that the call is put on, outputs that are
    views at 16-byte boundaries."""
    p = Blocks([100, 900, 33], 1, 8, 2, 128, 16, fp8=fp8, window=200, sinks=17)
    c = Call(p)
    wide = torch.full((3, c.table.shape[1] + 5), 1 << 29, dtype=torch.int32, device=DEV)
    wide[:, :c.table.shape[1]] = c.table
    c.table = wide[:, :c.table.shape[1]]
    room = torch.full((c.out.numel() + 64,), 5.0, dtype=c.out.dtype, device=DEV)
    c.out = room[8:8 + c.out.numel()].view(c.out.shape)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        torch.cuda._sleep(2_000_000)
        c.q = c.q.clone()
        c.run(stream=st)
    st.synchronize()
    got = _f64(c.out)
    for r in range(3):
        check_attention(got[r], p.want(r), "bf16")
    assert bool((room[:8] == 5).all()) and bool((room[8 + c.out.numel():] == 5).all())


@pytest.mark.parametrize("fp8", [False, True])
def test_two_graphs_replayed_at_once(fp8):
    """Two captured calls with a workspace each, replayed on two streams on new lengths and queries."""
    sets = []
    for seed in range(2):
        p = Blocks([600, 900, 33, 1], 2, 16, 4, 128, 16, fp8=fp8, seed=seed, window=250, sinks=17)
        c = Call(p)
        c.run()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run()
        sets.append((p, c, g))
    rng = np.random.default_rng(7)
    for turn in range(3):
        for p, c, _ in sets:
            # shorter requests whose windows and first blocks are all there: within the last 250 of the longest only
            p.lens = np.array([600 - turn, 900 - turn, 33 - 5 * turn, 2], np.int32)
            p.q = cast(rng.standard_normal(p.q.shape).astype(np.float32), "bf16")
            c.lens.copy_(_d(p.lens))
            c.q.copy_(_d(p.q))
        torch.cuda.synchronize()
        for st, (_, _, g) in zip((torch.cuda.Stream(), torch.cuda.Stream()), sets):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for p, c, _ in sets:
            for r in (0, 1, 2):
                check_attention(_f64(c.out)[r], p.want(r), "bf16")


def test_a_cache_of_more_than_2_to_the_31_elements():
    """Blocks near the end of caches of 2^31 codes and above: offsets are 64 bits wide."""
    for d, total in ((128, 17_000), (64, 34_000)):
        bs, hkv = 128, 8
        k = torch.zeros((total, bs, hkv, d), dtype=torch.uint8, device=DEV)
        v = torch.zeros_like(k)
        assert k.numel() > 2 ** 31
        ks, vs = (torch.ones((total, hkv), device=DEV) for _ in range(2))
        rng = np.random.default_rng(0)
        new = [_d(rng.standard_normal((300, hkv, d)).astype(np.float32)) for _ in range(2)]
        table = torch.tensor([[total - 1, total - 2, total - 3]], dtype=torch.int32, device=DEV)
        qsl, ctx = (torch.tensor(x, dtype=torch.int32, device=DEV) for x in ([0, 300], [300]))
        bkv.bkv_cache_write_fp8_blocks(*new, qsl, ctx, table, k, v, ks, vs)
        q = _d(cast(rng.standard_normal((1, 1, 16, d)).astype(np.float32), "bf16"))
        out = torch.zeros_like(q)
        ws = bkv.alloc_window_workspace(1, 1, 16, hkv, d, bs, 300)
        bkv.bkv_paged_decode_fp8_blocks(q, k, v, ks, vs, table, ctx, 300, out, ws)
        rows = table[0].long()
        keys, values = ((oracle.e4m3_decode(c[rows].cpu().numpy()) * s[rows].cpu().numpy()[:, None, :, None])
                        .reshape(-1, hkv, d)[:300] for c, s in ((k, ks), (v, vs)))
        check_attention(_f64(out)[0], attend(_f64(q)[0], keys, values, 300), "bf16")
        assert int((k[:total - 3] != 0).sum()) == 0
        del k, v


@pytest.mark.parametrize("fp8", [True, False])
def test_steps_of_a_server(fp8):
    """Prompts, then decode steps, through tables built on the GPU, the write and the attention in order, against the
    plain forms: requests of several lengths, a request that ends and one that takes its row and its blocks."""
    hq, hkv, d, bs, rows, cols, window, sinks = 8, 2, 128, 16, 5, 40, 60, 5
    rng = np.random.default_rng(11)
    total = 1 + rows * cols
    free = rng.permutation(np.arange(1, total)).astype(np.int32)
    shape = (total, bs, hkv, d)
    table = torch.full((rows, cols), -1, dtype=torch.int32, device=DEV)
    if fp8:
        caches = [torch.full(shape, 0x7F, dtype=torch.uint8, device=DEV) for _ in range(2)]
        scales = [torch.zeros((total, hkv), device=DEV) for _ in range(2)]
    else:
        caches = [torch.full(shape, float("nan"), dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        scales = []
    want_c = [t.cpu().numpy() if fp8 else t.view(torch.uint16).cpu().numpy() for t in caches]
    want_s = [t.cpu().numpy() for t in scales]
    want_table = table.cpu().numpy()
    cached = np.zeros(rows, np.int32)
    left, err = free, torch.zeros(1, dtype=torch.int32, device=DEV)
    steps = [[70, 0, 33, 1, 200]] + [[1, 0, 1, 1, 1]] * 3 + [[1, 90, 1, 20, 1]] + [[1, 1, 1, 1, 1]] * 14 + [[3, 3, 3, 3, 3]] * 2
    for i, new in enumerate(steps):
        new = np.array(new, np.int32)
        if i == 8:                                                  # request 4 ends; its row begins anew
            back = want_table[4][want_table[4] > 0]
            left = np.concatenate([left, back]).astype(np.int32)
            cached[4], new[4] = 0, 50
        n = int(new.sum()) + 3
        ctx, qsl, req = (torch.zeros(x, dtype=torch.int32, device=DEV) for x in (rows, rows + 1, n))
        pos, slots = (torch.zeros(n, dtype=torch.int64, device=DEV) for _ in range(2))
        used = torch.zeros(1, dtype=torch.int32, device=DEV)
        bkv.bkv_build_step(_d(cached), _d(new), _d(left), bs, table, ctx, qsl, req, pos, slots, used, err_count=err)
        m = n - 3
        x = rng.standard_normal((2, n, hkv, d)).astype(np.float32) * np.float32(1 + i / 8)
        kv = [_d(cast(y, "bf16")) for y in x]
        if fp8:
            bkv.bkv_cache_write_fp8_blocks(kv[0], kv[1], qsl, ctx, table, *caches, *scales, err_count=err)
        else:
            bkv.bkv_cache_write(kv[0], kv[1], slots, *caches, err_count=err)
        w = build_step(cached, new, left, bs, want_table, n)
        want_table, left = w[0], left[w[6]:]
        assert int(used) == w[6] and w[7] == 0
        cached = w[1]
        host = [cast(y, "bf16") for y in x]
        if fp8:
            write_blocks(host[0], host[1], w[2], cached, want_table, bs, *want_c, *want_s)
        else:
            for y, c in zip(host, want_c):
                for j in range(m):
                    c[w[5][j] // bs, w[5][j] % bs] = y[j]
        t = int(new.min())
        if t < 1 or (new != t).any():
            continue
        q = cast(rng.standard_normal((rows, t, hq, d)).astype(np.float32), "bf16")
        top = int(cached.max())
        out = torch.full((rows, t, hq, d), 8.0, dtype=torch.bfloat16, device=DEV)
        ws = bkv.alloc_window_workspace(rows, t, hq, hkv, d, bs, top)
        if fp8:
            bkv.bkv_paged_decode_fp8_blocks(_d(q), *caches, *scales, table, ctx, top, out, ws, window, sinks, err_count=err)
        else:
            bkv.bkv_paged_decode_sink(_d(q), *caches, table, ctx, top, out, ws, window, sinks, err_count=err)
        got, q64 = _f64(out), _f64(_d(q))
        for r in range(rows):
            L = int(cached[r])
            b = want_table[r][:-(-L // bs)]
            if fp8:
                keys, values = ((oracle.e4m3_decode(c[b]) * s[b][:, None, :, None]).reshape(-1, hkv, d)[:L]
                                for c, s in zip(want_c, want_s))
            else:
                keys, values = (_f64(_d(c[b])).reshape(-1, hkv, d)[:L] for c in want_c)
            check_attention(got[r], attend(q64[r], keys, values, L, True, window, sinks), "bf16", f"step {i} request {r}")
    torch.cuda.synchronize()
    assert int(err) == 0
    assert np.array_equal(table.cpu().numpy(), want_table)
    for g, w in zip(caches, want_c):
        assert np.array_equal((g if fp8 else g.view(torch.uint16)).cpu().numpy(), w)
    for g, w in zip(scales, want_s):
        assert np.array_equal(g.cpu().numpy(), w)

"""GPU tests of step building and of the block-scaled E4M3 write, against plain
forms on the host.

Everything here is exact: tables, lists, slots and counts are whole numbers;
scales are powers of two, so that quotients by them are exact and a code is one
rounding of an exact value on both sides."""
import numpy as np
import pytest
import torch

import oracle
from _spec import cast
from _window import build_step, write_blocks
from paged_kv_cache_slot_gb300 import bkv

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _d(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.uint16 and dtype is None:
        dtype = torch.bfloat16
    return (t.view(dtype) if dtype is not None else t).to(DEV)


class Step:
    """Outputs of a step of ``rows`` requests, filled with rubbish, in a table of row stride cols + extra."""

    def __init__(self, rows, cols, tokens, extra=0):
        self.wide = torch.full((max(rows, 1), cols + extra), 77, dtype=torch.int32, device=DEV)
        self.table = self.wide[:rows, :cols]
        self.ctx = torch.full((rows,), -5, dtype=torch.int32, device=DEV)
        self.qsl = torch.full((rows + 1,), -5, dtype=torch.int32, device=DEV)
        self.req = torch.full((tokens,), -5, dtype=torch.int32, device=DEV)
        self.pos = torch.full((tokens,), -5, dtype=torch.int64, device=DEV)
        self.slots = torch.full((tokens,), -5, dtype=torch.int64, device=DEV)
        self.used = torch.full((1,), -5, dtype=torch.int32, device=DEV)
        self.err = torch.zeros(1, dtype=torch.int32, device=DEV)

    def run(self, cached, new, free, bs, stream=None):
        return bkv.bkv_build_step(cached, new, free, bs, self.table, self.ctx, self.qsl, self.req, self.pos, self.slots,
                                  self.used, err_count=self.err, stream=stream)


def _check_step(cached, new, free, bs, cols, tokens, extra=0, seed=0):
    rng = np.random.default_rng(seed)
    rows = len(cached)
    table = rng.integers(1, 1 << 20, (rows, cols)).astype(np.int32)
    s = Step(rows, cols, tokens, extra)
    s.table.copy_(_d(table))
    s.run(_d(cached.astype(np.int32)), _d(new.astype(np.int32)), _d(free.astype(np.int32)), bs)
    torch.cuda.synchronize()
    want = build_step(cached, new, free, bs, table, tokens)
    got = (s.table, s.ctx, s.qsl, s.req, s.pos, s.slots)
    for g, w, name in zip(got, want, ("table", "ctx", "qsl", "req", "pos", "slots")):
        assert np.array_equal(g.cpu().numpy(), w), name
    assert int(s.used) == want[6] and int(s.err) == want[7]
    if extra:
        assert bool((s.wide[:rows, cols:] == 77).all())            # behind the columns nothing is written
    return s


@pytest.mark.parametrize("rows,bs,cols,hi,extra", [
    (1, 16, 7, 40, 0), (3, 16, 9, 50, 3), (31, 64, 5, 200, 0), (32, 1, 33, 16, 1), (33, 7, 30, 100, 2), (320, 16, 514, 4000, 0),
    (511, 16, 12, 90, 0), (513, 32, 8, 100, 4), (1500, 16, 21, 150, 3), (20000, 16, 6, 40, 2)])
def test_build_step(rows, bs, cols, hi, extra):
    """Requests from none to several blocks, new tokens from none to some blocks, padded rows among them, tables whose
    rows begin at any alignment."""
    rng = np.random.default_rng(rows)
    cached = rng.integers(0, hi + 1, rows)
    new = np.where(rng.random(rows) < 0.6, 1, rng.integers(0, 3 * bs, rows))
    cached[rng.random(rows) < 0.1] = 0
    new[rng.random(rows) < 0.2] = 0
    new = np.minimum(new, np.maximum(cols * bs - cached, 0))
    cached = np.minimum(cached, cols * bs)
    free = rng.permutation(1 << 20)[:int((new // bs + 1).sum()) + 5] + 1
    _check_step(cached, new, free, bs, cols, int(new.sum()) + 13, extra)


def test_build_step_of_a_chunk_and_of_nothing():
    one = np.array([5])
    _check_step(one, np.array([3000]), np.arange(9, 400), 16, 190, 3100)
    _check_step(np.array([0, 0, 0]), np.array([0, 0, 0]), np.arange(0), 16, 4, 5)
    _check_step(np.array([0]), np.array([0]), np.arange(0), 16, 4, 0)
    _check_step(np.zeros(0, np.int64), np.zeros(0, np.int64), np.arange(3), 16, 4, 6)
    _check_step(one, np.array([1]), np.arange(3), 16, 0, 2)          # a table without columns
    _check_step(np.array([1 << 20]), np.array([2]), np.arange(1, 9), 1, 1 << 21, 2)


def test_build_step_errors():
    """Free lists that run out, tables that are too narrow, lists that are too short, lengths that are none."""
    rng = np.random.default_rng(1)
    cached, new = rng.integers(0, 60, 40), rng.integers(0, 40, 40)
    for left in (0, 1, 17, 40):
        _check_step(cached, new, np.arange(1, left + 1), 16, 9, int(new.sum()) + 4)
    _check_step(cached, new, np.arange(1, 200), 16, 3, int(new.sum()) + 4)
    for tokens in (0, 1, 100, int(new.sum()) - 1):
        _check_step(cached, new, np.arange(1, 200), 16, 9, tokens)
    odd = np.array([3, -4, 2 ** 31 - 3, 2 ** 31 - 1, 5])
    _check_step(odd, np.array([-1, 20, 7, 0, 4]), np.arange(1, 50), 16, 6, 60)
    _check_step(np.array([2 ** 31 - 2, 3, -2 ** 31]), np.array([2 ** 31 - 1, 9, -2 ** 31]), np.arange(1, 50), 64, 6, 60)


def test_build_step_again_and_in_graphs():
    """The call repeated on its own outputs changes nothing; two captured graphs replay beside one another on new lengths."""
    rng = np.random.default_rng(2)
    sets = []
    for k in range(2):
        cached, new = rng.integers(0, 90, 70), rng.integers(0, 20, 70)
        free = np.arange(500, 900)
        s = _check_step(cached, new, free, 16, 9, 900, seed=k)
        ins = [_d(x.astype(np.int32)) for x in (cached, new, free)]
        before = [t.clone() for t in (s.table, s.qsl, s.req, s.pos, s.slots)]
        s.run(*ins, 16)
        assert all(torch.equal(a, b) for a, b in zip(before, (s.table, s.qsl, s.req, s.pos, s.slots)))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            s.run(*ins, 16)
        sets.append((s, ins, g, free))
    for turn in range(3):
        want = []
        for s, ins, g, free in sets:
            cached, new = rng.integers(0, 90, 70), rng.integers(0, 20, 70)
            table = rng.integers(1, 1 << 20, (70, 9)).astype(np.int32)
            ins[0].copy_(_d(cached.astype(np.int32)))
            ins[1].copy_(_d(new.astype(np.int32)))
            s.table.copy_(_d(table))
            want.append(build_step(cached, new, free, 16, table, 900))
        torch.cuda.synchronize()
        for st, (s, ins, g, free) in zip((torch.cuda.Stream(), torch.cuda.Stream()), sets):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        for (s, _, _, _), w in zip(sets, want):
            for got, x in zip((s.table, s.ctx, s.qsl, s.req, s.pos, s.slots), w):
                assert np.array_equal(got.cpu().numpy(), x)


# ---------------------------------------------------------------------------
# The block-scaled write
# ---------------------------------------------------------------------------
class Write:
    """A step's rows in a fused projection, tables, caches that hold codes and scales."""

    def __init__(self, prior, new, hkv, d, bs, dtype="bf16", seed=0, extra=8, cols_less=0):
        rng = np.random.default_rng(seed)
        prior, new = np.array(prior), np.array(new)
        self.ctx = (prior + new).astype(np.int32)
        self.qsl = np.concatenate([[0], new.cumsum()]).astype(np.int32)
        need = -(-self.ctx // bs)
        self.total = 3 + int(need.sum())
        ids = rng.permutation(np.arange(1, self.total))
        cols = max(int(need.max(initial=0)) + 1 - cols_less, 1)
        self.table = np.full((len(prior), cols), -1, np.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n][:cols]
            at += n
        n, row = int(new.sum()), hkv * d
        x = rng.standard_normal((n, 2 * row + extra)).astype(np.float32)
        x *= np.exp2(rng.uniform(-6, 6, (n, 1))).astype(np.float32)
        self.proj = cast(x, dtype)
        self.hkv, self.d, self.bs, self.row = hkv, d, bs, row
        self.kc, self.vc = (rng.integers(0, 0x7F, (self.total, bs, hkv, d)).astype(np.uint8) for _ in range(2))
        self.ks, self.vs = (np.exp2(rng.integers(-11, 1, (self.total, hkv))).astype(np.float32) for _ in range(2))

    def rows(self):
        n = len(self.proj)
        return (self.proj[:, :self.row].reshape(n, self.hkv, self.d),
                self.proj[:, self.row:2 * self.row].reshape(n, self.hkv, self.d))

    def run(self, times=1):
        p = _d(self.proj)
        n, s = p.shape[0], p.stride(0)
        k = p.as_strided((n, self.hkv, self.d), (s, self.d, 1))
        v = p.as_strided((n, self.hkv, self.d), (s, self.d, 1), self.row)
        err = torch.zeros(1, dtype=torch.int32, device=DEV)
        got = [_d(x) for x in (self.kc, self.vc, self.ks, self.vs)]
        for _ in range(times):
            bkv.bkv_cache_write_fp8_blocks(k, v, _d(self.qsl), _d(self.ctx), _d(self.table), *got, err_count=err)
        torch.cuda.synchronize()
        return [g.cpu().numpy() for g in got], int(err)

    def check(self):
        got, err = self.run()
        want = [x.copy() for x in (self.kc, self.vc, self.ks, self.vs)]
        k, v = self.rows()
        werr = write_blocks(k, v, self.qsl, self.ctx, self.table, self.bs, *want)
        assert err == werr
        for g, w, name in zip(got, want, ("k_cache", "v_cache", "k_scales", "v_scales")):
            assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5])
        return got


@pytest.mark.parametrize("hkv,d,bs,dtype", [
    (8, 128, 16, "bf16"), (2, 64, 32, "f32"), (5, 128, 64, "bf16"), (1, 256, 64, "bf16"), (3, 256, 128, "f32"),
    (2, 80, 16, "bf16"), (3, 20, 24, "f32"), (1, 2, 1, "bf16"), (2, 7, 5, "bf16"), (4, 128, 256, "bf16")])
@pytest.mark.parametrize("kind", ["decode", "mixed"])
def test_write(hkv, d, bs, dtype, kind):
    """Single tokens at every place of a block, and chunks that begin and end inside blocks, over one or several."""
    rng = np.random.default_rng(d * bs)
    if kind == "decode":
        prior = np.concatenate([np.arange(min(bs + 2, 40)), rng.integers(0, 4 * bs + 1, 20)])
        new = np.ones_like(prior)
    else:
        prior = rng.integers(0, 3 * bs + 1, 45)
        new = rng.integers(0, 3 * bs + 2, 45)
        new[rng.random(45) < 0.2] = 0
    for seed, extra in ((0, 8), (1, 3)):                            # rows at aligned and at odd strides
        Write(prior, new, hkv, d, bs, dtype, seed, extra).check()


def test_write_one_request_and_none():
    Write([0], [1], 8, 128, 16).check()
    Write([0], [700], 8, 128, 64).check()
    Write([5], [0], 8, 128, 64).check()
    Write([0, 0, 3], [0, 0, 0], 2, 64, 16).check()


def test_write_thousands_of_requests():
    rng = np.random.default_rng(3)
    new = rng.integers(0, 3, 3000)
    Write(rng.integers(0, 20, 3000), new, 2, 64, 16).check()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_write_edge_values(dtype):
    """Rows of zeros, of the border 448 x 2^e itself and just above it, subnormal and huge values, infinities and NaN."""
    w = Write([3, 0, 15, 16, 2, 7], [2, 16, 2, 1, 1, 9], 2, 64, 16, dtype)
    x = np.zeros((len(w.proj), w.proj.shape[1]), np.float32)
    rng = np.random.default_rng(0)
    x[:] = rng.standard_normal(x.shape)
    x[0] = 0.0
    x[1, :64] = 0.0
    x[2] = 7.0                                                      # 448 / 64
    x[3] = np.nextafter(np.float32(7.0), np.float32(8.0)) if dtype == "f32" else 7.03125
    x[4] *= 1e-38
    x[5] *= 1e30
    x[18, 3] = np.inf
    x[18, 70] = -np.inf
    x[19, 5] = np.nan
    x[20] = np.nan
    x[21] = np.inf
    w.proj = cast(x, dtype)
    got = w.check()
    assert np.isfinite(got[2]).all() and (got[2] > 0).all()


def test_write_scales_that_are_none():
    """Scales of 0, NaN, infinity or below 0 count as absent: the earlier rows stay as they are."""
    w = Write([3, 5, 7, 9, 20], [1, 1, 1, 1, 2], 1, 64, 16)
    for r, bad in enumerate((0.0, np.nan, np.inf, -1.0)):
        w.ks[w.table[r, 0]] = bad
    before = w.kc.copy()
    got = w.check()
    for r, p in enumerate((3, 5, 7, 9)):
        assert np.array_equal(got[0][w.table[r, 0], :p], before[w.table[r, 0], :p])


def test_write_errors():
    """Blocks past the table or the cache, null entries, more new tokens than the request is long."""
    w = Write([10, 3, 40, 0, 17], [30, 4, 9, 20, 1], 2, 64, 16, cols_less=2)
    w.check()
    w = Write([10, 3, 40, 0, 17], [30, 4, 9, 20, 1], 2, 64, 16)
    w.table[0, 1] = w.total + 4
    w.table[3, 0] = 0
    w.table[4, 1] = -1
    w.ctx[1] = 2
    _, err = w.run()
    w.check()
    assert err == 2


def test_write_twice_is_once():
    """A step written again finds the scales it made: nothing changes."""
    w = Write([3, 0, 30, 100, 17], [5, 40, 1, 64, 1], 4, 128, 32)
    once, _ = w.run()
    twice, _ = w.run(times=3)
    assert all(np.array_equal(a, b) for a, b in zip(once, twice))


def test_write_grows_step_by_step():
    """Tokens one at a time, ever larger and then small, against the plain form step by step: the scale grows, and what
    the block holds stays within half a step of E4M3 per growth of the values written."""
    hkv, d, bs, n = 2, 64, 16, 40
    rng = np.random.default_rng(5)
    x = (rng.standard_normal((n, 2, hkv, d)) * np.exp2(np.minimum(np.arange(n), 25) / 3)[:, None, None, None]).astype(np.float32)
    table = np.array([[2, 1, 3]], np.int32)
    caches = [torch.zeros((4, bs, hkv, d), dtype=torch.uint8, device=DEV) for _ in range(2)]
    scales = [torch.zeros((4, hkv), device=DEV) for _ in range(2)]
    want = [c.cpu().numpy() for c in caches + scales]
    for i in range(n):
        rows = [_d(x[i:i + 1, j]) for j in range(2)]
        bkv.bkv_cache_write_fp8_blocks(*rows, _d(np.array([0, 1], np.int32)), _d(np.array([i + 1], np.int32)), _d(table),
                                       *caches, *scales)
        write_blocks(x[i:i + 1, 0], x[i:i + 1, 1], np.array([0, 1]), np.array([i + 1]), table, bs, *want)
    got = [t.cpu().numpy() for t in caches + scales]
    assert all(np.array_equal(g, w) for g, w in zip(got, want))
    for j in range(2):
        held = oracle.e4m3_decode(got[j][table[0]]).reshape(-1, hkv, d)[:n] * got[2 + j][table[0]].repeat(bs, 0)[:n, :, None]
        # a value is rounded once, to 2^-4 of itself; a growth of the scale rounds it again only below 2^-6 of the scale,
        # by at most 2^-10 of the new one, and the growths' scales double, so that their sum is below 2^-9 of the last
        step = got[2 + j][table[0]].repeat(bs, 0)[:n, :, None]
        assert (np.abs(held - x[:, j]) <= np.abs(x[:, j]) * 2.0 ** -4 + step * 2.0 ** -9).all()


def test_write_in_a_graph():
    """A captured write replayed on new rows and lengths."""
    rng = np.random.default_rng(8)
    hkv, d, bs = 2, 128, 16
    w = Write([20] * 6, [5] * 6, hkv, d, bs)
    ins = [_d(x) for x in (w.proj, w.qsl, w.ctx, w.table, w.kc, w.vc, w.ks, w.vs)]
    p, qsl, ctx, table, kc, vc, ks, vs = ins
    s = p.stride(0)
    k = p.as_strided((30, hkv, d), (s, d, 1))
    v = p.as_strided((30, hkv, d), (s, d, 1), w.row)

    def call():
        bkv.bkv_cache_write_fp8_blocks(k, v, qsl, ctx, table, kc, vc, ks, vs)

    call()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        call()
    for turn in range(3):
        new = rng.multinomial(rng.integers(1, 31), [1 / 6] * 6)
        w.qsl = np.concatenate([[0], new.cumsum()]).astype(np.int32)
        w.ctx = (new + rng.integers(0, 10, 6)).astype(np.int32)
        w.proj = cast(rng.standard_normal(w.proj.shape).astype(np.float32) * 4.0 ** turn, "bf16")
        for t, x in zip(ins, (w.proj, w.qsl, w.ctx, w.table, w.kc, w.vc, w.ks, w.vs)):
            t.copy_(_d(x))
        g.replay()
        torch.cuda.synchronize()
        want = [x.copy() for x in (w.kc, w.vc, w.ks, w.vs)]
        write_blocks(*w.rows(), w.qsl, w.ctx, w.table, bs, *want)
        for t, x in zip((kc, vc, ks, vs), want):
            assert np.array_equal(t.cpu().numpy(), x)

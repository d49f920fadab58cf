"""GPU tests of the speculative step at its edges: infinite keys, heads turned in
place, batches of short contexts, the smallest random numbers.

Tolerances as in tests/test_gpu_spec.py: attention by tests/_parity.py; norm and
rotation the output's rounding plus 2e-6 of the row's largest value; tokens,
paths and counts equal."""
import itertools
from fractions import Fraction

import numpy as np
import pytest
import torch

import oracle
from _parity import check_attention
from _spec import Paged, ancestors, cast, parents, probs, rope_table, words
from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"


def _d(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.uint16 and dtype is None:
        dtype = torch.bfloat16
    return (t.view(dtype) if dtype is not None else t).to(DEV)


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _tree(p, mask):
    nr, t, hq, d = p.q.shape
    ws = bkv.alloc_tree_workspace(nr, t, hq, p.k.shape[2], d, p.bs, int(p.lens.max()))
    ws.fill_(0xFF)                                              # NaN: a partial nobody wrote would show
    q = _d(p.q)
    out = torch.full_like(q, 9.0)
    return bkv.bkv_paged_decode_tree(q, _d(p.k), _d(p.v), _d(p.table), _d(p.lens), int(p.lens.max()),
                                     _d(words(mask).view(np.int32)), out, ws)


@pytest.mark.parametrize("t,hq,hkv,seed", [(4, 32, 8, 0), (7, 32, 8, 1), (1, 16, 1, 2), (30, 32, 8, 3)])
def test_tree_decode_many_short_requests(t, hq, hkv, seed):
    """Batches whose units are mostly one tile long, so that a stream of the kernel has none, or one, of the next unit:
    every request's rows as the oracle's, and the same bits in every run."""
    rng = np.random.default_rng(seed)
    lens = np.where(rng.random(700) < 0.8, rng.integers(t, 129, 700), rng.integers(129, 600, 700))
    p = Paged(lens, t, hq, hkv, 128, 16, seed=seed)
    mask = ancestors(parents(rng, 700, t))
    first = _tree(p, mask)
    for _ in range(10):
        assert torch.equal(first, _tree(p, mask))
    got = _f64(first)
    for r in rng.permutation(700)[:60]:
        want, _ = oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens, words(mask))
        check_attention(got[r], want, "bf16")


@pytest.mark.parametrize("t,hq,hkv,d,dtype", [
    (6, 8, 2, 128, "bf16"), (40, 8, 2, 128, "bf16"), (6, 8, 2, 64, "bf16"), (6, 6, 3, 64, "f32"), (20, 4, 1, 128, "f32")])
def test_tree_decode_infinite_keys(t, hq, hkv, d, dtype):
    """An infinite key element makes scores of -inf (a weight of 0) or, by the query's sign, of +inf (a NaN row): among
    the committed positions (a first tile of nothing else included), in the tree, and where a row sees nothing else."""
    lens = [t + 300, t + 500, t + 90, t]
    p = Paged(lens, t, hq, hkv, d, 16, dtype)
    mask = ancestors(parents(np.random.default_rng(4), 4, t))
    mask[3, 4] = False
    mask[3, 4, 2] = True                                        # sees one key, and that one is infinite
    where = [(0, np.arange(5, 21)), (1, np.arange(0, 160)), (2, np.array([90 + 3])), (3, np.array([2]))]
    k = p.k.reshape(-1, hkv, d)
    for i, (r, pos) in enumerate(where):
        k[p.rows(r, pos), :, 3] = cast(np.array([-np.inf if i % 2 else np.inf], np.float32), dtype)[0]
    got = _f64(_tree(p, mask))
    finite = nans = empty = 0
    for r, n in enumerate(lens):
        rows = p.rows(r, np.arange(n))
        kr, vr = (wl.to_f32(c).reshape(-1, hkv, d)[rows].astype(np.float64) for c in (p.k, p.v))
        q = wl.to_f32(p.q[r]).astype(np.float64)
        for i in range(t):
            seen = np.ones(n, bool)
            seen[n - t:] = mask[r, i]
            for h in range(hq):
                s = (kr[seen, h // (hq // hkv)] @ q[i, h]) / np.sqrt(d)
                row = got[r, i, h]
                if np.isposinf(s).any():
                    assert np.isnan(row).all()
                    nans += 1
                elif np.isneginf(s).all():
                    assert not row.any()                        # nothing weighs anything
                    empty += 1
                else:
                    w = np.exp(s - s.max())
                    check_attention(row[None], (w @ vr[seen, h // (hq // hkv)] / w.sum())[None], dtype)
                    finite += 1
    assert finite and nans and empty


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot,dtype,norm", [
    (70, 4, 2, 80, 80, "bf16", True), (33, 3, 1, 10, 6, "f32", True), (50, 8, 2, 128, 24, "bf16", False),
    (41, 5, 1, 256, 250, "f32", False), (900, 7, 7, 96, 72, "bf16", True), (60, 8, 2, 64, 64, "bf16", True)])
def test_rope_write_in_place(n, hq, hkv, d, rot, dtype, norm, inter):
    """q_out may be q: the shapes whose elements turn with another lane's included."""
    rng = np.random.default_rng(7)
    q, k, v = (cast(rng.standard_normal((n, h, d)).astype(np.float32) * 2, dtype) for h in (hq, hkv, hkv))
    w = cast(1 + 0.3 * rng.standard_normal(d).astype(np.float32), dtype)
    cs, pos = rope_table(n, rot), np.arange(n)
    table = np.arange(1, -(-n // 16) + 1, dtype=np.int32).reshape(1, -1)
    td = torch.bfloat16 if dtype == "bf16" else torch.float32
    outs = []
    for in_place in (False, True):
        tq = _d(q)
        qo = tq if in_place else torch.zeros_like(tq)
        kc, vc = (torch.zeros(table.size + 1, 16, hkv, d, dtype=td, device=DEV) for _ in range(2))
        slots = torch.zeros(n, dtype=torch.int64, device=DEV)
        bkv.bkv_qk_norm_rope_cache_write(tq, _d(k), _d(v), _d(w) if norm else None, None, 1e-6, _d(cs), _d(table),
                                         torch.zeros(n, dtype=torch.int32, device=DEV), _d(pos), slots, qo, kc, vc,
                                         interleaved=inter)
        outs.append((qo, kc, vc))
    assert all(torch.equal(a, b) for a, b in zip(*outs))
    want, bad = oracle.norm_rope(q, w if norm else None, 1e-6, cs, pos, inter)
    assert bad == 0
    step = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]
    assert (np.abs(_f64(outs[1][0]) - want) <= step * np.abs(want) + 2e-6 * np.abs(want).max(-1, keepdims=True)).all()


# 2^-42 (1 + 2^-23) of a whole of 2^56 - 1 units of 2^-56 is just above 2^14 of them; without its last bit, just below
TINY = np.float32(2.0 ** -42 * (1 + 2.0 ** -23))


def test_verify_chain_smallest_numbers():
    """A sample by a number whose last bit lies below 2^-64: the running sum is compared with the exact product."""
    w = np.array([2.0 ** -42] + [2.0 ** (i - 56) for i in range(56) if i != 14], np.float32)
    us = np.array([TINY, 2.0 ** -42, np.nextafter(np.float32(2.0 ** -42), np.float32(0)), 2.0 ** -100, 2.0 ** -149, 0.0],
                  np.float32)
    p = np.broadcast_to(w, (6, 1, 56)).copy()
    out = torch.full((6, 1), -5, dtype=torch.int64, device=DEV)
    n = torch.full((6,), -5, dtype=torch.int32, device=DEV)
    none = torch.zeros(6, 0, device=DEV)
    bkv.bkv_verify_draft_chain(_d(p), torch.zeros(6, 0, 56, device=DEV), none.long(), none, _d(us), out, n)
    # u (2^56 - 1) against 2^14 units: above; 2^14 - 2^-42 and what is smaller: below
    assert out[:, 0].tolist() == [1, 0, 0, 0, 0, 0]
    # the definition in rational numbers (the whole has 56 bits: more than a double holds)
    weights = [Fraction(float(x)) for x in w]
    runs = list(itertools.accumulate(weights))
    assert out[:, 0].tolist() == [next(v for v, c in enumerate(runs) if c > Fraction(float(u)) * runs[-1]) for u in us]


def test_verify_tree_smallest_numbers():
    """A child against what its rejected sibling, of one unit, left: the product exact for a number below 2^-40."""
    v = 8
    p = np.zeros((3, 3, v), np.float32)
    p[:] = 0.1
    p[:, 0, 2], p[:, 0, 3] = 2.0 ** -56, 2.0 ** -42
    tok, par = np.array([[0, 2, 3]] * 3), np.array([[-1, 0, 0]] * 3, np.int32)
    u = np.array([[0, 0.5, TINY], [0, 0.5, 2.0 ** -42], [0, 0.5, 2.0 ** -120]], np.float32)
    out = torch.zeros(3, 3, dtype=torch.int64, device=DEV)
    path = torch.zeros(3, 3, dtype=torch.int32, device=DEV)
    n = torch.zeros(3, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_tree(_d(p), _d(tok), _d(par), _d(u), torch.full((3,), 0.5, device=DEV), out, path, n)
    assert n.tolist() == [0, 1, 1] and path[1:, 1].tolist() == [2, 2]


def test_verify_tree_never_takes_what_is_no_child():
    """A token outside the vocabulary or met before is rejected whatever its number."""
    rng = np.random.default_rng(3)
    p = probs(rng, (4, 4, 50), 1.0)
    p[:, 0, 7] = 0.0
    tok = np.array([[0, 50, -3, 9], [0, 7, 7, 7], [0, 9, 9, 9], [0, 11, 11, -1]])
    par = np.array([[-1, 0, 0, 0]] * 4, np.int32)
    u = np.array([[0, -1, -1, 0.999], [0, 0.5, -1, -1], [0, 0.999, -1, -1], [0, 0.999, -0.5, -1]], np.float32)
    out = torch.zeros(4, 4, dtype=torch.int64, device=DEV)
    path = torch.zeros(4, 4, dtype=torch.int32, device=DEV)
    n = torch.zeros(4, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_tree(_d(p), _d(tok), _d(par), _d(u), _d(np.float32([0.1, 0.3, 0.5, 0.9])), out, path, n)
    for got, want in zip((out, path, n), oracle.verify_tree(p, tok, par, u, np.float32([0.1, 0.3, 0.5, 0.9]))):
        assert np.array_equal(got.cpu().numpy(), want)
    assert n.tolist() == [0, 0, 0, 0] and (path[:, 1:] == -1).all() and (out[:, 0] >= 0).all()


@pytest.mark.parametrize("lens,t,hq,hkv,d,bs,dtype", [
    ([3, 70, 400], 5, 4, 2, 2, 16, "bf16"), ([3, 70, 400], 5, 4, 2, 8, 16, "f32"), ([40, 900], 9, 6, 2, 32, 16, "f32"),
    ([40, 900], 33, 6, 2, 32, 32, "bf16"), ([1, 31, 33, 257], 1, 2, 2, 24, 4, "bf16"),
    ([2, 3, 130] * 682 + [77, 1], 2, 2, 1, 128, 16, "bf16")],    # as many requests as the tensor-core kernel takes
    ids=lambda x: str(len(x)) if isinstance(x, list) else str(x))
def test_tree_decode_small_heads_and_full_tables(lens, t, hq, hkv, d, bs, dtype):
    p = Paged(lens, t, hq, hkv, d, bs, dtype)
    mask = ancestors(parents(np.random.default_rng(6), len(lens), t))
    want = np.stack([oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens, words(mask))[0]
                     for r in range(len(lens))])
    check_attention(_f64(_tree(p, mask)), want, dtype)


@pytest.mark.parametrize("bs", [128, 256])
@pytest.mark.parametrize("t,hq", [(6, 8), (50, 8)])
def test_tree_decode_tiles_that_are_not_there(bs, t, hq):
    """Null entries that leave whole tiles unloaded: the first, the last, one between, all."""
    p = Paged([700, 900, 1100, 520], t, hq, 2, 128, bs, holes=[(0, 0), (1, 2), (2, -(-1100 // bs) - 1)] +
              [(3, b) for b in range(-(-520 // bs))])
    mask = ancestors(parents(np.random.default_rng(6), 4, t))
    want = np.stack([oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens, words(mask))[0] for r in range(4)])
    assert not want[3].any()
    check_attention(_f64(_tree(p, mask)), want, "bf16")


def test_verify_rows_that_sum_to_just_below_256():
    """The largest sum that the units of 2^-56 hold: 255 weights of 1 and one of 1 - 2^-24."""
    p = np.ones((3, 1, 256), np.float32)
    p[:, 0, 255] = 1 - 2.0 ** -24
    us = np.array([0.0, 0.5, 1 - 2.0 ** -24], np.float32)
    out = torch.full((3, 1), -5, dtype=torch.int64, device=DEV)
    n, none, err = torch.zeros(3, dtype=torch.int32, device=DEV), torch.zeros(3, 0, device=DEV), torch.zeros(
        1, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_chain(_d(p), torch.zeros(3, 0, 256, device=DEV), none.long(), none, _d(us), out, n, err_count=err)
    runs = list(itertools.accumulate(Fraction(float(w)) for w in p[0, 0]))
    assert out[:, 0].tolist() == [next(v for v, c in enumerate(runs) if c > Fraction(float(u)) * runs[-1]) for u in us]
    assert out[:, 0].tolist() == [0, 127, 255] and int(err.item()) == 0

"""GPU tests of the speculative step over the paged cache against the fp64
oracle: norm + rotation + cache write, attention of drafted trees,
verification of drafts, and a run of them together.

Tolerances.  Attention: the bars of tests/_parity.py.  Norm and rotation: the
output's own rounding (bf16 2^-8, fp32 2^-24, E4M3 2^-4 of the value and
2^-10 where codes are subnormal, in units of the scale) plus 2e-6 of the
row's largest value for the fp32 arithmetic: at most 16 roundings of 2^-24
on each element of a pair, sqrt(2) for the pair, is 1.4e-6.  Slots, copied
values, error counts, tokens, paths and counts: equal."""
import numpy as np
import pytest
import torch

import oracle
from _parity import check_attention
from _spec import Paged, ancestors, cast, draws, parents, probs, rope_table, words
from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
TDT = {"bf16": torch.bfloat16, "f32": torch.float32}


def _d(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    if t.dtype == torch.uint16 and dtype is None:
        dtype = torch.bfloat16
    return (t.view(dtype) if dtype is not None else t).to(DEV)


def _i32(mask):
    return _d(mask.view(np.int32))


def _f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def _err():
    return torch.zeros(1, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# Norm, rotation, slots and cache write
# ---------------------------------------------------------------------------
def _rope_case(n, hq, hkv, d, rot, dtype, seed=0, reqs=3, bs=8, pad=0, extra=0):
    """Tokens of 3 requests with every kind of trouble among them, in a fused projection."""
    rng = np.random.default_rng(seed)
    cols = 6
    total = reqs * cols + 2
    table = rng.permutation(np.arange(1, total - 1))[: reqs * cols].reshape(reqs, cols).astype(np.int32)
    spots = rng.permutation(reqs * cols * bs)[:n]              # distinct (request, position) pairs
    req = (spots // (cols * bs)).astype(np.int32)
    pos = (spots % (cols * bs)).astype(np.int64)
    rpos = rng.integers(0, 90, n).astype(np.int64)
    if n > 12:
        req[1], req[4] = -1, reqs                              # padding; a request past the batch
        pos[5], pos[6] = cols * bs, -3                         # past the table; negative
        rpos[7], rpos[8] = 90, -1                              # past the rotation table; negative
        table[req[9], pos[9] // bs] = 0                        # a null entry
        table[req[10], pos[10] // bs] = total + 5              # a block past the cache
    width = (hq + 2 * hkv) * d + extra
    qkv = cast(rng.standard_normal((n, width)).astype(np.float32) * 2, dtype)
    w = [cast(1 + 0.3 * rng.standard_normal(d).astype(np.float32), dtype) for _ in range(2)]
    return dict(table=table, req=req, pos=pos, rpos=rpos, qkv=qkv, w=w, cs=rope_table(90, rot), total=total, bs=bs,
                max_n=n + pad)


def _split(qkv, hq, hkv, d):
    n = qkv.shape[0]
    q, k = hq * d, (hq + hkv) * d
    return (qkv[:, :q].reshape(n, hq, d), qkv[:, q:k].reshape(n, hkv, d), qkv[:, k:k + hkv * d].reshape(n, hkv, d))


def _views(qkv, hq, hkv, d):
    n, q, k = qkv.shape[0], hq * d, (hq + hkv) * d
    s = qkv.stride(0)
    return (qkv.as_strided((n, hq, d), (s, d, 1), qkv.storage_offset()),
            qkv.as_strided((n, hkv, d), (s, d, 1), qkv.storage_offset() + q),
            qkv.as_strided((n, hkv, d), (s, d, 1), qkv.storage_offset() + k))


def _run_rope(c, hq, hkv, d, dtype, fp8, norm, inter, k_scale=0.05, v_scale=0.07):
    q, k, v = _views(_d(c["qkv"]), hq, hkv, d)
    shape = (c["total"], c["bs"], hkv, d)
    if fp8:
        kc, vc = (torch.full(shape, 0x55, dtype=torch.uint8, device=DEV) for _ in range(2))
    else:
        kc, vc = (torch.full(shape, 7.0, dtype=TDT[dtype], device=DEV) for _ in range(2))
    q_out = torch.full((len(c["pos"]) + 2, hq, d), 7.0, dtype=TDT[dtype], device=DEV)
    slots = torch.full((c["max_n"],), -9, dtype=torch.int64, device=DEV)
    err = _err()
    args = [q, k, v, _d(c["w"][0]) if norm else None, _d(c["w"][1]) if norm else None, 1e-6, _d(c["cs"]), _d(c["table"]),
            _d(c["req"]), _d(c["pos"]), slots, q_out, kc, vc]
    kw = dict(rope_positions=_d(c["rpos"]), interleaved=inter, err_count=err)
    if fp8:
        bkv.bkv_qk_norm_rope_cache_write_fp8(*args, k_scale, v_scale, **kw)
    else:
        bkv.bkv_qk_norm_rope_cache_write(*args, **kw)
    torch.cuda.synchronize()
    return q_out, slots, kc, vc, int(err.item())


def _check_rope(c, hq, hkv, d, dtype, fp8, norm, inter, k_scale=0.05, v_scale=0.07):
    q_out, slots, kc, vc, err = _run_rope(c, hq, hkv, d, dtype, fp8, norm, inter, k_scale, v_scale)
    n = len(c["pos"])
    qn, kn, vn = _split(c["qkv"], hq, hkv, d)
    turned = (c["rpos"] >= 0) & (c["rpos"] < len(c["cs"]))
    req = np.where(turned, c["req"], -1).astype(np.int32)      # a token without a rotation is padding
    want_slots, serr = oracle.compute_slot_mapping(c["table"], req, c["pos"], c["bs"], n, c["max_n"])
    past = want_slots >= c["total"] * c["bs"]
    assert np.array_equal(slots.cpu().numpy(), want_slots)
    assert err == serr + int(past.sum()) + int(((c["req"] >= 0) & ~turned).sum())
    wq, _ = oracle.norm_rope(qn, c["w"][0] if norm else None, 1e-6, c["cs"], c["rpos"], inter)
    wk, _ = oracle.norm_rope(kn, c["w"][1] if norm else None, 1e-6, c["cs"], c["rpos"], inter)
    half_step = {"bf16": 2.0 ** -8, "f32": 2.0 ** -24}[dtype]

    def near(got, want):
        tol = half_step * np.abs(want) + 2e-6 * np.abs(want).max(-1, keepdims=True)
        assert (np.abs(got - want) <= tol).all()

    got = _f64(q_out)
    real = req >= 0
    near(got[:n][real], wq[real])
    assert (got[:n][~real] == 7).all() and (got[n:] == 7).all()  # padding and rows behind the last: as they were
    ok = (want_slots[:n] >= 0) & ~past[:n]
    at = want_slots[:n][ok]
    rest = np.ones(c["total"] * c["bs"], bool)
    rest[at] = False
    if fp8:
        ck, cv = (x.cpu().numpy().reshape(-1, hkv, d) for x in (kc, vc))
        assert (ck[rest] == 0x55).all() and (cv[rest] == 0x55).all()
        assert np.array_equal(cv[at], oracle.e4m3_encode((wl.to_f32(vn[ok]) / np.float32(v_scale)).astype(np.float32)))
        x = np.clip(wk[ok] / k_scale, -448, 448)
        tol = np.maximum(2.0 ** -4 * np.abs(x), 2.0 ** -10) + 2e-6 * np.abs(x).max(-1, keepdims=True)
        assert (np.abs(oracle.e4m3_decode(ck[at]) - x) <= tol).all()
    else:
        fk, fv = (_f64(x).reshape(-1, hkv, d) for x in (kc, vc))
        assert (fk[rest] == 7).all() and (fv[rest] == 7).all()
        near(fk[at], wk[ok])
        assert np.array_equal(fv[at], wl.to_f32(vn[ok]).astype(np.float64))


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("n,hq,hkv,d,rot,dtype,norm", [
    (1, 4, 1, 128, 128, "bf16", True), (13, 32, 8, 128, 128, "bf16", True), (77, 15, 5, 64, 64, "bf16", True),
    (40, 8, 2, 128, 64, "bf16", False), (33, 3, 1, 256, 256, "bf16", True), (29, 6, 2, 32, 16, "bf16", True),
    (40, 4, 4, 80, 80, "bf16", True), (21, 7, 7, 96, 32, "f32", True), (50, 12, 3, 128, 128, "f32", True),
    (31, 6, 2, 64, 32, "f32", False), (17, 2, 1, 256, 64, "f32", True), (19, 5, 1, 10, 6, "f32", True),
    (23, 4, 2, 64, 0, "bf16", True), (35, 16, 2, 128, 24, "bf16", True), (14, 40, 1, 64, 64, "f32", False)])
def test_rope_write(n, hq, hkv, d, rot, dtype, norm, inter, fp8):
    _check_rope(_rope_case(n, hq, hkv, d, rot, dtype, pad=n % 5), hq, hkv, d, dtype, fp8, norm, inter)


@pytest.mark.parametrize("extra", [1, 2, 4, 8])
def test_rope_write_row_strides(extra):
    """Projection rows at any stride: those off the 16-byte grid included."""
    _check_rope(_rope_case(40, 8, 2, 128, 128, "bf16", extra=extra), 8, 2, 128, "bf16", False, True, False)


@pytest.mark.parametrize("hq,hkv,d,rot,dtype,fp8", [
    (1, 1, 32, 32, "bf16", False),                               # two lanes' work in a warp
    (4, 1, 256, 128, "f32", True),                               # a warp a token
    (15, 5, 256, 256, "bf16", True),                             # five warps
    (64, 8, 128, 128, "bf16", False),                            # more heads than a CTA takes at once
    (40, 8, 64, 64, "f32", False),
    (33, 11, 64, 32, "bf16", True),
])
def test_rope_write_more_tokens_than_ctas(hq, hkv, d, rot, dtype, fp8):
    """Enough tokens that a CTA takes a token's heads together, several tokens in turn."""
    c = _rope_case(3500, hq, hkv, d, rot, dtype, reqs=40, bs=16, pad=3)
    for inter in (False, True):
        _check_rope(c, hq, hkv, d, dtype, fp8, True, inter)


def test_rope_write_many_tokens():
    c = _rope_case(3000, 32, 8, 128, 128, "bf16", reqs=40, bs=16)
    _check_rope(c, 32, 8, 128, "bf16", False, True, False)


def test_rope_write_saturates_and_keeps_nan():
    c = _rope_case(16, 2, 1, 128, 128, "f32")
    c["qkv"][2, 2 * 128:] *= 1e6
    c["qkv"][3, 3 * 128 + 5] = np.nan                          # in a value row
    c["qkv"][0, 3 * 128 + 5] = -np.inf
    _, slots, kc, vc, _ = _run_rope(c, 2, 1, 128, "f32", True, False, False)
    s = slots.cpu().numpy()
    codes = vc.cpu().numpy().reshape(-1, 128)
    assert (codes[s[3], 5] & 0x7F) == 0x7F and codes[s[0], 5] == 0xFE
    assert np.isin(codes[s[2]] & 0x7F, [0x7E]).mean() > 0.9


def test_rope_write_in_place_and_default_positions():
    """q_out may be q; without rope_positions the cache positions turn the heads."""
    c = _rope_case(12, 4, 2, 128, 128, "bf16")
    qn, kn, vn = _split(c["qkv"], 4, 2, 128)
    q, k, v = _d(qn), _d(kn), _d(vn)
    kc, vc = (torch.zeros(c["total"], c["bs"], 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.zeros(12, dtype=torch.int64, device=DEV)
    bkv.bkv_qk_norm_rope_cache_write(q, k, v, _d(c["w"][0]), None, 1e-6, _d(c["cs"]), _d(c["table"]), _d(c["req"]),
                                     _d(c["pos"]), slots, q, kc, vc)
    want, bad = oracle.norm_rope(qn, c["w"][0], 1e-6, c["cs"], c["pos"])
    assert bad == 0
    assert (np.abs(_f64(q) - want) <= 2.0 ** -8 * np.abs(want) + 2e-6 * np.abs(want).max(-1, keepdims=True)).all()


def test_rope_write_without_rotation_is_the_fused_write():
    """No weights and no rotation: the caches, slots and errors of bkv_slot_mapping_cache_write, the queries copied."""
    c = _rope_case(60, 4, 2, 64, 64, "bf16", pad=3)
    q, k, v = _views(_d(c["qkv"]), 4, 2, 64)
    got, want = [], []
    for out in (got, want):
        kc, vc = (torch.zeros(c["total"], c["bs"], 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
        slots = torch.zeros(c["max_n"], dtype=torch.int64, device=DEV)
        err = _err()
        table, req, pos = _d(c["table"]), _d(c["req"]), _d(c["pos"])
        if out is got:
            q_out = torch.zeros(60, 4, 64, dtype=torch.bfloat16, device=DEV)
            bkv.bkv_qk_norm_rope_cache_write(q, k, v, None, None, 0.0, None, table, req, pos, slots, q_out, kc, vc,
                                             err_count=err)
        else:
            bkv.bkv_slot_mapping_cache_write(table, req, pos, slots, k, v, kc, vc, num_tokens=60, err_count=err)
        out += [slots, kc, vc, err]
    # a negative position is no rotation row of a table of any size: padding with one error either way
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    real = (c["req"] >= 0) & (c["pos"] >= 0)
    assert torch.equal(q_out.cpu()[torch.from_numpy(real)], q.cpu()[torch.from_numpy(real)])


def test_rope_write_no_tokens():
    c = _rope_case(13, 4, 2, 64, 64, "bf16")
    q, k, v = _views(_d(c["qkv"]), 4, 2, 64)
    kc, vc = (torch.zeros(c["total"], c["bs"], 2, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.zeros(9, dtype=torch.int64, device=DEV)
    q_out = torch.zeros(13, 4, 64, dtype=torch.bfloat16, device=DEV)
    bkv.bkv_qk_norm_rope_cache_write(q, k, v, None, None, 0.0, _d(c["cs"]), _d(c["table"]), _d(c["req"]), _d(c["pos"]), slots,
                                     q_out, kc, vc, num_tokens=0)
    assert (slots == -1).all() and not kc.any() and not vc.any() and not q_out.any()


def test_rope_write_fewer_tokens_side_stream_and_graph():
    """num_tokens below the buffers' length (the rest is padding), on a side stream, and replayed from a graph
    after the projections changed in place."""
    c = _rope_case(40, 8, 2, 128, 128, "bf16")
    c["req"][:], c["pos"][:13], c["rpos"][:13] = np.maximum(c["req"], 0) % 3, np.arange(13), np.arange(13)
    c["table"][c["table"] <= 0] = 1
    c["table"][c["table"] >= c["total"]] = 1
    q, k, v = _views(_d(c["qkv"]), 8, 2, 128)
    kc, vc = (torch.zeros(c["total"], c["bs"], 2, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    slots = torch.full((40,), -9, dtype=torch.int64, device=DEV)
    q_out = torch.full((40, 8, 128), 7.0, dtype=torch.bfloat16, device=DEV)
    args = [q, k, v, _d(c["w"][0]), _d(c["w"][1]), 1e-6, _d(c["cs"]), _d(c["table"]), _d(c["req"]), _d(c["pos"]), slots, q_out,
            kc, vc]
    rpos = _d(c["rpos"])

    def check(qkv):
        want, _ = oracle.norm_rope(_split(qkv, 8, 2, 128)[0], c["w"][0], 1e-6, c["cs"], c["rpos"])
        got = _f64(q_out)
        w = want[:25]
        assert (np.abs(got[:25] - w) <= 2.0 ** -8 * np.abs(w) + 2e-6 * np.abs(w).max(-1, keepdims=True)).all()
        assert (got[25:] == 7).all() and (slots[25:] == -1).all() and (slots[:25] >= 0).all()

    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bkv.bkv_qk_norm_rope_cache_write(*args, rope_positions=rpos, num_tokens=25, stream=side)
    side.synchronize()
    check(c["qkv"])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bkv.bkv_qk_norm_rope_cache_write(*args, rope_positions=rpos, num_tokens=25)
    new = cast(np.random.default_rng(3).standard_normal(c["qkv"].shape).astype(np.float32), "bf16")
    for view, src in zip((q, k, v), _split(new, 8, 2, 128)):
        view.copy_(_d(src))
    g.replay()
    torch.cuda.synchronize()
    check(new)


# ---------------------------------------------------------------------------
# Attention of drafted trees
# ---------------------------------------------------------------------------
def _tree(p, mask, max_ctx=None, err=None, ws=None, stream=None, k=None, v=None, out=None):
    nr, t, hq, d = p.q.shape
    hkv = p.k.shape[2]
    max_ctx = int(p.lens.max()) if max_ctx is None else max_ctx
    if ws is None:
        ws = bkv.alloc_tree_workspace(nr, t, hq, hkv, d, p.bs, max_ctx)
        ws.fill_(0xFF)                                          # NaN: a partial nobody wrote would show
    q = _d(p.q)
    out = torch.full_like(q, 9.0) if out is None else out
    bkv.bkv_paged_decode_tree(q, _d(p.k) if k is None else k, _d(p.v) if v is None else v, _d(p.table), _d(p.lens), max_ctx,
                              _i32(words(mask)), out, ws, err_count=err, stream=stream)
    return out


def _want(p, mask, lens=None):
    rows, errs = [], 0
    for r in range(len(p.lens)):
        o, e = oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens if lens is None else lens, words(mask))
        rows.append(o)
        errs += e
    return np.stack(rows), errs


TREES = [  # lens, t, hq, hkv, d, bs, dtype
    ([1], 1, 1, 1, 128, 16, "bf16"),
    ([1, 2, 130, 0], 1, 8, 2, 128, 16, "bf16"),
    ([7, 128, 129, 500], 7, 32, 8, 128, 64, "bf16"),
    ([16, 17, 144, 1000, 385], 16, 32, 8, 128, 16, "bf16"),
    ([32, 700, 255], 32, 4, 1, 128, 32, "bf16"),                 # one full query tile
    ([33, 700, 257, 1], 33, 4, 1, 128, 32, "bf16"),              # a second one with one token
    ([61, 1500, 128], 61, 16, 2, 128, 64, "bf16"),               # two pairs
    ([64, 900], 64, 12, 4, 128, 128, "bf16"),                    # a group of 3
    ([40, 333, 90], 40, 10, 2, 128, 8, "bf16"),                  # a group of 5, small blocks
    ([256, 3000], 256, 2, 2, 128, 16, "bf16"),                   # the widest tree, no grouping
    ([129, 2000, 300], 129, 7, 1, 128, 256, "bf16"),             # a group of 7, blocks wider than a tile
    ([300] * 40, 5, 8, 8, 128, 16, "bf16"),                      # many equal requests
    ([20, 41, 333], 9, 4, 2, 128, 12, "bf16"),                   # a block size the tensor cores' loads do not take
    ([20, 300], 9, 6, 3, 64, 16, "bf16"),
    ([200, 31], 31, 4, 2, 256, 16, "bf16"),
    ([150, 12], 12, 2, 1, 80, 16, "bf16"),
    ([1, 44, 257], 1, 4, 2, 64, 4, "f32"),
    ([33, 800, 130], 11, 15, 5, 64, 16, "f32"),
    ([70, 513], 70, 8, 1, 128, 16, "f32"),
    ([25, 260], 3, 4, 4, 256, 32, "f32"),
    ([19, 90], 17, 3, 1, 34, 8, "f32"),
]


@pytest.mark.parametrize("case", TREES, ids=lambda c: f"t{c[1]}_h{c[2]}x{c[3]}_d{c[4]}_bs{c[5]}_{c[6]}")
def test_tree_decode(case):
    lens, t, hq, hkv, d, bs, dtype = case
    p = Paged(lens, t, hq, hkv, d, bs, dtype)
    rng = np.random.default_rng(5)
    mask = ancestors(parents(rng, len(lens), t))
    if t > 3:
        mask[-1, 2] = False                                      # a row of the tree that sees the prefix only
        mask[0, 3] = False
        mask[-1, :, 1] &= rng.random(t) < 0.5                    # and no tree at all
    want, errs = _want(p, mask)
    err = _err()
    got = _tree(p, mask, err=err)
    assert int(err.item()) == errs * hkv == 0
    check_attention(_f64(got), want, dtype)


@pytest.mark.parametrize("dtype,bs", [("bf16", 16), ("bf16", 64), ("bf16", 12), ("f32", 16)])
def test_tree_decode_random_masks_and_short_contexts(dtype, bs):
    """Any mask; caches shorter than the tree (its first tokens are not there); null and bad entries."""
    lens = [3, 11, 0, 200, 150, 90]
    p = Paged(lens, 11, 8, 2, 128, bs, dtype, holes=[(3, 1), (4, 0), (5, 3)])
    rng = np.random.default_rng(8)
    mask = rng.random((6, 11, 11)) < 0.4
    mask[3, 5] = False
    p.table[3, 2] = p.total + 4                                  # an id past the cache
    want, errs = _want(p, mask)
    err = _err()
    got = _tree(p, mask, err=err)
    assert errs > 0 and int(err.item()) == errs * 2
    check_attention(_f64(got), want, dtype)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_decode_narrow_table_and_clamped_length(dtype):
    p = Paged([100, 300, 60], 5, 8, 2, 128, 16, dtype, width=12)
    mask = ancestors(parents(np.random.default_rng(9), 3, 5))
    err = _err()
    want, errs = _want(p, mask)
    got = _tree(p, mask, err=err)
    assert errs == 7 and int(err.item()) == 14                   # 300 tokens are 19 blocks, the table has 12
    check_attention(_f64(got), want, dtype)
    err = _err()
    want, errs = _want(p, mask, np.minimum(p.lens, 90))
    got = _tree(p, mask, max_ctx=90, err=err)
    assert int(err.item()) == 2 + 2 * errs                       # two requests past the bound
    check_attention(_f64(got), want, dtype)


@pytest.mark.parametrize("t,g", [(7, 4), (40, 4), (61, 8)])
def test_tree_decode_causal_bits_are_the_decode(t, g):
    p = Paged([t, 400, 1300], t, 2 * g, 2, 128, 16)
    tri = np.broadcast_to(np.tril(np.ones((t, t), bool)), (3, t, t))
    got = _f64(_tree(p, tri))
    ws = bkv.alloc_workspace(3, t, 2 * g, 2, 128, 16, 1300)
    out = torch.zeros_like(_d(p.q))
    bkv.bkv_paged_decode(_d(p.q), _d(p.k), _d(p.v), _d(p.table), _d(p.lens), 1300, out, ws)
    # each side within 2^-7 of the exact row (its output's and its weights' rounding)
    w = _f64(out)
    assert (np.abs(got - w).max(-1) <= 2.0 ** -6 * np.abs(w).max(-1) + 1e-6).all()


def test_tree_decode_shared_mask_is_the_repeated_one():
    p = Paged([40, 300, 90], 20, 8, 2, 128, 16)
    mask = ancestors(parents(np.random.default_rng(3), 1, 20))
    a = _tree(p, np.repeat(mask, 3, 0))
    b = _tree(p, mask[0])
    assert torch.equal(a, b)


@pytest.mark.parametrize("t,hq,hkv,d,dtype,value", [
    (12, 8, 2, 128, "bf16", np.nan), (12, 8, 2, 128, "bf16", np.inf), (50, 8, 2, 128, "bf16", np.nan),
    (12, 8, 2, 64, "bf16", -np.inf), (12, 6, 2, 64, "f32", np.nan), (12, 6, 2, 64, "f32", np.inf)])
def test_tree_decode_masked_garbage_stays_out(t, hq, hkv, d, dtype, value):
    """K and V of two tree positions hold NaN or infinities: rows that see neither are untouched bit for bit,
    rows that see one are NaN.  Two requests whose trees end inside a tile and at its border."""
    p = Paged([300, 256], t, hq, hkv, d, 16, dtype)
    mask = ancestors(parents(np.random.default_rng(4), 2, t))
    clean = _tree(p, mask)
    for r, L in enumerate((300, 256)):
        for i, cache in ((t - 3, p.v), (t - 6, p.k)):
            row = p.rows(r, L - t + i)
            cache.reshape(-1, hkv, d)[row, :, 3] = cast(np.array([value], np.float32), dtype)[0]
    got = _tree(p, mask)
    g = _f64(got)
    for r in range(2):
        sees = mask[r, :, t - 3] | mask[r, :, t - 6]
        assert sees.any() and not sees.all()
        keep = torch.from_numpy(~sees)
        assert torch.equal(got[r].cpu()[keep], clean[r].cpu()[keep])
        v_only = mask[r, :, t - 3]
        assert np.isnan(g[r][v_only]).all()
        if not np.isinf(value):
            assert np.isnan(g[r][sees]).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_decode_garbage_behind_null_entries(dtype):
    """Requests whose caches hold NaN values run before one with null entries: a tile of the latter that is
    not loaded must not show what an earlier tile left behind."""
    p = Paged([260] * 30, 4, 4, 1, 128, 16, dtype, holes=[(r, b) for r in range(1, 30, 2) for b in (0, 3, 9)])
    mask = ancestors(parents(np.random.default_rng(4), 30, 4))
    want, _ = _want(p, mask)
    v = p.v.reshape(-1, 1, 128)
    for r in range(0, 30, 2):
        v[p.rows(r, np.arange(200))] = cast(np.array([np.nan], np.float32), dtype)[0]
    got = _f64(_tree(p, mask))
    check_attention(got[1::2], want[1::2], dtype)
    assert np.isnan(got[0::2]).all()


def test_tree_decode_long_contexts_are_split_and_repeatable():
    p = Paged([9000, 64, 3001], 61, 64, 8, 128, 64)
    mask = ancestors(parents(np.random.default_rng(4), 3, 61))
    a = _tree(p, mask)
    for _ in range(3):
        assert torch.equal(a, _tree(p, mask))
    for r in (0, 2):
        o, _ = oracle.paged_decode_tree_request(r, p.q[:, :, :8], p.k[:, :, :1], p.v[:, :, :1], p.table, p.lens, words(mask))
        check_attention(_f64(a)[r, :, :8], o, "bf16")


def test_tree_decode_offsets_past_32_bits():
    """Blocks whose element offsets pass 2^32."""
    bs, hkv, d, t = 64, 8, 128, 6
    p = Paged([70, 200], t, 8, hkv, d, bs)
    mask = ancestors(parents(np.random.default_rng(4), 2, t))
    want, _ = _want(p, mask)
    blocks = 2 ** 32 // (bs * hkv * d) + 40
    k = torch.zeros(blocks, bs, hkv, d, dtype=torch.bfloat16, device=DEV)
    v = torch.zeros_like(k)
    shift = blocks - p.total
    k[shift:], v[shift:] = _d(p.k), _d(p.v)
    p.table[p.table > 0] += shift
    check_attention(_f64(_tree(p, mask, k=k, v=v)), want, "bf16")


def test_tree_decode_streams_and_graphs():
    """On another stream than the current one; two captured graphs with workspaces of their own, replayed at once
    on new data."""
    ps = [Paged([300, 900, 40], 16, 8, 2, 128, 16, seed=s) for s in (1, 2)]
    mask = ancestors(parents(np.random.default_rng(4), 3, 16))
    want = [_tree(p, mask).clone() for p in ps]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    out = _tree(ps[0], mask, stream=side)
    side.synchronize()
    assert torch.equal(out, want[0])
    runs = []
    for p in ps:
        q, k, v, tb, ln, m = _d(p.q), _d(p.k), _d(p.v), _d(p.table), _d(p.lens), _i32(words(mask))
        o = torch.zeros_like(q)
        ws = bkv.alloc_tree_workspace(3, 16, 8, 2, 128, 16, 900)
        s = torch.cuda.Stream()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            bkv.bkv_paged_decode_tree(q, k, v, tb, ln, 900, m, o, ws)
        runs.append((g, s, o, q, k, v, tb, ln, m, ws))
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s, o, *_ in runs:
            with torch.cuda.stream(s):
                o.zero_()
                g.replay()
    torch.cuda.synchronize()
    for (g, s, o, *_), w in zip(runs, want):
        assert torch.equal(o, w)


@pytest.mark.parametrize("case", [
    ([30, 140], 5, 160, 160, 128, 16, "bf16"),                   # more KV heads than SMs
    ([9, 300, 70], 33, 88, 44, 128, 64, "bf16"),                 # KV heads that do not divide the SMs
    ([12, 70], 3, 130, 1, 128, 16, "bf16"),                      # a group wider than a query tile
    ([21, 400], 2, 128, 1, 128, 16, "bf16"),                     # one token a query tile
    ([40, 260], 33, 100, 4, 128, 16, "bf16"),                    # pairs of query tiles of 125 rows, a part of them idle
    ([60, 200], 3, 64, 1, 128, 32, "bf16"),                      # a pair whose second tile has one token
    ([3, 4, 5] * 750, 3, 2, 1, 128, 8, "bf16"),                  # more requests than the tensor-core kernel's tables hold
], ids=lambda c: f"n{len(c[0])}_t{c[1]}_h{c[2]}x{c[3]}")
def test_tree_decode_head_and_batch_counts(case):
    lens, t, hq, hkv, d, bs, dtype = case
    p = Paged(lens, t, hq, hkv, d, bs, dtype)
    mask = ancestors(parents(np.random.default_rng(6), len(lens), t))
    want, _ = _want(p, mask)
    check_attention(_f64(_tree(p, mask)), want, dtype)


@pytest.mark.parametrize("t,hq,hkv,d,bs,dtype", [
    (3, 4, 2, 66, 12, "f32"),
    (11, 15, 5, 64, 100, "f32"),                                 # blocks of no whole number of tiles
    (2, 4, 4, 128, 48, "f32"),
    (24, 3, 1, 36, 7, "bf16"),
    (40, 4, 2, 96, 16, "bf16"),                                  # several query tiles
    (1, 8, 1, 256, 1, "f32"),
])
def test_tree_decode_ragged_batches_without_tensor_cores(t, hq, hkv, d, bs, dtype):
    """Requests from none to 2,500 positions in one batch, many of them empty, with missing and bad entries: each of
    the bad ones counts once a KV head, however the columns share the positions."""
    rng = np.random.default_rng(11)
    lens = rng.integers(0, 120, 150) * (rng.random(150) < 0.6)
    lens[[7, 80, 149]] = 2500, 1, 1300
    p = Paged(lens, t, hq, hkv, d, bs, dtype)
    need = -(-p.lens // bs)
    for r in range(150):
        for b in range(need[r]):
            if rng.random() < 0.03:
                p.table[r, b] = rng.choice([0, -1, p.total, p.total + 5])
    mask = ancestors(parents(rng, 150, t))
    want, errs = _want(p, mask)
    err = _err()
    got = _tree(p, mask, err=err)
    assert errs > 0 and int(err.item()) == errs * hkv
    check_attention(_f64(got), want, dtype)
    assert torch.equal(got, _tree(p, mask))                      # and the same bits again


def test_tree_decode_nothing_cached():
    """A bound of 0 on the lengths, and lengths of 0 under a bound: zeros everywhere."""
    for dtype, lens, bound in (("bf16", [5, 9], 0), ("f32", [5, 9], 0), ("bf16", [0, 0], 500), ("f32", [0, 0], 500)):
        p = Paged(lens, 4, 8, 2, 128, 16, dtype)
        mask = np.ones((2, 4, 4), bool)
        err = _err()
        assert not _tree(p, mask, max_ctx=bound, err=err).any()
        assert int(err.item()) == (2 if bound == 0 else 0)


def test_tree_decode_very_long_context():
    """One request of 70,001 positions over every column of CTAs, against torch in fp64."""
    t, hq, hkv, L = 9, 8, 2, 70001
    p = Paged([L], t, hq, hkv, 128, 64)
    mask = ancestors(parents(np.random.default_rng(7), 1, t))
    got = _tree(p, mask)[0].double()
    rows = torch.from_numpy(p.rows(0, np.arange(L))).to(DEV)
    seen = torch.ones(t, L, dtype=torch.bool, device=DEV)
    seen[:, L - t:] = _d(mask[0])
    q = _d(p.q)[0].double()
    for h in range(hq):
        k, v = (_d(c).view(-1, hkv, 128)[rows, h // 4].double() for c in (p.k, p.v))
        s = (q[:, h] @ k.T / 128 ** 0.5).masked_fill(~seen, float("-inf"))
        want = s.softmax(-1) @ v
        assert ((got[:, h] - want).abs().amax(-1) <= 1e-2 * want.abs().amax(-1)).all()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_decode_graph_replays_on_new_lengths(dtype):
    """A captured call, replayed after lengths, table, mask and queries changed in place: nothing of the first
    run is kept."""
    a, b = (Paged(lens, 7, 8, 2, 128, 16, dtype, seed=s) for s, lens in ((1, [300, 20, 700]), (2, [9, 640, 0])))
    rng = np.random.default_rng(5)
    ma, mb = (ancestors(parents(rng, 3, 7)) for _ in range(2))
    n = max(a.total, b.total)
    w = max(a.table.shape[1], b.table.shape[1])
    bufs = [torch.zeros((n,) + a.k.shape[1:], dtype=TDT[dtype], device=DEV) for _ in range(2)]
    bufs += [torch.zeros(3, w, dtype=torch.int32, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV),
             torch.zeros(3, 7, 1, dtype=torch.int32, device=DEV), torch.zeros(a.q.shape, dtype=TDT[dtype], device=DEV)]
    k, v, table, lens, mask, q = bufs
    out = torch.zeros_like(q)
    ws = bkv.alloc_tree_workspace(3, 7, 8, 2, 128, 16, 700)

    def fill(p, m):
        k[: p.total], v[: p.total] = _d(p.k), _d(p.v)
        table.fill_(-1)
        table[:, : p.table.shape[1]] = _d(p.table)
        lens.copy_(_d(p.lens))
        mask.copy_(_i32(words(m)))
        q.copy_(_d(p.q))

    fill(a, ma)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bkv.bkv_paged_decode_tree(q, k, v, table, lens, 700, mask, out, ws)
    for p, m in ((a, ma), (b, mb), (a, ma)):
        fill(p, m)
        g.replay()
        torch.cuda.synchronize()
        check_attention(_f64(out), _want(p, m)[0], dtype)


# ---------------------------------------------------------------------------
# Verification
# ---------------------------------------------------------------------------
def _chain(p, q, tok, u, us, lens=None, err=None):
    r, k1, _ = p.shape
    out = torch.full((r, k1), -5, dtype=torch.int64, device=DEV)
    n = torch.full((r,), -5, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_chain(p, q, _d(tok), _d(u), _d(us), out, n, draft_lens=None if lens is None else _d(lens),
                               err_count=err)
    return out.cpu().numpy(), n.cpu().numpy()


def _tree_verify(p, tok, par, u, us, err=None):
    r, t, _ = p.shape
    out = torch.full((r, t), -5, dtype=torch.int64, device=DEV)
    path = torch.full((r, t), -5, dtype=torch.int32, device=DEV)
    n = torch.full((r,), -5, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_tree(p, _d(tok), _d(par), _d(u), _d(us), out, path, n, err_count=err)
    return out.cpu().numpy(), path.cpu().numpy(), n.cpu().numpy()


def _u(rng, *shape):
    return rng.random(shape, dtype=np.float32)


@pytest.mark.parametrize("reqs,k,v", [(1, 0, 5), (1, 1, 1), (3, 4, 2), (40, 3, 33), (17, 7, 1000), (9, 2, 32000),
                                      (5, 40, 4097), (300, 1, 1025), (4, 5, 131072)])
def test_verify_chain(reqs, k, v):
    rng = np.random.default_rng(11)
    p = probs(rng, (reqs, k + 1, v))
    q = probs(rng, (reqs, k, v)) if k else np.zeros((reqs, 0, v), np.float32)
    q = (0.6 * p[:, :k] + 0.4 * q).astype(np.float32)
    tok = draws(rng, q)
    lens = rng.integers(0, k + 1, reqs).astype(np.int32)
    u, us = _u(rng, reqs, k), _u(rng, reqs)
    us[0] = 0.0
    for ln in (None, lens):
        want = oracle.verify_chain(p, q, tok, u, us, ln)
        err = _err()
        got = _chain(_d(p), _d(q), tok, u, us, ln, err)
        assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1]) and int(err.item()) == want[2] == 0


@pytest.mark.parametrize("v", [127, 128, 2047, 2049, 4100, 6145, 8191, 8192, 10239, 12292, 16385, 20480])
def test_verify_parts_of_every_length(v):
    """Vocabularies whose parts of a warp end in every share of a round, rows aligned and not: the same tokens as the
    oracle's, bit for bit, in chains and trees."""
    rng = np.random.default_rng(v)
    p, q = probs(rng, (280, 2, v)), probs(rng, (280, 1, v))
    tok = draws(rng, q)
    u, us = np.ones((280, 1), np.float32), _u(rng, 280)          # every draft refused: the residual's sample
    u[::2] = 0.0                                                 # or taken: the row's own
    want = oracle.verify_chain(p, q, tok, u, us)
    got = _chain(_d(p), _d(q), tok, u, us)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    t = 3
    p = probs(rng, (100, t, v))
    par = parents(rng, 100, t)
    tok = rng.integers(0, v, (100, t))
    u, us = _u(rng, 100, t), _u(rng, 100)
    want = oracle.verify_tree(p, tok, par, u, us)
    got = _tree_verify(_d(p), tok, par, u, us)
    assert all(np.array_equal(g, w) for g, w in zip(got, want))


def test_verify_chain_bad_inputs_and_edges():
    rng = np.random.default_rng(12)
    p, q = probs(rng, (6, 4, 500)), probs(rng, (6, 3, 500))
    tok = draws(rng, q)
    tok[0, 0], tok[1, 1] = 500, -1
    u, us = _u(rng, 6, 3), _u(rng, 6)
    u[:, 0] = 0.0                                                # accepted wherever the target has it at all
    us[2], us[3] = 1.0, np.nan                                   # the border at the sum's end
    lens = np.array([3, 3, 4, -2, 3, 3], np.int32)
    q[4, 0] = p[4, 0]                                            # a residual of zeros: the row itself
    p[4, 0, tok[4, 0]] = 0.0
    q[4, 0] = np.maximum(p[4, 0], q[4, 0])
    p[5] = 0.0                                                   # no weight at all
    want = oracle.verify_chain(p, q, tok, u, np.nan_to_num(us, nan=1.0), lens)
    err = _err()
    got = _chain(_d(p), _d(q), tok, u, us, lens, err)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])
    assert int(err.item()) == want[2] > 0
    assert got[0][5, 0] == -1


def test_verify_chain_strided_and_unaligned_rows():
    rng = np.random.default_rng(13)
    wide_p = torch.zeros(7, 6, 1011, device=DEV)
    wide_q = torch.zeros(7, 5, 1013, device=DEV)
    p, q = probs(rng, (7, 5, 1001)), probs(rng, (7, 4, 1001))
    vp, vq = wide_p[:, 1:, 3:1004], wide_q[:, :4, 5:1006]
    vp.copy_(_d(p))
    vq.copy_(_d(q))
    tok, u, us = draws(rng, q), _u(rng, 7, 4), _u(rng, 7)
    want = oracle.verify_chain(p, q, tok, u, us)
    got = _chain(vp, vq, tok, u, us)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


@pytest.mark.parametrize("reqs,t,v", [(1, 1, 7), (2, 2, 3), (30, 9, 40), (13, 33, 1000), (5, 61, 50001), (3, 300, 2000),
                                      (2, 16, 131072), (70, 5, 4096)])
def test_verify_tree(reqs, t, v):
    rng = np.random.default_rng(14)
    p = probs(rng, (reqs, t, v), 2.0)
    par = parents(rng, reqs, t)
    likely = np.argsort(-p, -1)[:, :, : max(1, min(v, 6))]
    tok = np.zeros((reqs, t), np.int64)
    for r in range(reqs):
        for i in range(1, t):
            tok[r, i] = likely[r, par[r, i], rng.integers(likely.shape[2])]       # siblings may repeat a token
    u, us = _u(rng, reqs, t) * 0.6, _u(rng, reqs)
    want = oracle.verify_tree(p, tok, par, u, us)
    err = _err()
    got = _tree_verify(_d(p), tok, par, u, us, err)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
    assert int(err.item()) == want[3] == 0


def test_verify_tree_bad_inputs_and_edges():
    rng = np.random.default_rng(15)
    reqs, t, v = 6, 12, 300
    p = probs(rng, (reqs, t, v), 1.0)
    par = parents(rng, reqs, t)
    tok = draws(rng, np.take_along_axis(p, np.maximum(par, 0)[..., None], 1))
    u, us = _u(rng, reqs, t) * 0.01, _u(rng, reqs)
    par[0, 3], par[0, 4], par[1, 5], par[1, 6] = 3, 40, -1, -2   # itself, past the tree, padding, no node
    tok[2, 1], tok[2, 2] = v, -7
    par[3, 1:] = -1                                              # the root alone
    p[4, 0] = 0.0                                                # its only weights are its children's: none
    p[5, 0], par[5, 1], par[5, 2], tok[5, 1], tok[5, 2] = 0.0, 0, 0, 3, 5
    par[5, 3:] = -1
    p[5, 0, 3], p[5, 0, 5], u[5, 1], u[5, 2] = 0.5, 0.5, 1.0, 1.0   # all of the mass rejected: the row itself
    want = oracle.verify_tree(p, tok, par, u, us)
    err = _err()
    got = _tree_verify(_d(p), tok, par, u, us, err)
    for a, b in zip(got, want):
        assert np.array_equal(a, b)
    assert int(err.item()) == want[3] > 0
    assert got[0][4, 0] == -1 and got[0][5, 0] in (3, 5)


def test_verify_shared_rows_and_streams():
    """One set of target rows for all requests (request stride 0), on a side stream and replayed from a graph."""
    rng = np.random.default_rng(17)
    p = probs(rng, (1, 6, 777))
    par = parents(rng, 20, 6)
    tok = draws(rng, np.take_along_axis(np.repeat(p, 20, 0), np.maximum(par, 0)[..., None], 1))
    u, us = _u(rng, 20, 6) * 0.4, _u(rng, 20)
    want = oracle.verify_tree(np.repeat(p, 20, 0), tok, par, u, us)
    shared = _d(p).expand(20, 6, 777)
    for a, b in zip(_tree_verify(shared, tok, par, u, us), want):
        assert np.array_equal(a, b)
    args = [_d(tok), _d(par), _d(u), _d(us), torch.zeros(20, 6, dtype=torch.int64, device=DEV),
            torch.zeros(20, 6, dtype=torch.int32, device=DEV), torch.zeros(20, dtype=torch.int32, device=DEV)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    bkv.bkv_verify_draft_tree(shared, *args, stream=side)
    side.synchronize()
    assert np.array_equal(args[4].cpu().numpy(), want[0])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        bkv.bkv_verify_draft_tree(shared, *args)
    for x in args[4:]:
        x.fill_(-9)
    g.replay()
    torch.cuda.synchronize()
    for a, b in zip(args[4:], want):
        assert np.array_equal(a.cpu().numpy(), b)


def test_verify_wide_trees_and_long_chains():
    """The most nodes and drafts: a root with 1023 children, a chain of 1024."""
    rng = np.random.default_rng(18)
    p = np.zeros((2, 1024, 1500), np.float32)
    p[:] = probs(rng, (1, 1, 1500), 1.0)
    par = np.zeros((2, 1024), np.int32)
    par[:, 0] = -1
    par[1, 600:] = 599
    tok = np.stack([rng.permutation(1500)[:1024] for _ in range(2)])
    u = np.full((2, 1024), 0.999, np.float32)
    u[0, 1000:] = 0.0
    us = _u(rng, 2)
    want = oracle.verify_tree(p, tok, par, u, us)
    for a, b in zip(_tree_verify(_d(p), tok, par, u, us), want):
        assert np.array_equal(a, b)
    q = p[:, :1, :].repeat(1024, 1)
    t = np.concatenate([p, p[:, :1]], 1)
    u = np.full((2, 1024), 0.5, np.float32)
    u[1, 700] = 1.0
    want = oracle.verify_chain(t, q, tok, u, us)
    assert want[1].tolist() == [1024, 700]
    got = _chain(_d(t), _d(q), tok, u, us)
    assert np.array_equal(got[0], want[0]) and np.array_equal(got[1], want[1])


def test_verify_offsets_past_32_bits():
    """Rows whose element offsets pass 2^32."""
    v, t = 131072, 3
    rng = np.random.default_rng(16)
    p = probs(rng, (2, t, v))
    tok = draws(rng, p[:, [0, 0, 1]])
    par = np.array([[-1, 0, 1]] * 2, np.int32)
    u, us = _u(rng, 2, t) * 0.3, _u(rng, 2)
    want = oracle.verify_tree(p, tok, par, u, us)
    far = torch.empty(2 ** 32 + 2 * t * v, device=DEV)
    rows = far.as_strided((2, t, v), (2 ** 32 + 7, v, 1))
    rows.copy_(_d(p))
    for a, b in zip(_tree_verify(rows, tok, par, u, us), want):
        assert np.array_equal(a, b)


# ---------------------------------------------------------------------------
# A step of them together
# ---------------------------------------------------------------------------
def test_a_speculative_step():
    """Drafted trees through the whole step, as a program runs it: the tree's tokens are normalised, turned and
    written behind the committed ones; the tree is attended; drafts are verified; and the accepted tokens' rows
    are written to their final places with the cache write, rejected drafts as padding.  The cache then equals one
    that saw the accepted tokens alone, and the next decode step gives its outputs."""
    rng = np.random.default_rng(21)
    nr, t, hq, hkv, d, bs, v = 3, 13, 8, 2, 128, 16, 900
    base = np.array([50, 3, 121])                                # committed tokens; node 0 is the last emitted token
    par = parents(rng, nr, t)
    anc = ancestors(par)
    depth = anc.sum(-1) - 1
    p = Paged(base + 2 * t, t, hq, hkv, d, bs)                   # room for this step and the next
    k_cache, v_cache = _d(p.k), _d(p.v)
    cs, wq, wk = rope_table(400, d), *(cast(1 + 0.2 * rng.standard_normal(d).astype(np.float32), "bf16") for _ in range(2))
    qkv = cast(rng.standard_normal((nr * t, (hq + 2 * hkv) * d)).astype(np.float32), "bf16")
    q, k, vv = _views(_d(qkv), hq, hkv, d)
    req = np.repeat(np.arange(nr), t).astype(np.int32)
    pos = (base[:, None] + np.arange(t)).reshape(-1)
    rpos = (base[:, None] + depth).reshape(-1)
    slots = torch.zeros(nr * t, dtype=torch.int64, device=DEV)
    q_out = torch.zeros(nr * t, hq, d, dtype=torch.bfloat16, device=DEV)
    err = _err()
    bkv.bkv_qk_norm_rope_cache_write(q, k, vv, _d(wq), _d(wk), 1e-6, _d(cs), _d(p.table), _d(req), _d(pos), slots, q_out,
                                     k_cache, v_cache, rope_positions=_d(rpos), err_count=err)
    lens = (base + t).astype(np.int32)
    ws = bkv.alloc_tree_workspace(nr, t, hq, hkv, d, bs, int(lens.max()))
    out = torch.zeros(nr, t, hq, d, dtype=torch.bfloat16, device=DEV)
    bkv.bkv_paged_decode_tree(q_out.view(nr, t, hq, d), k_cache, v_cache, _d(p.table), _d(lens), int(lens.max()),
                              _i32(words(anc)), out, ws, err_count=err)
    # every token's output is what a decode of its own path gives
    kh, vh = (x.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, hkv, d) for x in (k_cache, v_cache))
    for r in range(nr):
        for node in (0, t // 2, t - 1):
            path = np.flatnonzero(anc[r, node])
            rows = np.concatenate([p.rows(r, np.arange(base[r])), p.rows(r, base[r] + path)])
            n = len(rows)
            kr, vr = (np.concatenate([c[rows[:1]], c[rows]])[:, None] for c in (kh, vh))   # block 0 is the null block
            table = np.arange(1, n + 1, dtype=np.int32)[None]
            qn = q_out.view(nr, t, hq, d)[r, node].view(torch.int16).cpu().numpy().view(np.uint16)[None, None]
            want, _ = oracle.paged_decode_request(0, qn, kr, vr, table, np.array([n], np.int32))
            check_attention(_f64(out)[r, node][None], want, "bf16")
    pr = probs(rng, (nr, t, v), 2.0)
    tok = draws(rng, np.take_along_axis(pr, np.maximum(par, 0)[..., None], 1))
    out_tok = torch.zeros(nr, t, dtype=torch.int64, device=DEV)
    path = torch.zeros(nr, t, dtype=torch.int32, device=DEV)
    count = torch.zeros(nr, dtype=torch.int32, device=DEV)
    bkv.bkv_verify_draft_tree(_d(pr), _d(tok), _d(par), _d(_u(rng, nr, t) * 0.05), _d(_u(rng, nr)), out_tok, path, count,
                              err_count=err)
    assert int(count.sum()) > 0
    # commit: the accepted nodes' rows to consecutive positions, everything else padding
    nodes = path.long()
    real = nodes >= 0
    flat = (nodes.clamp_min(0) + torch.arange(nr, device=DEV)[:, None] * t).reshape(-1)
    creq = torch.where(real, torch.arange(nr, device=DEV, dtype=torch.int32)[:, None], -1).reshape(-1)
    cpos = (torch.from_numpy(base).to(DEV)[:, None] + torch.arange(t, device=DEV)).reshape(-1)
    turned = k_cache.view(-1, hkv, d)[slots[flat]].contiguous()    # the rows as the step wrote them, before any moves
    bkv.bkv_slot_mapping_cache_write(_d(p.table), creq, cpos, slots, turned, vv[flat].contiguous(), k_cache, v_cache,
                                     err_count=err)
    assert int(err.item()) == 0
    kh2, vh2 = (x.view(torch.int16).cpu().numpy().view(np.uint16).reshape(-1, hkv, d) for x in (k_cache, v_cache))
    turned_k, _ = oracle.norm_rope(_split(qkv, hq, hkv, d)[1], wk, 1e-6, cs, rpos)
    for r in range(nr):
        for i, node in enumerate(path[r].cpu().numpy()):
            if node < 0:
                break
            row = p.rows(r, base[r] + i)
            w = turned_k[r * t + node]
            assert (np.abs(wl.to_f32(kh2[row]) - w) <= 2.0 ** -8 * np.abs(w) + 2e-6 * np.abs(w).max()).all()
            assert np.array_equal(vh2[row], _split(qkv, hq, hkv, d)[2][r * t + node])
        before = p.rows(r, np.arange(base[r]))
        assert np.array_equal(kh2[before], kh[before])
    new_lens = (base + count.cpu().numpy() + 1).astype(np.int32)
    dec = torch.zeros(nr, 1, hq, d, dtype=torch.bfloat16, device=DEV)
    ws = bkv.alloc_workspace(nr, 1, hq, hkv, d, bs, int(new_lens.max()))
    bkv.bkv_paged_decode(q_out.view(nr, t, hq, d)[:, :1].contiguous(), k_cache, v_cache, _d(p.table), _d(new_lens),
                         int(new_lens.max()), dec, ws)
    shape = (p.total, bs, hkv, d)
    for r in range(nr):
        want, _ = oracle.paged_decode_request(r, q_out.view(nr, t, hq, d)[:, :1].contiguous().view(torch.int16).cpu().numpy()
                                              .view(np.uint16), kh2.reshape(shape), vh2.reshape(shape), p.table, new_lens)
        check_attention(_f64(dec)[r], want, "bf16")

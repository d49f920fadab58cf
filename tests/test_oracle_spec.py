"""Pins of the oracle's speculative step (readings R18 .. R20) against torch
in fp64, reductions to pinned functions, closed forms, and the property that
makes verification right: the emitted tokens are distributed as the target's."""
import numpy as np
import pytest
import torch

import oracle
from _spec import Paged, ancestors, cast, draws, parents, probs, rope_table, words
from paged_kv_cache_slot_gb300 import workloads as wl


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("rot", [0, 6, 16])
@pytest.mark.parametrize("norm", [False, True])
def test_norm_rope_is_a_complex_turn(inter, rot, norm):
    """Pairs as complex numbers: the rotation multiplies pair i by cos + i sin of its angle."""
    rng = np.random.default_rng(1)
    x = rng.standard_normal((5, 3, 16)).astype(np.float32)
    w = rng.standard_normal(16).astype(np.float32) if norm else None
    cs = rope_table(50, rot)
    pos = np.array([0, 1, 7, 49, 50])
    got, bad = oracle.norm_rope(x, w, 1e-5, cs, pos, inter)
    assert bad == 1 and not got[4].any()
    y = torch.from_numpy(x).double()
    if norm:
        y = torch.nn.functional.rms_norm(y, (16,), torch.from_numpy(w).double(), 1e-5)
    z = y.clone()
    if rot:
        head = y[..., :rot]
        a, b = (head[..., 0::2], head[..., 1::2]) if inter else (head[..., :rot // 2], head[..., rot // 2:])
        c = torch.from_numpy(cs[np.minimum(pos, 49)]).double()[:, None]
        turned = torch.complex(a, b) * torch.complex(c[..., :rot // 2], c[..., rot // 2:])
        z[..., :rot] = (torch.view_as_real(turned).flatten(-2) if inter else torch.cat([turned.real, turned.imag], -1))
    assert np.abs(got[:4] - z.numpy()[:4]).max() < 1e-12


def test_rotated_products_depend_on_the_distance_only():
    rng = np.random.default_rng(2)
    q, k = rng.standard_normal((2, 1, 1, 32)).astype(np.float32)
    cs = rope_table(200, 32)
    dot = []
    for p in (3, 90):
        a, _ = oracle.norm_rope(q[None, 0], None, 0.0, cs, [p + 17])
        b, _ = oracle.norm_rope(k[None, 0], None, 0.0, cs, [p])
        dot.append((a * b).sum())
    assert abs(dot[0] - dot[1]) < 1e-5      # the table is fp32


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_tree_masks_reduce_to_the_decode(dtype):
    """Lower-triangular bits are the causal decode, all bits its all-ones mask."""
    t = 5
    p = Paged([5, 0, 23, 40], t, 4, 2, 16, 4, dtype, holes=[(3, 2)])
    causal = words(np.tril(np.ones((t, t), bool)))
    full = words(np.ones((t, t), bool))
    for r in range(4):
        for mode, mask in ((0, causal), (1, np.broadcast_to(full, (4,) + full.shape))):
            want, e0 = oracle.paged_decode_request(r, p.q, p.k, p.v, p.table, p.lens, mask_mode=mode)
            got, e1 = oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens, mask)
            assert e0 == e1 and np.abs(got - want).max() < 1e-13


def test_tree_decode_matches_sdpa():
    t, hq, hkv, d = 37, 6, 2, 16
    p = Paged([37, 90], t, hq, hkv, d, 8)
    rng = np.random.default_rng(3)
    mask = ancestors(parents(rng, 2, t))
    mask[1, 4] = False                                     # a row that sees the committed positions only
    mask[0, 6] = False                                     # and one that sees nothing
    for r, L in enumerate((37, 90)):
        got, err = oracle.paged_decode_tree_request(r, p.q, p.k, p.v, p.table, p.lens, words(mask))
        assert err == 0
        rows = p.rows(r, np.arange(L))
        k, v = (torch.from_numpy(wl.to_f32(c).reshape(-1, hkv, d)[rows].astype(np.float64)).permute(1, 0, 2)
                .repeat_interleave(hq // hkv, 0) for c in (p.k, p.v))
        q = torch.from_numpy(wl.to_f32(p.q[r]).astype(np.float64)).permute(1, 0, 2)
        seen = np.ones((t, L), bool)
        seen[:, L - t:] = mask[r]
        o = torch.nn.functional.scaled_dot_product_attention(q, k, v, attn_mask=torch.from_numpy(seen)[None])
        o = torch.nan_to_num(o.permute(1, 0, 2)).numpy()
        assert np.abs(got - o).max() < 1e-12
        if r == 0:
            assert not got[6].any()


def _grid(n):
    return (np.arange(n) + 0.5) / n


def test_chain_tokens_are_distributed_as_the_targets():
    """Over a draft drawn from q and even grids of both random numbers, the first emitted token has the
    target's distribution (grid error 1 / 64 a draw, weighted by q)."""
    rng = np.random.default_rng(4)
    p, q = probs(rng, (1, 2, 6), 1.0), probs(rng, (1, 1, 6), 1.0)
    seen = np.zeros(6)
    u, us = np.meshgrid(_grid(64), _grid(64))
    n = u.size
    for x in range(6):
        out, count, err = oracle.verify_chain(np.repeat(p, n, 0), np.repeat(q, n, 0), np.full((n, 1), x), u.reshape(n, 1),
                                              us.reshape(n))
        assert err == 0
        seen += np.bincount(out[:, 0], minlength=6) / n * q[0, 0, x]
        assert np.array_equal(out[:, 1] >= 0, count == 1)
    assert np.abs(seen - p[0, 0]).max() < 2 / 64


def test_tree_tokens_are_distributed_as_the_targets():
    """The first emitted token of a root with three children (two of the same token)."""
    rng = np.random.default_rng(5)
    p = probs(rng, (1, 5, 4), 0.7)
    g = _grid(24)
    u1, u2, us = (x.reshape(-1) for x in np.meshgrid(g, g, g))
    n = len(us)
    u = np.stack([np.zeros(n), u1, np.full(n, 0.5), u2, np.full(n, 0.9)], 1)
    par = np.broadcast_to(np.array([-1, 0, 0, 0, 1], np.int32), (n, 5))
    tok = np.broadcast_to(np.array([0, 2, 2, 1, 3]), (n, 5))
    out, path, count, err = oracle.verify_tree(np.repeat(p, n, 0), tok, par, u, us)
    assert err == 0
    assert np.abs(np.bincount(out[:, 0], minlength=4) / n - p[0, 0]).max() < 4 / 24
    assert np.array_equal((path >= 0).sum(1), count + 1)
    assert not (path == 2).any()                              # a token met before is never taken


def test_chain_closed_forms():
    rng = np.random.default_rng(6)
    p = probs(rng, (3, 4, 9))
    tok = draws(rng, p[:, :3])
    u, us = rng.random((3, 3)) * 0.999, np.array([0.0, 0.5, 1.0])
    out, count, err = oracle.verify_chain(p, p[:, :3], tok, u, us)      # the draft is the target: all stand
    assert (count == 3).all() and np.array_equal(out[:, :3], tok) and err == 0
    assert out[0, 3] == 0 and out[2, 3] == 8                            # u = 0 and u = 1: the first, the last token
    q = np.zeros((3, 3, 9), np.float32)
    q[:, :, 4] = 1.0
    p[:, :, 4] = 0.0
    out, count, _ = oracle.verify_chain(p, q, np.full((3, 3), 4), u, us)  # never the target's: none stand
    assert (count == 0).all() and not (out[:, 0] == 4).any()
    out, count, err = oracle.verify_chain(p, q, np.full((3, 3), 4), u, us, lens=[0, 9, -1])
    assert err == 2 and out[1, 0] >= 0
    out, _, err = oracle.verify_chain(p * 0, q, np.full((3, 3), 12), u, us)
    assert (out[:, 0] == -1).all() and err == 3 * 3 + 3

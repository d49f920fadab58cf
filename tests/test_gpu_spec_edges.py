"""GPU tests of the speculative step at its edges: infinite keys, heads turned in
place, batches of short contexts, the smallest random numbers.

Tolerances as in tests/test_gpu_spec.py: attention by tests/_parity.py; norm and
rotation the output's rounding plus 2e-6 of the row's largest value; tokens,
paths and counts equal."""
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

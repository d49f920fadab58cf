"""GPU tests of rows whose attention is one key's for the most part and thousands of keys' for the rest, each of which
weighs next to nothing: what the first token of a long request draws in many heads.

Requests share one cache, so that a batch is large enough for a column of the kernel's grid to take whole requests: where
a request is divided, each part has its own maximum.

Tolerance: tests/_parity.py's bar.  A weight of P V is within 2^-8 of itself, so that the tail's part of the output is
within 2^-8 of its own size and the output's rounding comes to 2^-9 more: 0.6% of the row's largest value at most."""
import numpy as np
import pytest
import torch

import oracle
from _parity import check_attention
from _spec import cast
from _window import attend, block_scale
from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import workloads as wl

pytestmark = pytest.mark.gpu

DEV = "cuda"
BS = 64


def _d(a, dtype=None):
    t = torch.from_numpy(np.ascontiguousarray(a))
    return (t.view(dtype) if dtype is not None else t).to(DEV)


def _codes(x, scale_of):
    """E4M3 codes of x (blocks, BS, hkv, d) with a scale a block and head, scale_of(largest) of its rows; their values."""
    top = np.abs(x).max((1, 3))
    scales = np.vectorize(scale_of)(top).astype(np.float32)
    codes = oracle.e4m3_encode((x / scales[:, None, :, None]).astype(np.float32))
    return codes, scales, oracle.e4m3_decode(codes) * scales[:, None, :, None].astype(np.float64)


class Tail:
    """One cache of L positions that every request of the batch reads: the key at position `at` has about `share` of the
    weight, all others' scores lie within a factor of about 1.4.  values: "mean" of 0.5 and deviation 1, "constant", or
    "blocks", the same in blocks whose largest values are a factor of up to 2^12 apart, the heavy key's among the large;
    the heavy key's own are next to nothing but for constant ones."""

    def __init__(self, L, share, t, hq, hkv, d, values, at=0, seed=0, window=0, sinks=0, fp8=True):
        rng = np.random.default_rng(seed)
        n = -(-L // BS)
        self.L, self.t, self.window, self.sinks, self.fp8 = L, t, window, sinks, fp8
        q = rng.standard_normal((t, hq, d)) * 0.2
        q[..., :8] = 2.0                                             # one direction that all queries share
        self.q = cast(q.astype(np.float32), "bf16")
        k = rng.standard_normal((n, BS, hkv, d)) * 0.15
        k[..., :8] *= 0.5
        seen = min(L, window + sinks) if window else L
        want = np.log(share / (1 - share) * seen * 1.06)             # the heavy key's score above the others'
        k[at // BS, at % BS] = 0.0
        k[at // BS, at % BS, :, :8] = want * d ** 0.5 / 16
        v = rng.standard_normal((n, BS, hkv, d)) + 0.5
        if values == "constant":
            v[:] = 0.75
        else:
            v[at // BS, at % BS] *= 2.0 ** -10
        if values == "blocks":
            v *= np.exp2(-rng.integers(0, 13, (n, 1, hkv, 1)))
            v[at // BS] *= 2.0 ** 6
        self.k, self.ks, keys = _codes(k, block_scale_of)
        self.v, self.vs, vals = _codes(v, block_scale_of)
        if not fp8:
            self.k, self.v = (cast(x.astype(np.float32), "bf16") for x in (k, v))
            keys, vals = (wl.to_f32(x).astype(np.float64) for x in (self.k, self.v))
        self.want = attend(wl.to_f32(self.q).astype(np.float64), keys.reshape(-1, hkv, d)[:L], vals.reshape(-1, hkv, d)[:L],
                           L, True, window, sinks)

    def run(self, reqs, bound=None):
        t, hq, d = self.q.shape
        n, _, hkv, _ = self.k.shape
        # block 0 is the null block: ids from 1 on
        k, v = (torch.cat([x[:1], x]) for x in (_d(self.k, None if self.fp8 else torch.bfloat16),
                                                _d(self.v, None if self.fp8 else torch.bfloat16)))
        scales = [torch.cat([x[:1], x]) for x in (_d(self.ks), _d(self.vs))]
        table = torch.arange(1, n + 1, dtype=torch.int32, device=DEV).expand(reqs, n).contiguous()
        ctx = torch.full((reqs,), self.L, dtype=torch.int32, device=DEV)
        q = _d(self.q, torch.bfloat16).expand(reqs, t, hq, d).contiguous()
        out, err = torch.full_like(q, 9.0), torch.zeros(1, dtype=torch.int32, device=DEV)
        ws = bkv.alloc_window_workspace(reqs, t, hq, hkv, d, BS, bound or self.L)
        if self.fp8:
            bkv.bkv_paged_decode_fp8_blocks(q, k, v, *scales, table, ctx, bound or self.L, out, ws, self.window,
                                            self.sinks, err_count=err)
        else:
            bkv.bkv_paged_decode_sink(q, k, v, table, ctx, bound or self.L, out, ws, self.window, self.sinks, err_count=err)
        got = out.float().cpu().numpy().astype(np.float64)
        assert int(err) == 0
        return got

    def check(self, reqs, bound=None):
        got = self.run(reqs, bound)
        for r in range(reqs):
            check_attention(got[r], self.want, "bf16", f"request {r}")


def block_scale_of(top):
    return block_scale(np.array([top]))


@pytest.mark.parametrize("values", ["mean", "constant", "blocks"])
@pytest.mark.parametrize("share", [0.5, 0.9, 0.99])
@pytest.mark.parametrize("L,reqs", [(1028, 160), (4100, 160), (8192, 160), (32768, 100)])
def test_one_heavy_key_and_a_long_flat_tail(L, reqs, share, values):
    Tail(L, share, 1, 8, 2, 128, values).check(reqs)


@pytest.mark.parametrize("t,hq", [(1, 2), (1, 16), (2, 16), (4, 8)])
@pytest.mark.parametrize("d", [128, 64])
def test_query_rows_and_head_sizes(t, hq, d):
    """One row a KV head and groups of 8 and 16, several tokens; heads of 64 run on the CUDA cores."""
    Tail(8192, 0.9, t, hq, 2, d, "mean", seed=t).check(100)


@pytest.mark.parametrize("fp8", [True, False])
@pytest.mark.parametrize("window,sinks", [(4096, 4), (8000, 64)])
def test_windows_beside_a_heavy_first_token(fp8, window, sinks):
    Tail(20000, 0.9, 2, 16, 2, 128, "mean", window=window, sinks=sinks, fp8=fp8).check(160)
    Tail(20000, 0.97, 1, 8, 2, 128, "constant", window=window, sinks=sinks, fp8=fp8).check(160)


@pytest.mark.parametrize("at", [700, 8191])
def test_a_heavy_key_behind_the_tail(at):
    """The reference moves after most of the tail has been summed."""
    Tail(8192, 0.9, 1, 8, 2, 128, "mean", at=at).check(160)


@pytest.mark.parametrize("share", [0.5, 0.9])
def test_the_longest_tail(share):
    """131072 positions whole and divided among columns, and one request alone."""
    p = Tail(131072, share, 1, 4, 1, 128, "mean")
    p.check(1)
    p.check(160)


@pytest.mark.parametrize("t,hq", [(1, 8), (4, 8)])
def test_bounds_of_long_caches(t, hq):
    """A bound on the lengths from which the kernel holds small weights more finely; the requests are short."""
    for bound in (1 << 22, (1 << 22) + 1, 1 << 26):
        Tail(8192, 0.9, t, hq, 2, 128, "mean", seed=3).check(100, bound)

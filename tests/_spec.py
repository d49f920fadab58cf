"""Inputs of the speculative step's tests: small paged caches, random trees,
probabilities, as numpy arrays (bf16 as uint16 bits)."""
import numpy as np

from paged_kv_cache_slot_gb300 import workloads as wl


def cast(x, dtype):
    return wl.f32_to_bf16_bits(x) if dtype == "bf16" else np.ascontiguousarray(x, np.float32)


def nan_like(shape, dtype):
    return np.full(shape, 0x7FC0, np.uint16) if dtype == "bf16" else np.full(shape, np.nan, np.float32)


def parents(rng, reqs, t, bushy=1.5):
    """Random trees: parents (reqs, t) int32, each before its child, the root's -1."""
    par = np.full((reqs, t), -1, np.int32)
    for i in range(1, t):
        par[:, i] = np.minimum((rng.random(reqs) ** bushy * i).astype(np.int32), i - 1)
    return par


def ancestors(par):
    """bool (reqs, t, t): [r, t, i] whether i is t or an ancestor of t."""
    reqs, t = par.shape
    anc = np.zeros((reqs, t, t), bool)
    for r in range(reqs):
        for i in range(t):
            if par[r, i] >= 0:
                anc[r, i] = anc[r, par[r, i]]
            anc[r, i, i] = True
    return anc


def words(mask):
    """uint32 words (.., t, ceil(t / 32)) of a bool mask (.., t, t)."""
    t = mask.shape[-1]
    w = -(-t // 32)
    bits = np.zeros(mask.shape[:-1] + (w * 32,), np.uint64)
    bits[..., :t] = mask
    return (bits.reshape(mask.shape[:-1] + (w, 32)) << np.arange(32, dtype=np.uint64)).sum(-1).astype(np.uint32)


class Paged:
    """Requests of the given cache lengths in a paged cache whose unwritten memory is NaN."""

    def __init__(self, lens, t, hq, hkv, d, bs, dtype="bf16", seed=0, holes=(), width=None):
        rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        need = -(-self.lens // bs)
        total = 1 + int(need.sum()) + 3
        ids = rng.permutation(np.arange(1, total))[: int(need.sum())]
        self.table = np.full((len(lens), int(need.max(initial=0)) + 2 if width is None else width), -1, np.int32)
        self.k = nan_like((total, bs, hkv, d), dtype)
        self.v = nan_like((total, bs, hkv, d), dtype)
        at = 0
        for r, n in enumerate(need):
            mine = ids[at:at + n]
            at += n
            cols = min(n, self.table.shape[1])
            self.table[r, :cols] = mine[:cols]
            for b in range(n):
                rows = min(bs, self.lens[r] - b * bs)
                self.k[mine[b], :rows] = cast(rng.standard_normal((rows, hkv, d), np.float32) * 1.4, dtype)
                self.v[mine[b], :rows] = cast(rng.standard_normal((rows, hkv, d), np.float32), dtype)
        for r, b in holes:
            self.table[r, b] = (r + b) % 2 - 1     # a null entry, 0 or -1
        self.q = cast(rng.standard_normal((len(lens), t, hq, d), np.float32) * 1.4, dtype)
        self.dtype, self.total, self.bs, self.d = dtype, total, bs, d

    def rows(self, r, pos):
        """Flat cache row of position pos of request r."""
        return self.table[r, pos // self.bs] * self.bs + pos % self.bs


def probs(rng, shape, spread=2.5):
    """Rows of probabilities (fp32) along the last axis."""
    x = rng.standard_normal(shape).astype(np.float64) * spread
    x = np.exp(x - x.max(-1, keepdims=True))
    return (x / x.sum(-1, keepdims=True)).astype(np.float32)


def draws(rng, p):
    """One token of each row of p (.., V)."""
    flat = p.reshape(-1, p.shape[-1]).astype(np.float64)
    c = flat.cumsum(-1)
    x = rng.random(len(flat)) * c[:, -1]
    return (c > x[:, None]).argmax(-1).reshape(p.shape[:-1]).astype(np.int64)


def rope_table(n, rot, base=10000.0):
    half = rot // 2
    ang = np.arange(n)[:, None] * base ** (-np.arange(half) / max(half, 1))
    return np.concatenate([np.cos(ang), np.sin(ang)], 1).astype(np.float32)

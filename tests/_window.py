"""Inputs and plain 64-bit forms for the tests of step building, block-scaled E4M3
caches and windows whose first tokens stay visible (numpy; bf16 as uint16 bits)."""
import numpy as np

import oracle
from _spec import cast, nan_like
from paged_kv_cache_slot_gb300 import workloads as wl


def build_step(cached, new, free, bs, table, max_tokens):
    """bkv_build_step, request after request: table, context_lens, query_start_loc, req, pos, slots, used, errors."""
    table = table.copy()
    cols = table.shape[1]
    ctx, qsl, req, pos, slots, used, err = [], [0], [], [], [], 0, 0
    for r, (c, n) in enumerate(zip(cached.tolist(), new.tolist())):
        big = 2 ** 31 - 1
        if c < 0 or n < 0 or max(c, 0) + n > big:
            err += 1
            c = max(c, 0)
            n = min(max(n, 0), big - c)
        have, blocks = -(-c // bs), -(-(c + n) // bs)
        if n > 0 and blocks > cols:
            err += 1
        table[r, have:] = -1
        for j in range(have, min(blocks, cols)):
            if used < len(free):
                table[r, j] = free[used]
            else:
                err += 1
            used += 1
        ctx.append(c + n)
        qsl.append(min(qsl[-1] + n, big))
        for p in range(c, min(c + n, c + max_tokens + 1)):
            b = int(table[r, p // bs]) if p // bs < cols else -1
            req.append(r)
            pos.append(p)
            slots.append(b * bs + p % bs if b > 0 else -1)
    if len(req) > max_tokens:
        err += 1
    pad = max(0, max_tokens - len(req))
    cut = slice(0, max_tokens)
    return (table, np.array(ctx, np.int32), np.array(qsl, np.int32), np.array((req + [-1] * pad)[cut], np.int32),
            np.array((pos + [0] * pad)[cut], np.int64), np.array((slots + [-1] * pad)[cut], np.int64),
            min(used, len(free)), err)


def block_scale(x):
    """The smallest power of two s with max |x| <= 448 s over the finite x, its exponent in [-40, 40]."""
    x = np.abs(x.astype(np.float64))
    x = x[np.isfinite(x)]
    top = x.max(initial=0.0)
    for e in range(-40, 41):
        if top <= 448.0 * 2.0 ** e:
            return 2.0 ** e
    return 2.0 ** 40


def write_blocks(k_new, v_new, qsl, ctx, table, bs, k_cache, v_cache, k_scales, v_scales):
    """bkv_cache_write_fp8_blocks in place, block after block; the number of errors."""
    err, total = 0, len(k_cache)
    for r in range(len(ctx)):
        n = int(qsl[r + 1] - qsl[r])
        start = int(ctx[r]) - n
        if n > 0 and start < 0:
            err += 1
            continue
        p = start
        while p < ctx[r]:
            m = min(bs - p % bs, int(ctx[r]) - p)
            lb, first, tok = p // bs, p % bs, int(qsl[r]) + p - start
            p += m
            b = int(table[r, lb]) if lb < table.shape[1] else total
            if b >= total:
                err += 1
            if b <= 0 or b >= total:
                continue
            for new, cache, scales in ((k_new, k_cache, k_scales), (v_new, v_cache, v_scales)):
                x = wl.to_f32(new[tok:tok + m])
                for h in range(cache.shape[2]):
                    s, old = block_scale(x[:, h]), float(scales[b, h])
                    if first > 0 and np.isfinite(old) and old > 0:
                        if old >= s:
                            s = old
                        else:
                            held = oracle.e4m3_decode(cache[b, :first, h]) * (old / s)
                            cache[b, :first, h] = oracle.e4m3_encode(held.astype(np.float32))
                    scales[b, h] = s
                    with np.errstate(over="ignore"):
                        cache[b, first:first + m, h] = oracle.e4m3_encode((x[:, h].astype(np.float64) / s).astype(np.float32))
    return err


def visible(L, q_len, t, causal, window, sinks):
    """Positions of a request of length L that its query token t sees."""
    p = L - q_len + t
    j = np.arange(L)
    see = j <= (p if causal else L - 1)
    if window:
        see &= (j > p - window) | (j < sinks)
    return j[see]


def attend(q, keys, values, L, causal=True, window=0, sinks=0, scale=None, there=None):
    """Output rows (q_len, H_q, D) of one request in 64 bits: q (q_len, H_q, D), keys / values (L, H_kv, D) float64;
    there (L): whether a position's block entry is a real block."""
    ql, hq, d = q.shape
    hkv = keys.shape[1]
    g = hq // hkv
    scale = d ** -0.5 if scale is None else scale
    out = np.zeros((ql, hq, d))
    for t in range(ql):
        j = visible(L, ql, t, causal, window, sinks)
        if there is not None:
            j = j[there[j]]
        if not len(j):
            continue
        for h in range(hkv):
            s = (q[t, h * g:(h + 1) * g] @ keys[j, h].T) * scale
            w = np.exp(s - s.max(-1, keepdims=True))
            out[t, h * g:(h + 1) * g] = (w @ values[j, h]) / w.sum(-1, keepdims=True)
    return out


class Blocks:
    """Requests of the given lengths in a paged cache whose unwritten memory is NaN: bf16 or fp32, or E4M3 codes with a
    scale a block and head (fp8).  Blocks that lie wholly outside the first ``keep`` and the last ``window`` positions
    (with the step's q_len) are not there: their entries are null and nothing was written."""

    def __init__(self, lens, t, hq, hkv, d, bs, dtype="bf16", fp8=False, seed=0, window=0, sinks=0, holes=(), spread=2.0,
                 pow2=True):
        rng = np.random.default_rng(seed)
        self.lens = np.array(lens, np.int32)
        need = -(-self.lens // bs)
        total = 1 + int(need.sum()) + 3
        ids = rng.permutation(np.arange(1, total))[: int(need.sum())]
        self.table = np.full((len(lens), int(need.max(initial=0)) + 2), -1, np.int32)
        shape = (total, bs, hkv, d)
        if fp8:
            self.k, self.v = (np.full(shape, 0x7F, np.uint8) for _ in range(2))
        else:
            self.k, self.v = (nan_like(shape, dtype) for _ in range(2))
        self.ks, self.vs = (np.full((total, hkv), np.nan, np.float32) for _ in range(2))
        self.keys, self.values, self.there = [], [], []
        at = 0
        for r, n in enumerate(need):
            L = int(self.lens[r])
            keys, values = (np.zeros((L, hkv, d)) for _ in range(2))
            there = np.zeros(L, bool)
            lo = max(0, L - t - window + 1) if window else 0
            for b in range(n):
                i = ids[at + b]
                rows = min(bs, L - b * bs)
                if window and b * bs >= sinks and (b + 1) * bs <= lo:
                    continue
                self.table[r, b] = i
                part = slice(b * bs, b * bs + rows)
                there[part] = True
                for cache, scales, to, amp in ((self.k, self.ks, keys, 1.4), (self.v, self.vs, values, 1.0)):
                    x = rng.standard_normal((rows, hkv, d)).astype(np.float32) * np.float32(amp)
                    if fp8:
                        if to is values:
                            x *= np.exp2(spread * (2 * rng.random((1, hkv, 1)) - 1)).astype(np.float32)
                        s = np.array([block_scale(x[:, h]) for h in range(hkv)], np.float32)
                        if not pow2:
                            s *= (1 + rng.random(hkv)).astype(np.float32)
                        scales[i] = s
                        cache[i, :rows] = oracle.e4m3_encode(x / s[:, None])
                        to[part] = oracle.e4m3_decode(cache[i, :rows]) * s[:, None].astype(np.float64)
                    else:
                        cache[i, :rows] = cast(x, dtype)
                        to[part] = wl.to_f32(cache[i, :rows])
            at += n
            self.keys.append(keys)
            self.values.append(values)
            self.there.append(there)
        for r, b in holes:
            self.table[r, b] = (r + b) % 2 - 1     # a null entry, 0 or -1
            self.there[r][b * bs:(b + 1) * bs] = False
        self.q = cast(rng.standard_normal((len(lens), t, hq, d)).astype(np.float32) * np.float32(1.4), dtype)
        self.dtype, self.total, self.bs, self.d, self.fp8 = dtype, total, bs, d, fp8
        self.window, self.sinks = window, sinks

    def want(self, r, causal=True, scale=None):
        return attend(wl.to_f32(self.q[r]).astype(np.float64), self.keys[r], self.values[r], int(self.lens[r]), causal,
                      self.window, self.sinks, scale, self.there[r])

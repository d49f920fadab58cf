"""The operators of a serving step over an 8-bit paged cache and over sliding-window layers, as they are measured.

A step hands out the blocks that its new tokens need and lists the tokens with their slots (``step``), writes their keys
and values as E4M3 codes with one scale for each block of tokens and head (``write``), and attends over such a cache
(``attn8``), or over a bf16 / fp32 one in a layer with a sliding window whose first tokens stay visible (``sink``).
``run`` does one of these in elementary torch operations, or, where ``own`` is set, through the calls of
``paged_kv_cache_slot_gb300.bkv``.
"""
import math

import torch

own = False

NEG = float("-inf")
TOP = 448.0        # E4M3's largest value
EXP_MIN, EXP_MAX = -40, 40   # exponents that a block's scale may have


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # -- block tables, token lists and slots from the requests' lengths (op "step") --
        # a decode step of 32 requests, a token each: launch latency counts
        dict(name="step_decode", op="step", reqs=32, pad=0, singles=32, new_lo=0, new_hi=0, prior_hi=4096, one=1, bs=64,
             cols=65, pad_tokens=0),
        # 256 speculating requests (1 + 3 tokens) in a batch padded to 320 rows, blocks of 16
        dict(name="step_spec", op="step", reqs=256, pad=64, singles=256, new_lo=0, new_hi=0, prior_hi=8192, one=4, bs=16,
             cols=514, pad_tokens=256),
        # 4096 rows of up to 2048 blocks, decode tokens beside prompt chunks: bandwidth counts
        dict(name="step_large", op="step", reqs=4096, pad=0, singles=3840, new_lo=64, new_hi=1024, prior_hi=16384, one=1,
             bs=16, cols=2048, pad_tokens=100),
        # -- writes into an E4M3 cache with a scale a block and head (op "write") --
        # a decode step of 256 requests
        dict(name="write_decode", op="write", reqs=256, singles=256, new_lo=0, new_hi=0, prior_hi=8192, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # a mixed step of 48 decode tokens and 16 prompt chunks of 64..1024 tokens
        dict(name="write_step", op="write", reqs=64, singles=48, new_lo=64, new_hi=1024, prior_hi=2048, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # 32 whole prompts: the largest
        dict(name="write_prompt", op="write", reqs=32, singles=0, new_lo=512, new_hi=4096, prior_hi=1, hkv=8, d=128, bs=64,
             dtype="bf16"),
        # -- attention over that cache (op "attn8") --
        # one request with a short context: the latency of a chat with one user
        dict(name="attn8_one", op="attn8", reqs=1, lo=700, hi=700, t=1, hq=32, hkv=8, d=128, bs=64, dtype="bf16", window=0,
             sinks=0),
        # a decode step of 32 requests of 512..4096 tokens
        dict(name="attn8_batch", op="attn8", reqs=32, lo=512, hi=4096, t=1, hq=32, hkv=8, d=128, bs=64, dtype="bf16",
             window=0, sinks=0),
        # 8 long requests with 64 query heads and 1 + 1 tokens: the most bytes
        dict(name="attn8_long", op="attn8", reqs=8, lo=4000, hi=131071, t=2, hq=64, hkv=8, d=128, bs=64, dtype="bf16",
             window=0, sinks=0),
        # -- sliding window with first tokens that stay visible (op "sink") --
        # one long conversation through a window of 1024
        dict(name="sink_one", op="sink", reqs=1, lo=100003, hi=100003, t=1, hq=32, hkv=8, d=128, bs=64, dtype="bf16",
             window=1024, sinks=4),
        # 256 speculating requests of very mixed lengths through a window of 2048, blocks of 16
        dict(name="sink_batch", op="sink", reqs=256, lo=9, hi=16384, t=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16",
             window=2048, sinks=4),
        # fp32 caches with small heads, an odd group, an odd number of requests and a sink that ends inside a block
        dict(name="sink_f32", op="sink", reqs=13, lo=33, hi=5000, t=1, hq=15, hkv=5, d=64, bs=16, dtype="f32", window=777,
             sinks=21),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step", "write", "write", "attn8", "attn8", "attn8", "sink", "sink"])
    bs = rng.choice([16, 32, 64])
    if op == "step":
        reqs = _log(rng, 1, 2000)
        lo = _log(rng, 1, 64)
        prior = _log(rng, 16, 16000)
        one = rng.choice([1, 1, 4, 7])
        hi = lo + _log(rng, 1, 500)
        return dict(op="step", reqs=reqs, pad=rng.choice([0, 0, 1, 17]), singles=rng.randint(reqs * 3 // 4, reqs), new_lo=lo,
                    new_hi=hi, prior_hi=prior, one=one, bs=bs, cols=-(-(prior + max(hi, one)) // bs) + rng.randint(0, 40),
                    pad_tokens=rng.choice([0, 1, 19]))
    if op == "write":
        reqs = _log(rng, 1, 200)
        lo = _log(rng, 1, 64)
        return dict(op="write", reqs=reqs, singles=rng.randint(reqs // 2, reqs), new_lo=lo, new_hi=lo + _log(rng, 1, 900),
                    prior_hi=_log(rng, 16, 3000), hkv=rng.choice([1, 2, 5, 8]), d=rng.choice([64, 128, 128, 128, 256]),
                    bs=bs, dtype=rng.choice(["bf16", "bf16", "f32"]))
    plain = rng.random() < 0.25   # other types and head sizes
    hkv = rng.choice([1, 2, 4, 5, 8])
    g = rng.choice([1, 3, 4, 4, 7, 8])
    reqs = _log(rng, 1, 16 if plain else 64)
    hi = _log(rng, 200, 3000 if plain else 60000 if reqs <= 8 else 6000)
    t = 1 if rng.random() < 0.5 else rng.randint(2, 5)
    windowed = op == "sink" or rng.random() < 0.3
    return dict(op=op, reqs=reqs, lo=t + _log(rng, 1, hi // 4), hi=hi + t, t=t, hq=hkv * g, hkv=hkv,
                d=rng.choice([64, 128, 256]) if plain else 128, bs=bs, dtype=rng.choice(["bf16", "f32"]) if plain else "bf16",
                window=_log(rng, 16, 5000) if windowed else 0, sinks=rng.choice([0, 1, 4, 21, 64]) if windowed else 0)


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------
def _gen(seed, salt):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed * 16 + salt)
    return g


def _dtype(case):
    return torch.bfloat16 if case["dtype"] == "bf16" else torch.float32


def _spread(n, lo, hi):
    """n lengths spread over [lo, hi] in equal steps of their logarithm (their sum is the case's, not the seed's)."""
    if n == 0:
        return []
    if lo >= hi:
        return [lo] * n
    return [int(round(lo * (hi / lo) ** ((i + 0.5) / n))) for i in range(n)]


def _news(case):
    n = case["reqs"] - case["singles"]
    step = (case["new_hi"] - case["new_lo"]) / max(1, n - 1)
    return [case.get("one", 1)] * case["singles"] + [case["new_lo"] + int(i * step) for i in range(n)]


def _shuffled(values, seed):
    order = torch.randperm(len(values), generator=torch.Generator().manual_seed(seed)).tolist()
    return [values[i] for i in order]


def _tables(lens, bs, g, cols=None):
    """Block tables of requests of these lengths: ids a permutation of 1..total-1, unused entries -1.  The pool's size
    follows from the lengths' sum.  Also the ids that no request has."""
    need = torch.tensor([-(-n // bs) for n in lens])
    most = sum(lens) // bs + len(lens)
    total = most + most // 4 + 2
    ids = (torch.randperm(total - 1, generator=g, device="cuda") + 1).to(torch.int32)
    cols = int(need.max()) + 1 if cols is None else cols
    at = torch.arange(cols)[None] < need[:, None]
    table = torch.full((len(lens), cols), -1, dtype=torch.int32, device="cuda")
    table[at.cuda()] = ids[:int(need.sum())]
    return table, total, ids[int(need.sum()):]


def _prepare_step(c, seed):
    g = _gen(seed, 1)
    news, rows = _news(c) + [0] * c["pad"], c["reqs"] + c["pad"]
    prior = _shuffled(_spread(c["reqs"], 1, c["prior_hi"]), seed) + [0] * c["pad"]
    table, total, free = _tables(prior, c["bs"], g, c["cols"])
    extra = sum(news) // c["bs"] + rows
    free = torch.cat([free, torch.arange(total, total + extra, dtype=torch.int32, device="cuda")])
    n = sum(news) + c["pad_tokens"]

    def ints(*shape, dtype=torch.int32):
        return torch.zeros(shape, dtype=dtype, device="cuda")

    return dict(c, cached=torch.tensor(prior, dtype=torch.int32, device="cuda"),
                new=torch.tensor(news, dtype=torch.int32, device="cuda"), free=free, table=table, ctx=ints(rows),
                qsl=ints(rows + 1), req=ints(n), pos=ints(n, dtype=torch.int64), slots=ints(n, dtype=torch.int64),
                used=ints(1))


def _amplitudes(shape, g):
    """Sizes that rows of one head or block have beside one another's: a factor of 4 either way."""
    return torch.exp2(4 * torch.rand(shape, generator=g, device="cuda") - 2)


def _prepare_write(c, seed):
    g = _gen(seed, 2)
    dt = _dtype(c)
    news = _news(c)
    prior = _shuffled(_spread(c["reqs"], 1, c["prior_hi"]), seed)
    lens = [p + m for p, m in zip(prior, news)]
    table, total, _ = _tables(lens, c["bs"], g)
    n, row = sum(news), c["hkv"] * c["d"]
    # keys and values lie in one projection beside the queries
    kv = torch.randn(n, 2 * row + 128, generator=g, device="cuda", dtype=dt)
    kv[:, :2 * row].view(n, 2 * c["hkv"], c["d"]).mul_(_amplitudes((n, 2 * c["hkv"], 1), g).to(dt))
    scales = [_two_to(torch.randint(-10, -6, (total, c["hkv"]), generator=g, device="cuda")) for _ in range(2)]
    # codes of finite values
    caches = [torch.randint(0, 0x7F, (total, c["bs"], c["hkv"], c["d"]), generator=g, device="cuda", dtype=torch.uint8)
              for _ in range(2)]
    qsl = [0]
    for m in news:
        qsl.append(qsl[-1] + m)
    return dict(c, k=kv[:, :row].view(n, c["hkv"], c["d"]), v=kv[:, row:2 * row].view(n, c["hkv"], c["d"]), table=table,
                qsl=torch.tensor(qsl, dtype=torch.int32, device="cuda"),
                ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"), k_cache=caches[0], v_cache=caches[1],
                k_scales=scales[0], v_scales=scales[1])


def _lens(case):
    return _spread(case["reqs"], case["lo"], case["hi"])


def _scale_of(top):
    """The smallest power of two s with top <= 448 s, its exponent held to what a scale may have."""
    m, e = torch.frexp(top)
    return _two_to((e - 9 + (m > 0.875).int()).clamp(EXP_MIN, EXP_MAX))


def _two_to(e):
    """2^e exactly, by the number's bits (torch's own powers are an ulp off for some e)."""
    return ((e.int() + 127) << 23).view(torch.float32)


def _prepare_attn(c, seed):
    g = _gen(seed, 3)
    dt = _dtype(c)
    lens = _shuffled(_lens(c), seed)
    table, total, _ = _tables(lens, c["bs"], g)
    cache = (total, c["bs"], c["hkv"], c["d"])
    # scores of standard deviation 2, so that some keys matter much more than others
    q = torch.randn(c["reqs"], c["t"], c["hq"], c["d"], generator=g, device="cuda").mul_(2 ** 0.5).to(dt)
    kt = torch.float32 if c["op"] == "attn8" else dt
    k = torch.randn(cache, generator=g, device="cuda", dtype=kt).mul_(2 ** 0.5)
    v = torch.randn(cache, generator=g, device="cuda", dtype=kt)
    st = dict(c, q=q, table=table, ctx=torch.tensor(lens, dtype=torch.int32, device="cuda"), max_ctx=max(lens),
              out=torch.zeros_like(q), workspace=_Workspace((c["reqs"], c["t"], c["hq"], c["hkv"], c["d"], c["bs"], max(lens))))
    if c["op"] == "sink":
        return dict(st, k_cache=k, v_cache=v)
    v.mul_(_amplitudes((total, 1, c["hkv"], 1), g))
    for name, x in (("k", k), ("v", v)):
        scale = _scale_of(x.abs().amax((1, 3)))
        st[name + "_scales"] = scale
        st[name + "_cache"] = (x / scale[:, None, :, None]).to(torch.float8_e4m3fn).view(torch.uint8)
    return st


class _Workspace:
    """Scratch memory that a program keeps for its calls, made at the first of them."""

    def __init__(self, sizes):
        self.sizes, self.mem = sizes, None

    def get(self, bkv):
        if self.mem is None:
            self.mem = bkv.alloc_window_workspace(*self.sizes)
        return self.mem


def prepare(case, seed):
    return {"step": _prepare_step, "write": _prepare_write, "attn8": _prepare_attn, "sink": _prepare_attn}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# One pass, plain
# ---------------------------------------------------------------------------
def _plain_step(s):
    bs, table = s["bs"], s["table"]
    rows, cols = table.shape
    dev = table.device
    cached, new = s["cached"].long(), s["new"].long()
    ctx = cached + new
    have = (cached + bs - 1) // bs
    need = (((ctx + bs - 1) // bs).clamp_max(cols) - have).clamp_min(0)
    run = need.cumsum(0)
    j = torch.arange(cols, device=dev)[None]
    fresh = (j >= have[:, None]) & (j < (have + need)[:, None])
    at = ((run - need - have)[:, None] + j).clamp(0, s["free"].numel() - 1)
    table = torch.where(fresh, s["free"][at], torch.where(j < have[:, None], table, -1))
    ends = new.cumsum(0)
    i = torch.arange(s["slots"].numel(), device=dev)
    req = torch.searchsorted(ends, i, right=True)
    real = req < rows
    req = req.clamp_max(rows - 1)
    pos = torch.where(real, i - (ends - new)[req] + cached[req], 0)
    block = table[req, pos // bs].long()
    slots = torch.where(real & (block > 0), block * bs + pos % bs, -1)
    qsl = torch.cat([torch.zeros_like(ends[:1]), ends])
    return (table, ctx.int(), qsl.int(), torch.where(real, req, -1).int(), pos, slots, run[-1:].int())


def _token_places(s):
    """Of every new token: its cache row and block; of every (token, block) pair whether the block is begun by it."""
    n = s["k"].shape[0]
    i = torch.arange(n, device=s["k"].device)
    req = torch.searchsorted(s["qsl"][1:].long(), i, right=True)
    start, ctx = s["qsl"].long()[req], s["ctx"].long()[req]
    end = s["qsl"].long()[req + 1]
    pos = ctx - (end - start) + i - start
    block = s["table"][req, pos // s["bs"]].long()
    return block, pos % s["bs"]


def _plain_write(s):
    bs = s["bs"]
    total = s["k_cache"].shape[0]
    block, off = _token_places(s)
    n = block.numel()
    # the first row of each block that is written, where it is one of this step's (bs: none)
    first = torch.full((total,), bs, dtype=torch.int64, device=block.device).scatter_reduce_(0, block, off, "amin")
    got = []
    for new, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        x = new.float()
        top = torch.zeros_like(scales).scatter_reduce_(0, block[:, None].expand(n, s["hkv"]), x.abs().amax(-1), "amax")
        now = torch.where((first == bs)[:, None], scales, _scale_of(top))
        now = torch.where(((first > 0) & (first < bs))[:, None], torch.maximum(now, scales), now)
        # rows that the block held before, in the units of its scale now
        ids = block[off == first[block]]
        old = cache[ids].view(torch.float8_e4m3fn).float() * (scales[ids] / now[ids])[:, None, :, None]
        keep = torch.arange(bs, device=ids.device)[None] < first[ids][:, None]
        cache[ids] = torch.where(keep[:, :, None, None], old.to(torch.float8_e4m3fn).view(torch.uint8), cache[ids])
        cache[block, off] = (x / now[block][..., None]).clamp(-TOP, TOP).to(torch.float8_e4m3fn).view(torch.uint8)
        scales.copy_(now)
        got += [cache.view(torch.float8_e4m3fn), scales]
    return tuple(got)


def _seen_positions(s):
    """Positions that some query token of a request may see, as (R, n) with those past its end among them."""
    ctx, t, w = s["ctx"].long(), s["t"], s["window"]
    if w == 0:
        return torch.arange(s["max_ctx"], device=ctx.device)[None].expand(s["reqs"], -1)
    begin = (ctx - t - w + 1).clamp_min(0)
    n = min(w + t - 1, s["max_ctx"])
    near = begin[:, None] + torch.arange(n, device=ctx.device)[None]
    first = torch.arange(s["sinks"], device=ctx.device)[None].expand(s["reqs"], -1)
    # a first token inside the window stands there already: put past the end here
    return torch.cat([torch.where(first < begin[:, None], first, 1 << 40), near], 1)


def _plain_attn(s):
    r, t, hq, d = s["q"].shape
    hkv, bs, g = s["hkv"], s["bs"], s["hq"] // s["hkv"]
    ctx = s["ctx"].long()
    j = _seen_positions(s)                                          # (r, n)
    n = j.shape[1]
    inside = j < ctx[:, None]
    at = torch.where(inside, j, 0)
    block = torch.gather(s["table"].long(), 1, at // bs)
    inside = inside & (block > 0)
    block = block.clamp_min(0)
    row = block * bs + at % bs
    k, v = (s[x].view(-1, hkv, d)[row] for x in ("k_cache", "v_cache"))       # (r, n, hkv, d)
    if s["op"] == "attn8":
        k = k.view(torch.float8_e4m3fn).float() * s["k_scales"][block][..., None]
        v = v.view(torch.float8_e4m3fn).float() * s["v_scales"][block][..., None]
    k = k.permute(0, 2, 3, 1).float()
    v = torch.where(inside[..., None, None], v, 0.0).permute(0, 2, 1, 3).float()
    q = s["q"].float().view(r, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(r, hkv, t * g, d)
    scores = (q @ k).view(r, hkv, t, g, n) / math.sqrt(d)
    own_pos = ctx[:, None] - t + torch.arange(t, device=ctx.device)[None]      # (r, t)
    seen = inside[:, None] & (j[:, None] <= own_pos[..., None])
    if s["window"]:
        seen = seen & ((j[:, None] > own_pos[..., None] - s["window"]) | (j[:, None] < s["sinks"]))
    scores = scores.masked_fill(~seen[:, None, :, None, :], NEG)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    w = torch.exp(scores - top)
    w = (w / w.sum(-1, keepdim=True).clamp_min(1e-37)).view(r, hkv, t * g, n)
    out = (w @ v).view(r, hkv, t, g, d).permute(0, 2, 1, 3, 4).reshape(r, t, hq, d)
    return out.to(s["q"].dtype)


# ---------------------------------------------------------------------------
# One pass, through the framework
# ---------------------------------------------------------------------------
def _own(s):
    from paged_kv_cache_slot_gb300 import bkv

    if s["op"] == "step":
        return bkv.bkv_build_step(s["cached"], s["new"], s["free"], s["bs"], s["table"], s["ctx"], s["qsl"], s["req"],
                                  s["pos"], s["slots"], s["used"])
    if s["op"] == "write":
        bkv.bkv_cache_write_fp8_blocks(s["k"], s["v"], s["qsl"], s["ctx"], s["table"], s["k_cache"], s["v_cache"],
                                       s["k_scales"], s["v_scales"])
        return (s["k_cache"].view(torch.float8_e4m3fn), s["k_scales"], s["v_cache"].view(torch.float8_e4m3fn), s["v_scales"])
    if s["op"] == "attn8":
        return bkv.bkv_paged_decode_fp8_blocks(s["q"], s["k_cache"], s["v_cache"], s["k_scales"], s["v_scales"], s["table"],
                                               s["ctx"], s["max_ctx"], s["out"], s["workspace"].get(bkv),
                                               sliding_window=s["window"], num_sinks=s["sinks"])
    return bkv.bkv_paged_decode_sink(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["max_ctx"], s["out"],
                                     s["workspace"].get(bkv), s["window"], s["sinks"])


def run(state):
    if own:
        return _own(state)
    return {"step": _plain_step, "write": _plain_write, "attn8": _plain_attn, "sink": _plain_attn}[state["op"]](state)


def _keys(case):
    """Cached positions that a request's query tokens see between them, summed over the requests."""
    w, span = case["window"], case["window"] + case["t"] - 1
    return sum(n if not w or n <= span else span + min(case["sinks"], n - span) for n in _lens(case))


def work(case):
    c = case
    if c["op"] == "step":
        news = _news(c)
        n = sum(news) + c["pad_tokens"]
        rows = c["reqs"] + c["pad"]
        prior = _spread(c["reqs"], 1, c["prior_hi"])
        entries = rows * c["cols"] - sum(-(-p // c["bs"]) for p in prior)
        return {"bytes": rows * 16 + 4 * entries + n * 24 + 4 * (sum(news) // c["bs"]), "flops": rows * 4 + n * 4}
    if c["op"] == "write":
        e = 2 if c["dtype"] == "bf16" else 4
        n = sum(_news(c))
        return {"bytes": n * 2 * c["hkv"] * c["d"] * (e + 1) + 16 * c["hkv"] * (n // c["bs"] + c["reqs"]),
                "flops": n * 4 * c["hkv"] * c["d"]}
    e = 2 if c["dtype"] == "bf16" else 4
    keys, rows = _keys(c), c["reqs"] * c["t"] * c["hq"]
    ek = e if c["op"] == "sink" else 1 + 4 / (c["bs"] * c["d"])
    return {"bytes": int(keys * 2 * c["hkv"] * c["d"] * ek) + 2 * rows * c["d"] * e + 4 * keys // c["bs"],
            "flops": 4 * c["d"] * keys * c["t"] * c["hq"]}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_write(s):
    bs, dev = s["bs"], "cuda"
    table, qsl, ctx = s["table"].cpu(), s["qsl"].tolist(), s["ctx"].tolist()
    # every touched block: (id, first written row, first token, tokens)
    parts = []
    for r in range(len(ctx)):
        i, p = qsl[r], ctx[r] - (qsl[r + 1] - qsl[r])
        while i < qsl[r + 1]:
            m = min(bs - p % bs, qsl[r + 1] - i)
            parts.append((int(table[r, p // bs]), p % bs, i, m))
            i, p = i + m, p + m
    ids = torch.tensor([b for b, _, _, _ in parts], device=dev)
    first = torch.tensor([o for _, o, _, _ in parts], device=dev)
    powers = torch.tensor([2.0 ** e for e in range(EXP_MIN, EXP_MAX + 1)], dtype=torch.float64, device=dev)
    got = []
    for new, cache, scales in ((s["k"], s["k_cache"], s["k_scales"]), (s["v"], s["v_cache"], s["v_scales"])):
        whole = cache.view(torch.float8_e4m3fn).double()
        now = scales.double()
        part = torch.repeat_interleave(torch.arange(len(parts)), torch.tensor([m for _, _, _, m in parts])).to(dev)
        row = torch.cat([torch.arange(o, o + m) for _, o, _, m in parts]).to(dev)
        tok = torch.cat([torch.arange(i, i + m) for _, _, i, m in parts]).to(dev)
        x = torch.zeros(len(parts), bs, s["hkv"], s["d"], dtype=torch.float64, device=dev)
        x[part, row] = new.double()[tok]
        # the first power whose 448-fold reaches the largest value
        scale = powers[torch.searchsorted(448.0 * powers, x.abs().amax((1, 3))).clamp_max(len(powers) - 1)]
        scale = torch.where(first[:, None] > 0, torch.maximum(scale, now[ids]), scale)
        old = torch.arange(bs, device=dev)[None] < first[:, None]
        written = torch.zeros(len(parts), bs, dtype=torch.bool, device=dev)
        written[part, row] = True
        held = whole[ids]
        held = torch.where(old[..., None, None], held * (now[ids] / scale)[:, None, :, None], held)
        held = torch.where(written[..., None, None], (x / scale[:, None, :, None]).clamp(-448.0, 448.0), held)
        whole[ids] = held
        now[ids] = scale
        got += [whole, now]   # values in units of their scale, and the scales
    return tuple(got)


def _exact_attn(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t, g, w = s["t"], s["hq"] // s["hkv"], s["window"]
    table, lens = s["table"].cpu(), s["ctx"].tolist()
    for r, n in enumerate(lens):
        blocks = table[r][:-(-n // s["bs"])].long().cuda()
        k, v = s["k_cache"][blocks], s["v_cache"][blocks]
        if s["op"] == "attn8":
            k = k.view(torch.float8_e4m3fn).double() * s["k_scales"][blocks].double()[:, None, :, None]
            v = v.view(torch.float8_e4m3fn).double() * s["v_scales"][blocks].double()[:, None, :, None]
        k, v = k.flatten(0, 1)[:n].double(), v.flatten(0, 1)[:n].double()
        j = torch.arange(n, device="cuda")
        for i in range(t):
            p = n - t + i
            see = (j <= p) & ((j >= p - w + 1) | (j < s["sinks"])) if w else j <= p
            q = s["q"][r, i].double().view(s["hkv"], g, -1)
            logits = torch.einsum("hgd,nhd->hgn", q, k[see]) * s["d"] ** -0.5
            out[r, i] = torch.einsum("hgn,nhd->hgd", logits.softmax(-1), v[see]).flatten(0, 1)
    return out


def _exact_step(s):
    """Whole numbers: the requests one after the other, on the host."""
    bs = s["bs"]
    cached, new, free = s["cached"].tolist(), s["new"].tolist(), s["free"].tolist()
    table, n = s["table"].cpu().numpy().copy(), s["slots"].numel()
    ctx, qsl, req, pos, slots, used = [], [0], [], [], [], 0
    for r, (c, m) in enumerate(zip(cached, new)):
        a, b = -(-c // bs), min(-(-(c + m) // bs), table.shape[1])
        table[r, a:] = -1
        if b > a:
            table[r, a:b] = free[used:used + b - a]
            used += b - a
        ctx.append(c + m)
        qsl.append(qsl[-1] + m)
        req += [r] * m
        pos += range(c, c + m)
        slots += [int(table[r, p // bs]) * bs + p % bs for p in range(c, c + m)]
    rest = n - len(req)
    ten = [torch.from_numpy(table), ctx, qsl, req + [-1] * rest, pos + [0] * rest, slots + [-1] * rest, [used]]
    types = [torch.int32] * 4 + [torch.int64] * 2 + [torch.int32]
    return tuple((x if torch.is_tensor(x) else torch.tensor(x, dtype=y)).cuda() for x, y in zip(ten, types))


def exact(case, seed):
    s = prepare(case, seed)
    return {"step": _exact_step, "write": _exact_write, "attn8": _exact_attn, "sink": _exact_attn}[case["op"]](s)

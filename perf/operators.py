"""The operators of a speculative step over a paged KV cache, as they are measured.

A step prepares its tokens (norm of every query and key head, position rotation, slots, cache write), attends over the
cache with a tree of drafted tokens, and verifies the drafts against the target's probabilities.  ``run`` does one of
these in elementary torch operations, or, where ``own`` is set, through the calls of ``paged_kv_cache_slot_gb300.bkv``.
"""
import math

import torch

own = False

NEG = float("-inf")


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------
def listed():
    return [
        # -- norm, rotation, slots and cache write (op "prep") --
        # a decode step of 32 requests, one token each: launch latency counts
        dict(name="prep_decode", op="prep", reqs=32, singles=32, new_lo=0, new_hi=0, prior_hi=4096, hq=32, hkv=8, d=128,
             rot=128, inter=False, norm=True, bs=64, dtype="bf16", fp8=False, tree=False, pad=0),
        # drafted trees of 2..30 tokens on an E4M3 cache with the hybrid block size, a padded tail, half of a head rotated
        dict(name="prep_tree_fp8", op="prep", reqs=64, singles=1, new_lo=2, new_hi=30, prior_hi=2048, hq=32, hkv=8, d=128,
             rot=64, inter=False, norm=True, bs=16, dtype="bf16", fp8=True, tree=True, pad=37),
        # a mixed step of 48 decode tokens and 16 prompt chunks of 64..1024 tokens: bandwidth counts
        dict(name="prep_step", op="prep", reqs=64, singles=48, new_lo=64, new_hi=1024, prior_hi=2048, hq=32, hkv=8, d=128,
             rot=128, inter=False, norm=True, bs=16, dtype="bf16", fp8=False, tree=False, pad=0),
        # -- attention of a drafted tree over the cache (op "attn") --
        # one request with a short context and a small tree: the latency of a chat with one user
        dict(name="attn_one", op="attn", reqs=1, lo=700, hi=700, t=7, hq=32, hkv=8, d=128, bs=64, dtype="bf16"),
        # 32 requests of 512..4096 tokens, trees of 16 drafts
        dict(name="attn_batch", op="attn", reqs=32, lo=512, hi=4096, t=16, hq=32, hkv=8, d=128, bs=64, dtype="bf16"),
        # 256 requests of very mixed lengths with 1 + 3 drafts in blocks of 16
        dict(name="attn_hybrid", op="attn", reqs=256, lo=9, hi=8192, t=4, hq=32, hkv=8, d=128, bs=16, dtype="bf16"),
        # 8 long requests, 64 query heads, trees of 61 drafts: the most arithmetic per byte
        dict(name="attn_long", op="attn", reqs=8, lo=1000, hi=16693, t=61, hq=64, hkv=8, d=128, bs=64, dtype="bf16"),
        # fp32 caches with small heads, an odd group and an odd number of requests
        dict(name="attn_f32", op="attn", reqs=13, lo=33, hi=2500, t=11, hq=15, hkv=5, d=64, bs=16, dtype="f32"),
        # -- verification of a chain of drafts with the draft model's probabilities (op "chain") --
        dict(name="chain_small", op="chain", reqs=4, k=3, v=32000, ragged=False),
        dict(name="chain_batch", op="chain", reqs=256, k=7, v=100003, ragged=True),
        # -- verification of a tree of drafts from the target's probabilities alone (op "tree") --
        dict(name="tree_small", op="tree", reqs=5, t=16, v=50001),
        dict(name="tree_batch", op="tree", reqs=64, t=61, v=131072),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["prep", "prep", "attn", "attn", "attn", "chain", "tree"])
    if op == "prep":
        reqs = _log(rng, 1, 64)
        singles = rng.randint(0, reqs)
        hkv = rng.choice([1, 2, 5, 8])
        d = rng.choice([64, 128, 128, 128, 256])
        hq = hkv * rng.choice([1, 3, 4, 4, 8])
        if hq * d > 4096:
            hq = max(1, 4096 // d // hkv) * hkv
        lo = _log(rng, 2, 64)
        tree = rng.random() < 0.4
        return dict(op="prep", reqs=reqs, singles=singles, new_lo=lo, new_hi=lo + _log(rng, 1, 60 if tree else 900),
                    prior_hi=_log(rng, 64, 2048), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2]),
                    inter=rng.random() < 0.4, norm=rng.random() < 0.7, bs=rng.choice([16, 32, 64]),
                    dtype=rng.choice(["bf16", "bf16", "f32"]), fp8=rng.random() < 0.4, tree=tree,
                    pad=rng.choice([0, 1, 19]))
    if op == "attn":
        f32 = rng.random() < 0.25
        hkv = rng.choice([1, 2, 4, 5, 8])
        g = rng.choice([1, 3, 4, 4, 6, 8])
        reqs = _log(rng, 1, 64)
        hi = _log(rng, 128, 16000 if reqs <= 8 and not f32 else 4096 if not f32 else 2000)
        t = _log(rng, 1, 64)
        if f32:
            reqs, t = min(reqs, 16), min(t, 24)
        if reqs > 8:
            t = min(t, 32)
        return dict(op="attn", reqs=reqs, lo=t + _log(rng, 1, max(2, hi // 4)), hi=hi + t, t=t, hq=hkv * g, hkv=hkv,
                    d=rng.choice([32, 64, 128]) if f32 else 128, bs=rng.choice([16, 32, 64]),
                    dtype="f32" if f32 else "bf16")
    v = _log(rng, 1000, 131072)
    if op == "chain":
        return dict(op="chain", reqs=_log(rng, 1, 190), k=rng.randint(1, 7), v=v, ragged=rng.random() < 0.5)
    return dict(op="tree", reqs=_log(rng, 1, 64), t=_log(rng, 2, 61), v=v)


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
    return [1] * case["singles"] + [case["new_lo"] + int(i * step) for i in range(n)]


def _tables(lens, bs, g):
    """Block tables of requests of these lengths: ids a permutation of 1..total-1, unused entries -1.  The pool's size
    follows from the lengths' sum."""
    need = [-(-n // bs) for n in lens]
    most = sum(lens) // bs + len(lens)
    total = most + most // 4 + 2
    ids = (torch.randperm(total - 1, generator=g, device="cuda") + 1).to(torch.int32)
    table = torch.full((len(lens), max(need) + 1), -1, dtype=torch.int32, device="cuda")
    at = 0
    for r, n in enumerate(need):
        table[r, :n] = ids[at:at + n]
        at += n
    return table, total


def _trees(reqs, t, seed):
    """Random trees: parents int32 (reqs, t), every parent before its child, root -1; ancestors-or-self bool (reqs, t, t)
    and depths int64.  Shallow and bushy, as drafters build them."""
    g = torch.Generator()
    g.manual_seed(seed * 16 + 9)
    parents = torch.full((reqs, t), -1, dtype=torch.int64)
    anc = torch.zeros(reqs, t, t, dtype=torch.bool)
    anc[:, 0, 0] = True
    rows = torch.arange(reqs)
    for i in range(1, t):
        p = (torch.rand(reqs, generator=g) ** 1.5 * i).long().clamp_(max=i - 1)
        parents[:, i] = p
        anc[:, i] = anc[rows, p]
        anc[:, i, i] = True
    return parents.to(torch.int32).cuda(), anc.cuda(), (anc.sum(-1) - 1).cuda()


def _words(anc):
    """Ancestor masks as 32-bit words: bit i of row t is whether token t sees token i."""
    r, t, _ = anc.shape
    w = -(-t // 32)
    bits = torch.zeros(r, t, w * 32, dtype=torch.int64, device=anc.device)
    bits[:, :, :t] = anc
    words = (bits.view(r, t, w, 32) << torch.arange(32, device=anc.device)).sum(-1)
    return torch.where(words >= 1 << 31, words - (1 << 32), words).to(torch.int32)


def _prepare_prep(c, seed):
    g = _gen(seed, 1)
    dt, dev = _dtype(c), "cuda"
    news = _news(c)
    prior = torch.tensor(_spread(c["reqs"], 1, c["prior_hi"]))[torch.randperm(c["reqs"], generator=torch.Generator().manual_seed(seed))]
    prior = prior.tolist()
    n = sum(news)
    table, total = _tables([p + m for p, m in zip(prior, news)], c["bs"], g)
    req = torch.repeat_interleave(torch.arange(c["reqs"]), torch.tensor(news)).to(torch.int32).cuda()
    base = torch.repeat_interleave(torch.tensor(prior), torch.tensor(news)).cuda()
    at = torch.cat([torch.arange(m) for m in news]).cuda()
    pos = base + at
    rpos = pos
    if c["tree"]:
        _, _, depth = _trees(c["reqs"], max(news), seed)
        rpos = base + depth[req.long(), at]
    width = (c["hq"] + 2 * c["hkv"]) * c["d"]
    qkv = torch.randn(n, width, generator=g, device=dev, dtype=torch.float32).mul_(2.0).to(dt)
    nq, nk = c["hq"] * c["d"], c["hkv"] * c["d"]
    cache = (total, c["bs"], c["hkv"], c["d"])
    if c["fp8"]:
        k_cache, v_cache = (torch.zeros(cache, dtype=torch.uint8, device=dev) for _ in range(2))
    else:
        k_cache, v_cache = (torch.randn(cache, generator=g, device=dev, dtype=dt) for _ in range(2))
    half = c["rot"] // 2
    inv = 10000.0 ** (-torch.arange(half, dtype=torch.float64, device=dev) / half)
    ang = torch.arange(c["prior_hi"] + max(news) + 1, dtype=torch.float64, device=dev)[:, None] * inv
    mx = n + c["pad"]
    return dict(c, q=qkv[:, :nq].view(n, c["hq"], c["d"]), k=qkv[:, nq:nq + nk].view(n, c["hkv"], c["d"]),
                v=qkv[:, nq + nk:].view(n, c["hkv"], c["d"]),
                q_weight=(1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt) if c["norm"] else None,
                k_weight=(1 + 0.2 * torch.randn(c["d"], generator=g, device=dev)).to(dt) if c["norm"] else None,
                eps=1e-6, cos_sin=torch.cat([ang.cos(), ang.sin()], 1).float(), table=table, req=req, pos=pos, rpos=rpos,
                slots=torch.full((mx,), -7, dtype=torch.int64, device=dev),
                q_out=torch.zeros(n, c["hq"], c["d"], dtype=dt, device=dev), k_cache=k_cache, v_cache=v_cache,
                k_scale=0.02, v_scale=0.03)


def _lens(case):
    return _spread(case["reqs"], case["lo"], case["hi"])


def _prepare_attn(c, seed):
    g = _gen(seed, 2)
    dt, dev = _dtype(c), "cuda"
    lens = torch.tensor(_lens(c))[torch.randperm(c["reqs"], generator=torch.Generator().manual_seed(seed))]
    table, total = _tables(lens.tolist(), c["bs"], g)
    parents, anc, _ = _trees(c["reqs"], c["t"], seed)
    cache = (total, c["bs"], c["hkv"], c["d"])
    # scores of standard deviation 2, so that some keys matter much more than others
    q = torch.randn(c["reqs"], c["t"], c["hq"], c["d"], generator=g, device=dev).mul_(2 ** 0.5).to(dt)
    k = torch.randn(cache, generator=g, device=dev, dtype=dt).mul_(2 ** 0.5)
    v = torch.randn(cache, generator=g, device=dev, dtype=dt)
    st = dict(c, q=q, k_cache=k, v_cache=v, table=table, ctx=lens.to(torch.int32).cuda(), max_ctx=int(max(lens)),
              anc=anc, mask=_words(anc), out=torch.zeros_like(q))
    # a program allocates its workspace once; its size is settled by the framework where that is there
    st["workspace"] = _Workspace((c["reqs"], c["t"], c["hq"], c["hkv"], c["d"], c["bs"], st["max_ctx"]))
    return st


class _Workspace:
    """Scratch memory that a program keeps for its calls, made at the first of them."""

    def __init__(self, sizes):
        self.sizes, self.mem = sizes, None

    def get(self, bkv):
        if self.mem is None:
            self.mem = bkv.alloc_tree_workspace(*self.sizes)
        return self.mem


def _gumbel_argmax(logp, g):
    u = torch.rand(logp.shape, generator=g, device=logp.device).clamp_min_(1e-30)
    return (logp - torch.log(-torch.log(u))).argmax(-1)


def _prepare_chain(c, seed):
    g = _gen(seed, 3)
    r, k, v = c["reqs"], c["k"], c["v"]
    target = torch.randn(r, k + 1, v, generator=g, device="cuda").mul_(3.0)
    draft = target[:, :k] + 0.7 * torch.randn(r, k, v, generator=g, device="cuda")
    draft = draft.log_softmax(-1)
    tokens = torch.stack([_gumbel_argmax(draft[:, i], g) for i in range(k)], 1)
    lens = torch.full((r,), k, dtype=torch.int32, device="cuda")
    if c["ragged"]:
        lens = torch.randint(0, k + 1, (r,), generator=g, device="cuda", dtype=torch.int32)
    return dict(c, target=target.softmax(-1), draft=draft.exp_(), tokens=tokens, lens=lens,
                u=torch.rand(r, k, generator=g, device="cuda"), us=torch.rand(r, generator=g, device="cuda"),
                out=torch.zeros(r, k + 1, dtype=torch.int64, device="cuda"),
                count=torch.zeros(r, dtype=torch.int32, device="cuda"))


def _prepare_tree(c, seed):
    g = _gen(seed, 4)
    r, t, v = c["reqs"], c["t"], c["v"]
    parents, anc, _ = _trees(r, t, seed)
    logits = torch.randn(r, t, v, generator=g, device="cuda").mul_(3.0)
    # the drafter proposes, under each node, tokens that the target finds likely
    noisy = logits + 0.7 * torch.randn(r, t, v, generator=g, device="cuda")
    likely = noisy.topk(min(t, v), -1).indices
    del noisy
    rank = ((parents[:, :, None] == parents[:, None, :]) & torch.ones(t, t, dtype=torch.bool, device="cuda").tril(-1)).sum(-1)
    tokens = likely[torch.arange(r, device="cuda")[:, None], parents.clamp_min(0).long(), rank]
    return dict(c, target=logits.softmax(-1), tokens=tokens, parents=parents, anc=anc,
                u=torch.rand(r, t, generator=g, device="cuda"), us=torch.rand(r, generator=g, device="cuda"),
                out=torch.zeros(r, t, dtype=torch.int64, device="cuda"),
                path=torch.zeros(r, t, dtype=torch.int32, device="cuda"),
                count=torch.zeros(r, dtype=torch.int32, device="cuda"))


def prepare(case, seed):
    return {"prep": _prepare_prep, "attn": _prepare_attn, "chain": _prepare_chain, "tree": _prepare_tree}[case["op"]](case, seed)


# ---------------------------------------------------------------------------
# One pass, plain
# ---------------------------------------------------------------------------
def _norm_rope(x, weight, eps, cs, rot, inter):
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + eps) * weight.float()
    c, s = cs[:, None, :rot // 2], cs[:, None, rot // 2:]
    if inter:
        a, b = y[..., 0:rot:2], y[..., 1:rot:2]
        z = torch.stack([a * c - b * s, b * c + a * s], -1).flatten(-2)
    else:
        a, b = y[..., :rot // 2], y[..., rot // 2:rot]
        z = torch.cat([a * c - b * s, b * c + a * s], -1)
    return torch.cat([z, y[..., rot:]], -1)


def _codes(x, scale):
    return (x.float() / scale).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _plain_prep(s):
    n = s["pos"].numel()
    cs = s["cos_sin"][s["rpos"]]
    q = _norm_rope(s["q"], s["q_weight"], s["eps"], cs, s["rot"], s["inter"])
    k = _norm_rope(s["k"], s["k_weight"], s["eps"], cs, s["rot"], s["inter"])
    block = s["table"][s["req"].long(), s["pos"] // s["bs"]].long()
    slot = torch.where(block > 0, block * s["bs"] + s["pos"] % s["bs"], -1)
    slots = torch.full_like(s["slots"], -1)
    slots[:n] = slot
    for cache, new, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"], s["v_scale"])):
        rows = cache.view(-1, s["hkv"], s["d"])
        new = _codes(new, scale) if s["fp8"] else new.to(cache.dtype)
        keep = (slot >= 0)[:, None, None]
        rows[slot.clamp_min(0)] = torch.where(keep, new, rows[0])
    return q.to(s["q"].dtype), slots, s["k_cache"], s["v_cache"]


def _plain_attn(s):
    r, t, hq, d = s["q"].shape
    hkv, bs, g = s["hkv"], s["bs"], s["hq"] // s["hkv"]
    cols = -(-s["max_ctx"] // bs)
    table = s["table"][:, :cols].long()
    n = cols * bs
    k = s["k_cache"][table.clamp_min(0)].view(r, n, hkv, d).permute(0, 2, 3, 1).float()
    v = s["v_cache"][table.clamp_min(0)].view(r, n, hkv, d).permute(0, 2, 1, 3).float()
    q = s["q"].float().view(r, t, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(r, hkv, t * g, d)
    scores = (q @ k).view(r, hkv, t, g, n) / math.sqrt(d)
    j = torch.arange(n, device=q.device)
    first = s["ctx"].long() - t                                     # position of the tree's first token
    i = j[None] - first[:, None]                                    # (r, n): tree index of position j
    seen = torch.gather(s["anc"], 2, i.clamp(0, t - 1)[:, None, :].expand(r, t, n))
    seen = (i < 0)[:, None, :] | (seen & (i < t)[:, None, :])       # (r, t, n)
    seen = seen & (table > 0).repeat_interleave(bs, 1)[:, None, :]
    scores = scores.masked_fill(~seen[:, None, :, None, :], NEG)
    top = scores.amax(-1, keepdim=True).clamp_min(-1e30)
    w = torch.exp(scores - top)
    total = w.sum(-1, keepdim=True)
    w = (w / total.clamp_min(1e-37)).view(r, hkv, t * g, n)
    v = torch.where((j[None] < s["ctx"][:, None])[:, None, :, None], v, 0.0)
    out = (w @ v).view(r, hkv, t, g, d).permute(0, 2, 1, 3, 4).reshape(r, t, hq, d)
    return out.to(s["q"].dtype)


def _sample(w, fallback, u):
    """Lowest index whose running sum of w passes u times the whole (of `fallback` where w is all 0)."""
    w = torch.where((w.sum(-1, keepdim=True) > 0), w, fallback)
    c = w.cumsum(-1)
    x = u.double()[:, None] * c[:, -1:]
    return torch.searchsorted(c, x, right=True)[:, 0].clamp_max(w.shape[-1] - 1)


def _plain_chain(s):
    r, k, v = s["draft"].shape
    dev = s["draft"].device
    p = torch.gather(s["target"][:, :k], 2, s["tokens"][..., None])[..., 0].double()
    q = torch.gather(s["draft"], 2, s["tokens"][..., None])[..., 0].double()
    i = torch.arange(k, device=dev)
    good = (s["u"].double() * q < p) & (i[None] < s["lens"][:, None])
    n = good.long().cumprod(1).sum(1)
    rows = torch.arange(r, device=dev)
    pr = s["target"][rows, n].double()
    qr = s["draft"][rows, n.clamp_max(k - 1)].double()
    w = torch.where((n < s["lens"])[:, None], (pr - qr).clamp_min(0.0), pr)
    nxt = _sample(w, pr, s["us"])
    at = torch.arange(k + 1, device=dev)[None]
    toks = torch.cat([s["tokens"], s["tokens"][:, :1]], 1)
    out = torch.where(at < n[:, None], toks, torch.where(at == n[:, None], nxt[:, None], -1))
    return out, n.to(torch.int32)


def _plain_tree(s):
    r, t, v = s["target"].shape
    dev = s["target"].device
    idx = torch.arange(t, device=dev)
    par = s["parents"].long()
    rows = torch.arange(r, device=dev)[:, None]
    p = s["target"][rows, par.clamp_min(0), s["tokens"]].double()
    p[:, 0] = 0.0
    older = (par[:, :, None] == par[:, None, :]) & (idx[:, None] > idx[None])[None]      # sibling j before i
    same = (older & (s["tokens"][:, :, None] == s["tokens"][:, None, :])).any(-1)
    p = torch.where(same, 0.0, p)                                   # a token counts once under a node
    rem = (1.0 - (older.double() @ p[..., None])[..., 0]).clamp_min(0.0)
    test = s["u"].double() * rem < p
    taken = test & ~(older & test[:, None, :]).any(-1)
    taken[:, 0] = True
    reached = ~(s["anc"] & ~taken[:, None, :]).any(-1)              # every ancestor and the node itself taken
    n = reached.sum(1) - 1
    path = torch.where(reached, idx, t).sort(1).values
    last = path.gather(1, n[:, None])[:, 0]
    pr = s["target"][rows[:, 0], last].double()
    kids = par == last[:, None]
    kids[:, 0] = False
    w = pr.scatter_reduce(1, s["tokens"], torch.where(kids, 0.0, torch.inf).double(), "amin")
    nxt = _sample(w, pr, s["us"])
    toks = s["tokens"].gather(1, path.clamp_max(t - 1).roll(-1, 1))
    out = torch.where(idx[None] < n[:, None], toks, torch.where(idx[None] == n[:, None], nxt[:, None], -1))
    return out, torch.where(path < t, path, -1).to(torch.int32), n.to(torch.int32)


# ---------------------------------------------------------------------------
# One pass, through the framework
# ---------------------------------------------------------------------------
def _own(s):
    from paged_kv_cache_slot_gb300 import bkv

    if s["op"] == "prep":
        if s["fp8"]:
            bkv.bkv_qk_norm_rope_cache_write_fp8(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"], s["cos_sin"],
                                                 s["table"], s["req"], s["pos"], s["slots"], s["q_out"], s["k_cache"],
                                                 s["v_cache"], s["k_scale"], s["v_scale"], rope_positions=s["rpos"],
                                                 interleaved=s["inter"])
        else:
            bkv.bkv_qk_norm_rope_cache_write(s["q"], s["k"], s["v"], s["q_weight"], s["k_weight"], s["eps"], s["cos_sin"],
                                             s["table"], s["req"], s["pos"], s["slots"], s["q_out"], s["k_cache"],
                                             s["v_cache"], rope_positions=s["rpos"], interleaved=s["inter"])
        return s["q_out"], s["slots"], s["k_cache"], s["v_cache"]
    if s["op"] == "attn":
        return bkv.bkv_paged_decode_tree(s["q"], s["k_cache"], s["v_cache"], s["table"], s["ctx"], s["max_ctx"], s["mask"],
                                         s["out"], s["workspace"].get(bkv))
    if s["op"] == "chain":
        return bkv.bkv_verify_draft_chain(s["target"], s["draft"], s["tokens"], s["u"], s["us"], s["out"], s["count"],
                                          draft_lens=s["lens"])
    return bkv.bkv_verify_draft_tree(s["target"], s["tokens"], s["parents"], s["u"], s["us"], s["out"], s["path"], s["count"])


def run(state):
    if own:
        got = _own(state)
    else:
        got = {"prep": _plain_prep, "attn": _plain_attn, "chain": _plain_chain, "tree": _plain_tree}[state["op"]](state)
    if state["op"] == "prep" and state["fp8"]:   # codes as the values that they stand for
        got = (got[0], got[1], got[2].view(torch.float8_e4m3fn), got[3].view(torch.float8_e4m3fn))
    return got


def work(case):
    c = case
    if c["op"] == "prep":
        e = 2 if c["dtype"] == "bf16" else 4
        ec = 1 if c["fp8"] else e
        n = sum(_news(c))
        row = 2 * c["hq"] * c["d"] * e + 2 * c["hkv"] * c["d"] * (e + ec)
        return {"bytes": n * (row + 4 * c["rot"] + 28), "flops": n * (c["hq"] + c["hkv"]) * (4 * c["d"] + 3 * c["rot"])}
    if c["op"] == "attn":
        e = 2 if c["dtype"] == "bf16" else 4
        keys, rows = sum(_lens(c)), c["reqs"] * c["t"] * c["hq"]
        return {"bytes": keys * 2 * c["hkv"] * c["d"] * e + 2 * rows * c["d"] * e + c["reqs"] * (c["t"] * -(-c["t"] // 32) * 4 + 4),
                "flops": 4 * c["d"] * keys * c["t"] * c["hq"]}
    # one row of the target's probabilities a request, and in a chain the draft's beside it
    return {"bytes": c["reqs"] * c["v"] * 4 * (2 if c["op"] == "chain" else 1), "flops": c["reqs"] * c["v"] * 2}


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------
def _exact_head(x, w, eps, ang_c, ang_s, rot, inter):
    y = x.double().clone()
    if w is not None:
        y = w.double() * y / (y.pow(2).sum(-1, keepdim=True) / y.shape[-1] + eps).sqrt()
    z = y.clone()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        c, s = ang_c[:, i:i + 1], ang_s[:, i:i + 1]
        z[:, :, a] = y[:, :, a] * c - y[:, :, b] * s
        z[:, :, b] = y[:, :, b] * c + y[:, :, a] * s
    return z


def _exact_prep(s):
    half = s["rot"] // 2
    cs = s["cos_sin"].double()[s["rpos"]]
    q = _exact_head(s["q"], s["q_weight"], s["eps"], cs[:, :half], cs[:, half:], s["rot"], s["inter"])
    k = _exact_head(s["k"], s["k_weight"], s["eps"], cs[:, :half], cs[:, half:], s["rot"], s["inter"])
    pos, req, table = s["pos"].tolist(), s["req"].tolist(), s["table"].tolist()
    slots = [table[r][p // s["bs"]] * s["bs"] + p % s["bs"] for r, p in zip(req, pos)]
    at = torch.tensor(slots, device=q.device)
    caches = []
    for cache, new, scale in ((s["k_cache"], k, s["k_scale"]), (s["v_cache"], s["v"].double(), s["v_scale"])):
        if s["fp8"]:   # values are kept in units of the scale
            whole = torch.zeros(cache.shape, dtype=torch.float64, device=q.device)
            new = (new / scale).clamp(-448.0, 448.0)
        else:
            whole = cache.double()
        whole.view(-1, s["hkv"], s["d"])[at] = new
        caches.append(whole)
    return q, torch.tensor(slots + [-1] * s["pad"], device=q.device), caches[0], caches[1]


def _exact_attn(s):
    out = torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    t, g = s["t"], s["hq"] // s["hkv"]
    table, ctx = s["table"].tolist(), s["ctx"].tolist()
    for r in range(s["reqs"]):
        blocks = torch.tensor(table[r][:-(-ctx[r] // s["bs"])], device="cuda")
        k = s["k_cache"][blocks].flatten(0, 1)[:ctx[r]].double()
        v = s["v_cache"][blocks].flatten(0, 1)[:ctx[r]].double()
        hidden = torch.zeros(t, ctx[r], dtype=torch.bool, device="cuda")
        hidden[:, ctx[r] - t:] = ~s["anc"][r]
        for h in range(s["hkv"]):
            q = s["q"][r, :, h * g:(h + 1) * g].double()
            logits = torch.einsum("tgd,nd->tgn", q, k[:, h]) * s["d"] ** -0.5
            logits[hidden[:, None].expand_as(logits)] = NEG
            out[r, :, h * g:(h + 1) * g] = torch.einsum("tgn,nd->tgd", logits.softmax(-1), v[:, h])
    return out


def _first_past(weights, u):
    run = torch.cumsum(weights, 0)
    return int((run <= u * float(run[-1])).sum())


def _exact_chain(s):
    out, count = [], []
    lens, tokens = s["lens"].tolist(), s["tokens"].tolist()
    u, us = s["u"].double().tolist(), s["us"].double().tolist()
    for r in range(s["reqs"]):
        got = []
        while len(got) < lens[r]:
            i = len(got)
            x = tokens[r][i]
            if not u[r][i] * float(s["draft"][r, i, x]) < float(s["target"][r, i, x]):
                break
            got.append(x)
        w = p = s["target"][r, len(got)].double()
        if len(got) < lens[r]:
            w = (p - s["draft"][r, len(got)].double()).clamp_min(0.0)
        count.append(len(got))
        got.append(_first_past(w if float(w.sum()) > 0 else p, us[r]))
        out.append(got + [-1] * (s["k"] + 1 - len(got)))
    return torch.tensor(out, device="cuda"), torch.tensor(count, dtype=torch.int32, device="cuda")


def _exact_tree(s):
    out, paths, count = [], [], []
    tokens, parents = s["tokens"].tolist(), s["parents"].tolist()
    u, us = s["u"].double().tolist(), s["us"].double().tolist()
    for r in range(s["reqs"]):
        path, got = [0], []
        while True:
            p = s["target"][r, path[-1]].double()
            w, left, child = p.clone(), 1.0, None
            for c in range(1, s["t"]):
                if parents[r][c] != path[-1]:
                    continue
                x = float(w[tokens[r][c]])
                if u[r][c] * max(left, 0.0) < x:
                    child = c
                    break
                left -= x
                w[tokens[r][c]] = 0.0
            if child is None:
                break
            path.append(child)
            got.append(tokens[r][child])
        count.append(len(got))
        got.append(_first_past(w if float(w.sum()) > 0 else p, us[r]))
        out.append(got + [-1] * (s["t"] - len(got)))
        paths.append(path + [-1] * (s["t"] - len(path)))
    return (torch.tensor(out, device="cuda"), torch.tensor(paths, dtype=torch.int32, device="cuda"),
            torch.tensor(count, dtype=torch.int32, device="cuda"))


def exact(case, seed):
    s = prepare(case, seed)
    return {"prep": _exact_prep, "attn": _exact_attn, "chain": _exact_chain, "tree": _exact_tree}[case["op"]](s)

"""A host model of the tree attention's schedule and of its kernel's barriers.

The schedule (which column of CTAs takes which tiles, and where partials go) is
restated from its definition and checked for what the merge relies on: every
tile taken once, partial slots distinct and where the merge looks for them, the table of
split streams complete.  The barrier protocol of the kernel's warps (rings of
K and V slots, query buffers, two softmax streams, the unit's end) is run as
agents with random delays: no wait may be left unanswered, none answered a
phase early, and every product must see the operands of its own tile."""
import heapq
import random

import numpy as np
import pytest

KERNELS = [(128, 2, 2), (32, 1, 1)]   # positions a tile, tiles that a unit's end takes as long as, a column's least cost


def _columns(lens, P, TILE, END_COST, MIN_COST):
    """Column q's units: (request, first tile, tiles, whole, slot)."""
    tiles = [-(-n // TILE) for n in lens]
    cost = [t + END_COST if t else 0 for t in tiles]
    pre = np.concatenate([[0], np.cumsum(cost)]).tolist()
    C = pre[-1]
    peff = min(-(-C // MIN_COST), P)
    out = []
    for q in range(P):
        lo, hi = (C * q // peff, C * (q + 1) // peff) if q < peff else (C, C)
        units = []
        for r, t in enumerate(tiles):
            a, b = max(lo, pre[r]), min(hi, pre[r] + t)
            if a < b:
                units.append((r, a - pre[r], b - a, b - a == t, P + q if a == pre[r] else q))
        split = (0, 0)
        for r, t in enumerate(tiles):   # the stream that this column begins and does not end
            s, e = pre[r], pre[r] + t
            if t and lo <= s < hi < e:
                split = (r, (e * peff - 1) // C - q + 1)
        out.append((units, split))
    return tiles, out


@pytest.mark.parametrize("seed", range(40))
@pytest.mark.parametrize("TILE,END_COST,MIN_COST", KERNELS)
def test_every_tile_once_and_slots_for_the_merge(seed, TILE, END_COST, MIN_COST):
    rng = random.Random(seed)
    P = rng.choice([1, 2, 5, 9, 19, 76, 152])
    lens = [rng.choice([0, 1, 127, 128, 129, rng.randint(1, 20000), rng.randint(1, 700)]) for _ in range(rng.randint(1, 60))]
    tiles, cols = _columns(lens, P, TILE, END_COST, MIN_COST)
    seen = [np.zeros(t, int) for t in tiles]
    parts, slots = {}, set()
    for q, (units, split) in enumerate(cols):
        for r, f, n, whole, slot in units:
            seen[r][f:f + n] += 1
            assert slot < 2 * P
            if whole:
                assert n == tiles[r]
            else:
                assert slot not in slots
                slots.add(slot)
                parts.setdefault(r, []).append(slot)
    assert all((s == 1).all() for s in seen)
    table = {s[0]: (q, s[1]) for q, (_, s) in enumerate(cols) if s[1]}
    assert set(table) == set(parts)              # every split stream, once
    for r, got in parts.items():
        q, n = table[r]
        assert got == [P + q] + list(range(q + 1, q + n)) and n >= 2
    load = [sum(n for _, _, n, _, _ in u) + END_COST * len(u) for u, _ in cols]
    assert max(load) <= sum(tiles + [END_COST for t in tiles if t]) / P + 2 + 2 * END_COST or MIN_COST * P > sum(tiles)


class _Bar:
    """An mbarrier: arrivals complete a phase; a parity wait is answered when the current phase's parity differs."""

    def __init__(self, count):
        self.count = self.pending = count
        self.phase = 0

    def arrive(self):
        assert self.pending > 0
        self.pending -= 1
        if self.pending == 0:
            self.pending, self.phase = self.count, self.phase + 1


def _run(rng, units, nK, nV, nbuf, dual, aq):
    now, events, count = [0], [], [0]

    def later(d, f):
        count[0] += 1
        heapq.heappush(events, (now[0] + d, count[0], f))

    def wait(bar, k):
        """Phase k of a barrier (in order: the model checks that the parity could not have meant another)."""
        assert bar.phase in (k, k + 1), "a parity wait a phase early or late"
        return bar, k

    issuers = 1 if dual else 2
    kf, ke = [_Bar(1) for _ in range(8)], [_Bar(1) for _ in range(3)]
    vf, ve = [_Bar(1) for _ in range(8)], [_Bar(1) for _ in range(3)]
    qf, qe = [_Bar(1), _Bar(1)], [_Bar(issuers), _Bar(issuers)]
    sf = [_Bar(1), _Bar(1)]
    pf = [_Bar(4), _Bar(aq[1] if dual else 4)]
    of, oe = _Bar(2 * issuers), _Bar(aq[0] + aq[1])
    mk, pair = [_Bar(1) for _ in range(8)], [_Bar(2) for _ in range(4)]
    K, V, Q, mask = [None] * 3, [None] * 3, [None] * 2, [None] * 8
    S, Pw, O = [None, None], [None, None], [[], []]
    own = {}
    j = 0
    for u, n in enumerate(units):
        for _ in range(n):
            for x in ((0, 1) if dual else (j & 1,)):
                own.setdefault((u, x), []).append(j)
            j += 1
    pace = [rng.randint(1, 40) for _ in range(8)]
    free = [0, 0]

    def mma(x, f):   # one issuing thread's products run in order
        free[x] = max(now[0], free[x]) + rng.randint(5, 9)
        later(free[x] - now[0], f)

    def commit(x, bar):
        later(max(now[0], free[x]) - now[0] + rng.randint(0, 3), bar.arrive)

    def use(k):   # a slot's or buffer's k-th use waits for the end of its (k - 1)-th
        return k - 1

    def loads(is_v):
        n_slots, full, empty, store = (nV, vf, ve, V) if is_v else (nK, kf, ke, K)
        j = 0
        for u, n in enumerate(units):
            if not is_v:
                b, k = (u & 1, u >> 1) if nbuf == 2 else (0, u)
                if k:
                    yield wait(qe[b], use(k))

                def q_land(b=b, u=u):
                    Q[b] = u
                    qf[b].arrive()
                later(rng.randint(1, pace[0]), q_land)
            for _ in range(n):
                s, k = j % n_slots, j // n_slots
                if k:
                    yield wait(empty[s], use(k))
                if not is_v:
                    mask[j & 7] = j
                    mk[j & 7].arrive()
                store[s] = None

                def land(s=s, j=j):
                    store[s] = j
                    full[j & 7].arrive()
                later(rng.randint(1, pace[1 + is_v]), land)
                j += 1
                yield rng.randint(0, 2)

    done = [0, 0]   # P tiles used of each stream

    def finish(i):
        commit(i, of)
        of.arrive()

    def pv(i, x, j, first, u):
        yield wait(vf[j & 7], j >> 3)
        yield wait(pf[x], done[x])
        done[x] += 1
        if first and u:
            yield wait(oe, u - 1)

        def f():
            assert V[j % nV] == j and Pw[x] == j
            Pw[x] = None
            if first:
                O[x] = []
            O[x].append(j)
        mma(i, f)

    def score(i, x, j, u, b):
        def f():
            assert K[j % nK] == j and Q[b] == u and Pw[x] is None
            S[x] = j
        mma(i, f)
        commit(i, sf[x])

    def issuer_of_both():   # two query tiles: one thread
        j = 0
        for u, n in enumerate(units):
            yield wait(qf[0], u)
            for t in range(n + 1):
                if t < n:
                    yield wait(kf[(j + t) & 7], (j + t) >> 3)
                for x in range(2):
                    if t:
                        yield from pv(0, x, j + t - 1, t == 1, u)
                    if t < n:
                        score(0, x, j + t, u, 0)
                    yield rng.randint(0, 6)
                if t:
                    commit(0, ve[(j + t - 1) % nV])
                if t < n:
                    commit(0, ke[(j + t) % nK])
                    if t == n - 1:
                        commit(0, qe[0])
                else:
                    finish(0)
            j += n

    def issuer(x):   # one query tile: a thread a stream
        pend = None  # the tile whose P V is to come

        def settle():
            nonlocal pend
            if pend is None:
                return
            (j, first, last, u), pend = pend, None
            yield from pv(x, x, j, first, u)
            commit(x, ve[j % nV])
            if last:
                finish(x)
        j = 0
        for u, n in enumerate(units):
            b, k = (u & 1, u >> 1) if nbuf == 2 else (0, u)
            had = False
            for t in range(n):
                if (j & 1) == x:
                    yield from settle()
                    if not had:
                        yield wait(qf[b], k)
                    yield wait(kf[j & 7], j >> 3)
                    score(x, x, j, u, b)
                    commit(x, ke[j % nK])
                    last = t + 2 >= n
                    pend, had = (j, not had, last, u), True
                    if last:
                        commit(x, qe[b])
                    yield rng.randint(0, 6)
                j += 1
            if not had:   # no tile of the unit is this stream's
                yield from settle()
                yield wait(qf[b], k)
                if u:
                    yield wait(oe, u - 1)
                qe[b].arrive()
                finish(x)
        yield from settle()

    posted = {}

    def softmax(x, w):
        idle, fixes = w >= aq[x], not dual or x == 0
        if idle and not fixes:
            return
        ns = 0
        for u, n in enumerate(units):
            for j in own.get((u, x), []):
                yield wait(sf[x], ns)
                yield wait(mk[j & 7], j >> 3)
                ns += 1
                assert S[x] == j and mask[j & 7] == j
                yield rng.randint(1, pace[3 + x])
                assert mask[j & 7] == j
                if fixes and rng.random() < 0.5:
                    yield wait(vf[j & 7], j >> 3)
                    assert V[j % nV] == j
                yield rng.randint(1, pace[5])
                assert S[x] == j and (not fixes or V[j % nV] in (j, None, j - nV))
                posted[x, j] = posted.get((x, j), 0) + 1
                if posted[x, j] == (4 if fixes else aq[1]):
                    Pw[x] = j
                pf[x].arrive()
            if idle:
                continue
            if not dual:
                pair[w].arrive()
                yield wait(pair[w], u)
            yield wait(of, u)
            for _ in range(2):
                for y in ((x,) if dual else (0, 1)):
                    assert not own.get((u, y)) or O[y] == own[u, y]
                yield rng.randint(1, pace[6])
            oe.arrive()

    agents = [loads(False), loads(True)] + ([issuer_of_both()] if dual else [issuer(0), issuer(1)]) + [softmax(x, w) for x in range(2) for w in range(4)]
    at, blocked, alive = [0] * len(agents), [None] * len(agents), set(range(len(agents)))
    while alive:
        while events and events[0][0] <= now[0]:
            heapq.heappop(events)[2]()
        moved, order = False, list(alive)
        rng.shuffle(order)
        for i in order:
            if at[i] > now[0] or (blocked[i] and blocked[i][0].phase <= blocked[i][1]):
                continue
            moved = True
            try:
                got = next(agents[i])
                blocked[i] = got if isinstance(got, tuple) else None
                at[i] = now[0] + (got if isinstance(got, int) else 0)
            except StopIteration:
                alive.discard(i)
        if not moved:
            nxt = [e[0] for e in events[:1]] + [at[i] for i in alive if at[i] > now[0]]
            assert nxt, "every agent waits"
            now[0] = max(now[0] + 1, min(nxt))


@pytest.mark.parametrize("seed", range(200))
def test_barriers_answer_every_wait(seed):
    rng = random.Random(seed)
    dual = rng.random() < 0.4
    units = [rng.choice([1, 1, 2, 3, 4, 5, 7, 12]) for _ in range(rng.randint(1, 8))]
    nbuf = 1 if dual else rng.choice([1, 2])
    nK, nV = (2, 2) if dual else rng.choice([(2, 2), (2, 3), (3, 3)])
    a = rng.randint(1, 4)
    _run(rng, units, nK, nV, nbuf, dual, (a, rng.randint(1, a) if dual else a))

"""A host model of the tree attention kernel's unit end where key tiles alternate on
two softmax streams: a lane quarter's two warps (one a stream) exchange a row's
maximum and sum through shared memory, an entry a stream, by a barrier of two
arrivals; sets of entries are used in turn.  Run as agents at random paces: what
a warp reads must be both streams' entries of its own unit, whatever the units'
lengths.  And the constants that the model of the schedule was written with, against
the sources'."""
import os
import random
import re

import pytest

from paged_kv_cache_slot_gb300 import build as bkv_build
from test_tree_schedule_host import KERNELS, _Bar


def _source(name):
    with open(os.path.join(bkv_build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def _run(rng, units, sets):
    """units: tiles of each; sets of entries that the units take in turn."""
    sf, pf = [_Bar(1), _Bar(1)], [_Bar(1), _Bar(1)]
    of, oe, pair = _Bar(4), _Bar(2), _Bar(2)
    own, j = {}, 0
    for u, n in enumerate(units):
        for _ in range(n):
            own.setdefault((u, j & 1), []).append(j)
            j += 1
    pipe = [[], []]          # arrivals that wait for an issuing thread's products
    xm = [[None, None] for _ in range(sets)]
    live = [2, 2]

    def products(x):
        while live[x] or pipe[x]:
            if pipe[x]:
                pipe[x].pop(0).arrive()
            yield None

    def issuer(x):
        pend, tiles = None, 0

        def settle():
            nonlocal pend, tiles
            if pend is None:
                return
            (first, last, u), pend = pend, None
            yield pf[x], tiles
            tiles += 1
            if first and u:
                yield oe, u - 1
            if last:
                pipe[x].append(of)
                of.arrive()
        for u, n in enumerate(units):
            mine = own.get((u, x), [])
            for i in range(len(mine)):
                yield from settle()
                pipe[x].append(sf[x])
                pend = (i == 0, i == len(mine) - 1, u)
                yield None
            if not mine:
                yield from settle()
                if u:
                    yield oe, u - 1
                pipe[x].append(of)
                of.arrive()
        yield from settle()
        live[x] -= 1

    def softmax(x):
        ns = 0
        for u in range(len(units)):
            for _ in own.get((u, x), []):
                yield sf[x], ns
                ns += 1
                yield None
                pf[x].arrive()
            xm[u % sets][x] = u
            pair.arrive()
            yield pair, u
            for y in rng.sample((0, 1), 2):
                yield None
                assert xm[u % sets][y] == u, "an entry of another unit"
            yield of, u
            yield None
            oe.arrive()
        live[x] -= 1

    agents = {i: a for i, a in enumerate((products(0), products(1), issuer(0), issuer(1), softmax(0), softmax(1)))}
    pace = [10.0 ** rng.uniform(-2, 0) for _ in agents]
    blocked = {}
    for _ in range(400 * (sum(units) + len(units)) + 100000):
        if not agents:
            return
        ready = [i for i in agents if i not in blocked or blocked[i][0].phase > blocked[i][1]]
        assert ready, "every agent waits"
        i = rng.choices(ready, [pace[i] for i in ready])[0]
        blocked.pop(i, None)
        try:
            got = next(agents[i])
        except StopIteration:
            del agents[i]
            continue
        if got is not None:
            assert got[0].phase in (got[1], got[1] + 1), "a parity wait a phase early or late"
            blocked[i] = got
    raise AssertionError("no end")


def _units(rng):
    return [rng.choice([1, 1, 1, 2, 2, 3, 5]) for _ in range(rng.randint(2, 10))]


def _sets():
    """The kernel's sets of entries, which its warps index by the unit's number."""
    src = _source("bkv_tree_tc.cu")
    found = re.findall(r"kXmSets = (\d+);", src)
    if not found:
        return 1
    assert re.search(r"xm \+ no % kXmSets \* 2 \* kTile", src) and re.search(r"kOffXm \+ kXmSets \* 2 \* kTile \* 8", src)
    return int(found[0])


@pytest.mark.parametrize("seed", range(200))
def test_a_quarters_warps_read_their_own_units_entries(seed):
    rng = random.Random(seed)
    _run(rng, _units(rng), _sets())


def test_the_model_sees_a_single_set():
    bad = 0
    for seed in range(300):
        rng = random.Random(seed)
        try:
            _run(rng, _units(rng), 1)
        except AssertionError as e:
            assert "another unit" in str(e)
            bad += 1
    assert bad > 0


def test_the_schedules_model_has_the_kernels_constants():
    cc, tc, shared = (_source(n) for n in ("bkv_tree.cu", "bkv_tree_tc.cu", "bkv_tree.cuh"))

    def value(src, name):
        return int(re.search(rf"\b{name} = (\d+)[,;]", src).group(1))
    assert re.search(r"kTile = kTreeTile;", tc)
    # the CUDA-core kernel's columns: at least a cost of one each
    assert re.search(r"peff = C < a\.P \? C : a\.P;", cc)
    assert KERNELS == [(value(shared, "kTreeTile"), value(tc, "kEndCost"), value(tc, "kMinCost")),
                       (value(cc, "kBK"), value(cc, "kCcEnd"), 1)]

"""The schedule of the attention over windows and block-scaled caches, as its own
header computes it, run on the host: a request's span holds every position that
some query sees, each once, and begins its runs at segments' borders; columns
take every tile of every request once; partial slots are distinct and where the
merge looks for them."""
import os
import random
import subprocess

import numpy as np
import pytest

from paged_kv_cache_slot_gb300 import build as bkv_build

CSRC = os.path.join(os.path.dirname(os.path.abspath(bkv_build.__file__)), "csrc")
INCLUDE = os.path.join(os.path.dirname(os.path.dirname(CSRC)), "include")

# reads: n P tile seg q_len window sinks max_ctx, then n lengths.  Prints a span a request, then a column a line.
PROGRAM = r"""
#include <cstdio>
#include <vector>
#include "bkv_window.cuh"
int main() {
    using namespace bkv::win;
    Args a{};
    int n, P;
    while (std::scanf("%d %d %d %d %d %d %d %d", &n, &P, &a.tile, &a.seg, &a.q_len, &a.window, &a.sinks, &a.max_ctx) == 8) {
        std::vector<int> pre(n + 1, 0);
        for (int r = 0, x; r < n; ++r) {
            if (std::scanf("%d", &x) != 1) return 1;
            const Span s = span_of(a, x);
            pre[r + 1] = pre[r] + (s.len > 0 ? (s.len + a.tile - 1) / a.tile + kEndCost : 0);
            std::printf("%d %d %d %d\n", s.L, s.sb, s.gap, s.len);
        }
        for (int q = 0; q < P; ++q) {
            Units u(pre.data(), n, q, P);
            const int2 sp = u.split();
            std::printf("%d %d", sp.x, sp.y);
            Unit x;
            while (u.next(x)) std::printf(" %d %d %d %d %d", x.r, x.f, x.nt, (int)x.whole, x.slot);
            std::printf("\n");
        }
    }
    return 0;
}
"""


@pytest.fixture(scope="module")
def schedule(tmp_path_factory):
    d = tmp_path_factory.mktemp("schedule")
    src, exe = d / "schedule.cu", d / "schedule"
    src.write_text(PROGRAM)
    nvcc = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    subprocess.run([nvcc, "-gencode", "arch=compute_103a,code=sm_103a", "-std=c++17", "-I", CSRC, "-I", INCLUDE, "-o",
                    str(exe), str(src)], check=True, capture_output=True)

    def run(lens, P, tile, seg, q_len, window, sinks, max_ctx):
        text = " ".join(map(str, [len(lens), P, tile, seg, q_len, window, sinks, max_ctx, *lens]))
        out = subprocess.run([str(exe)], input=text, capture_output=True, text=True, check=True).stdout.splitlines()
        rows = [list(map(int, line.split())) for line in out]
        return rows[:len(lens)], rows[len(lens):]

    return run


@pytest.mark.parametrize("seed", range(60))
def test_spans_tiles_and_slots(schedule, seed):
    rng = random.Random(seed)
    P = rng.choice([1, 2, 5, 9, 19, 57, 152])
    tile, seg = rng.choice([(64, 1), (128, 8), (128, 16), (128, 64), (128, 128)])
    q_len, window, sinks = rng.choice([1, 2, 5, 40]), rng.choice([0, 0, 1, 50, 777, 2048]), rng.choice([0, 1, 4, 100, 500])
    lens = [rng.choice([0, 1, 127, 128, 129, rng.randint(1, 9000), rng.randint(1, 700)]) for _ in range(rng.randint(1, 60))]
    max_ctx = max(lens) if rng.random() < 0.8 else max(1, max(lens) // 2)
    spans, cols = schedule(lens, P, tile, seg, q_len, window, sinks, max_ctx)
    for n, (L, sb, gap, size) in zip(lens, spans):
        assert L == min(n, max_ctx) and size == L - gap and sb % seg == 0 and gap % seg == 0
        v = np.arange(size)
        at = set(np.where(v < sb, v, v + gap).tolist())
        assert len(at) == size and all(0 <= p < L for p in at)
        first = max(0, L - q_len - window + 1) if window else 0
        assert at >= set(range(first, L)) | (set(range(min(sinks, L))) if window else set())
        if gap:   # no segment more than holds a first token or a window's
            assert sb - seg < sinks and first - (sb + gap) < seg
    tiles = [-(-s[3] // tile) for s in spans]
    seen = [np.zeros(t, int) for t in tiles]
    parts, slots, table = {}, set(), {}
    for q, col in enumerate(cols):
        if col[1]:
            assert col[0] not in table
            table[col[0]] = (q, col[1])
        for r, f, n, whole, slot in np.reshape(col[2:], (-1, 5)).tolist():
            assert n > 0
            seen[r][f:f + n] += 1
            assert 0 <= slot < 2 * P and bool(whole) == (n == tiles[r])
            if not whole:
                assert slot not in slots
                slots.add(slot)
                parts.setdefault(r, []).append(slot)
    assert all((s == 1).all() for s in seen)
    assert set(table) == set(parts)
    for r, got in parts.items():
        q, n = table[r]
        assert got == [P + q] + list(range(q + 1, q + n)) and n >= 2

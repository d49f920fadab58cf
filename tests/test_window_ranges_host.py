"""Host-side refusals of step building, block-scaled writes and windowed attention at the ends of their ranges."""
from paged_kv_cache_slot_gb300 import bkv
from test_window_host import _Entry, lib  # noqa: F401 (a fixture)


def test_tables_too_wide_for_the_step(lib):  # noqa: F811
    """Walks over a row's columns stay within int32."""
    some = {n: 64 * (i + 1) for i, n in enumerate(("cached", "new", "free", "bt", "ctx", "qsl", "req", "pos", "slots", "used"))}
    entry = _Entry(lib.bkv_build_step, "ppipiipqiqpppppppp")
    for cols in ((1 << 30) + 1, (1 << 31) - 1):
        assert entry(some["cached"], some["new"], 1, some["free"], 3, 16, some["bt"], 1 << 31, cols, 5, some["ctx"], some["qsl"],
                     some["req"], some["pos"], some["slots"], some["used"], 0, 0) == bkv.BKV_ERR_INVALID_ARG, cols

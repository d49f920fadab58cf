"""Host-side checks of step building, block-scaled E4M3 caches and windows whose
first tokens stay visible: the C ABI's refusals (before any CUDA call), the
binding's checks and argument marshalling, the plain forms of the GPU tests."""
import ctypes

import numpy as np
import pytest
import torch

from _window import attend, block_scale, build_step, visible
from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import build as bkv_build
from test_spec_binding_host import SAME_DEVICE, _Elsewhere
from test_spec_host import fake  # noqa: F401 (a fixture)

NULL = None
I32, I64, U8 = torch.int32, torch.int64, torch.uint8


@pytest.fixture(scope="module")
def lib():
    bkv_build.build()
    return bkv.load()


class _Entry:
    """A C entry point under the argument types of include/bkv.h (the binding passes records instead)."""

    def __init__(self, f, types):
        c = {"p": ctypes.c_void_p, "i": ctypes.c_int32, "q": ctypes.c_int64, "f": ctypes.c_float, "n": ctypes.c_size_t}
        self.f = ctypes.CFUNCTYPE(ctypes.c_int, *[c[x] for x in types])(ctypes.cast(f, ctypes.c_void_p).value)

    def __call__(self, *args):
        return self.f(*args)


def test_build_step_refusals(lib):
    entry = _Entry(lib.bkv_build_step, "ppipiipqiqpppppppp")

    base = dict(cached=NULL, new=NULL, nr=2, free=NULL, nf=3, bs=16, bt=NULL, st=4, cols=4, mx=5, ctx=NULL, qsl=NULL,
                req=NULL, pos=NULL, slots=NULL, used=NULL, err=NULL, stream=NULL)

    def call(**kw):
        return entry(*dict(base, **kw).values())

    some = {n: 64 * (i + 1) for i, n in enumerate(("cached", "new", "free", "bt", "ctx", "qsl", "req", "pos", "slots", "used"))}
    for bad in (dict(nr=-1), dict(nr=(1 << 30) + 1), dict(nf=-1), dict(bs=0), dict(cols=-1), dict(st=3), dict(mx=-1),
                dict(ctx=some["cached"]), dict(ctx=some["new"]), *({n: NULL} for n in some)):
        assert call(**dict(some, **bad)) == bkv.BKV_ERR_INVALID_ARG, bad


def test_write_refusals(lib):
    entry = _Entry(lib.bkv_cache_write_fp8_blocks, "ppqqppipqippppqiiiipp")
    base = dict(k=NULL, v=NULL, n=4, stride=1024, qsl=NULL, ctx=NULL, nr=2, bt=NULL, st=4, cols=4, kc=NULL, vc=NULL, ks=NULL,
                vs=NULL, tb=9, bs=16, hkv=8, d=128, dt=0, err=NULL, stream=NULL)

    def call(**kw):
        return entry(*dict(base, **kw).values())

    assert call(dt=3) == bkv.BKV_ERR_UNSUPPORTED
    some = {n: 64 * (i + 1) for i, n in enumerate(("k", "v", "qsl", "ctx", "bt", "kc", "vc", "ks", "vs"))}
    for bad in (dict(n=-1), dict(nr=-1), dict(tb=-1), dict(bs=0), dict(hkv=0), dict(d=0), dict(cols=-1), dict(st=3),
                dict(stride=1023), dict(bs=65537), dict(d=65544, stride=1 << 20), dict(n=1 << 31), *({n: NULL} for n in some)):
        assert call(**dict(some, **bad)) == bkv.BKV_ERR_INVALID_ARG, bad
    assert call(n=0) == bkv.BKV_OK and call(nr=0) == bkv.BKV_OK      # nothing to do launches nothing


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_refusals(lib, fp8):
    base = dict(q=NULL, k=NULL, v=NULL)
    if fp8:
        base.update(ks=NULL, vs=NULL)
    base.update(bt=NULL, st=4, cols=4, ctx=NULL, mx=16, nr=2, ql=1, hq=32, hkv=8, d=128, bs=16, tb=8, scale=0.0, mode=0,
                window=8, sinks=4, dt=0, out=NULL, ws=NULL, wsb=0, err=NULL, stream=NULL)
    types = "pqipiiiiiiiqfiiiippnpp"
    f = (_Entry(lib.bkv_paged_decode_fp8_blocks, "ppppp" + types) if fp8 else _Entry(lib.bkv_paged_decode_sink, "ppp" + types))

    def call(**kw):
        return f(*dict(base, **kw).values())

    size = lib.bkv_paged_decode_window_workspace_size
    need = size(2, 1, 32, 8, 128, 16, 16)
    some = {n: 64 * (i + 1) for i, n in enumerate(x for x in ("q", "k", "v", "ks", "vs", "bt", "ctx", "out", "ws") if x in base)}
    some["wsb"] = need
    for bad in (dict(dt=5), dict(d=258), dict(d=63)):
        assert call(**dict(some, **bad)) == bkv.BKV_ERR_UNSUPPORTED, bad
    for bad in (dict(st=3), dict(cols=-1), dict(hq=30), dict(nr=0), dict(ql=0), dict(hkv=0), dict(bs=0), dict(bs=65537),
                dict(mx=-1), dict(mx=(1 << 26) + 1), dict(ql=20000), dict(tb=-1), dict(mode=2), dict(window=-1), dict(sinks=-1),
                dict(wsb=need - 1), dict(ws=16), *({n: NULL} for n in some if n != "wsb")):
        assert call(**dict(some, **bad)) == bkv.BKV_ERR_INVALID_ARG, bad
    for bad in ((0, 1, 32, 8, 128, 16, 16), (2, 0, 32, 8, 128, 16, 16), (2, 1, 30, 8, 128, 16, 16), (2, 1, 32, 8, 0, 16, 16),
                (2, 1, 32, 8, 258, 16, 16), (2, 1, 32, 8, 127, 16, 16), (2, 1, 32, 8, 128, 0, 16), (2, 1, 32, 8, 128, 16, -1),
                (2, 1, 32, 8, 128, 16, (1 << 26) + 1)):
        assert size(*bad) == 0, bad
    # what a call needs does not grow with the lengths or the batch
    assert size(1, 1, 32, 8, 128, 16, 100) == size(4000, 1, 32, 8, 128, 16, 1 << 26) > 0


def _step():
    z = torch.zeros
    return dict(cached_lens=z(3, dtype=I32), new_lens=z(3, dtype=I32), free_blocks=z(7, dtype=I32), block_size=16,
                block_table=z(3, 9, dtype=I32)[:, :5], context_lens=z(3, dtype=I32), query_start_loc=z(4, dtype=I32),
                req_indices=z(11, dtype=I32), positions=z(11, dtype=I64), slot_mapping=z(11, dtype=I64),
                blocks_used=z(1, dtype=I32))


def _write(n=6, hkv=2, d=64):
    z = torch.zeros
    kv = z(n, 2 * hkv * d + 16, dtype=torch.bfloat16)
    return dict(k_new=kv[:, :hkv * d].view(n, hkv, d), v_new=kv[:, hkv * d:2 * hkv * d].view(n, hkv, d),
                query_start_loc=z(4, dtype=I32), context_lens=z(3, dtype=I32), block_table=z(3, 5, dtype=I32),
                k_cache=z(8, 16, hkv, d, dtype=U8), v_cache=z(8, 16, hkv, d, dtype=U8), k_scales=z(8, hkv), v_scales=z(8, hkv))


def _attn(fp8, nr=3, t=2, hq=8, hkv=2, d=64, dtype=torch.bfloat16):
    z = torch.zeros
    a = dict(q=z(nr, t, hq, d, dtype=dtype), k_cache=z(8, 16, hkv, d, dtype=U8 if fp8 else dtype),
             v_cache=z(8, 16, hkv, d, dtype=U8 if fp8 else dtype))
    if fp8:
        a.update(k_scales=z(8, hkv), v_scales=z(8, hkv))
    a.update(block_table=z(nr, 5, dtype=I32), context_lens=z(nr, dtype=I32), max_context_len=70,
             out=z(nr, t, hq, d, dtype=dtype), workspace=z(99, dtype=U8), sliding_window=33, num_sinks=4)
    return a


def _attn_fn(fp8):
    return bkv.bkv_paged_decode_fp8_blocks if fp8 else bkv.bkv_paged_decode_sink


def _sent(fake, fn):  # noqa: F811
    """The arguments of a call, out of its record."""
    (record,) = fake.calls[fn + "_record"]
    return bkv._RECORDS[fn].unpack(record)


def test_marshalling(fake):  # noqa: F811
    bkv.bkv_build_step(**_step())
    p = fake.ptrs
    assert _sent(fake, "bkv_build_step") == (
        p["cached_lens"], p["new_lens"], 3, p["free_blocks"], 7, 16, p["block_table"], 9, 5, 11, p["context_lens"],
        p["query_start_loc"], p["req_indices"], p["positions"], p["slot_mapping"], p["blocks_used"], 0, 999)
    bkv.bkv_cache_write_fp8_blocks(**_write())
    assert _sent(fake, "bkv_cache_write_fp8_blocks") == (
        p["k_new"], p["v_new"], 6, 272, p["query_start_loc"], p["context_lens"], 3, p["block_table"], 5, 5, p["k_cache"],
        p["v_cache"], p["k_scales"], p["v_scales"], 8, 16, 2, 64, bkv.BKV_BF16, 0, 999)
    for fp8 in (False, True):
        fn = "bkv_paged_decode_fp8_blocks" if fp8 else "bkv_paged_decode_sink"
        _attn_fn(fp8)(**_attn(fp8), softmax_scale=0.5, mask_mode=bkv.BKV_MASK_ALL)
        scales = (p["k_scales"], p["v_scales"]) if fp8 else (0, 0)
        assert _sent(fake, fn) == (p["q"], p["k_cache"], p["v_cache"], *scales, p["block_table"], 5, 5, p["context_lens"], 70,
                                   3, 2, 8, 2, 64, 16, 8, 0.5, 1, 33, 4, bkv.BKV_BF16, p["out"], p["workspace"], 99, 0, 999)
    with pytest.raises(ValueError, match="C type"):              # no argument is cut to fit
        bkv.bkv_paged_decode_sink(**dict(_attn(False), sliding_window=1 << 33))


def test_records_are_the_entry_points_arguments(lib):
    """A record read by the library refuses exactly what its entry point refuses: every field sits where the C struct has
    it (a wrong size before it would move what is refused)."""
    good = dict(step=[64, 64, 2, 64, 3, 16, 64, 4, 4, 5, 128, 64, 64, 64, 64, 64, 0, 0],
                write=[64, 64, 4, 1024, 64, 64, 2, 64, 4, 4, 64, 64, 64, 64, 9, 16, 8, 128, 0, 0, 0],
                attn=[64, 64, 64, 64, 64, 64, 4, 4, 64, 16, 2, 1, 32, 8, 128, 16, 8, 0.0, 0, 8, 4, 0, 64, 64,
                      lib.bkv_paged_decode_window_workspace_size(2, 1, 32, 8, 128, 16, 16), 0, 0])

    def refused(fn, args, at, value, status=bkv.BKV_ERR_INVALID_ARG):
        args = list(args)
        args[at] = value
        got = getattr(lib, fn + "_record")(bkv._RECORDS[fn].pack(*args))
        assert got == status, (fn, at, value, got)

    for at, value in ((0, 0), (1, 0), (2, -1), (3, 0), (4, -1), (5, 0), (6, 0), (7, 3), (8, -1), (9, -1), (10, 64), (11, 0),
                      (12, 0), (13, 0), (14, 0), (15, 0)):
        refused("bkv_build_step", good["step"], at, value)
    for at, value in ((0, 0), (1, 0), (2, -1), (3, 1023), (4, 0), (5, 0), (6, -1), (7, 0), (8, 3), (9, -1), (10, 0), (11, 0),
                      (12, 0), (13, 0), (14, -1), (15, 0), (16, 0), (17, 0)):
        refused("bkv_cache_write_fp8_blocks", good["write"], at, value)
    refused("bkv_cache_write_fp8_blocks", good["write"], 18, 7, bkv.BKV_ERR_UNSUPPORTED)
    for fn in ("bkv_paged_decode_sink", "bkv_paged_decode_fp8_blocks"):
        for at, value in ((0, 0), (1, 0), (2, 0), (5, 0), (6, 3), (7, -1), (8, 0), (9, -1), (10, 0), (11, 0), (12, 30), (13, 0),
                          (15, 0), (16, -1), (18, 3), (19, -1), (20, -1), (22, 0), (23, 0), (23, 16), (24, 100)):
            refused(fn, good["attn"], at, value)
        refused(fn, good["attn"], 14, 63, bkv.BKV_ERR_UNSUPPORTED)
        refused(fn, good["attn"], 21, 3, bkv.BKV_ERR_UNSUPPORTED)
    refused("bkv_paged_decode_fp8_blocks", good["attn"], 3, 0)
    refused("bkv_paged_decode_fp8_blocks", good["attn"], 4, 0)


STEP_BAD = [(dict(new_lens=torch.zeros(2, dtype=I32)), ValueError), (dict(context_lens=torch.zeros(4, dtype=I32)), ValueError),
            (dict(query_start_loc=torch.zeros(3, dtype=I32)), ValueError), (dict(blocks_used=torch.zeros(2, dtype=I32)), ValueError),
            (dict(positions=torch.zeros(10, dtype=I64)), ValueError), (dict(req_indices=torch.zeros(12, dtype=I32)), ValueError),
            (dict(block_table=torch.zeros(2, 5, dtype=I32)), ValueError), (dict(block_table=torch.zeros(5, dtype=I32)), ValueError),
            (dict(block_table=torch.zeros(5, 3, dtype=I32).t()), ValueError)]
WRITE_BAD = [(dict(k_new=torch.zeros(6, 3, 64, dtype=torch.bfloat16)), ValueError), (dict(k_scales=torch.zeros(8, 3)), ValueError),
             (dict(v_scales=torch.zeros(9, 2)), ValueError), (dict(k_cache=torch.zeros(8, 8, 2, 64, dtype=U8)), ValueError),
             (dict(k_cache=torch.zeros(8, 16, 2, 64), v_cache=torch.zeros(8, 16, 2, 64)), TypeError),
             (dict(v_new=torch.zeros(6, 2, 64, dtype=torch.bfloat16)), ValueError),
             (dict(k_new=torch.zeros(6, 2, 64), v_new=torch.zeros(6, 2, 64, dtype=torch.bfloat16)), TypeError),
             (dict(k_new=torch.zeros(6, 2, 64, dtype=torch.float16), v_new=torch.zeros(6, 2, 64, dtype=torch.float16)), TypeError),
             (dict(context_lens=torch.zeros(2, dtype=I32)), ValueError), (dict(query_start_loc=torch.zeros(0, dtype=I32)), ValueError),
             (dict(query_start_loc=torch.zeros(6, dtype=I32), context_lens=torch.zeros(5, dtype=I32)), ValueError),
             (dict(k_new=torch.zeros(2, 6, 64, dtype=torch.bfloat16).transpose(0, 1)), ValueError)]


@pytest.mark.parametrize("change,exc", STEP_BAD)
def test_build_step_checks(fake, change, exc):  # noqa: F811
    with pytest.raises(exc):
        bkv.bkv_build_step(**dict(_step(), **change))
    assert not fake.calls


@pytest.mark.parametrize("change,exc", WRITE_BAD)
def test_write_checks(fake, change, exc):  # noqa: F811
    with pytest.raises(exc):
        bkv.bkv_cache_write_fp8_blocks(**dict(_write(), **change))
    assert not fake.calls


@pytest.mark.parametrize("fp8", [False, True])
def test_decode_checks(fake, fp8):  # noqa: F811
    z, bf = torch.zeros, torch.bfloat16
    bad = [(dict(q=z(3, 2, 8, 32, dtype=bf), out=z(3, 2, 8, 32, dtype=bf)), ValueError), (dict(out=z(3, 2, 7, 64, dtype=bf)), ValueError),
           (dict(out=z(3, 2, 8, 64)), TypeError), (dict(k_cache=z(8, 16, 2, 64), v_cache=z(8, 16, 2, 64)), TypeError),
           (dict(v_cache=z(8, 16, 2, 32, dtype=U8)), ValueError), (dict(block_table=z(2, 5, dtype=I32)), ValueError),
           (dict(context_lens=z(2, dtype=I32)), ValueError), (dict(workspace=z(99)), TypeError),
           (dict(q=z(3, 2, 8, 64, dtype=torch.float16)), TypeError)]
    if fp8:
        bad += [(dict(k_scales=z(8, 3)), ValueError), (dict(v_scales=z(7, 2)), ValueError)]
    for change, exc in bad:
        with pytest.raises(exc):
            _attn_fn(fp8)(**dict(_attn(fp8), **change))
        assert not fake.calls, change


@pytest.mark.parametrize("at", range(4))
def test_every_tensor_is_looked_at_for_its_device(fake, monkeypatch, at):  # noqa: F811
    fn, kw = [(bkv.bkv_build_step, _step()), (bkv.bkv_cache_write_fp8_blocks, _write()), (_attn_fn(False), _attn(False)),
              (_attn_fn(True), _attn(True))][at]
    kw["err_count"] = torch.zeros(1, dtype=I32)
    monkeypatch.setattr(bkv, "_same_device", SAME_DEVICE)
    monkeypatch.setattr(bkv, "_current_device", lambda: -1)      # the device that host tensors say they are on
    monkeypatch.setattr(bkv, "_gpus", 2)
    fn(**kw)
    assert len(fake.calls) == 1
    for name in [n for n, x in kw.items() if isinstance(x, torch.Tensor)]:
        fake.calls.clear()
        with pytest.raises(ValueError, match="current device"):
            fn(**dict(kw, **{name: kw[name].as_subclass(_Elsewhere)}))
        assert not fake.calls


def test_dimensions_of_size_one_may_carry_any_stride(fake):  # noqa: F811
    one = torch.zeros(5, dtype=I32).as_strided((1, 5), (0, 1))
    a = _attn(True, nr=1)
    bkv.bkv_paged_decode_fp8_blocks(**dict(a, block_table=one))
    assert _sent(fake, "bkv_paged_decode_fp8_blocks")[6:8] == (5, 5)
    heads = torch.zeros(2, 6, 64, dtype=torch.bfloat16)
    w = dict(_write(hkv=1), k_new=heads[:1].transpose(0, 1), v_new=heads[1:].transpose(0, 1))
    bkv.bkv_cache_write_fp8_blocks(**w)
    assert _sent(fake, "bkv_cache_write_fp8_blocks")[3] == 64


def test_plain_forms():
    """The tests' own plain forms on worked examples."""
    # the page's blocks: positions 62 .. 65 of a request with blocks 10 and 15 of 64
    table = np.array([[10, 7, 9]], np.int32)
    got = build_step(np.array([62]), np.array([4]), [15, 16], 64, table, 6)
    assert got[0].tolist() == [[10, 15, -1]] and got[5].tolist() == [702, 703, 960, 961, -1, -1]
    assert got[4].tolist() == [62, 63, 64, 65, 0, 0] and got[6:] == (1, 0) and got[2].tolist() == [0, 4]
    assert block_scale(np.array([448.0])) == 1.0 and block_scale(np.array([-448.1])) == 2.0
    assert block_scale(np.array([0.0])) == 2.0 ** -40 and block_scale(np.array([np.inf, 224.0, np.nan])) == 0.5
    assert visible(10, 2, 0, True, 3, 2).tolist() == [0, 1, 6, 7, 8] and visible(10, 2, 1, False, 3, 0).tolist() == [7, 8, 9]
    rng = np.random.default_rng(0)
    q, k, v = (rng.standard_normal(s) for s in ((2, 4, 8), (12, 2, 8), (12, 2, 8)))
    t = [torch.from_numpy(x) for x in (q, k, v)]
    mask = torch.zeros(2, 12, dtype=torch.bool)
    for i in range(2):
        mask[i, torch.from_numpy(visible(12, 2, i, True, 4, 3))] = True
    want = torch.nn.functional.scaled_dot_product_attention(
        t[0].transpose(0, 1), t[1].transpose(0, 1).repeat_interleave(2, 0), t[2].transpose(0, 1).repeat_interleave(2, 0),
        attn_mask=mask).transpose(0, 1).numpy()
    assert np.allclose(attend(q, k, v, 12, True, 4, 3), want, atol=1e-12)

"""Host-side checks of the speculative step's entry points: the C ABI's refusals
(before any CUDA call) and the binding's checks and argument marshalling."""
import pytest
import torch

from paged_kv_cache_slot_gb300 import bkv
from paged_kv_cache_slot_gb300 import build as bkv_build

NULL = None


@pytest.fixture(scope="module")
def lib():
    bkv_build.build()
    return bkv.load()


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_refusals(lib, fp8):
    f = getattr(lib, "bkv_qk_norm_rope_cache_write" + ("_fp8" if fp8 else ""))

    def call(**kw):
        a = dict(q=NULL, k=NULL, v=NULL, qs=4096, ks=1024, vs=1024, qw=NULL, kw=NULL, eps=1e-6, cs=NULL, maxp=10, rot=128,
                 inter=0, bt=NULL, nr=1, st=4, cols=4, req=NULL, pos=NULL, rpos=NULL, n=1, mx=1, slots=NULL, qo=NULL,
                 kc=NULL, vc=NULL, tb=4, bs=16, hq=32, hkv=8, d=128, dt=0)
        if fp8:
            a.update(kscale=1.0, vscale=1.0)
        a.update(kw)
        return f(*a.values(), NULL, NULL)

    assert call(dt=7) == bkv.BKV_ERR_UNSUPPORTED
    assert call(d=258, qs=9999, ks=9999, vs=9999) == bkv.BKV_ERR_UNSUPPORTED
    assert call(d=127) == bkv.BKV_ERR_UNSUPPORTED
    for bad in (dict(n=5, mx=4), dict(st=2), dict(bs=0), dict(hq=0), dict(hkv=0), dict(qs=4095), dict(ks=1023),
                dict(vs=1023), dict(rot=130), dict(rot=-2), dict(rot=5), dict(eps=-1.0), dict(eps=float("nan")),
                dict(maxp=-1), dict(n=-1), dict(tb=-1), dict(nr=-1)):
        assert call(**bad) == bkv.BKV_ERR_INVALID_ARG, bad
    if fp8:
        for bad in (dict(kscale=0.0), dict(vscale=float("inf")), dict(kscale=float("nan"))):
            assert call(**bad) == bkv.BKV_ERR_INVALID_ARG
    assert call() == bkv.BKV_ERR_INVALID_ARG                   # null pointers
    assert call(n=0, mx=0) == bkv.BKV_OK                       # nothing to do launches nothing


def test_tree_decode_refusals(lib):
    f = lib.bkv_paged_decode_tree
    base = dict(q=NULL, k=NULL, v=NULL, bt=NULL, bt_stride=4, bt_cols=4, ctx=NULL, max_ctx=16, num_reqs=2, q_len=5,
                hq=32, hkv=8, d=128, bs=16, tb=8, scale=0.0, mask=NULL, mstride=0, dtype=0, out=NULL, ws=NULL, wsb=0,
                err=NULL, stream=NULL)

    def call(**kw):
        return f(*dict(base, **kw).values())

    for bad in (dict(dtype=5), dict(d=512), dict(d=63), dict(q_len=257)):
        assert call(**bad) == bkv.BKV_ERR_UNSUPPORTED, bad
    for bad in (dict(bt_stride=2), dict(hq=30), dict(num_reqs=0), dict(q_len=0), dict(bs=0), dict(max_ctx=-1),
                dict(mstride=4), dict(mstride=-1), dict(tb=-1), dict()):
        assert call(**bad) == bkv.BKV_ERR_INVALID_ARG, bad
    size = lib.bkv_paged_decode_tree_workspace_size
    assert size(2, 5, 32, 8, 128, 16, 100) > 0
    for bad in ((0, 5, 32, 8, 128, 16, 100), (2, 0, 32, 8, 128, 16, 100), (2, 257, 32, 8, 128, 16, 100),
                (2, 5, 30, 8, 128, 16, 100), (2, 5, 32, 8, 258, 16, 100), (2, 5, 32, 8, 128, 0, 100),
                (2, 5, 32, 8, 128, 16, -1)):
        assert size(*bad) == 0, bad


def test_tree_decode_longest_context(lib):
    size = lib.bkv_paged_decode_tree_workspace_size
    assert size(2, 5, 32, 8, 128, 16, 1 << 30) > 0
    for bound in ((1 << 30) + 1, (1 << 31) - 1):
        assert size(2, 5, 32, 8, 128, 16, bound) == 0
    # what a call needs does not grow with the lengths or the batch
    assert size(2, 5, 32, 8, 128, 16, 100) == size(4000, 5, 32, 8, 128, 16, 1 << 20)


def test_verify_refusals(lib):
    def chain(**kw):
        a = dict(p=NULL, pr=400, prow=100, q=NULL, qr=300, qrow=100, tok=NULL, lens=NULL, u=NULL, us=NULL, nr=1, k=3, v=100,
                 out=NULL, cnt=NULL, err=NULL, stream=NULL)
        return lib.bkv_verify_draft_chain(*dict(a, **kw).values())

    def tree(**kw):
        a = dict(p=NULL, pr=400, prow=100, tok=NULL, par=NULL, u=NULL, us=NULL, nr=1, t=4, v=100, out=NULL, path=NULL,
                 cnt=NULL, err=NULL, stream=NULL)
        return lib.bkv_verify_draft_tree(*dict(a, **kw).values())

    for call, nodes in ((chain, "k"), (tree, "t")):
        assert call(**{nodes: 1025}) == bkv.BKV_ERR_UNSUPPORTED
        for bad in (dict(nr=-1), {nodes: -1}, dict(v=0), dict(prow=99), dict(pr=-1), dict()):
            assert call(**bad) == bkv.BKV_ERR_INVALID_ARG, bad
        assert call(nr=0) == bkv.BKV_OK
    assert chain(qrow=99) == bkv.BKV_ERR_INVALID_ARG
    assert tree(t=0) == bkv.BKV_ERR_INVALID_ARG


class _FakeLib:
    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def f(*args):
            self.calls[name] = args
            return 0
        return f


@pytest.fixture
def fake(monkeypatch):
    fake = _FakeLib()
    monkeypatch.setattr(bkv, "load", lambda: fake)
    fake.ptrs = {}
    monkeypatch.setattr(bkv, "_dev", lambda t, name, dtype=None, contiguous=True: fake.ptrs.setdefault(
        name, len(fake.ptrs) + 1))
    monkeypatch.setattr(bkv, "_stream", lambda s: 999)
    monkeypatch.setattr(bkv, "_same_device", lambda *t: None)
    return fake


def _rope_inputs(n=5, hq=8, hkv=2, d=64, dtype=torch.bfloat16, cache=torch.bfloat16):
    qkv = torch.zeros(n, (hq + 2 * hkv) * d, dtype=dtype)
    q = qkv[:, :hq * d].view(n, hq, d)
    k = qkv[:, hq * d:(hq + hkv) * d].view(n, hkv, d)
    v = qkv[:, (hq + hkv) * d:].view(n, hkv, d)
    i64 = torch.int64
    return dict(q=q, k=k, v=v, q_weight=torch.ones(d, dtype=dtype), k_weight=torch.ones(d, dtype=dtype), norm_eps=1e-6,
                cos_sin=torch.zeros(100, 32), block_table=torch.zeros(3, 9, dtype=torch.int32)[:, :7],
                req_indices=torch.zeros(n, dtype=torch.int32), positions=torch.zeros(n, dtype=i64),
                slot_mapping=torch.zeros(n + 2, dtype=i64), q_out=torch.zeros(n, hq, d, dtype=dtype),
                k_cache=torch.zeros(4, 16, hkv, d, dtype=cache), v_cache=torch.zeros(4, 16, hkv, d, dtype=cache))


@pytest.mark.parametrize("fp8", [False, True])
def test_norm_rope_marshalling(fake, fp8):
    a = _rope_inputs(cache=torch.uint8 if fp8 else torch.bfloat16)
    fn = "bkv_qk_norm_rope_cache_write" + ("_fp8" if fp8 else "")
    if fp8:
        bkv.bkv_qk_norm_rope_cache_write_fp8(**a, k_scale=0.5, v_scale=2.0, interleaved=True, num_tokens=4)
    else:
        bkv.bkv_qk_norm_rope_cache_write(**a, interleaved=True, num_tokens=4)
    p = fake.ptrs
    assert fake.calls[fn] == (
        p["q"], p["k"], p["v"], 768, 768, 768, p["q_weight"], p["k_weight"], 1e-6, p["cos_sin"], 100, 32, 1,
        p["block_table"], 3, 9, 7, p["req_indices"], p["positions"], None, 4, 7, p["slot_mapping"], p["q_out"],
        p["k_cache"], p["v_cache"], 4, 16, 8, 2, 64, bkv.BKV_BF16) + ((0.5, 2.0) if fp8 else ()) + (None, 999)


@pytest.mark.parametrize("change,exc", [
    (dict(q=torch.zeros(5, 8, 32, dtype=torch.bfloat16)), ValueError),
    (dict(k=torch.zeros(5, 3, 64, dtype=torch.bfloat16)), ValueError),
    (dict(v=torch.zeros(5, 2, 64)), TypeError),
    (dict(q_out=torch.zeros(4, 8, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q_out=torch.zeros(5, 8, 64)), TypeError),
    (dict(k_cache=torch.zeros(4, 16, 2, 64), v_cache=torch.zeros(4, 16, 2, 64)), TypeError),
    (dict(v_cache=torch.zeros(3, 16, 2, 64, dtype=torch.bfloat16)), ValueError),
    (dict(q_weight=torch.ones(32, dtype=torch.bfloat16)), ValueError),
    (dict(cos_sin=torch.zeros(100)), ValueError),
    (dict(num_tokens=6), ValueError),
    (dict(rope_positions=torch.zeros(4, dtype=torch.int64)), ValueError),
    (dict(q=torch.zeros(5, 64, 8, dtype=torch.bfloat16).transpose(1, 2)), ValueError)])
def test_norm_rope_binding_refuses(fake, change, exc):
    with pytest.raises(exc):
        bkv.bkv_qk_norm_rope_cache_write(**dict(_rope_inputs(), **change))


def _tree_inputs(nr=3, t=40, hq=8, hkv=2, d=64, dtype=torch.float32):
    z = torch.zeros
    return dict(q=z(nr, t, hq, d, dtype=dtype), k_cache=z(4, 16, hkv, d, dtype=dtype), v_cache=z(4, 16, hkv, d, dtype=dtype),
                block_table=z(nr, 6, dtype=torch.int32), context_lens=z(nr, dtype=torch.int32), max_context_len=90,
                tree_mask=z(nr, t, 2, dtype=torch.int32), out=z(nr, t, hq, d, dtype=dtype),
                workspace=z(1000, dtype=torch.uint8))


def test_tree_decode_marshalling(fake):
    a = _tree_inputs()
    for mask, stride in ((a["tree_mask"], 80), (a["tree_mask"][0], 0)):
        bkv.bkv_paged_decode_tree(**dict(a, tree_mask=mask), softmax_scale=0.25)
        p = fake.ptrs
        assert fake.calls["bkv_paged_decode_tree"] == (
            p["q"], p["k_cache"], p["v_cache"], p["block_table"], 6, 6, p["context_lens"], 90, 3, 40, 8, 2, 64, 16, 4, 0.25,
            p["tree_mask"], stride, bkv.BKV_F32, p["out"], p["workspace"], 1000, None, 999)


@pytest.mark.parametrize("change,exc", [
    (dict(tree_mask=torch.zeros(3, 40, 1, dtype=torch.int32)), ValueError),
    (dict(tree_mask=torch.zeros(2, 40, 2, dtype=torch.int32)), ValueError),
    (dict(out=torch.zeros(3, 40, 8, 64, dtype=torch.bfloat16)), TypeError),
    (dict(k_cache=torch.zeros(4, 16, 2, 64, dtype=torch.uint8), v_cache=torch.zeros(4, 16, 2, 64, dtype=torch.uint8)),
     TypeError),
    (dict(block_table=torch.zeros(2, 6, dtype=torch.int32)), ValueError),
    (dict(context_lens=torch.zeros(2, dtype=torch.int32)), ValueError),
    (dict(workspace=torch.zeros(1000)), TypeError)])
def test_tree_decode_binding_refuses(fake, change, exc):
    with pytest.raises(exc):
        bkv.bkv_paged_decode_tree(**dict(_tree_inputs(), **change))


def test_verify_marshalling(fake):
    z, i64, i32 = torch.zeros, torch.int64, torch.int32
    wide = z(3, 5, 120)
    bkv.bkv_verify_draft_chain(wide[:, :4, :100], z(3, 3, 100), z(3, 3, dtype=i64), z(3, 3), z(3), z(3, 4, dtype=i64),
                               z(3, dtype=i32), draft_lens=z(3, dtype=i32))
    p = fake.ptrs
    assert fake.calls["bkv_verify_draft_chain"] == (
        p["target_probs"], 600, 120, p["draft_probs"], 300, 100, p["draft_tokens"], p["draft_lens"], p["accept_u"],
        p["sample_u"], 3, 3, 100, p["out_tokens"], p["num_accepted"], None, 999)
    bkv.bkv_verify_draft_tree(wide[:, :, 20:], z(3, 5, dtype=i64), z(3, 5, dtype=i32), z(3, 5), z(3), z(3, 5, dtype=i64),
                              z(3, 5, dtype=i32), z(3, dtype=i32))
    assert fake.calls["bkv_verify_draft_tree"] == (
        p["target_probs"], 600, 120, p["draft_tokens"], p["parents"], p["accept_u"], p["sample_u"], 3, 5, 100,
        p["out_tokens"], p["path"], p["num_accepted"], None, 999)


def test_verify_binding_refuses(fake):
    z, i64, i32 = torch.zeros, torch.int64, torch.int32
    good = [z(3, 4, 100), z(3, 3, 100), z(3, 3, dtype=i64), z(3, 3), z(3), z(3, 4, dtype=i64), z(3, dtype=i32)]
    bkv.bkv_verify_draft_chain(*good)
    for at, bad in ((1, z(3, 4, 100)), (1, z(3, 3, 99)), (2, z(3, 4, dtype=i64)), (3, z(3, 2)), (4, z(2)),
                    (5, z(3, 3, dtype=i64)), (6, z(4, dtype=i32)), (0, z(3, 100, 4).transpose(1, 2))):
        with pytest.raises(ValueError):
            bkv.bkv_verify_draft_chain(*good[:at], bad, *good[at + 1:])
    good = [z(3, 5, 100), z(3, 5, dtype=i64), z(3, 5, dtype=i32), z(3, 5), z(3), z(3, 5, dtype=i64), z(3, 5, dtype=i32),
            z(3, dtype=i32)]
    bkv.bkv_verify_draft_tree(*good)
    for at in (1, 2, 3, 5, 6):
        with pytest.raises(ValueError):
            bkv.bkv_verify_draft_tree(*good[:at], good[at][:, :4], *good[at + 1:])


def test_binding_refuses_host_tensors():
    with pytest.raises(TypeError, match="CUDA tensor"):
        bkv.bkv_qk_norm_rope_cache_write(**_rope_inputs())
    with pytest.raises(TypeError, match="CUDA tensor"):
        bkv.bkv_paged_decode_tree(**_tree_inputs())
    z, i64, i32 = torch.zeros, torch.int64, torch.int32
    with pytest.raises(TypeError, match="CUDA tensor"):
        bkv.bkv_verify_draft_chain(z(3, 4, 100), z(3, 3, 100), z(3, 3, dtype=i64), z(3, 3), z(3), z(3, 4, dtype=i64),
                                   z(3, dtype=i32))

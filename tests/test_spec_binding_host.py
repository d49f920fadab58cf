"""Host-side checks of the speculative step's binding: devices and layouts."""
import inspect

import pytest
import torch

from paged_kv_cache_slot_gb300 import bkv
from test_spec_host import _rope_inputs, _tree_inputs, fake  # noqa: F401 (a fixture)

I64, I32 = torch.int64, torch.int32


def _calls():
    z = torch.zeros
    err = dict(err_count=z(1, dtype=I32))
    rope = dict(_rope_inputs(), rope_positions=z(5, dtype=I64), **err)
    yield bkv.bkv_qk_norm_rope_cache_write, rope
    yield bkv.bkv_qk_norm_rope_cache_write_fp8, dict(_rope_inputs(cache=torch.uint8), k_scale=1.0, v_scale=1.0, **err)
    yield bkv.bkv_paged_decode_tree, dict(_tree_inputs(), **err)
    yield bkv.bkv_verify_draft_chain, dict(
        target_probs=z(3, 4, 100), draft_probs=z(3, 3, 100), draft_tokens=z(3, 3, dtype=I64), accept_u=z(3, 3),
        sample_u=z(3), out_tokens=z(3, 4, dtype=I64), num_accepted=z(3, dtype=I32), draft_lens=z(3, dtype=I32), **err)
    yield bkv.bkv_verify_draft_tree, dict(
        target_probs=z(3, 5, 100), draft_tokens=z(3, 5, dtype=I64), parents=z(3, 5, dtype=I32), accept_u=z(3, 5),
        sample_u=z(3), out_tokens=z(3, 5, dtype=I64), path=z(3, 5, dtype=I32), num_accepted=z(3, dtype=I32), **err)


class _Elsewhere(torch.Tensor):
    """A tensor that says it is on the next GPU."""

    def get_device(self):
        return 1


@pytest.mark.parametrize("at", range(5))
def test_every_tensor_is_looked_at_for_its_device(fake, monkeypatch, at):  # noqa: F811
    """A tensor of any argument on another device than the current one is refused before the call."""
    fn, kw = list(_calls())[at]
    monkeypatch.setattr(bkv, "_same_device", SAME_DEVICE)
    monkeypatch.setattr(bkv, "_current_device", lambda: -1)      # the device that host tensors say they are on
    monkeypatch.setattr(bkv, "_gpus", 2)
    fn(**kw)
    assert len(fake.calls) == 1
    names = [n for n, x in kw.items() if isinstance(x, torch.Tensor)]
    assert len(names) >= 9 and set(names) <= set(inspect.signature(fn).parameters)
    for name in names:
        fake.calls.clear()
        with pytest.raises(ValueError, match="current device"):
            fn(**dict(kw, **{name: kw[name].as_subclass(_Elsewhere)}))
        assert not fake.calls


SAME_DEVICE = bkv._same_device


def test_dimensions_of_size_one_may_carry_any_stride(fake):  # noqa: F811
    """One head taken out of a (heads, tokens, D) layout, a table of one row or one column: dense, whatever torch calls
    the strides of those dimensions."""
    a = _rope_inputs(hq=1, hkv=1)
    heads = torch.zeros(3, 5, 64, dtype=torch.bfloat16)
    a.update(q=heads[:1].transpose(0, 1), k=heads[1:2].transpose(0, 1), v=heads[2:].transpose(0, 1),
             block_table=torch.zeros(7, dtype=torch.int32).as_strided((1, 7), (0, 1)))
    assert a["k"].stride() == (64, 320, 1)
    bkv.bkv_qk_norm_rope_cache_write(**a)
    got = fake.calls["bkv_qk_norm_rope_cache_write"]
    assert got[3:6] == (64, 64, 64) and got[14:17] == (1, 7, 7)
    for table, want in ((torch.zeros(6, dtype=torch.int32).as_strided((1, 6), (0, 1)), (6, 6)),
                        (torch.zeros(3, 4, dtype=torch.int32).as_strided((1, 1), (4, 4)), (4, 1)),
                        (torch.zeros(6, dtype=torch.int32).as_strided((3, 1), (2, 2)), (2, 1))):
        t = _tree_inputs(nr=min(3, len(table)))
        bkv.bkv_paged_decode_tree(**dict(t, block_table=table))
        assert fake.calls["bkv_paged_decode_tree"][4:6] == want
    one = torch.zeros(3, 1, 4).transpose(1, 2)                   # a vocabulary of one token
    bkv.bkv_verify_draft_chain(one, one[:, :3], torch.zeros(3, 3, dtype=I64), torch.zeros(3, 3), torch.zeros(3),
                               torch.zeros(3, 4, dtype=I64), torch.zeros(3, dtype=I32))
    assert fake.calls["bkv_verify_draft_chain"][1:3] == (4, 1) and fake.calls["bkv_verify_draft_chain"][4:6] == (4, 1)
    with pytest.raises(ValueError):
        bkv.bkv_qk_norm_rope_cache_write(**dict(_rope_inputs(), k=torch.zeros(2, 5, 64, dtype=torch.bfloat16).transpose(0, 1)))

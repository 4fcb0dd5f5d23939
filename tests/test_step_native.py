"""The native binding without a GPU: what it leaves to ctypes, and when a built one is used."""
import pytest
import torch

from packed_variable_length_varlen_gb300 import build


@pytest.fixture(scope="module")
def va():
    build.build()
    build.binding()
    from packed_variable_length_varlen_gb300 import varlen_attn
    if varlen_attn.NATIVE is None:  # built only now
        varlen_attn.NATIVE = varlen_attn._load_binding(varlen_attn.LIB)
    return varlen_attn


def test_tensors_of_the_host_are_left_to_ctypes(va):
    n = va.NATIVE
    rope = va.Rotary([1.0, 0.5], device="cpu")
    table, lens, free, count = (torch.zeros(s, dtype=torch.int32) for s in ((3, 4), (3,), (9,), (1,)))
    pool, plan = va.PagePool(table, lens, free, count, 16), va.StepPlan(3, 10, "cpu")
    q, pos = torch.zeros(5, 4, 64, dtype=torch.bfloat16), torch.zeros(5, dtype=torch.int32)
    assert rope.at[1] == pool.at[1] == -1
    assert n.rotary(rope.at, 0, q, None, pos, None, None, None) is NotImplemented
    assert n.cache_plan(pool.at, 3, lens, None, 10, plan.args) is NotImplemented
    assert n.cache_trim(pool.at, 3, lens, None) is NotImplemented
    assert n.cache_move([], 3, lens, table, lens) is NotImplemented


@pytest.mark.parametrize("args", [(), (None,), ((1, 2), 3), ((1, -1),) * 6, ((1, -1),) * 9, ("x",) * 8, ((1.5, -1),) + (None,) * 7,
                                  ((1 << 70, -1),) + (None,) * 7, ([],) * 5, ([None],) * 5, ([(1, -1)], 1, 2, 3, 4)])
def test_other_arguments_are_left_to_ctypes(va, args):
    for name in ("rotary", "rotary_cache_write", "cache_plan", "cache_trim", "cache_move", "attention_fwd_paged_tree", "bind"):
        if name == "bind" and len(args) == 7:
            continue
        assert getattr(va.NATIVE, name)(*args) is NotImplemented


def test_handles_carry_their_address(va):
    import ctypes
    rope = va.Rotary([1.0, 0.5], device="cpu")
    assert rope.at == (ctypes.addressof(rope.struct), -1)
    with pytest.raises(AttributeError):
        rope.at = (0, 0)


def test_a_binding_of_another_torch_is_not_loaded(va, monkeypatch):
    assert build.binding_built()
    assert torch.__version__ in build.binding_tag()
    monkeypatch.setattr(build, "binding_tag", lambda: "another")
    assert not build.binding_built()
    assert va._load_binding(va.LIB) is None


def test_plans_past_32_bits(va):
    for args in ((3, 1 << 31), (1 << 31, 3), (-1, 3), (3, -1)):
        with pytest.raises(ValueError):
            va.StepPlan(*args, "cpu")
    with pytest.raises(ValueError):
        va.StepPlan(3, 3, "cpu", mask_words=1 << 31)

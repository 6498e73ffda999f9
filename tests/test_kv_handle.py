"""The cache's handle and its tensors: what a call reaches is what the attributes hold."""
import copy

import pytest
import torch

import fp8_block_scaled_12_b200 as F
from fp8_block_scaled_12_b200.kv import _CacheStruct


def reached(c):
    """The structure that a call on this cache is given."""
    s = c._ref._obj
    return {n: getattr(s, n) for n, _ in _CacheStruct._fields_}


def test_assigned_tensors_are_the_ones_that_calls_reach():
    c = F.KVCache(4, 16, 2, 64, device="cpu")
    for name in ("k", "v", "k_scale", "v_scale"):
        t = getattr(c, name).clone()
        setattr(c, name, t)
        assert getattr(c, name) is t and reached(c)[name] == t.data_ptr()
    c.fmt, c.scale_fmt = F.E5M2, F.SCALE_UE8M0
    assert reached(c)["fmt"] == F.E5M2 and reached(c)["scale_fmt"] == F.SCALE_UE8M0


def test_tensors_that_do_not_fit_are_refused_and_nothing_changes():
    c = F.KVCache(4, 16, 2, 64, device="cpu")
    before, k = reached(c), c.k
    for name, bad, err in (("k", c.k[:2], ValueError), ("v", c.v.float(), TypeError),
                           ("k", c.k.transpose(1, 2).contiguous().transpose(1, 2), ValueError),
                           ("v_scale", c.v_scale.double(), TypeError), ("k_scale", c.k_scale[:, :1], ValueError),
                           ("v", c.v.to("meta"), ValueError), ("fmt", 7, ValueError), ("scale_fmt", -1, ValueError)):
        with pytest.raises(err):
            setattr(c, name, bad)
    for name in ("num_pages", "heads", "page_size", "head_dim", "device", "index"):
        with pytest.raises(AttributeError):
            setattr(c, name, getattr(c, name))
    assert c.k is k and reached(c) == before
    c.owner = "a user's own attribute"
    assert reached(c) == before


def test_a_copy_has_its_own_tensors():
    c = F.KVCache(4, 16, 2, 64, device="cpu")
    before, d = reached(c), copy.copy(c)
    d.k = c.k.clone()
    assert reached(c) == before and reached(d)["k"] == d.k.data_ptr() != before["k"]


@pytest.mark.gpu
def test_a_write_after_an_assignment_goes_to_the_new_memory(cuda_device):
    P, H, D, T = 16, 2, 64, 40
    c = F.KVCache(4, P, H, D)
    old = {n: getattr(c, n) for n in ("k", "v", "k_scale", "v_scale")}
    for t in old.values():
        t.fill_(3)
    for n, t in old.items():
        setattr(c, n, torch.empty_like(t))
    k, v = (torch.randn((T, H, D), device="cuda").to(torch.bfloat16) for _ in range(2))
    slots = torch.arange(T, device="cuda")
    F.kv_write(k, v, slots, c)
    d = F.KVCache(4, P, H, D)
    F.kv_write(k, v, slots, d)
    n = T // P
    for name in old:
        assert torch.equal(getattr(c, name)[:n], getattr(d, name)[:n])
        assert (old[name] == 3).all()
    table = torch.arange(4, dtype=torch.int32, device="cuda").view(1, 4)
    lens = torch.tensor([T], dtype=torch.int32, device="cuda")
    q = torch.randn((1, 8, D), device="cuda").to(torch.bfloat16)
    assert torch.equal(F.paged_attention(q, c, table, lens), F.paged_attention(q, d, table, lens))
    assert F.fp8_device_error() == 0

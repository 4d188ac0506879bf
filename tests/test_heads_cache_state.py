"""What a KVCache holds and what its calls are given stay the same thing, on the host."""
import copy
import ctypes
import pickle

import pytest
import torch

from tests.test_layers_host import sc  # noqa: F401  (a fixture)

MEMORY = ("k", "v", "k_scale", "v_scale")


def agrees(c):
    s = c._struct
    assert [getattr(s, n) for n in MEMORY] == [getattr(c, n).data_ptr() for n in MEMORY]
    assert s.table == (None if c.table is None else c.table.data_ptr())
    assert (s.B, s.N, s.P, s.Hkv, s.D) == (c.B, c.N, c.blocks, c.Hkv, c.D)
    assert ctypes.addressof(c._ref._obj) == ctypes.addressof(s)


def test_replaced_memory_reaches_the_calls(sc):
    c = sc.KVCache(3, 128, 2, 32, device="cpu")
    agrees(c)
    order = torch.tensor([4, 5, 0, 1, 2, 3])      # the sequences in another order
    for n in MEMORY:
        old = getattr(c, n)
        setattr(c, n, old[order])
        assert getattr(c, n).data_ptr() != old.data_ptr()
        agrees(c)
    c.table = torch.arange(6, dtype=torch.int32).view(3, 2)
    agrees(c)


def test_memory_of_another_kind_is_refused(sc):
    c = sc.KVCache(3, 128, 2, 32, device="cpu")
    before = [getattr(c, n) for n in MEMORY]
    for n in MEMORY:
        t = getattr(c, n)
        for bad in (t[:4], t.double(), t[:, :1], torch.cat([t, t], -1)[..., :t.shape[-1]], t.to("meta")):
            with pytest.raises(ValueError):
                setattr(c, n, bad)
    assert all(a is b for a, b in zip(before, (getattr(c, n) for n in MEMORY)))
    agrees(c)
    for n in ("B", "N", "blocks", "Hkv", "D", "code", "device"):
        with pytest.raises(AttributeError):
            setattr(c, n, getattr(c, n))


def test_copies_do_not_share_a_struct(sc):
    table = torch.arange(6, dtype=torch.int32).view(3, 2)
    a = sc.KVCache(3, 128, 2, 32, "e4m3", device="cpu")
    b = copy.copy(a)
    assert b.k is a.k and b.v_scale is a.v_scale
    b.table = table
    b.k = a.k.clone()
    assert a.table is None and a._struct.table is None
    agrees(a)
    agrees(b)
    d = copy.deepcopy(b)
    e = pickle.loads(pickle.dumps(b))
    for c in (d, e):
        assert torch.equal(c.table, table) and c.table is not table and c.code == "e4m3"
        assert all(getattr(c, n).data_ptr() != getattr(b, n).data_ptr() for n in MEMORY)
        agrees(c)

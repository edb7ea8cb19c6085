"""Refusals of the layer operators' further entry points and attributes, without a GPU."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from test_layer_cpu import OK, _cache, layer, moe  # noqa: E402, F401


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(ks=4), -2), (dict(v=None), -1), (dict(c=None), -1), (dict(held=0x10001), -1),
    (dict(ws=None), -3), (dict(n=1024), -3),
])
def test_append_held_refuses(moe, kw, status):  # noqa: F811
    a = dict(k=OK, ks=256, v=OK, vs=256, starts=OK, t=3, c=ctypes.byref(_cache(moe)), held=OK, ws=OK, n=1 << 30)
    a.update(kw)
    assert moe.load_library().moe_kv_append_held(*a.values(), None) == status


@pytest.mark.parametrize("name", ["codes", "scales", "tail", "table", "lens", "held", "ws"])
def test_cache_tensors_cannot_be_replaced(layer, name):  # noqa: F811
    """The kernels keep the addresses of the first ones."""
    cache = object.__new__(layer.KvCache)
    with pytest.raises(AttributeError):
        setattr(cache, name, torch.zeros(1))

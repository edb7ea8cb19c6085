"""Refusals of the layer operators, before any CUDA call: argument errors the
C ABI reports, and those the Python binding catches because the library sees
bare pointers only."""

import ctypes

import pytest

torch = pytest.importorskip("torch")

from routed_expert_prefill_gb300 import build as B  # noqa: E402


@pytest.fixture(scope="module")
def moe():
    B.build()
    from routed_expert_prefill_gb300 import moe as m

    m.load_library()
    return m


@pytest.fixture(scope="module")
def layer(moe):
    from routed_expert_prefill_gb300 import layer as m

    return m


OK, ODD = 0x10000, 0x10002  # 16-byte aligned and misaligned addresses; never dereferenced here


def _norm(moe, **kw):
    a = dict(x=OK, xs=256, r=OK, rs=256, g=OK, eps=1e-6, t=4, h=256, sum=OK, y=OK, codes=None, scales=None)
    a.update(kw)
    return moe.load_library().moe_add_rms_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(h=0), -2), (dict(h=20), -2), (dict(h=16392), -2),
    (dict(xs=4), -2), (dict(xs=-8), -2), (dict(rs=12), -2), (dict(h=72, codes=OK, scales=OK), -2),
    (dict(x=None), -1), (dict(g=None), -1), (dict(x=ODD), -1), (dict(r=ODD), -1), (dict(y=ODD), -1),
    (dict(sum=None, y=None), -1), (dict(codes=OK), -1), (dict(scales=OK), -1), (dict(eps=-1.0), -1),
    (dict(eps=float("nan")), -1),
])
def test_norm_refuses(moe, kw, status):
    assert _norm(moe, **kw) == status
    assert moe.load_library().moe_last_error().decode()


def _qmv(moe, **kw):
    w = moe.MoeQWeights(kw.pop("codes", OK), kw.pop("scales", OK), kw.pop("biases", OK))
    a = dict(x=OK, xs=256, xc=None, xsc=None, w=ctypes.byref(w), t=4, n=100, k=256, y=OK, f=0)
    a.update(kw)
    return moe.load_library().moe_qmv(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(n=0), -2), (dict(n=1 << 21), -2), (dict(k=0), -2), (dict(k=96), -2),
    (dict(k=65600), -2), (dict(xs=4), -2), (dict(x=None), -1), (dict(xc=OK, xsc=OK), -1), (dict(x=None, xc=OK), -1),
    (dict(xsc=OK), -1), (dict(x=ODD), -1), (dict(x=None, xc=ODD, xsc=OK), -1), (dict(w=None), -1),
    (dict(codes=ODD), -1), (dict(scales=None), -1), (dict(biases=0x10001), -1), (dict(y=None), -1),
    (dict(y=ODD, f=1), -1),
])
def test_qmv_refuses(moe, kw, status):
    assert _qmv(moe, **kw) == status
    assert moe.load_library().moe_last_error().decode()


def _cache(moe, **kw):
    a = dict(codes=OK, scales=OK, tail=OK, table=OK, lens=OK, n_seq=2, n_pages=8, max_blocks=4, block=64, hkv=2,
             d=128)
    a.update(kw)
    return moe.MoeKvCache(*a.values())


CACHE_REFUSALS = [
    (dict(d=96), -2), (dict(d=256), -2), (dict(block=48), -2), (dict(block=256), -2), (dict(hkv=0), -2),
    (dict(n_seq=0), -2), (dict(n_pages=0), -2), (dict(max_blocks=0), -2), (dict(max_blocks=1 << 25), -2),
    (dict(codes=None), -1), (dict(scales=None), -1), (dict(tail=ODD), -1), (dict(table=0x10001), -1),
    (dict(lens=None), -1),
]


def _append(moe, cache=None, **kw):
    a = dict(k=OK, ks=256, v=OK, vs=256, starts=OK, t=3, c=ctypes.byref(cache or _cache(moe)), ws=OK,
             n=1 << 30)
    a.update(kw)
    return moe.load_library().moe_kv_append(*a.values(), None)


def _attend(moe, cache=None, **kw):
    a = dict(q=OK, qs=512, starts=OK, t=3, hq=4, scale=1.0, c=ctypes.byref(cache or _cache(moe)), out=OK, ws=OK,
             n=1 << 30)
    a.update(kw)
    return moe.load_library().moe_kv_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", CACHE_REFUSALS)
def test_cache_refused_by_both_calls(moe, kw, status):
    assert _append(moe, _cache(moe, **kw)) == status
    assert _attend(moe, _cache(moe, **kw)) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(ks=4), -2), (dict(vs=-8), -2), (dict(k=None), -1), (dict(v=ODD), -1),
    (dict(starts=None), -1), (dict(c=None), -1), (dict(ws=None), -3), (dict(ws=0x10010), -3), (dict(n=1024), -3),
])
def test_append_refuses(moe, kw, status):
    assert _append(moe, **kw) == status


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(qs=12), -2), (dict(hq=3), -2), (dict(hq=1), -2), (dict(q=ODD), -1), (dict(out=None), -1),
    (dict(scale=float("inf")), -1), (dict(c=None), -1), (dict(starts=None), -1), (dict(ws=None), -3),
    (dict(n=1024), -3),
])
def test_attention_refuses(moe, kw, status):
    assert _attend(moe, **kw) == status


def test_workspace_bytes(moe):
    lib = moe.load_library()
    assert lib.moe_kv_workspace_bytes(96) == 0
    assert 0 < lib.moe_kv_workspace_bytes(64) < lib.moe_kv_workspace_bytes(128)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_norm_binding_refuses(layer):
    x, g = bf(4, 256), bf(256)
    with pytest.raises(TypeError, match="x must have dtype"):
        layer.moe_add_rms_norm(x.float(), g)
    with pytest.raises(ValueError, match="contiguous"):
        layer.moe_add_rms_norm(bf(256, 4).t(), g)
    with pytest.raises(ValueError, match="multiple of 8"):
        layer.moe_add_rms_norm(bf(4, 260)[:, :256], g)
    with pytest.raises(ValueError, match="gamma"):
        layer.moe_add_rms_norm(x, bf(128))
    with pytest.raises(ValueError, match="residual must have 4 rows"):
        layer.moe_add_rms_norm(x, g, bf(3, 256))
    with pytest.raises(ValueError, match="sum_out"):
        layer.moe_add_rms_norm(x, g, sum_out=bf(4, 128))
    with pytest.raises(ValueError, match="multiple of 64"):
        layer.moe_add_rms_norm(bf(4, 72), bf(72), quantize=True)
    with pytest.raises(ValueError, match="CUDA device"):
        layer.moe_add_rms_norm(x, g)


def test_qmv_binding_refuses(layer):
    w = (torch.zeros(100, 128, dtype=torch.uint8), torch.zeros(100, 4, dtype=torch.float16),
         torch.zeros(100, 4, dtype=torch.float16))
    x = bf(4, 256)
    with pytest.raises(TypeError, match="weight codes"):
        layer.moe_qmv(x, (w[0].int(), w[1], w[2]))
    with pytest.raises(ValueError, match="weight scales"):
        layer.moe_qmv(x, (w[0], w[1][:, :3].contiguous(), w[2]))
    with pytest.raises(ValueError, match="x must have shape"):
        layer.moe_qmv(bf(4, 128), w)
    with pytest.raises(TypeError, match="x codes"):
        layer.moe_qmv((torch.zeros(4, 256, dtype=torch.uint8), torch.zeros(4, 4)), w)
    with pytest.raises(ValueError, match="x scales"):
        layer.moe_qmv((torch.zeros(4, 256, dtype=torch.int8), torch.zeros(4, 3)), w)
    with pytest.raises(TypeError, match="out_dtype"):
        layer.moe_qmv(x, w, out_dtype=torch.float16)
    with pytest.raises(ValueError, match="out must have shape"):
        layer.moe_qmv(x, w, out=torch.zeros(4, 99))
    with pytest.raises(ValueError, match="CUDA device"):
        layer.moe_qmv(x, w)


def test_cache_binding_refuses(layer):
    i32 = dict(dtype=torch.int32)
    ok = dict(codes=torch.zeros(2, 8, 2, 64, 128, dtype=torch.int8), scales=torch.zeros(2, 8, 2),
              tail=bf(3, 2, 2, 128, 128), table=torch.zeros(3, 4, **i32), lens=torch.zeros(3, **i32))
    for name, bad, err in (("codes", ok["codes"][0], ValueError), ("codes", ok["codes"].to(torch.uint8), TypeError),
                           ("scales", torch.zeros(2, 8), ValueError), ("tail", bf(3, 2, 2, 64, 128), ValueError),
                           ("table", torch.zeros(3, 4), TypeError), ("lens", torch.zeros(2, **i32), ValueError)):
        with pytest.raises(err, match=name):
            layer.KvCache(**{**ok, name: bad})
    with pytest.raises(ValueError, match="CUDA device"):
        layer.KvCache(**ok)
    with pytest.raises(TypeError, match="KvCache"):
        layer.moe_kv_append(bf(4, 2, 128), bf(4, 2, 128), torch.zeros(4, **i32), ok)

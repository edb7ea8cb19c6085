"""Refusals of the operators of a serving step (norms around a block, page
plan, linear attention, log probabilities), before any CUDA call: argument
errors the C ABI reports, and those the Python binding catches because the
library sees bare pointers only."""

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


def _refused(moe, status, got):
    assert got == status
    assert moe.load_library().moe_last_error().decode()


def _gated(moe, gate=None, **kw):
    g = None if gate is None else ctypes.byref(moe.MoeGate(*gate))
    a = dict(x=OK, xs=256, post=OK, g=g, r=OK, rs=256, scale=1.0, gamma=OK, eps=1e-6, t=4, h=256, sum=OK, y=OK,
             codes=None, scales=None)
    a.update(kw)
    return moe.load_library().moe_gated_rms_norm(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(h=0), -2), (dict(h=20), -2), (dict(h=16392), -2),
    (dict(xs=4), -2), (dict(xs=-8), -2), (dict(rs=12), -2), (dict(h=72, codes=OK, scales=OK), -2),
    (dict(x=None), -1), (dict(gamma=None), -1), (dict(post=ODD), -1), (dict(x=ODD), -1), (dict(r=ODD), -1),
    (dict(y=ODD), -1), (dict(sum=None, y=None), -1), (dict(codes=OK), -1), (dict(scales=OK), -1),
    (dict(eps=-1.0), -1), (dict(eps=float("nan")), -1), (dict(scale=float("inf")), -1), (dict(scale=float("nan")), -1),
    (dict(gate=(None, 0, 1, 0)), -1), (dict(gate=(ODD, 0, 1, 0)), -1), (dict(gate=(0x10001, 1, 0, 0)), -1),
    (dict(gate=(OK, 12, 1, 0)), -2), (dict(gate=(OK, -8, 1, 0)), -2), (dict(gate=(OK, -1, 0, 0)), -2),
])
def test_gated_norm_refuses(moe, kw, status):
    _refused(moe, status, _gated(moe, **kw))


def _plan(moe, pages=(OK, OK, OK), **kw):
    a = dict(fresh=OK, before=OK, lens=OK, table=OK, pages=None if pages is None else ctypes.byref(moe.MoeKvPages(*pages)),
             n_seq=3, n_pages=8, max_blocks=4, block=64, t=5, starts=OK, seq=OK, pos=OK, slot=OK, ws=OK, n=1 << 20)
    a.update(kw)
    return moe.load_library().moe_kv_plan(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(n_seq=0), -2), (dict(n_seq=65537), -2), (dict(n_pages=0), -2),
    (dict(block=48), -2), (dict(block=256), -2), (dict(max_blocks=0), -2), (dict(max_blocks=1 << 25), -2),
    (dict(fresh=None), -1), (dict(before=None), -1), (dict(lens=0x10001), -1), (dict(table=None), -1),
    (dict(pages=None), -1), (dict(pages=(None, OK, OK)), -1), (dict(pages=(OK, ODD, OK)), -1),
    (dict(pages=(OK, OK, None)), -1), (dict(starts=None), -1), (dict(seq=ODD), -1), (dict(slot=0x10004), -1),
    (dict(ws=None), -3), (dict(ws=0x10010), -3), (dict(n=512), -3),
])
def test_plan_refuses(moe, kw, status):
    _refused(moe, status, _plan(moe, **kw))


def _linear(moe, **kw):
    a = dict(q=OK, qs=256, k=OK, ks=256, v=OK, vs=512, g=OK, gs=4, starts=OK, t=5, n_seq=2, hk=2, hv=4, d=128, scale=1.0,
             states=OK, n_slots=2, slots=None, out_slots=None, out=OK, ws=OK, n=1 << 30)
    a.update(kw)
    return moe.load_library().moe_linear_attention(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(n_seq=0), -2), (dict(n_seq=65537), -2), (dict(d=96), -2),
    (dict(d=256), -2), (dict(hk=0), -2), (dict(hk=3), -2), (dict(hk=8), -2), (dict(hv=0), -2), (dict(hk=1, hv=1025), -2),
    (dict(n_slots=0), -2), (dict(n_slots=1), -2), (dict(qs=4), -2), (dict(ks=-8), -2), (dict(vs=12), -2), (dict(gs=-1), -2),
    (dict(scale=float("inf")), -1), (dict(q=None), -1), (dict(k=ODD), -1), (dict(v=None), -1), (dict(g=ODD), -1),
    (dict(starts=None), -1), (dict(states=None), -1), (dict(states=0x10004), -1), (dict(slots=ODD), -1),
    (dict(out_slots=ODD), -1), (dict(out=None), -1), (dict(ws=None), -3), (dict(ws=0x10010), -3), (dict(n=64), -3),
])
def test_linear_attention_refuses(moe, kw, status):
    _refused(moe, status, _linear(moe, **kw))


def _logprobs(moe, **kw):
    a = dict(x=OK, stride=100, f32=1, t=4, n=100, ids=OK, ids64=1, n_ids=1, top=5, lp=OK, ent=OK, lse=OK, tid=OK, tlp=OK)
    a.update(kw)
    return moe.load_library().moe_logprobs(*a.values(), None)


@pytest.mark.parametrize("kw,status", [
    (dict(t=0), -2), (dict(t=65537), -2), (dict(n=0), -2), (dict(n=(1 << 20) + 1), -2), (dict(stride=-1), -2),
    (dict(n_ids=-1), -2), (dict(n_ids=257), -2), (dict(top=-1), -2), (dict(top=33), -2), (dict(n=4), -2),
    (dict(x=None), -1), (dict(x=ODD), -1), (dict(x=0x10001, f32=0), -1), (dict(ids=None), -1), (dict(ids=0x10004), -1),
    (dict(ids=ODD, ids64=0), -1), (dict(lp=None), -1), (dict(ent=ODD), -1), (dict(tid=None), -1), (dict(tlp=ODD), -1),
])
def test_logprobs_refuses(moe, kw, status):
    _refused(moe, status, _logprobs(moe, **kw))


def test_workspace_bytes(moe):
    lib = moe.load_library()
    assert lib.moe_linear_workspace_bytes(96) == 0 and lib.moe_linear_workspace_bytes(128) > 0
    assert lib.moe_kv_plan_workspace_bytes(0) == 0 == lib.moe_kv_plan_workspace_bytes(65537)
    assert 0 < lib.moe_kv_plan_workspace_bytes(1) < lib.moe_kv_plan_workspace_bytes(65536)


def bf(*shape):
    return torch.zeros(shape, dtype=torch.bfloat16)


def test_gated_norm_binding_refuses(layer):
    x, g = bf(4, 256), bf(256)
    f = layer.moe_gated_rms_norm
    with pytest.raises(TypeError, match="x must have dtype"):
        f(x.float(), g)
    with pytest.raises(ValueError, match="gamma"):
        f(x, bf(128))
    with pytest.raises(ValueError, match="post_gamma"):
        f(x, g, post_gamma=bf(128))
    with pytest.raises(ValueError, match="residual must have 4 rows"):
        f(x, g, bf(3, 256))
    with pytest.raises(ValueError, match="gate must have shape"):
        f(x, g, gate=bf(4))
    with pytest.raises(ValueError, match="gate must have shape"):
        f(x, g, gate=bf(3, 256))
    with pytest.raises(TypeError, match="gate must have dtype"):
        f(x, g, gate=torch.zeros(256))
    with pytest.raises(ValueError, match="gate: rows"):
        f(x, g, gate=bf(4, 260)[:, :256])
    with pytest.raises(ValueError, match="sum_out"):
        f(x, g, sum_out=bf(4, 128))
    with pytest.raises(ValueError, match="multiple of 64"):
        f(bf(4, 72), bf(72), quantize=True)
    with pytest.raises(ValueError, match="CUDA device"):
        f(x, g, gate=bf(4, 1))


def test_plan_binding_refuses(layer):
    with pytest.raises(TypeError, match="KvCache"):
        layer.KvPages(None)
    with pytest.raises(TypeError, match="KvPages"):
        layer.moe_kv_plan(torch.zeros(3, dtype=torch.int32), None, None, 4)


def test_linear_state_refuses(layer):
    for bad in (torch.zeros(3, 2, 128), torch.zeros(3, 2, 128, 64)):
        with pytest.raises(ValueError, match="states must be"):
            layer.LinearState(bad)
    with pytest.raises(TypeError, match="states must have dtype"):
        layer.LinearState(bf(3, 2, 64, 64))
    with pytest.raises(ValueError, match="CUDA device"):
        layer.LinearState(torch.zeros(3, 2, 64, 64))
    with pytest.raises(TypeError, match="LinearState"):
        layer.moe_linear_attention(bf(3, 2, 64), bf(3, 2, 64), bf(3, 2, 64), torch.zeros(2), torch.zeros(2), None)


def test_logprobs_binding_refuses(layer):
    x = torch.zeros(4, 100)
    f = layer.moe_logprobs
    with pytest.raises(ValueError, match=r"\[t, n\]"):
        f(x[0])
    with pytest.raises(TypeError, match="logits must have dtype"):
        f(x.double())
    with pytest.raises(ValueError, match="contiguous"):
        f(torch.zeros(100, 4).t())
    with pytest.raises(ValueError, match="ids must have shape"):
        f(x, torch.zeros(3, dtype=torch.int64))
    with pytest.raises(TypeError, match="ids must have dtype"):
        f(x, torch.zeros(4))
    with pytest.raises(ValueError, match="CUDA device"):
        f(x, torch.zeros(4, dtype=torch.int64))


def test_names_of_the_package(layer):
    """The calls and handles are names of the package itself, as those of the other layer operators."""
    import routed_expert_prefill_gb300 as package

    for name in ("moe_gated_rms_norm", "KvPages", "moe_kv_plan", "LinearState", "moe_linear_attention", "moe_logprobs"):
        assert name in package.__all__
        assert getattr(package, name) is getattr(layer, name)

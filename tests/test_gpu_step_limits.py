"""The operators of a serving step at the ends of their ranges: kernel forms
that only large sizes reach, chains of chunks that several CTAs share, waits
that run out, offsets past 32 bits, rows that lie over one another."""

import math
import time

import pytest

torch = pytest.importorskip("torch")

from test_gpu_layer import BF16, F64, gen, i32, layer, randn, within  # noqa: E402, F401
from test_gpu_step import F32, check_linear, check_logprobs, gated_ref, plan_state, run_plan, starts_of  # noqa: E402

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- norms around a block

# many rows, walked by a grid that fills the SMs: a CTA a row of one, two and four vectors a thread, a warp a row
@pytest.mark.parametrize("t,h", [(1500, 2056), (1400, 1032), (1100, 8200), (700, 16384), (9001, 128), (8200, 1024),
                                 (8200, 264), (20011, 512), (65536, 8)])
@pytest.mark.parametrize("gate,sigmoid", [("none", False), ("channel", True), ("row", False), ("full", False)])
def test_gated_norm_of_many_rows(layer, t, h, gate, sigmoid):
    g = gen(t + h)
    x, res, gamma, post = ((randn(g, *s) * m).bfloat16() for s, m in (((t, h), 3), ((t, h), 1), ((h,), 1), ((h,), 1)))
    x[0, :: max(1, h // 3)] = 200.0
    shape = {"none": None, "channel": (h,), "row": (t, 1), "full": (t, h)}[gate]
    z = None if shape is None else randn(g, *shape).bfloat16()
    stream = res.clone()
    for post_, res_, into in ((post, res, None), (post, stream, stream), (None, res, None), (post, None, None)):
        q8 = h % 64 == 0 and into is None
        out = layer.moe_gated_rms_norm(x, gamma, res_, post_, z, gate_sigmoid=sigmoid, residual_scale=0.37, eps=1e-5,
                                       quantize=q8, want_y=True, sum_out=into)
        a, y, ea, ey = gated_ref(x, gamma, res if into is not None else res_, post_, z, sigmoid, 0.37, 1e-5)
        within(out.y, y, BF16 * y.abs() + 1.01 * ey + 1e-38)
        if res_ is not None:
            within(out.sum, a, BF16 * a.abs() + 1.01 * ea)
        if q8:
            m = y.view(t, h // 64, 64).abs().amax(-1)
            e = ey.view(t, h // 64, 64).amax(-1)
            within(out.scales, m / 127, (e + 4 * F32 * m) / 127)
            within(out.codes.view(t, h // 64, 64).to(F64) * out.scales.to(F64).unsqueeze(-1), y.view(t, h // 64, 64),
                   ((0.5 + 127 * 8 * F32) * m / 127 + 3 * e).unsqueeze(-1))
    only = layer.moe_gated_rms_norm(x, gamma, res, post, z, gate_sigmoid=sigmoid, residual_scale=0.37, want_y=False)
    assert only.y is None
    a, _, ea, _ = gated_ref(x, gamma, res, post, z, sigmoid, 0.37, 1e-6)
    within(only.sum, a, BF16 * a.abs() + 1.01 * ea)


def test_gated_norm_one_row_for_all(layer):
    """Stride 0: the residual, the gate or the block's output is one row for many."""
    g = gen(5)
    t, h = 2000, 4096
    x, one, z = randn(g, t, h).bfloat16(), randn(g, 1, h).bfloat16(), randn(g, 1, h).bfloat16()
    gamma = randn(g, h).bfloat16()
    a = layer.moe_gated_rms_norm(x, gamma, one.expand(t, h), gamma, z.expand(t, h))
    b = layer.moe_gated_rms_norm(x, gamma, one.expand(t, h).contiguous(), gamma, z[0])
    assert torch.equal(a.sum, b.sum) and torch.equal(a.y, b.y)
    c = layer.moe_gated_rms_norm(one.expand(t, h), gamma, x, gamma)
    d = layer.moe_gated_rms_norm(one.expand(t, h).contiguous(), gamma, x, gamma)
    assert torch.equal(c.sum, d.sum) and torch.equal(c.y, d.y)


# ---------------------------------------------------------------- plan

def test_plan_of_the_most_sequences_and_rows(layer):
    n = 65536
    cache, pages = plan_state(layer, n, n // 2, 1, 16)
    assert run_plan(layer, cache, pages, [1, 0] * (n // 2), n)
    assert not run_plan(layer, cache, pages, [0, 1] + [0] * (n - 2), 1)  # no page is left
    assert run_plan(layer, cache, pages, [-1, 0] * (n // 4) + [0, 0] * (n // 4), 1)
    assert run_plan(layer, cache, pages, [0, 2] * (n // 4) + [1, 0] * (n // 4), n)


# ---------------------------------------------------------------- linear attention

@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,hk,hv", [([600, 130, 257, 0, 700], 8, 32), ([129] * 20, 4, 12), ([3000], 1, 1), ([900, 30], 3, 6),
                                        ([40] * 40, 2, 8)])
def test_linear_attention_chains_that_ctas_share(layer, d, lens, hk, hv):
    """Runs of chunks that begin and end inside a chain, hold several, or lie inside one."""
    check_linear(layer, lens, hk, hv, d, True, seed=len(lens))


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens,hk,hv", [([600] * 7, 4, 16), ([700, 600, 513] * 5, 2, 8), ([1100, 30, 0, 1000] * 4, 4, 8)])
def test_linear_attention_runs_about_as_long_as_chains(layer, d, lens, hk, hv):
    check_linear(layer, lens, hk, hv, d, True, seed=len(lens) + d)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n", [5, 300])
def test_linear_attention_states_at_an_odd_place(layer, d, n):
    """A pool that begins at a multiple of 16 bytes that is none of 32."""
    g = gen(d + n)
    q, k, v = (randn(g, 2 * n, 2, d).bfloat16() for _ in range(3))
    logs = -torch.rand(2 * n, 2, generator=g, device="cuda")
    starts = i32([0, n, 2 * n])
    first = randn(g, 2, 2, d, d)
    a = layer.LinearState(first.clone())
    b = layer.LinearState(torch.empty(first.numel() + 4, device="cuda")[4:].view(first.shape).copy_(first))
    assert a.states.data_ptr() % 32 == 0 and b.states.data_ptr() % 32 == 16
    assert torch.equal(layer.moe_linear_attention(q, k, v, logs, starts, a), layer.moe_linear_attention(q, k, v, logs, starts, b))
    assert torch.equal(a.states, b.states)
    assert a.read_device_status() == 0 == b.read_device_status()


def test_linear_attention_moves_states_of_sequences_without_rows(layer):
    """Between long ones: a sequence without rows leaves its state in another slot, or keeps it."""
    check_linear(layer, [300, 0, 0, 200, 0], 2, 4, 64, True, n_slots=9, pick=([7, 1, 3, -1, -1], [2, 1, 5, 8, 0]))
    check_linear(layer, [0, 0, 300], 2, 4, 128, False, n_slots=9, pick=([7, 4, 3], [-1, 6, -1]))


@pytest.mark.parametrize("n", [5, 300])
def test_linear_attention_rows_that_lie_over_one_another(layer, n):
    """One row of queries for all (stride 0), slices of wider decays."""
    g = gen(2)
    q, k, v = randn(g, 1, 2, 64).bfloat16(), randn(g, n, 2, 64).bfloat16(), randn(g, n, 4, 64).bfloat16()
    wide = -0.3 * torch.rand(n, 11, generator=g, device="cuda")
    starts = i32([0, n])
    a, b = layer.LinearState.new(1, 4, 64), layer.LinearState.new(1, 4, 64)
    one = layer.moe_linear_attention(q.expand(n, 2, 64), k, v, wide[:, 3:7], starts, a)
    other = layer.moe_linear_attention(q.expand(n, 2, 64).contiguous(), k, v, wide[:, 3:7].contiguous(), starts, b)
    ref = b.states.to(F64)
    # two orders of the same sums: each within its own bound of the definition, so within twice that of the other
    size = torch.zeros(1, 4, 64, 64, dtype=F64, device="cuda")
    for r in range(n):
        lam = torch.exp(wide[r, 3:7].to(F64))[:, None, None]
        size = size * lam + (k[r].to(F64).abs().repeat_interleave(2, 0).unsqueeze(-1) * v[r].to(F64).abs().unsqueeze(-2))
    within(a.states, ref, 2 * (6 * n + 64) * F32 * size + 1e-38)
    mag = (q[0].to(F64).abs().repeat_interleave(2, 0).unsqueeze(-1) * size).sum(-2) / 8
    within(one[-1], other[-1].to(F64), 2 * BF16 * other[-1].to(F64).abs() + 2 * ((6 * n + 128) * F32 + 2.0 ** -16) * mag)


def test_linear_attention_wait_that_runs_out(layer):
    """A part that is never published: the call ends with MOE_ETIMEOUT, and the next one on the workspace is right."""
    from routed_expert_prefill_gb300 import moe

    g = gen(6)
    q, k, v = (randn(g, 900, 2, 128).bfloat16() for _ in range(3))
    logs = torch.full((2,), -0.05, device="cuda")
    starts = i32([0, 900])
    clean = layer.LinearState.new(1, 2, 128)
    ref = layer.moe_linear_attention(q, k, v, logs, starts, clean)
    state = layer.LinearState.new(1, 2, 128)
    moe.debug_stall(state.ws, moe.MOE_STALL_GRID_BARRIER)
    torch.cuda.synchronize()
    t0 = time.monotonic()
    layer.moe_linear_attention(q, k, v, logs, starts, state)
    assert state.read_device_status() == -6  # MOE_ETIMEOUT
    assert time.monotonic() - t0 < 20
    state.states.zero_()
    out = layer.moe_linear_attention(q, k, v, logs, starts, state)
    assert state.read_device_status() == 0
    assert torch.equal(out, ref) and torch.equal(state.states, clean.states)


def test_linear_attention_states_past_32_bits(layer):
    """The last slots of a pool of more than 2^31 values, by either kernel."""
    hv, d, n_slots = 16, 128, 8300
    if torch.cuda.mem_get_info()[0] < 12e9:
        pytest.skip("needs 9 GB")
    states = torch.zeros(n_slots, hv, d, d, device="cuda")
    state = layer.LinearState(states)
    small = layer.LinearState.new(2, hv, d)
    g = gen(1)
    for n in (3, 150):
        q, k, v = (randn(g, n, hv, d).bfloat16() for _ in range(3))
        logs = torch.full((hv,), -0.1, device="cuda")
        a = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), state, i32([n_slots - 1]), i32([n_slots - 2]))
        b = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), small, i32([1]), i32([0]))
        assert torch.equal(a, b) and torch.equal(states[-2], small.states[0]) and not states[-1].any()
    assert not states[:-2].any() and state.read_device_status() == 0


@pytest.mark.parametrize("d", [64, 128])
def test_linear_attention_two_calls_at_once(layer, d):
    """Pools of their own on streams of their own, each call's CTAs waiting for one another's states."""
    g = gen(31)
    calls = []
    for n, hv in ((1500, 3), (1100, 5)):
        q, k, v = (randn(g, n, hv, d).bfloat16() for _ in range(3))
        logs = -0.1 * torch.rand(n, hv, generator=g, device="cuda")
        starts = i32([0, n // 3, n])
        state = layer.LinearState.new(2, hv, d)
        out = layer.moe_linear_attention(q, k, v, logs, starts, state)
        calls.append((q, k, v, logs, starts, out, state.states.clone(), layer.LinearState.new(2, hv, d), torch.cuda.Stream()))
    torch.cuda.synchronize()
    for _ in range(20):
        got = []
        for q, k, v, logs, starts, _, _, state, stream in calls:
            with torch.cuda.stream(stream):
                state.states.zero_()
                got.append(layer.moe_linear_attention(q, k, v, logs, starts, state))
        torch.cuda.synchronize()
        for out, (*_, ref, states, state, _) in zip(got, calls):
            assert torch.equal(out, ref) and torch.equal(state.states, states) and state.read_device_status() == 0


@pytest.mark.parametrize("n", [6, 250])
def test_linear_attention_decay_that_is_nan(layer, n):
    """From its row on that head is NaN; rows before it and other heads are not touched."""
    g = gen(17)
    q, k, v = (randn(g, n, 2, 64).bfloat16() for _ in range(3))
    logs = torch.full((n, 2), -0.1, device="cuda")
    a, b = layer.LinearState.new(1, 2, 64), layer.LinearState.new(1, 2, 64)
    ref = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), a)
    logs[n // 2, 0] = math.nan
    out = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), b)
    assert torch.equal(out[:, 1], ref[:, 1]) and torch.equal(b.states[:, 1], a.states[:, 1])
    assert torch.equal(out[:n // 2, 0], ref[:n // 2, 0])
    assert out[n // 2:, 0].isnan().all() and b.states[0, 0].isnan().all()


def test_two_pools_in_one_captured_graph(layer):
    """Calls of both kernels in a graph, replayed while the same leaves are used eagerly between."""
    g = gen(14)
    q, k, v = (randn(g, 400, 2, 64).bfloat16() for _ in range(3))
    logs = torch.full((2,), -0.1, device="cuda")
    starts, one = i32([0, 300, 400]), i32([0, 1])
    a, b = layer.LinearState.new(2, 2, 64), layer.LinearState.new(1, 2, 64)

    def step():
        return (layer.moe_linear_attention(q, k, v, logs, starts, a),
                layer.moe_linear_attention(q[:1], k[:1], v[:1], logs, one, b))

    ref = []
    for _ in range(3):
        ref.append([t.clone() for t in step()] + [a.states.clone(), b.states.clone()])
    a.states.zero_(), b.states.zero_()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            made = step()
        a.states.zero_(), b.states.zero_()
        for i, r in enumerate(ref):
            if i == 1:
                got = step()  # eager, between two replays
            else:
                graph.replay()
                got = made
            for x, y in zip(list(got) + [a.states, b.states], r):
                assert torch.equal(x, y)
    side.synchronize()
    assert a.read_device_status() == 0 == b.read_device_status()


# ---------------------------------------------------------------- log probabilities

def test_logprobs_rows_past_32_bits(layer):
    if torch.cuda.mem_get_info()[0] < 12e9:
        pytest.skip("needs 9 GB")
    t, stride, n = 2100, 1050000, 5001
    big = torch.empty(t * stride, device="cuda")
    x = big.as_strided((t, n), (stride, 1))
    x.copy_(randn(gen(3), t, n))
    ids = torch.randint(0, n, (t,), generator=gen(4), device="cuda")
    check_logprobs(layer, x, ids, 5)


@pytest.mark.parametrize("t", [65536, 40, 77, 153, 305])
def test_logprobs_row_counts(layer, t):
    """The most rows; those around which fewer CTAs share a row."""
    n = 70 if t > 1000 else 40000
    x = randn(gen(t), t, n).bfloat16()
    check_logprobs(layer, x, torch.randint(0, n, (t, 2), generator=gen(1), device="cuda", dtype=torch.int32), 8)


def test_logprobs_most_tokens_and_alternatives(layer):
    x = randn(gen(8), 3, 300)
    ids = torch.randint(0, 300, (3, 256), generator=gen(9), device="cuda")
    check_logprobs(layer, x, ids, 32)
    r = layer.moe_logprobs(x, torch.zeros(3, 0, dtype=torch.int64, device="cuda"))
    assert r.logprob.shape == (3, 0) and torch.isfinite(r.lse).all()
    none = layer.moe_logprobs(x)
    assert none.logprob is None and torch.equal(none.entropy, r.entropy)


def test_logprobs_of_the_products_that_feed_them(layer):
    """fp32 logits of a vocabulary product, and their own tokens' log probabilities summing to one over the row."""
    g = gen(11)
    x = randn(g, 4, 77)
    every = torch.arange(77, device="cuda").expand(4, 77).contiguous()
    lp = layer.moe_logprobs(x, every, top=32)
    total = lp.logprob.to(F64).exp().sum(-1)
    # 77 probabilities, each off by its exponent's error, and they add up to one
    within(total, torch.ones_like(total), 77 * 2 * F32 * (1 + lp.logprob.to(F64).abs().amax(-1)) + (77 / 256 + 80) * F32)
    assert torch.equal(lp.top_logprobs, torch.gather(lp.logprob, 1, lp.top_ids.long()))
    assert math.isclose(float(lp.top_logprobs[0, 0]), float(lp.logprob[0].max()), rel_tol=0, abs_tol=0)

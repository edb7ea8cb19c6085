"""The operators of a serving step (norms around a block, page plan, linear
attention, log probabilities) against plain 64-bit implementations.

Tolerances are derived, not fitted: a rounding to bf16 is off by 2^-8 of the
exact value at most (half a step), one to fp32 by 2^-24, and each test states
the bound of its own sums.
"""

import math
import random

import pytest

torch = pytest.importorskip("torch")

from test_gpu_layer import BF16, F64, gen, i32, layer, randn, weights, within  # noqa: E402, F401

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24


def starts_of(lens):
    a = [0]
    for n in lens:
        a.append(a[-1] + n)
    return a


# ---------------------------------------------------------------- norms around a block

def gated_ref(x, gamma, residual, post, gate, sigmoid, scale, eps):
    """a, y, and bounds of the fp32 errors before either is rounded."""
    f, h = (lambda v: v.to(F64)), x.shape[1]
    b = f(x)
    if post is not None:
        b = b / ((b * b).mean(-1, keepdim=True) + eps).sqrt() * f(post)
    if gate is not None:
        b = b * (torch.sigmoid(f(gate)) if sigmoid else f(gate))
    r = torch.zeros_like(b) if residual is None else scale * f(residual)
    a = r + b
    # a sum of h squares without cancellation: h / 8 + 16 roundings, halved by the root; the
    # gate's exponential, quotients and products are 16 more; then the sum of the two terms
    ea = (h / 16 + 32) * F32 * (b.abs() + r.abs())
    rstd = 1 / ((a * a).mean(-1, keepdim=True) + eps).sqrt()
    y = a * rstd * f(gamma)
    off = (a.abs() * ea).sum(-1, keepdim=True) / (a * a).sum(-1, keepdim=True).clamp(min=1e-300)
    return a, y, ea, rstd * f(gamma).abs() * ea + (off + (h / 16 + 16) * F32) * y.abs()


@pytest.mark.parametrize("t,h", [(1, 8), (1, 2048), (3, 64), (5, 264), (37, 4096), (2, 4104), (3, 16384), (1000, 128),
                                 (513, 2056)])
@pytest.mark.parametrize("gate,sigmoid", [("none", False), ("channel", False), ("row", True), ("full", True), ("full", False),
                                          ("row", False)])
def test_gated_norm(layer, t, h, gate, sigmoid):
    g = gen(t * 31 + h)
    x, res, gamma, post = ((randn(g, *s) * m).bfloat16() for s, m in (((t, h), 3), ((t, h), 1), ((h,), 1), ((h,), 1)))
    x[0, :: max(1, h // 3)] = 200.0
    shape = {"none": None, "channel": (h,), "row": (t, 1), "full": (t, h)}[gate]
    z = None if shape is None else randn(g, *shape).bfloat16()
    for post_, res_ in ((post, res), (None, res), (post, None)):
        out = layer.moe_gated_rms_norm(x, gamma, res_, post_, z, gate_sigmoid=sigmoid, residual_scale=0.37, eps=1e-5,
                                       quantize=h % 64 == 0, want_y=True)
        a, y, ea, ey = gated_ref(x, gamma, res_, post_, z, sigmoid, 0.37, 1e-5)
        within(out.y, y, BF16 * y.abs() + 1.01 * ey + 1e-38)
        if res_ is None:
            assert out.sum is None
        else:
            within(out.sum, a, BF16 * a.abs() + 1.01 * ea)
        if h % 64 == 0:
            y, ey = y.view(t, h // 64, 64), ey.view(t, h // 64, 64).amax(-1)
            m = y.abs().amax(-1)
            within(out.scales, m / 127, (ey + 4 * F32 * m) / 127)
            # half a step of the code, the step's own error 127 times, the value's error
            within(out.codes.view(y.shape).to(F64) * out.scales.to(F64).unsqueeze(-1), y,
                   ((0.5 + 127 * 8 * F32) * m / 127 + 3 * ey).unsqueeze(-1))


def test_gated_norm_without_its_parts_is_the_plain_norm(layer):
    g = gen(5)
    x, r = randn(g, 33, 1024).bfloat16(), randn(g, 33, 1024).bfloat16()
    gamma = randn(g, 1024).bfloat16()
    a = layer.moe_add_rms_norm(x, gamma, r, quantize=True, want_y=True)
    b = layer.moe_gated_rms_norm(x, gamma, r, quantize=True, want_y=True)
    for one, other in zip(a, b):
        assert torch.equal(one, other)


def test_gated_norm_strides_and_in_place(layer):
    g = gen(6)
    wide = randn(g, 9, 1200).bfloat16()
    x, z = wide[:, 8:520], wide[:, 600:1112]  # slices of one projection: the block's output and its gate
    stream = randn(g, 9, 512).bfloat16()
    gamma = randn(g, 512).bfloat16()
    first = layer.moe_gated_rms_norm(x.contiguous(), gamma, stream.clone(), gamma, z.contiguous(), gate_sigmoid=True)
    got = layer.moe_gated_rms_norm(x, gamma, stream, gamma, z, gate_sigmoid=True, sum_out=stream)
    assert got.sum is stream and torch.equal(stream, first.sum) and torch.equal(got.y, first.y)
    rows = wide[:, 1::300][:, :1]  # one value a row, rows 1200 apart, at an odd place
    one = layer.moe_gated_rms_norm(x, gamma, stream, gate=rows)
    other = layer.moe_gated_rms_norm(x, gamma, stream, gate=rows.expand(9, 512).contiguous())
    assert torch.equal(one.sum, other.sum) and torch.equal(one.y, other.y)
    only = layer.moe_gated_rms_norm(x, gamma, stream, gate=rows, want_y=False)
    assert only.y is None and torch.equal(only.sum, one.sum)


def test_gated_norm_zero_rows_and_values_that_are_not_finite(layer):
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    r, one = torch.zeros_like(x), torch.ones(128, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = float("nan")
    r[2, 5] = float("inf")
    x[3] = 2.0
    out = layer.moe_gated_rms_norm(x, one, r, one, one, eps=1e-6, quantize=True, want_y=True)
    assert not out.sum[0].any() and not out.y[0].any() and not out.codes[0].any() and not out.scales[0].any()
    assert out.sum[1].isnan().all() and out.y[1].isnan().all() and out.scales[1].isnan().all()
    assert out.sum[2, 5].isinf() and out.y[2, 5].isnan() and not out.y[2, 6].any()
    assert (out.codes[3] == 127).all()


# ---------------------------------------------------------------- plan

def plan_ref(fresh, before, table, free, account, block, t, width):
    """The definition, step by step; None where the batch does not fit."""
    table, free, account = [list(r) for r in table], list(free), list(account)
    n_pages, top = len(free), account[-1]
    for i, n in enumerate(fresh):
        if n < 0:
            for b in range(account[i]):
                free[top] = table[i][b]
                top += 1
            account[i] = 0
    lens, starts, seq, pos, slot = [], [0], [], [], []
    for i, (n, old) in enumerate(zip(fresh, before)):
        if n >= 0 and (old > account[i] * block or old + n > width * block):
            return None
        while n >= 0 and account[i] * block < old + n:
            if top == 0:
                return None
            top -= 1
            table[i][account[i]] = free[top]
            account[i] += 1
        lens.append(0 if n < 0 else old + n)
        for p in range(old, old + n):
            seq.append(i)
            pos.append(p)
            slot.append(table[i][p // block] * block + p % block)
        starts.append(len(seq))
    if len(seq) > t:
        return None
    account[-1] = top
    blank = [-1] * (t - len(seq))
    assert len(free) == n_pages
    return dict(starts=starts, seq=seq + blank, pos=pos + blank, slot=slot + blank, lens=lens, table=table, free=free,
                account=account)


def plan_state(layer, n_seq, n_pages, width, block, seed=0):
    c = layer.KvCache.new(n_seq, n_pages, width, 1, 64, block)
    free = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).to(torch.int32).cuda()
    account = torch.zeros(n_seq + 1, dtype=torch.int32, device="cuda")
    account[-1] = n_pages
    return c, layer.KvPages(c, free, account)


def run_plan(layer, cache, pages, fresh, t, lens=None):
    """One call beside the definition; whether the batch fitted."""
    was = [v.tolist() for v in (cache.table, pages.free, pages.account, cache.lens)]
    ref = plan_ref(fresh, was[3] if lens is None else lens, *was[:3], cache.block, t, cache.table.shape[1])
    p = layer.moe_kv_plan(i32(fresh), cache, pages, t, None if lens is None else i32(lens))
    got = dict(starts=p.starts, seq=p.seq, pos=p.pos, slot=p.slot, lens=cache.lens, table=cache.table, free=pages.free,
               account=pages.account)
    assert [v.dtype for v in p] == [torch.int32] * 3 + [torch.int64]
    status = pages.read_device_status()
    if ref is None:
        assert status == -5
        ref = dict(starts=[0] * (len(fresh) + 1), seq=[-1] * t, pos=[-1] * t, slot=[-1] * t, lens=was[3], table=was[0],
                   free=was[1], account=was[2])
        fits = False
    else:
        assert status == 0
        fits = True
    for name, v in got.items():
        assert v.tolist() == ref[name], name
    return fits


# one kernel or two: up to 1024 sequences and 8192 rows, and above
@pytest.mark.parametrize("n_seq,t,block", [(1, 1, 16), (1, 300, 64), (7, 40, 16), (33, 64, 32), (1000, 1500, 16),
                                           (1025, 1100, 16), (2500, 9000, 128), (20, 10000, 64)])
def test_plan_follows_a_server(layer, n_seq, t, block):
    """Sequences begin, grow, stand still, are cut back, end and give their places to others."""
    r = random.Random(n_seq * 7 + block)
    width = 3 + 2 * t // (block * n_seq) + (t // block if n_seq < 50 else 0)
    n_pages = max(2, n_seq * width // 2)
    cache, pages = plan_state(layer, n_seq, n_pages, width, block)
    fitted = 0
    for step in range(12):
        lens = cache.lens.tolist()
        fresh, left = [0] * n_seq, t
        for s in r.sample(range(n_seq), n_seq):
            if lens[s] and r.random() < 0.15:
                fresh[s] = -r.randint(1, 5)
                continue
            n = min(left, r.choice([0, 1, 1, r.randint(0, 2 * t // n_seq + 2)]), width * block - lens[s])
            fresh[s] = n
            left -= n
        cut = None
        if step % 3 == 2:  # cut back, to any length: pages beyond it stay
            cut = [r.randint(0, n) if r.random() < 0.3 else n for n in lens]
        fitted += run_plan(layer, cache, pages, fresh, t, cut)
    assert fitted >= 6


def test_plan_refuses_a_batch_as_a_whole(layer):
    cache, pages = plan_state(layer, 4, 6, 4, 16)
    assert run_plan(layer, cache, pages, [17, 0, 16, 1], 40)  # 4 pages of 6
    assert not run_plan(layer, cache, pages, [16, 16, 16, 0], 60)  # three pages, two are free
    assert run_plan(layer, cache, pages, [-1, 16, 16, 16], 60)  # but with those of the sequence that ends
    assert not run_plan(layer, cache, pages, [1, 1, 1, 1], 3)  # more rows than t
    assert not run_plan(layer, cache, pages, [0, 49, 0, 0], 60)  # behind the table's width
    assert not run_plan(layer, cache, pages, [0, 0, 1, 0], 60, [0, 16, 33, 17])  # tokens before it without pages
    assert not run_plan(layer, cache, pages, [2**31 - 1, 2**31 - 1, 2**31 - 1, 0], 60)
    assert run_plan(layer, cache, pages, [-1, -1, -1, -1], 1)
    assert sorted(pages.free.tolist()) == list(range(6)) and int(pages.count) == 6
    assert run_plan(layer, cache, pages, [0, 0, 0, 0], 5)


@pytest.mark.parametrize("n_seq", [3, 1500])
def test_plan_reports_what_is_out_of_range(layer, n_seq):
    """Page ids, accounts and lengths that do not exist: nothing is changed, nothing is followed."""
    def broken(change, fresh):
        cache, pages = plan_state(layer, n_seq, 8, 4, 16)
        assert run_plan(layer, cache, pages, [20] + [0] * (n_seq - 1), 20)
        change(cache, pages)
        was = [v.clone() for v in (cache.lens, cache.table, pages.free, pages.account)]
        p = layer.moe_kv_plan(i32(fresh + [0] * (n_seq - len(fresh))), cache, pages, 30)
        assert pages.read_device_status() == -5
        assert not p.starts.any() and (p.seq == -1).all() and (p.slot == -1).all() and (p.pos == -1).all()
        for a, b in zip(was, (cache.lens, cache.table, pages.free, pages.account)):
            assert torch.equal(a, b)

    broken(lambda c, p: p.free.__setitem__(5, 8), [0, 1])
    broken(lambda c, p: p.free.__setitem__(5, -1), [20])
    broken(lambda c, p: c.table.__setitem__((0, 1), 99), [-1])
    broken(lambda c, p: p.account.__setitem__(0, 5), [-1])  # more blocks than the table is wide
    broken(lambda c, p: p.account.__setitem__(1, -1), [1])
    broken(lambda c, p: p.account.__setitem__(-1, 9), [1])
    broken(lambda c, p: p.account.__setitem__(-1, 7), [-1])  # more free pages than there are
    broken(lambda c, p: c.lens.__setitem__(2, -1), [1])
    broken(lambda c, p: c.lens.__setitem__(0, 33), [1])


# ---------------------------------------------------------------- linear attention

def linear_ref(q, k, v, g, starts, states, slots, slots_out, scale):
    """out, states, and the magnitudes that pass through the sums of both."""
    t, hk, d = q.shape
    hv = v.shape[1]
    f = lambda x: x.to(F64)  # noqa: E731
    q, k = (f(x).repeat_interleave(hv // hk, 1) for x in (q, k))
    v, lam = f(v), torch.exp(f(g).clamp(max=0)).expand(t, hv)
    out, mag = torch.zeros(t, hv, d, dtype=F64, device="cuda"), torch.zeros(t, hv, d, dtype=F64, device="cuda")
    new, size = f(states).clone(), f(states).abs()
    for s in range(len(starts) - 1):
        S = f(states[slots[s]]) if slots[s] >= 0 else torch.zeros(hv, d, d, dtype=F64, device="cuda")
        A = S.abs()
        for r in range(starts[s], starts[s + 1]):
            kv = k[r].unsqueeze(-1) * v[r].unsqueeze(-2)
            S = S * lam[r][:, None, None] + kv
            A = A * lam[r][:, None, None] + kv.abs()
            out[r] = scale * (q[r].unsqueeze(-1) * S).sum(-2)
            mag[r] = scale * (q[r].abs().unsqueeze(-1) * A).sum(-2)
        if slots_out[s] >= 0:
            new[slots_out[s]], size[slots_out[s]] = S, A
    return out, mag, new, size


def check_linear(layer, lens, hk, hv, d, each, seed=0, scale=None, decay=1.0, n_slots=None, pick=None, stride=False):
    g = gen(seed)
    starts = starts_of(lens)
    t, n_seq = starts[-1], len(lens)
    pad = 8 if stride else 0
    q, k, v = (randn(g, t, h, d).bfloat16() for h in (hk, hk, hv))
    if stride:  # slices of one projection
        wide = randn(g, t, 2 * hk * d + hv * d + pad).bfloat16()
        q, k = (wide[:, i * hk * d:(i + 1) * hk * d].unflatten(1, (hk, d)) for i in range(2))
        v = wide[:, 2 * hk * d:2 * hk * d + hv * d].unflatten(1, (hv, d))
    rate = decay * torch.exp(-5 * torch.rand(hv, generator=g, device="cuda"))
    logs = -rate * (2 * torch.rand(t, hv, generator=g, device="cuda") if each else torch.ones(hv, device="cuda"))
    n_slots = n_slots or n_seq
    first = randn(g, n_slots, hv, d, d) * 2
    state = layer.LinearState(first.clone())
    slots, slots_out = pick or (list(range(n_seq)), list(range(n_seq)))
    out = layer.moe_linear_attention(q, k, v, logs, i32(starts), state, *((i32(slots), i32(slots_out)) if pick else ()),
                                     scale=scale)
    assert state.read_device_status() == 0
    ref, mag, new, size = linear_ref(q, k, v, logs, starts, first, slots, slots_out, 1 / math.sqrt(d) if scale is None else scale)
    # A state is a sum of its rows' products, each with the product of the
    # decays behind it: for every row of the sequence the decay's exponential
    # (2^-22 of it), a product and a sum, and 64 for the joins.  A result is a
    # sum of d such values; where operands are taken in parts of 8 bits, two of
    # them leave 2^-17 each of a weight and of a state.
    n = max(lens)
    within(state.states, new, (6 * n + 64) * F32 * size + 1e-38)
    within(out, ref, BF16 * ref.abs() + ((6 * n + d + 64) * F32 + 2.0 ** -16) * mag * 1.01 + 1e-38)
    return state, out


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("lens,hk,hv", [
    ([1], 1, 1), ([1, 1, 1], 2, 4), ([2, 5, 0, 16], 4, 4), ([17], 3, 9), ([63], 1, 2), ([64], 2, 2), ([65], 1, 1),
    ([127, 1], 1, 4), ([128], 2, 4), ([129, 0, 64, 200], 1, 2), ([500], 1, 3), ([0, 0, 3], 2, 2), ([300, 310, 290], 4, 8)])
def test_linear_attention(layer, lens, hk, hv, d, each):
    check_linear(layer, lens, hk, hv, d, each, seed=sum(lens) + hk)


@pytest.mark.parametrize("lens", [[1, 1, 1], [70, 1, 200], [0, 5, 0]])
def test_linear_attention_slots_and_strides(layer, lens):
    check_linear(layer, lens, 2, 4, 128, True, n_slots=9, pick=([7, -1, 3], [2, 5, 8]), stride=True)
    check_linear(layer, lens, 2, 4, 64, False, n_slots=9, pick=([7, 1, -1], [7, -1, 4]), scale=1.7)


@pytest.mark.parametrize("decay", [0.0, 1e-4, 30.0, 1000.0])
@pytest.mark.parametrize("lens", [[3], [150], [400, 333]])
def test_linear_attention_slow_and_fast_decays(layer, lens, decay):
    check_linear(layer, lens, 1, 2, 128, True, decay=decay)
    check_linear(layer, lens, 1, 2, 64, False, decay=decay)


@pytest.mark.parametrize("n", [4, 200])
def test_linear_attention_decays_at_the_ends_of_their_range(layer, n):
    """-inf forgets all before it, values above zero count as zero; strong ones beside weak ones lose nothing of these."""
    g = gen(3)
    q, k, v = (randn(g, n, 2, 64).bfloat16() for _ in range(3))
    logs = torch.full((n, 2), -0.01, device="cuda")
    logs[n // 2, 0] = -math.inf
    logs[: n // 2, 1] = -20.0
    logs[n // 2 + 1:, 1] = 3.0
    first = randn(g, 1, 2, 64, 64)
    state = layer.LinearState(first.clone())
    out = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), state)
    ref, mag, new, size = linear_ref(q, k, v, logs, [0, n], first, [0], [0], 1 / 8)
    within(state.states, new, (6 * n + 64) * F32 * size + 1e-38)
    within(out, ref, BF16 * ref.abs() + ((6 * n + 128) * F32 + 2.0 ** -16) * mag * 1.01 + 1e-38)


@pytest.mark.parametrize("n,at", [(5, 2), (200, 100), (200, 199), (300, 70)])
@pytest.mark.parametrize("what", ["q", "k", "v"])
@pytest.mark.parametrize("bad", [math.inf, math.nan])
def test_linear_attention_values_that_are_not_finite(layer, n, at, what, bad):
    """A row's infinity or NaN does not reach the rows before it, other heads or sequences."""
    g = gen(9)
    x = {name: randn(g, n + 40, 2, 64).bfloat16() for name in "qkv"}
    logs = torch.full((2,), -0.02, device="cuda")
    starts = i32([0, 20, n + 20, n + 40])
    clean = layer.LinearState.new(3, 2, 64)
    ref = layer.moe_linear_attention(*x.values(), logs, starts, clean)
    x[what][20 + at, 0, 5] = bad
    state = layer.LinearState.new(3, 2, 64)
    out = layer.moe_linear_attention(*x.values(), logs, starts, state)
    for rows in (slice(0, 20 + at), slice(n + 20, n + 40)):
        assert torch.equal(out[rows], ref[rows])
    assert torch.equal(out[:, 1], ref[:, 1])
    assert torch.equal(state.states[[0, 2]], clean.states[[0, 2]]) and torch.equal(state.states[1, 1], clean.states[1, 1])
    hit = out[20 + at:20 + n, 0]
    assert not torch.isfinite(hit[0]).all()
    if what == "q":
        assert torch.equal(hit[1:], ref[20 + at + 1:20 + n, 0]) and torch.equal(state.states, clean.states)
    elif what == "v":  # one column of the state, and that channel of the rows behind
        assert not torch.isfinite(hit[:, 5]).any() and not torch.isfinite(state.states[1, 0, :, 5]).any()
        others = [i for i in range(64) if i != 5]
        assert torch.isfinite(hit[:, others]).all() and torch.isfinite(state.states[1, 0][:, others]).all()
    else:
        assert not torch.isfinite(state.states[1, 0, 5]).any()


def test_linear_attention_rows_and_slots_out_of_range(layer):
    g = gen(12)
    q, k, v = (randn(g, 90, 2, 64).bfloat16() for _ in range(3))
    logs = torch.full((2,), -0.1, device="cuda")
    first = randn(g, 4, 2, 64, 64)

    def call(starts, slots=None, slots_out=None):
        state = layer.LinearState(first.clone())
        out = torch.full_like(q, 7.0)
        layer.moe_linear_attention(q, k, v, logs, i32(starts), state, None if slots is None else i32(slots),
                                   None if slots_out is None else i32(slots_out), out=out)
        return state, out

    good, ref = call([0, 30, 90])
    assert good.read_device_status() == 0
    for starts, slots, slots_out in (([0, 30, 91], None, None), ([0, 30, 90], [0, 4], None), ([0, 30, 90], [0, -2], None),
                                     ([0, 30, 90], [0, 1], [0, 4]), ([0, 30, 20], None, None)):
        state, out = call(starts, slots, slots_out)
        assert state.read_device_status() == -5
        assert torch.equal(out[:30], ref[:30]) and (out[30:] == 7).all()
        assert torch.equal(state.states[0], good.states[0]) and torch.equal(state.states[1:], first[1:])
    # rows that no sequence owns are neither read nor written
    q[:5] = math.nan
    state, out = call([5, 30, 60])
    assert state.read_device_status() == 0 and (out[:5] == 7).all() and (out[60:] == 7).all()
    assert torch.isfinite(out).all()


@pytest.mark.parametrize("n,cuts", [(9, [0, 1, 4, 9]), (700, [0, 128, 129, 400, 401, 640, 700])])
def test_linear_attention_in_pieces(layer, n, cuts):
    """A prompt in one call, and in several: the same up to the sums' roundings."""
    g = gen(4)
    q, k, v = (randn(g, n, 4, 128).bfloat16() for _ in range(3))
    logs = -0.2 * torch.rand(n, 4, generator=g, device="cuda")
    whole, parts = layer.LinearState.new(1, 4, 128), layer.LinearState.new(1, 4, 128)
    out = layer.moe_linear_attention(q, k, v, logs, i32([0, n]), whole)
    got = torch.cat([layer.moe_linear_attention(q[a:b], k[a:b], v[a:b], logs[a:b], i32([0, b - a]), parts)
                     for a, b in zip(cuts, cuts[1:])])
    _, mag, _, size = linear_ref(q, k, v, logs, [0, n], torch.zeros(1, 4, 128, 128, device="cuda"), [0], [0], 128 ** -0.5)
    within(parts.states, whole.states.to(F64), 2 * (6 * n + 64) * F32 * size)
    within(got, out.to(F64), 2 * BF16 * out.to(F64).abs() + 2 * ((6 * n + 192) * F32 + 2.0 ** -16) * mag)


def test_linear_attention_is_the_same_every_time(layer):
    g = gen(8)
    lens = [900, 3, 411]
    starts = i32(starts_of(lens))
    q, k, v = (randn(g, sum(lens), 2, 128).bfloat16() for _ in range(3))
    logs = -0.1 * torch.rand(sum(lens), 2, generator=g, device="cuda")
    runs = []
    for _ in range(3):
        state = layer.LinearState.new(3, 2, 128)
        runs.append((layer.moe_linear_attention(q, k, v, logs, starts, state), state.states))
    for out, states in runs[1:]:
        assert torch.equal(out, runs[0][0]) and torch.equal(states, runs[0][1])


# ---------------------------------------------------------------- log probabilities

def logprobs_ref(x, ids, top):
    x = x.to(F64)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    s = e.sum(-1, keepdim=True)
    d = torch.where(e > 0, x - m, torch.zeros_like(x))
    spread = (e * d.abs()).sum(-1) / s[:, 0]  # mean distance from the largest
    ln_s = s.log()
    lp = x - m - ln_s
    best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :top]
    given = lp.gather(1, ids.long().view(len(x), -1)).view(ids.shape)
    return dict(lse=(m + ln_s)[:, 0], entropy=ln_s[:, 0] + spread, logprob=given, top_ids=best.to(torch.int32),
                top_logprobs=lp.gather(1, best), spread=spread, ln_s=ln_s[:, 0])


def check_logprobs(layer, x, ids, top):
    got, ref = layer.moe_logprobs(x, ids, top=top), logprobs_ref(x, ids, top)
    n = x.shape[1]
    # of the sum: n / 256 + 64 sums on the way of a value, its exponential (2^-22) and the
    # exponent's own roundings, which weigh as much as the value is below the largest
    es = (n / 256 + 80) * F32 + 2 * F32 * ref["spread"]
    within(got.lse, ref["lse"], es + 2 * F32 * (ref["ln_s"] + ref["lse"].abs()))
    within(got.entropy, ref["entropy"], es + 2 * F32 * ref["ln_s"] + (es + (n / 256 + 80) * F32) * (1 + ref["spread"]) + 4 * F32)
    tol = es + 2 * F32 * ref["ln_s"]

    def logs(a, lp):
        # what lies past fp32's largest value, 2^128 (1 - 2^-24), rounds to -inf: two logits of 3e38 are 6e38 apart
        fine = lp.abs() < 2.0 ** 128 * (1 - F32)
        assert torch.equal(torch.isfinite(a), fine) and (a[~fine] == -math.inf).all()
        rows = (slice(None),) + (None,) * (lp.dim() - 1)
        within(a[fine], lp[fine], (tol[rows] + 4 * F32 * (lp.abs() + ref["ln_s"][rows]))[fine])

    logs(got.logprob, ref["logprob"])
    if top:
        assert torch.equal(got.top_ids, ref["top_ids"])
        logs(got.top_logprobs, ref["top_logprobs"])
    else:
        assert got.top_ids is None and got.top_logprobs is None


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("t,n,top", [(1, 1, 1), (1, 2, 0), (3, 7, 7), (2, 33, 32), (1, 1000, 20), (5, 4096, 32), (9, 4099, 5),
                                     (1, 131072, 5), (2, 40001, 32), (20, 32003, 20), (70, 20000, 1), (200, 9001, 20),
                                     (400, 5000, 0), (1, 1 << 20, 32)])
def test_logprobs(layer, dtype, t, n, top):
    g = gen(t + n + top)
    x = (randn(g, t, n) * 3).to(dtype)
    ids = torch.randint(0, n, (t,), generator=g, device="cuda", dtype=torch.int32)
    check_logprobs(layer, x, ids, top)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "few", "steps", "large", "peak", "masked", "hole"])
@pytest.mark.parametrize("t,n", [(2, 20000), (320, 6007)])
def test_logprobs_orders_and_masks(layer, dtype, kind, t, n):
    g = gen(n)
    at = torch.arange(n, device="cuda", dtype=torch.float32)
    x = {"equal": torch.zeros(n, device="cuda"), "rising": at / 1000, "falling": -at / 1000,
         "few": (at % 3), "steps": torch.floor(at / 5000), "large": torch.where(at == 777, 3e38, -3e38),
         "peak": torch.where(at == n - 1, 50.0, at % 7), "masked": torch.where(at == n - 3, 1.0, -math.inf),
         "hole": torch.where((at > 4200) & (at < 4300), at / 100, -math.inf)}[kind]
    x = x.repeat(t, 1).to(dtype)
    ids = torch.full((t, 3), n - 3, device="cuda")
    if kind == "hole":
        ids[:] = 4250
    check_logprobs(layer, x, ids, 32)
    check_logprobs(layer, x, ids, 3)


def test_logprobs_rows_that_are_not_finite(layer):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(5, 9000, device="cuda", dtype=dtype)
        x[0] = -math.inf
        x[1, 8000] = math.nan
        x[2, 17] = math.inf
        x[3, 1] = -math.inf
        ids = torch.tensor([3, 4, 17, 1, -1], device="cuda")
        r = layer.moe_logprobs(x, ids, top=3)
        assert r.lse[0] == -math.inf and r.logprob[0].isnan() and r.entropy[0].isnan()
        assert r.top_ids[0].tolist() == [0, 1, 2] and r.top_logprobs[0].isnan().all()
        for i in (1, 2):
            assert r.logprob[i].isnan() and r.entropy[i].isnan() and r.lse[i].isnan()
            assert r.top_ids[i].tolist() == [-1] * 3 and r.top_logprobs[i].isnan().all()
        assert r.logprob[3] == -math.inf and r.top_ids[3].tolist() == [0, 2, 3]
        assert r.logprob[4].isnan() and r.top_ids[4].tolist() == [0, 1, 2] and r.entropy[4].isfinite()
        assert layer.moe_logprobs(x, torch.tensor([9000, 2**40, 1, 1, 2**31], device="cuda")).logprob.isnan().tolist() == [
            True, True, True, False, True]


def test_logprobs_strides(layer):
    g = gen(2)
    for dtype in (torch.float32, torch.bfloat16):
        wide = randn(g, 6, 30011).to(dtype)
        for lo, hi in ((0, 30011), (1, 30008), (7, 30000), (3, 12), (5, 6)):
            x = wide[:, lo:hi]
            top = min(4, hi - lo)
            ids = torch.randint(0, hi - lo, (6, 5), generator=g, device="cuda")
            a, b = layer.moe_logprobs(x, ids, top=top), layer.moe_logprobs(x.contiguous(), ids, top=top)
            check_logprobs(layer, x, ids, top)
            assert torch.equal(a.top_ids, b.top_ids)
        one = layer.moe_logprobs(wide[:1].expand(3, 30011), torch.zeros(3, dtype=torch.int64, device="cuda"))
        assert (one.lse == one.lse[0]).all()


# ---------------------------------------------------------------- together

class Hybrid:
    """Two layers, one with attention over a cache and one with linear attention, and a vocabulary."""

    def __init__(self, layer, g, h=256, hq=4, hkv=2, d=64, vocab=1003):
        self.layer, self.hq, self.hkv, self.d = layer, hq, hkv, d
        gamma = lambda: (1 + 0.1 * randn(g, h)).bfloat16()  # noqa: E731
        self.gammas = [gamma() for _ in range(5)]
        small = lambda n, k: tuple(w if w.dtype is torch.uint8 else (w * 0.15).half() for w in weights(g, n, k)[0])  # noqa: E731
        self.qkv = [small((hq + 2 * hkv) * d, h) for _ in range(2)]
        self.gate = [small(hq * d, h) for _ in range(2)]
        self.o = [small(h, hq * d) for _ in range(2)]
        self.head = small(vocab, h)
        self.decay = -torch.rand(hq, generator=g, device="cuda") * 0.2
        self.embed = randn(g, vocab, h).bfloat16()

    def step(self, tokens, plan, cache, state, slots, targets):
        L, hq, hkv, d = self.layer, self.hq, self.hkv, self.d
        x = self.embed[tokens]
        n = L.moe_add_rms_norm(x, self.gammas[0])
        for i in range(2):
            qkv = L.moe_qmv(n.y, self.qkv[i]).unflatten(1, (-1, d))
            q, k, v = qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:]
            if i == 0:
                L.moe_kv_append(k, v, plan.starts, cache)
                o = L.moe_kv_attention(q, plan.starts, cache)
            else:  # the keys' heads serve two value heads each
                o = L.moe_linear_attention(k, v, q, self.decay, plan.starts, state, slots)
            z = L.moe_qmv(n.y, self.gate[i])
            out = L.moe_qmv((o.flatten(1).float() * torch.sigmoid(z.float())).bfloat16(), self.o[i])
            n = L.moe_gated_rms_norm(out, self.gammas[2 + i], x, self.gammas[4], residual_scale=0.9)
            x = n.sum
        return L.moe_logprobs(L.moe_qmv(n.y, self.head, out_dtype=torch.float32), targets, top=4)


def test_a_step_from_lengths_to_log_probabilities(layer):
    """Prompts in one step: with the plan's tables as with tables made by hand,
    and in a place that another sequence has left.  Token by token: a captured
    graph as the calls themselves.  All bit for bit."""
    g = gen(77)
    net = Hybrid(layer, g)
    lens = [37, 20, 64]
    t = sum(lens)
    tokens = torch.randint(0, 1003, (t,), generator=g, device="cuda")
    starts, slots = starts_of(lens), i32([2, 0, 1])

    def begin():
        cache = layer.KvCache.new(3, 16, 8, net.hkv, net.d, 16)
        return cache, layer.KvPages(cache), layer.LinearState.new(3, net.hq, net.d)

    def clean(cache, pages, state):
        assert pages.read_device_status() == 0 == cache.read_device_status() == state.read_device_status()

    def same(a, b):
        for x, y in zip(a, b):
            assert torch.equal(x, y)

    cache, pages, state = begin()
    whole = net.step(tokens, layer.moe_kv_plan(i32(lens), cache, pages, t + 3), cache, state, slots, tokens)
    clean(cache, pages, state)
    by_hand, _, other = begin()
    by_hand.lens.copy_(i32(lens))
    by_hand.table.copy_(i32([[4], [0], [12]]) + i32([0, 1, 2, 3, 0, 0, 0, 0]))  # 3, 2 and 4 pages, none shared
    none = torch.zeros(1)
    same(whole, net.step(tokens, layer.KvPlan(i32(starts), none, none, none), by_hand, other, slots, tokens))
    assert torch.equal(state.states, other.states) and torch.isfinite(whole.logprob).all()

    # they end, and the same prompts come again, on other pages
    was = cache.table.clone()
    layer.moe_kv_plan(i32([-1, 30, -1]), cache, pages, 30)
    layer.moe_kv_plan(i32([0, -1, 0]), cache, pages, 1)
    plan = layer.moe_kv_plan(i32(lens), cache, pages, t)
    assert not torch.equal(cache.table, was)
    state.states.zero_()
    same(whole, net.step(tokens, plan, cache, state, slots, tokens))
    clean(cache, pages, state)

    # row by row: every sequence's next token, those that are done idle, three rows always
    def rows(run, feed, fresh):
        seen = []
        for i in range(max(lens)):
            live = [s for s in range(3) if i < lens[s]]
            fresh.copy_(torch.tensor([int(s in live) for s in range(3)], dtype=torch.int32))
            feed[:len(live)] = tokens[torch.tensor([starts[s] + i for s in live], device="cuda")]
            plan, got = run()
            assert plan.seq.tolist() == live + [-1] * (3 - len(live)) and plan.pos[:len(live)].tolist() == [i] * len(live)
            seen += [[v[:len(live)].clone() for v in got]]
        return seen

    cache, pages, state = begin()
    feed, fresh = torch.zeros(3, dtype=torch.int64, device="cuda"), i32([0, 0, 0])

    def eager():
        plan = layer.moe_kv_plan(fresh, cache, pages, 3)
        return plan, net.step(feed, plan, cache, state, slots, feed)

    ref, ref_state = rows(eager, feed, fresh), state.states
    clean(cache, pages, state)
    cache, pages, state = begin()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        fresh.zero_()
        eager()
        side.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            made = eager()

        def replay():
            graph.replay()
            return made

        got = rows(replay, feed, fresh)
        clean(cache, pages, state)
    torch.cuda.synchronize()
    for a, b in zip(ref, got):
        same(a, b)
    assert torch.equal(state.states, ref_state)


def test_calls_on_a_stream_of_their_own(layer):
    """`stream` names where the work goes and whom the results belong to."""
    g = gen(21)
    s = torch.cuda.Stream()
    x = randn(g, 64, 512).bfloat16()
    gamma = randn(g, 512).bfloat16()
    logits = randn(g, 64, 5000)
    ids = torch.randint(0, 5000, (64,), generator=g, device="cuda")
    q = randn(g, 64, 2, 64).bfloat16()
    logs = torch.full((2,), -0.1, device="cuda")
    a, b = layer.LinearState.new(1, 2, 64), layer.LinearState.new(1, 2, 64)
    cache, pages = plan_state(layer, 1, 8, 8, 16)
    starts = i32([0, 64])
    fresh = i32([64])
    ref = [layer.moe_gated_rms_norm(x, gamma, x).y, layer.moe_logprobs(logits, ids, top=3).top_logprobs,
           layer.moe_linear_attention(q, q, q, logs, starts, a)]
    torch.cuda.synchronize()
    got = [layer.moe_gated_rms_norm(x, gamma, x, stream=s).y, layer.moe_logprobs(logits, ids, top=3, stream=s).top_logprobs,
           layer.moe_linear_attention(q, q, q, logs, starts, b, stream=s)]
    p = layer.moe_kv_plan(fresh, cache, pages, 64, stream=s)
    s.synchronize()
    for u, v in zip(ref, got):
        assert torch.equal(u, v)
    assert p.starts.tolist() == [0, 64] and p.pos.tolist() == list(range(64))

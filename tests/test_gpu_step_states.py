"""States of linear attention over long prompts: how many bits they keep, and
those that a call only carries from one slot to another.

The bounds here are on a state as a whole (its norm, head by head) and on sums
of one sign, whose size is that of their magnitudes, so that a lost part of an
operand or of a decay shows.
"""

import math

import pytest

torch = pytest.importorskip("torch")

from test_gpu_layer import F64, gen, i32, layer, randn, within  # noqa: E402, F401

pytestmark = pytest.mark.gpu

F32 = 2.0 ** -24


def final_state(k, v, logs, first):
    """The state of one sequence behind its last row, in 64 bits, a head at a time, and the sum of its log decays."""
    n, hk, _ = k.shape
    hv = v.shape[1]
    state, total = first.to(F64), logs.to(F64).expand(n, hv).sum(0)
    for h in range(hv):
        g = logs.to(F64).expand(n, hv)[:, h]
        behind = torch.exp(g.sum() - torch.cumsum(g, 0))  # of the decays behind each row
        kw = k[:, h // (hv // hk)].to(F64) * behind[:, None]
        state[h] = state[h] * torch.exp(total[h]) + kw.T @ v[:, h].to(F64)
    return state, total


@pytest.mark.parametrize("each", [False, True])
@pytest.mark.parametrize("n,hk,hv,d", [(60, 1, 2, 128), (60, 2, 2, 64), (600, 1, 4, 128), (8191, 1, 2, 128), (8191, 2, 16, 64),
                                       (65536, 1, 16, 128), (65536, 1, 48, 128), (65536, 2, 64, 64)])
def test_linear_attention_states_of_slow_decays(layer, n, hk, hv, d, each):
    """Decays so slow that nothing is forgotten: a call of 65536 rows keeps as many bits as one of 60."""
    g = gen(n + hv)
    q = randn(g, n, hk, d).bfloat16()
    k, v = (randn(g, n, h, d).abs().bfloat16() for h in (hk, hv))
    rate = torch.logspace(-7, -4, hv, device="cuda")
    logs = -rate * (2 * torch.rand(n, hv, generator=g, device="cuda") if each else torch.ones(hv, device="cuda"))
    first = randn(g, hv, d, d).abs() * (n / 4)
    state = layer.LinearState(first.clone()[None])
    layer.moe_linear_attention(q, k, v, logs, i32([0, n]), state)
    assert state.read_device_status() == 0
    ref, total = final_state(k, v, logs, first)
    # All terms are positive, so that an error relative to the state at some row
    # is as large relative to the last one at most.  Of what a chunk's rows
    # add, 100: a key's factor 2^-22 (4), its product (1), 24 sums, of which
    # the first eight grow, each cut by up to 2^-23 (41), the same once more
    # for cuts inside a product, and the factors 2^-22 of joins that are not
    # slow, each of which lessens those before it by a quarter (13).
    # Roundings of the state, two a chunk and three a join of CTAs, have no
    # common sign: the norm of their sum is the root of their count times
    # 2^-24 / sqrt(3), here four times that.  A slow factor is off by 2^-22 of
    # its own (small) exponent, which adds up to that of the whole decay.
    chunks = -(-n // 128)
    bound = (100 + 4 * math.sqrt(2 * chunks + 3 * min(chunks, 152)) + 4 * total.abs()) * F32
    off = (state.states[0].to(F64) - ref).norm(dim=(1, 2)) / ref.norm(dim=(1, 2))
    assert (off <= bound).all(), f"worst {float((off / bound).max()):.3g} of the bound, off by {float(off.max()):.3g}"


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("at", [0, 37, 99])
def test_linear_attention_keeps_the_bits_of_a_key(layer, d, at):
    """One row of a chunk: its key times the decays behind it and its value, to fp32's last bits."""
    g = gen(at + d)
    n, hv = 100, 4
    q, k, v = (randn(g, n, h, d).bfloat16() for h in (1, 1, hv))
    k[:at], k[at + 1:] = 0, 0
    logs = -0.02 * torch.rand(n, hv, generator=g, device="cuda")
    state = layer.LinearState.new(1, hv, d)
    layer.moe_linear_attention(q, k, v, logs, i32([0, n]), state)
    behind = torch.exp(logs[at + 1:].to(F64).sum(0))
    ref = behind[:, None, None] * k[at, 0].to(F64)[None, :, None] * v[at].to(F64)[:, None, :]
    # the exponent, at most 3, as fp32 (3), the exponential (4), its product
    # with the key (1), the sums of its three parts, cut (6), and into the
    # state (2): 16 times 2^-24.  Without the third part it would be 2^-16.
    within(state.states[0], ref, 16 * F32 * ref.abs() + 1e-38)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("lens", [[300, 0, 0, 200, 0], [3, 0, 0, 1, 0], [0, 0, 700, 0, 0]])
def test_linear_attention_carries_states_over_bit_for_bit(layer, d, lens):
    """A sequence without rows: the state in its other slot is the one that it had, whatever its values."""
    g = gen(d + lens[0])
    n, hv = sum(lens), 3
    q, k, v = (randn(g, n, hv, d).bfloat16() for _ in range(3))
    starts = [0]
    for x in lens:
        starts.append(starts[-1] + x)
    first = randn(g, 10, hv, d, d)
    first[:, 0, 0, :4] = torch.tensor([math.inf, -math.inf, -0.0, 1e-42], device="cuda")
    first[:, 1, 5] = 3.4028e38
    first[:, 2, :, 7].view(torch.int32).fill_(0x7fa00001)  # a NaN of its own
    state = layer.LinearState(first.clone())
    slots, slots_out = [0, 1, -1, 3, 4], [5, 6, 7, 8, 9]
    layer.moe_linear_attention(q, k, v, torch.full((hv,), -0.1, device="cuda"), i32(starts), state, i32(slots), i32(slots_out))
    assert state.read_device_status() == 0
    bits = lambda x: x.view(torch.int32)  # noqa: E731
    for s, (a, b) in enumerate(zip(slots, slots_out)):
        if lens[s] == 0:
            was = first[a] if a >= 0 else torch.zeros_like(first[0])
            assert torch.equal(bits(state.states[b]), bits(was)), f"sequence {s}"
    assert torch.equal(bits(state.states[:5]), bits(first[:5]))

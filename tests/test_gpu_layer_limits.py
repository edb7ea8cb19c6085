"""The layer operators at the ends of their ranges: shapes that fill shared
memory, kernel forms that only large sizes reach, caches that are cut back,
waits that run out, very long contexts, very large scores."""

import math
import time

import pytest

torch = pytest.importorskip("torch")

from test_gpu_layer import (BF16, F64, check_attention, check_cache, feed, filled, gen, i32, layer,  # noqa: E402, F401
                            make_kv, new_cache, randn, starts_of, weights, within)

pytestmark = pytest.mark.gpu


# ---------------------------------------------------------------- qmv

def qmv_case(layer, t, n, k, q8):
    """Every weight row in fp32 against the exact product; the error bound is test_qmv's."""
    g = gen(t + 7 * n + k)
    w, ref_w, mag = weights(g, n, k)
    if q8:
        xc = torch.randint(-127, 128, (t, k), dtype=torch.int8, generator=g, device="cuda")
        xs = torch.rand(t, k // 64, generator=g, device="cuda") * 0.1
        x, rx = (xc, xs), xc.to(F64) * xs.to(F64).repeat_interleave(64, 1)
    else:
        x = randn(g, t, k).bfloat16()
        rx = x.to(F64)
    out = layer.moe_qmv(x, w, out_dtype=torch.float32)
    for i in range(0, n, 8192):
        sl = slice(i, i + 8192)
        tol = (k / 64 + 32) * 2.0 ** -23 * (rx.abs() @ mag[sl].t())
        within(out[:, sl], rx @ ref_w[sl].t(), tol)


# Sizes whose rows of x leave less than 128 bytes of a CTA's shared memory.
@pytest.mark.parametrize("t,n,k", [(4, 4000, 3968), (7, 4000, 4864), (3, 4000, 8640), (2, 4000, 10688), (16, 1000, 3776),
                                   (5, 1000, 12864)])
def test_qmv_rows_that_fill_shared_memory(layer, t, n, k):
    qmv_case(layer, t, n, k, False)


WIDE = 38912 + 89  # 256 weight rows for each of 152 SMs, and an odd rest


# 32 weight rows a warp: 8, 16, 32 and 64 rows of x a tile; k of whole units and not
@pytest.mark.parametrize("t", [5, 12, 27, 50])
@pytest.mark.parametrize("k", [512, 448])
@pytest.mark.parametrize("q8", [False, True])
def test_qmv_wide_tiles(layer, t, k, q8):
    qmv_case(layer, t, WIDE, k, q8)


# The largest k of every form of the streaming kernel (one or two teams, three
# or four stages, 8 or 16 rows), and sizes one step above, which take the next
# form or the tile kernel; 152 SMs.
@pytest.mark.parametrize("t,n,k,q8", [
    (1, 4000, 7680, False), (1, 4000, 13824, False), (1, 4000, 13888, False), (8, 4000, 2368, False),
    (8, 4000, 2432, False), (8, 4000, 4352, False), (8, 4000, 4416, False), (4, 4000, 7168, False),
    (9, 4000, 1408, False), (9, 4000, 1472, False), (9, 4000, 3136, False), (9, 4000, 3200, False),
    (12, 4000, 4864, False), (9, 4000, 7232, False), (9, 4000, 7296, False), (16, 4000, 832, False),
    (16, 4000, 1984, False), (16, 4000, 2048, False), (4, 1000, 13312, False), (4, 1000, 15360, False),
    (4, 1000, 15424, False), (8, 1000, 8704, False), (16, 1000, 4352, False), (16, 1000, 4416, False),
    (1, 4000, 7104, True), (1, 4000, 12800, True), (2, 4000, 5504, True), (8, 4000, 4224, True),
    (8, 4000, 4288, True), (10, 4000, 1216, True), (10, 4000, 2816, True), (16, 4000, 1920, True),
    (13, 4000, 4416, True), (16, 4000, 4224, True), (16, 4000, 4288, True), (4, 1000, 14656, True),
    (16, 1000, 3648, True), (16, 1000, 4224, True), (3, 1000, 16384, True), (3, 1000, 16448, True)])
def test_qmv_streaming_forms(layer, t, n, k, q8):
    qmv_case(layer, t, n, k, q8)


# ---------------------------------------------------------------- append

def test_append_cut_back_past_the_tail_is_reported(layer):
    """Two cuts in a row that each drop at most a block: the second one goes
    back into a block whose tokens the tail no longer holds."""
    block, total = 16, [33]
    kv = make_kv(gen(21), total, 2, 64)
    cache = new_cache(layer, total, block, 2, 64)
    feed(layer, cache, kv, [0], [33])
    feed(layer, cache, kv, [17], [1])  # into the block before the last: the tail holds it
    check_cache(cache, kv, [18])
    assert cache.read_device_status() == 0
    feed(layer, cache, kv, [2], [1])  # block 0: its places hold block 2's tokens
    assert cache.read_device_status() == -5
    feed(layer, cache, kv, [0], [20])  # from a block's start on nothing is read back
    check_cache(cache, kv, [20])
    feed(layer, cache, kv, [20], [1])
    assert cache.read_device_status() == 0
    feed(layer, cache, kv, [24], [1])  # tokens 21 .. 23 were never given
    assert cache.read_device_status() == -5


def test_append_tail_given_by_the_caller_is_taken(layer):
    """A cache around tensors that another one has filled: what its tail holds is not known, and taken as it is."""
    total = [45, 20]
    kv = make_kv(gen(22), total, 2, 64)
    a = new_cache(layer, total, 16, 2, 64)
    lens = feed(layer, a, kv, [0, 0], [40, 3])
    b = layer.KvCache(a.codes, a.scales, a.tail, a.table, a.lens)
    lens = feed(layer, b, kv, lens, [5, 17])
    check_cache(b, kv, lens)
    assert b.read_device_status() == 0


def test_append_reports_starts_out_of_order(layer):
    """A sequence whose rows end before they begin, between two whose rows are in range."""
    total = [200, 64, 295]
    kv = make_kv(gen(23), [300], 1, 64)[0]
    cache = new_cache(layer, total, 64, 1, 64)
    cache.lens.copy_(i32(total))
    layer.moe_kv_append(kv[:, 0], kv[:, 1], i32([0, 200, 5, 300]), cache)
    assert cache.read_device_status() == -5


# ---------------------------------------------------------------- attention

def test_attention_wait_runs_out_and_workspace_recovers(layer):
    """The first CTA brings no codes, and gives up its part of items that all
    CTAs share; the others count theirs.  The next calls, of either kernel,
    find the counts as if nothing had been."""
    from routed_expert_prefill_gb300 import moe

    g = gen(25)
    new, lens = [40], [200000]  # some eight units of 128 tokens a CTA
    cache = filled(layer, g, new, lens, 1, 64, 64)
    q = randn(g, 40, 4, 64).bfloat16()
    ref = check_attention(layer, cache, q, new, lens)
    for _ in range(2):
        out = torch.full_like(q, 7.0)
        moe.debug_stall(cache.ws, moe.MOE_STALL_WEIGHT_COPIES)
        torch.cuda.synchronize()
        t0 = time.monotonic()
        layer.moe_kv_attention(q, starts_of(new), cache, out=out)
        assert cache.read_device_status() == -6
        assert time.monotonic() - t0 < 20  # waits of 2 s, side by side
        assert (out == 7).all()  # the item was not joined
    assert torch.equal(layer.moe_kv_attention(q, starts_of(new), cache), ref)
    one = check_attention(layer, cache, q[39:], [1], lens)
    assert torch.equal(layer.moe_kv_attention(q, starts_of(new), cache), ref)
    assert torch.equal(layer.moe_kv_attention(q[39:], starts_of([1]), cache), one)
    assert cache.read_device_status() == 0


@pytest.mark.parametrize("n_seq,new,bits", [(500, 1, 39), (200, 40, 32)])
def test_attention_small_weights_of_a_long_context(layer, n_seq, new, bits):
    """One token with nearly all of the weight and no value, before 2^18 with
    2^-26.25 of its weight each: what they add up to is the result.  A weight
    may be off by 2^-11 and by 2^-bits of the row's largest.  All sequences
    share their pages; there are enough for most to stay within one CTA."""
    ln, d, block = 2 ** 18, 64, 64
    pages = ln // block
    cache = layer.KvCache.new(n_seq, pages, pages, 1, d, block)
    cache.table[:] = torch.randperm(pages, generator=torch.Generator().manual_seed(0)).to(torch.int32).cuda()
    place = torch.arange(ln, device="cuda")
    v = (32 + (place[:, None] * 7 + torch.arange(d, device="cuda")) % 64).to(torch.int8)
    v[0] = 0
    cache.codes[1, cache.table[0].long(), 0] = v.view(pages, block, d)
    cache.codes[0, int(cache.table[0, 0]), 0, 0, 0] = 64  # the first token's key: 1 in channel 0
    cache.scales.fill_(1 / 64)
    cache.lens.fill_(ln)
    q = torch.zeros(n_seq * new, 1, d, dtype=torch.bfloat16, device="cuda")
    q[:, 0, 0] = 1
    got = layer.moe_kv_attention(q, starts_of([new] * n_seq), cache, scale=26.25 * math.log(2))
    w = 2.0 ** -26.25
    sums = v.to(F64).cumsum(0)[ln - new:] / 64  # of what each row sees
    seen = torch.arange(ln - new, ln, device="cuda", dtype=F64)[:, None]  # tokens beside the first
    ref = (w * sums / (1 + w * seen)).repeat(n_seq, 1)[:, None]
    tol = (2.0 ** -11 + 2.0 ** -14) * ref + ln * 2.0 ** -bits * 95 / 64
    within(got, ref, tol + BF16 * (ref + tol))

def one_hot_case(layer, new, exponent, q_exponent, scale):
    """Scores so large that each row's best token has all of the weight, with
    value scales that differ: the result is that token's value."""
    g = gen(24 + new)
    ln, hq, d, block = 300, 4, 64, 16
    cache = filled(layer, g, [new], [ln], 2, d, block)
    pages = cache.table[0, :-(-ln // block)].long()
    cache.scales[1, pages] *= 10 ** (2 * torch.rand(len(pages), 2, generator=g, device="cuda") - 1)
    q = (randn(g, new, hq, d) * 2.0 ** q_exponent).bfloat16()
    got = layer.moe_kv_attention(q, i32([0, new]), cache, scale=scale)
    checked = 0
    for h in range(hq):
        k, v = ((cache.codes[i, pages, h // 2].to(F64) * cache.scales[i, pages, h // 2].to(F64)[:, None, None])
                .reshape(-1, d)[:ln] for i in range(2))
        z = q[:, h].to(F64) @ k.t() * scale
        size = (q[:, h].to(F64).abs() @ k.abs().t() * scale).amax(-1)
        see = torch.arange(ln, device="cuda")[None, :] <= torch.arange(ln - new, ln, device="cuda")[:, None]
        two = z.masked_fill(~see, -math.inf).topk(2, -1)
        gap = two.values[:, 0] - two.values[:, 1]
        # scores are off by less than 2^-18 of `size`; beside a token 200 ahead nothing counts
        clear = gap > 200 + 2.0 ** -16 * size
        assert float(size.max()) > 2.0 ** exponent
        checked += int(clear.sum())
        ref = v[two.indices[:, 0]][clear]
        # one weight rounded to fp16, the value scale's logarithm and power
        tol = (2.0 ** -11 + 2.0 ** -16) * ref.abs()
        within(got[clear, h], ref, tol + BF16 * (ref.abs() + tol))
    assert checked >= max(2, new)  # of 4 * new rows


@pytest.mark.parametrize("exponent", [12, 17, 21, 25, 28, 40])
def test_attention_large_scores_of_many_rows(layer, exponent):
    one_hot_case(layer, 40, exponent, 0, 2.0 ** (exponent - 3))


def test_attention_large_queries_of_many_rows(layer):
    one_hot_case(layer, 40, 110, 116, 2.0 ** -3)


@pytest.mark.parametrize("exponent", [12, 17, 21, 25, 28, 40])
def test_attention_large_scores_of_single_tokens(layer, exponent):
    one_hot_case(layer, 1, exponent, 0, 2.0 ** (exponent - 3))


@pytest.mark.parametrize("exponent", [12, 21, 28])
def test_attention_large_scores_joined_across_the_gpu(layer, exponent):
    """The same from the parts of many CTAs, in two levels: each row's best
    token is one of three far apart, the other parts are far below it."""
    g = gen(26)
    ln, d, block = 70001, 64, 64
    cache = filled(layer, g, [1], [ln], 1, d, block)
    pages = cache.table[0, :-(-ln // block)].long()
    cache.scales[1, pages] *= 10 ** (2 * torch.rand(len(pages), 1, generator=g, device="cuda") - 1)
    for at in (77, 35000, ln - 1):
        page, place = int(cache.table[0, at // block]), at % block
        kept = cache.codes[0, page, 0, place].clone()
        cache.codes[0, page, 0, place] = 127
        q = torch.ones(1, 2, d, dtype=torch.bfloat16, device="cuda")
        got = layer.moe_kv_attention(q, i32([0, 1]), cache, scale=2.0 ** (exponent - 6))
        ref = cache.codes[1, page, 0, place].to(F64) * cache.scales[1, page, 0].to(F64)
        tol = (2.0 ** -11 + 2.0 ** -16) * ref.abs()
        within(got[0], ref.expand(2, d), tol + BF16 * (ref.abs() + tol))
        cache.codes[0, page, 0, place] = kept


@pytest.mark.parametrize("new", [1, 40])
@pytest.mark.parametrize("q_exponent,scale", [(116, 2.0 ** -3), (122, 2.0 ** -6)])
def test_attention_largest_queries(layer, new, q_exponent, scale):
    one_hot_case(layer, new, 110, q_exponent, scale)

"""The layer operators against plain 64-bit implementations.

Tolerances are derived, not fitted.  A bf16 result may be off by its rounding,
2^-8 of the exact value; what comes before it is fp32, and each test states
the bound of its own sums.
"""

import math

import pytest

torch = pytest.importorskip("torch")

pytestmark = pytest.mark.gpu

BF16 = 2.0 ** -8  # largest relative error of one rounding to bf16
F64 = torch.float64


@pytest.fixture(scope="module")
def layer():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    from routed_expert_prefill_gb300 import build

    build.build()
    from routed_expert_prefill_gb300 import layer as m

    return m


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def randn(g, *shape):
    return torch.randn(shape, generator=g, device="cuda")


def within(got, ref, tol):
    d = (got.to(F64) - ref).abs()
    bad = ~(d <= tol)
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} off, worst {float((d - tol).max()):.3g} over"


# ---------------------------------------------------------------- norm

def norm_ref(x, gamma, residual, eps):
    a = x.to(F64) + (0 if residual is None else residual.to(F64))
    return a, a / ((a * a).mean(-1, keepdim=True) + eps).sqrt() * gamma.to(F64)


@pytest.mark.parametrize("t,h", [(1, 8), (1, 2048), (3, 64), (5, 264), (37, 4096), (2, 4104), (7, 8192), (3, 16384),
                                 (1000, 128), (513, 2056), (4, 1536)])
@pytest.mark.parametrize("res", [False, True])
def test_norm(layer, t, h, res):
    g = gen(t * 31 + h)
    x = (randn(g, t, h) * 3).bfloat16()
    x[0, :: max(1, h // 3)] = 200.0
    r = randn(g, t, h).bfloat16() if res else None
    gamma = randn(g, h).bfloat16()
    out = layer.moe_add_rms_norm(x, gamma, r, eps=1e-5, quantize=h % 64 == 0, want_y=True)
    a, y = norm_ref(x, gamma, r, 1e-5)
    # the sum of squares has no cancellation: at most h / 8 + 16 roundings of
    # 2^-24 each, halved by the root; four more roundings follow
    f32 = (h / 16 + 16) * 2.0 ** -24
    within(out.y, y, (BF16 + 2 * f32) * y.abs() + 1e-38)
    if res:
        within(out.sum, a, BF16 * a.abs())
    else:
        assert out.sum is None
    if h % 64 == 0:
        y = y.view(t, h // 64, 64)
        m = y.abs().amax(-1)
        within(out.scales, m / 127, 2 * f32 * m / 127)
        # half a step, and the fp32 error of 127 steps
        within(out.codes.view(t, h // 64, 64).to(F64) * out.scales.to(F64).unsqueeze(-1), y,
               ((0.5 + 127 * 4 * f32) * m / 127).unsqueeze(-1))
        assert int(out.codes.abs().amax()) == 127


def test_norm_strides_broadcast_and_in_place(layer):
    g = gen(3)
    wide = randn(g, 9, 600).bfloat16()
    x, one = wide[:, 8:520], randn(g, 1, 512).bfloat16()
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    res = one.expand(9, 512)  # one row for all: stride 0
    a, y = norm_ref(x, gamma, res, 1e-6)
    stream = x.contiguous()
    out = layer.moe_add_rms_norm(x, gamma, res)
    within(out.y, y, 1.01 * BF16 * y.abs())
    again = layer.moe_add_rms_norm(stream, gamma, res, sum_out=stream)  # the stream's own rows
    assert again.sum is stream
    assert torch.equal(stream, out.sum) and torch.equal(again.y, out.y)


def test_norm_zero_rows_and_values_that_are_not_finite(layer):
    x = torch.zeros(4, 128, dtype=torch.bfloat16, device="cuda")
    x[1, 3] = float("inf")
    x[2, 70] = float("nan")
    x[3] = 1.0
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    out = layer.moe_add_rms_norm(x, gamma, eps=0.25, quantize=True, want_y=True)
    assert torch.equal(out.y[0].float(), torch.zeros(128, device="cuda"))
    assert torch.equal(out.codes[0], torch.zeros(128, dtype=torch.int8, device="cuda")) and not out.scales[0].any()
    assert out.y[1, 3].isnan() and not out.y[1, 4].any()  # inf * (1 / inf), 0 * (1 / inf)
    assert out.scales[1, 0].isnan() and out.scales[1, 1] == 0 and not out.codes[1].any()
    assert out.y[2].isnan().all() and out.scales[2].isnan().all()
    assert (out.codes[3] == 127).all()


# ---------------------------------------------------------------- qmv

def weights(g, n, k):
    codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g, device="cuda")
    scales = (randn(g, n, k // 64) * 0.02).half()
    biases = (randn(g, n, k // 64) * 0.1).half()
    q = torch.stack([codes & 15, codes >> 4], -1).view(n, k // 64, 64).to(F64)
    w = q * scales.to(F64)[..., None] + biases.to(F64)[..., None]
    # magnitude that passes through the fp32 sums: |16 s (1 + q / 16)| + |b - 16 s|
    mag = (q + 32) * scales.to(F64).abs()[..., None] + biases.to(F64).abs()[..., None]
    return (codes, scales, biases), w.view(n, k), mag.view(n, k)


QMV_SHAPES = [(1, 1, 64), (1, 2560, 2048), (2, 17, 128), (3, 100, 320), (5, 333, 704), (8, 1000, 4096),
              (9, 48, 1024), (16, 640, 192), (23, 129, 2048), (32, 64, 64), (40, 31, 448), (64, 512, 1024),
              (65, 200, 256), (200, 96, 512), (1, 20011, 256), (2, 50, 65536)]


@pytest.mark.parametrize("t,n,k", QMV_SHAPES)
@pytest.mark.parametrize("f32", [False, True])
@pytest.mark.parametrize("q8", [False, True])
def test_qmv(layer, t, n, k, f32, q8):
    g = gen(t + 7 * n + k)
    w, ref_w, mag = weights(g, n, k)
    if q8:
        xc = torch.randint(-127, 128, (t, k), dtype=torch.int8, generator=g, device="cuda")
        xs = torch.rand(t, k // 64, generator=g, device="cuda") * 0.1
        x, rx = (xc, xs), xc.to(F64) * xs.to(F64).repeat_interleave(64, 1)
    else:
        x = randn(g, t, k).bfloat16()
        rx = x.to(F64)
    out = layer.moe_qmv(x, w, out_dtype=torch.float32 if f32 else torch.bfloat16)
    ref = rx @ ref_w.t()
    # exact products; k / 64 groups are added in fp32 after 4 steps each of
    # the tensor core, whose sums may be cut instead of rounded (2^-22)
    tol = (k / 64 + 32) * 2.0 ** -23 * (rx.abs() @ mag.t())
    within(out, ref, tol if f32 else tol + BF16 * (ref.abs() + tol))


def test_qmv_strided_rows_out_and_special_values(layer):
    g = gen(5)
    w, ref_w, _ = weights(g, 70, 256)
    wide = randn(g, 6, 3 * 256).bfloat16()
    x = wide[:, 256:512]
    out = torch.empty(6, 70, dtype=torch.float32, device="cuda")
    assert layer.moe_qmv(x, w, out=out) is out
    assert torch.equal(out, layer.moe_qmv(x.contiguous(), w, out_dtype=torch.float32))
    same = layer.moe_qmv(x[2:3].expand(6, 256), w, out_dtype=torch.float32)
    assert torch.equal(same, out[2:3].expand(6, 70))
    bad = x.contiguous()
    bad[1, 7] = float("nan")
    bad[3, 200] = float("inf")
    got = layer.moe_qmv(bad, w, out_dtype=torch.float32)
    assert got[1].isnan().all() and not got[3].isfinite().any()
    for r in (0, 2, 4, 5):
        assert torch.equal(got[r], out[r])  # rows do not mix


def test_norm_feeds_qmv_in_8_bits(layer):
    g = gen(6)
    x = randn(g, 11, 1024).bfloat16()
    gamma = (1 + 0.1 * randn(g, 1024)).bfloat16()
    w, ref_w, _ = weights(g, 256, 1024)
    o = layer.moe_add_rms_norm(x, gamma, quantize=True)
    got = layer.moe_qmv((o.codes, o.scales), w, out_dtype=torch.float32)
    _, y = norm_ref(x, gamma, None, 1e-6)
    # every activation is within half a step (and fp32) of the norm's value
    step = (y.view(11, 16, 64).abs().amax(-1) / 127).repeat_interleave(64, 1)
    within(got, y @ ref_w.t(), 0.51 * step @ ref_w.abs().t() + 1e-3)


# ---------------------------------------------------------------- cache

def new_cache(layer, total, block, hkv, d, spare=3, seed=0, slots=None):
    """A cache with scattered pages for sequences of `total` tokens; unused
    pages and tails hold garbage and NaN."""
    blocks = [-(-n // block) for n in total]
    n_pages, n_seq = sum(blocks) + spare, len(total)
    perm = torch.randperm(n_pages, generator=torch.Generator().manual_seed(seed)).tolist()
    table = torch.full((n_seq, max(max(blocks), 1) + 1), n_pages + 12345, dtype=torch.int32)
    at = 0
    for s, b in enumerate(blocks):
        table[s, :b] = torch.tensor(perm[at:at + b], dtype=torch.int32)
        at += b
    codes = torch.randint(-128, 128, (2, n_pages, hkv, block, d), dtype=torch.int8, device="cuda")
    scales = torch.full((2, n_pages, hkv), float("nan"), device="cuda")
    tail = torch.full((n_seq, 2, hkv, 2 * block, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    return layer.KvCache(codes, scales, tail, table.cuda(), torch.zeros(n_seq, dtype=torch.int32, device="cuda"))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device="cuda")


def starts_of(new):
    a = [0]
    for n in new:
        a.append(a[-1] + n)
    return i32(a)


def feed(layer, cache, kv, lens, new):
    """Append the next new[s] tokens of kv[s] ([tokens, 2, hkv, d]) to every sequence; returns the new lengths."""
    rows = torch.cat([kv[s][lens[s]:lens[s] + n] for s, n in enumerate(new)])
    lens = [a + n for a, n in zip(lens, new)]
    cache.lens.copy_(i32(lens))
    layer.moe_kv_append(rows[:, 0], rows[:, 1], starts_of(new), cache)
    return lens


def quantised(v):
    """v [tokens, hkv, d] of one block in 64 bits: codes and the fp32 step of each head."""
    v = v.to(F64)
    m = v.abs().amax((0, 2))
    q = torch.where(m[None, :, None] > 0, (v * 127 / m[None, :, None]).round(), torch.zeros_like(v))
    return q, (m / 127).float()


def check_cache(cache, kv, lens):
    for s, n in enumerate(lens):
        for b in range(-(-n // cache.block)):
            page = int(cache.table[s, b])
            part = kv[s][b * cache.block:min(n, (b + 1) * cache.block)]
            for i in range(2):
                q, step = quantised(part[:, i])
                got = cache.codes[i, page].transpose(0, 1)
                assert torch.equal(got[:len(part)].to(F64), q), (s, b, i)
                assert not got[len(part):].any()
                assert torch.equal(cache.scales[i, page], step)


def make_kv(g, total, hkv, d):
    out = []
    for n in total:
        kv = randn(g, n, 2, hkv, d) * (0.2 + torch.rand(2, hkv, d, generator=g, device="cuda"))
        out.append(kv.bfloat16())
    return out


@pytest.mark.parametrize("block", [16, 32, 64, 128])
@pytest.mark.parametrize("hkv,d", [(1, 64), (3, 128)])
def test_append_in_pieces(layer, block, hkv, d):
    """One token, odd pieces, runs over many blocks and idle sequences: after
    every call each touched block is its tokens' quantisation, bit for bit."""
    total = [1, 2 * block + 1, 5 * block + 7, block]
    g = gen(block + hkv)
    kv = make_kv(g, total, hkv, d)
    cache = new_cache(layer, total, block, hkv, d)
    lens = [0] * 4
    for new in ([1, 1, block, 0], [0, block - 1, 1, 0], [0, 0, 3 * block, block], [0, block, block - 2, 0],
                [0, 1, 8, 0]):
        lens = feed(layer, cache, kv, lens, new)
        check_cache(cache, kv, lens)
    assert lens == total and cache.read_device_status() == 0


def test_append_one_by_one_is_append_at_once(layer):
    total = [37, 70]
    kv = make_kv(gen(1), total, 2, 64)
    a, b = (new_cache(layer, total, 16, 2, 64) for _ in range(2))
    feed(layer, a, kv, [0, 0], total)
    lens = [0, 0]
    for i in range(70):
        lens = feed(layer, b, kv, lens, [1 if i < 37 else 0, 1])
    check_cache(b, kv, total)
    for s, n in enumerate(total):
        pages = a.table[s, :-(-n // 16)].long()
        assert torch.equal(a.codes[:, pages], b.codes[:, pages])
        assert torch.equal(a.scales[:, pages], b.scales[:, pages])


def test_append_after_cutting_back(layer):
    """Draft tokens written over a block's end, dropped and replaced."""
    block, total = 32, [70]
    kv, other = make_kv(gen(2), total, 2, 64), make_kv(gen(3), total, 2, 64)
    for cut, draft in ((31, 2), (30, 6), (62, 5), (64, 1), (40, 32)):
        cache = new_cache(layer, total, block, 2, 64)
        lens = feed(layer, cache, kv, [0], [cut])
        mixed = [torch.cat([kv[0][:cut], other[0][cut:]])]
        feed(layer, cache, mixed, lens, [min(draft, 70 - cut)])
        lens = feed(layer, cache, kv, [cut], [3])  # back at `cut`
        check_cache(cache, kv, lens)


def test_append_strided_values_zero_and_not_finite(layer):
    hkv, d, block = 2, 64, 16
    qkv = randn(gen(4), 20, (4 + 2 * hkv) * d).bfloat16()
    k = qkv[:, 4 * d:(4 + hkv) * d].unflatten(1, (hkv, d))
    v = qkv[:, (4 + hkv) * d:].unflatten(1, (hkv, d))
    k[:16, 1] = 0  # a block of zeros
    v[3, 0, 5], v[17, 1, 0], k[18, 0, 2] = float("nan"), float("inf"), -float("inf")
    cache = new_cache(layer, [20], block, hkv, d)
    cache.lens.fill_(20)
    layer.moe_kv_append(k, v, i32([0, 20]), cache)
    kv = torch.stack([k, v], 1).clone()
    kv[~kv.isfinite()] = 0
    check_cache(cache, [kv], [20])
    assert cache.read_device_status() == -5
    assert cache.read_device_status() == 0
    assert cache.tail.view(2, hkv, 2 * block, d)[:, :, :20].isfinite().all()


def test_append_skips_what_is_out_of_range(layer):
    total = [20, 20, 20]
    kv = make_kv(gen(5), total, 1, 64)
    cache = new_cache(layer, total, 16, 1, 64)
    rows, starts = torch.cat(kv), starts_of(total)
    cache.lens.copy_(i32([20, 500, 20]))  # more than the table has room for
    cache.table[2, 1] = -1
    before = cache.codes.clone()
    layer.moe_kv_append(rows[:, 0], rows[:, 1], starts, cache)
    assert cache.read_device_status() == -5
    check_cache(cache, kv, [20])  # the first sequence is whole
    touched = (cache.codes != before).flatten(2).any(-1).any(0).nonzero().flatten().tolist()
    assert set(touched) <= {*cache.table[0, :2].tolist(), int(cache.table[2, 0])}
    # lengths below the new tokens' count, and starts past the rows
    for lens, starts in (([20, 5, 20], starts), ([20, 20, 20], i32([0, 20, 40, 61])),
                         ([20, 20, 20], i32([0, 20, 10, 60])), ([20, 20, 20], i32([-4, 20, 40, 60]))):
        cache.lens.copy_(i32(lens))
        cache.table[2, 1] = cache.table[0, 0]
        layer.moe_kv_append(rows[:, 0], rows[:, 1], starts, cache)
        assert cache.read_device_status() == -5


# ---------------------------------------------------------------- attention

def attention_ref(cache, q, new, lens, scale):
    """Exact output, and per element the bound of its error before the last rounding."""
    t, hq, d = q.shape
    group = hq // cache.hkv
    out = torch.zeros(q.shape, dtype=F64, device="cuda")
    tol = torch.zeros_like(out)
    row = 0
    for s, (n, ln) in enumerate(zip(new, lens)):
        if n == 0:
            continue
        pages = cache.table[s, :-(-ln // cache.block)].long()
        for h in range(cache.hkv):
            k, v = ((cache.codes[i, pages, h].to(F64) * cache.scales[i, pages, h].to(F64)[:, None, None])
                    .reshape(-1, d)[:ln] for i in range(2))
            x = q[row:row + n, h * group:(h + 1) * group].to(F64)  # [n, group, d]
            z = torch.einsum("ngd,ld->ngl", x, k) * scale
            size = torch.einsum("ngd,ld->ngl", x.abs(), k.abs()) * abs(scale)
            see = torch.arange(ln, device="cuda")[None, :] <= torch.arange(ln - n, ln, device="cuda")[:, None]
            p = torch.softmax(z.masked_fill(~see[:, None], -math.inf), -1)
            size = size.masked_fill(~see[:, None], 0)
            sl = slice(h * group, (h + 1) * group)
            out[row:row + n, sl] = torch.einsum("ngl,ld->ngd", p, v)
            mean = torch.einsum("ngl,ld->ngd", p, v.abs())
            # weights: fp16 (2^-11) and fp32 steps; a score is d / 16 + 8 fp32
            # sums, possibly cut (2^-22), of terms of that size; weights below
            # fp16's range lose 2^-25 of the largest each
            rel = 2.0 ** -11 + 2.0 ** -12 + (d / 16 + 8) * 2.0 ** -22 * size.amax(-1, keepdim=True)
            tol[row:row + n, sl] = 2 * rel * mean + ln * 2.0 ** -24 * v.abs().amax()
        row += n
    return out, tol


def check_attention(layer, cache, q, new, lens, scale=None, **kw):
    got = layer.moe_kv_attention(q, starts_of(new), cache, scale=scale, **kw)
    ref, tol = attention_ref(cache, q, new, lens, 1 / math.sqrt(cache.d) if scale is None else scale)
    within(got, ref, tol + BF16 * (ref.abs() + tol))
    return got


ATTENTION = [
    # new tokens, lengths after them, hq, hkv, d, block
    ([1], [1], 1, 1, 64, 16),
    ([1], [1], 8, 1, 128, 64),
    ([1], [16], 8, 2, 128, 16),
    ([1], [127], 16, 2, 128, 64),
    ([1], [129], 32, 8, 64, 32),
    ([1, 1, 1], [5, 1000, 64], 16, 2, 128, 64),
    ([1, 0, 2, 0], [33, 70, 2, 9], 10, 2, 64, 16),
    ([3, 5], [3, 205], 12, 4, 128, 32),
    ([17], [17], 4, 4, 64, 128),
    ([1, 7], [4097, 2050], 16, 1, 128, 128),
    ([40, 1, 130], [40, 300, 700], 8, 2, 128, 64),
    ([300], [333], 5, 1, 128, 64),
    ([1] * 70, [1 + 13 * i for i in range(70)], 4, 2, 64, 16),
    ([1] * 300, [1 + i % 37 for i in range(300)], 2, 1, 64, 16),
    ([257], [257], 8, 8, 64, 32),
    ([129, 200], [1129, 200], 24, 1, 128, 64),
]


def filled(layer, g, new, lens, hkv, d, block):
    cache = new_cache(layer, lens, block, hkv, d)
    kv = make_kv(g, lens, hkv, d)
    before = [a - b for a, b in zip(lens, new)]
    at = [0] * len(lens)
    while at != before:  # at most 30000 rows of a sequence per call
        at = feed(layer, cache, kv, at, [min(30000, b - a) for a, b in zip(at, before)])
    if any(new):
        feed(layer, cache, kv, at, new)
    return cache


@pytest.mark.parametrize("case", ATTENTION, ids=lambda c: f"{len(c[0])}seq-{max(c[0])}new-{max(c[1])}len-{c[2]}q{c[3]}kv"
                         f"-d{c[4]}-b{c[5]}")
def test_attention(layer, case):
    new, lens, hq, hkv, d, block = case
    g = gen(sum(lens) + hq)
    cache = filled(layer, g, new, lens, hkv, d, block)
    q = (randn(g, sum(new), hq, d) * 1.5).bfloat16()
    got = check_attention(layer, cache, q, new, lens)
    assert cache.read_device_status() == 0
    assert torch.equal(got, layer.moe_kv_attention(q, starts_of(new), cache))  # the same bits again


def test_attention_long_context_split_over_the_gpu(layer):
    g = gen(9)
    cache = filled(layer, g, [1], [70001], 2, 128, 64)
    q = (randn(g, 1, 8, 128) * 2).bfloat16()
    check_attention(layer, cache, q, [1], [70001])
    # the workspace's counters are as before: other work splits right after it
    q = randn(g, 1, 16, 128).bfloat16()
    check_attention(layer, cache, q, [1], [70001], scale=0.3)


@pytest.mark.parametrize("new,lens", [([1], [200]), ([50], [200])])
def test_attention_reads_nothing_past_the_length(layer, new, lens):
    """Blocks past the length have no pages (garbage table entries); places
    past it in the last block, and unused pages, hold garbage and NaN."""
    g = gen(10)
    cache = filled(layer, g, new, lens, 2, 128, 64)
    q = randn(g, sum(new), 6, 128).bfloat16()
    ref = check_attention(layer, cache, q, new, lens)
    page = int(cache.table[0, 3])
    cache.codes[:, page, :, 200 - 192:] = 99
    assert torch.equal(ref, layer.moe_kv_attention(q, starts_of(new), cache))


@pytest.mark.parametrize("new", [1, 40])
def test_attention_uneven_scales(layer, new):
    """Blocks whose keys or values are all zero, and value scales ten orders
    apart, so that the largest weight and the largest product differ."""
    g = gen(11)
    lens = [300]
    cache = filled(layer, g, [new], lens, 2, 64, 16)
    pages = cache.table[0, :19].long()
    cache.scales[1, pages[3]] = 0
    cache.scales[0, pages[4]] = 0
    cache.scales[1, pages[5]] *= 1e6
    cache.scales[1, pages[7:12]] *= 1e-4
    q = randn(g, new, 4, 64).bfloat16() * 3
    check_attention(layer, cache, q, [new], lens)
    cache.scales[1] = 0
    assert not layer.moe_kv_attention(q, starts_of([new]), cache).any()


@pytest.mark.parametrize("new", [1, 33])
def test_attention_scale_and_query_range(layer, new):
    """Query rows whose magnitudes are far apart, zero rows, scale 0 and
    negative, peaked and flat softmax; a NaN query spoils its own row only."""
    g = gen(12)
    lens = [150]
    cache = filled(layer, g, [new], lens, 1, 128, 32)
    q = randn(g, new, 4, 128)
    q[0, 0] *= 1e-20
    q[0, 1] *= 50
    q[0, 2] = 0
    q = q.bfloat16()
    for scale in (None, 0.0, -0.05, 0.5):
        check_attention(layer, cache, q, [new], lens, scale=scale)
    huge = q.float()
    huge[0, 3] *= 1e20
    check_attention(layer, cache, huge.bfloat16(), [new], lens, scale=1e-20)
    q[0, 3, 7] = float("nan")
    got = layer.moe_kv_attention(q, starts_of([new]), cache)
    assert got[0, 3].isnan().all() and got.isnan().sum() == 128


@pytest.mark.parametrize("new", [2, 48])
def test_attention_strided_queries_and_other_stream(layer, new):
    g = gen(13)
    lens = [90]
    cache = filled(layer, g, [new], lens, 2, 64, 16)
    wide = randn(g, new, 8 * 64).bfloat16()
    q = wide[:, 64:64 + 256].unflatten(1, (4, 64))
    ref = check_attention(layer, cache, q, [new], lens)
    side = torch.cuda.Stream()
    starts = starts_of([new])
    side.wait_stream(torch.cuda.current_stream())
    got = layer.moe_kv_attention(q, starts, cache, stream=side)
    side.synchronize()
    assert torch.equal(got, ref)


def test_attention_flags_what_is_out_of_range(layer):
    g = gen(14)
    new, lens = [1, 2, 1], [100, 90, 80]
    cache = filled(layer, g, new, lens, 1, 64, 16)
    q = randn(g, 4, 2, 64).bfloat16()
    ref = check_attention(layer, cache, q, new, lens)
    out = torch.full_like(q, 7.0)
    cache.lens[1] = 1  # fewer tokens than it has new ones
    layer.moe_kv_attention(q, starts_of(new), cache, out=out)
    assert cache.read_device_status() == -5
    assert torch.equal(out[0], ref[0]) and torch.equal(out[3], ref[3]) and (out[1:3] == 7).all()
    cache.lens[1] = 90
    cache.table[2, :] = -3  # no page is left to the third sequence
    layer.moe_kv_attention(q, starts_of(new), cache, out=out)
    assert cache.read_device_status() == -5
    assert torch.equal(out[:3], ref[:3]) and not out[3].any()


@pytest.mark.parametrize("new", [1, 24])
def test_cache_offsets_past_32_bits(layer, new):
    """Pages whose bytes lie more than 4 GB into the cache."""
    hkv, d, block = 2, 128, 64
    n_pages = 2 ** 32 // (hkv * d * block) + 1000
    cache = layer.KvCache.new(1, n_pages, 4, hkv, d, block)
    cache.table[0] = i32([n_pages - 1, 3, n_pages - 7, n_pages - 2])
    g = gen(15)
    kv = make_kv(g, [200], hkv, d)
    lens = feed(layer, cache, kv, [0], [200 - new])
    lens = feed(layer, cache, kv, lens, [new])
    check_cache(cache, kv, lens)
    q = randn(g, new, 4, d).bfloat16()
    check_attention(layer, cache, q, [new], lens)


# ---------------------------------------------------------------- together

def test_decoder_layer_example():
    """The example's layer: a prompt in one chunk, in two, and token by token agree."""
    import importlib.util
    import os

    path = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples", "decoder_layer.py")
    spec = importlib.util.spec_from_file_location("decoder_layer", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    assert mod.main(["--tokens", "70", "--hidden", "256", "--experts", "8"]) == 0


def test_calls_capture_in_a_graph(layer):
    """The four calls of a decode step replay from a CUDA graph with new inputs in place."""
    g = gen(16)
    h, hq, hkv, d = 256, 4, 2, 64
    total = [40]
    cache = new_cache(layer, [60], 16, hkv, d)
    kv = make_kv(g, total, hkv, d)
    feed(layer, cache, kv, [0], total)
    w, _, _ = weights(g, (hq + 2 * hkv) * d, h)
    x, gamma = randn(g, 1, h).bfloat16(), torch.ones(h, dtype=torch.bfloat16, device="cuda")
    starts = i32([0, 1])

    def step():
        y = layer.moe_add_rms_norm(x, gamma, quantize=True)
        qkv = layer.moe_qmv((y.codes, y.scales), w).unflatten(1, (hq + 2 * hkv, d))
        layer.moe_kv_append(qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], starts, cache)
        return layer.moe_kv_attention(qkv[:, :hq], starts, cache)

    cache.lens.fill_(41)
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    x.copy_(randn(g, 1, h).bfloat16())
    cache.lens.fill_(41)
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, step())

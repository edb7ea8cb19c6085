"""Cases of the layer operators around the routed mixture-of-experts block.

Four operators of a decoder layer: the RMS norm with the residual's addition
(``norm``), the product with 4-bit weights (``qmv``), the append to a paged
8-bit key/value cache (``append``) and the attention over it (``attention``).
``run`` computes them in plain torch operations in 32 bits, or, where ``own``
is true, through ``routed_expert_prefill_gb300.layer``.
"""

import math
import random

import torch

own = False

GROUP = 64  # weights per scale, and activations per scale of an 8-bit row
EPS = 1e-6


def listed():
    return [
        # one decoded token enters a layer: the call's own time is what counts
        dict(name="norm t1 h2048", op="norm", t=1, h=2048, q8=False),
        # a verify batch of an odd row count, quantised for the 4-bit product that follows
        dict(name="norm t37 h4096 q8", op="norm", t=37, h=4096, q8=True),
        # a full prompt chunk: the stream's sum and the norm's rows, bounded by memory
        dict(name="norm t4096 h4096", op="norm", t=4096, h=4096, q8=False),
        # the query/key/value projection of one decoded token
        dict(name="qmv t1 k2048 n2560", op="qmv", t=1, k=2048, n=2560, q8=False, f32=False),
        # a verify batch whose rows the norm has left in 8 bits
        dict(name="qmv t5 k4096 n6144 q8", op="qmv", t=5, k=4096, n=6144, q8=True, f32=False),
        # the vocabulary's logits of a small decode batch, in 32 bits
        dict(name="qmv t4 k4096 n131072", op="qmv", t=4, k=4096, n=131072, q8=False, f32=True),
        # a decode batch writes one token a sequence, most of them into a block that is partly filled
        dict(name="append s32 one", op="append", seqs=32, new=1, ragged=False, ctx=1021, hkv=4, d=128, block=64),
        # a prompt chunk of three uneven sequences
        dict(name="append s3 chunk", op="append", seqs=3, new=2311, ragged=True, ctx=300, hkv=8, d=128, block=64),
        # one decoded token at a short odd context: the call's own time
        dict(name="attention s1 c1013", op="attention", seqs=1, new=1, ragged=False, ctx=1013, hq=16, hkv=2, d=128,
             block=64),
        # a decode batch of ragged contexts: bounded by the cache's bytes
        dict(name="attention s48 c20000", op="attention", seqs=48, new=1, ragged=True, ctx=20000, hq=32, hkv=4, d=128,
             block=64),
        # verify batches of up to five rows, narrow heads and small blocks
        dict(name="attention s16 verify", op="attention", seqs=16, new=5, ragged=True, ctx=4099, hq=16, hkv=4, d=64,
             block=32),
        # a prompt chunk behind a context: bounded by the matrix products
        dict(name="attention s2 prefill", op="attention", seqs=2, new=2600, ragged=True, ctx=3001, hq=32, hkv=8, d=128,
             block=64),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {"bytes": max(work(c)["bytes"] for c in listed()), "flops": max(work(c)["flops"] for c in listed())}
    while True:
        op = rng.choice(["norm", "qmv", "append", "attention", "attention"])
        if op == "norm":
            q8 = rng.random() < 0.5
            step = 64 if q8 else 8
            c = dict(op=op, t=_spread(rng, 1, 4096), h=step * _spread(rng, 1024 // step, 8192 // step), q8=q8)
        elif op == "qmv":
            c = dict(op=op, t=_spread(rng, 1, 64), k=128 * _spread(rng, 4, 64), n=_spread(rng, 500, 131072),
                     q8=rng.random() < 0.5, f32=rng.random() < 0.5)
        else:
            hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128])
            block = rng.choice([16, 32, 64])
            kind = rng.choice(["one", "verify", "chunk"])
            seqs = _spread(rng, 1, 64) if kind != "chunk" else rng.randint(1, 4)
            new = 1 if kind == "one" else rng.randint(2, 16) if kind == "verify" else _spread(rng, 17, 4096)
            c = dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, ctx=_spread(rng, 1, 32768), hkv=hkv, d=d,
                     block=block)
            if op == "append":
                c["ctx"] = min(c["ctx"], 2048)
            else:
                c["hq"] = hkv * rng.choice([1, 2, 4, 5, 8])
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _plain_bytes(c) <= 12e9:
            return c


def _plain_bytes(c):
    """Bytes of the plain form's largest table, so that drawn cases fit beside one another."""
    if c["op"] != "attention":
        return 0
    return 4 * c["seqs"] * c["hq"] * c["new"] * (c["ctx"] + c["new"])


def _lengths(c):
    """New tokens and total length of each sequence: the first as the case says, the others below it where it is ragged."""
    r = random.Random("%d %d %d" % (c["seqs"], c["new"], c["ctx"]))
    new, total = [], []
    for s in range(c["seqs"]):
        n = c["new"] if s == 0 or not c["ragged"] else r.randint(max(1, c["new"] // 2), c["new"])
        before = c["ctx"] if s == 0 else r.randint(c["ctx"] // 8, c["ctx"]) if c["ragged"] else max(0, c["ctx"] - 5 * s)
        new.append(n)
        total.append(before + n)
    return new, total


def work(c):
    if c["op"] == "norm":
        t, h = c["t"], c["h"]
        out = t * h + 4 * t * h // GROUP if c["q8"] else 2 * t * h
        return {"bytes": 6 * t * h + 2 * h + out, "flops": 6 * t * h}
    if c["op"] == "qmv":
        t, k, n = c["t"], c["k"], c["n"]
        rows = t * k + 4 * t * k // GROUP if c["q8"] else 2 * t * k
        return {"bytes": n * k // 2 + 4 * n * k // GROUP + rows + (4 if c["f32"] else 2) * t * n, "flops": 2 * t * n * k}
    new, total = _lengths(c)
    hkv, d, block = c["hkv"], c["d"], c["block"]
    if c["op"] == "append":
        moved = 0
        for n, tot in zip(new, total):
            old = tot - n
            first, last = old // block, (tot - 1) // block
            read = n + old - first * block  # the new tokens, and what the first block held
            kept = tot - max(old, max(0, last - 1) * block)  # new tokens of the last two blocks
            moved += 2 * hkv * (d * (2 * read + (last - first + 1) * block + 2 * kept) + 4 * (last - first + 1))
        return {"bytes": moved, "flops": 4 * sum(new) * 2 * hkv * d}
    hq = c["hq"]
    blocks = sum(-(-tot // block) for tot in total)
    seen = sum(n * (tot - n) + n * (n + 1) // 2 for n, tot in zip(new, total))
    return {"bytes": 2 * hkv * (sum(total) * d + 4 * blocks) + 4 * sum(new) * hq * d, "flops": 4 * hq * d * seen}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _rows(g, t, h):
    """Rows of a residual stream: a few channels far larger than the others."""
    x = torch.randn(t, h, generator=g, device="cuda")
    big = 1 + 15 * (torch.rand(h, generator=g, device="cuda") < 0.01).float()
    return (x * big * 0.7).to(torch.bfloat16)


def _to_8_bits(v):
    """v [..., n] to whole numbers in [-127, 127] of one step for all n, and the step."""
    most = v.abs().amax(-1, keepdim=True)
    q = torch.where(most > 0, torch.round(v * 127 / most), torch.zeros_like(v))
    return q, (most / torch.full_like(most, 127))[..., 0]


def _keys(g, shape):
    """Keys or values: channels of uneven size, as projections give them."""
    size = 0.3 + 1.4 * torch.rand(shape[-2:], generator=g, device="cuda")
    return (torch.randn(shape, generator=g, device="cuda") * size).to(torch.bfloat16)


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    if c["op"] == "norm":
        s = {"op": "norm", "x": _rows(g, c["t"], c["h"]), "residual": _rows(g, c["t"], c["h"]), "q8": c["q8"]}
        s["gamma"] = (1 + 0.2 * torch.randn(c["h"], generator=g, device="cuda")).to(torch.bfloat16)
        if c["q8"]:
            s["values"] = torch.empty(c["t"], c["h"] // GROUP, GROUP, dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "qmv":
        t, k, n = c["t"], c["k"], c["n"]
        s = {"op": "qmv", "f32": c["f32"], "q8": c["q8"]}
        codes = torch.randint(0, 256, (n, k // 2), dtype=torch.uint8, generator=g, device="cuda")
        scales = (0.004 + 0.004 * torch.rand(n, k // GROUP, generator=g, device="cuda")).to(torch.float16)
        biases = (scales.float() * (-7.5 + torch.randn(n, k // GROUP, generator=g, device="cuda"))).to(torch.float16)
        s["weights"] = (codes, scales, biases)
        x = _rows(g, t, k)
        if c["q8"]:
            q, step = _to_8_bits(x.float().view(t, k // GROUP, GROUP))
            s["x"] = (q.view(t, k).to(torch.int8), step)
        else:
            s["x"] = x
        return s
    new, total = _lengths(c)
    hkv, d, block, seqs = c["hkv"], c["d"], c["block"], c["seqs"]
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    most = max(-(-tot // block) for tot in total)
    # for the append only the blocks that it touches have pages of their own; the others share page 0
    first = [(tot - n) // block if c["op"] == "append" else 0 for n, tot in zip(new, total)]
    table = torch.zeros(seqs, most, dtype=torch.int32)
    pages = 1
    for i, tot in enumerate(total):
        count = -(-tot // block) - first[i]
        table[i, first[i]:first[i] + count] = torch.arange(pages, pages + count, dtype=torch.int32)
        pages += count
    order = torch.randperm(pages - 1, generator=torch.Generator().manual_seed(seed)).to(torch.int32) + 1
    table = torch.cat([torch.zeros(1, dtype=torch.int32), order])[table.long()].to("cuda")
    s = {"op": c["op"], "starts": whole(starts), "lens": whole(total), "table": table, "most_new": max(new),
         "block": block, "hkv": hkv, "d": d, "seqs": seqs}
    if c["op"] == "append":
        s["codes"] = torch.zeros(2, pages, hkv, block, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.zeros(2, pages, hkv, device="cuda")
        s["tail"] = _keys(g, (seqs, 2, 2 * block, hkv, d)).transpose(2, 3).contiguous()
        s["k"], s["v"] = _keys(g, (2, starts[-1], hkv, d)).unbind(0)
    else:
        s["codes"] = torch.empty(2, pages, hkv, block, d, dtype=torch.int8, device="cuda")
        s["scales"] = torch.empty(2, pages, hkv, device="cuda")
        for i in range(2):
            v = _keys(g, (pages, block, hkv, d)).transpose(1, 2).float()
            q, step = _to_8_bits(v.reshape(pages, hkv, block * d))
            s["codes"][i] = q.view(pages, hkv, block, d).to(torch.int8)
            s["scales"][i] = step
        s["tail"] = torch.zeros(seqs, 2, hkv, 2 * block, d, dtype=torch.bfloat16, device="cuda")
        s["q"] = (1.5 * torch.randn(starts[-1], c["hq"], d, generator=g, device="cuda")).to(torch.bfloat16)
    if own:  # the handle that a program keeps: it holds the tensors above
        from routed_expert_prefill_gb300 import layer

        s["cache"] = layer.KvCache(s["codes"], s["scales"], s["tail"], s["table"], s["lens"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        from routed_expert_prefill_gb300 import layer

        if s["op"] == "norm":
            r = layer.moe_add_rms_norm(s["x"], s["gamma"], s["residual"], eps=EPS, quantize=s["q8"])
            if not s["q8"]:
                return {"sum": r.sum, "y": r.y}
            torch.mul(r.codes.view(s["values"].shape), r.scales.unsqueeze(-1), out=s["values"])
            return {"sum": r.sum, "values": s["values"], "scales": r.scales}
        if s["op"] == "qmv":
            return layer.moe_qmv(s["x"], s["weights"], out_dtype=torch.float32 if s["f32"] else torch.bfloat16)
        if s["op"] == "append":
            layer.moe_kv_append(s["k"], s["v"], s["starts"], s["cache"])
            return {"values": s["codes"] * s["scales"][..., None, None], "tail": s["tail"]}
        return layer.moe_kv_attention(s["q"], s["starts"], s["cache"])
    return {"norm": _norm, "qmv": _qmv, "append": _append, "attention": _attention}[s["op"]](s)


def _norm(s):
    a = s["x"].float() + s["residual"].float()
    y = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    if not s["q8"]:
        return {"sum": a.to(torch.bfloat16), "y": y.to(torch.bfloat16)}
    q, step = _to_8_bits(y.view(s["values"].shape))
    return {"sum": a.to(torch.bfloat16), "values": (q * step[..., None]).to(torch.bfloat16), "scales": step}


def _qmv(s):
    codes, scales, biases = s["weights"]
    n, groups = scales.shape
    q = torch.stack([codes & 15, codes >> 4], -1).view(n, groups, GROUP)
    w = (q.float() * scales.float()[..., None] + biases.float()[..., None]).view(n, -1)
    x = (s["x"][0].view(-1, groups, GROUP) * s["x"][1][..., None]).view(-1, groups * GROUP) if s["q8"] else s["x"].float()
    y = x @ w.t()
    return y if s["f32"] else y.to(torch.bfloat16)


def _append(s):
    block, dev = s["block"], s["k"].device
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["table"].long()
    old = lens - (starts[1:] - starts[:-1])
    first = old // block
    count = -(-(s["most_new"] - 1) // block) + 1  # blocks that the longest run of new tokens may touch
    at = first[:, None] + torch.arange(count, device=dev)  # [sequence, block]
    pos = at[..., None] * block + torch.arange(block, device=dev)
    seq = torch.arange(s["seqs"], device=dev)[:, None, None]
    fresh = torch.stack([s["k"], s["v"]], 1)  # [token, 2, head, channel]
    new = fresh[(starts[:-1, None, None] + pos - old[:, None, None]).clamp(0, fresh.shape[0] - 1)]
    held = s["tail"].permute(0, 3, 1, 2, 4)[seq, pos % (2 * block)]
    some = pos[..., None, None, None]
    v = torch.where(some < old[:, None, None, None, None, None], held, new).float()
    v = torch.where(some < lens[:, None, None, None, None, None], v, torch.zeros_like(v))
    v = v.permute(3, 0, 1, 4, 2, 5)  # [2, sequence, block, head, place, channel]
    q, step = _to_8_bits(v.reshape(*v.shape[:4], -1))
    live = (at * block < lens[:, None]).nonzero(as_tuple=True)
    page = table[live[0], at[live]]
    s["codes"][:, page] = q.view(v.shape)[:, live[0], live[1]].to(torch.int8)
    s["scales"][:, page] = step[:, live[0], live[1]]
    token = torch.arange(fresh.shape[0], device=dev)
    owner = torch.searchsorted(starts[1:].contiguous(), token, right=True)
    place = old[owner] + token - starts[owner]
    kept = (place >= ((lens[owner] - 1) // block - 1) * block).nonzero(as_tuple=True)[0]
    s["tail"].permute(0, 3, 1, 2, 4)[owner[kept], place[kept] % (2 * block)] = fresh[kept]
    return {"values": s["codes"] * s["scales"][..., None, None], "tail": s["tail"]}


def _attention(s):
    q, dev = s["q"], s["q"].device
    t, hq, d = q.shape
    seqs, hkv, block, group = s["seqs"], s["hkv"], s["block"], hq // s["hkv"]
    starts, lens, table = s["starts"].long(), s["lens"].long(), s["table"].long()
    n = starts[1:] - starts[:-1]
    k, v = ((s["codes"][i][table].float() * s["scales"][i][table][..., None, None]).transpose(1, 2).reshape(
        seqs, hkv, -1, d) for i in range(2))  # [sequence, head, position, channel]
    row = torch.arange(s["most_new"], device=dev)
    at = (starts[:-1, None] + row).clamp(max=t - 1)
    x = q[at].float().view(seqs, -1, hkv, group, d).permute(0, 2, 3, 1, 4).reshape(seqs, hkv, -1, d)
    scores = (x @ k.transpose(2, 3)).view(seqs, hkv, group, s["most_new"], -1) / math.sqrt(d)
    last = (lens - n)[:, None] + row  # the last position that each row sees
    hidden = torch.arange(k.shape[2], device=dev) > last[..., None]
    scores.masked_fill_(hidden[:, None, None], -math.inf)
    p = torch.exp(scores.sub_(scores.amax(-1, keepdim=True)))
    total = p.sum(-1)
    o = (p.view(seqs, hkv, -1, p.shape[-1]) @ v).view(seqs, hkv, group, -1, d) / total[..., None]
    o = o.permute(0, 3, 1, 2, 4).reshape(seqs, -1, hq, d)
    return o[(row < n[:, None])].to(torch.bfloat16)


# ---------------------------------------------------------------------------
# The definitions in 64 bits
# ---------------------------------------------------------------------------

def exact(case, seed):
    global own
    was, own = own, False
    try:
        s = prepare(case, seed)
    finally:
        own = was
    f = torch.float64

    def steps(v):  # whole numbers of one step over the last axis, and the step
        top = v.abs().max(-1, keepdim=True).values
        q = (v * 127 / top.clamp(min=1e-300)).round()
        return q, top.squeeze(-1) / 127

    if case["op"] == "norm":
        a = s["x"].to(f) + s["residual"].to(f)
        y = a / ((a * a).sum(-1, keepdim=True) / case["h"] + EPS).sqrt() * s["gamma"].to(f)
        if not case["q8"]:
            return {"sum": a, "y": y}
        q, step = steps(y.reshape(case["t"], -1, GROUP))
        return {"sum": a, "values": q * step.unsqueeze(-1), "scales": step}
    if case["op"] == "qmv":
        codes, scales, biases = s["weights"]
        out = []
        x = s["x"]
        if case["q8"]:
            x = x[0].to(f) * x[1].to(f).repeat_interleave(GROUP, 1)
        x = x.to(f)
        for i in range(0, case["n"], 16384):  # rows of the weights, in pieces
            c = codes[i:i + 16384]
            w = torch.empty(c.shape[0], case["k"], dtype=f, device="cuda")
            w[:, 0::2] = (c % 16).to(f)
            w[:, 1::2] = (c // 16).to(f)
            w *= scales[i:i + 16384].to(f).repeat_interleave(GROUP, 1)
            w += biases[i:i + 16384].to(f).repeat_interleave(GROUP, 1)
            out.append(torch.einsum("tk,nk->tn", x, w))
        return torch.cat(out, 1)
    new, total = _lengths(case)
    block, hkv, d = case["block"], case["hkv"], case["d"]
    begin = 0
    if case["op"] == "append":
        values, tail = torch.zeros(s["codes"].shape, dtype=f, device="cuda"), s["tail"].to(f)
        kv = torch.stack([s["k"], s["v"]]).to(f)
        for i, (n, tot) in enumerate(zip(new, total)):
            seen = torch.zeros(2, hkv, tot, d, dtype=f, device="cuda")
            begin_block = (tot - n) // block * block
            for p in range(begin_block, tot - n):
                seen[:, :, p] = tail[i, :, :, p % (2 * block)]
            seen[:, :, tot - n:] = kv[:, begin:begin + n].transpose(1, 2)
            for b in range(begin_block, tot, block):
                part = seen[:, :, b:b + block]
                q, step = steps(part.reshape(2, hkv, -1))
                page = int(s["table"][i, b // block])
                values[:, page, :, :part.shape[2]] = q.view(part.shape) * step[..., None, None]
            for p in range(max(tot - n, ((tot - 1) // block - 1) * block), tot):
                tail[i, :, :, p % (2 * block)] = seen[:, :, p]
            begin += n
        return {"values": values, "tail": tail}
    out = torch.empty(s["q"].shape, dtype=f, device="cuda")
    for i, (n, tot) in enumerate(zip(new, total)):
        pages = s["table"][i, :-(-tot // block)].long()
        see = torch.arange(tot, device="cuda")[None, :] <= torch.arange(tot - n, tot, device="cuda")[:, None]
        for h in range(hkv):
            k, v = ((s["codes"][j, pages, h].to(f) * s["scales"][j, pages, h].to(f)[:, None, None]).reshape(-1, d)[:tot]
                    for j in range(2))
            for head in range(h * case["hq"] // hkv, (h + 1) * case["hq"] // hkv):
                z = s["q"][begin:begin + n, head].to(f) @ k.t() / d ** 0.5
                p = torch.softmax(z.masked_fill(~see, -math.inf), -1)
                out[begin:begin + n, head] = p @ v
        begin += n
    return out

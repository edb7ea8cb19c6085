"""Cases of the operators that take a decoder from request lengths to log probabilities.

Four operators beside those of ``perf/operators.py``: the norms before and
after a block with its gate and residual scale (``norms``), the page tables and
row maps of a batch (``plan``), linear attention with a decay for each head
(``linear``) and the log probabilities of given tokens with entropy and top
alternatives (``logprobs``).  ``run`` computes them in plain torch operations
in 32 bits, or, where ``own`` is true, through
``routed_expert_prefill_gb300.layer``.
"""

import math
import random

import torch

own = False

GROUP = 64  # channels per scale of an 8-bit row
EPS = 1e-6
CHUNK = 64  # rows that the plain form of linear attention takes at a time


def listed():
    return [
        # one decoded token between two blocks: the call's own time is what counts
        dict(name="norms t1 h2048", op="norms", t=1, h=2048, gate="channel", sigmoid=False, q8=False),
        # a verify batch of an odd row count, gated per channel and row, quantised for the 4-bit product that follows
        dict(name="norms t37 h4096 q8", op="norms", t=37, h=4096, gate="full", sigmoid=True, q8=True),
        # a full prompt chunk: bounded by memory
        dict(name="norms t4096 h4096", op="norms", t=4096, h=4096, gate="channel", sigmoid=False, q8=False),
        # a decode batch: one token a sequence, a page now and then, a few sequences that end
        dict(name="plan s48 one", op="plan", seqs=48, new=1, ctx=20000, block=64, ends=3),
        # prompts of uneven length enter many slots at once
        dict(name="plan s700 prompts", op="plan", seqs=700, new=160, ctx=900, block=16, ends=41),
        # the sampled token of one sequence, with five alternatives
        dict(name="logprobs t1 n131072", op="logprobs", t=1, n=131072, bf16=False, top=5),
        # a verify batch over an odd vocabulary in 16 bits, where many logits are equal
        dict(name="logprobs t33 n32003", op="logprobs", t=33, n=32003, bf16=True, top=20),
        # a prompt is scored: bounded by the logits' bytes
        dict(name="logprobs t2048 n131072", op="logprobs", t=2048, n=131072, bf16=False, top=20),
        # a decode batch: every state is read and written once
        dict(name="linear s64 one", op="linear", seqs=64, new=1, ragged=False, hk=16, hv=32, d=128, each=False),
        # verify batches of a few rows, narrow heads, a decay for each row
        dict(name="linear s16 verify", op="linear", seqs=16, new=5, ragged=True, hk=8, hv=16, d=64, each=True),
        # one prompt of few heads: the length itself has to be split
        dict(name="linear s1 prompt", op="linear", seqs=1, new=8191, ragged=False, hk=16, hv=16, d=128, each=False),
        # uneven prompts of many heads, a decay for each row: bounded by memory
        dict(name="linear s6 prompts", op="linear", seqs=6, new=2900, ragged=True, hk=16, hv=32, d=128, each=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, spread over its logarithm."""
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    most = {"bytes": max(work(c)["bytes"] for c in listed()), "flops": max(work(c)["flops"] for c in listed())}
    while True:
        op = rng.choice(["norms", "plan", "logprobs", "linear", "linear"])
        if op == "norms":
            q8 = rng.random() < 0.5
            step = 64 if q8 else 8
            c = dict(op=op, t=_spread(rng, 1, 4096), h=step * _spread(rng, 512 // step, 8192 // step),
                     gate=rng.choice(["none", "channel", "row", "full"]), sigmoid=rng.random() < 0.5, q8=q8)
        elif op == "plan":
            seqs = _spread(rng, 1, 2048)
            c = dict(op=op, seqs=seqs, new=rng.choice([1, rng.randint(2, 16), _spread(rng, 17, 4096)]),
                     ctx=_spread(rng, 1, min(32768, 8_000_000 // seqs)), block=rng.choice([16, 32, 64, 128]),
                     ends=rng.randint(0, seqs // 4))
        elif op == "logprobs":
            c = dict(op=op, t=_spread(rng, 1, 4096), n=_spread(rng, 500, 262144), bf16=rng.random() < 0.5,
                     top=rng.choice([0, 1, rng.randint(2, 32), 32]))
        else:
            kind = rng.choice(["one", "verify", "prompt", "prompt"])
            hk = rng.choice([1, 2, 4, 8, 16])
            seqs = _spread(rng, 1, 128) if kind != "prompt" else _spread(rng, 1, 12)
            new = 1 if kind == "one" else rng.randint(2, 16) if kind == "verify" else _spread(rng, 17, 8192)
            c = dict(op=op, seqs=seqs, new=new, ragged=rng.random() < 0.5, hk=hk, hv=hk * rng.choice([1, 2, 4]),
                     d=rng.choice([64, 128]), each=rng.random() < 0.5)
        w = work(c)
        if w["bytes"] <= most["bytes"] and w["flops"] <= most["flops"] and _plain_bytes(c) <= 10e9 and _rows(c) <= 65536:
            return c


def _rows(c):
    return sum(n for n in _plan(c)[1] if n > 0) if c["op"] == "plan" else c["t"] if "t" in c else sum(_lengths(c))


def _plain_bytes(c):
    """Bytes of the plain form's largest tables, so that drawn cases fit beside one another."""
    if c["op"] == "linear":
        chunks = -(-c["new"] // CHUNK)
        return 4 * c["seqs"] * c["hv"] * chunks * (3 * c["d"] ** 2 + 3 * CHUNK ** 2 + 6 * CHUNK * c["d"])
    if c["op"] == "logprobs":
        return 24 * c["t"] * c["n"]
    return 0


def _lengths(c):
    """New rows of each sequence: the first as the case says, the others below it where it is ragged."""
    r = random.Random("%d %d" % (c["seqs"], c["new"]))
    return [c["new"] if s == 0 or not c["ragged"] else r.randint(max(1, c["new"] // 2), c["new"]) for s in range(c["seqs"])]


def _plan(c):
    """Tokens of each sequence before the call, and its new ones (-1: it ends)."""
    r = random.Random("%d %d %d" % (c["seqs"], c["new"], c["ctx"]))
    before = [r.randint(0, c["ctx"]) for _ in range(c["seqs"])]
    new = [c["new"] if c["new"] < 17 else r.randint(0, c["new"]) for _ in range(c["seqs"])]
    for s in r.sample(range(c["seqs"]), c["ends"]):
        new[s] = -1
    return before, new


def work(c):
    if c["op"] == "norms":
        t, h = c["t"], c["h"]
        out = t * h + 4 * t * h // GROUP if c["q8"] else 2 * t * h
        gate = {"none": 0, "channel": 2 * h, "row": 2 * t, "full": 2 * t * h}[c["gate"]]
        return {"bytes": 6 * t * h + 4 * h + gate + out, "flops": 12 * t * h}
    if c["op"] == "plan":
        before, new = _plan(c)
        b = c["block"]
        rows = sum(n for n in new if n > 0)
        taken = sum(-(-(o + n) // b) - -(-o // b) for o, n in zip(before, new) if n > 0)
        given = sum(-(-o // b) for o, n in zip(before, new) if n < 0)
        seen = sum(-(-o // b) * b > o for o, n in zip(before, new) if n > 0)  # pages held before that rows go into
        # new, lengths and held blocks in, lengths, held blocks and starts out, three maps, pages
        return {"bytes": 24 * c["seqs"] + 16 * rows + 8 * taken + 8 * given + 4 * seen, "flops": 4 * rows}
    if c["op"] == "logprobs":
        t, n = c["t"], c["n"]
        return {"bytes": t * n * (2 if c["bf16"] else 4) + t * (8 + 12 + 8 * c["top"]), "flops": 5 * t * n}
    rows, hk, hv, d = sum(_lengths(c)), c["hk"], c["hv"], c["d"]
    moved = 2 * rows * d * 2 * (hk + hv) + (4 * rows * hv if c["each"] else 4 * hv) + 8 * c["seqs"] * hv * d * d
    return {"bytes": moved, "flops": 4 * rows * hv * d * d}


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _stream_rows(g, t, h):
    """Rows of a residual stream: a few channels far larger than the others."""
    x = torch.randn(t, h, generator=g, device="cuda")
    big = 1 + 15 * (torch.rand(h, generator=g, device="cuda") < 0.01).float()
    return (x * big * 0.7).to(torch.bfloat16)


def _to_8_bits(v):
    """v [..., n] to whole numbers in [-127, 127] of one step for all n, and the step."""
    most = v.abs().amax(-1, keepdim=True)
    q = torch.where(most > 0, torch.round(v * 127 / most), torch.zeros_like(v))
    return q, (most / torch.full_like(most, 127))[..., 0]


def prepare(case, seed):
    c = case
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    rand = lambda *shape: torch.randn(shape, generator=g, device="cuda")  # noqa: E731
    whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    s = {"op": c["op"]}
    if c["op"] == "norms":
        t, h = c["t"], c["h"]
        s |= {"x": _stream_rows(g, t, h), "residual": _stream_rows(g, t, h), "q8": c["q8"], "sigmoid": c["sigmoid"],
              "post": (1 + 0.2 * rand(h)).to(torch.bfloat16), "gamma": (1 + 0.2 * rand(h)).to(torch.bfloat16),
              "scale": 0.25 + 0.05 * (seed % 16)}
        shape = {"none": None, "channel": (h,), "row": (t, 1), "full": (t, h)}[c["gate"]]
        s["gate"] = None if shape is None else (0.6 * rand(*shape)).to(torch.bfloat16)
        if c["q8"]:
            s["values"] = torch.empty(t, h // GROUP, GROUP, dtype=torch.bfloat16, device="cuda")
        return s
    if c["op"] == "plan":
        before, new = _plan(c)
        block, seqs = c["block"], c["seqs"]
        r = random.Random(seed)
        r.shuffle(both := list(zip(before, new)))  # which sequence holds what
        before, new = [list(v) for v in zip(*both)]
        held = [-(-b // block) for b in before]
        width = max(1, max(-(-(b + max(n, 0)) // block) for b, n in zip(before, new)))
        taken = sum(max(0, -(-(b + n) // block) - h) for b, n, h in zip(before, new, held) if n > 0)
        pages = sum(held) + taken + 7
        order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)
        table = torch.zeros(seqs, width, dtype=torch.int32, device="cuda")
        at = torch.arange(width, device="cuda")
        mine = at < whole(held)[:, None]
        table[mine] = order[:sum(held)]
        s |= {"new": whole(new), "before": whole(before), "t": max(1, sum(n for n in new if n > 0)), "block": block,
              "lens": whole(before), "table": table, "free": torch.cat([order[sum(held):], order[:sum(held)]]),
              # what the pool's account holds before a pass: the blocks of each sequence, then the free pages
              "account": whole(held + [pages - sum(held)])}
        if own:  # the handles that a program keeps: they hold the tensors above
            from routed_expert_prefill_gb300 import layer

            codes = torch.zeros(2, pages, 1, block, 64, dtype=torch.int8, device="cuda")
            scales = torch.zeros(2, pages, 1, device="cuda")
            tail = torch.zeros(seqs, 2, 1, 2 * block, 64, dtype=torch.bfloat16, device="cuda")
            s["cache"] = layer.KvCache(codes, scales, tail, s["table"], s["lens"])
            s["pages"] = layer.KvPages(s["cache"], s["free"], s["account"].clone())
        return s
    if c["op"] == "logprobs":
        t, n = c["t"], c["n"]
        x = rand(t, n).mul_(2.5).add_(rand(n))
        s |= {"logits": x.to(torch.bfloat16) if c["bf16"] else x, "top": c["top"],
              "ids": torch.randint(0, n, (t,), generator=g, device="cuda")}
        return s
    new, hk, hv, d = _lengths(c), c["hk"], c["hv"], c["d"]
    starts = [0]
    for n in new:
        starts.append(starts[-1] + n)
    t, seqs = starts[-1], c["seqs"]
    rate = torch.exp(-torch.linspace(0.7, 6.5, hv, device="cuda")[torch.randperm(hv, generator=g, device="cuda")])
    s |= {"q": (1.5 * rand(t, hk, d)).to(torch.bfloat16), "k": rand(t, hk, d).to(torch.bfloat16),
          "v": (rand(t, hv, d) * (0.3 + 1.4 * torch.rand(hv, d, generator=g, device="cuda"))).to(torch.bfloat16),
          "starts": whole(starts), "most_new": max(new),
          "decay": -rate * torch.rand(t, hv, generator=g, device="cuda").mul_(2) if c["each"] else -rate,
          # each sequence reads the state of one slot and leaves its own in another
          "states": rand(2 * seqs, hv, d, d).mul_(2)}
    at = torch.randperm(2 * seqs, generator=g, device="cuda").to(torch.int32)
    s["slots"], s["slots_out"] = at[:seqs].contiguous(), at[seqs:].contiguous()
    if own:
        from routed_expert_prefill_gb300 import layer

        s["state"] = layer.LinearState(s["states"])
    return s


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if own:
        from routed_expert_prefill_gb300 import layer

        if s["op"] == "norms":
            r = layer.moe_gated_rms_norm(s["x"], s["gamma"], s["residual"], s["post"], s["gate"], gate_sigmoid=s["sigmoid"],
                                         residual_scale=s["scale"], eps=EPS, quantize=s["q8"])
            if not s["q8"]:
                return {"sum": r.sum, "y": r.y}
            torch.mul(r.codes.view(s["values"].shape), r.scales.unsqueeze(-1), out=s["values"])
            return {"sum": r.sum, "values": s["values"], "scales": r.scales}
        if s["op"] == "plan":
            s["pages"].account.copy_(s["account"])  # as the pool stood before the call
            p = layer.moe_kv_plan(s["new"], s["cache"], s["pages"], s["t"], lens=s["before"])
            return {"starts": p.starts, "seq": p.seq, "pos": p.pos, "slot": p.slot, "lens": s["lens"],
                    "table": s["table"], "free": s["free"], "account": s["pages"].account}
        if s["op"] == "logprobs":
            r = layer.moe_logprobs(s["logits"], s["ids"], top=s["top"])
            out = {"logprob": r.logprob, "entropy": r.entropy, "lse": r.lse}
            return out | {"top_ids": r.top_ids, "top_logprobs": r.top_logprobs} if s["top"] else out
        o = layer.moe_linear_attention(s["q"], s["k"], s["v"], s["decay"], s["starts"], s["state"], slots=s["slots"],
                                       slots_out=s["slots_out"])
        return {"out": o, "states": s["states"]}
    return {"norms": _norms, "plan": _tables, "logprobs": _logprobs, "linear": _linear}[s["op"]](s)


def _norms(s):
    x = s["x"].float()
    b = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + EPS) * s["post"].float()
    if s["gate"] is not None:
        gate = s["gate"].float()
        b = b * (1 / (1 + torch.exp(-gate)) if s["sigmoid"] else gate)
    a = s["residual"].float() * s["scale"] + b
    y = a * torch.rsqrt(a.square().mean(-1, keepdim=True) + EPS) * s["gamma"].float()
    if not s["q8"]:
        return {"sum": a.to(torch.bfloat16), "y": y.to(torch.bfloat16)}
    q, step = _to_8_bits(y.view(s["values"].shape))
    return {"sum": a.to(torch.bfloat16), "values": (q * step[..., None]).to(torch.bfloat16), "scales": step}


def _tables(s):
    new, before, table, free, block = s["new"], s["before"], s["table"], s["free"], s["block"]
    dev = new.device
    seqs, width = table.shape
    held, count = s["account"][:-1], s["account"][-1]
    grow = new.clamp(min=0)
    lens = torch.where(new < 0, torch.zeros_like(before), before + grow)
    starts = torch.cat([torch.zeros_like(grow[:1]), grow.cumsum(0, dtype=torch.int32)])
    # pages of the sequences that end go on top of the pool, in order
    b = torch.arange(width, device=dev)
    given = torch.where(new < 0, held, torch.zeros_like(held))
    place = count + given.cumsum(0)[:, None] - given[:, None] + b
    place = torch.where(b < given[:, None], place, torch.full_like(place, free.shape[0]))
    pool = torch.cat([free, free[:1]]).scatter(0, place.reshape(-1), table.reshape(-1))[:-1]
    # the others take theirs from the top
    need = torch.where(new < 0, torch.zeros_like(held), torch.maximum(held, (lens + block - 1) // block))
    more = torch.where(new < 0, torch.zeros_like(held), need - held)
    top = count + given.sum()
    nth = more.cumsum(0)[:, None] - more[:, None] + b - held[:, None]
    takes = (b >= held[:, None]) & (b < need[:, None])
    page = pool[(top - 1 - nth).clamp(0, free.shape[0] - 1)]
    table.copy_(torch.where(takes, page, table))
    free.copy_(pool)
    s["lens"].copy_(lens)
    row = torch.arange(s["t"], dtype=torch.int32, device=dev)
    seq = torch.searchsorted(starts[1:].contiguous(), row, right=True, out_int32=True)
    live = row < starts[-1]
    own_seq = seq.clamp(max=seqs - 1).long()
    pos = before[own_seq] + row - starts[own_seq]
    slot = table[own_seq, (pos // block).clamp(0, width - 1).long()].long() * block + pos % block
    none = torch.full_like(seq, -1)
    return {"starts": starts, "seq": torch.where(live, seq, none), "pos": torch.where(live, pos, none),
            "slot": torch.where(live, slot, none.long()), "lens": s["lens"], "table": table, "free": free,
            "account": torch.cat([need, (top - more.sum())[None]]).to(torch.int32)}


def _logprobs(s):
    x = s["logits"].float()
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1)
    lse = m[:, 0] + torch.log(total)
    entropy = torch.log(total) - (e * (x - m)).sum(-1) / total
    given = x.gather(1, s["ids"][:, None])[:, 0]
    out = {"logprob": given - lse, "entropy": entropy, "lse": lse}
    if s["top"]:
        bits = (x + 0.0).view(torch.int32)  # whole numbers in the order of the values, the lower index first among equals
        order = torch.where(bits < 0, bits ^ 0x7FFFFFFF, bits).long()
        key = (order << 32) + (x.shape[1] - torch.arange(x.shape[1], device=x.device))
        best = (x.shape[1] - (key.topk(s["top"], -1).values & 0xFFFFFFFF)).to(torch.int32)
        out |= {"top_ids": best, "top_logprobs": x.gather(1, best.long()) - lse[:, None]}
    return out


def _linear(s):
    dev, d = s["q"].device, s["q"].shape[2]
    starts, hv = s["starts"].long(), s["v"].shape[1]
    n = starts[1:] - starts[:-1]
    seqs, chunks = n.shape[0], -(-s["most_new"] // CHUNK)
    row = torch.arange(chunks * CHUNK, device=dev)
    live = row < n[:, None]
    at = (starts[:-1, None] + row).clamp(max=s["q"].shape[0] - 1)
    group = hv // s["q"].shape[1]

    def tiles(x, repeat):  # [sequence, head, chunk, row, channel], zero behind the sequence's end
        x = torch.where(live[..., None, None], x[at].float(), torch.zeros((), device=dev))
        return x.repeat_interleave(repeat, 2).view(seqs, chunks, CHUNK, hv, d).permute(0, 3, 1, 2, 4)

    q, k, v = tiles(s["q"], group) / math.sqrt(d), tiles(s["k"], group), tiles(s["v"], 1)
    g = s["decay"].double()
    g = g[at] if g.dim() == 2 else g.expand(seqs, chunks * CHUNK, hv)
    g = torch.where(live[..., None], g, torch.zeros_like(g)).view(seqs, chunks, CHUNK, hv).permute(0, 3, 1, 2)
    inside = g.cumsum(-1)  # [sequence, head, chunk, row]
    whole = inside[..., -1]
    ends = whole.cumsum(-1)
    causal = torch.ones(CHUNK, CHUNK, dtype=torch.bool, device=dev).tril()
    w = torch.exp((inside[..., :, None] - inside[..., None, :]).masked_fill(~causal, -math.inf)).float()
    o = (q @ k.transpose(-1, -2) * w) @ v
    added = (k * torch.exp(whole[..., None] - inside).float()[..., None]).transpose(-1, -2) @ v
    # the state before chunk i (and behind the last one): what chunks j < i added and the first state, decayed
    begins = torch.cat([torch.zeros_like(ends[..., :1]), ends], -1)
    before = torch.ones(chunks + 1, chunks, dtype=torch.bool, device=dev).tril(-1)
    w = torch.exp((begins[..., :, None] - ends[..., None, :]).masked_fill(~before, -math.inf)).float()
    first = s["states"][s["slots"].long()]
    state = (w @ added.reshape(seqs, hv, chunks, d * d)).view(seqs, hv, chunks + 1, d, d)
    state += torch.exp(begins).float()[..., None, None] * first[:, :, None]
    o += torch.exp(inside).float()[..., None] * (q @ state[:, :, :-1])
    s["states"][s["slots_out"].long()] = state[:, :, -1]
    o = o.permute(0, 2, 3, 1, 4).reshape(seqs, chunks * CHUNK, hv, d)
    return {"out": o[live].to(torch.bfloat16), "states": s["states"]}


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
    if case["op"] == "norms":
        def normed(z, weight):
            return z / ((z * z).sum(-1, keepdim=True) / case["h"] + EPS).sqrt() * weight.to(f)

        b = normed(s["x"].to(f), s["post"])
        if case["gate"] != "none":
            b = b * (torch.sigmoid(s["gate"].to(f)) if case["sigmoid"] else s["gate"].to(f))
        a = s["scale"] * s["residual"].to(f) + b
        y = normed(a, s["gamma"])
        if not case["q8"]:
            return {"sum": a, "y": y}
        z = y.reshape(case["t"], -1, GROUP)
        top = z.abs().max(-1).values
        q = (z * 127 / top.clamp(min=1e-300).unsqueeze(-1)).round()
        return {"sum": a, "values": q * (top / 127).unsqueeze(-1), "scales": top / 127}
    if case["op"] == "plan":
        new, before, block = s["new"].tolist(), s["before"].tolist(), case["block"]
        table, free, account = s["table"].tolist(), s["free"].tolist(), s["account"].tolist()
        lens, starts, seq, pos, slot = [], [0], [], [], []
        top = account[-1]
        for i, n in enumerate(new):
            if n < 0:
                for b in range(account[i]):
                    free[top] = table[i][b]
                    top += 1
                account[i] = 0
        for i, (n, old) in enumerate(zip(new, before)):
            while n > 0 and account[i] * block < old + n:
                top -= 1
                table[i][account[i]] = free[top]
                account[i] += 1
            lens.append(0 if n < 0 else old + n)
            for p in range(old, old + n):
                seq.append(i)
                pos.append(p)
                slot.append(table[i][p // block] * block + p % block)
            starts.append(len(seq))
        account[-1] = top
        blank = [-1] * (s["t"] - len(seq))
        whole = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
        return {"starts": whole(starts), "seq": whole(seq + blank), "pos": whole(pos + blank),
                "slot": torch.tensor(slot + blank, device="cuda"), "lens": whole(lens), "table": whole(table),
                "free": whole(free), "account": whole(account)}
    if case["op"] == "logprobs":
        found = {"logprob": [], "entropy": [], "lse": [], "top_ids": [], "top_logprobs": []}
        step = max(1, (1 << 26) // case["n"])
        for i in range(0, case["t"], step):  # rows, in pieces
            x = s["logits"][i:i + step].to(f)
            lse = torch.logsumexp(x, -1, keepdim=True)
            lp = x - lse
            found["lse"].append(lse[:, 0])
            found["logprob"].append(lp[torch.arange(x.shape[0], device="cuda"), s["ids"][i:i + step]])
            found["entropy"].append(-(lp.exp() * lp).sum(-1))
            best = torch.sort(x, dim=-1, descending=True, stable=True).indices[:, :case["top"]]
            found["top_ids"].append(best.to(torch.int32))
            found["top_logprobs"].append(torch.take_along_dim(lp, best, 1))
        return {p: torch.cat(v) for p, v in found.items() if case["top"] or not p.startswith("top")}
    new = _lengths(case)
    if max(new) > 8192:
        return None
    hv, d, group = case["hv"], case["d"], case["hv"] // case["hk"]
    first = s["starts"][:-1].long()
    n = torch.tensor(new, device="cuda")
    out = torch.zeros(s["v"].shape, dtype=f, device="cuda")
    states = s["states"].to(f)
    a = states[s["slots"].long()]
    g = s["decay"].to(f)
    for i in range(max(new)):  # one row of every sequence that has as many
        some = [j for j, m in enumerate(new) if m > i]
        at = slice(None) if len(some) == len(new) else torch.tensor(some, device="cuda")
        r = first[at] + i
        q, k = (s[p][r].to(f).repeat_interleave(group, 1) for p in "qk")
        lam = torch.exp(g[r] if g.dim() == 2 else g.expand(len(some), hv))
        b = a[at] * lam[..., None, None] + k.unsqueeze(-1) * s["v"][r].to(f).unsqueeze(-2)
        a[at] = b
        out[r] = (q.unsqueeze(-1) * b).sum(-2) / math.sqrt(d)
    states[s["slots_out"].long()] = a
    return {"out": out, "states": states}

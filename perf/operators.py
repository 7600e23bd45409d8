"""The serving operators beside the quantised activations, as cases that can be timed and compared.

One decode step of a model whose activations are rotated (`rht_heads`, `rht_head_mix_quant`) needs four more
operators next to them: a plan of the paged cache built on the GPU from the requests' lengths (`kv8_plan`), the
append of new keys and values to a cache of 8-bit codes with one scale for each block of tokens and head
(`kv8_append`), the attention that reads that cache (`kv8_attention`), and the matrix products of a few token rows
with 4-bit weights that carry a scale for each group of inputs (`w4_matvec`).

`own` chooses who computes: the plain torch form below, or the package's entry points."""
import math
import random

import torch

own = False

DEV = "cuda"


def _rsq():
    from w3a3_quantization_online_b200 import rsq
    return rsq


# ------------------------------------------------------------------------------------------------- cases

def listed():
    return [
        # one decode step of 64 running requests: 64 lengths in, 64 slots out (latency)
        {"name": "plan-decode", "op": "plan", "batch": 64, "block": 64, "ctx": 8192, "new": 1, "pad": 0, "lens": 1},
        # the admission of 48 prompts of ragged lengths into a batch padded to whole rows of 256
        {"name": "plan-prompts", "op": "plan", "batch": 48, "block": 16, "ctx": 2000, "new": 1024, "pad": 256, "lens": 2},
        # one token of each of 64 requests into partly filled blocks
        {"name": "append-decode", "op": "append", "batch": 64, "block": 64, "ctx": 1024, "new": 1, "kv": 8, "dh": 128,
         "dtype": "bf16", "fused": True, "lens": 3},
        # the keys and values of 16384 prompt tokens, 32 heads of 128, read out of a fused projection's rows
        {"name": "append-prompts", "op": "append", "batch": 12, "block": 64, "ctx": 100, "new": 2000, "kv": 32, "dh": 128,
         "dtype": "bf16", "fused": True, "lens": 4},
        # the first steps of one short request, a head of keys for each head of queries
        {"name": "decode-short", "op": "attention", "batch": 1, "block": 16, "ctx": 200, "new": 1, "heads": 32, "kv": 32,
         "dh": 128, "dtype": "bf16", "lens": 5},
        # a serving batch: 64 requests from a few tokens to 8192, four query heads to a key head
        {"name": "decode-batch", "op": "attention", "batch": 64, "block": 64, "ctx": 8192, "new": 1, "heads": 32, "kv": 8,
         "dh": 128, "dtype": "bf16", "lens": 6},
        # two long documents: the keys of one head are spread over the whole GPU
        {"name": "decode-long", "op": "attention", "batch": 2, "block": 128, "ctx": 131072, "new": 1, "heads": 32, "kv": 8,
         "dh": 128, "dtype": "bf16", "lens": 7},
        # prompts in chunks of up to 2048 tokens on top of what the cache holds
        {"name": "prompt-chunks", "op": "attention", "batch": 3, "block": 64, "ctx": 8000, "new": 2048, "heads": 32, "kv": 8,
         "dh": 128, "dtype": "bf16", "lens": 8},
        # a few guessed tokens a request are checked at once, in float32, five query heads to a key head
        {"name": "verify-f32", "op": "attention", "batch": 17, "block": 32, "ctx": 1900, "new": 4, "heads": 20, "kv": 4,
         "dh": 64, "dtype": "f32", "lens": 9},
        # one token through a hidden-size projection
        {"name": "matvec-1", "op": "matvec", "rows": 1, "n": 4096, "k": 4096, "group": 128, "dtype": "bf16"},
        # a float32 batch of odd size through the down projection
        {"name": "matvec-down-f32", "op": "matvec", "rows": 5, "n": 4096, "k": 12288, "group": 64, "dtype": "f32"},
        # a decode batch of 48 through the wide hidden size, small groups
        {"name": "matvec-48", "op": "matvec", "rows": 48, "n": 8192, "k": 8192, "group": 32, "dtype": "bf16"},
    ]


def _log(rng, lo, hi):
    """A whole number of [lo, hi], spread over the logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "append", "attention", "attention", "attention", "matvec", "matvec"])
    c = {"op": op, "lens": rng.randrange(1, 1 << 30)}
    if op == "plan":
        c |= {"batch": _log(rng, 1, 512), "block": rng.choice([16, 32, 64, 128]), "ctx": _log(rng, 1, 16384),
              "new": rng.choice([1, 1, _log(rng, 2, 256)]), "pad": rng.choice([0, 1, 64])}
    elif op == "append":
        new = rng.choice([1, _log(rng, 2, 2000)])
        c |= {"batch": _log(rng, 1, 128 if new == 1 else 10), "block": rng.choice([16, 32, 64, 128]),
              "ctx": _log(rng, 1, 1024), "new": new, "kv": _log(rng, 1, 32), "dh": rng.choice([64, 128]),
              "dtype": rng.choice(["bf16", "bf16", "f32"]), "fused": rng.random() < 0.5}
    elif op == "attention":
        new = rng.choice([1, 1, 1, _log(rng, 2, 8), _log(rng, 64, 1024)])
        batch = _log(rng, 1, 96 if new == 1 else 16 if new <= 8 else 3)
        kv = rng.choice([1, 2, 4, 8, 8])
        c |= {"batch": batch, "block": rng.choice([16, 32, 64, 128]),
              "ctx": _log(rng, 8, min(65536, 262144 // batch) if new <= 8 else 6000), "new": new,
              "heads": kv * rng.choice([1, 2, 3, 4, 4, 5, 8]), "kv": kv, "dh": rng.choice([64, 128, 128]),
              "dtype": rng.choice(["bf16", "bf16", "f32"]) if new <= 8 else "bf16"}
        c["heads"] = min(c["heads"], 40)
        c["heads"] -= c["heads"] % kv
    else:
        group = rng.choice([32, 64, 128, 128])
        c |= {"rows": _log(rng, 1, 64), "n": _log(rng, 500, 12288), "k": group * _log(rng, max(2, 1024 // group), 12288 // group),
              "group": group, "dtype": rng.choice(["bf16", "bf16", "f32"])}
    return c


def _lengths(c):
    """(tokens in the cache before the call, new tokens) of each request: part of the case, whatever the seed. Lengths are
    spread over their logarithm, one request is as long as the case allows, and in a larger batch some places are empty."""
    rng = random.Random(c["lens"])
    ctx = [c["ctx"]] + [_log(rng, 1, c["ctx"]) for _ in range(c["batch"] - 1)]
    if c["new"] == 1:
        new = [1] * c["batch"]
    else:
        new = [c["new"]] + [_log(rng, max(1, c["new"] // 3), c["new"]) for _ in range(c["batch"] - 1)]
    for i in range(1, c["batch"]):
        r = rng.random()
        if c["batch"] > 8 and r < 0.05:
            ctx[i] = new[i] = 0            # an empty place of the batch
        elif r < 0.1:
            ctx[i] = 0                     # a request's first tokens
    if c["op"] == "attention":
        ctx[0] -= min(ctx[0], c["new"])    # the longest one ends at the case's length
    order = list(range(c["batch"]))
    rng.shuffle(order)
    return [ctx[i] for i in order], [new[i] for i in order]


def _blocks(n, size):
    return -(-n // size)


def _rows(c):
    """Rows of the token arrays: the new tokens, and what pads them."""
    n = sum(_lengths(c)[1])
    return _blocks(n, c["pad"]) * c["pad"] if c.get("pad") else n


def _dtype(c):
    return torch.bfloat16 if c["dtype"] == "bf16" else torch.float32


def _visible(c):
    """Pairs of a new token and a key that it sees."""
    return sum(n * k + n * (n + 1) // 2 for k, n in zip(*_lengths(c)))


def work(case):
    c = case
    if c["op"] == "matvec":
        e = 2 if c["dtype"] == "bf16" else 4
        return {"bytes": c["n"] * c["k"] // 2 + 4 * c["n"] * (c["k"] // c["group"]) + c["rows"] * (c["k"] + c["n"]) * e,
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    ctx, new = _lengths(c)
    seq = [a + b for a, b in zip(ctx, new)]
    if c["op"] == "plan":
        fresh = sum(_blocks(s, c["block"]) - _blocks(a, c["block"]) for a, s in zip(ctx, seq))
        # lengths in, running sums and lengths out, ids of fresh blocks in and out, a position and a slot of each row out
        return {"bytes": 8 * c["batch"] + 8 * c["batch"] + 8 * fresh + 12 * _rows(c), "flops": 0}
    if c["op"] == "append":
        e = 2 if c["dtype"] == "bf16" else 4
        touched = sum(_blocks(s, c["block"]) - a // c["block"] for a, s, n in zip(ctx, seq, new) if n)
        return {"bytes": 2 * sum(new) * c["kv"] * c["dh"] * (e + 1) + 8 * sum(new) + 2 * 8 * touched * c["kv"], "flops": 0}
    e = 2 if c["dtype"] == "bf16" else 4
    live = [s for s, n in zip(seq, new) if n]
    blocks = sum(_blocks(s, c["block"]) for s in live)
    return {"bytes": 2 * sum(live) * c["kv"] * c["dh"] + blocks * (8 * c["kv"] + 4) + 2 * sum(new) * c["heads"] * c["dh"] * e,
            "flops": 4 * c["dh"] * c["heads"] * _visible(c)}


# ------------------------------------------------------------------------------------------------- inputs

def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _codes(shape, g):
    """8-bit codes of rotated keys or values: near Gaussian, the largest of a block at the end of the range."""
    return (torch.randn(shape, generator=g, device=DEV, dtype=torch.float16) * 38).round_().clamp_(-127, 127).to(torch.int8)


def _scales(shape, g):
    return torch.exp(torch.randn(shape, generator=g, device=DEV) * 0.25) * 0.026


def _i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    c, g = case, _gen(seed)
    s = {"case": c}
    if c["op"] == "matvec":
        x = torch.randn((c["rows"], c["k"]), generator=g, device=DEV)
        x[:, torch.randint(0, c["k"], (8,), generator=g, device=DEV)] *= 20.0     # channels of outliers
        s["x"] = x.to(_dtype(c))
        s["codes"] = torch.randint(0, 256, (c["n"], c["k"] // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = torch.exp(torch.randn((c["n"], c["k"] // c["group"]), generator=g, device=DEV) * 0.3) * 0.004
        return s
    ctx, new = _lengths(c)
    seq = [a + b for a, b in zip(ctx, new)]
    size = c["block"]
    width = max(1, max(_blocks(n, size) for n in seq))
    s |= {"ctx": _i32(ctx), "new": _i32(new), "width": width, "most": max(new)}
    total = sum(_blocks(n, size) for n in seq)
    pool = total + max(2, total // 16)
    order = torch.randperm(pool, generator=g, device=DEV).to(torch.int32)
    held = _i32([_blocks(a if c["op"] == "plan" else n, size) for a, n in zip(ctx, seq)])
    cols = torch.arange(width, device=DEV, dtype=torch.int32)
    first = torch.cumsum(held, 0) - held
    at = first[:, None] + cols[None]
    s["table"] = torch.where(cols[None] < held[:, None], order[at.clamp(max=pool - 1).long()], torch.full_like(at, -1))
    if c["op"] == "plan":
        # the ids behind those in use are free; the first two of them went to an earlier call
        taken = int(sum(_blocks(a, size) for a in ctx))
        s["free"] = order[taken:].contiguous()
        s["cursor"] = _i32([2])
        s["rows"] = _rows(c)
        return s
    s["cu"] = _i32([0] + new).cumsum(0).to(torch.int32)
    s["seq"] = _i32(seq)
    shape = (pool, c["kv"], size, c["dh"])
    s["kc"], s["vc"] = _codes(shape, g), _codes(shape, g)
    s["ks"], s["vs"] = _scales(shape[:2], g), _scales(shape[:2], g)
    n, dt = sum(new), _dtype(c)
    if c["op"] == "append":
        w = c["kv"] * c["dh"]
        if c["fused"]:      # keys and values are columns of one projection's output
            rows = torch.randn((n, 3 * w), generator=g, device=DEV, dtype=dt)
            s["k"], s["v"] = rows[:, w:2 * w], rows[:, 2 * w:]
        else:
            s["k"] = torch.randn((n, w), generator=g, device=DEV, dtype=dt)
            s["v"] = torch.randn((n, w), generator=g, device=DEV, dtype=dt)
        pos = torch.cat([torch.arange(a, b) for a, b in zip(ctx, seq)]).to(DEV)
        req = torch.repeat_interleave(torch.arange(c["batch"], device=DEV), s["new"].long())
        s["slots"] = s["table"][req, pos // size].long() * size + pos % size
        return s
    s["q"] = (torch.randn((n, c["heads"] * c["dh"]), generator=g, device=DEV) * 2.0).to(dt)
    s["scale"] = 1.0 / math.sqrt(c["dh"])
    return s


# ------------------------------------------------------------------------------------------------- plain forms

def _plan(s):
    size, dev = s["case"]["block"], s["ctx"].device
    ctx, new = s["ctx"].long().clamp(min=0), s["new"].long().clamp(min=0)
    table, free = s["table"], s["free"]
    width = table.shape[1]
    seq = ctx + new
    cu = torch.zeros(len(ctx) + 1, dtype=torch.int64, device=dev)
    cu[1:] = torch.cumsum(new, 0)
    had = ((ctx + size - 1) // size).clamp(max=width)
    has = ((seq + size - 1) // size).clamp(max=width)
    ends = torch.cumsum(has - had, 0) + s["cursor"]
    cols = torch.arange(width, device=dev)
    src = (ends - (has - had))[:, None] + cols - had[:, None]
    ids = torch.where(src < len(free), free[src.clamp(0, len(free) - 1)], -1)
    table = torch.where((cols >= had[:, None]) & (cols < has[:, None]), ids, table)
    t = torch.arange(s["rows"], device=dev)
    req = torch.searchsorted(cu[1:], t, right=True)
    live = req < len(ctx)
    req = req.clamp(max=len(ctx) - 1)
    pos = torch.where(live, ctx[req] + t - cu[req], -1)
    col = pos // size
    block = table[req, col.clamp(0, width - 1)].long()
    slots = torch.where(live & (col < width) & (block >= 0), block * size + pos % size, -1)
    return [table, cu.int(), seq.int(), pos.int(), slots, ends[-1:].int()]


def _store(new, codes, scales, slots, size):
    """The codes and scales of the blocks after the rows `new` are written at `slots`, for one of keys and values."""
    n_blocks, heads = scales.shape
    x = new.reshape(len(slots), heads, -1).float()
    block, off = slots // size, slots % size
    ids = block[:, None].expand(-1, heads)
    most = torch.zeros_like(scales).scatter_reduce(0, ids, x.abs().amax(-1), "amax")
    first = torch.full((n_blocks,), size, device=x.device).scatter_reduce(0, block, off, "amin")
    touched = (first < size)[:, None]
    old = torch.where((first > 0)[:, None], scales, 0.0)            # a block that starts anew forgets its scale
    scale = torch.where(touched, torch.maximum(old, most / 127.0), scales)
    keep = touched & (scale > old) & (first > 0)[:, None]
    ratio = torch.where(keep, old / scale, 1.0)[:, :, None, None]
    held = torch.arange(size, device=x.device) < torch.where(first < size, first, 0)[:, None]
    again = torch.round(codes.float() * ratio).to(torch.int8)
    codes = torch.where(held[:, None, :, None], again, codes)
    by = scale[block][:, :, None]
    q = torch.where((by > 0) & by.isfinite(), torch.round(x / by), 0.0).clamp(-127, 127).to(torch.int8)
    codes[block, :, off] = q
    return codes, scale


def _append(s):
    size = s["case"]["block"]
    kc, ks = _store(s["k"], s["kc"], s["ks"], s["slots"], size)
    vc, vs = _store(s["v"], s["vc"], s["vs"], s["slots"], size)
    return [kc, ks, vc, vs]


def _read(codes, scales, table):
    """[batch, heads, tokens, width] of the values that a cache holds, in the order of the tables."""
    at = table.clamp(min=0).long()
    x = codes[at].float() * scales[at][..., None, None]
    b, n, h, size, d = x.shape
    return x.transpose(1, 2).reshape(b, h, n * size, d)


def _attend(s):
    c = s["case"]
    kv, d, q = c["kv"], c["dh"], s["q"]
    g, b, most = c["heads"] // kv, c["batch"], s["most"]
    k, v = _read(s["kc"], s["ks"], s["table"]), _read(s["vc"], s["vs"], s["table"])
    i = torch.arange(most, device=q.device)
    live = i < s["new"][:, None]
    rows = (s["cu"][:-1, None] + i).clamp(max=len(q) - 1).long()
    x = q.float().reshape(-1, kv, g, d)[rows].permute(0, 2, 3, 1, 4).reshape(b, kv, g * most, d)
    w = torch.matmul(x, k.transpose(2, 3)).mul_(s["scale"]).reshape(b, kv, g, most, -1)
    pos = (s["seq"] - s["new"])[:, None] + i
    w.masked_fill_(torch.arange(w.shape[-1], device=q.device) > pos[:, None, None, :, None], float("-inf"))
    w.sub_(w.amax(-1, keepdim=True)).exp_()
    w.div_(w.sum(-1, keepdim=True))
    o = torch.matmul(w.reshape(b, kv, g * most, -1), v).reshape(b, kv, g, most, d).permute(0, 3, 1, 2, 4)
    return [o[live].reshape(len(q), -1).to(q.dtype)]


def _matvec(s):
    c, b = s["case"], s["codes"]
    w = torch.stack([b & 15, b >> 4], -1).reshape(c["n"], -1).to(torch.int8)
    w = torch.where(w > 7, w - 16, w).float().reshape(c["n"], -1, c["group"]) * s["scales"][:, :, None]
    return [torch.matmul(s["x"].float(), w.reshape(c["n"], c["k"]).t()).to(s["x"].dtype)]


# The 8-bit codes of an append are whole numbers of the cache itself and have to be equal; with the scales beside them they
# say what the cache holds. An append writes the same a second time: the scales have grown, and the codes follow from them.

def run(state):
    s, op = state, state["case"]["op"]
    if own:
        rsq = _rsq()
        if op == "plan":
            cu, seq, pos, slots, cursor = rsq.kv8_plan(s["ctx"], s["new"], s["table"], s["free"], s["cursor"], s["rows"],
                                                       s["case"]["block"])
            return [s["table"], cu, seq, pos, slots, cursor]
        if op == "append":
            rsq.kv8_append(s["k"], s["v"], s["slots"], s["kc"], s["ks"], s["vc"], s["vs"])
            return [s["kc"], s["ks"], s["vc"], s["vs"]]
        if op == "attention":
            return [rsq.kv8_attention(s["q"], s["kc"], s["ks"], s["vc"], s["vs"], s["table"], s["seq"], s["cu"],
                                      sm_scale=s["scale"])]
        return [rsq.w4_matvec(s["x"], s["codes"], s["scales"])]
    return {"plan": _plan, "append": _append, "attention": _attend, "matvec": _matvec}[op](s)


# ------------------------------------------------------------------------------------------------- 64 bits

def exact(case, seed):
    c = case
    if c["op"] == "plan":
        return None
    s = prepare(case, seed)
    if c["op"] == "matvec":
        y = torch.zeros((c["rows"], c["n"]), dtype=torch.float64, device=DEV)
        step = max(1, (1 << 26) // c["k"])
        for a in range(0, c["n"], step):
            b = s["codes"][a:a + step].long()
            w = torch.empty((len(b), c["k"]), dtype=torch.float64, device=DEV)
            w[:, 0::2] = ((b % 16 + 8) % 16 - 8).double()
            w[:, 1::2] = ((b // 16 + 8) % 16 - 8).double()
            w *= s["scales"][a:a + step].double().repeat_interleave(c["group"], 1)
            y[:, a:a + step] = s["x"].double() @ w.T
        return [y]
    if c["op"] == "append":
        # the scales alone have a value in 64 bits: the codes are whole numbers
        out = []
        for new, scale in ((s["k"], s["ks"]), (s["v"], s["vs"])):
            x = new.double().reshape(len(new), c["kv"], c["dh"]).abs().max(2).values / 127
            blocks = (s["slots"] // c["block"]).tolist()
            offs = (s["slots"] % c["block"]).tolist()
            x, want = x.cpu(), scale.double().cpu()
            for t, (b, o) in enumerate(zip(blocks, offs)):
                if o == 0:
                    want[b] = x[t]
                else:
                    want[b] = torch.maximum(want[b], x[t])
            out.append(want.to(DEV))
        return [None, out[0], None, out[1]]
    ctx, new = _lengths(c)
    g, d, size = c["heads"] // c["kv"], c["dh"], c["block"]
    out, at = torch.zeros((sum(new), c["heads"], d), dtype=torch.float64, device=DEV), 0
    for b, (a, n) in enumerate(zip(ctx, new)):
        if n == 0:
            continue
        ids = s["table"][b, :_blocks(a + n, size)].long()
        for h in range(c["kv"]):
            k = (s["kc"][ids, h].double() * s["ks"][ids, h].double()[:, None, None]).reshape(-1, d)[:a + n]
            v = (s["vc"][ids, h].double() * s["vs"][ids, h].double()[:, None, None]).reshape(-1, d)[:a + n]
            for j in range(h * g, h * g + g):
                z = (s["q"][at:at + n, j * d:(j + 1) * d].double() @ k.T) * s["scale"]
                seen = torch.ones((n, a + n), dtype=torch.bool, device=DEV).tril(a)
                out[at:at + n, j] = torch.softmax(z.masked_fill(~seen, -math.inf), -1) @ v
        at += n
    return [out.reshape(len(out), -1)]

"""The attention operators of the decode layer, as cases that can be timed and checked.

Three operators fill the place between the input projection and the out-projection:
  tables     positions, slots and block-table entries of a step's tokens, from the requests' lengths
  rope       rotary positions of q and k, and the write of k and v into the paged cache
  attention  softmax(scale q k) v over a shared prefix and each request's own cached tokens
Each has a plain form in elementary torch operations and the library's call. The head layout of the
ordinary cases is the decode layer's own: an input projection 12288 wide holds 64 query heads and
16 key and 16 value heads of 128, and 64 x 128 = 8192 is the out-projection's input.
"""
import math

import torch

own = False
DEV = "cuda"
_kept = {}


def listed():
    return [
        # every decode step begins with this: 64 requests, one token each
        dict(op="tables", name="tables, 64 requests of one token", requests=64, ctx_lo=1, ctx_hi=8192, prompts=0,
             new_lo=1, new_hi=1, block=16, pad_rows=0),
        # admission: a few prompts arrive beside running requests; the largest table work
        dict(op="tables", name="tables, 24 prompts beside 200 running", requests=224, ctx_lo=3, ctx_hi=30000, prompts=24,
             new_lo=900, new_hi=6000, block=16, pad_rows=77),
        # one user's token, the latency case
        dict(op="rope", name="rope, one token", tokens=1, heads=64, kv=16, dim=128, rot=128, inter=False,
             scaling="none", factor=1.0, pos_lo=5000, pos_hi=5001, block=16, skip=0),
        # a full decode batch far into long contexts, with frequencies stretched for them
        dict(op="rope", name="rope, 64 tokens at far positions", tokens=64, heads=64, kv=16, dim=128, rot=64, inter=True,
             scaling="yarn", factor=32.0, pos_lo=1000, pos_hi=1000000, block=32, skip=3),
        # a prompt that is written to the cache in one piece
        dict(op="rope", name="rope, prompt of 8192", tokens=8192, heads=64, kv=16, dim=128, rot=128, inter=False,
             scaling="bands", factor=8.0, pos_lo=0, pos_hi=8192, block=16, skip=0),
        # small heads, odd token count
        dict(op="rope", name="rope, 1531 tokens of small heads", tokens=1531, heads=56, kv=8, dim=64, rot=48, inter=False,
             scaling="linear", factor=4.0, pos_lo=100, pos_hi=40000, block=64, skip=11),
        # one user's short chat, the latency case
        dict(op="attention", name="attention, one request of 777", requests=1, new=1, heads=64, kv=16, dim=128, block=16,
             prefix=0, ctx_lo=777, ctx_hi=777, idle=0, pad_rows=0),
        # a full batch of ordinary chats, ragged, with rows that no request uses
        dict(op="attention", name="attention, 61 ragged requests", requests=61, new=1, heads=64, kv=16, dim=128, block=16,
             prefix=0, ctx_lo=1, ctx_hi=4096, idle=2, pad_rows=3),
        # one user with a very long document: the work of one row has to spread over the whole chip
        dict(op="attention", name="attention, one request of 131000", requests=1, new=1, heads=64, kv=16, dim=128, block=64,
             prefix=0, ctx_lo=131000, ctx_hi=131000, idle=0, pad_rows=0),
        # a verify batch of eight drafts for each of eight requests
        dict(op="attention", name="attention, 8 requests of 8 drafts", requests=8, new=8, heads=64, kv=16, dim=128, block=32,
             prefix=0, ctx_lo=2000, ctx_hi=16000, idle=0, pad_rows=0),
        # agents that share a long system prompt and documents: the most arithmetic
        dict(op="attention", name="attention, 64 requests on a prefix of 32768", requests=64, new=1, heads=64, kv=16,
             dim=128, block=16, prefix=32768, ctx_lo=1, ctx_hi=2000, idle=0, pad_rows=0),
        # the same at a tensor-parallel shard's heads: few heads, a prefix that ends inside a block
        dict(op="attention", name="attention, 16 requests of small heads on a prefix of 5003", requests=16, new=1, heads=32,
             kv=4, dim=64, block=16, prefix=5003, ctx_lo=30, ctx_hi=900, idle=1, pad_rows=0),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["tables", "rope", "attention", "attention"])
    if op == "tables":
        prompts = rng.choice([0, 0, rng.randint(1, 24)])
        hi = _log(rng, 20, 30000)
        new_hi = _log(rng, 16, 6000)
        return dict(op=op, requests=prompts + _log(rng, 1, 200), ctx_lo=rng.randint(1, 20), ctx_hi=hi, prompts=prompts,
                    new_lo=max(1, new_hi // 8), new_hi=new_hi, block=rng.choice([16, 32, 64, 128]),
                    pad_rows=rng.choice([0, rng.randint(1, 64)]))
    if op == "rope":
        heads, kv, dim = rng.choice([(64, 16, 128), (32, 8, 128), (56, 8, 64), (8, 1, 128), (16, 16, 64), (71, 1, 64)])
        rot = rng.choice([dim, dim // 2, dim // 4, dim - 16])
        tokens = _log(rng, 1, 8192)
        lo = _log(rng, 1, 100000)
        return dict(op=op, tokens=tokens, heads=heads, kv=kv, dim=dim, rot=rot, inter=rng.random() < 0.5,
                    scaling=rng.choice(["none", "linear", "ntk", "bands", "yarn"]), factor=rng.choice([2.0, 8.0, 40.0]),
                    pos_lo=lo, pos_hi=lo + tokens + _log(rng, 1, 900000), block=rng.choice([16, 32, 64, 128]),
                    skip=rng.choice([0, min(tokens - 1, rng.randint(1, 9))]))
    heads, kv, dim = rng.choice([(64, 16, 128), (32, 8, 128), (32, 4, 64), (28, 4, 128), (16, 16, 64), (8, 2, 128), (20, 1, 64)])
    new = rng.choice([1, 1, 1, 2, 4, 8, rng.randint(3, 16)])
    requests = _log(rng, 1, 64 // new)
    prefix = rng.choice([0, 0, _log(rng, 50, 32768)])
    # the keys that a case of this size may hold without passing the largest listed ones
    token = kv * dim * 4
    most = min(130000, int(1e9 / (token * requests)))
    hi = _log(rng, 2, max(4, most))
    idle = rng.choice([0, rng.randint(0, max(0, (requests - 1) // 4))])
    room = 64 - (requests - idle) * new
    return dict(op=op, requests=requests, new=new, heads=heads, kv=kv, dim=dim, block=rng.choice([16, 32, 64, 128]),
                prefix=prefix, ctx_lo=max(1, hi // rng.choice([1, 2, 100])), ctx_hi=hi, idle=idle,
                pad_rows=rng.choice([0, min(room, rng.randint(0, 5))]))


def _spread(n, lo, hi):
    """n whole numbers from lo to hi, even on a logarithmic scale and out of order; the last is hi."""
    f = [((i + 1) * 0.6180339887498949) % 1.0 for i in range(n)]
    v = [int(round(lo * (hi / lo) ** x)) if hi > lo else lo for x in f]
    v[n - 1] = hi
    return v


def _lengths(case):
    """(tokens in the cache, new tokens) of each request."""
    n = case["requests"]
    ctx = _spread(n, case["ctx_lo"], case["ctx_hi"])
    if case["op"] == "tables":
        new = [1] * n
        if case["prompts"]:
            # prompts are new requests, with nothing in the cache, spread among the others
            at = [int((i + 0.5) * n / case["prompts"]) for i in range(case["prompts"])]
            for i, length in zip(at, _spread(len(at), case["new_lo"], case["new_hi"])):
                new[i], ctx[i] = length, 0
        return ctx, new
    new = [case["new"]] * n
    for i in range(case["idle"]):  # slots of the batch whose request has finished
        new[(7 * i + 1) % n] = 0
    return ctx, new


def _blocks(tokens, size):
    return (tokens + size - 1) // size


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape, scale=1.0):
    return (torch.randn(*shape, device=DEV, generator=g) * scale).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        size = case["block"]
        held = [_blocks(c, size) for c in ctx]
        total = [_blocks(c + n, size) for c, n in zip(ctx, new)]
        order = torch.randperm(sum(total) + 100, device=DEV, generator=g).to(torch.int32)
        width = max(total) + 5
        table = torch.full((len(ctx), width), -1, dtype=torch.int32, device=DEV)
        inside = torch.arange(width, device=DEV)[None, :] < _ints(held)[:, None]
        table[inside] = order[:sum(held)]
        free = torch.zeros(sum(total) + 100, dtype=torch.int32, device=DEV)
        left = sum(total) + 100 - sum(held)
        free[:left] = order[sum(held):]
        rows = sum(new) + case["pad_rows"]
        # the prefix that all requests share comes before their own tokens
        s.update(ctx=_ints(ctx), new=_ints(new), free=free, count=_ints([left]), table=table, rows=rows,
                 offset=1 + int(torch.randint(0, 5000, (1,), device=DEV, generator=g)),
                 row_start=torch.empty(len(ctx) + 1, dtype=torch.int32, device=DEV),
                 own_len=torch.empty(len(ctx), dtype=torch.int32, device=DEV),
                 positions=torch.empty(rows, dtype=torch.int32, device=DEV),
                 slots=torch.empty(rows, dtype=torch.int32, device=DEV),
                 left=torch.empty(2, dtype=torch.int32, device=DEV))
    elif case["op"] == "rope":
        t, hq, kv, d, size = case["tokens"], case["heads"], case["kv"], case["dim"], case["block"]
        # q, k and v are columns of one projection's output
        y = _normal(g, t, (hq + 2 * kv) * d)
        blocks = _blocks(t, size) + 3
        slots = torch.randperm(blocks, device=DEV, generator=g)[:, None] * size + torch.arange(size, device=DEV)
        slots = slots.reshape(-1)[:t].to(torch.int32)
        slots[t - case["skip"]:] = -1
        s.update(q=y[:, :hq * d], k=y[:, hq * d:(hq + kv) * d], v=y[:, (hq + kv) * d:],
                 positions=torch.randint(case["pos_lo"], case["pos_hi"], (t,), device=DEV, generator=g).to(torch.int32),
                 slots=slots, kc=_normal(g, blocks, kv, size, d), vc=_normal(g, blocks, kv, size, d),
                 out=torch.empty((t, hq * d), dtype=torch.bfloat16, device=DEV))
        s["freq"], s["mag"] = _frequencies(case)
    else:
        ctx, new = _lengths(case)
        hq, kv, d, size, prefix = case["heads"], case["kv"], case["dim"], case["block"], case["prefix"]
        held = [_blocks(c + n, size) for c, n in zip(ctx, new)]
        ahead = _blocks(prefix, size)
        blocks = sum(held) + ahead + 2
        order = torch.randperm(blocks, device=DEV, generator=g).to(torch.int32)
        table = torch.full((len(ctx), max(held)), -1, dtype=torch.int32, device=DEV)
        inside = torch.arange(max(held), device=DEV)[None, :] < _ints(held)[:, None]
        table[inside] = order[ahead:ahead + sum(held)]
        rows = sum(new) + case["pad_rows"]
        # q sharp enough that a few keys of a long context carry most of the weight
        y = _normal(g, rows, (hq + 2 * kv) * d, scale=2.5)
        start = [0]
        for n in new:
            start.append(start[-1] + n)
        s.update(q=y[:, :hq * d], kc=_normal(g, blocks, kv, size, d), vc=_normal(g, blocks, kv, size, d),
                 table=table, prefix_table=order[:ahead].contiguous(), row_start=_ints(start),
                 own_len=_ints([c + n for c, n in zip(ctx, new)]), longest=max(c + n for c, n in zip(ctx, new)),
                 scale=d ** -0.5, out=torch.zeros((rows, hq * d), dtype=torch.bfloat16, device=DEV))
    if own:
        # the handle and the descriptors of long-lived buffers that a user's program keeps
        import moe_layers_gb300 as ml
        if "handle" not in _kept:
            _kept["handle"] = ml.Handle(0)
        s["h"] = _kept["handle"]
        if case["op"] == "tables":
            s["step"] = ml.StepTables(s["row_start"], s["own_len"], s["positions"], s["slots"], s["left"])
        else:
            s["cache"] = ml.KvCache(s["kc"], s["vc"])
        if case["op"] == "rope":
            s["rope"] = ml.Rope(s["h"], case["rot"], base=500000.0, interleaved=case["inter"], scaling=case["scaling"],
                                factor=case["factor"], original_len=8192, magnitude=s["mag"])
        if case["op"] == "attention":
            s["batch"] = ml.Batch(s["row_start"], s["own_len"], s["table"], max_new=case["new"],
                                  prefix_table=s["prefix_table"], prefix_len=case["prefix"])
    return s


def _frequencies(case):
    """Radians a position turns each pair by (float64), and the factor on cos and sin."""
    r, f, length, base = case["rot"], case["factor"], 8192.0, 500000.0
    i = torch.arange(r // 2, device=DEV, dtype=torch.float64)
    freq = base ** (-2.0 * i / r)
    if case["scaling"] == "linear":
        return freq / f, 1.0
    if case["scaling"] == "ntk":
        return (base * f ** (r / (r - 2.0))) ** (-2.0 * i / r), 1.0
    if case["scaling"] == "bands":
        # whole turns within the original length: under 1 divided by the factor, over 4 kept, a blend between
        keep = ((length * freq / (2 * math.pi) - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        return keep * freq + (1.0 - keep) * freq / f, 1.0
    if case["scaling"] == "yarn":
        # the same with 32 and 1 turns as a ramp over the pair's index
        def index(turns):
            return r * math.log(length / (turns * 2 * math.pi)) / (2.0 * math.log(base))
        lo, hi = max(math.floor(index(32.0)), 0), min(math.ceil(index(1.0)), r - 1)
        keep = 1.0 - ((i - lo) / max(hi - lo, 0.001)).clamp(0.0, 1.0)
        return keep * freq + (1.0 - keep) * freq / f, 0.1 * math.log(f) + 1.0
    return freq, 1.0


def run(s):
    case = s["case"]
    if case["op"] == "tables":
        return _run_tables(s, case)
    if case["op"] == "rope":
        return _run_rope(s, case)
    return _run_attention(s, case)


def _run_tables(s, case):
    if own:
        import moe_layers_gb300 as ml
        ml.dec_batch_tables(s["h"], s["ctx"], s["new"], s["free"], s["count"], s["table"], case["block"], s["step"],
                            position_offset=s["offset"])
    else:
        size, table, rows = case["block"], s["table"], s["rows"]
        n, width = table.shape
        end = torch.cumsum(s["new"], 0)
        held, total = (s["ctx"] + size - 1) // size, (s["ctx"] + s["new"] + size - 1) // size
        first = torch.cumsum(total - held, 0) - (total - held)
        column = torch.arange(width, device=DEV)[None, :]
        at = (s["count"] - 1 - first[:, None] - (column - held[:, None])).clamp(min=0)
        fresh = (column >= held[:, None]) & (column < total[:, None])
        table.copy_(torch.where(fresh, s["free"][at], table))
        row = torch.arange(rows, device=DEV)
        request = torch.searchsorted(end, row, right=True)
        used = request < n
        request = request.clamp(max=n - 1)
        place = s["ctx"][request] + row - (end - s["new"])[request]
        s["row_start"][0] = 0
        s["row_start"][1:] = end
        s["own_len"].copy_(s["ctx"] + s["new"])
        s["positions"].copy_(torch.where(used, s["offset"] + place, 0))
        slot = table[request, (place // size).clamp(max=width - 1)] * size + place % size
        s["slots"].copy_(torch.where(used, slot, -1))
        s["left"][0] = s["count"][0] - (total - held).sum()
        s["left"][1] = 0
    return dict(row_start=s["row_start"], own_len=s["own_len"], positions=s["positions"], slots=s["slots"],
                table=s["table"], left=s["left"])


def _run_rope(s, case):
    if own:
        import moe_layers_gb300 as ml
        ml.dec_rope_append(s["h"], s["rope"], s["q"], s["k"], s["v"], s["positions"], s["slots"], s["cache"],
                           q_out=s["out"])
    else:
        t, hq, kv, d, r, size = case["tokens"], case["heads"], case["kv"], case["dim"], case["rot"], case["block"]
        angle = s["positions"].double()[:, None] * s["freq"][None, :]
        cos, sin = (torch.cos(angle) * s["mag"]).float()[:, None, :], (torch.sin(angle) * s["mag"]).float()[:, None, :]

        def turn(x):
            x = x.float()
            a, b = (x[..., 0:r:2], x[..., 1:r:2]) if case["inter"] else (x[..., :r // 2], x[..., r // 2:r])
            a, b = a * cos - b * sin, b * cos + a * sin
            both = torch.stack((a, b), -1).flatten(-2) if case["inter"] else torch.cat((a, b), -1)
            return torch.cat((both, x[..., r:]), -1).to(torch.bfloat16)

        s["out"].copy_(turn(s["q"].reshape(t, hq, d)).reshape(t, hq * d))
        # rows without a slot (-1, at the end) are not written
        slot = s["slots"][:t - case["skip"]].long()
        n = t - case["skip"]
        s["kc"][slot // size, :, slot % size] = turn(s["k"].reshape(t, kv, d))[:n]
        s["vc"][slot // size, :, slot % size] = s["v"].reshape(t, kv, d)[:n]
    return dict(q=s["out"], k=s["kc"], v=s["vc"])


def _run_attention(s, case):
    if own:
        import moe_layers_gb300 as ml
        ml.dec_attention(s["h"], s["q"], s["cache"], s["batch"], s["scale"], out=s["out"])
        return s["out"]
    hq, kv, d, size, prefix, new = (case[k] for k in ("heads", "kv", "dim", "block", "prefix", "new"))
    n, group = case["requests"], hq // kv
    rows = s["q"].shape[0]
    q = s["q"].float().reshape(rows, kv, group, d) * s["scale"]

    def keys(cache, table, length):
        """[requests, kv, length, d] in 32 bits; places without a block read block 0 and are masked by the caller."""
        place = torch.arange(length, device=DEV)
        block = table[:, place // size].clamp(min=0).long()
        return cache[block, :, place % size].float().permute(0, 2, 1, 3)

    # each request's own tokens: row i of a request sees all but the last new - 1 - i of them
    longest = s["longest"]
    count = s["row_start"][1:] - s["row_start"][:-1]
    i = torch.arange(new, device=DEV)[None, :]
    row = (s["row_start"][:-1, None] + i).clamp(max=rows - 1).long()
    mine = q[row].permute(0, 2, 1, 3, 4).reshape(n, kv, new * group, d)
    score = torch.matmul(mine, keys(s["kc"], s["table"], longest).transpose(2, 3)).reshape(n, kv, new, group, longest)
    sees = s["own_len"][:, None] - count[:, None] + i + 1
    hidden = torch.arange(longest, device=DEV)[None, None, :] >= sees[:, :, None]
    score.masked_fill_(hidden[:, None, :, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - top)
    total = weight.sum(-1, keepdim=True)
    mixed = torch.matmul(weight.reshape(n, kv, new * group, longest), keys(s["vc"], s["table"], longest))
    mixed = mixed.reshape(n, kv, new, group, d)
    del score, weight
    if prefix:
        # the prefix once for all rows, joined with each row's own part by the larger maximum
        k, v = keys(s["kc"], s["prefix_table"][None], prefix)[0], keys(s["vc"], s["prefix_table"][None], prefix)[0]
        score = torch.matmul(q.permute(1, 0, 2, 3).reshape(kv, rows * group, d), k.transpose(1, 2))
        far = score.amax(-1, keepdim=True)
        score = torch.exp(score - far)
        parts = [x.reshape(kv, rows, group, -1).permute(1, 0, 2, 3)[row].permute(0, 2, 1, 3, 4)
                 for x in (far, score.sum(-1, keepdim=True), torch.matmul(score, v))]
        both = torch.maximum(top, parts[0])
        near, far = torch.exp(top - both), torch.exp(parts[0] - both)
        mixed, total = mixed * near + parts[2] * far, total * near + parts[1] * far
    used = i < count[:, None]
    s["out"][row[used]] = (mixed / total).permute(0, 2, 1, 3, 4)[used].reshape(-1, hq * d).to(torch.bfloat16)
    return s["out"]


def work(case):
    if case["op"] == "tables":
        ctx, new = _lengths(case)
        size, n = case["block"], case["requests"]
        fresh = sum(_blocks(c + t, size) - _blocks(c, size) for c, t in zip(ctx, new))
        # lengths in; a held block's id where a request continues inside it; new ids; the tables and maps out
        return dict(bytes=4 * (2 * n + n + 2 * fresh + 2 * n + 2 * (sum(new) + case["pad_rows"])), flops=4 * sum(new))
    if case["op"] == "rope":
        t, hq, kv, d = case["tokens"], case["heads"], case["kv"], case["dim"]
        return dict(bytes=4 * t * (hq + 2 * kv) * d - 4 * case["skip"] * kv * d + 8 * t,
                    flops=3 * t * (hq + kv) * case["rot"])
    ctx, new = _lengths(case)
    hq, kv, d, prefix = case["heads"], case["kv"], case["dim"], case["prefix"]
    held = sum(c + t for c, t in zip(ctx, new) if t)
    pairs = sum(t * (prefix + c) + t * (t + 1) // 2 for c, t in zip(ctx, new))
    return dict(bytes=4 * (prefix + held) * kv * d + 4 * sum(new) * hq * d, flops=4 * pairs * hq * d)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "tables":
        return None
    if case["op"] == "rope":
        t, hq, kv, d, r = case["tokens"], case["heads"], case["kv"], case["dim"], case["rot"]
        turn = torch.polar(torch.full((t, r // 2), s["mag"], dtype=torch.float64, device=DEV),
                           s["positions"].double()[:, None] * s["freq"])

        def rotate(x, heads):
            x = x.double().reshape(t, heads, d).clone()
            head = x[:, :, :r]
            pair = head.reshape(t, heads, r // 2, 2) if case["inter"] else head.reshape(t, heads, 2, r // 2).transpose(2, 3)
            pair = torch.view_as_real(torch.view_as_complex(pair.contiguous()) * turn[:, None])
            x[:, :, :r] = (pair if case["inter"] else pair.transpose(2, 3)).reshape(t, heads, r)
            return x

        k, v = s["kc"].double(), s["vc"].double()
        flat_k, flat_v = k.transpose(1, 2).reshape(-1, kv, d), v.transpose(1, 2).reshape(-1, kv, d)
        keep = torch.nonzero(s["slots"] >= 0)[:, 0]
        flat_k[s["slots"][keep].long()] = rotate(s["k"], kv)[keep]
        flat_v[s["slots"][keep].long()] = s["v"].double().reshape(t, kv, d)[keep]
        back = (k.shape[0], k.shape[2], kv, d)
        return dict(q=rotate(s["q"], hq).reshape(t, hq * d), k=flat_k.reshape(back).transpose(1, 2).contiguous(),
                    v=flat_v.reshape(back).transpose(1, 2).contiguous())
    # attention: each request by itself, over its prefix and own tokens in one row of scores
    ctx, new = _lengths(case)
    hq, kv, d, size, prefix = case["heads"], case["kv"], case["dim"], case["block"], case["prefix"]
    out = torch.zeros(s["out"].shape, dtype=torch.float64, device=DEV)
    at = 0
    for b in range(case["requests"]):
        if not new[b]:
            continue
        own_blocks = s["table"][b, :_blocks(ctx[b] + new[b], size)].long()

        def laid(cache):
            parts = [cache[x].transpose(1, 2).reshape(-1, kv, d)[:m]
                     for x, m in ((s["prefix_table"].long(), prefix), (own_blocks, ctx[b] + new[b]))]
            return torch.cat(parts).double()

        k, v = laid(s["kc"]), laid(s["vc"])
        q = s["q"][at:at + new[b]].double().reshape(new[b], kv, hq // kv, d)
        score = torch.einsum("tkgd,nkd->tkgn", q, k) * s["scale"]
        place = torch.arange(k.shape[0], device=DEV)
        last = prefix + ctx[b] + torch.arange(new[b], device=DEV)
        score = score.masked_fill((place[None, :] > last[:, None])[:, None, None, :], -math.inf)
        out[at:at + new[b]] = torch.einsum("tkgn,nkd->tkgd", torch.softmax(score, -1), v).reshape(new[b], hq * d)
        at += new[b]
    return out

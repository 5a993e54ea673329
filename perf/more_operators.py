"""The decode layer's products on 8-bit weights, as cases that can be timed and checked.

Three operators carry a layer whose weights are e4m3 numbers with one 32-bit scale for each block of 128 x 128, and
whose activations are e4m3 numbers with one scale for each 128 values of a row:
  norm     the residual's addition, a root-mean-square norm with gains, and its output in 8 bits with scales
  linear   y = [r +] x W^T from rows and weights in 8 bits
  experts  the routed and shared SwiGLU experts of a batch on 8-bit weights, with the weighted combine
Each has a plain form in elementary torch operations and the library's call. The sizes of the ordinary cases are the
decode layer's own: hidden size 7168, an input projection of 12288 columns, an out-projection from 8192, experts of
2048 (256 on each GPU of a tensor-parallel group of eight), 384 of them, 8 for each token, and one shared.
"""
import math

import torch

own = False
DEV = "cuda"
E4M3 = torch.float8_e4m3fn
TOP = 448.0  # the largest e4m3 number
_kept = {}


def listed():
    return [
        # the latency case: one user's token between two blocks of the layer, with the residual stream kept
        dict(op="norm", name="norm, one token", rows=1, width=7168, residual=True, normed=False, gains=True),
        # a full decode batch before the experts: the router reads the normed row in 16 bits as well
        dict(op="norm", name="norm, 64 tokens, 16-bit output too", rows=64, width=7168, residual=True, normed=True, gains=True),
        # the rows of a prompt
        dict(op="norm", name="norm, prompt of 8192", rows=8192, width=7168, residual=True, normed=False, gains=True),
        # one user's token in the largest projection: weight reads alone
        dict(op="linear", name="linear, input projection, one token", rows=1, n=12288, k=7168, residual=False),
        # the smallest projection that is measured anywhere here: latency counts
        dict(op="linear", name="linear, 4096 x 4096, two tokens", rows=2, n=4096, k=4096, residual=False),
        # a middle batch in the out-projection, which adds the residual
        dict(op="linear", name="linear, out-projection, 16 tokens", rows=16, n=7168, k=8192, residual=True),
        # the full decode batch
        dict(op="linear", name="linear, input projection, 64 tokens", rows=64, n=12288, k=7168, residual=False),
        # nothing fits a tile: rows, columns and the last block of 128 are all ragged
        dict(op="linear", name="linear, ragged, 333 rows", rows=333, n=1000, k=2064, residual=True),
        # a prompt in one piece: arithmetic alone
        dict(op="linear", name="linear, input projection, prompt of 4096", rows=4096, n=12288, k=7168, residual=False),
        # one user's token on one GPU of a tensor-parallel group
        dict(op="experts", name="experts, one token, shard", rows=1, experts=384, top=8, hidden=7168, inner=256, shared=True),
        # eight users, whole experts
        dict(op="experts", name="experts, 8 tokens, 32 experts", rows=8, experts=32, top=8, hidden=7168, inner=2048, shared=True),
        # the full decode batch on one GPU of a tensor-parallel group: most experts are read
        dict(op="experts", name="experts, 64 tokens, shard", rows=64, experts=384, top=8, hidden=7168, inner=256, shared=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "linear", "linear", "experts"])
    if op == "norm":
        width = 16 * _log(rng, 4, 1024)
        return dict(op=op, rows=_log(rng, 1, min(8192, 8192 * 7168 // width)), width=width, residual=rng.random() < 0.7,
                    normed=rng.random() < 0.4, gains=rng.random() < 0.8)
    if op == "linear":
        n, k = _log(rng, 64, 16384), 16 * _log(rng, 8, 1024)
        # decode batches as often as prompts
        rows = _log(rng, 1, 64) if rng.random() < 0.6 else _log(rng, 65, max(66, min(4096, 4096 * 12288 * 7168 // (n * k))))
        return dict(op=op, rows=rows, n=n, k=k, residual=rng.random() < 0.5)
    hidden, inner = 128 * _log(rng, 2, 56), 128 * _log(rng, 1, 16)
    one = hidden * inner
    experts = _log(rng, 8, max(9, min(384, 384 * 7168 * 256 // one)))
    top = rng.choice([1, 2, 4, 6, 8])
    return dict(op=op, rows=_log(rng, 1, max(1, min(64, 512 * 7168 * 256 // (one * top)))), experts=experts, top=top,
                hidden=hidden, inner=inner, shared=rng.random() < 0.7)


def _gen(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _normal(g, *shape):
    return torch.randn(*shape, device=DEV, generator=g)


def _activations(g, rows, width):
    """Rows as a layer's stream holds them: channels of very different sizes, a few of them far larger."""
    channel = torch.exp(0.5 * _normal(g, width))
    channel[torch.randint(0, width, (1 + width // 500,), device=DEV, generator=g)] *= 20.0
    return _normal(g, rows, width) * channel


def _in_groups(x):
    """[..., width] as [..., groups, 128], zeros behind the last value."""
    width = x.shape[-1]
    return torch.nn.functional.pad(x, (0, -width % 128)).unflatten(-1, (-1, 128))


def _rows_in_8_bits(y):
    """A row's groups of 128 by their largest value: (e4m3 values, scales). A group of zeros has scale 0."""
    grouped = _in_groups(y)
    most = grouped.abs().amax(-1)
    up = torch.where(most > 0, TOP / most, 0.0)
    q = (grouped * up.unsqueeze(-1)).flatten(-2)[..., :y.shape[-1]].to(E4M3)
    return q.contiguous(), most / TOP


def _weights(g, *shape, scale):
    """Weights [..., n, k] by blocks of 128 x 128: (e4m3 values, scales)."""
    w = _normal(g, *shape) * scale
    n, k = shape[-2:]
    b = torch.nn.functional.pad(w, (0, -k % 128, 0, -n % 128)).unflatten(-1, (-1, 128)).unflatten(-3, (-1, 128))
    most = b.abs().amax((-1, -3), keepdim=True)
    q = (b * (TOP / most.clamp(min=1e-30))).flatten(-4, -3).flatten(-2)[..., :n, :k].to(E4M3)
    return q.contiguous(), (most / TOP).squeeze(-1).squeeze(-2).contiguous()


def prepare(case, seed):
    g = _gen(seed)
    s = dict(case=case)
    if case["op"] == "norm":
        m, width = case["rows"], case["width"]
        s["x"] = _activations(g, m, width).to(torch.bfloat16)
        s["residual"] = (3.0 * _activations(g, m, width)).to(torch.bfloat16) if case["residual"] else None
        s["gains"] = (1.0 + 0.3 * _normal(g, width)).to(torch.bfloat16) if case["gains"] else None
        s["q"] = torch.empty((m, width), dtype=E4M3, device=DEV)
        s["scale"] = torch.empty((m, -(-width // 128)), dtype=torch.float32, device=DEV)
        s["total"] = torch.empty_like(s["x"]) if case["residual"] else None
        s["y"] = torch.empty_like(s["x"]) if case["normed"] else None
    elif case["op"] == "linear":
        m, n, k = case["rows"], case["n"], case["k"]
        s["x"], s["xs"] = _rows_in_8_bits(_activations(g, m, k))
        s["w"], s["ws"] = _weights(g, n, k, scale=k ** -0.5)
        s["residual"] = _normal(g, m, n).to(torch.bfloat16) if case["residual"] else None
        s["y"] = torch.empty((m, n), dtype=torch.bfloat16, device=DEV)
    else:
        m, e, h, i = case["rows"], case["experts"], case["hidden"], case["inner"]
        s["x"], s["xs"] = _rows_in_8_bits(_normal(g, m, h))
        # every token has its own few experts, with weights that sum to one
        best = torch.sigmoid(_normal(g, m, e)).topk(min(case["top"], e), dim=-1)
        s["idx"], s["weight"] = best.indices.to(torch.int32), best.values / best.values.sum(-1, keepdim=True)
        s["gate"], s["up"] = _weights(g, e, i, h, scale=h ** -0.5), _weights(g, e, i, h, scale=h ** -0.5)
        s["down"] = _weights(g, e, h, i, scale=i ** -0.5)
        s["shared"] = None
        if case["shared"]:
            s["shared"] = (_weights(g, i, h, scale=h ** -0.5), _weights(g, i, h, scale=h ** -0.5),
                           _weights(g, h, i, scale=i ** -0.5))
        s["residual"] = _normal(g, m, h).to(torch.bfloat16)
        s["out"] = torch.empty((m, h), dtype=torch.bfloat16, device=DEV)
    if own:
        # the handle and the descriptors of long-lived buffers that a user's program keeps
        import moe_layers_gb300 as ml
        if "handle" not in _kept:
            _kept["handle"] = ml.Handle(0)
        s["h"] = _kept["handle"]
        if case["op"] == "norm":
            s["rows"] = ml.Fp8Rows(s["q"], s["scale"])
        else:
            s["rows"] = ml.Fp8Rows(s["x"], s["xs"])
        if case["op"] == "linear":
            s["weights"] = ml.Fp8Weight(s["w"], s["ws"])
        if case["op"] == "experts":
            shared = [None] * 3 if s["shared"] is None else [ml.Fp8Weight(*w) for w in s["shared"]]
            s["weights"] = ml.MoeFp8Weights(ml.Fp8Weight(*s["gate"]), ml.Fp8Weight(*s["up"]), ml.Fp8Weight(*s["down"]),
                                            *shared)
    return s


def run(s):
    case = s["case"]
    if case["op"] == "norm":
        return _run_norm(s)
    if case["op"] == "linear":
        return _run_linear(s)
    return _run_experts(s)


def _run_norm(s):
    if own:
        import moe_layers_gb300 as ml
        ml.dec_rmsnorm_quant(s["h"], s["x"], s["gains"], residual=s["residual"], eps=1e-6, total=s["total"], y=s["y"],
                             out=s["rows"])
    else:
        a = s["x"]
        if s["residual"] is not None:
            # the stream is kept in 16 bits, and what is normed is what is kept
            a = (a.float() + s["residual"].float()).to(torch.bfloat16)
            s["total"].copy_(a)
        y = a.float()
        if s["gains"] is not None:
            mean = y.double().square().mean(-1, keepdim=True)
            y = y * torch.rsqrt(mean + 1e-6).float() * s["gains"].float()
        if s["y"] is not None:
            s["y"].copy_(y)
        q, scale = _rows_in_8_bits(y)
        s["q"].copy_(q)
        s["scale"].copy_(scale)
    return {name: s[name] for name in ("q", "scale", "total", "y") if s[name] is not None}


def _values(q, scale):
    """Rows in 8 bits as what they stand for, in 32 bits."""
    return (_in_groups(q.float()) * scale.unsqueeze(-1)).flatten(-2)[..., :q.shape[-1]]


def _weight_values(q, scale):
    """The same of weights [..., n, k] with scales [..., n / 128, k / 128]."""
    n, k = q.shape[-2:]
    return q.float() * scale.repeat_interleave(128, -2)[..., :n, :].repeat_interleave(128, -1)[..., :k]


def _run_linear(s):
    if own:
        import moe_layers_gb300 as ml
        ml.dec_linear_fp8(s["h"], s["rows"], s["weights"], residual=s["residual"], y=s["y"])
    else:
        y = torch.matmul(_values(s["x"], s["xs"]), _weight_values(s["w"], s["ws"]).t())
        if s["residual"] is not None:
            y = y + s["residual"].float()
        s["y"].copy_(y)
    return s["y"]


def _run_experts(s):
    if own:
        import moe_layers_gb300 as ml
        ml.moe_experts_fp8(s["h"], s["rows"], s["idx"], s["weight"], s["weights"], residual=s["residual"], out=s["out"])
        return s["out"]
    x = _values(s["x"], s["xs"])
    m, top = s["idx"].shape
    at = s["idx"].reshape(-1).long()

    def expert(x, gate, up, down):
        """[n, width] through weights [n, ...] or, with one set for all, [1, ...]."""
        def times(x, w):
            return torch.matmul(x.unsqueeze(-2) if w.shape[0] > 1 else x, w.transpose(-1, -2)).reshape(x.shape[0], -1)
        z = times(x, gate)
        inner = z / (1.0 + torch.exp(-z)) * times(x, up)
        return times(_values(*_rows_in_8_bits(inner)), down)

    chosen = [_weight_values(q[at], scale[at]) for q, scale in (s["gate"], s["up"], s["down"])]
    y = expert(x.repeat_interleave(top, 0), *chosen)
    y = (y.reshape(m, top, -1) * s["weight"].unsqueeze(-1)).sum(1)
    if s["shared"] is not None:
        y = y + expert(x, *(_weight_values(q, scale).unsqueeze(0) for q, scale in s["shared"]))
    s["out"].copy_(y + s["residual"].float())
    return s["out"]


def work(case):
    m = case["rows"]
    if case["op"] == "norm":
        width, kept = case["width"], 2 if case["residual"] else 0
        # a residual is one more input and its sum one more output
        return dict(bytes=m * width * (2 + 2 * kept + 1 + (2 if case["normed"] else 0)) + 4 * m * -(-width // 128)
                    + (2 * width if case["gains"] else 0), flops=6 * m * width)
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        blocks = -(-k // 128)
        return dict(bytes=n * k + 4 * -(-n // 128) * blocks + m * (k + 4 * blocks) + m * n * (4 if case["residual"] else 2),
                    flops=2 * m * n * k)
    e, top, h, i = case["experts"], min(case["top"], case["experts"]), case["hidden"], case["inner"]
    # experts that at least one token of m chooses, in the mean
    read = e * (1.0 - (1.0 - top / e) ** m) + (1 if case["shared"] else 0)
    one = 3 * h * i * (1 + 4 / 128 ** 2)
    return dict(bytes=int(read * one) + m * (h + 4 * h // 128 + 8 * top + 4 * h),
                flops=6 * h * i * m * (top + (1 if case["shared"] else 0)))


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        a = s["x"].double()
        if s["residual"] is not None:
            a = (a + s["residual"].double())
        kept = a.to(torch.bfloat16).double()
        y = kept
        if s["gains"] is not None:
            y = kept / torch.sqrt((kept * kept).sum(-1, keepdim=True) / case["width"] + 1e-6) * s["gains"].double()
        scale = torch.stack([part.abs().amax(-1) for part in y.split(128, -1)], -1) / TOP
        spread = torch.stack([scale[:, j // 128] for j in range(0, case["width"], 16)], -1)
        q = y.reshape(case["rows"], -1, 16) / spread.clamp(min=1e-300).unsqueeze(-1)
        found = dict(q=q.reshape(y.shape), scale=scale)
        if s["residual"] is not None:
            found["total"] = a
        if case["normed"]:
            found["y"] = y
        return found

    def whole(q, scale):
        v = q.double()
        for i in range(scale.shape[-2]):
            for j in range(scale.shape[-1]):
                v[128 * i:128 * (i + 1), 128 * j:128 * (j + 1)] *= scale[i, j].double()
        return v

    def wide(q, scale):
        """The same for rows: one scale for each 128 values."""
        v = q.double()
        for j in range(scale.shape[-1]):
            v[:, 128 * j:128 * (j + 1)] *= scale[:, j:j + 1].double()
        return v

    x = wide(s["x"], s["xs"])
    if case["op"] == "linear":
        y = x @ whole(s["w"], s["ws"]).t()
        return y if s["residual"] is None else y + s["residual"].double()
    out = s["residual"].double()

    def through(rows, gate, up, down):
        z = rows @ whole(*gate).t()
        inner = z * torch.sigmoid(z) * (rows @ whole(*up).t())
        scale = torch.stack([part.abs().amax(-1) for part in inner.split(128, -1)], -1) / TOP
        by = scale.repeat_interleave(128, -1)
        # the inner row is an 8-bit row by the operator's definition
        return ((inner / by.clamp(min=1e-300)).to(E4M3).double() * by) @ whole(*down).t()

    for e in sorted(set(s["idx"].reshape(-1).tolist())):
        token, place = torch.nonzero(s["idx"] == e, as_tuple=True)
        y = through(x[token], *((q[e], scale[e]) for q, scale in (s["gate"], s["up"], s["down"])))
        out[token] += s["weight"][token, place].double().unsqueeze(-1) * y
    if s["shared"] is not None:
        out += through(x, *s["shared"])
    return out

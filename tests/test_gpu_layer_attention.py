"""The decode layer with attention (decode_layer_attention): steps of a small
batch from tables to hidden state against the oracle's layer, stage by stage."""
import numpy as np
import pytest

import oracle
import synth
from _util import SEED, assert_bf16_close, dev_bf16, dev_f32, host_bits

pytestmark = pytest.mark.gpu

H, E, I, K = 256, 16, 128, 4


@pytest.fixture(scope="module")
def h():
    import torch
    import moe_layers_gb300 as M
    assert torch.cuda.is_available()
    M.build()
    with M.Handle(0) as hd:
        yield hd
        assert hd.check_device_error() == M.DEC_OK


def i32(a):
    import torch
    return torch.tensor(np.ascontiguousarray(a, dtype=np.int32), device="cuda")


class Layer:
    def __init__(self, heads, kv, d, rest, shared):
        import moe_layers_gb300 as ML
        self.heads, self.kv, self.d = heads, kv, d
        n_in, k_out = (heads + 2 * kv) * d + rest, heads * d
        mk = lambda tid, *shape, s=0.05: synth.bf16(int(np.prod(shape)), SEED, 7000 + tid, 0, s).reshape(shape)  # noqa: E731
        one = (np.asarray(1.0, np.float32).view(np.uint32) >> 16).astype(np.uint16)
        self.g1, self.g2 = np.full(H, one), np.full(H, one)
        self.W_in, self.W_o = mk(0, n_in, H, s=0.1), mk(1, H, k_out)
        self.Wr = synth.f32(E * H, SEED, 7002, 0, 0.05).reshape(E, H)
        self.bank = [mk(3, E, I, H), mk(4, E, I, H), mk(5, E, H, I)]
        self.shared = [mk(6, I, H), mk(7, I, H), mk(8, H, I)] if shared else None
        dev = lambda a: dev_bf16(a, a.shape)  # noqa: E731
        sh = [dev(a) for a in self.shared] if shared else [None] * 3
        self.w = ML.LayerWeights(gamma1=dev(self.g1), W_in=dev(self.W_in), W_o=dev(self.W_o), gamma2=dev(self.g2),
                                 W_r=dev_f32(self.Wr), Wg=dev(self.bank[0]), Wu=dev(self.bank[1]), Wd=dev(self.bank[2]),
                                 Wg_s=sh[0], Wu_s=sh[1], Wd_s=sh[2], k=K, k_out=k_out)


@pytest.mark.parametrize("shared", [True, False])
@pytest.mark.parametrize("heads,kv,d,rest", [(4, 2, 64, 8), (2, 1, 128, 0), (6, 6, 64, 64)])
@pytest.mark.parametrize("news,prefix,pad", [([[1], [1]], 0, 0), ([[1, 1], [1, 1]], 20, 0), ([[3, 1], [1, 1]], 37, 1),
                                             ([[2, 0, 5, 1], [1, 1, 1, 1]], 0, 2), ([[16, 20, 9, 11], [1] * 4], 65, 3)])
def test_steps(h, heads, kv, d, rest, news, prefix, pad, shared):
    import torch
    import moe_layers_gb300 as ML
    L = Layer(heads, kv, d, rest, shared)
    size, blocks, n = 16, 40, len(news[0])
    rng = np.random.default_rng(len(news[0]) + prefix)
    kc, vc = (torch.tensor(rng.standard_normal((blocks, kv, size, d)), dtype=torch.float32).to(torch.bfloat16).cuda()
              for _ in range(2))
    ids = [int(x) for x in rng.permutation(blocks)]
    prefix_table = ids[:-(-prefix // size)]
    free = ids[len(prefix_table):]
    table, ctx, count = np.full((n, 4), -1), np.zeros(n, int), len(free)
    d_table, d_free = i32(table), i32(free)
    rope, freq = ML.Rope(h, 32, base=10000.0), oracle.rope_frequencies(32, 10000.0)
    for step, new in enumerate(news):
        M = sum(new) + pad
        tables = ML.dec_batch_tables(h, i32(ctx), i32(new), d_free, i32([count]), d_table, size, rows=M,
                                     position_offset=prefix)
        batch = ML.Batch(tables.row_start, tables.own_len, d_table, max_new=max(new),
                         prefix_table=i32(prefix_table) if prefix else None, prefix_len=prefix)
        att = ML.LayerAttention(heads, d ** -0.5, ML.KvCache(kc, vc), batch, tables.positions, tables.slots, rope)
        hb = synth.bf16(M * H, SEED, 7100 + step, 0, 1.0).reshape(M, H)
        hidden = dev_bf16(hb, (M, H))
        k0, v0 = host_bits(kc), host_bits(vc)
        tr = ML.decode_layer_attention(h, L.w, att, hidden, trace=True)
        torch.cuda.synchronize()
        want = oracle.batch_tables(ctx, new, free, count, table, size, prefix, M)
        table, ctx, count = want["table"], want["own_len"], int(want["left"][0])

        def core(y):
            y = y.reshape(M, -1)
            q, k, v = (y[:, a * d:b * d].reshape(M, b - a, d) for a, b in ((0, heads), (heads, heads + kv),
                                                                          (heads + kv, heads + 2 * kv)))
            q, k = (oracle.round_bf16(oracle.rope(x, want["positions"], freq)) for x in (q, k))
            ck, cv = oracle.as_f64(k0).copy(), oracle.as_f64(v0).copy()
            for t in range(sum(new)):
                b, o = want["slots"][t] // size, want["slots"][t] % size
                ck[b, :, o], cv[b, :, o] = k[t], v[t]
            core.cache = ck, cv
            out, _, _ = oracle.attention(q, ck, cv, want["row_start"], ctx, table, d ** -0.5, prefix_table, prefix)
            return oracle.round_bf16(np.nan_to_num(out)).reshape(M, heads * d)

        expert = lambda e: tuple(oracle.bf16_to_f64(b[e]) for b in L.bank)  # noqa: E731
        ref = oracle.decode_layer(hb, L.g1, L.W_in, L.W_o, L.g2, L.Wr, K, expert, L.shared, k_out=heads * d, core=core)
        # against the sum before its storage rounding: the rule allows the stored value one
        # half-ulp, and a reference that had been rounded as well could lie another one off
        assert_bf16_close(host_bits(tr["h1"]), ref["unrounded"]["h1"], "h1")
        # the cache: the step's tokens to a rounding of the projection and of the turn, the rest untouched
        for got, exp, before in zip((host_bits(kc), host_bits(vc)), core.cache, (k0, v0)):
            touched = np.zeros(got.shape, bool)
            for t in range(sum(new)):
                touched[want["slots"][t] // size, :, want["slots"][t] % size] = True
            assert np.array_equal(got[~touched], before[~touched])
            assert np.all(np.abs(oracle.as_f64(got) - exp)[touched] <= 2.0 ** -6 * np.abs(exp)[touched] + 2e-2)
        # rows of no request pass without attention
        assert np.array_equal(host_bits(tr["h1"])[sum(new):], hb[sum(new):])
        # the MoE block on the stored h1 with the routing it chose
        h1 = oracle.as_f64(host_bits(tr["h1"]))
        b = oracle.round_bf16(oracle.rmsnorm(h1, L.g2))
        out = h1 + oracle.moe(b, tr["idx"].cpu().numpy(), tr["w"].cpu().numpy().astype(np.float64), expert, L.shared)
        assert_bf16_close(host_bits(hidden), out, "out")


def test_layer_attention_under_a_graph(h):
    """A captured step replayed with the tables' own outputs as the next lengths gives the eager steps' bits."""
    import torch
    import moe_layers_gb300 as ML
    heads, kv, d, size, n = 4, 2, 64, 16, 3
    L = Layer(heads, kv, d, 0, True)
    rng = np.random.default_rng(1)
    init = torch.tensor(rng.standard_normal((2, 20, kv, size, d)), dtype=torch.float32).to(torch.bfloat16).cuda()
    x0 = dev_bf16(synth.bf16(n * H, SEED, 7200, 0, 1.0).reshape(n, H), (n, H))
    rope = ML.Rope(h, 64)

    def run(graph):
        pool = init.clone()
        ctx, new, free, count = i32([0, 3, 15]), i32([1, 1, 1]), i32(range(3, 20)), i32([17, 0])
        table = i32([[-1] * 4, [0] + [-1] * 3, [1] + [-1] * 3])
        out = ML.StepTables(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), ctx,
                            torch.zeros(n, dtype=torch.int32, device="cuda"),
                            torch.zeros(n, dtype=torch.int32, device="cuda"), count)
        batch = ML.Batch(out.row_start, out.own_len, table)
        att = ML.LayerAttention(heads, 0.125, ML.KvCache(pool[0], pool[1]), batch, out.positions, out.slots, rope)
        x = x0.clone()
        ws = torch.zeros(ML.decode_layer_attention_workspace_size(h, L.w, att, n), dtype=torch.uint8, device="cuda")

        def step():
            ML.dec_batch_tables(h, ctx, new, free, count, table, size, out)
            ML.decode_layer_attention(h, L.w, att, x, ws=ws)

        if graph:
            g = torch.cuda.CUDAGraph()
            side = torch.cuda.Stream()
            side.wait_stream(torch.cuda.current_stream())
            with torch.cuda.graph(g, stream=side):
                step()
            for _ in range(20):
                g.replay()
        else:
            for _ in range(20):
                step()
        torch.cuda.synchronize()
        return host_bits(x), host_bits(pool), ctx.cpu().numpy(), table.cpu().numpy()

    for a, b in zip(run(False), run(True)):
        assert np.array_equal(a, b)


def test_layer_attention_workspace_and_captures(h):
    """A capture that would have to make the workspace is refused; one made before keeps it, whatever other
    shapes run in between."""
    import torch
    import moe_layers_gb300 as ML
    L = Layer(4, 2, 64, 0, True)
    pool = torch.zeros((40, 2, 16, 64), dtype=torch.bfloat16, device="cuda")

    def layer(M):
        step = ML.StepTables.empty(M, M)
        table = torch.full((M, 2), -1, dtype=torch.int32, device="cuda")
        ML.dec_batch_tables(h, i32([0] * M), i32([1] * M), i32(range(40)), i32([40]), table, 16, step)
        batch = ML.Batch(step.row_start, step.own_len, table)
        return ML.LayerAttention(4, 0.125, ML.KvCache(pool, pool.clone()), batch, step.positions, step.slots)

    x0 = {M: dev_bf16(synth.bf16(M * H, SEED, 7300 + M, 0, 1.0).reshape(M, H), (M, H)) for M in (3, 8, 33)}
    att = {M: layer(M) for M in x0}
    s = torch.cuda.Stream()
    x = x0[3].clone()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            ML.decode_layer_attention(h, L.w, att[3], x)
    torch.cuda.synchronize()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        want = x0[3].clone()
        ML.decode_layer_attention(h, L.w, att[3], want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        ML.decode_layer_attention(h, L.w, att[3], x)
    for M in (8, 33, 8):
        with torch.cuda.stream(s):
            ML.decode_layer_attention(h, L.w, att[M], x0[M].clone())
        torch.cuda.synchronize()
        torch.cuda.empty_cache()
        x.copy_(x0[3])
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(x.view(torch.int16), want.view(torch.int16))


def test_layer_attention_refuses(h):
    import torch
    import moe_layers_gb300 as ML
    L = Layer(4, 2, 64, 0, True)
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    batch = ML.Batch(i32([0, 1]), i32([1]), i32([[0]]))
    one = i32([0])
    x = torch.zeros((1, H), dtype=torch.bfloat16, device="cuda")

    def call(heads=4, scale=0.125, cache=pool, rope=None):
        ML.decode_layer_attention(h, L.w, ML.LayerAttention(heads, scale, ML.KvCache(cache, cache), batch, one, one, rope), x)

    for bad in (dict(heads=3), dict(heads=2), dict(scale=0.0), dict(scale=float("inf")),
                dict(cache=torch.zeros((4, 4, 16, 64), dtype=torch.bfloat16, device="cuda")),
                dict(rope=ML.Rope(h, 128))):
        with pytest.raises(ML.DecodeError) as e:
            call(**bad)
        assert e.value.status == ML.DEC_ERR_INVALID_ARG
    with pytest.raises(ValueError):
        ML.decode_layer_attention(h, L.w, ML.LayerAttention(4, 0.125, ML.KvCache(pool, pool), batch, one, one),
                                  torch.zeros((2, H), dtype=torch.bfloat16, device="cuda"))
    torch.cuda.synchronize()


def test_layer_attention_refuses_another_width(h):
    """The weights' H values of each row are read and written: a narrower or wider hidden state is refused."""
    import torch
    import moe_layers_gb300 as ML
    L = Layer(4, 2, 64, 0, True)
    pool = torch.zeros((4, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    batch = ML.Batch(i32([0, 1]), i32([1]), i32([[0]]))
    att = ML.LayerAttention(4, 0.125, ML.KvCache(pool, pool), batch, i32([0]), i32([0]))
    for width in (H - 8, H + 8, 8):
        x = torch.zeros((1, width), dtype=torch.bfloat16, device="cuda")
        with pytest.raises(ValueError):
            ML.decode_layer_attention(h, L.w, att, x)


@pytest.fixture(scope="module")
def wide():
    """The workload's projections (7168 -> 12288 -> 8192 -> 7168, 64 + 16 + 16 heads of 128) before 16 experts."""
    import torch
    import moe_layers_gb300 as ML
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    width, n_in, k_out, experts, inner = 7168, 12288, 8192, 16, 2048

    def rand(*shape, s=0.02):
        return (torch.randn(*shape, device="cuda", generator=g) * s).to(torch.bfloat16)

    return ML.LayerWeights(gamma1=1 + rand(width, s=0.1), W_in=rand(n_in, width), W_o=rand(width, k_out),
                           gamma2=1 + rand(width, s=0.1),
                           W_r=torch.randn(experts, width, device="cuda", generator=g) * 0.01,
                           Wg=rand(experts, inner, width), Wu=rand(experts, inner, width), Wd=rand(experts, width, inner),
                           Wg_s=rand(inner, width), Wu_s=rand(inner, width), Wd_s=rand(width, inner), k=8, k_out=k_out)


@pytest.mark.parametrize("n,new,own,prefix,pad", [(1, 1, 777, 0, 0), (1, 1, 2000, 300, 0), (2, 1, 90, 0, 0), (4, 2, 500, 0, 0),
                                                  (1, 64, 1000, 0, 0), (60, 1, 70, 2048, 4), (7, 1, 33, 40, 2)])
@pytest.mark.parametrize("spare", [True, False])
def test_layer_attention_at_the_workloads_width(h, wide, n, new, own, prefix, pad, spare):
    """One step against float64: h1 by the formulas from the hidden state on, the rest as moe_layer gives it.
    Without spare blocks, new tokens that begin a block have no place and are not there."""
    import torch
    import moe_layers_gb300 as ML
    heads, kv, d, size, M = 64, 16, 128, 16, n * new + pad
    g = torch.Generator(device="cuda")
    g.manual_seed(M + prefix)
    lens = [own + new + 3 * b for b in range(n)]  # with this step's rows
    held, ahead = [-(-x // size) for x in lens], -(-prefix // size)
    blocks = sum(held) + ahead + n * 5  # a request begins five blocks at most
    pool = torch.randn((2, blocks, kv, size, d), device="cuda", generator=g).to(torch.bfloat16)
    order = torch.randperm(blocks, device="cuda", generator=g).to(torch.int32)
    table = torch.full((n, max(held)), -1, dtype=torch.int32, device="cuda")
    at = ahead
    for b in range(n):
        table[b, :held[b]] = order[at:at + held[b]]
        at += held[b]
    step = ML.dec_batch_tables(h, i32([x - new for x in lens]), i32([new] * n), order[at:].contiguous(),
                               i32([n * 5 if spare else 0]), table, size, rows=M, position_offset=prefix)
    batch = ML.Batch(step.row_start, step.own_len, table, max_new=new,
                     prefix_table=order[:ahead].contiguous() if prefix else None, prefix_len=prefix)
    rope = ML.Rope(h, d, base=500000.0)
    att = ML.LayerAttention(heads, d ** -0.5, ML.KvCache(pool[0], pool[1]), batch, step.positions, step.slots, rope)
    x = torch.randn((M, 7168), device="cuda", generator=g).to(torch.bfloat16)
    old, hidden = pool.clone(), x.clone()
    trace = ML.decode_layer_attention(h, wide, att, hidden, trace=True)
    torch.cuda.synchronize()

    stored = lambda t: t.to(torch.bfloat16).double()  # noqa: E731
    a = x.double()
    a = stored(a * torch.rsqrt((a * a).mean(-1, keepdim=True) + wide.eps) * wide.gamma1.double())
    y = stored(a @ wide.W_in.double().T)
    q, k, v = (t.reshape(M, -1, d) for t in (y[:, :heads * d], y[:, heads * d:(heads + kv) * d], y[:, (heads + kv) * d:]))
    angle = step.positions.double()[:, None] * 500000.0 ** (-2.0 * torch.arange(d // 2, device="cuda").double() / d)
    c, s = torch.cos(angle)[:, None], torch.sin(angle)[:, None]
    turn = lambda t: stored(torch.cat((t[..., :64] * c - t[..., 64:] * s, t[..., 64:] * c + t[..., :64] * s), -1))  # noqa: E731
    q, k = turn(q), turn(k)
    core = torch.zeros((M, heads, d), dtype=torch.float64, device="cuda")
    for b in range(n):
        keys = [torch.cat([old[i, t.long()].transpose(1, 2).reshape(-1, kv, d)[:m]
                           for t, m in ((order[:ahead], prefix), (table[b, :held[b]], lens[b] - new))]).double() for i in (0, 1)]
        rows = slice(b * new, (b + 1) * new)
        kk, vv = (torch.cat((t, mine[rows])) for t, mine in zip(keys, (k, v)))
        score = torch.einsum("tkgd,nkd->tkgn", q[rows].reshape(new, kv, heads // kv, d), kk) * d ** -0.5
        place = torch.arange(kk.shape[0], device="cuda")
        hidden_from = prefix + lens[b] - new + torch.arange(new, device="cuda")
        gone = (place >= prefix) & (table[b, ((place - prefix) // size).clamp(min=0)] < 0)  # in a block that is not there
        score = score.masked_fill(((place[None] > hidden_from[:, None]) | gone)[:, None, None], -torch.inf)
        core[rows] = torch.einsum("tkgn,nkd->tkgd", torch.softmax(score, -1), vv).reshape(new, heads, d)
    h1 = x.double() + stored(core.reshape(M, -1)) @ wide.W_o.double().T
    assert_bf16_close(host_bits(trace["h1"]), h1.cpu().numpy(), "h1")
    assert torch.equal(trace["h1"][n * new:], x[n * new:])  # rows of no request
    moe = ML.MoeWeights(W_r=wide.W_r, Wg=wide.Wg, Wu=wide.Wu, Wd=wide.Wd, Wg_s=wide.Wg_s, Wu_s=wide.Wu_s, Wd_s=wide.Wd_s,
                        gamma=wide.gamma2, k=wide.k)
    out, same = ML.moe_layer(h, moe, trace["h1"], residual=trace["h1"], trace=True)
    torch.cuda.synchronize()
    assert torch.equal(same["idx"], trace["idx"])
    assert_bf16_close(host_bits(hidden), out.double().cpu().numpy(), "out")


@pytest.mark.parametrize("M", [1, 2, 4, 40])
def test_two_layers_at_once(h, wide, M):
    """Steps of two batches on two streams through one handle, and two captured ones replayed at the same time:
    the bits of each alone."""
    import torch
    import moe_layers_gb300 as ML
    kv, d, size, streams = 16, 128, 16, [torch.cuda.Stream() for _ in range(2)]
    runs = []
    for i in range(2):
        g = torch.Generator(device="cuda")
        g.manual_seed(i)
        own = 300 + 50 * i
        pool = torch.randn((2, M * 25, kv, size, d), device="cuda", generator=g).to(torch.bfloat16)
        table = torch.arange(M * 25, device="cuda").to(torch.int32).reshape(M, 25)
        batch = ML.Batch(i32(range(M + 1)), i32([own] * M), table)
        slots = table[:, (own - 1) // size].contiguous() * size + (own - 1) % size
        att = ML.LayerAttention(64, d ** -0.5, ML.KvCache(pool[0], pool[1]), batch, i32([own - 1] * M), slots,
                                ML.Rope(h, 128))
        x0 = torch.randn((M, 7168), device="cuda", generator=g).to(torch.bfloat16)
        x, alone = x0.clone(), x0.clone()
        ws = torch.zeros(ML.decode_layer_attention_workspace_size(h, wide, att, M), dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        for _ in range(6):
            ML.decode_layer_attention(h, wide, att, alone, ws=ws)
        torch.cuda.synchronize()
        runs.append((att, x0, x, ws, alone))
    for _ in range(5):
        for att, x0, x, ws, alone in runs:
            x.copy_(x0)
        torch.cuda.synchronize()
        for _ in range(6):
            for s, (att, x0, x, ws, alone) in zip(streams, runs):
                ML.decode_layer_attention(h, wide, att, x, stream=s, ws=ws)
        torch.cuda.synchronize()
        assert all(torch.equal(x, alone) for att, x0, x, ws, alone in runs)
    graphs = [torch.cuda.CUDAGraph() for _ in runs]
    for g, (att, x0, x, ws, alone) in zip(graphs, runs):
        with torch.cuda.graph(g):
            for _ in range(6):
                ML.decode_layer_attention(h, wide, att, x, ws=ws)
    for _ in range(5):
        for att, x0, x, ws, alone in runs:
            x.copy_(x0)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, alone) for att, x0, x, ws, alone in runs)

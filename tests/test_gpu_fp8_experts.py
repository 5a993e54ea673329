"""The 8-bit experts where calls follow one another, choices are left out, and rows and weights hold what is not finite."""
import pytest
import torch

from _fp8 import assert_within, experts64, rand_rows
from test_gpu_fp8 import bits, choices, expert_weights, gen

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ml():
    import moe_layers_gb300 as M
    M.build()
    return M


@pytest.fixture()
def h(ml):
    with ml.Handle(0) as handle:
        yield handle


# ---------------------------------------------------------------------------- calls back to back
def routings(g, m, e, k):
    """Few problems after many and the other way round: even choices, all tokens on the same experts, most or all left out."""
    out = []
    for i in range(12):
        idx, w = choices(g, m, e, k)
        if i % 4 == 1:
            idx[:] = idx[0].clone()
        elif i % 4 == 2:
            idx[:, 1:] = -1
        elif i % 4 == 3 and i > 4:
            idx[:] = e
        out.append((idx, w))
    return out


@pytest.mark.parametrize("m,shared", [(1, True), (1, False), (4, True), (24, False), (64, True)])
def test_routing_that_changes_from_call_to_call(ml, h, m, shared):
    """The second product reads the routing before the first one has ended, at one address for all calls."""
    g = gen(40 + m)
    E, k, H, I = 40, 4, 512, 256
    banks, one, W = expert_weights(ml, g, E, H, I, shared)
    x = rand_rows(g, m, H)
    X = ml.Fp8Rows(*x)
    ways = routings(g, m, E, k)
    n = -(-m * k // 4) * 4  # the copying kernel takes whole 16 bytes
    held = torch.zeros(len(ways), 2, n, dtype=torch.int32, device="cuda")  # each call's ids and weights
    for i, (idx, w) in enumerate(ways):
        held[i, 0, :m * k], held[i, 1, :m * k] = idx.flatten(), w.flatten().view(torch.int32)
    now = torch.zeros(2, n, dtype=torch.int32, device="cuda")
    idx0, w0 = now[0, :m * k].view(m, k), now[1, :m * k].view(torch.float32).view(m, k)
    alone = []
    for idx, w in ways:
        alone.append(ml.moe_experts_fp8(h, X, idx, w, W))
        torch.cuda.synchronize()
        want, room = experts64(*x, idx, w, *banks, one)
        assert_within(alone[-1], want, room + 1e-300)
    ws = torch.empty(ml.moe_experts_fp8_workspace_size(h, W, m, k), dtype=torch.uint8, device="cuda")
    outs = torch.empty(len(ways), m, H, dtype=torch.bfloat16, device="cuda")
    stream = torch.cuda.Stream()

    def run():
        for i, _ in enumerate(ways):
            ml.test_delayed_copy(h, now, held[i], 0, stream=stream)
            ml.moe_experts_fp8(h, X, idx0, w0, W, out=outs[i], ws=ws, stream=stream)

    def check():
        torch.cuda.synchronize()
        for i, want in enumerate(alone):
            assert torch.equal(bits(outs[i]), bits(want)), i
        outs.zero_()
        torch.cuda.synchronize()

    torch.cuda.synchronize()
    for _ in range(5):
        run()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    for _ in range(5):
        graph.replay()
    check()
    assert h.check_device_error() == 0


# ---------------------------------------------------------------------------- choices left out
def replay_us(run):
    """A call in a replayed graph of ten, the quickest of seven replays."""
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        for _ in range(10):
            run()
    took = []
    for _ in range(7):
        a, b = (torch.cuda.Event(enable_timing=True) for _ in range(2))
        with torch.cuda.stream(stream):
            a.record()
            graph.replay()
            b.record()
        torch.cuda.synchronize()
        took.append(a.elapsed_time(b) * 100)
    return min(took)


@pytest.mark.parametrize("m", [1, 2])
def test_choices_left_out_stream_no_weights(ml, h, m):
    """One choice of sixteen is here, as on a rank that holds a part of the experts. An expert's weights (400 MB) pass in
    some 60 us, all sixteen's in a millisecond: twice the time of a call with that choice alone leaves room for noise."""
    E, k, H, I = 2, 16, 16384, 8192
    g = gen(m)

    def bank(*shape):
        q = torch.empty(*shape, dtype=torch.uint8, device="cuda").random_(0x20, 0x58, generator=g)
        return ml.Fp8Weight(q.view(torch.float8_e4m3fn), torch.full((*shape[:-2], shape[-2] // 128, shape[-1] // 128), 1e-4,
                                                                    device="cuda"))

    W = ml.MoeFp8Weights(bank(E, I, H), bank(E, I, H), bank(E, H, I))
    X = ml.Fp8Rows(*rand_rows(g, m, H))
    idx = torch.full((m, k), -1, dtype=torch.int32, device="cuda")
    idx[:, 5] = 1
    w = torch.rand(m, k, generator=g, device="cuda")
    one, w1 = idx[:, 5:6].contiguous(), w[:, 5:6].contiguous()
    out, out1 = (torch.empty(m, H, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    few = replay_us(lambda: ml.moe_experts_fp8(h, X, one, w1, W, out=out1))
    left_out = replay_us(lambda: ml.moe_experts_fp8(h, X, idx, w, W, out=out))
    assert torch.equal(bits(out), bits(out1))
    assert left_out < 2 * few, f"{left_out:.1f} us with fifteen choices left out, {few:.1f} us without them"


@pytest.mark.parametrize("shared", [False, True])
def test_one_token_s_choices_in_and_out(ml, h, shared):
    """Every pattern of four choices here or not."""
    g = gen(17)
    E, k, H, I = 6, 4, 256, 128
    banks, one, W = expert_weights(ml, g, E, H, I, shared)
    x = rand_rows(g, 1, H)
    r = torch.randn(1, H, generator=g, device="cuda").bfloat16()
    for pattern in range(16):
        idx, w = choices(g, 1, E, k)
        for j in range(k):
            if not pattern >> j & 1:
                idx[0, j] = (-1, E, -2 ** 31, 2 ** 31 - 1)[j]
                w[0, j] = float("nan")  # a weight that nothing takes
        out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W, residual=r)
        assert_within(out, *experts64(*x, idx, w.nan_to_num(), *banks, one, r))


# ---------------------------------------------------------------------------- rows
@pytest.mark.parametrize("m", [1, 2, 11, 64])
def test_strided_rows(ml, h, m):
    """Columns of wider rows, from a group's start on: values and scales with strides of their own."""
    g = gen(60 + m)
    E, k, H, I = 9, 3, 640, 256
    banks, one, W = expert_weights(ml, g, E, H, I, True)
    q, s = rand_rows(g, m, 2048)
    x = (q[:, 384:384 + H], s[:, 3:8])
    idx, w = choices(g, m, E, k)
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    assert_within(out, *experts64(*x, idx, w, *banks, one))
    dense = ml.moe_experts_fp8(h, ml.Fp8Rows(x[0].contiguous(), x[1].contiguous()), idx, w, W)
    assert torch.equal(bits(out), bits(dense))


@pytest.mark.parametrize("m", [1, 3, 40])
@pytest.mark.parametrize("what", ["value", "nan scale", "inf scale", "nan weight", "inf weight", "overflow"])
def test_what_is_not_finite_stays_with_its_token(ml, h, m, what):
    """The last token's row or routing weight; the others are as without it. An inner row past fp32's range counts as
    infinite, and a group that holds an infinity is not finite."""
    g = gen(70 + m)
    E, k, H, I = 5, 3, 384, 256
    banks, one, W = expert_weights(ml, g, E, H, I, True)
    q, s = rand_rows(g, m, H)
    idx, w = choices(g, m, E, k)
    before = ml.moe_experts_fp8(h, ml.Fp8Rows(q, s), idx, w, W)
    assert_within(before, *experts64(q, s, idx, w, *banks, one))
    q, s, w = q.clone(), s.clone(), w.clone()
    if what == "value":
        bits(q)[m - 1, 200] = 0x7F
    elif what == "nan weight":
        w[m - 1, 1] = float("nan")
    elif what == "inf weight":
        w[m - 1, 1] = float("inf")
    else:
        s[m - 1, 1] = {"nan scale": float("nan"), "inf scale": float("inf"), "overflow": 1e25}[what]
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(q, s), idx, w, W)
    assert torch.equal(bits(out[:m - 1]), bits(before[:m - 1]))
    assert not torch.isfinite(out[m - 1]).any()
    assert h.check_device_error() == 0

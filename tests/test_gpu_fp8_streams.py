"""The 8-bit operators on other streams, in captured graphs, with shared workspaces and at sizes past 32 bits."""
import pytest
import torch

from _fp8 import E4M3, assert_within, experts64, linear64, rand_rows, rand_weight, value_rows, value_weight
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


def some_linear(g, m, n=640, k=1040):
    return rand_rows(g, m, k), rand_weight(g, n, k)


@pytest.mark.parametrize("m", [1, 12, 64, 300])
def test_linear_captured_and_replayed_with_new_rows(ml, h, m):
    g = gen(m)
    (q, s), w = some_linear(g, m)
    y = torch.empty(m, 640, dtype=torch.bfloat16, device="cuda")
    x, W = ml.Fp8Rows(q, s), ml.Fp8Weight(*w)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        ml.dec_linear_fp8(h, x, W, y=y)  # its workspace
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        ml.dec_linear_fp8(h, x, W, y=y)
    for seed in range(3):
        q2, s2 = rand_rows(gen(100 + seed), m, 1040)
        q.copy_(q2)
        s.copy_(s2)
        y.zero_()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert_within(y, *linear64(q, s, *w))
    assert h.check_device_error() == 0


def test_layer_run_captured(ml, h):
    g = gen(7)
    m, H, I, E, k = 6, 512, 256, 12, 3
    x, r = (torch.randn(m, H, generator=g, device="cuda").bfloat16() for _ in range(2))
    gamma = torch.randn(H, generator=g, device="cuda").bfloat16()
    banks, one, W = expert_weights(ml, g, E, H, I, True)
    idx, wt = choices(g, m, E, k)
    rows, out = ml.Fp8Rows.empty(m, H), torch.empty_like(x)

    def run(stream=None):
        ml.dec_rmsnorm_quant(h, x, gamma, residual=r, out=rows, stream=stream)
        ml.moe_experts_fp8(h, rows, idx, wt, W, residual=r, out=out, stream=stream)

    run()
    torch.cuda.synchronize()
    want = out.clone()
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        run()
    out.zero_()
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(bits(out), bits(want))
    idx.copy_(choices(gen(8), m, E, k)[0])
    torch.cuda.synchronize()
    graph.replay()
    torch.cuda.synchronize()
    assert_within(out, *experts64(rows.q, rows.scale, idx, wt, *banks, one, r))


def padded(t):
    """(buffer of whole 16 bytes, a view of it with t's shape and values): what the copying hook takes."""
    flat = torch.zeros(-(-t.numel() // 16) * 16, dtype=t.dtype, device="cuda") if t.dtype != E4M3 else \
        torch.zeros(-(-t.numel() // 16) * 16, dtype=torch.uint8, device="cuda").view(E4M3)
    view = flat[:t.numel()].view(t.shape)
    view.copy_(t)
    return flat, view


@pytest.mark.parametrize("m", [1, 16, 40, 200])
def test_rows_that_a_slow_kernel_before_writes(ml, h, m):
    """The launch may start before the kernel ahead of it ends: only weights are read before that."""
    g = gen(m)
    (q, s), w = some_linear(g, m)
    (qf, _), (sf, _) = padded(q), padded(s)
    (qf0, q0), (sf0, s0) = padded(torch.zeros_like(q)), padded(torch.zeros_like(s))
    stream = torch.cuda.Stream()
    x, W = ml.Fp8Rows(q0, s0), ml.Fp8Weight(*w)
    torch.cuda.synchronize()
    ml.dec_linear_fp8(h, x, W, stream=stream)
    torch.cuda.synchronize()
    ml.test_delayed_copy(h, qf0, qf, 300_000, stream=stream)
    ml.test_delayed_copy(h, sf0, sf, 300_000, stream=stream)
    y = ml.dec_linear_fp8(h, x, W, stream=stream)
    torch.cuda.synchronize()
    assert_within(y, *linear64(q, s, *w))


def test_experts_after_a_slow_router(ml, h):
    g = gen(3)
    banks, one, W = expert_weights(ml, g, 10, 256, 128, True)
    for m in (1, 7):
        x = rand_rows(g, m, 256)
        idx, wt = choices(g, m, 10, 4)
        (if_, _), (wf, _) = padded(idx), padded(wt)
        (if0, idx0), (wf0, w0) = padded(torch.zeros_like(idx)), padded(torch.zeros_like(wt))
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        ml.test_delayed_copy(h, if0, if_, 300_000, stream=stream)
        ml.test_delayed_copy(h, wf0, wf, 300_000, stream=stream)
        out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx0, w0, W, stream=stream)
        torch.cuda.synchronize()
        assert_within(out, *experts64(*x, idx, wt, *banks, one))


def test_weights_quantised_just_before(ml, h):
    g = gen(5)
    Wb = torch.randn(2048, 1024, generator=g, device="cuda").bfloat16()
    for m in (2, 30):
        x = rand_rows(g, m, 1024)
        torch.cuda.synchronize()
        W = ml.dec_quant_weight(h, Wb)
        y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), W)
        assert_within(y, *linear64(*x, W.q, W.scale))


def test_graphs_with_their_own_workspaces_at_the_same_time(ml, h):
    g = gen(6)
    n, k, m = 4096, 4096, 100
    W = rand_weight(g, n, k)
    weight = ml.Fp8Weight(*W)
    parts = []
    for i in range(2):
        x = rand_rows(g, m, k)
        size = ml.dec_linear_fp8_workspace_size(h, m, n, k)
        ws = torch.zeros(size, dtype=torch.uint8, device="cuda")
        y = torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(20):
                ml.dec_linear_fp8(h, ml.Fp8Rows(*x), weight, y=y, ws=ws)
        parts.append((x, y, stream, graph, ws))
    for _ in range(3):
        for x, y, stream, graph, ws in parts:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for x, y, *_ in parts:
        assert_within(y, *linear64(*x, *W))


def test_one_workspace_for_many_shapes(ml, h):
    """Counters are zero between calls, whatever the shape."""
    g = gen(11)
    shapes = [(64, 4096, 1024), (17, 300, 2064), (300, 1000, 2064), (40, 640, 16384), (128, 7168, 512), (64, 4096, 1024)]
    ws = torch.zeros(max(ml.dec_linear_fp8_workspace_size(h, *s) for s in shapes), dtype=torch.uint8, device="cuda")
    for m, n, k in shapes:
        x, w = rand_rows(g, m, k), rand_weight(g, n, k)
        y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), ws=ws)
        assert_within(y, *linear64(*x, *w))


def test_workspaces_refused(ml, h):
    g = gen(12)
    (q, s), w = some_linear(g, 64)
    x, W = ml.Fp8Rows(q, s), ml.Fp8Weight(*w)
    with pytest.raises(ml.DecodeError):
        ml.dec_linear_fp8(h, x, W, ws=torch.zeros(16, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError):
        ml.dec_linear_fp8(h, x, W, ws=torch.zeros(1 << 20, dtype=torch.uint8))
    stream = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    y = torch.empty(64, 640, dtype=torch.bfloat16, device="cuda")
    with torch.cuda.graph(graph, stream=stream):
        with pytest.raises(RuntimeError, match="before the"):
            ml.dec_linear_fp8(h, x, W, y=y)
        y.zero_()


def test_binding_refuses_what_does_not_fit(ml, h):
    dev = "cuda"
    q, s = torch.zeros(4, 256, device=dev).to(E4M3), torch.zeros(4, 2, device=dev)
    x = ml.Fp8Rows(q, s)
    W = ml.Fp8Weight(torch.zeros(128, 256, device=dev).to(E4M3), torch.zeros(1, 2, device=dev))
    for bad in [(q, s[:, :1]), (q[:, ::2], s), (q, s.double()), (q.float(), s), (q[:, :24], s[:, :1]), (q[0], s[0])]:
        with pytest.raises(ValueError):
            ml.Fp8Rows(*bad)
    for bad in [(W.q, s), (W.q.t(), torch.zeros(2, 1, device=dev)), (torch.zeros(2, 64, 128, device=dev).to(E4M3), torch.zeros(2, 1, 1, device=dev))]:
        with pytest.raises(ValueError):
            ml.Fp8Weight(*bad)
    b = torch.bfloat16
    with pytest.raises(ValueError):
        ml.dec_linear_fp8(h, x, ml.Fp8Weight(torch.zeros(128, 128, device=dev).to(E4M3), torch.zeros(1, 1, device=dev)))
    for kw in [dict(y=torch.zeros(4, 127, dtype=b, device=dev)), dict(residual=torch.zeros(4, 128, device=dev)),
               dict(y=torch.zeros(128, 4, dtype=b, device=dev).t())]:
        with pytest.raises(ValueError):
            ml.dec_linear_fp8(h, x, W, **kw)
    v = torch.zeros(4, 256, dtype=b, device=dev)
    for kw in [dict(residual=v[:3]), dict(y=v.float()), dict(gamma=v[0, :128]), dict(out=ml.Fp8Rows.empty(3, 256)),
               dict(total=v.t().contiguous().t())]:
        with pytest.raises(ValueError):
            ml.dec_rmsnorm_quant(h, v, **kw)
    with pytest.raises(ml.DecodeError):
        ml.dec_rmsnorm_quant(h, v, total=torch.zeros_like(v))  # a sum without a residual
    banks, one, moe = expert_weights(ml, gen(1), 4, 256, 128, False)
    idx, wt = choices(gen(2), 4, 4, 2)
    for a in [(idx[:3], wt), (idx, wt[:, :1]), (idx.long(), wt), (idx, wt.half())]:
        with pytest.raises(ValueError):
            ml.moe_experts_fp8(h, x, *a, moe)
    with pytest.raises(ValueError):
        ml.moe_experts_fp8(h, ml.Fp8Rows(q[:, :128], s[:, :1]), idx, wt, moe)
    with pytest.raises(ValueError):
        ml.MoeFp8Weights(ml.Fp8Weight(*banks[0]), ml.Fp8Weight(*banks[1]), ml.Fp8Weight(*banks[0]))


def test_kernels_are_this_library_s(ml, h):
    g = gen(4)
    x, w = some_linear(g, 20)
    before = h.launch_count
    ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w))
    ml.dec_rmsnorm_quant(h, torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda"))
    assert h.launch_count == before + 2


# ---------------------------------------------------------------------------- past 32 bits
def random_e4m3(g, *shape):
    return torch.empty(shape, dtype=torch.uint8, device="cuda").random_(0x20, 0x58, generator=g).view(E4M3)


@pytest.mark.parametrize("m", [2, 20])
def test_linear_weights_past_32_bits(ml, h, m):
    g = gen(m)
    n, k = 540_000, 8192
    wq, ws = random_e4m3(g, n, k), torch.rand(-(-n // 128), k // 128, generator=g, device="cuda") * 1e-3
    x = rand_rows(g, m, k)
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(wq, ws))
    for at in (0, n - n % 128 - 256):
        to = min(at + 384, n)
        assert_within(y[:, at:to], *linear64(*x, wq[at:to], ws[at // 128:-(-to // 128)]))


def test_rows_past_32_bits(ml, h):
    g = gen(1)
    m, k, n = 264_000, 16400, 48
    q, s = random_e4m3(g, m, k), torch.rand(m, 129, generator=g, device="cuda") * 1e-2
    w = rand_weight(g, n, k)
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(q, s), ml.Fp8Weight(*w))
    for at in (0, m - 300):
        assert_within(y[at:at + 300], *linear64(q[at:at + 300], s[at:at + 300], *w))


def test_norm_past_32_bits(ml, h):
    g = gen(1)
    m, width = 66_000, 65536
    x = torch.empty(m, width, dtype=torch.bfloat16, device="cuda")
    x[:3].normal_(generator=g)
    x[-3:].normal_(generator=g)
    out = ml.dec_rmsnorm_quant(h, x, torch.ones(width, dtype=torch.bfloat16, device="cuda"), total=None)
    for part in (slice(0, 3), slice(m - 3, m)):
        alone = ml.dec_rmsnorm_quant(h, x[part].contiguous(), torch.ones(width, dtype=torch.bfloat16, device="cuda"))
        assert torch.equal(bits(out.q[part]), bits(alone.q)) and torch.equal(bits(out.scale[part]), bits(alone.scale))


def test_experts_past_32_bits(ml, h):
    g = gen(1)
    E, I, H = 312, 2048, 7168
    made = [(random_e4m3(g, *s), torch.rand(s[0], s[1] // 128, s[2] // 128, generator=g, device="cuda") * 1e-3)
            for s in ((E, I, H), (E, I, H), (E, H, I))]
    W = ml.MoeFp8Weights(*(ml.Fp8Weight(*b) for b in made))
    for m in (1, 3):
        x = rand_rows(g, m, H)
        idx = torch.tensor([[E - 1, 0, E - 2, 295]] * m, dtype=torch.int32, device="cuda")
        wt = torch.rand(m, 4, generator=g, device="cuda")
        out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, wt, W)
        assert_within(out, *experts64(*x, idx, wt, *made))


# ---------------------------------------------------------------------------- waits
@pytest.mark.parametrize("m,n,k", [(1, 12288, 7168), (16, 4096, 4096), (64, 4096, 4096), (40, 300, 1040), (300, 20000, 7168)])
def test_a_slow_kernel_ahead_is_no_wait_that_runs_out(ml, h, m, n, k):
    """The launch starts early and has filled its rings long before its rows are there: the limit of a wait counts from then."""
    g = gen(m)
    (q, s), w = rand_rows(g, m, k), rand_weight(g, n, k)
    (qf, _), (qf0, q0) = padded(q), padded(torch.zeros_like(q))
    x, W = ml.Fp8Rows(q0, s), ml.Fp8Weight(*w)
    ml.dec_linear_fp8(h, x, W)
    ml.test_delayed_copy(h, qf0, qf, 1000)
    qf0.view(torch.uint8).zero_()
    torch.cuda.synchronize()
    h.set_wait_limit_ns(20_000_000)
    for _ in range(2):
        ml.test_delayed_copy(h, qf0, qf, 100_000_000)
        y = ml.dec_linear_fp8(h, x, W)
        assert h.check_device_error() == 0
        assert_within(y, *linear64(q, s, *w))

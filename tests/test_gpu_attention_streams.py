"""The attention operators on streams other than the current one: the memory that a
call makes for itself is memory of the call's stream."""
import pytest

from _util import host_bits
from test_gpu_attention import Case

pytestmark = pytest.mark.gpu


@pytest.fixture
def h():
    """A handle of its own for each test: its workspaces are made there."""
    import torch
    import moe_layers_gb300 as M
    assert torch.cuda.is_available()
    M.build()
    with M.Handle(0) as hd:
        yield hd
        assert hd.check_device_error() == M.DEC_OK


def read_late(h, nbytes):
    """A copy on the current stream that begins in 0.2 s, out of memory that is given back before.
    Returns (what it copies, where to)."""
    import torch
    import moe_layers_gb300 as ML
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    want = (torch.arange(nbytes, device="cuda") % 251).to(torch.uint8)
    got = torch.zeros_like(want)
    src = want.clone()
    torch.cuda.synchronize()
    ML.test_delayed_copy(h, got, src, 200_000_000)
    del src
    return want, got


def test_attention_workspace_is_memory_of_its_stream(h):
    import torch
    import moe_layers_gb300 as ML
    c = Case([1] * 20, list(range(30, 830, 40)), 16, 4, 128, 16, prefix=500, seed=6)
    alone = c.run(h)
    size = ML.dec_attention_workspace_size(h, 20, 16, c.cache, c.batch)
    s = torch.cuda.Stream()
    out = torch.full((20, 16 * 128), 7.5, dtype=torch.bfloat16, device="cuda")
    want, got = read_late(h, size)
    for _ in range(3):
        ML.dec_attention(h, c.q, c.cache, c.batch, c.scale, out=out, stream=s)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert (host_bits(out).reshape(alone.shape) == alone).all()


def test_layer_trace_is_memory_of_its_stream(h):
    import torch
    import moe_layers_gb300 as ML
    from test_gpu_layer_attention import H, Layer, i32
    M, size = 40, 16
    L = Layer(4, 2, 64, 0, True)
    pool = torch.randn((2, M, 2, size, 64), device="cuda").to(torch.bfloat16)
    lens = i32([5] * M)
    batch = ML.Batch(i32(range(M + 1)), lens, i32([[b] for b in range(M)]))
    x0 = torch.randn((M, H), device="cuda").to(torch.bfloat16)
    streams = [torch.cuda.current_stream(), torch.cuda.Stream()]
    results = []
    for s in streams:
        # a cache of its own for each run, which writes its rows' own tokens
        cache = ML.KvCache(pool[0].clone(), pool[1].clone())
        att = ML.LayerAttention(4, 0.125, cache, batch, lens, i32([b * size + 4 for b in range(M)]))
        first, x = x0.clone(), x0.clone()
        torch.cuda.synchronize()
        ML.decode_layer_attention(h, L.w, att, first, stream=s)  # makes the workspace
        want, got = read_late(h, 2 * M * H)  # the size of h1
        trace = ML.decode_layer_attention(h, L.w, att, x, trace=True, stream=s)
        torch.cuda.synchronize()
        assert torch.equal(got, want)
        results.append(dict(trace, x=x))
    for n, t in results[0].items():
        assert torch.equal(t, results[1][n]), n


def test_layer_workspace_is_not_made_in_a_capture_of_the_given_stream(h):
    import torch
    import moe_layers_gb300 as ML
    from test_gpu_layer_attention import H, Layer, i32
    L = Layer(4, 2, 64, 0, True)
    pool = torch.zeros((2, 2, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    batch = ML.Batch(i32([0, 1]), i32([1]), i32([[0]]))
    att = ML.LayerAttention(4, 0.125, ML.KvCache(pool[0], pool[1]), batch, i32([0]), i32([0]))
    x0 = torch.randn((1, H), device="cuda").to(torch.bfloat16)
    want = x0.clone()
    s, other = torch.cuda.Stream(), torch.cuda.Stream()
    x = x0.clone()
    torch.cuda.synchronize()
    with pytest.raises(RuntimeError, match="before the capture"):
        with torch.cuda.graph(torch.cuda.CUDAGraph(), stream=s):
            with torch.cuda.stream(other):
                ML.decode_layer_attention(h, L.w, att, x, stream=s)
    torch.cuda.synchronize()
    assert not h._layer_ws and torch.equal(x, x0)
    ML.decode_layer_attention(h, L.w, att, want, stream=s)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        with torch.cuda.stream(other):
            ML.decode_layer_attention(h, L.w, att, x, stream=s)
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(x, want)

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

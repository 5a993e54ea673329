"""What the binding of the attention operators does around a call (where it makes
its tensors, what it refuses, what it passes on), checked without a GPU.

Tensors, streams and the library are stand-ins: a tensor remembers the stream
that was current when it was made, and a call only records its arguments.
"""
import contextlib
import types

import pytest
import torch


class Stream:
    def __init__(self, number, capturing=False):
        self.cuda_stream, self.capturing = number, capturing


class Tensor:
    """The part of a CUDA tensor that the binding looks at."""
    is_cuda = True
    made = 0

    def __init__(self, shape, dtype=torch.bfloat16, device=0, stride=None, stream=None):
        self.shape, self.dtype, self.index, self.made_on = tuple(shape), dtype, device, stream
        self.device = f"cuda:{device}"
        if stride is None:
            stride, n = [], 1
            for s in reversed(self.shape):
                stride.insert(0, n)
                n *= s
        self.strides = tuple(stride)
        Tensor.made += 1
        self.address = Tensor.made << 24 if self.numel() else 0

    def stride(self, i=None):
        return self.strides if i is None else self.strides[i]

    def is_contiguous(self):
        return self.strides == Tensor(self.shape).strides

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return torch.empty((), dtype=self.dtype, device="cpu").element_size()

    def get_device(self):
        return self.index

    def data_ptr(self):
        return self.address


class Library:
    """Every entry point answers OK and keeps its arguments; size queries answer `size`."""
    size = 5000

    def __init__(self):
        self.calls = {}

    def __getattr__(self, name):
        def call(*args):
            self.calls[name] = args
            if name.endswith("_workspace_size"):
                args[-1]._obj.value = self.size
            return 0
        return call


@pytest.fixture
def b(monkeypatch):
    """The binding on stand-ins: b.ml, b.lib, b.h, and b.current, the current stream."""
    import moe_layers_gb300 as ml
    at = types.SimpleNamespace(ml=ml, lib=Library(), current=Stream(1))

    @contextlib.contextmanager
    def stream(s):
        before, at.current = at.current, s
        try:
            yield
        finally:
            at.current = before

    def make(*shape, dtype=None, device=None):
        shape = shape[0] if isinstance(shape[0], (tuple, list)) else shape
        return Tensor(shape, dtype, int(str(device).rpartition(":")[2]), stream=at.current)

    real_empty = torch.empty

    def empty(*shape, dtype=None, device=None):
        return real_empty(*shape, dtype=dtype) if device == "cpu" else make(*shape, dtype=dtype, device=device)

    monkeypatch.setattr(ml, "_load", lambda: at.lib)
    monkeypatch.setattr(ml, "_bf16", torch.bfloat16)
    monkeypatch.setattr(ml, "_i32", torch.int32)
    monkeypatch.setattr(ml, "_raw_stream", lambda device: at.current.cuda_stream)
    monkeypatch.setattr(torch, "empty", empty)
    monkeypatch.setattr(torch, "zeros", make)
    monkeypatch.setattr(torch, "empty_like", lambda t: make(t.shape, dtype=t.dtype, device=t.device))
    monkeypatch.setattr(torch.cuda, "stream", stream)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: at.current)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: at.current.capturing)
    at.h = ml.Handle(0)
    at.h._h.value = 1
    at.lib.calls.clear()
    yield at
    at.h._h.value = None  # nothing to destroy


def ints(*shape, **kw):
    return Tensor(shape, torch.int32, **kw)


def attention_call(b, rows=2, heads=4, **kw):
    cache = b.ml.KvCache(Tensor((10, 2, 16, 64)), Tensor((10, 2, 16, 64)))
    batch = b.ml.Batch(ints(rows + 1), ints(rows), ints(rows, 4))
    return b.ml.dec_attention(b.h, Tensor((rows, heads * 64)), cache, batch, 0.125, **kw)


def test_attention_workspace_is_made_on_the_stream_of_the_call(b):
    """A block that the current stream has just given back may still be read there: only memory of
    the call's own stream may be written by the call."""
    s = Stream(7)
    attention_call(b, stream=s)
    (ws,) = b.h._stream_ws[("attention", 7)]
    assert ws.made_on is s and ws.numel() >= Library.size
    attention_call(b)
    (ws,) = b.h._stream_ws[("attention", 1)]
    assert ws.made_on is b.current
    # one that is outgrown, too, is replaced by one of its own stream
    b.lib.size = 50000
    attention_call(b, rows=3, stream=s)
    assert len(b.h._stream_ws[("attention", 7)]) == 2
    assert all(ws.made_on is s for ws in b.h._stream_ws[("attention", 7)])


class Weights:
    """A layer of 64 columns with 6 experts, top 2."""

    def __init__(self, ml):
        self.ml = ml

    def c_struct(self):
        c = self.ml._LayerWeights()
        c.H, c.N_in, c.K_out, c.E, c.k, c.I = 64, 512, 256, 6, 2, 128
        return c


def layer_call(b, M=2, hidden=None, **kw):
    cache = b.ml.KvCache(Tensor((10, 2, 16, 64)), Tensor((10, 2, 16, 64)))
    batch = b.ml.Batch(ints(M + 1), ints(M), ints(M, 4))
    att = b.ml.LayerAttention(4, 0.125, cache, batch, ints(M), ints(M))
    return b.ml.decode_layer_attention(b.h, Weights(b.ml), att, Tensor((M, 64)) if hidden is None else hidden, **kw)


def test_layer_trace_is_made_on_the_stream_of_the_call(b):
    s = Stream(7)
    trace = layer_call(b, trace=True, stream=s)
    assert sorted(trace) == ["h1", "idx", "scores", "w"]
    assert all(t.made_on is s for t in trace.values())
    assert all(ws.made_on is s for ws in b.h._layer_ws.values())
    trace = layer_call(b, trace=True)
    assert all(t.made_on is b.current for t in trace.values())


def test_layer_workspace_is_not_made_in_a_capture_of_the_given_stream(b):
    """The zeroes would be recorded instead of written, and the workspace kept for eager calls."""
    s = Stream(7, capturing=True)
    with pytest.raises(RuntimeError, match="before the capture"):
        layer_call(b, stream=s)
    assert not b.h._layer_ws and "decode_layer_attention" not in b.lib.calls
    s.capturing = False
    layer_call(b, stream=s)
    s.capturing = True
    layer_call(b, stream=s)  # the workspace is there
    # a capture of the current stream does not concern a call on another one
    b.current.capturing = True
    layer_call(b, M=3, stream=Stream(8))
    with pytest.raises(RuntimeError, match="before the capture"):
        layer_call(b, M=3)


@pytest.mark.parametrize("hidden", [Tensor((2, 56)), Tensor((2, 72)), Tensor((2, 64), stride=(128, 1)), Tensor((3, 64)),
                                    Tensor((2, 64), device=1), Tensor((2, 64), torch.float16), Tensor((128,))],
                         ids=lambda t: f"{t.shape}{t.stride()}{t.dtype}{t.device}")
def test_layer_refuses_hidden_states_of_another_form(b, hidden):
    """The layer's width comes from the weights: M x H values are read and written."""
    with pytest.raises(ValueError):
        layer_call(b, hidden=hidden)
    assert not b.lib.calls


TRACE = dict(h1=lambda **kw: Tensor((2, 64), **kw), idx=lambda **kw: Tensor((2, 2), torch.int32, **kw),
             w=lambda **kw: Tensor((2, 2), torch.float32, **kw), scores=lambda **kw: Tensor((2, 6), torch.float32, **kw))
BAD_TRACE = [dict(h1=Tensor((1, 64))), dict(h1=Tensor((2, 56))), dict(h1=Tensor((2, 64), torch.float32)),
             dict(h1=Tensor((2, 64), stride=(72, 1))), dict(h1=Tensor((2, 64), device=1)),
             dict(idx=Tensor((2, 1), torch.int32)), dict(idx=Tensor((2, 2), torch.int64)),
             dict(w=Tensor((2, 2))), dict(w=Tensor((1, 2), torch.float32)), dict(scores=Tensor((2, 2), torch.float32)),
             dict(scores=Tensor((2, 6), torch.float32, stride=(1, 2))), dict(idx=torch.zeros((2, 2), dtype=torch.int32))]


@pytest.mark.parametrize("bad", BAD_TRACE, ids=lambda d: f"{next(iter(d))}-{BAD_TRACE.index(d)}")
def test_layer_refuses_trace_tensors_of_another_form(b, bad):
    """M x H, M x k and M x E values are written to them."""
    trace = {n: make() for n, make in TRACE.items()}
    trace.update(bad)
    with pytest.raises(ValueError):
        layer_call(b, trace=trace)
    with pytest.raises(ValueError):
        layer_call(b, trace=bad)
    assert not b.lib.calls


def test_layer_takes_trace_tensors(b):
    for names in ("h1", "idx w", "scores", "h1 idx w scores", ""):
        trace = {n: TRACE[n]() for n in names.split()}
        assert layer_call(b, trace=trace) is trace
        given = b.lib.calls["decode_layer_attention"][5]
        if trace:
            for n in TRACE:
                assert getattr(given._obj, n) == (trace[n].data_ptr() if n in trace else None)
    layer_call(b, trace=dict(h1=Tensor((64, 64))))  # of a larger batch
    assert layer_call(b, trace=False) is None and layer_call(b, trace=dict(h1=None, idx=TRACE["idx"]()))


BAD_WS = [torch.zeros(10000, dtype=torch.uint8), Tensor((10000,), torch.uint8, device=1),
          Tensor((10000,), torch.uint8, stride=(0,)), Tensor((100, 100), torch.uint8, stride=(1, 100))]


@pytest.mark.parametrize("ws", BAD_WS, ids=["host", "other device", "expanded", "not contiguous"])
@pytest.mark.parametrize("call", [attention_call, layer_call])
def test_workspaces_of_another_form_are_refused(b, call, ws):
    with pytest.raises(ValueError):
        call(b, ws=ws)
    assert not b.lib.calls


@pytest.mark.parametrize("call,name,size_at", [(attention_call, "dec_attention", 11), (layer_call, "decode_layer_attention", 7)])
def test_workspaces_count_in_bytes(b, call, name, size_at):
    for t in (Tensor((6000,), torch.uint8), Tensor((60, 100), torch.float32)):
        call(b, ws=t)
        assert b.lib.calls[name][size_at - 1:size_at + 1] == (t.data_ptr(), t.numel() * t.element_size())


def tables_call(b, free, n=2, rows=3):
    out = b.ml.StepTables(ints(n + 1), ints(n), ints(rows), ints(rows), ints(2))
    count = ints(1)
    b.ml.dec_batch_tables(b.h, ints(n), ints(n), free, count, ints(n, 4), 16, out)
    return b.lib.calls["dec_batch_tables"][4:6] + (count,)


def test_tables_take_an_empty_free_list(b):
    """A tensor without elements has no address, which the library takes for a missing argument:
    another one stands for it (with a count of 0 nothing is read there)."""
    free, at, count = tables_call(b, ints(0))
    assert free == at == count.data_ptr() != 0
    given = ints(5)
    free, at, count = tables_call(b, given)
    assert free == given.data_ptr() and at == count.data_ptr()
    with pytest.raises(ValueError):
        tables_call(b, ints(0, device=1))
    with pytest.raises(ValueError):
        tables_call(b, Tensor((0,), torch.int64))

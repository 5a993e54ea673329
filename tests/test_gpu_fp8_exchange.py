"""The 8-bit product where CTAs exchange pieces of a tile through the workspace: whole rounds of tiles, then left-over
ones that two to four CTAs share."""
import pytest
import torch

from _fp8 import assert_within, linear64, rand_rows, rand_weight
from test_gpu_fp8 import bits, gen

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


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


def counter_bytes():
    return (sms() * 4 + 255) // 256 * 256


def ragged(left, row_tiles, k, rounds=1, tile=256):
    """(m, n, k) of `rounds` whole rounds and about `left` tiles of `tile` weights, rows and columns ragged."""
    return row_tiles * 128 - 51, -(-(rounds * sms() + left) // row_tiles) * tile - 57, k


def workspace(ml, h, m, n, k, tile=256):
    """A zeroed workspace; its size says that pieces go through it."""
    size = ml.dec_linear_fp8_workspace_size(h, m, n, k)
    assert size == counter_bytes() + sms() * tile * 128 * 4
    return torch.zeros(size, dtype=torch.uint8, device="cuda")


def counters(ws):
    return ws[:counter_bytes()].view(torch.int32)


@pytest.mark.parametrize("every", [1, 2, 3, 5])
@pytest.mark.parametrize("at,kw", [((30, 3, 7168), {}), ((40, 3, 7184), {}), ((52, 3, 16384), {})], ids=str)
def test_a_wait_that_runs_out_leaves_the_workspace_ready(ml, h, at, kw, every):
    """Part of the CTAs give up: of a tile that four, three or two share some, all or none. The call is lost, and the error
    word says so; the next one on the workspace is not."""
    m, n, k = ragged(*at, **kw)
    g = gen(5)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    X, W = ml.Fp8Rows(*x), ml.Fp8Weight(*w)
    ws = workspace(ml, h, m, n, k)
    h.test_set_linear_fp8_give_up(every)
    for _ in range(2):
        ml.dec_linear_fp8(h, X, W, ws=ws)
        assert h.check_device_error() == ml.DEC_ERR_TIMEOUT
        assert not counters(ws).any()
    h.test_set_linear_fp8_give_up(0)
    y = ml.dec_linear_fp8(h, X, W, ws=ws)
    assert h.check_device_error() == ml.DEC_OK
    assert_within(y, *linear64(*x, *w))


@pytest.mark.parametrize("every", [1, 2, 3])
@pytest.mark.parametrize("m,n,k", [(64, 4096, 4096), (64, 12288, 7168), (20, 300, 1040), (700, 7168, 1024)])
def test_a_wait_that_runs_out_in_clusters_and_whole_tiles(ml, h, m, n, k, every):
    g = gen(6)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    X, W = ml.Fp8Rows(*x), ml.Fp8Weight(*w)
    h.test_set_linear_fp8_give_up(every)
    ml.dec_linear_fp8(h, X, W)
    assert h.check_device_error() == ml.DEC_ERR_TIMEOUT
    h.test_set_linear_fp8_give_up(0)
    y = ml.dec_linear_fp8(h, X, W)
    assert h.check_device_error() == ml.DEC_OK
    assert_within(y, *linear64(*x, *w))


# about (left-over tiles, tiles of rows, K, whole rounds, weights of a tile); on 152 SMs they are shared by as many CTAs as
# behind them
SHARED = [((8, 3, 16400), {}), ((30, 3, 7168), {}),                   # 4
          ((16, 8, 16384), dict(rounds=4)),                           # 4
          ((40, 3, 7184), {}), ((44, 8, 7168), dict(rounds=2)),       # 3
          ((52, 3, 16384), {}), ((60, 3, 16400), {}),                 # 2
          ((52, 3, 7168), dict(tile=192)), ((50, 4, 7168), dict(tile=192))]


@pytest.mark.parametrize("at,kw", SHARED, ids=str)
@pytest.mark.parametrize("residual", [False, True])
def test_shared_tiles(ml, h, at, kw, residual):
    m, n, k = ragged(*at, **kw)
    g = gen(n)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    r = torch.randn(m, n + 3, generator=g, device="cuda").bfloat16()[:, 1:n + 1] if residual else None
    ws = workspace(ml, h, m, n, k, kw.get("tile", 256))
    X, W = ml.Fp8Rows(*x), ml.Fp8Weight(*w)
    y = ml.dec_linear_fp8(h, X, W, residual=r, ws=ws)
    assert_within(y, *linear64(*x, *w, r))
    assert not counters(ws).any()
    # what the workspace holds beside the counters does not matter, and the order in which CTAs finish neither
    ws[counter_bytes():] = 0xFF
    for _ in range(3):
        assert torch.equal(bits(ml.dec_linear_fp8(h, X, W, residual=r, ws=ws)), bits(y))
    if residual:  # in the residual's place
        ml.dec_linear_fp8(h, X, W, residual=r, y=r, ws=ws)
        assert torch.equal(bits(r), bits(y))
    assert not counters(ws).any() and h.check_device_error() == 0


def test_one_workspace_for_shared_tiles_and_others(ml, h):
    """Back to back: shared tiles of several kinds, clusters and whole tiles between them."""
    shapes = [ragged(30, 3, 7168), (64, 4096, 1024), ragged(52, 3, 16384), (300, 1000, 2064), ragged(44, 8, 7168, rounds=2),
              (17, 300, 2064), ragged(52, 3, 7168, tile=192), (200, 640, 384), ragged(30, 3, 7168)]
    ws = torch.zeros(max(ml.dec_linear_fp8_workspace_size(h, *s) for s in shapes), dtype=torch.uint8, device="cuda")
    g = gen(21)
    made = [(rand_rows(g, m, k), rand_weight(g, n, k)) for m, n, k in shapes]
    alone = [ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w)) for x, w in made]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    outs = [[ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), ws=ws, stream=stream) for x, w in made]
            for _ in range(3)]
    torch.cuda.synchronize()
    for x, w, y in zip([x for x, _ in made], [w for _, w in made], alone):
        assert_within(y, *linear64(*x, *w))
    for again in outs:
        for y, want in zip(again, alone):
            assert torch.equal(bits(y), bits(want))
    assert not counters(ws).any() and h.check_device_error() == 0


def test_shared_tiles_in_two_graphs_at_the_same_time(ml, h):
    m, n, k = ragged(30, 3, 7168)
    g = gen(22)
    w = rand_weight(g, n, k)
    W = ml.Fp8Weight(*w)
    parts = []
    for _ in range(2):
        x = rand_rows(g, m, k)
        ws, y = workspace(ml, h, m, n, k), torch.empty(m, n, dtype=torch.bfloat16, device="cuda")
        stream, graph = torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            for _ in range(8):
                ml.dec_linear_fp8(h, ml.Fp8Rows(*x), W, y=y, ws=ws)
        parts.append((x, y, ws, stream, graph))
    for _ in range(3):
        for *_, stream, graph in parts:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    for x, y, ws, *_ in parts:
        assert_within(y, *linear64(*x, *w))
        assert not counters(ws).any()
    assert h.check_device_error() == 0


@pytest.mark.parametrize("m,k,family", [(16, 65536, 2), (3, 65536, 2), (2, 65536, 1), (16, 16384, 2), (8, 16384, 1), (16, 8192, 1)])
def test_few_rows_too_long_for_shared_memory(ml, h, m, k, family):
    """The streaming kernel forced: rows that its shared memory does not hold go to the tcgen05 kernel."""
    g = gen(m + k)
    x, w = rand_rows(g, m, k), rand_weight(g, 130, k)
    h.set_force_variant(ml.VARIANT_SMALL_M)
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w))
    assert h.last_variant == family
    assert_within(y, *linear64(*x, *w))

"""The 8-bit product where CTAs exchange pieces of a tile through the workspace: whole rounds of tiles, then left-over
ones that two to four CTAs share."""
import time

import pytest
import torch

from _fp8 import assert_within, linear64, rand_rows, rand_weight
from test_gpu_fp8 import gen

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


def test_a_wait_that_runs_out_leaves_the_workspace_ready(ml, h):
    """Part of the CTAs give up: those that start while the kernel ahead is still running wait for its rows past the
    handle's limit, the others start when an SM is free again. A shared tile of CTAs of both kinds is lost, and the
    error word says so; the next call on the workspace is not."""
    m, n, k = ragged(30, 3, 7168)  # 31 tiles of four CTAs each where a device has 152 SMs
    g = gen(5)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    X, W = ml.Fp8Rows(*x), ml.Fp8Weight(*w)
    ws = workspace(ml, h, m, n, k)
    early = 3 * sms() // 16 * 4 + 2  # CTAs that start at once, less one where the kernel ahead has its SM
    src, dst = (torch.zeros(4, device="cuda") for _ in range(2))
    main, side = torch.cuda.Stream(), torch.cuda.Stream()
    ml.dec_linear_fp8(h, X, W, ws=ws)  # the code is loaded
    ml.test_delayed_copy(h, dst, src, 1000)
    ml.test_occupy_sms(h, 1, 1000)
    torch.cuda.synchronize()
    h.set_wait_limit_ns(20_000_000)
    try:
        ml.test_occupy_sms(h, sms() - early, 900_000_000, stream=side)
        time.sleep(0.002)  # it is resident before the others are launched
        ml.test_delayed_copy(h, dst, src, 500_000_000, stream=main)
        ml.dec_linear_fp8(h, X, W, ws=ws, stream=main)
        torch.cuda.synchronize()
    finally:
        h.set_wait_limit_ns(500_000_000)
    assert h.check_device_error() == ml.DEC_ERR_TIMEOUT
    assert not counters(ws).any()
    y = ml.dec_linear_fp8(h, X, W, ws=ws)
    assert h.check_device_error() == ml.DEC_OK
    assert_within(y, *linear64(*x, *w))

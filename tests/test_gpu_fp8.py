"""The operators on 8-bit rows and weights against plain forms in 64 bits."""
import pytest
import torch

from _fp8 import (E4M3, TOP, amax_groups, assert_within, experts64, groups, linear64, quant_rows, rand_rows, rand_weight,
                  spread, value_rows, value_weight)

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def ml():
    import moe_layers_gb300 as M
    M.build()
    return M


@pytest.fixture(scope="module")
def h(ml):
    with ml.Handle(0) as handle:
        yield handle


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def bits(t):
    return t.contiguous().view({1: torch.uint8, 2: torch.int16, 4: torch.int32}[t.element_size()])


# ---------------------------------------------------------------------------- norm
NORMS = [(1, 7168), (3, 16), (2, 128), (5, 144), (64, 2048), (7, 2064), (3, 4112), (130, 1040), (2, 8192), (2, 16400),
         (1, 33008), (2, 65536)]


@pytest.mark.parametrize("rows,width", NORMS)
@pytest.mark.parametrize("residual", [False, True])
def test_norm(ml, h, rows, width, residual):
    g = gen(rows * width)
    x = torch.randn(rows, width, generator=g, device="cuda").bfloat16()
    r = (3 * torch.randn(rows, width, generator=g, device="cuda")).bfloat16() if residual else None
    gamma = (1 + 0.3 * torch.randn(width, generator=g, device="cuda")).bfloat16()
    total = torch.empty_like(x) if residual else None
    y = torch.empty_like(x)
    out = ml.dec_rmsnorm_quant(h, x, gamma, residual=r, eps=1e-5, total=total, y=y)
    a = (x.float() + r.float()).bfloat16() if residual else x
    if residual:
        assert torch.equal(bits(total), bits(a))
    if rows <= 64:
        assert torch.equal(bits(y), bits(ml.dec_rmsnorm(h, a, gamma, eps=1e-5)))
    d = a.double()
    want = d / torch.sqrt(d.square().mean(-1, keepdim=True) + 1e-5) * gamma.double()
    # a thread's additions, five shuffles and eight warps, halved by the root; then the root, the mean and two products
    rel = ((8 * -(-width // 2048) + 13) / 2 + 8) * 2.0 ** -24
    assert_within(y, want, (2.0 ** -8 + rel) * want.abs())
    s = amax_groups(want) / TOP
    assert_within(out.scale, s, (rel + 2.0 ** -23) * s)
    v = want / spread(s, width)
    # half a step: 2^-4 of a normal number, 2^-10 below
    assert_within(out.q, v, torch.maximum(v.abs() * 2.0 ** -4, torch.tensor(2.0 ** -10, dtype=torch.float64, device="cuda"))
                  + 3 * rel * v.abs() + 1e-300)


@pytest.mark.parametrize("rows,width", NORMS)
def test_quantised_rows_are_the_formula_s(ml, h, rows, width):
    """Without a norm every step is one rounding that torch makes as well."""
    x = (torch.randn(rows, width, generator=gen(width), device="cuda") * 7).bfloat16()
    x[-1, : width // 2] = 0
    out = ml.dec_rmsnorm_quant(h, x)
    q, s = quant_rows(x.float())
    assert torch.equal(bits(out.scale), bits(s)) and torch.equal(bits(out.q), bits(q))


def test_norm_in_place_and_strided(ml, h):
    g = gen(4)
    wide = torch.randn(6, 3 * 1040, generator=g, device="cuda").bfloat16()
    x, r = wide[:, 1040:2080], torch.randn(6, 1040, generator=g, device="cuda").bfloat16()
    gamma = torch.randn(1040, generator=g, device="cuda").bfloat16()
    want_total = torch.empty_like(r)
    want_y = torch.empty_like(r)
    want = ml.dec_rmsnorm_quant(h, x.contiguous(), gamma, residual=r, total=want_total, y=want_y)
    rest = wide.clone()
    big = ml.Fp8Rows.empty(6, 2048)
    out = ml.Fp8Rows(big.q[:, 512:512 + 1040], big.scale[:, 4:13])
    y = torch.zeros(6, 1040 + 8, dtype=torch.bfloat16, device="cuda")
    ml.dec_rmsnorm_quant(h, x, gamma, residual=r, total=x, y=y[:, :1040], out=out)
    assert torch.equal(bits(x), bits(want_total)) and torch.equal(bits(y[:, :1040]), bits(want_y))
    assert torch.equal(bits(out.q), bits(want.q)) and torch.equal(bits(out.scale), bits(want.scale))
    assert torch.equal(wide[:, :1040], rest[:, :1040]) and torch.equal(wide[:, 2080:], rest[:, 2080:])
    assert not y[:, 1040:].any()
    # the sum in the residual's place, as a layer keeps its stream
    x2 = rest[:, 1040:2080]
    out2 = ml.dec_rmsnorm_quant(h, x2, gamma, residual=r, total=r)
    assert torch.equal(bits(r), bits(want_total)) and torch.equal(bits(out2.q), bits(want.q))


def test_norm_of_zeros_infinities_and_nan(ml, h):
    x = torch.zeros(5, 400, dtype=torch.bfloat16, device="cuda")
    x[1, 5], x[2, 130], x[3, :] = float("inf"), float("nan"), 2.0 ** -120
    x[4, 7] = 3.0
    out = ml.dec_rmsnorm_quant(h, x)
    s, v = out.scale.cpu(), (out.q.float() * spread(out.scale, 400)).cpu()
    assert (s[0] == 0).all() and (v[0] == 0).all() and (s[3] == 0).all() and (v[3] == 0).all()
    assert s[1, 0] == float("inf") and torch.isnan(v[1, :128]).all() and (v[1, 128:] == 0).all()
    assert torch.isnan(s[2, 1]) and torch.isnan(v[2, 128:256]).all() and (v[2, :128] == 0).all()
    assert v[4, 7] == 3.0 and v[4].sum() == 3.0


@pytest.mark.parametrize("shape", [(128, 128), (1, 16), (100, 272), (384, 2048), (3, 128, 1040)])
def test_weights(ml, h, shape):
    W = torch.randn(*shape, generator=gen(len(shape)), device="cuda").bfloat16()
    got = ml.dec_quant_weight(h, W)
    n, k = shape[-2:]
    flat, q, s = W.reshape(-1, n, k).float(), got.q.reshape(-1, n, k), got.scale.reshape(-1, groups(n), groups(k))
    for e in range(flat.shape[0]):
        for i in range(groups(n)):
            for j in range(groups(k)):
                at = (slice(128 * i, 128 * i + 128), slice(128 * j, 128 * j + 128))
                block = flat[e][at]
                most = block.abs().max()
                top = torch.full_like(most, TOP)
                assert s[e, i, j] == most / top
                assert torch.equal(bits(q[e][at]), bits((block * (top / most)).to(E4M3)))


# ---------------------------------------------------------------------------- linear
LINEARS = [(1, 128, 128), (1, 1, 16), (2, 17, 144), (3, 1000, 2064), (8, 304, 7168), (9, 129, 512), (16, 12288, 256),
           (15, 500, 4096), (17, 640, 384), (33, 77, 1040), (64, 1536, 7168), (65, 256, 128), (128, 130, 640),
           (200, 1000, 2064), (333, 129, 272), (1, 12288, 7168), (4, 4096, 4096), (1, 40, 65536), (5, 33, 30000), (40, 100, 16384), (17, 64, 65536),
           (130, 128, 8192), (64, 2048, 8208), (100, 4096, 1024)]


@pytest.mark.parametrize("m,n,k", LINEARS)
@pytest.mark.parametrize("residual", [False, True])
def test_linear(ml, h, m, n, k, residual):
    g = gen(m * n + k)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    r = torch.randn(m, n, generator=g, device="cuda").bfloat16() if residual else None
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), residual=r)
    assert_within(y, *linear64(*x, *w, r))
    assert h.check_device_error() == 0
    again = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), residual=r)
    assert torch.equal(bits(y), bits(again))


@pytest.mark.parametrize("m,n,k", [(20, 1, 16), (300, 5, 16), (1 << 20, 8, 16), (1, 1 << 20, 16), (70, 1 << 20, 16),
                                   (16, 300, 65536), (2, 3, 65536), (129, 257, 65536)])
def test_linear_at_its_limits(ml, h, m, n, k):
    g = gen(m + n)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w))
    assert_within(y, *linear64(*x, *w))


@pytest.mark.parametrize("family", [1, 2])
@pytest.mark.parametrize("m,n,k", [(1, 300, 1040), (5, 4096, 4096), (8, 640, 16384), (9, 1000, 2064), (16, 7168, 1024),
                                   (16, 12288, 7168), (13, 130, 144)])
def test_linear_kernel_families(ml, h, family, m, n, k):
    g = gen(m)
    x, w = rand_rows(g, m, k), rand_weight(g, n, k)
    r = torch.randn(m, n, generator=g, device="cuda").bfloat16()
    h.set_force_variant(family)
    try:
        y = ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), residual=r)
        assert h.last_variant == (2 if k * m > 200_000 else family)
    finally:
        h.set_force_variant(0)
    assert_within(y, *linear64(*x, *w, r))


@pytest.mark.parametrize("m", [5, 40, 150])
def test_linear_in_place_and_strided(ml, h, m):
    g = gen(m)
    n, k = 1032, 640
    q, s = rand_rows(g, m, 2048)
    w = rand_weight(g, n, k)
    x = (q[:, 256:256 + k], s[:, 2:7])
    r = torch.randn(m, n + 9, generator=g, device="cuda").bfloat16()
    keep = r.clone()
    want = linear64(x[0], x[1], *w, r[:, 3:3 + n])
    ml.dec_linear_fp8(h, ml.Fp8Rows(*x), ml.Fp8Weight(*w), residual=r[:, 3:3 + n], y=r[:, 3:3 + n])
    assert_within(r[:, 3:3 + n], *want)
    assert torch.equal(r[:, :3], keep[:, :3]) and torch.equal(r[:, 3 + n:], keep[:, 3 + n:])


@pytest.mark.parametrize("m", [1, 12, 50, 140])
def test_linear_nan_stays_in_its_row_and_column(ml, h, m):
    g = gen(m)
    n, k = 300, 272
    (q, s), (wq, ws) = rand_rows(g, m, k), rand_weight(g, n, k)
    want, room = linear64(q, s, wq, ws)
    qb, wb = bits(q).clone(), bits(wq).clone()
    qb[m - 1, 3], wb[130, 200] = 0x7F, 0x7F
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(qb.view(E4M3), s), ml.Fp8Weight(wb.view(E4M3), ws))
    assert torch.isnan(y[m - 1]).all() and torch.isnan(y[:, 130]).all()
    keep = torch.ones(m, n, dtype=torch.bool, device="cuda")
    keep[m - 1], keep[:, 130] = False, False
    if m > 1:
        assert_within(y[keep], want[keep], room[keep])
    # a scale of its own: rows and blocks of columns
    s2, ws2 = s.clone(), ws.clone()
    s2[0, 1], ws2[2, 0] = float("nan"), float("inf")
    y = ml.dec_linear_fp8(h, ml.Fp8Rows(q, s2), ml.Fp8Weight(wq, ws2))
    assert torch.isnan(y[0]).all() and not torch.isfinite(y[:, 256:]).any()
    if m > 1:
        assert_within(y[1:, :256], want[1:, :256], room[1:, :256])


# ---------------------------------------------------------------------------- experts
def expert_weights(ml, g, e, hidden, inner, shared):
    banks = [rand_weight(g, e, inner, hidden), rand_weight(g, e, inner, hidden), rand_weight(g, e, hidden, inner)]
    one = [rand_weight(g, inner, hidden), rand_weight(g, inner, hidden), rand_weight(g, hidden, inner)] if shared else None
    made = ml.MoeFp8Weights(*(ml.Fp8Weight(*b) for b in banks), *([ml.Fp8Weight(*b) for b in one] if shared else []))
    return banks, one, made


def choices(g, m, e, k):
    best = torch.rand(m, e, generator=g, device="cuda").topk(k, -1)
    return best.indices.int().contiguous(), (best.values / best.values.sum(-1, keepdim=True)).contiguous()


EXPERTS = [(1, 8, 2, 128, 128), (1, 384, 8, 512, 256), (1, 4, 1, 1024, 384), (2, 16, 8, 256, 512), (3, 8, 8, 384, 128),
           (8, 32, 8, 512, 256), (9, 5, 3, 256, 128), (16, 24, 6, 640, 256), (17, 16, 4, 256, 256), (64, 64, 8, 256, 128),
           (64, 9, 8, 384, 256), (64, 1, 1, 256, 128), (40, 1024, 16, 128, 128), (4, 12, 2, 7168, 2048)]


@pytest.mark.parametrize("m,e,k,hidden,inner", EXPERTS)
@pytest.mark.parametrize("shared", [False, True])
def test_experts(ml, h, m, e, k, hidden, inner, shared):
    g = gen(m * e + k)
    banks, one, W = expert_weights(ml, g, e, hidden, inner, shared)
    x = rand_rows(g, m, hidden)
    idx, w = choices(g, m, e, k)
    r = torch.randn(m, hidden, generator=g, device="cuda").bfloat16()
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W, residual=r)
    assert_within(out, *experts64(*x, idx, w, *banks, one, r))
    again = r.clone()
    ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W, residual=again, out=again)
    assert torch.equal(bits(out), bits(again))
    bare = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    assert_within(bare, *experts64(*x, idx, w, *banks, one))


@pytest.mark.parametrize("m,e,k,hidden,inner", [(1, 2, 2, 16384, 128), (5, 2, 1, 128, 16384), (64, 1024, 16, 256, 128),
                                                (3, 4, 2, 16384, 256), (1, 1, 1, 128, 128)])
def test_experts_at_their_limits(ml, h, m, e, k, hidden, inner):
    g = gen(m + e)
    banks, one, W = expert_weights(ml, g, e, hidden, inner, True)
    x = rand_rows(g, m, hidden)
    idx, w = choices(g, m, e, k)
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    assert_within(out, *experts64(*x, idx, w, *banks, one))


@pytest.mark.parametrize("m,k", [(1, 4), (6, 4), (64, 3)])
def test_experts_twice_and_out_of_range(ml, h, m, k):
    """The same expert twice for a token adds twice; ids outside [0, E) add nothing; a token may have no expert at all."""
    g = gen(m)
    banks, one, W = expert_weights(ml, g, 6, 256, 128, m != 6)
    x = rand_rows(g, m, 256)
    idx, w = choices(g, m, 6, k)
    idx[:, 1] = idx[:, 0]
    idx[0, 2] = -1
    if m > 1:
        idx[1, :] = torch.tensor([6, -7, 2 ** 31 - 1, -2 ** 31][:k], dtype=torch.int32)
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    want, room = experts64(*x, idx, w, *banks, one)
    assert_within(out, want, room + 1e-300)
    if m == 6:
        assert not out[1].any()


def test_experts_all_tokens_to_the_same(ml, h):
    g = gen(9)
    banks, one, W = expert_weights(ml, g, 12, 512, 256, True)
    x = rand_rows(g, 64, 512)
    idx = torch.tensor([[3, 7, 11]], dtype=torch.int32, device="cuda").repeat(64, 1)
    w = torch.rand(64, 3, generator=g, device="cuda")
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    assert_within(out, *experts64(*x, idx, w, *banks, one))


def test_experts_nan_of_an_expert_reaches_its_tokens_alone(ml, h):
    g = gen(2)
    banks, one, W = expert_weights(ml, g, 8, 256, 128, True)
    x = rand_rows(g, 5, 256)
    idx, w = choices(g, 5, 8, 2)
    idx[0, 0], idx[1:, :] = 3, torch.where(idx[1:, :] == 3, 4, idx[1:, :])
    want, room = experts64(*x, idx, w, *banks, one)
    bits(banks[2][0])[3, 17, 5] = 0x7F
    out = ml.moe_experts_fp8(h, ml.Fp8Rows(*x), idx, w, W)
    assert torch.isnan(out[0, 17]) and torch.isfinite(out[0, :17]).all()
    assert_within(out[1:], want[1:], room[1:])


# ---------------------------------------------------------------------------- together
def test_a_layer_s_run(ml, h):
    """Norm, projection, quantised middle, projection with the residual, norm for router and experts: each step's input
    is the step's before, and each is checked by itself in 64 bits."""
    g = gen(1)
    m, H, mid, E, I, k = 5, 512, 768, 16, 256, 4
    x = torch.randn(m, H, generator=g, device="cuda").bfloat16()
    g1, g2 = ((1 + 0.2 * torch.randn(H, generator=g, device="cuda")).bfloat16() for _ in range(2))
    w_in, w_o = rand_weight(g, mid, H), rand_weight(g, H, mid)
    banks, one, W = expert_weights(ml, g, E, H, I, True)
    Wr = torch.randn(E, H, generator=g, device="cuda") * H ** -0.5
    a = ml.dec_rmsnorm_quant(h, x, g1)
    y = ml.dec_linear_fp8(h, a, ml.Fp8Weight(*w_in))
    assert_within(y, *linear64(a.q, a.scale, *w_in))
    b = ml.dec_rmsnorm_quant(h, y)
    attended = ml.dec_linear_fp8(h, b, ml.Fp8Weight(*w_o))
    assert_within(attended, *linear64(b.q, b.scale, *w_o))
    normed = torch.empty_like(x)
    c = ml.dec_rmsnorm_quant(h, attended, g2, residual=x, total=x, y=normed)
    idx, w, _ = ml.moe_route_topk(h, normed, Wr, k)
    ml.moe_experts_fp8(h, c, idx, w, W, residual=x, out=attended)
    assert_within(attended, *experts64(c.q, c.scale, idx, w, *banks, one, x))

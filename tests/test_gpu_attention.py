"""GPU parity of the attention operators against their fp64 oracle.

Tolerances. A bf16 rounding is off by at most 2^-8 of the value. Rotary
positions: one such rounding, and fp32 products and sums of two terms with
cosines good to 2^-22: 2^-20 (|a| + |b|) covers them. Attention: one rounding
of the output (2^-8 of it), one of each weight p (2^-8 of sum p |v|), fp32
sums over D products (scores off by at most D 2^-23 of the largest
scale sum |q k|, which changes every p by that much, numerator and
denominator), fp32 sums over n keys (n 2^-23 of sum p |v|) and exponentials
good to 2^-20.
"""
import numpy as np
import pytest

import oracle
from _util import host_bits

pytestmark = pytest.mark.gpu


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


def bf16(a):
    import torch
    return torch.tensor(np.ascontiguousarray(a, dtype=np.float32)).to(torch.bfloat16).cuda()


# ---------------------------------------------------------------------------- tables
def run_tables(h, ctx, new, free, count, table, size, offset, rows):
    import torch
    import moe_layers_gb300 as ML
    t = i32(table)
    out = ML.dec_batch_tables(h, i32(ctx), i32(new), i32(free), i32([count]), t, size, rows=rows,
                              position_offset=offset)
    torch.cuda.synchronize()
    got = {n: getattr(out, n).cpu().numpy() for n in ("row_start", "own_len", "positions", "slots", "left")}
    return dict(got, table=t.cpu().numpy())


def check_tables(h, ctx, new, free, count, table, size, offset, rows):
    want = oracle.batch_tables(ctx, new, free, count, table, size, offset, rows)
    got = run_tables(h, ctx, new, free, count, table, size, offset, rows)
    for n in want:
        assert np.array_equal(got[n], want[n]), n


@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("n,seed", [(1, 0), (2, 1), (31, 2), (32, 3), (33, 4), (64, 5), (300, 6), (1024, 7)])
def test_tables(h, size, n, seed):
    rng = np.random.default_rng(seed)
    ctx = rng.integers(0, 5 * size, n)
    ctx[rng.random(n) < 0.3] //= size
    ctx[rng.random(n) < 0.2] *= 0
    new = np.where(rng.random(n) < 0.2, rng.integers(0, 3 * size, n), 1)
    new[rng.random(n) < 0.1] = 0
    ids = rng.permutation(20 * n).astype(np.int64)
    table = np.full((n, 9), -1)
    at = 0
    for b in range(n):
        m = -(-int(ctx[b]) // size)
        table[b, :m] = ids[at:at + m]
        at += m
    free = ids[at:]
    for rows in (int(new.sum()) + 7, max(int(new.sum()), 1)):
        check_tables(h, ctx, new, free, len(free), table, size, 1000, rows)


def test_tables_at_the_edges(h):
    size = 16
    # the free list runs dry in the middle of a request, and later requests get nothing
    check_tables(h, [10, 16, 0, 5], [1, 1, 40, 20], [3, 8], 2, np.full((4, 6), 2), size, 0, 70)
    # no free block at all, a count below zero, negative lengths
    check_tables(h, [16, -5], [1, -3], [3], 0, np.full((2, 2), 1), size, 0, 3)
    check_tables(h, [16, 0], [1, 4], [3], -2, np.full((2, 2), 1), size, 0, 6)
    # rows past the capacity are left out, and their blocks are not taken
    check_tables(h, [3, 0, 7], [1, 50, 9], np.arange(20), 20, np.full((3, 8), 5), size, 7, 30)
    # a request that has outgrown its row of the table, a held entry that is not there
    check_tables(h, [40, 3], [5, 1], np.arange(9), 9, [[1, 2], [-1, -1]], size, 0, 8)
    # one request, one row
    check_tables(h, [0], [1], [4], 1, [[-1]], size, 0, 1)
    # nothing new
    check_tables(h, [5, 6], [0, 0], [4], 1, [[1], [2]], size, 0, 4)


def test_tables_large_prompt_batch(h):
    rng = np.random.default_rng(11)
    n, size = 40, 16
    ctx = rng.integers(0, 200, n)
    new = rng.integers(1, 9000, n)
    width = -(-int((ctx + new).max()) // size)
    ids = rng.permutation(n * width + 100)
    table = np.full((n, width), -1)
    at = 0
    for b in range(n):
        m = -(-int(ctx[b]) // size)
        table[b, :m] = ids[at:at + m]
        at += m
    check_tables(h, ctx, new, ids[at:], len(ids) - at, table, size, 31000, int(new.sum()) + 3)


def test_tables_step_after_step_in_place_under_a_graph(h):
    """own_len over ctx_len and left over free_count: a captured step continues by itself."""
    import torch
    import moe_layers_gb300 as ML
    size, n = 16, 5
    ctx0 = [0, 14, 15, 16, 40]
    table0 = np.full((n, 8), -1)
    ids = list(range(60))
    for b in range(n):
        for j in range(-(-ctx0[b] // size)):
            table0[b, j] = ids.pop(0)
    ctx, new, free, count, table = i32(ctx0), i32([1, 1, 0, 1, 1]), i32(ids), i32([len(ids), 0]), i32(table0)
    out = ML.StepTables(torch.zeros(n + 1, dtype=torch.int32, device="cuda"), ctx,
                        torch.zeros(6, dtype=torch.int32, device="cuda"),
                        torch.zeros(6, dtype=torch.int32, device="cuda"), count)
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g, stream=side):
        ML.dec_batch_tables(h, ctx, new, free, count, table, size, out)
    want = dict(own_len=np.array(ctx0), left=np.array([len(ids), 0]), table=table0)
    for _ in range(40):
        g.replay()
        want = oracle.batch_tables(want["own_len"], [1, 1, 0, 1, 1], ids, want["left"][0], want["table"], size, 0, 6)
    torch.cuda.synchronize()
    got = dict(own_len=ctx, left=count, table=table, positions=out.positions, slots=out.slots)
    for k, t in got.items():
        assert np.array_equal(t.cpu().numpy(), want[k]), k


# ---------------------------------------------------------------------------- rotary positions
def rope_case(h, T, heads, kv, d, rot, inter, size, scaling="none", factor=1.0, mag=1.0, positions=None, seed=0,
              wide=0, in_place=False, bad=()):
    import torch
    import moe_layers_gb300 as ML
    rng = np.random.default_rng(seed)
    width = (heads + 2 * kv) * d + wide
    y = bf16(rng.standard_normal((T, width)))
    q, k, v = (y[:, a:b] for a, b in ((0, heads * d), (heads * d, (heads + kv) * d),
                                      ((heads + kv) * d, (heads + 2 * kv) * d)))
    blocks = -(-T // size) + 2
    positions = rng.integers(0, 1 << 17, T) if positions is None else np.resize(positions, T)
    slots = rng.permutation(blocks * size)[:T]
    for i, s in bad:
        slots[i] = s
    pool = bf16(rng.standard_normal((blocks, 2, kv, size, d)))  # k and v interleaved in one pool
    kc, vc = pool[:, 0], pool[:, 1]
    y0, kc0, vc0 = (host_bits(t) for t in (y, kc, vc))
    r = ML.Rope(h, rot, base=10000.0, interleaved=inter, scaling=scaling, factor=factor, magnitude=mag)
    out = ML.dec_rope_append(h, r, q if heads else None, k, v, i32(positions), i32(slots), ML.KvCache(kc, vc),
                             q_out=q if in_place else None)
    torch.cuda.synchronize()
    freq = oracle.rope_frequencies(rot, 10000.0, scaling, factor, high=32.0 if scaling == "yarn" else 4.0)
    x = oracle.as_f64(y0)[:, :(heads + 2 * kv) * d].reshape(T, heads + 2 * kv, d)
    want = oracle.rope(x, positions, freq, inter, mag)
    near = np.abs(want) * 2.0 ** -8
    size_of = np.zeros_like(x)
    a_at, b_at = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    size_of[..., a_at] = size_of[..., b_at] = np.abs(x[..., a_at]) + np.abs(x[..., b_at])
    near += size_of * abs(mag) * 2.0 ** -20
    near[..., rot:] = 0.0
    if heads:
        got = oracle.as_f64(host_bits(out)).reshape(T, heads, d)
        assert np.all(np.abs(got - want[:, :heads]) <= near[:, :heads])
    y1 = host_bits(y)
    if in_place:
        y1[:, :heads * d] = y0[:, :heads * d]
    assert np.array_equal(y1, y0)
    kc1, vc1 = host_bits(kc), host_bits(vc)
    for t in range(T):
        s = int(slots[t])
        if not 0 <= s < blocks * size:
            continue
        b, o = s // size, s % size
        got = oracle.as_f64(kc1[b, :, o])
        assert np.all(np.abs(got - want[t, heads:heads + kv]) <= near[t, heads:heads + kv])
        assert np.array_equal(vc1[b, :, o], y0[t, (heads + kv) * d:(heads + 2 * kv) * d].reshape(kv, d))
        kc1[b, :, o], vc1[b, :, o] = kc0[b, :, o], vc0[b, :, o]
    assert np.array_equal(kc1, kc0) and np.array_equal(vc1, vc0)  # nothing else was written


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,heads,kv,d,rot,size", [(1, 8, 2, 64, 64, 16), (1, 64, 16, 128, 128, 16), (3, 4, 4, 128, 64, 32),
                                                   (64, 20, 1, 64, 48, 64), (65, 7, 7, 128, 112, 128), (2, 3, 1, 64, 16, 16),
                                                   (5, 6, 2, 128, 0, 16), (200, 71, 1, 64, 32, 16), (9, 0, 3, 64, 64, 16)])
def test_rope(h, T, heads, kv, d, rot, size, inter):
    rope_case(h, T, heads, kv, d, rot, inter, size, wide=8 * (T % 3))


@pytest.mark.parametrize("scaling,factor,mag", [("none", 1.0, 1.0), ("linear", 4.0, 1.0), ("ntk", 8.0, 1.0),
                                                ("bands", 8.0, 1.0), ("yarn", 40.0, 0.1 * np.log(40.0) + 1.0),
                                                ("yarn", 1.0, 1.0)])
def test_rope_scalings_at_far_positions(h, scaling, factor, mag):
    far = [0, 1, 2, 8191, 8192, 1 << 20, (1 << 24) + 1, (1 << 30) + 12345, -3]
    rope_case(h, 9, 4, 2, 128, 96, False, 16, scaling, factor, mag, positions=far)
    rope_case(h, 9, 4, 2, 64, 64, True, 16, scaling, factor, mag, positions=far)


def test_rope_in_place_and_rows_without_a_slot(h):
    bad = [(0, -1), (3, -7), (5, 1 << 30), (6, 16 * 3), (7, 2 ** 31 - 1)]
    rope_case(h, 12, 6, 2, 64, 64, False, 16, in_place=True, bad=bad[:3])
    rope_case(h, 12, 6, 2, 128, 64, True, 16, in_place=True, bad=bad)


def test_rope_phases_are_exact(h):
    import moe_layers_gb300 as ML
    for scaling, factor in (("none", 1.0), ("linear", 3.0), ("ntk", 5.0), ("bands", 8.0), ("yarn", 16.0)):
        r = ML.Rope(h, 128, base=500000.0, scaling=scaling, factor=factor)
        got = r.phases.cpu().numpy().view(np.uint64).astype(np.float64) / 2.0 ** 64
        want = oracle.rope_frequencies(128, 500000.0, scaling, factor, high=32.0 if scaling == "yarn" else 4.0) / (2 * np.pi)
        assert np.all(np.abs(got - want) <= want * 2.0 ** -46 + 2.0 ** -64)


def test_rope_cache_offsets_past_32_bits(h):
    """A pool whose last block begins past 2^32 elements."""
    import torch
    import moe_layers_gb300 as ML
    kv, size, d = 2, 16, 64
    blocks = 2200000
    pool = torch.empty((blocks, kv, size, d), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 32
    x = bf16(np.random.default_rng(0).standard_normal((2, 3 * kv * d)))
    r = ML.Rope(h, 0)
    slots = [blocks * size - 1, 5]
    ML.dec_rope_append(h, r, None, x[:, :kv * d], x[:, kv * d:2 * kv * d], i32([1, 2]), i32(slots), ML.KvCache(pool, pool))
    torch.cuda.synchronize()
    # v is written after or before k into the same pool: either row is one of the two
    for t, s in enumerate(slots):
        got = host_bits(pool[s // size, :, s % size])
        rows = [host_bits(x[t, a:a + kv * d]).reshape(kv, d) for a in (0, kv * d)]
        assert np.all((got == rows[0]) | (got == rows[1]))
    del pool
    torch.cuda.empty_cache()


# ---------------------------------------------------------------------------- attention
class Case:
    """A batch over a paged cache whose unused places hold NaN and infinities."""

    def __init__(self, new, own, heads, kv, d, size, prefix=0, pad=0, seed=0, sharp=1.0, extra_blocks=0, wide=0):
        rng = np.random.default_rng(seed)
        self.new, self.own, self.heads, self.kv, self.d, self.size, self.prefix = new, own, heads, kv, d, size, prefix
        n = len(new)
        held = [-(-max(o, 0) // size) for o in own]
        ahead = -(-prefix // size)
        self.blocks = sum(held) + ahead + 2
        order = rng.permutation(self.blocks)
        self.table = np.full((n, max(max(held), 1) + extra_blocks), -1)
        at = ahead
        for b in range(n):
            self.table[b, :held[b]] = order[at:at + held[b]]
            at += held[b]
        self.prefix_table = order[:ahead]
        self.row_start = np.concatenate([[0], np.cumsum(new)])
        self.M = int(self.row_start[-1]) + pad
        junk = np.array([np.nan, np.inf, -np.inf, 3e38])
        shape = (self.blocks, kv, size, d)
        k, v = junk[rng.integers(0, 4, shape)], junk[rng.integers(0, 4, shape)]

        def fill(table, length):
            for j in range(length):
                blk, o = table[j // size], j % size
                k[blk, :, o], v[blk, :, o] = rng.standard_normal((kv, d)), rng.standard_normal((kv, d))

        fill(self.prefix_table, prefix)
        for b in range(n):
            fill(self.table[b], max(own[b], 0))
        self.k, self.v = bf16(k), bf16(v)
        self.wide = wide
        self.q = bf16(sharp * rng.standard_normal((max(self.M, 1), heads * d + wide)))[:, :heads * d]
        self.scale = d ** -0.5

    def run(self, h, stream=None, ws=None, scale=None):
        import torch
        import moe_layers_gb300 as ML
        out = torch.full((self.q.shape[0], self.heads * self.d + self.wide), 7.5, dtype=torch.bfloat16, device="cuda")
        self.batch = ML.Batch(i32(self.row_start), i32(self.own), i32(self.table), max_new=max(max(self.new), 1),
                              prefix_table=i32(self.prefix_table) if self.prefix else None, prefix_len=self.prefix)
        self.cache = ML.KvCache(self.k, self.v)
        ML.dec_attention(h, self.q, self.cache, self.batch, scale or self.scale, out=out[:, :self.heads * self.d],
                         stream=stream, ws=ws)
        torch.cuda.synchronize()
        assert np.all(oracle.as_f64(host_bits(out[:, self.heads * self.d:])) == 7.5)
        return host_bits(out[:, :self.heads * self.d]).reshape(-1, self.heads, self.d)

    def want(self):
        return oracle.attention(host_bits(self.q).reshape(-1, self.heads, self.d), host_bits(self.k), host_bits(self.v),
                                self.row_start, self.own, self.table, self.scale, self.prefix_table, self.prefix)

    def check(self, bits, reference=None):
        want, spread, reach = (reference or Case.want)(self)
        got = oracle.as_f64(bits)
        used = ~np.isnan(want[:, 0, 0])
        assert np.all(got[~used] == 7.5)  # rows of no request
        keys = self.prefix + max(max(self.own), 0)
        score = self.d * 2.0 ** -23 * reach[..., None]
        tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * score + keys * 2.0 ** -23 + 2.0 ** -20)
        err = np.abs(got - want)
        assert np.all(err[used] <= tol[used] * 1.01), float(np.max(err[used] - tol[used]))
        return got, want


def reference64(c):
    """Like oracle.attention, in float64 on the GPU (elementary operations, one request at a time), for
    cases that are long for a loop over rows on the host. Returns (out, sum p |v|, reach)."""
    import torch
    k, v = (torch.nan_to_num(t.double(), 0.0, 0.0, 0.0) for t in (c.k, c.v))
    q = c.q.double().reshape(-1, c.kv, c.heads // c.kv, c.d)
    shape = (q.shape[0], c.heads, c.d)
    out, spread = np.full(shape, np.nan), np.zeros(shape)
    reach = np.zeros(shape[:2])
    for b, n in enumerate(c.new):
        if not n:
            continue
        place = [(int(c.prefix_table[j // c.size]), j % c.size, -1) for j in range(c.prefix)]
        place += [(int(c.table[b][j // c.size]), j % c.size, j) for j in range(c.own[b])]
        blk, off, own = torch.tensor([p for p in place if 0 <= p[0] < c.blocks], device="cuda").T
        first = int(c.row_start[b])
        kk, vv, qq = k[blk, :, off], v[blk, :, off], q[first:first + n]
        s = torch.einsum("tkgd,nkd->tkgn", qq, kk) * c.scale
        last = c.own[b] - n + torch.arange(n, device="cuda")
        s = s.masked_fill((own[None, :] > last[:, None])[:, None, None, :], -np.inf)
        p = torch.softmax(s, -1)
        out[first:first + n] = torch.einsum("tkgn,nkd->tkgd", p, vv).reshape(n, c.heads, c.d).cpu().numpy()
        spread[first:first + n] = torch.einsum("tkgn,nkd->tkgd", p, vv.abs()).reshape(n, c.heads, c.d).cpu().numpy()
        far = torch.einsum("tkgd,nkd->tkgn", qq.abs(), kk.abs()).amax(-1) * c.scale
        reach[first:first + n] = far.reshape(n, c.heads).cpu().numpy()
    return out, spread, reach


LAYOUTS = [(8, 2, 64), (8, 2, 128), (4, 4, 128), (6, 1, 64), (20, 1, 128), (3, 3, 64), (40, 2, 128)]


@pytest.mark.parametrize("heads,kv,d", LAYOUTS)
@pytest.mark.parametrize("size", [16, 64])
def test_attention_single_tokens(h, heads, kv, d, size):
    own = [1, 2, 15, 16, 17, 63, 64, 65, 127, 128, 129, 300]
    c = Case([1] * len(own), own, heads, kv, d, size, pad=2, seed=heads + d)
    c.check(c.run(h))


@pytest.mark.parametrize("own", [1, 16, 17, 64, 100, 1000, 2049])
@pytest.mark.parametrize("size", [16, 32, 64, 128])
def test_attention_one_request(h, own, size):
    c = Case([1], [own], 8, 2, 128, size, seed=own, wide=16)
    c.check(c.run(h))


@pytest.mark.parametrize("heads,kv,d", LAYOUTS)
@pytest.mark.parametrize("prefix", [1, 16, 50, 128, 777])
def test_attention_shared_prefix(h, heads, kv, d, prefix):
    own = [1, 5, 16, 33, 64, 130, 2]
    c = Case([1] * len(own), own, heads, kv, d, 16, prefix=prefix, pad=1, seed=prefix + d)
    c.check(c.run(h))


@pytest.mark.parametrize("M", [1, 2, 3, 8, 31, 32, 33, 63, 64])
@pytest.mark.parametrize("heads,kv,d", [(8, 2, 128), (8, 1, 64), (12, 3, 128)])
def test_attention_prefix_batches(h, M, heads, kv, d):
    rng = np.random.default_rng(M)
    c = Case([1] * M, [int(x) for x in rng.integers(1, 90, M)], heads, kv, d, 32, prefix=600 + M, seed=M)
    c.check(c.run(h))


@pytest.mark.parametrize("heads,kv,d,new", [(8, 2, 128, 2), (8, 2, 64, 4), (8, 2, 128, 8), (8, 2, 64, 8), (8, 2, 128, 16),
                                            (4, 1, 64, 30), (8, 2, 128, 64), (16, 1, 64, 64), (2, 2, 128, 8)])
@pytest.mark.parametrize("prefix", [0, 70])
def test_attention_later_tokens_that_are_not_finite(h, heads, kv, d, new, prefix):
    """Infinities and NaN in k and v of a step's own tokens reach the rows that see them alone: the rows
    before are as without them, and in those behind, an element of v only its own column."""
    n = min(4, 64 // new)
    own = [127 + new, 120 + new // 2, new, 1000][:n]  # the new tokens begin and end in all parts of a tile
    c = Case([new] * n, own, heads, kv, d, 16, prefix=prefix, seed=new + d)
    rng = np.random.default_rng(new)
    planted = np.zeros((c.M, heads, d), dtype=bool)
    sick = np.zeros(c.M, dtype=bool)  # rows that see a NaN score
    values = []
    for b in range(n):
        for i in {0, 1, new // 2, new - 1}:
            j, g, col = own[b] - new + i, int(rng.integers(kv)), int(rng.integers(d))
            at = (int(c.table[b][j // 16]), g, j % 16)
            values.append((at, col, (np.inf, -np.inf, np.nan)[(i + b) % 3]))
            first = int(c.row_start[b]) + i
            planted[first:int(c.row_start[b + 1]), g * heads // kv:(g + 1) * heads // kv, col] = True
    for at, col, _ in values:
        c.v[at][col] = 0.0
    want, spread, reach = c.want()
    for at, col, x in values:
        c.v[at][col] = x
    j = own[-1] - 1  # the last row of the last request sees a key of NaN
    c.k[int(c.table[-1][j // 16]), :, j % 16] = float("nan")
    sick[-1] = True
    got = oracle.as_f64(c.run(h))
    assert np.all(np.isnan(got[sick]))
    assert not np.any(np.isfinite(got[planted & ~sick[:, None, None]]))
    ok = ~planted & ~sick[:, None, None]
    score = d * 2.0 ** -23 * reach[..., None]
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2 * score + (prefix + 1000) * 2.0 ** -23 + 2.0 ** -20)
    assert np.all((np.abs(got - want) <= tol * 1.01)[ok])


@pytest.mark.parametrize("heads,kv,d", [(8, 2, 128), (4, 1, 64), (16, 16, 64), (64, 4, 128)])
@pytest.mark.parametrize("new", [[8] * 8, [3, 1, 7, 0, 16], [64], [33, 31], [2] * 5, [1, 0, 0, 1]])
@pytest.mark.parametrize("prefix", [0, 70])
def test_attention_drafts(h, heads, kv, d, new, prefix):
    rng = np.random.default_rng(len(new))
    own = [n + int(rng.integers(0, 200)) for n in new]
    own[0] = new[0]  # a first chunk: the first row sees itself alone
    c = Case(new, own, heads, kv, d, 16, prefix=prefix, seed=5)
    c.check(c.run(h))


def test_attention_rows_that_see_nothing(h):
    """own_len 0 or short of the rows, holes in the table: zeros, and no NaN from the junk around."""
    c = Case([1, 4, 1, 2, 1], [0, 2, -3, 40, 20], 8, 2, 64, 16, seed=3)
    c.table[3, 1:] = -1
    c.table[4, 0] = c.blocks  # past the cache
    got, want = c.check(c.run(h))
    assert np.all(got[0] == 0) and np.all(got[1] == 0) and np.all(got[2] == 0) and np.any(got[3] != 0)
    c = Case([1, 4, 1], [0, 2, 0], 8, 2, 64, 16, prefix=19, seed=3)
    got, want = c.check(c.run(h))
    assert np.any(got[0] != 0)


def test_attention_block_ids_out_of_range(h):
    """Entries outside the cache are not there, in the prefix as well: nothing is read through them."""
    for bad in (-1, 1 << 30, -(1 << 31), 2 ** 31 - 1):
        c = Case([1, 2], [300, 200], 8, 2, 128, 16, prefix=100, seed=9)
        c.table[0, [0, 7, 18]] = bad
        c.table[1, 3:9] = bad
        c.prefix_table[2] = bad
        c.check(c.run(h))


def test_attention_lengths_past_the_table(h):
    """own_len beyond max_blocks blocks: the tokens past the table are not there."""
    c = Case([1, 1], [64, 40], 4, 2, 64, 16, seed=2)
    c.own = [1 << 30, 2 ** 31 - 1]
    c.table[1, 3:] = -1
    # request 1's third block is part full: give its tail values
    import torch
    c.k[c.table[1, 2], :, 8:] = 0
    c.v[c.table[1, 2], :, 8:] = 0
    torch.cuda.synchronize()
    got = oracle.as_f64(c.run(h))
    c.own = [64, 48]
    want, spread, reach = c.want()
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2.0 ** -12)
    assert np.all(np.abs(got - want) <= tol)


@pytest.mark.parametrize("prefix", [0, 100])
def test_attention_finds_one_key(h, prefix):
    """A key that outweighs all others by e^60: the output is its value to one rounding, at every
    place of the visible tokens; the same key one place behind the last visible token changes nothing."""
    import torch
    own, d, size = 150, 64, 16
    c = Case([1], [own], 4, 2, d, size, prefix=prefix, seed=1, extra_blocks=1)
    base = c.run(h)
    k0, v0 = c.k.clone(), c.v.clone()
    q = oracle.as_f64(host_bits(c.q)).reshape(4, d)
    for place in list(range(0, prefix + own, 7)) + [prefix - 1, prefix, prefix + own - 1]:
        if place < 0:
            continue
        t, j = (c.prefix_table, place) if place < prefix else (c.table[0], place - prefix)
        for kvh in (0, 1):
            direction = q[2 * kvh] / (q[2 * kvh] @ q[2 * kvh])
            c.k[t[j // size], kvh, j % size] = bf16(direction * 70.0 / c.scale)
        got = oracle.as_f64(c.run(h))
        for g in (0, 2):
            want = oracle.as_f64(host_bits(c.v[t[j // size], g // 2, j % size]))
            assert np.all(np.abs(got[0, g] - want) <= 2.0 ** -8 * np.abs(want) + 1e-9), place
        c.k.copy_(k0)
    j = own  # the first place behind the last token, in a part-full block
    c.k[c.table[0][j // size], :, j % size] = 1000.0
    assert np.array_equal(c.run(h), base)
    torch.cuda.synchronize()


def test_attention_large_scores_do_not_overflow(h):
    c = Case([1, 2, 1], [300, 77, 64], 8, 2, 128, 16, prefix=200, seed=4, sharp=60.0)
    got = oracle.as_f64(c.run(h))
    want, spread, reach = c.want()
    # scores up to about 1000: off by D 2^-23 of reach, p by a factor e^that
    score = 128 * 2.0 ** -23 * reach[..., None]
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2.0 ** -9) + 2 * score * np.abs(host_max(c))
    assert np.all(np.isfinite(got)) and np.all(np.abs(got - want) <= tol)


def host_max(c):
    v = oracle.as_f64(host_bits(c.v))
    return np.max(np.abs(v[np.isfinite(v) & (np.abs(v) < 100)]))


def test_attention_same_bits_again_and_on_another_stream(h):
    import torch
    c = Case([1] * 20, list(range(30, 830, 40)), 16, 4, 128, 16, prefix=500, seed=6)
    first = c.run(h)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    assert np.array_equal(c.run(h), first)
    assert np.array_equal(c.run(h, stream=s), first)


def test_attention_two_calls_at_once(h):
    """Two streams, two workspaces: neither disturbs the other."""
    import torch
    import moe_layers_gb300 as ML
    cs = [Case([1] * 12, list(range(900, 1500, 50)), 16, 4, 128, 16, prefix=p, seed=p) for p in (0, 900)]
    alone = [c.run(h) for c in cs]
    streams = [torch.cuda.Stream() for _ in cs]
    outs = [[torch.full((12, 16 * 128), 7.5, dtype=torch.bfloat16, device="cuda") for _ in range(10)] for _ in cs]
    torch.cuda.synchronize()
    for i in range(10):
        for c, s, o in zip(cs, streams, outs):
            with torch.cuda.stream(s):
                ML.dec_attention(h, c.q, c.cache, c.batch, c.scale, out=o[i])
    torch.cuda.synchronize()
    for a, o in zip(alone, outs):
        for x in o:
            assert np.array_equal(host_bits(x).reshape(a.shape), a)


def test_attention_under_a_graph_with_new_lengths(h):
    import torch
    import moe_layers_gb300 as ML
    c = Case([1] * 9, list(range(20, 200, 20)), 8, 2, 64, 16, prefix=130, seed=8)
    c.run(h)
    out = torch.full((9, 8 * 64), 7.5, dtype=torch.bfloat16, device="cuda")
    side = torch.cuda.Stream()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=side):
        ML.dec_attention(h, c.q, c.cache, c.batch, c.scale, out=out)
    for k in (0, 3):
        c.own = [x - k for x in range(20, 200, 20)]
        c.batch.own_len.copy_(i32(c.own))
        g.replay()
        torch.cuda.synchronize()
        c.check(host_bits(out).reshape(9, 8, 64))


@pytest.mark.parametrize("heads,kv,d,M", [(32, 32, 128, 64), (128, 8, 64, 64), (8, 2, 64, 9)])
def test_two_graphs_at_once(h, heads, kv, d, M):
    """Captured calls with a workspace each, replayed on two streams at the same time, many times."""
    import torch
    import moe_layers_gb300 as ML
    prefix = 6085 if kv == 32 else 1600
    cs = [Case([1] * M, [3 + (7 * i + s) % 60 for i in range(M)], heads, kv, d, 16, prefix=prefix, seed=s) for s in (0, 1)]
    alone = [c.run(h) for c in cs]
    # a graph keeps addresses, not tensors: its workspace and output stay alive here
    outs, spaces, graphs, streams = [], [], [], [torch.cuda.Stream() for _ in cs]
    for c in cs:
        out = torch.zeros((M, heads * d), dtype=torch.bfloat16, device="cuda")
        ws = torch.empty(ML.dec_attention_workspace_size(h, M, heads, c.cache, c.batch), dtype=torch.uint8, device="cuda")
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ML.dec_attention(h, c.q, c.cache, c.batch, c.scale, out=out, ws=ws)
        outs.append(out)
        spaces.append(ws)
        graphs.append(g)
    for _ in range(20):
        for o in outs:
            o.zero_()
        torch.cuda.synchronize()
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, want in zip(outs, alone):
            assert np.array_equal(host_bits(o).reshape(want.shape), want)


@pytest.mark.parametrize("prefix", [0, 40])
def test_attention_of_an_idle_batch(h, prefix):
    """No request has a row: nothing is written."""
    c = Case([0, 0, 0], [5, 0, 90], 8, 2, 64, 16, prefix=prefix, pad=3, seed=1)
    assert np.all(oracle.as_f64(c.run(h)) == 7.5)


def test_attention_long_context_offsets(h):
    """A cache whose blocks lie past 2^32 elements."""
    import torch
    import moe_layers_gb300 as ML
    kv, size, d, own = 2, 64, 128, 700
    blocks = 300000
    k = torch.zeros((blocks, kv, size, d), dtype=torch.bfloat16, device="cuda")
    assert k.numel() > 1 << 32
    rng = np.random.default_rng(0)
    v = torch.zeros_like(k)
    ids = [blocks - 1 - 7 * i for i in range(11)]
    small = Case([1], [own], 4, kv, d, size, seed=12)
    for i, b in enumerate(ids):
        k[b], v[b] = small.k[small.table[0, i]], small.v[small.table[0, i]]
    want = small.run(h)
    out = torch.full((1, 4 * d), 7.5, dtype=torch.bfloat16, device="cuda")
    batch = ML.Batch(i32([0, 1]), i32([own]), i32([ids]))
    ML.dec_attention(h, small.q, ML.KvCache(k, v), batch, small.scale, out=out)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(out).reshape(1, 4, d), want)
    del k, v
    torch.cuda.empty_cache()


@pytest.mark.parametrize("heads,kv,d,M,prefix", [(64, 32, 64, 32, 6100), (32, 32, 128, 64, 6085), (128, 8, 64, 64, 1600),
                                                 (64, 8, 128, 40, 5003), (16, 16, 128, 64, 16000), (64, 16, 128, 24, 20000),
                                                 (64, 16, 128, 64, 12345), (32, 4, 64, 63, 30001)])
def test_attention_large_prefix_work(h, heads, kv, d, M, prefix):
    """Enough prefix for the tensor-memory kernel and a launch apart for the own tokens: one and two streams,
    a few tiles a CTA and many; the same bits every time."""
    rng = np.random.default_rng(M)
    c = Case([1] * (M - 1) + [0], [int(x) for x in rng.integers(1, 70, M)], heads, kv, d, 16, prefix=prefix, pad=1, seed=M,
             sharp=2.5)
    c.prefix_table[3] = c.blocks + 5  # one block of the prefix is not there
    first = c.run(h)
    got, want = c.check(first, reference64)
    used = slice(0, M - 1)
    # both roundings are independent and at most 2^-8 of each term: 2^0.5 2^-8 in the 2-norm
    assert np.linalg.norm((got - want)[used]) <= 2.0 ** -7.5 * np.linalg.norm(want[used])
    for _ in range(5):
        assert np.array_equal(c.run(h), first)


@pytest.mark.parametrize("heads,kv,d,new,own", [(64, 32, 128, [24], [8000]), (64, 16, 128, [64], [9000]),
                                                (40, 1, 64, [1] * 16, [5000 + 77 * i for i in range(16)]),
                                                (64, 8, 64, [16, 9, 0, 20], [12000, 30, 500, 7000])])
def test_attention_many_rows_on_long_contexts(h, heads, kv, d, new, own):
    """More than 32 rows of one request to a key head: the tensor-memory kernel on own tokens, many tiles a CTA."""
    c = Case(new, own, heads, kv, d, 32, seed=sum(new), sharp=2.5)
    first = c.run(h)
    c.check(first, reference64)
    for _ in range(5):
        assert np.array_equal(c.run(h), first)


@pytest.mark.parametrize("heads,kv,d,M", [(1024, 128, 64, 2), (128, 1, 64, 3), (128, 1, 128, 64), (1024, 8, 64, 1)])
def test_attention_many_heads(h, heads, kv, d, M):
    c = Case([1] * M, [40 + i for i in range(M)], heads, kv, d, 32, prefix=70, seed=heads + M)
    c.check(c.run(h))


def test_attention_row_lengths_at_the_int_limit(h):
    """own_len near 2^31 with several rows: each sees the whole table."""
    c = Case([4], [64], 4, 2, 64, 16, seed=2)
    c.own = [2 ** 31 - 1]
    got = oracle.as_f64(c.run(h))
    want, spread, reach = c.want()
    tol = 2.0 ** -8 * np.abs(want) + spread * (2.0 ** -8 + 2.0 ** -12)
    assert np.all(np.abs(got - want) <= tol)


def test_attention_without_dependent_launches_and_while_profiling(h):
    """The same bits with kernels strictly one after another."""
    for prefix, heads, M in ((0, 8, 9), (90, 8, 9), (6085, 32, 64)):
        c = Case([1] * M, [30 + 5 * i for i in range(M)], heads, 32 if heads == 32 else 2, 64, 16, prefix=prefix, seed=M)
        first = c.run(h)
        h.set_pdl(False)
        assert np.array_equal(c.run(h), first)
        h.set_pdl(True)
        h.set_profiling(True)
        assert np.array_equal(c.run(h), first)
        tags = h.profile_read()
        h.set_profiling(False)
        assert "attention" in tags and ("attention_prefix" in tags) == (prefix == 6085)


def test_attention_single_row_of_any_stride(h):
    import torch
    import moe_layers_gb300 as ML
    c = Case([1], [50], 4, 2, 64, 16, seed=3)
    want = c.run(h)
    odd = torch.zeros((1, 4 * 64 + 3), dtype=torch.bfloat16, device="cuda")
    odd[:, :256] = c.q
    got = ML.dec_attention(h, odd[:, :256], c.cache, c.batch, c.scale)
    torch.cuda.synchronize()
    assert np.array_equal(host_bits(got).reshape(1, 4, 64), want)


def test_outputs_made_on_the_stream_of_the_call(h):
    """Without an output tensor, the zeros of idle rows and the result belong to the call's stream."""
    import torch
    import moe_layers_gb300 as ML
    c = Case([1, 0, 1], [500, 7, 300], 8, 2, 64, 16, pad=2, seed=7)
    want = c.run(h)
    want[2:] = 0
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    ML.test_occupy_sms(h, 8, 20_000_000)  # the current stream is busy meanwhile
    got = ML.dec_attention(h, c.q, c.cache, c.batch, c.scale, stream=s)
    s.synchronize()
    assert np.array_equal(host_bits(got).reshape(want.shape), want)


def test_operators_together(h):
    """Three decode steps of a small batch: tables, rotary positions with the cache write, attention,
    against the oracle's own chain; the cache is written by the operators alone."""
    import torch
    import moe_layers_gb300 as ML
    rng = np.random.default_rng(21)
    heads, kv, d, size, prefix, n, blocks = 8, 2, 64, 16, 21, 5, 40
    kc, vc = bf16(rng.standard_normal((blocks, kv, size, d))), bf16(rng.standard_normal((blocks, kv, size, d)))
    ids = [int(x) for x in rng.permutation(blocks)]
    prefix_table, ids = ids[:2], ids[2:]
    table, ctx, count, free = np.full((n, 4), -1), np.zeros(n, int), len(ids), ids
    d_table, d_free = i32(table), i32(free)
    rope, freq = ML.Rope(h, 32, base=10000.0), oracle.rope_frequencies(32, 10000.0)
    host_k, host_v = host_bits(kc), host_bits(vc)
    for new in ([5, 1, 0, 14, 2], [1, 1, 1, 1, 1], [2, 0, 4, 3, 1]):
        T = sum(new) + 2
        y = bf16(rng.standard_normal((T, (heads + 2 * kv) * d)))
        step = ML.dec_batch_tables(h, i32(ctx), i32(new), d_free, i32([count]), d_table, size, rows=T,
                                   position_offset=prefix)
        q = ML.dec_rope_append(h, rope, y[:, :heads * d], y[:, heads * d:(heads + kv) * d], y[:, (heads + kv) * d:],
                               step.positions, step.slots, ML.KvCache(kc, vc))
        batch = ML.Batch(step.row_start, step.own_len, d_table, max_new=max(new), prefix_table=i32(prefix_table),
                         prefix_len=prefix)
        out = ML.dec_attention(h, q, ML.KvCache(kc, vc), batch, d ** -0.5)
        torch.cuda.synchronize()
        want = oracle.batch_tables(ctx, new, free, count, table, size, prefix, T)
        table, ctx, count = want["table"], want["own_len"], int(want["left"][0])
        x = oracle.as_f64(host_bits(y)).reshape(T, heads + 2 * kv, d)
        turned = oracle.round_bf16(oracle.rope(x, want["positions"], freq))
        got_k, got_v = host_bits(kc), host_bits(vc)
        for t in range(sum(new)):
            s = want["slots"][t]
            b, o = s // size, s % size
            assert np.all(np.abs(oracle.as_f64(got_k[b, :, o]) - turned[t, heads:heads + kv]) <=
                          2.0 ** -7 * np.abs(turned[t, heads:heads + kv]) + 2.0 ** -16)
            assert np.array_equal(got_v[b, :, o], host_bits(y).reshape(T, -1, d)[t, heads + kv:])
            host_k[b, :, o], host_v[b, :, o] = got_k[b, :, o], got_v[b, :, o]
        assert np.array_equal(got_k, host_k) and np.array_equal(got_v, host_v)
        ref, spread, reach = oracle.attention(host_bits(q).reshape(T, heads, d), got_k, got_v, want["row_start"], ctx,
                                              table, d ** -0.5, prefix_table, prefix)
        got = oracle.as_f64(host_bits(out)).reshape(T, heads, d)
        used = slice(0, sum(new))
        tol = 2.0 ** -8 * np.abs(ref) + spread * (2.0 ** -8 + 2.0 ** -12 + 2 * d * 2.0 ** -23 * reach[..., None])
        assert np.all(np.abs(got - ref)[used] <= tol[used])
        assert np.all(got[sum(new):] == 0)


def test_tables_with_an_empty_free_list(h):
    """A free list without elements is a list that is used up: requests within their blocks go on, others get -1."""
    check_tables(h, [3, 16, 0], [2, 1, 4], [], 0, [[1, -1], [2, -1], [-1, -1]], 16, 5, 9)
    check_tables(h, [3], [2], [], 0, [[1, -1]], 16, 0, 2)
    check_tables(h, [0] * 3, [3000, 1, 2000], [], 0, np.full((3, 200), 7), 16, 0, 5010)


# own tokens, with and without a prefix, and a prefix with one own token a row; one and two streams
@pytest.mark.parametrize("heads,kv,d,new,more,prefix", [(64, 16, 128, [16] * 3, 700, 0), (64, 16, 128, [64], 700, 500),
                                                        (8, 2, 64, [30], 700, 0), (32, 32, 128, [1] * 64, 1, 6085)])
def test_attention_averages_equal_values_to_that_value(h, heads, kv, d, new, more, prefix):
    """In the tensor-memory kernel, whatever the weights are, their average of one value is that value, exactly:
    the weights that are summed are the rounded ones that are multiplied. (fp32 sums of at most 7000 terms are
    off by less than 2^-11, and 255/128 would round to its neighbour 2^-9 away. A single own token has weight 1.)"""
    for seed, sharp in ((1, 1.0), (2, 4.0), (3, 12.0)):
        rng = np.random.default_rng(seed)
        own = [n + int(rng.integers(0, more)) for n in new]
        c = Case(new, own, heads, kv, d, 16, prefix=prefix, seed=seed, sharp=sharp)
        values = 255.0 / 128 * np.exp2(rng.integers(-3, 4, d)) * rng.choice([-1.0, 1.0], d)
        c.v[:] = bf16(values)
        wrong = np.sum(oracle.as_f64(c.run(h)) != values)
        assert wrong == 0


@pytest.mark.parametrize("heads,kv,d,new,prefix", [(8, 2, 128, [1] * 5, 0), (8, 2, 64, [1] * 5, 200), (16, 1, 128, [1] * 3, 0),
                                                   (32, 1, 64, [1] * 3, 300), (8, 2, 128, [16] * 2, 100), (8, 2, 64, [30], 0),
                                                   (32, 32, 128, [1] * 64, 6085)])
@pytest.mark.parametrize("scale", [1e4, 1e9, 1e12, 1e30])
def test_attention_of_huge_scores_takes_the_largest(h, heads, kv, d, new, prefix, scale):
    """Scores far apart (a large scale): the output is the value of the largest score's key, or, where keys
    are the same, the mean of theirs. q and k hold small whole numbers, so that scores are exact in fp32 and
    the gap between two of them is at least 1 before the scale."""
    rng = np.random.default_rng(len(new) + prefix)
    own = [n + int(rng.integers(0, 400)) for n in new]
    c = Case(new, own, heads, kv, d, 16, prefix=prefix, seed=prefix + d)
    c.q[:] = bf16(rng.integers(-40, 41, tuple(c.q.shape)))
    c.k[:] = bf16(rng.integers(-40, 41, tuple(c.k.shape)))
    c.scale = scale
    got = oracle.as_f64(c.run(h))
    want, spread, _ = reference64(c)
    # the mean of equally large scores: weights of 1 are exact, one rounding of the output, fp32 sums
    assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + spread * 2.0 ** -20)


def test_attention_of_large_values(h):
    """Scores of 10^12 from large q and k, with the usual scale: as above."""
    rng = np.random.default_rng(3)
    for new, heads, prefix in (([1] * 4, 8, 130), ([16, 16], 16, 0)):
        c = Case(new, [n + 150 for n in new], heads, 2, 64, 16, prefix=prefix, seed=3)
        c.q[:] = bf16(rng.integers(-40, 41, tuple(c.q.shape)) * 2.0 ** 14)
        c.k[:] = bf16(rng.integers(-40, 41, tuple(c.k.shape)) * 2.0 ** 14)
        got = oracle.as_f64(c.run(h))
        want, spread, _ = reference64(c)
        assert np.all(np.abs(got - want) <= 2.0 ** -8 * np.abs(want) + spread * 2.0 ** -20)


@pytest.mark.parametrize("prefix,heads,kv,d", [(0, 8, 2, 64), (500, 8, 2, 64), (6085, 32, 32, 128)])
@pytest.mark.parametrize("start,same", [([0, 20, 12], [0, 12, 12]), ([5, 2, 30], [5, 5, 30]), ([4, 30, 10], [4, 10, 10]),
                                        ([-9, 3, 99], [0, 3, 40]), ([3, 40, 39], [3, 39, 39]), ([20, 3, 0], [20, 20, 20])])
def test_attention_row_starts_out_of_order(h, prefix, heads, kv, d, start, same):
    """Rows at and behind row_start[requests] belong to no request, and none before row_start[0] does,
    whatever lies between."""
    c = Case([40, 0], [300, 200], heads, kv, d, 16, prefix=prefix, seed=1)
    got = []
    for s in (same, start):
        c.row_start = s
        got.append(c.run(h))
    assert np.array_equal(got[0], got[1])
    idle = oracle.as_f64(got[0]) == 7.5
    assert np.all(idle[:max(same[0], 0)]) and np.all(idle[same[2]:]) and not np.any(np.all(idle[same[0]:same[2]], (1, 2)))


def test_rope_places_in_a_pool_past_32_bits(h):
    """k and v interleaved in one pool of more than 2^32 elements: both at their slots, exactly, and nothing where a
    wrapped offset or the other one's place would be."""
    import torch
    import moe_layers_gb300 as ML
    kv, size, d = 2, 16, 64
    blocks, per = 1200000, 2 * 16 * 64  # elements of one block of k, and of v
    pool = torch.empty((blocks, 2, kv, size, d), dtype=torch.bfloat16, device="cuda")
    assert pool.numel() > 1 << 32
    pool.view(torch.int16).fill_(0x1234)
    x = bf16(np.random.default_rng(0).standard_normal((4, 2 * kv * d)))
    far = (1 << 32) // (2 * per)  # the block that begins at element 2^32
    slots = [blocks * size - 1, 5, far * size + 3, (far - 1) * size + 15]
    r = ML.Rope(h, 0)
    ML.dec_rope_append(h, r, None, x[:, :kv * d], x[:, kv * d:], i32([1, 2, 3, 4]), i32(slots),
                       ML.KvCache(pool[:, 0], pool[:, 1]))
    torch.cuda.synchronize()
    for t, s in enumerate(slots):
        place = pool[s // size, :, :, s % size].view(torch.int16)  # [k or v][head][element]
        assert torch.equal(place.reshape(-1), x[t].view(torch.int16))
        place.fill_(0x1234)
    for part in pool.view(torch.int16).split(100000):
        assert bool((part == 0x1234).all())
    del pool, place, part
    torch.cuda.empty_cache()


def tables_in_place(h, rows, offsets, seed):
    """A step whose own_len lies over ctx_len and whose left over free_count, with outputs that begin at `offsets`
    4-byte words behind a 16-byte boundary."""
    import torch
    import moe_layers_gb300 as ML
    rng = np.random.default_rng(seed)
    n, size = 60, 16
    ctx = rng.integers(0, 400, n)
    new = rng.multinomial(rows - 5, np.ones(n) / n)
    new[3] = 0
    width = -(-int((ctx + new).max()) // size)
    ids = rng.permutation(n * width)
    table = np.full((n, width), -1)
    at = 0
    for b in range(n):
        m = -(-int(ctx[b]) // size)
        table[b, :m] = ids[at:at + m]
        at += m
    free = ids[at:]
    count = len(free) if seed % 2 else 50  # plenty, or used up in the middle

    def words(k, values, fill):
        buf = torch.full((len(values) + 8,), fill, dtype=torch.int32, device="cuda")
        view = buf[k:k + len(values)]
        view.copy_(i32(values))
        return buf, view

    bufs, views = zip(*(words(k, v, -77) for k, v in zip(
        offsets, ([0] * (n + 1), ctx, [0] * rows, [0] * rows, [count, 0]))))
    row_start, own, positions, slots, left = views
    t = i32(table)
    ML.dec_batch_tables(h, own, i32(new), i32(free), left, t, size, ML.StepTables(*views), position_offset=11)
    torch.cuda.synchronize()
    want = oracle.batch_tables(ctx, new, free, count, table, size, 11, rows)
    for name, v in dict(row_start=row_start, own_len=own, positions=positions, slots=slots, left=left, table=t).items():
        assert np.array_equal(v.cpu().numpy(), want[name]), name
    for k, buf, v in zip(offsets, bufs, views):  # nothing around the outputs
        rest = torch.cat((buf[:k], buf[k + len(v):]))
        assert bool((rest == -77).all())


@pytest.mark.parametrize("rows", [6, 700, 4095, 4096, 4099, 20002])
@pytest.mark.parametrize("offsets", [(0, 0, 0, 0, 0), (1, 2, 3, 1, 3), (0, 0, 4, 2, 1), (3, 1, 1, 4, 0)], ids=str)
def test_tables_in_place_and_at_any_alignment(h, rows, offsets):
    """own_len over ctx_len and left over free_count in one CTA and in the cluster, whose CTAs all have to have read
    both before one writes; positions and slots that are not 16-byte aligned."""
    for seed in range(4):
        tables_in_place(h, rows, offsets, seed)


@pytest.mark.parametrize("size", [16, 32, 64, 128])
@pytest.mark.parametrize("heads,kv,d,new,own,prefix", [(64, 16, 128, [1] * 40, 60, 9001), (32, 32, 64, [1] * 60, 60, 8333),
                                                       (64, 16, 128, [17, 30], 1500, 0), (8, 2, 64, [20, 0, 44], 900, 333)])
def test_tensor_memory_kernel_with_every_block_size(h, size, heads, kv, d, new, own, prefix):
    """Prefixes and contexts that end inside a block and a tile, blocks that are not there, requests whose last
    block has a token of the step alone."""
    rng = np.random.default_rng(size + d)
    lens = [n + int(rng.integers(0, own)) for n in new]
    lens[0] = new[0] + 3 * size
    c = Case(new, lens, heads, kv, d, size, prefix=prefix, pad=64 - sum(new), seed=size, sharp=2.0)
    for b in range(0, len(new), 2):
        c.table[b, int(rng.integers(0, -(-lens[b] // size)))] = (-1, c.blocks)[b % 4 // 2]
    if prefix:
        c.prefix_table[[1, -(-prefix // size) // 2]] = (c.blocks, -5)
    first = c.run(h)
    c.check(first, reference64)
    assert np.array_equal(c.run(h), first)


@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("T,heads,kv,d,rot,size", [(3000, 64, 16, 128, 128, 16), (5000, 8, 1, 128, 64, 64),
                                                   (9001, 16, 16, 64, 48, 128), (2433, 2, 1, 64, 16, 32),
                                                   (20000, 0, 1, 64, 64, 16), (700, 71, 1, 64, 0, 16)])
def test_rope_of_many_rows(h, T, heads, kv, d, rot, size, inter):
    """As many rows as one CTA turns several of, in place and not, and rows without a slot among them."""
    import torch
    import moe_layers_gb300 as ML
    g = torch.Generator(device="cuda")
    g.manual_seed(T)
    y = torch.randn((T, (heads + 2 * kv) * d + 8), device="cuda", generator=g).to(torch.bfloat16)
    q, k, v = (y[:, a * d:b * d] for a, b in ((0, heads), (heads, heads + kv), (heads + kv, heads + 2 * kv)))
    blocks = -(-T // size) + 2
    slots = torch.randperm(blocks * size, device="cuda", generator=g)[:T].to(torch.int32)
    slots[::7] = -1
    slots[5::91] = blocks * size
    positions = torch.randint(0, 1 << 20, (T,), device="cuda", generator=g).to(torch.int32)
    pool = torch.randn((2, blocks, kv, size, d), device="cuda", generator=g).to(torch.bfloat16)
    freq = torch.tensor(oracle.rope_frequencies(rot, 500000.0) if rot else np.zeros(0), device="cuda")
    angle = positions.double()[:, None, None] * freq
    x = y[:, :(heads + 2 * kv) * d].double().reshape(T, -1, d)
    a_at, b_at = (slice(0, rot, 2), slice(1, rot, 2)) if inter else (slice(0, rot // 2), slice(rot // 2, rot))
    want, size_of = x.clone(), torch.zeros_like(x)
    want[..., a_at] = x[..., a_at] * torch.cos(angle) - x[..., b_at] * torch.sin(angle)
    want[..., b_at] = x[..., b_at] * torch.cos(angle) + x[..., a_at] * torch.sin(angle)
    size_of[..., a_at] = size_of[..., b_at] = x[..., a_at].abs() + x[..., b_at].abs()
    near = want.abs() * 2.0 ** -8 + size_of * 2.0 ** -20
    near[..., rot:] = 0
    there = (slots >= 0) & (slots < blocks * size)
    at = slots[there].long()
    rope = ML.Rope(h, rot, base=500000.0, interleaved=inter)
    for in_place in (False, True) if heads else (False,):
        old_y, old = y.clone(), pool.clone()
        cache = pool.clone()
        out = ML.dec_rope_append(h, rope, q if heads else None, k, v, positions, slots, ML.KvCache(cache[0], cache[1]),
                                 q_out=q if in_place else None)
        torch.cuda.synchronize()
        if heads:
            assert bool(((out.double().reshape(T, heads, d) - want[:, :heads]).abs() <= near[:, :heads]).all())
        rest = slice(heads * d if in_place else 0, None)
        assert torch.equal(y[:, rest].view(torch.int16), old_y[:, rest].view(torch.int16))
        for part, mine, by in ((0, want[:, heads:heads + kv], near[:, heads:heads + kv]),
                               (1, x[:, heads + kv:], torch.zeros_like(x[:, heads + kv:]))):
            places = cache[part].transpose(1, 2)  # [block][token][head][element]
            got = places[at // size, at % size].double()
            assert bool(((got - mine[there]).abs() <= by[there]).all())
            untouched = torch.ones((blocks, size), dtype=torch.bool, device="cuda")
            untouched[at // size, at % size] = False
            assert torch.equal(places[untouched].view(torch.int16), old[part].transpose(1, 2)[untouched].view(torch.int16))

"""What the attention entry points refuse, checked without a GPU: every bad
argument is refused before anything touches the device.

The handle here is a block of zeros, which the argument checks never read.
"""
import ctypes

import numpy as np
import pytest

INVALID = 1
A = 1 << 20  # an aligned, never dereferenced device address


@pytest.fixture(scope="module")
def ml():
    import moe_layers_gb300 as M
    M.build()
    M._load()
    return M


@pytest.fixture(scope="module")
def handle():
    return ctypes.create_string_buffer(4096)


def cache(ml, **kw):
    d = dict(k=A, v=A, block_stride=2 * 16 * 64, blocks=10, block_size=16, kv_heads=2, head_dim=64)
    d.update(kw)
    return ml._KvCache(**d)


def batch(ml, **kw):
    d = dict(requests=2, max_new=1, row_start=A, own_len=A, block_table=A, max_blocks=4, prefix_table=None, prefix_len=0)
    d.update(kw)
    return ml._Batch(**d)


BAD_CACHE = [dict(k=None), dict(v=None), dict(k=A + 8), dict(v=A + 2), dict(blocks=0), dict(block_size=8),
             dict(block_size=24), dict(block_size=256), dict(kv_heads=0), dict(kv_heads=129, block_stride=1 << 24),
             dict(head_dim=96), dict(head_dim=0), dict(block_stride=2 * 16 * 64 - 8), dict(block_stride=2 * 16 * 64 + 4),
             dict(blocks=1 << 27), dict(block_stride=1 << 38)]
BAD_BATCH = [dict(requests=0), dict(requests=65), dict(max_new=0), dict(max_new=65), dict(row_start=None),
             dict(own_len=None), dict(block_table=None), dict(max_blocks=0), dict(max_blocks=1 << 25), dict(max_blocks=(1 << 24), block_size=128), dict(prefix_len=(1 << 31) - 1, prefix_table=A),
             dict(prefix_len=-1), dict(prefix_len=5), dict(row_start=A + 2)]
BAD_CALL = [dict(q=None), dict(out=None), dict(q=A + 8), dict(out=A + 8), dict(M=0), dict(M=65), dict(q_heads=0),
            dict(q_heads=3), dict(q_heads=2 * 129), dict(ldq=255), dict(ldq=252), dict(ldo=248), dict(scale=0.0),
            dict(scale=-1.0), dict(scale=1e-31), dict(scale=1e31), dict(scale=float("inf")), dict(scale=float("nan")), dict(out=2 * A),
            dict(ldq=(1 << 31) + 8)]


@pytest.mark.parametrize("kw", BAD_CACHE + BAD_BATCH + BAD_CALL, ids=str)
def test_attention_refuses(ml, handle, kw):
    c = cache(ml, **{k: v for k, v in kw.items() if k in dict(ml._KvCache._fields_)})
    b = batch(ml, **{k: v for k, v in kw.items() if k in dict(ml._Batch._fields_)})
    a = dict(q=2 * A, ldq=256, scale=0.125, out=3 * A, ldo=256, M=2, q_heads=4)
    a.update({k: v for k, v in kw.items() if k in a})
    got = ml._load().dec_attention(handle, a["q"], a["ldq"], ctypes.byref(c), ctypes.byref(b), a["scale"], a["out"],
                                   a["ldo"], a["M"], a["q_heads"], 4 * A, 1 << 40, None)
    assert got == INVALID


def test_attention_refuses_nothing_given(ml, handle):
    lib, c, b = ml._load(), cache(ml), batch(ml)
    assert lib.dec_attention(None, A, 256, ctypes.byref(c), ctypes.byref(b), 1.0, 2 * A, 256, 2, 4, A, 1 << 40, None) == INVALID
    assert lib.dec_attention(handle, A, 256, None, ctypes.byref(b), 1.0, 2 * A, 256, 2, 4, A, 1 << 40, None) == INVALID
    assert lib.dec_attention(handle, A, 256, ctypes.byref(c), None, 1.0, 2 * A, 256, 2, 4, A, 1 << 40, None) == INVALID
    n = ctypes.c_size_t()
    assert lib.dec_attention_workspace_size(handle, 65, 4, ctypes.byref(c), ctypes.byref(b), ctypes.byref(n)) == INVALID
    assert lib.dec_attention_workspace_size(handle, 2, 4, ctypes.byref(c), ctypes.byref(b), None) == INVALID


TABLES = dict(ctx=A, new=A, n=2, free=A, count=A, table=A, max_blocks=4, size=16, offset=0, rows=2)
BAD_TABLES = [dict(ctx=None), dict(new=None), dict(free=None), dict(count=None), dict(table=None), dict(n=0),
              dict(n=1025), dict(max_blocks=0), dict(max_blocks=(1 << 24) + 1), dict(size=15), dict(size=8),
              dict(size=256), dict(offset=-1), dict(rows=0), dict(rows=(1 << 20) + 1), dict(ctx=A + 1)]


@pytest.mark.parametrize("kw", BAD_TABLES, ids=str)
def test_tables_refuse(ml, handle, kw):
    a = dict(TABLES, **kw)
    out = ml._StepTables(A, A, A, A, A)
    assert ml._load().dec_batch_tables(handle, a["ctx"], a["new"], a["n"], a["free"], a["count"], a["table"],
                                       a["max_blocks"], a["size"], a["offset"], a["rows"], ctypes.byref(out),
                                       None) == INVALID


@pytest.mark.parametrize("name", ["row_start", "own_len", "positions", "slots", "left"])
def test_tables_refuse_missing_outputs(ml, handle, name):
    out = ml._StepTables(A, A, A, A, A)
    setattr(out, name, None)
    a = TABLES
    assert ml._load().dec_batch_tables(handle, a["ctx"], a["new"], a["n"], a["free"], a["count"], a["table"],
                                       a["max_blocks"], a["size"], a["offset"], a["rows"], ctypes.byref(out),
                                       None) == INVALID


BAD_PHASES = [dict(phases=None), dict(phases=A + 8), dict(rot=0), dict(rot=8), dict(rot=24), dict(rot=144),
              dict(base=1.0), dict(base=float("nan")), dict(base=float("inf")), dict(scaling=-1), dict(scaling=5),
              dict(factor=0.5), dict(factor=float("inf")), dict(scaling=3, length=0.0), dict(scaling=3, low=0.0),
              dict(scaling=4, low=4.0, high=4.0), dict(scaling=4, high=float("inf"))]


@pytest.mark.parametrize("kw", BAD_PHASES, ids=str)
def test_phases_refuse(ml, handle, kw):
    a = dict(phases=A, rot=64, base=1e4, scaling=0, factor=2.0, length=8192.0, low=1.0, high=4.0)
    a.update(kw)
    assert ml._load().dec_rope_phases(handle, a["phases"], a["rot"], a["base"], a["scaling"], a["factor"], a["length"],
                                      a["low"], a["high"], None) == INVALID


BAD_ROPE = [dict(rotary_dim=-16), dict(rotary_dim=80), dict(rotary_dim=24), dict(phases=None), dict(phases=A + 8),
            dict(magnitude=float("inf")), dict(interleaved=2), dict(q=None), dict(q_out=None), dict(q_heads=0),
            dict(q_heads=1025), dict(k=None), dict(v=None), dict(positions=None), dict(slots=None), dict(rows=0),
            dict(rows=(1 << 20) + 1), dict(ldk=120), dict(ldv=132), dict(ldq=248), dict(ldqo=260), dict(k=A + 2),
            dict(q_out=2 * A, ldqo=264), dict(head_dim=80), dict(blocks=0)]


@pytest.mark.parametrize("kw", BAD_ROPE, ids=str)
def test_rope_append_refuses(ml, handle, kw):
    c = cache(ml, **{k: v for k, v in kw.items() if k in ("head_dim", "blocks")})
    r = dict(rotary_dim=64, interleaved=0, magnitude=1.0, phases=A)
    r.update({k: v for k, v in kw.items() if k in r})
    rope = ml._Rope(*r.values())
    a = dict(q=2 * A, ldq=256, k=A, ldk=128, v=A, ldv=128, q_out=3 * A, ldqo=256, rows=2, q_heads=4, positions=A, slots=A)
    a.update({k: v for k, v in kw.items() if k in a})
    assert ml._load().dec_rope_append(handle, ctypes.byref(rope), *a.values(), ctypes.byref(c), None) == INVALID


def test_binding_refuses_host_tensors_and_odd_layouts(ml):
    import torch
    with pytest.raises(ValueError):
        ml.KvCache(torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16), torch.zeros(2, 1, 16, 64, dtype=torch.bfloat16))
    with pytest.raises(ValueError):
        ml.Batch(torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, 1, dtype=torch.int32))
    with pytest.raises(ValueError):
        ml.StepTables.empty(1, 1, "cpu")


def test_oracle_attention_against_brute_force():
    """Two keys by hand, a row that sees nothing, and a block that is not there."""
    import oracle
    k = np.zeros((3, 1, 16, 64))
    v = np.zeros((3, 1, 16, 64))
    k[1, 0, 0, 0], k[1, 0, 1, 0] = 1.0, 3.0
    v[1, 0, 0, 5], v[1, 0, 1, 5] = 10.0, 20.0
    q = np.zeros((3, 1, 64))
    q[:, 0, 0] = 2.0
    out, _, _ = oracle.attention(q, k, v, [0, 1, 2], [2, 2], [[1], [7]], 0.5)
    w = np.exp([1.0, 3.0]) / np.exp([1.0, 3.0]).sum()
    assert abs(out[0, 0, 5] - w @ [10.0, 20.0]) < 1e-12
    assert np.all(out[1] == 0.0) and np.all(np.isnan(out[2]))


def test_oracle_tables_by_hand():
    import oracle
    r = oracle.batch_tables([16, 0, 3], [1, 0, 15], [4, 9, 2], 3, [[7, -1], [-1, -1], [5, -1]], 16, 100, 18)
    assert r["row_start"].tolist() == [0, 1, 1, 16] and r["own_len"].tolist() == [17, 0, 18]
    assert r["table"].tolist() == [[7, 2], [-1, -1], [5, 9]]
    assert r["left"].tolist() == [1, 0]
    assert r["slots"].tolist() == [32] + [5 * 16 + j for j in range(3, 16)] + [144, 145] + [-1, -1]
    assert r["positions"].tolist() == [116] + list(range(103, 118)) + [0, 0]


def test_oracle_rope_is_a_rotation():
    import oracle
    rng = np.random.default_rng(0)
    x = rng.standard_normal((4, 2, 64))
    f = oracle.rope_frequencies(32, 1e4)
    for inter in (False, True):
        y = oracle.rope(x, [0, 1, 7, 100000], f, inter)
        assert np.array_equal(y[0], x[0]) and np.array_equal(y[..., 32:], x[..., 32:])
        assert np.allclose((y ** 2).sum(-1), (x ** 2).sum(-1))
        # scores depend on the distance alone
        a, b = oracle.rope(x, [5] * 4, f, inter), oracle.rope(x, [1005] * 4, f, inter)
        z = rng.standard_normal((4, 2, 64))
        c, d = oracle.rope(z, [2] * 4, f, inter), oracle.rope(z, [1002] * 4, f, inter)
        assert np.allclose((a * c).sum(-1), (b * d).sum(-1))


@pytest.mark.parametrize("M", [2, 40])
def test_nothing_is_launched_where_the_device_is_not_there(ml, M):
    """The entry points make the handle's device current before the first launch: on the default stream of
    another device, kernels would take this one's addresses."""
    import torch
    if torch.cuda.is_available():
        pytest.skip("shows by the launch count that no call reaches a device, for a machine without one")
    handle = ctypes.create_string_buffer(4096)
    handle[0:4] = (1000).to_bytes(4, "little")  # the device
    lib, c, b = ml._load(), cache(ml), batch(ml)
    rope, tables = ml._Rope(64, 0, 1.0, A), ml._StepTables(A, A, A, A, A)
    att = ml._LayerAttention(4, 0.125, ctypes.addressof(rope), ctypes.addressof(c), ctypes.addressof(b), A, A)
    w = ml._LayerWeights()
    w.H, w.N_in, w.K_out, w.E, w.k, w.I, w.eps = 256, 512, 256, 16, 4, 128, 1e-6
    for n in ("gamma1", "W_in", "W_o", "gamma2", "W_r", "Wg", "Wu", "Wd"):
        setattr(w, n, A)
    ref = ctypes.byref
    answers = [
        lib.dec_batch_tables(handle, A, A, 2, A, A, A, 4, 16, 0, 2, ref(tables), None),
        lib.dec_rope_phases(handle, A, 64, 1e4, 0, 1.0, 8192.0, 1.0, 4.0, None),
        lib.dec_rope_append(handle, ref(rope), 2 * A, 256, A, 128, A, 128, 3 * A, 256, M, 4, A, A, ref(c), None),
        lib.dec_attention(handle, 2 * A, 256, ref(c), ref(b), 0.125, 3 * A, 256, M, 4, A, 1 << 40, None),
        lib.decode_layer_attention(handle, ref(w), ref(att), A, M, None, A, 1 << 40, None),
        lib.decode_layer(handle, ref(w), A, M, None, A, 1 << 40, None)]
    assert answers == [3] * 6  # DEC_ERR_CUDA
    assert lib.dec_launch_count(handle) == 0


# Each limit by itself: everything else about the call is allowed, as the first case of each list shows by
# passing the checks (it then ends at the device, which is not there).
WIDE = dict(block_stride=1 << 24, ldq=1 << 20, ldo=1 << 20)
ATTENTION_LIMITS = [
    (dict(WIDE), dict(), None),
    (dict(WIDE, block_size=128, max_blocks=(1 << 24) - 2), dict(max_blocks=(1 << 24) - 1), "keys"),
    (dict(WIDE, max_blocks=1 << 24), dict(max_blocks=(1 << 24) + 1), "blocks of a request"),
    (dict(WIDE, q_heads=2 * 128), dict(q_heads=2 * 129), "heads to a key head"),
    (dict(WIDE, kv_heads=16, q_heads=1024), dict(q_heads=1040), "heads"),
    (dict(WIDE, kv_heads=128, q_heads=128), dict(kv_heads=129, q_heads=129), "key heads"),
    (dict(WIDE, head_dim=128), dict(head_dim=96), "head dim"),
    (dict(WIDE, head_dim=64), dict(head_dim=80), "head dim"),
    (dict(WIDE, block_size=16), dict(block_size=24), "block size"),
    (dict(WIDE, block_size=128), dict(block_size=256), "block size"),
    (dict(WIDE, block_size=16), dict(block_size=8), "block size"),
    (dict(WIDE, blocks=(1 << 27) - 1), dict(blocks=1 << 27), "tokens of the cache"),
    (dict(WIDE, block_stride=(1 << 38) - 8), dict(block_stride=1 << 38), "block stride"),
    (dict(WIDE, prefix_table=A, prefix_len=(1 << 31) - 256), dict(prefix_len=(1 << 31) - 255), "prefix"),
    (dict(WIDE, prefix_table=A, prefix_len=5), dict(prefix_table=A + 2), "alignment"),
    (dict(WIDE, requests=64, M=64, max_new=64), dict(requests=65), "requests"),
    (dict(WIDE, requests=64, M=64, max_new=64), dict(M=65), "rows"),
    (dict(WIDE, requests=64, M=64, max_new=64), dict(max_new=65), "new rows"),
    (dict(WIDE, scale=1e30), dict(scale=1.1e30), "scale"),
    (dict(WIDE, scale=1.1e-30), dict(scale=0.9e-30), "scale"),
    (dict(WIDE, ldq=1 << 31), dict(ldq=(1 << 31) + 8), "row stride"),
    (dict(WIDE, ldo=1 << 31), dict(ldo=(1 << 31) + 8), "row stride"),
    (dict(WIDE, ldo=256), dict(ldo=248), "row stride"),
]


def attention_answer(ml, handle, kw):
    c = cache(ml, **{k: v for k, v in kw.items() if k in dict(ml._KvCache._fields_)})
    b = batch(ml, **{k: v for k, v in kw.items() if k in dict(ml._Batch._fields_)})
    a = dict(q=2 * A, ldq=256, scale=0.125, out=3 * A, ldo=256, M=2, q_heads=4)
    a.update({k: v for k, v in kw.items() if k in a})
    return ml._load().dec_attention(handle, a["q"], a["ldq"], ctypes.byref(c), ctypes.byref(b), a["scale"], a["out"],
                                    a["ldo"], a["M"], a["q_heads"], 4 * A, 1 << 40, None)


@pytest.fixture(scope="module")
def nowhere():
    """A handle of a device that no machine has: a call that passes the checks ends there, as a CUDA error."""
    h = ctypes.create_string_buffer(4096)
    h[0:4] = (1000).to_bytes(4, "little")
    return h


@pytest.mark.parametrize("good,bad,what", ATTENTION_LIMITS, ids=lambda x: x if isinstance(x, str) else "")
def test_attention_limits_one_by_one(ml, nowhere, good, bad, what):
    assert attention_answer(ml, nowhere, good) == 3
    if bad:
        assert attention_answer(ml, nowhere, dict(good, **bad)) == INVALID


ROPE_LIMITS = [
    (dict(q_heads=1024), dict(q_heads=1025)), (dict(head_dim=128, rotary_dim=128), dict(rotary_dim=144)),
    (dict(head_dim=64), dict(head_dim=80)), (dict(rotary_dim=16), dict(rotary_dim=8)),
    (dict(rotary_dim=0, phases=None), dict(rotary_dim=-16)),
    (dict(ldk=1 << 31), dict(ldk=(1 << 31) + 8)), (dict(ldv=1 << 31), dict(ldv=(1 << 31) + 8)),
    (dict(ldq=1 << 31), dict(ldq=(1 << 31) + 8)), (dict(ldqo=1 << 31), dict(ldqo=(1 << 31) + 8)),
    (dict(ldk=128), dict(ldk=124)), (dict(ldk=136), dict(ldk=132)), (dict(ldv=128), dict(ldv=120)),
    (dict(q_out=2 * A), dict(q_out=2 * A, ldqo=(1 << 20) + 8)), (dict(rows=1 << 20), dict(rows=(1 << 20) + 1)),
    (dict(magnitude=-2.0), dict(magnitude=float("nan"))), (dict(slots=A + 4), dict(slots=A + 2)),
    (dict(positions=A + 4), dict(positions=A + 1)), (dict(q=None, q_out=None, q_heads=0), dict(q_out=3 * A)),
    (dict(q=None, q_out=None, q_heads=0), dict(q_heads=4)), (dict(interleaved=1), dict(interleaved=-1))]


@pytest.mark.parametrize("good,bad", ROPE_LIMITS, ids=str)
def test_rope_append_limits_one_by_one(ml, nowhere, good, bad):
    def answer(kw):
        c = cache(ml, block_stride=1 << 24, **{k: v for k, v in kw.items() if k == "head_dim"})
        r = dict(rotary_dim=64, interleaved=0, magnitude=1.0, phases=A)
        r.update({k: v for k, v in kw.items() if k in r})
        rope = ml._Rope(*r.values())
        a = dict(q=2 * A, ldq=1 << 20, k=A, ldk=256, v=A, ldv=256, q_out=3 * A, ldqo=1 << 20, rows=2, q_heads=4,
                 positions=A, slots=A)
        a.update({k: v for k, v in kw.items() if k in a})
        return ml._load().dec_rope_append(nowhere, ctypes.byref(rope), *a.values(), ctypes.byref(c), None)

    assert answer(good) == 3
    assert answer(dict(good, **bad)) == INVALID


TABLE_LIMITS = [(dict(n=1024), dict(n=1025)), (dict(max_blocks=1 << 24), dict(max_blocks=(1 << 24) + 1)),
                (dict(size=128), dict(size=256)), (dict(size=16), dict(size=8)),
                (dict(rows=1 << 20), dict(rows=(1 << 20) + 1)),
                (dict(offset=(1 << 31) - 1), dict(offset=-1)), (dict(free=A + 4), dict(free=A + 2)),
                (dict(table=A + 4), dict(table=A + 3)), (dict(new=A + 4), dict(new=A + 1)), (dict(count=A + 4), dict(count=A + 2))]


@pytest.mark.parametrize("good,bad", TABLE_LIMITS, ids=str)
def test_tables_limits_one_by_one(ml, nowhere, good, bad):
    def answer(kw):
        a = dict(TABLES, **kw)
        out = ml._StepTables(A, A, A, A, A)
        return ml._load().dec_batch_tables(nowhere, a["ctx"], a["new"], a["n"], a["free"], a["count"], a["table"],
                                           a["max_blocks"], a["size"], a["offset"], a["rows"], ctypes.byref(out), None)

    assert answer(good) == 3
    assert answer(dict(good, **bad)) == INVALID

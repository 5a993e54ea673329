"""What the 8-bit entry points refuse, checked without a GPU: every bad argument is refused before anything touches the
device. The handle here is a block of zeros, which the argument checks never read."""
import ctypes

import pytest

INVALID, UNSUPPORTED = 1, 2
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


def rows(ml, **kw):
    d = dict(q=A, ldq=256, scales=A, lds=2)
    d.update(kw)
    return ml._Fp8Rows(*d.values())


BAD_ROWS = [dict(q=None), dict(scales=None), dict(q=A + 8), dict(scales=A + 2), dict(ldq=240), dict(ldq=264),
            dict(lds=1), dict(ldq=(1 << 31) + 16), dict(lds=(1 << 31) + 1)]


@pytest.mark.parametrize("kw", BAD_ROWS + [
    dict(x=None), dict(x=A + 8), dict(ldx=248), dict(ldx=260), dict(M=0), dict(M=(1 << 20) + 1), dict(H=0), dict(H=8),
    dict(H=264), dict(H=65552), dict(residual=A + 2), dict(ldr=8), dict(residual=None), dict(sum=A + 4), dict(lds_sum=8),
    dict(y=A + 8), dict(ldy=12), dict(y=7 * A), dict(gamma=A + 2), dict(eps=-1.0), dict(eps=float("nan")),
    dict(eps=float("inf")), dict(sum=2 * A, lds_sum=512), dict(sum=3 * A, lds_sum=512), dict(y=2 * A, ldy=512),
    dict(y=3 * A, ldy=512)], ids=str)
def test_norm_refuses(ml, handle, kw):
    a = dict(x=2 * A, ldx=256, residual=3 * A, ldr=256, gamma=5 * A, eps=1e-6, sum=7 * A, lds_sum=256, y=9 * A, ldy=256,
             M=2, H=256)
    a.update({k: v for k, v in kw.items() if k in a})
    out = rows(ml, **{k: v for k, v in kw.items() if k in ("q", "ldq", "scales", "lds")})
    got = ml._load().dec_rmsnorm_quant(handle, a["x"], a["ldx"], a["residual"], a["ldr"], a["gamma"], a["eps"], a["sum"],
                                       a["lds_sum"], a["y"], a["ldy"], ctypes.byref(out), a["M"], a["H"], None)
    assert got == INVALID


def test_null_descriptors(ml, handle):
    lib, r, w = ml._load(), rows(ml), ml._Fp8Weight(A, A)
    moe = ml._MoeFp8Weights(256, 4, 128, *[w] * 6)
    n = ctypes.c_size_t()
    assert lib.dec_rmsnorm_quant(handle, A, 256, None, 0, None, 0.0, None, 0, None, 0, None, 1, 256, None) == INVALID
    assert lib.dec_rmsnorm_quant(None, A, 256, None, 0, None, 0.0, None, 0, None, 0, ctypes.byref(r), 1, 256, None) == INVALID
    assert lib.dec_linear_fp8(handle, None, ctypes.byref(w), None, 0, A, 64, 1, 64, 256, A, 1 << 40, None) == INVALID
    assert lib.dec_linear_fp8(handle, ctypes.byref(r), None, None, 0, A, 64, 1, 64, 256, A, 1 << 40, None) == INVALID
    assert lib.dec_linear_fp8(None, ctypes.byref(r), ctypes.byref(w), None, 0, A, 64, 1, 64, 256, A, 1 << 40, None) == INVALID
    assert lib.moe_experts_fp8(handle, None, A, A, 1, 2, ctypes.byref(moe), None, A, A, 1 << 40, None) == INVALID
    assert lib.moe_experts_fp8(handle, ctypes.byref(r), A, A, 1, 2, None, None, A, A, 1 << 40, None) == INVALID
    assert lib.moe_experts_fp8(None, ctypes.byref(r), A, A, 1, 2, ctypes.byref(moe), None, A, A, 1 << 40, None) == INVALID
    assert lib.dec_linear_fp8_workspace_size(None, 1, 1, 16, ctypes.byref(n)) == INVALID
    assert lib.dec_linear_fp8_workspace_size(handle, 1, 1, 16, None) == INVALID
    assert lib.moe_experts_fp8_workspace_size(None, ctypes.byref(moe), 1, 1, ctypes.byref(n)) == INVALID
    assert lib.moe_experts_fp8_workspace_size(handle, ctypes.byref(moe), 1, 1, None) == INVALID
    assert lib.dec_quant_weight(None, A, 128, 128, A, A, None) == INVALID


@pytest.mark.parametrize("kw", [dict(W=None), dict(q=None), dict(s=None), dict(W=A + 8), dict(q=A + 8), dict(s=A + 2),
                                dict(N=0), dict(N=(1 << 32) + 1), dict(K=0), dict(K=8), dict(K=24), dict(K=65552)], ids=str)
def test_weight_refuses(ml, handle, kw):
    a = dict(W=A, N=128, K=256, q=2 * A, s=3 * A)
    a.update(kw)
    assert ml._load().dec_quant_weight(handle, *a.values(), None) == INVALID


@pytest.mark.parametrize("kw", BAD_ROWS + [
    dict(wq=None), dict(ws=None), dict(wq=A + 8), dict(ws=A + 1), dict(y=None), dict(y=A + 1), dict(ldy=63),
    dict(ldy=(1 << 31) + 1), dict(residual=A + 1), dict(residual=5 * A, ldr=63), dict(residual=2 * A, ldr=128),
    dict(M=0), dict(M=(1 << 20) + 1), dict(N=0, ldy=64), dict(N=(1 << 20) + 1, ldy=1 << 21), dict(K=0), dict(K=8),
    dict(K=264), dict(K=65552, ldq=65552, lds=600)], ids=str)
def test_linear_refuses(ml, handle, kw):
    a = dict(residual=None, ldr=64, y=2 * A, ldy=64, M=2, N=64, K=256)
    a.update({k: v for k, v in kw.items() if k in a})
    r = rows(ml, **{k: v for k, v in kw.items() if k in ("q", "ldq", "scales", "lds")})
    w = ml._Fp8Weight(kw.get("wq", A), kw.get("ws", A))
    got = ml._load().dec_linear_fp8(handle, ctypes.byref(r), ctypes.byref(w), *a.values(), 4 * A, 1 << 40, None)
    assert got == INVALID


NAMES = ("gate", "up", "down", "gate_s", "up_s", "down_s")


@pytest.mark.parametrize("kw", BAD_ROWS + [dict(zip(("name", "part"), (n, p))) for n in NAMES for p in ("q", "scales")] + [
    dict(idx=None), dict(w=None), dict(idx=A + 2), dict(w=A + 1), dict(out=None), dict(out=A + 8), dict(residual=A + 8),
    dict(ws=None), dict(ws=A + 8), dict(ws_bytes=1000), dict(M=0), dict(M=65), dict(k=0), dict(k=17), dict(H=0), dict(H=192),
    dict(E=0), dict(E=1025), dict(I=0), dict(I=64)], ids=str)
def test_experts_refuse(ml, handle, kw):
    a = dict(idx=A, w=A, M=2, k=2)
    a.update({k: v for k, v in kw.items() if k in a})
    b = dict(residual=None, out=2 * A, ws=4 * A, ws_bytes=1 << 40)
    b.update({k: v for k, v in kw.items() if k in b})
    r = rows(ml, **{k: v for k, v in kw.items() if k in ("q", "ldq", "scales", "lds")})
    sizes = dict(H=256, E=4, I=128)
    sizes.update({k: v for k, v in kw.items() if k in sizes})
    moe = ml._MoeFp8Weights(*sizes.values(), *[ml._Fp8Weight(A, A) for _ in NAMES])
    if "name" in kw:
        setattr(getattr(moe, kw["name"]), kw["part"], None)
    got = ml._load().moe_experts_fp8(handle, ctypes.byref(r), *a.values(), ctypes.byref(moe), *b.values(), None)
    assert got == INVALID


@pytest.mark.parametrize("kw", [dict(H=16512), dict(I=16512)], ids=str)
def test_experts_too_wide(ml, handle, kw):
    sizes = dict(H=256, E=4, I=128)
    sizes.update(kw)
    moe = ml._MoeFp8Weights(*sizes.values(), *[ml._Fp8Weight(A, A) for _ in NAMES])
    r = rows(ml, ldq=65536, lds=512)
    n = ctypes.c_size_t()
    lib = ml._load()
    assert lib.moe_experts_fp8(handle, ctypes.byref(r), A, A, 1, 1, ctypes.byref(moe), None, 2 * A, 4 * A, 1 << 40,
                               None) == UNSUPPORTED
    assert lib.moe_experts_fp8_workspace_size(handle, ctypes.byref(moe), 1, 1, ctypes.byref(n)) == UNSUPPORTED


def test_binding_refuses(ml):
    """Descriptors of the binding: shapes, types, gaps (on the CPU every tensor is refused for its place, first of all)."""
    import torch
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.zeros(4, 2)
    with pytest.raises(ValueError, match="CUDA"):
        ml.Fp8Rows(q, s)
    with pytest.raises(ValueError, match="CUDA"):
        ml.Fp8Weight(q, s)

"""8-bit rows and weights in plain torch, in 64 bits, with the bounds of their arithmetic."""
import torch

E4M3 = torch.float8_e4m3fn
TOP = 448.0


def groups(width):
    return -(-width // 128)


def spread(scale, width):
    """[.., groups] scales as one for each of `width` values."""
    return scale.repeat_interleave(128, -1)[..., :width]


def value_rows(q, scale):
    return q.double() * spread(scale.double(), q.shape[-1])


def value_weight(q, scale):
    n, k = q.shape[-2:]
    return q.double() * spread(scale.double().repeat_interleave(128, -2)[..., :n, :], k)


def amax_groups(y):
    return torch.stack([p.abs().amax(-1) for p in y.split(128, -1)], -1)


def quant_rows(y):
    """By the formula, in y's own type (both divisions between tensors: torch divides by a number with its reciprocal)."""
    most = amax_groups(y)
    top = torch.full_like(most, TOP)
    up = torch.where(most > 0, top / most, torch.zeros_like(most))
    return (y * spread(up, y.shape[-1])).float().to(E4M3), most / top


def rand_rows(g, m, k, device="cuda"):
    q, s = quant_rows(torch.randn(m, k, generator=g, device=device) * torch.exp(torch.randn(k, generator=g, device=device)))
    return q, s.float()


def rand_weight(g, *shape, device="cuda"):
    n, k = shape[-2:]
    q = (torch.randn(*shape, generator=g, device=device) * 60).to(E4M3)
    s = torch.exp(torch.randn(*shape[:-2], groups(n), groups(k), generator=g, device=device)) * k ** -0.5 / 60
    return q, s


def sum_bound(k):
    """Relative to the sum of the products' absolute values: an addition in a product unit loses at most a unit in the
    last place (2^-23, it may cut instead of round), over a block's 128 products, then one rounded fused
    multiply-add a block with two scales multiplied before."""
    return (128 + groups(k) + 4) * 2.0 ** -23


def linear64(x, xs, w, ws, residual=None):
    """(result, how far a bf16 result may be off)."""
    a, b = value_rows(x, xs), value_weight(w, ws)
    y = a @ b.t()
    room = (a.abs() @ b.abs().t()) * sum_bound(x.shape[1])
    if residual is not None:
        y = y + residual.double()
        room = room + 2.0 ** -24 * y.abs()
    return y, room + 2.0 ** -8 * (y.abs() + room)


def inner64(x, xs, gate, up):
    """silu(gate x) * (up x) and how far an fp32 form may be off."""
    a = value_rows(x, xs)
    wg, wu = value_weight(*gate), value_weight(*up)
    z, u = a @ wg.t(), a @ wu.t()
    dz, du = (a.abs() @ wg.abs().t()) * sum_bound(x.shape[1]), (a.abs() @ wu.abs().t()) * sum_bound(x.shape[1])
    h = z * torch.sigmoid(z) * u
    # |silu'| <= 1.1; the exponential, division and products add a few roundings
    return h, 1.1 * dz * (u.abs() + du) + (z.abs() + dz) * du + 8 * 2.0 ** -24 * h.abs()


def expert64(x, xs, gate, up, down):
    """One expert's output for rows x and how far it may be off, rows near a tie of the 8-bit rounding included."""
    h, dh = inner64(x, xs, gate, up)
    most, dmost = amax_groups(h), amax_groups(dh)
    s = most / TOP
    off = spread(dmost / most.clamp(min=1e-300), h.shape[1]) + 2.0 ** -22  # of the group's factor
    v = h / spread(s, h.shape[1]).clamp(min=1e-300)
    dv = dh / spread(s, h.shape[1]).clamp(min=1e-300) + off * v.abs()
    q, hi, lo = (t.clamp(-TOP, TOP).float().to(E4M3).double() for t in (v, v + dv, v - dv))
    by = spread(s, h.shape[1])
    wd = value_weight(*down)
    room = ((hi - lo) * by + q.abs() * by * off) @ wd.abs().t()
    mass = ((q.abs() + (hi - lo)) * by) @ wd.abs().t()
    return (q * by) @ wd.t(), room + mass * sum_bound(h.shape[1])


def experts64(x, xs, idx, w, gate, up, down, shared=None, residual=None):
    m, k = idx.shape
    e = gate[0].shape[0]
    y = torch.zeros(m, gate[0].shape[2], dtype=torch.float64, device=x.device)
    room = torch.zeros_like(y)
    mass = torch.zeros_like(y)
    for i in sorted(set(idx.reshape(-1).tolist())):
        if not 0 <= i < e:
            continue
        t, j = torch.nonzero(idx == i, as_tuple=True)
        o, d = expert64(x[t], xs[t], *((a[0][i], a[1][i]) for a in (gate, up, down)))
        by = w[t, j].double()[:, None]
        y.index_add_(0, t, by * o)
        room.index_add_(0, t, by.abs() * d)
        mass.index_add_(0, t, by.abs() * o.abs())
    if shared is not None:
        o, d = expert64(x, xs, *shared)
        y, room, mass = y + o, room + d, mass + o.abs()
    if residual is not None:
        y, mass = y + residual.double(), mass + residual.double().abs()
    room = room + (k + 2) * 2.0 ** -24 * mass
    return y, room + 2.0 ** -8 * (y.abs() + room)


def assert_within(got, want, room, what=""):
    off = (got.double() - want).abs()
    worst = (off / room.clamp(min=1e-300)).max().item()
    assert torch.isfinite(got.float()).all() and worst <= 1.0, f"{what}: {worst:.3f} of the bound"

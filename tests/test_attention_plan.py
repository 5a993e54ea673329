"""The attention kernels' plan restated on the host: how a step's units are cut into
pieces and where the joining kernel finds them. Checked for the row starts that
a caller may leave in device memory, in order or not: every row's pieces are
those that were written, and no place outside the workspace is read.

The restatement follows build_parts, Piece and the joining kernel's span_of."""
import itertools

import numpy as np
import pytest

LEAD, TILE, SMS = 1, 64, 152


def clamp(x, lo, hi):
    return min(max(x, lo), hi)


def parts_of(row_start, own_len, prefix, M, group, kv, shift):
    """(first row, rows, keys, chunks, units) of part 0, the prefix, and of each request."""
    begin = clamp(row_start[0], 0, M)
    end = clamp(row_start[-1], begin, M)
    spans = [(row_start[0], row_start[-1])] + list(zip(row_start, row_start[1:]))
    parts = []
    for i, (r0, r1) in enumerate(spans):
        first = clamp(r0, begin, end)
        rows = clamp(r1, first, end) - first
        keys = prefix if i == 0 else max(own_len[i - 1], 0)
        chunks = -(-rows * group // (1 << shift))
        tiles = -(-keys // TILE)
        parts.append((first, rows, keys, chunks, kv * chunks * (tiles + LEAD) if tiles else 0))
    return parts


def written(parts, kv, ctas):
    """The pieces (part, head, chunk, first tile, CTA) that the CTAs keep, by their walk over the units."""
    first = np.concatenate([[0], np.cumsum([p[4] for p in parts])]).astype(int)
    W = int(first[-1])
    G = clamp(W, 1, ctas)
    out = set()
    for c in range(G):
        u, end = c * W // G, (c + 1) * W // G
        while u < end:
            part = int(np.searchsorted(first, u, side="right")) - 1
            each = -(-parts[part][2] // TILE) + LEAD
            hc, x = divmod(u - first[part], each)
            units = min(each - x, end - u)
            t0, t1 = max(0, x - LEAD), max(0, x + units - LEAD)
            if t1 > t0:
                out.add((part, hc // parts[part][3], hc % parts[part][3], t0, c))
            u += units
    return first, W, G, out


@pytest.mark.parametrize("seed", range(40))
def test_rows_find_their_pieces(seed):
    rng = np.random.default_rng(seed)
    n, M, kv, group, shift = int(rng.integers(1, 9)), int(rng.integers(1, 65)), int(rng.integers(1, 4)), 4, 3
    starts = np.sort(rng.integers(0, M + 1, n + 1))
    if seed % 4:
        starts = rng.permutation(starts)  # not in order
    if seed % 5 == 0:
        starts = starts + rng.integers(-80, 80, n + 1)  # outside the rows
    own = [int(x) for x in rng.integers(-3, 700, n)]
    prefix = int(rng.choice([0, 100, 5000]))
    parts = parts_of([int(x) for x in starts], own, prefix, M, group, kv, shift)
    ctas = 2 * SMS
    first, W, G, pieces = written(parts, kv, ctas)
    for t, kvh in itertools.product(range(M), range(kv)):
        hit = [i for i in range(1, n + 1) if parts[i][0] <= t < parts[i][0] + parts[i][1]]
        if not hit:
            continue
        for i in ([0] if prefix else []) + [hit[-1]]:
            if first[i + 1] == first[i]:
                continue
            rows0, rows, keys, chunks, _ = parts[i]
            rr = (t - rows0) * group
            assert 0 <= rr < rows * group  # within the part
            chunk, tiles = rr >> shift, -(-keys // TILE)
            u = int(first[i]) + (kvh * chunks + chunk) * (tiles + LEAD) + LEAD
            c0, c1 = -(-(u + 1) * G // W) - 1, -(-(u + tiles) * G // W) - 1
            assert 0 <= c0 <= c1 < G
            for c in range(c0, c1 + 1):
                assert any(p[:3] == (i, kvh, chunk) and p[4] == c and (p[3] == 0) == (c == c0) for p in pieces)

"""The paged 4-bit key/value cache and the page operations, restated plainly.

fp64 NumPy and Python lists, sharing no code with the library: the quantiser as
the formulas give it, a tile as bytes found one by one by their places, and the
page operations as a scheduler would do them one slot at a time.
"""

from __future__ import annotations

from fractions import Fraction

import numpy as np

from oracle import dca_oracle as orc

GROUP = 64
TILE = 64


# ---------------------------------------------------------------- roundings
def bf16(x):
    """float64 rounded once to bf16 (nearest even), as float64.  NaN and
    infinities pass; values at or above the overflow threshold become inf."""
    x = np.asarray(x, np.float64)
    m, e = np.frexp(x)
    e = np.maximum(e, -125)  # subnormals share the last place of the smallest normal
    step = np.ldexp(1.0, e - 8)
    with np.errstate(invalid="ignore", over="ignore"):
        y = np.rint(x / step) * step
    y = np.where(np.abs(y) >= 2.0 ** 128, np.copysign(np.inf, x), y)
    return np.where(np.isfinite(x), y, x)


def bf16_up(x):
    """The smallest bf16 value that is not below x >= 0."""
    x = np.asarray(x, np.float64)
    _, e = np.frexp(x)
    step = np.ldexp(1.0, np.maximum(e, -125) - 8)
    return np.ceil(x / step) * step


def bf16_bits(x):
    """Bit patterns (uint16) of float64 values that are bf16 values."""
    f = np.asarray(x, np.float32)
    return (f.view(np.uint32) >> 16).astype(np.uint16)


# ---------------------------------------------------------------- quantiser
def quantise(x):
    """x [..., D] float64 bf16 values -> codes uint8 [..., D], scale and offset
    float64 [..., D/64]; NaN parameters and zero codes where a group is not
    finite."""
    x = np.asarray(x, np.float64)
    g = x.reshape(*x.shape[:-1], -1, GROUP)
    fine = np.isfinite(g).all(-1)
    g = np.where(fine[..., None], g, 0.0)
    off, top = g.min(-1) + 0.0, g.max(-1)  # an offset of -0 is stored as 0
    scale = bf16_up((top - off) / 15 + 0.0)
    with np.errstate(invalid="ignore", divide="ignore"):
        quotient = (g - off[..., None]) / scale[..., None]
    quotient = np.where(scale[..., None] > 0, quotient, 0)
    c = np.rint(quotient).astype(np.uint8)
    # next to a border fp64 may have lost what decides: rational numbers there
    for at in np.argwhere(np.abs(quotient - np.floor(quotient) - 0.5) < 1e-9):
        at = tuple(at)
        exact = (Fraction(g[at]) - Fraction(off[at[:-1]])) / Fraction(scale[at[:-1]])
        c[at] = round(exact)  # half to even
    scale, off = np.where(fine, scale, np.nan), np.where(fine, off, np.nan)
    return c.reshape(x.shape), scale, off


def values(codes, scale, off):
    g = codes.astype(np.float64).reshape(*codes.shape[:-1], -1, GROUP)
    return (g * scale[..., None] + off[..., None]).reshape(codes.shape)


# ---------------------------------------------------------------- tiles
def tile_bytes(D):
    return 72 * D


def _places(D):
    """Byte place and nibble of every (row, dim) code and byte place of every
    (row, group) parameter, for keys and for values."""
    gr = D // GROUP
    out = {}
    base = 0
    for what in ("k", "v"):
        at = np.zeros((TILE, D), np.int64)
        nib = np.zeros((TILE, D), np.int64)
        par = np.zeros((TILE, gr), np.int64)
        for r in range(TILE):
            for d in range(D):
                g, i, n = d // 64, d % 64 // 8, d % 8
                if what == "k":
                    word = ((r * 4 + i // 2) * gr + g) * 2 + i % 2
                else:
                    word = ((r // 16 * gr + g) * 8 + i) * 16 + r % 16
                at[r, d] = base + 4 * word + n // 2
                nib[r, d] = n % 2
            for g in range(gr):
                par[r, g] = base + TILE * D // 2 + 4 * (r * gr + g)
        out[what] = at, nib, par
        base += TILE * D // 2 + TILE * gr * 4
    assert base == tile_bytes(D)
    return out


_PLACES = {D: _places(D) for D in (64, 128)}


def write_row(tile, what, r, codes, scale, off):
    """Store one quantised row in a tile (uint8 [tile_bytes], in place)."""
    D = codes.shape[0]
    at, nib, par = _PLACES[D][what]
    for n in (0, 1):
        sel = nib[r] == n
        keep = 0xF0 if n == 0 else 0x0F
        tile[at[r, sel]] = (tile[at[r, sel]] & keep) | (codes[sel] << (4 * n)).astype(np.uint8)
    for g in range(D // GROUP):
        if np.isnan(scale[g]):
            words = np.array([0x7FFF, 0x7FFF], np.uint16)
        else:
            words = np.array([bf16_bits(scale[g]), bf16_bits(off[g])], np.uint16)
        tile[par[r, g]:par[r, g] + 4] = words.view(np.uint8)


def read_rows(tile, what, D):
    """(codes, scale, offset) of the 64 rows of a tile."""
    at, nib, par = _PLACES[D][what]
    codes = (tile[at] >> (4 * nib).astype(np.uint8)) & 15
    words = np.stack([tile[par + j].astype(np.uint32) << (8 * j) for j in range(4)]).sum(0)
    words = words.astype(np.uint32)
    with np.errstate(invalid="ignore"):
        scale = (words << 16).astype(np.uint32).view(np.float32).astype(np.float64)
        off = (words & 0xFFFF0000).astype(np.uint32).view(np.float32).astype(np.float64)
    return codes, scale, off


def _tile(pool, table, b, pos, h):
    R = pool.shape[2] * TILE
    return pool[table[b, pos // R], h, pos % R // TILE]


def append(k, v, pool, table, cu, t0, s, base=10000.0):
    """Store packed rows k, v [T, Hkv, D] (float64 bf16 values) in pool, in place."""
    for b in range(len(t0)):
        for r in range(cu[b], cu[b + 1]):
            pos = t0[b] + r - cu[b]
            key = bf16(orc.rotate(k[r], pos % s, base))
            for h in range(k.shape[1]):
                tile = _tile(pool, table, b, pos, h)
                write_row(tile, "k", pos % TILE, *quantise(key[h]))
                write_row(tile, "v", pos % TILE, *quantise(v[r, h]))


def cache(pool, table, b, n, D):
    """{what: (codes [n, Hkv, D], scale, offset [n, Hkv, D/64])} of rows 0 .. n-1."""
    got = {}
    for what in ("k", "v"):
        rows = []
        for j0 in range(0, n, TILE):
            per_head = [read_rows(_tile(pool, table, b, j0, h), what, D)
                        for h in range(pool.shape[1])]
            rows.append([np.stack(x, 1) for x in zip(*per_head)])
        got[what] = tuple(np.concatenate([r[i] for r in rows])[:n] for i in range(3))
    return got


def decode(q, pool, table, t, s, c, base=10000.0, scale=0.0):
    """(O, LSE, bound_O, bound_LSE): the attention, and how far a kernel may be
    from it.  bound_O: the output is rounded to bf16 (half a step is 2^-8 of it).
    Every weight P times the value scale, which multiplies a code of 0 .. 15, is
    rounded to fp16 (half a step is 2^-11 of it) after a normalisation that puts
    the largest scale of a group among the 64 keys of a tile between 2^14 and
    2^15: below fp16's normal range half a step is 2^-25, which is 2^-39 of that
    scale, times a code of 15.  fp32 sums of codes and offsets besides.
    bound_LSE: the largest error a score can have from fp32 sums over D products
    and a query of 22 bits, and the fp32 sum of the exponentials."""
    B, Hq, D = q.shape
    Hkv = pool.shape[1]
    sc = scale if scale else 1.0 / np.sqrt(D)
    O, LSE = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    bO, bL = np.zeros((B, Hq, D)), np.zeros((B, Hq))
    for b in range(B):
        i = int(t[b])
        got = cache(pool, table, b, i + 1, D)
        key, val = values(*got["k"]), values(*got["v"])
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            O[b, h], LSE[b, h] = orc.dca_row(q[b, h], key[:, hk], val[:, hk], i, s, c, base, sc)
            codes, vs, vo = (x[:, hk] for x in got["v"])
            pos = orc.query_position(i, np.arange(i + 1), s, c)
            qr = {p: orc.rotate(q[b, h], p, base) for p in set(pos.tolist())}
            z = np.array([qr[p] @ key[j, hk] for j, p in enumerate(pos.tolist())]) * sc
            w = np.exp(z - LSE[b, h])
            part = np.repeat(vs, 64, 1) * codes
            whole = part + np.repeat(np.abs(vo), 64, 1)
            least = sum(len(x) * x.max(0) for x in np.split(vs, range(64, i + 1, 64)))
            least = np.repeat(least, 64) * 15 * 2.0 ** -39
            # errors of the scores change every weight by as much, relatively
            kc, ks, ko = (x[:, hk] for x in got["k"])
            size = np.repeat(np.abs(ko), 64, 1) + np.repeat(ks, 64, 1) * kc
            qa = max(np.abs(x).max() for x in qr.values())
            err = abs(sc) * (D + 16) * 2.0 ** -23 * qa * size.sum(1).max()
            sums = (16 + (i + 1) / 64) * 2.0 ** -23
            bL[b, h] = err + sums + abs(LSE[b, h]) * 2.0 ** -22
            bO[b, h] = 2.0 ** -8 * np.abs(O[b, h]) + 2.0 ** -11 * (w @ part) + (
                2 * err + 2 * sums) * (w @ whole) + least + 1e-30
    return O, LSE, bO, bL


# ---------------------------------------------------------------- pages
def _used(row, n, R):
    return list(row[:-(-n // R)])


def remap(src, old_len, new_len, table, refs, R):
    """One step of the slots: (table, refs, info, [(from, to, rows)]), or the
    state as it came when pages are missing.  Lists in, lists out."""
    refs_in, refs = list(refs), list(refs)
    B, most = len(table), len(table[0]) if table else 0
    for row, n in zip(table, old_len):
        for p in _used(row, n, R):
            refs[p] -= 1
    kept = []
    for b in range(B):
        keep = 0 if src[b] < 0 else min(old_len[src[b]], new_len[b])
        kept.append(divmod(keep, R))
        for p in (table[src[b]][:keep // R] if keep else []):
            refs[p] += 1
    held = {p for p, n in enumerate(refs) if n > 0}
    mine = []
    for b, (full, rest) in enumerate(kept):
        tail = table[src[b]][full] if rest else None
        mine.append(rest > 0 and tail not in held)
        if mine[-1]:
            held.add(tail)
            refs[tail] = 1
    free = [p for p, n in enumerate(refs) if n == 0]
    need = sum(-(-new_len[b] // R) - kept[b][0] - mine[b] for b in range(B))
    if need > len(free):
        return [list(r) for r in table], refs_in, [len(free) - need, 0], []
    out, copies = [], []
    for b, (full, rest) in enumerate(kept):
        row = list(table[src[b]][:full + mine[b]]) if full or rest else []
        if rest and not mine[b]:
            copies.append((table[src[b]][full], free[0], rest))
            row.append(free.pop(0))
        while len(row) < -(-new_len[b] // R):
            row.append(free.pop(0))
        for p in row[full + mine[b]:]:
            refs[p] = 1
        out.append(row + [-1] * (most - len(row)))
    return out, refs, [len(free), len(copies)], copies


def compact(lens, table, refs, R):
    """Pages in use to the front: (table, refs, moved, info, [(from, to, R)])."""
    n = sum(r > 0 for r in refs)
    holes = [p for p in range(n) if refs[p] == 0]
    late = [p for p in range(n, len(refs)) if refs[p] > 0]
    moved = [p if refs[p] > 0 else -1 for p in range(len(refs))]
    out_refs = [r if p < n else 0 for p, r in enumerate(refs)]
    for a, z in zip(late, holes):
        moved[a] = z
        out_refs[z] = refs[a]
    out = []
    for row, m in zip(table, lens):
        now = [moved[p] for p in _used(row, m, R)]
        out.append(now + [-1] * (len(row) - len(now)))
    return out, out_refs, moved, [n, len(late)], [(a, z, R) for a, z in zip(late, holes)]

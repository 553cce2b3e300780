"""The 4-bit cache and the page operations without a GPU: the oracle pinned by
hand-worked numbers, bounds and invariants, and every refusal that the library
makes before it touches the device."""

import ctypes

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
from oracle import dca_oracle as orc
from oracle import kv4_oracle as ko
from tests import kv4_util as ku


@pytest.fixture(scope="module")
def lib():
    from long_context_attention_dca_b200 import build
    build.build()
    return dca.lib()


# ------------------------------------------------------------- the oracle
def test_bf16_rounding_matches_torch():
    rng = np.random.default_rng(0)
    x = (rng.standard_normal(20000) * 10.0 ** rng.uniform(-40, 38, 20000)).astype(np.float32)
    x = np.concatenate([x, np.float32([0, -0.0, np.inf, -np.inf, 3.4e38, 1e-45, 1.00390625])])
    want = torch.from_numpy(x).to(torch.bfloat16).double().numpy()
    assert np.array_equal(ko.bf16(x.astype(np.float64)), want)


def test_quantiser_by_hand():
    x = np.zeros(64)
    x[:4] = [-1.0, 2.0, 0.5, -0.4]
    codes, scale, off = ko.quantise(ko.bf16(x))
    # range 3 / 15 = 0.2 -> the next bf16 above is 0.2001953125 (0x3E4D)
    assert off[0] == -1.0 and scale[0] == 0.2001953125
    assert codes[:4].tolist() == [0, 15, 7, 3] and codes[4] == 5
    # a constant group, a group with a tie (half to even), a group with an inf
    assert ko.quantise(np.full(64, 0.75))[1][0] == 0.0
    y = np.zeros(64)
    y[:4] = [-15.0, 15.0, 0.0, 2.0]  # scale 2: (0 + 15) / 2 = 7.5 -> 8, 8.5 -> 8
    codes, scale, off = ko.quantise(y)
    assert scale[0] == 2.0 and codes[:4].tolist() == [0, 15, 8, 8]
    y[5] = np.inf
    codes, scale, off = ko.quantise(y)
    assert np.isnan(scale[0]) and np.isnan(off[0]) and not codes.any()


@pytest.mark.parametrize("spread", [1.0, 1e-30, 1e30, 3e38])
def test_quantiser_error_is_at_most_half_a_step(spread):
    rng = np.random.default_rng(1)
    x = ko.bf16(np.clip(rng.standard_normal((500, 128)) * spread, -3.3e38, 3.3e38))
    codes, scale, off = ko.quantise(x)
    err = np.abs(ko.values(codes, scale, off) - x)
    assert (err <= np.repeat(scale, 64, 1) * 0.5 * (1 + 1e-12)).all()
    assert codes.max() == 15 and codes.min() == 0
    # the scale is the smallest that will do: one bf16 step less is too small
    top = x.reshape(500, 2, 64).max(-1) - off
    assert (scale * (1 - 2.0 ** -7) * 15 < top).all() and (scale * 15 >= top).all()


@pytest.mark.parametrize("D", [64, 128])
def test_tile_round_trip_and_no_two_values_share_a_place(D):
    rng = np.random.default_rng(2)
    tile = np.zeros(ko.tile_bytes(D), np.uint8)
    want = {}
    for what in ("k", "v"):
        x = ko.bf16(rng.standard_normal((64, D)))
        for r in rng.permutation(64):
            ko.write_row(tile, what, r, *ko.quantise(x[r]))
        want[what] = ko.quantise(x)
    for what in ("k", "v"):
        for a, b in zip(ko.read_rows(tile, what, D), want[what]):
            assert np.array_equal(a, b)
    places = [4 * (2 * ko._PLACES[D][w][0] + ko._PLACES[D][w][1]) for w in ("k", "v")]
    assert len(np.unique(np.concatenate([p.ravel() for p in places]))) == 2 * 64 * D


def test_oracle_decode_matches_attention_over_the_read_back_cache():
    rng = np.random.default_rng(3)
    D, Hq, Hkv, R, s, c = 64, 4, 2, 64, 20, 30
    table, num = ku.random_tables(rng, [130, 7], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    q = rng.standard_normal((2, Hq, D))
    O, LSE, bO, bL = ko.decode(q, pool, table, [129, 6], s, c)
    for b, n in enumerate((130, 7)):
        got = ko.cache(pool, table, b, n, D)
        K, V = ko.values(*got["k"])[None], ko.values(*got["v"])[None]
        o, l = orc.dca_decode(q[b:b + 1], K, V, [n - 1], s, c)
        assert np.allclose(o[0], O[b]) and np.allclose(l[0], LSE[b])
    assert (bO > 0).all() and bO.max() < 0.1 and (bL > 0).all() and bL.max() < 1e-2


def _consistent(table, refs, lens, R, pins):
    count = [0] * len(refs)
    for row, n in zip(table, lens):
        used = row[:-(-n // R)]
        assert all(0 <= p < len(refs) for p in used) and all(p == -1 for p in row[len(used):])
        assert len(set(used)) == len(used)
        for p in used:
            count[p] += 1
    assert [a - b for a, b in zip(refs, count)] == pins
    # whoever will write into a partial page has it alone
    for row, n in zip(table, lens):
        if n % R:
            assert refs[row[n // R]] == 1


def _rows(table, lens, pages, R):
    return [[pages[row[i // R]][i % R] for i in range(n)] for row, n in zip(table, lens)]


@pytest.mark.parametrize("k", range(12))
def test_remap_keeps_contents_and_counts(k):
    rng = np.random.default_rng(100 + k)
    R, most, B = int(rng.choice([1, 3, 64])), 5, int(rng.integers(1, 9))
    lens, table, refs, num = ku.random_slots(rng, B, most, R, extra=40, pins=k % 3)
    held = [refs[p] - sum(r[:-(-n // R)].count(p) for r, n in zip(table, lens))
            for p in range(num)]
    pages = [[(p, i) for i in range(R)] for p in range(num)]
    before = _rows(table, lens, pages, R)
    src = [int(x) for x in rng.integers(-1, B, B)]
    new = [int(rng.integers(0, most * R + 1)) for _ in range(B)]
    out, refs2, info, copies = ko.remap(src, lens, new, table, refs, R)
    assert info[0] >= 0
    _consistent(out, refs2, new, R, held)
    for a, z, n in copies:
        assert refs2[z] == 1 and refs2[a] > 0 and 0 < n < R
        pages[z] = pages[a][:n] + pages[z][n:]
    assert not {z for _, z, _ in copies} & {a for a, _, _ in copies}
    after = _rows(out, new, pages, R)
    for b in range(B):
        keep = 0 if src[b] < 0 else min(lens[src[b]], new[b])
        assert after[b][:keep] == (before[src[b]][:keep] if keep else [])


def test_remap_by_hand():
    # two slots of 5 rows in pages of 4: a fork of slot 0 into slot 1
    out, refs, info, copies = ko.remap([0, 0], [5, 5], [6, 6], [[3, 1], [0, 4]],
                                       [1, 1, 0, 1, 1, 0], 4)
    # slot 1's old pages 0 and 4 are free again; the copy takes page 0
    assert out == [[3, 1], [3, 0]] and refs == [1, 1, 0, 2, 0, 0]
    assert copies == [(1, 0, 1)] and info == [3, 1]
    # not enough pages: nothing changes
    out, refs, info, copies = ko.remap([0], [4], [20], [[1, -1, -1, -1, -1]], [0, 1, 0], 4)
    assert out == [[1, -1, -1, -1, -1]] and refs == [0, 1, 0] and info == [-2, 0] and not copies


@pytest.mark.parametrize("k", range(8))
def test_compact_keeps_contents_and_counts(k):
    rng = np.random.default_rng(200 + k)
    R, B = 4, int(rng.integers(0, 9))
    lens, table, refs, num = ku.random_slots(rng, B, 6, R, extra=int(rng.integers(0, 30)),
                                             pins=k % 3)
    held = [refs[p] - sum(r[:-(-n // R)].count(p) for r, n in zip(table, lens))
            for p in range(num)]
    pages = [[(p, i) for i in range(R)] for p in range(num)]
    before = _rows(table, lens, pages, R)
    out, refs2, moved, info, copies = ko.compact(lens, table, refs, R)
    n = info[0]
    assert all(r > 0 for r in refs2[:n]) and not any(refs2[n:])
    held2 = [0] * num
    for p, z in enumerate(moved):
        if z >= 0:
            held2[z] = held[p]
    count = [0] * num
    for row, m in zip(out, lens):
        for p in row[:-(-m // R)]:
            count[p] += 1
    assert [a - b for a, b in zip(refs2, count)] == held2
    for a, z, _ in copies:
        pages[z] = pages[a]
    assert _rows(out, lens, pages, R) == before


# ------------------------------------------------------------- refusals (host)
P = ctypes.c_void_p
FAKE, ODD, WS = P(0x10000), P(0x10008), P(0x20000)  # never dereferenced


def test_tile_and_workspace_sizes(lib):
    assert dca.dca_kv4_tile_bytes(128) == 9216 and dca.dca_kv4_tile_bytes(64) == 4608
    assert dca.dca_kv4_tile_bytes(96) == 0
    assert dca.dca_attn_decode_kv4_workspace(0, 8, 1, 128, 64) == 0
    # a slot of 8 heads x (D + 2) floats for every unit (sequence, kv head, 8
    # query heads) and every share; a share is four tiles, a unit its tiles and
    # 8 more, and there are 3 shares an SM at most unless one passes 512 tiles
    def slots(B, Hkv, groups, Tcap):
        units = B * Hkv * groups
        tiles = units * (-(-Tcap // 64) + 8)
        return units + max(1, min(tiles // 4, max(148 * 3, -(-tiles // 512))))

    for B, Hq, Hkv, D, Tcap in ((1, 8, 1, 128, 64), (1, 8, 1, 64, 129), (16, 64, 8, 128, 65536),
                                (3, 20, 2, 64, 1000), (64, 64, 64, 128, 1 << 20)):
        want = slots(B, Hkv, -(-(Hq // Hkv) // 8), Tcap) * 8 * (D + 2) * 4
        assert dca.dca_attn_decode_kv4_workspace(B, Hq, Hkv, D, Tcap) == want
    assert dca.dca_attn_decode_kv4_workspace(1, 8, 3, 128, 64) == 0
    assert dca.dca_attn_decode_kv4_workspace(1, 8, 1, 128, 0) == 0
    assert dca.dca_pages_workspace(0, 1, 1) > 0 and dca.dca_pages_workspace(-1, 1, 1) == 0
    assert dca.dca_pages_workspace(4, 0, 10) == 0 and dca.dca_pages_workspace(4, 3, 0) == 0


def _append(lib, k=FAKE, v=FAKE, pool=FAKE, table=FAKE, mb=4, br=64, nb=8, cu=FAKE, t0=FAKE, B=2,
            T=5, Hkv=2, D=128, s=8, c=12, base=1e4):
    return int(lib.dca_kv4_append_paged(k, v, pool, table, mb, br, nb, cu, t0, B, T, Hkv, D, s, c,
                                        base, None))


@pytest.mark.parametrize("want,args", [
    (1, dict(k=None)), (1, dict(v=ODD)), (1, dict(pool=None)), (1, dict(table=None)),
    (1, dict(cu=None)), (1, dict(t0=P(0x10002))), (1, dict(table=P(0x10001))),
    (1, dict(mb=0)), (1, dict(nb=0)), (2, dict(br=32)), (2, dict(br=96)), (2, dict(D=96)),
    (1, dict(B=-1)), (1, dict(T=-1)), (1, dict(Hkv=0)), (2, dict(s=13)), (1, dict(s=0)),
    (1, dict(base=0.0)), (1, dict(mb=1 << 25)), (2, dict(Hkv=70000)), (2, dict(B=70000)),
    (0, dict(B=0)), (0, dict(T=0, table=None)),
])
def test_append_refusals(lib, want, args):
    assert _append(lib, **args) == want


def _read(lib, pool=FAKE, table=FAKE, mb=4, br=64, nb=8, cu=FAKE, t0=FAKE, K=FAKE, V=FAKE, B=2,
          T=5, Hkv=2, D=128, out_rows=0):
    return int(lib.dca_kv4_read_paged(pool, table, mb, br, nb, cu, t0, K, V, B, T, Hkv, D,
                                      out_rows, None))


@pytest.mark.parametrize("want,args", [
    (1, dict(pool=ODD)), (1, dict(table=None)), (1, dict(cu=None)), (1, dict(t0=None)),
    (1, dict(K=None)), (1, dict(V=ODD)), (1, dict(out_rows=-1)), (2, dict(br=65)),
    (2, dict(D=32)), (0, dict(T=0)),
])
def test_read_refusals(lib, want, args):
    assert _read(lib, **args) == want


def _decode(lib, q=FAKE, pool=FAKE, table=FAKE, mb=4, br=64, nb=8, t=FAKE, O=FAKE, LSE=FAKE, B=2,
            Hq=4, Hkv=2, D=128, s=8, c=12, base=1e4, ws=WS, nbytes=None):
    if nbytes is None:
        nbytes = dca.dca_attn_decode_kv4_workspace(B, Hq, Hkv, D, mb * br)
    return int(lib.dca_attn_decode_kv4_paged(q, pool, table, mb, br, nb, t, O, LSE, B, Hq, Hkv, D,
                                             s, c, base, 0.0, ws, nbytes, None))


@pytest.mark.parametrize("want,args", [
    (1, dict(q=None)), (1, dict(pool=ODD)), (1, dict(table=None)), (1, dict(t=None)),
    (1, dict(O=None)), (1, dict(LSE=None)), (1, dict(ws=None)), (5, dict(nbytes=16)),
    (2, dict(Hq=5)), (2, dict(D=80)), (2, dict(br=100)), (1, dict(mb=0)), (2, dict(s=20)),
    (1, dict(B=-1)), (0, dict(B=0)),
])
def test_decode_refusals(lib, want, args):
    assert _decode(lib, **args) == want


class _PagePool(ctypes.Structure):
    _fields_ = [("base", ctypes.c_void_p), ("unit_bytes", ctypes.c_size_t),
                ("outer", ctypes.c_int), ("unit_rows", ctypes.c_int)]


def _pool(base=0x30000, unit=256, outer=1, rows=1):
    p = (_PagePool * 1)()
    p[0] = (base, unit, outer, rows)
    return ctypes.byref(p)


def _remap(lib, src=FAKE, old=FAKE, new=FAKE, table=FAKE, refs=FAKE, tout=FAKE, rout=FAKE,
           info=FAKE, B=2, mb=4, nb=8, br=64, pools=None, n=0, ws=WS, nbytes=1 << 20):
    return int(lib.dca_pages_remap(src, old, new, table, refs, tout, rout, info, B, mb, nb, br,
                                   pools, n, ws, nbytes, None))


def _compact(lib, lens=FAKE, table=FAKE, refs=FAKE, tout=FAKE, rout=FAKE, moved=FAKE, info=FAKE,
             B=2, mb=4, nb=8, br=64, pools=None, n=0, ws=WS, nbytes=1 << 20):
    return int(lib.dca_pages_compact(lens, table, refs, tout, rout, moved, info, B, mb, nb, br,
                                     pools, n, ws, nbytes, None))


SHARED = [
    (1, dict(table=None)), (1, dict(refs=None)), (1, dict(tout=P(0x10001))), (1, dict(rout=None)),
    (1, dict(info=None)), (1, dict(B=-1)), (1, dict(mb=0)), (1, dict(nb=0)), (1, dict(br=0)),
    (1, dict(n=1)), (1, dict(n=-1)), (1, dict(n=300, pools=1)), (1, dict(ws=None)),
    (5, dict(nbytes=100)), (2, dict(mb=1 << 30)), (2, dict(nb=(1 << 30) + 1)),
    (1, dict(n=1, pools=dict(base=0))), (1, dict(n=1, pools=dict(base=0x30008))),
    (1, dict(n=1, pools=dict(unit=0))), (1, dict(n=1, pools=dict(unit=24))),
    (1, dict(n=1, pools=dict(outer=0))), (1, dict(n=1, pools=dict(rows=0))),
    (1, dict(n=1, pools=dict(rows=48))), (2, dict(n=1, pools=dict(unit=1 << 30, outer=1 << 20))),
]


@pytest.mark.parametrize("call", [_remap, _compact])
@pytest.mark.parametrize("want,args", SHARED)
def test_page_refusals(lib, call, want, args):
    args = dict(args)
    if "pools" in args:
        args["pools"] = _pool(**(args["pools"] if isinstance(args["pools"], dict) else {}))
    assert call(lib, **args) == want


@pytest.mark.parametrize("call", [_remap, _compact])
def test_page_pools_too_large_together(lib, call):
    # each page is 2^40 bytes, which one pool may have; 256 of them are more than
    # the copies can number
    pools = (_PagePool * 256)(*[(0x30000, 1 << 20, 1 << 20, 64)] * 256)
    assert call(lib, n=256, pools=ctypes.byref(pools)) == 2


@pytest.mark.parametrize("call,args", [(_remap, dict(src=None)), (_remap, dict(old=None)),
                                       (_remap, dict(new=P(0x10001))),
                                       (_compact, dict(lens=None)), (_compact, dict(moved=None))])
def test_page_list_refusals(lib, call, args):
    assert call(lib, **args) == 1


def test_wrappers_refuse_cpu_tensors():
    x = torch.zeros(1, 1, 128, dtype=torch.bfloat16)
    i = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(dca.DcaError):
        dca.dca_kv4_append_paged(x, x, i, i, i, i, 4, 6)
    with pytest.raises(dca.DcaError):
        dca.dca_attn_decode_kv4_paged(x, i, i, i, 4, 6)
    with pytest.raises(dca.DcaError):
        dca.dca_pages_remap(i, i, i, i, i, [], 64)
    with pytest.raises(dca.DcaError):
        dca.dca_pages_compact(i, i, i, [], 64)

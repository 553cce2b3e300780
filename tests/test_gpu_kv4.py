"""The paged 4-bit cache on the GPU: append, read back and decode against the
plain fp64 restatement.

Append is held to equality, byte for byte: its roundings are those of the exact
result, which the oracle forms in fp64 (an element nearer to a border than fp64
can tell would need a coincidence of about 1e-12).  Decode is held to the
oracle's own bounds: an fp16 rounding of P times the value scale, a bf16 one of
the output, and fp32 arithmetic besides.
"""

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
from oracle import dca_oracle as orc
from oracle import kv4_oracle as ko
from tests import kv4_util as ku

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_attention_dca_b200 import build
    build.build()
    dca.lib()
    yield
    dca.dca_sync_status()


def _cu(lens):
    return np.concatenate(([0], np.cumsum(lens))).astype(np.int32)


def _append_case(seed, lens, t0, Hkv, D, R, s, base=10000.0, pad=0, k=None, v=None):
    """Append on the GPU and in the oracle; both pools (uint8 NumPy)."""
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    cu = _cu(lens)
    T = int(cu[-1]) + pad
    k = ku.bf16_rows(gen, T, Hkv, D) if k is None else k
    v = ku.bf16_rows(gen, T, Hkv, D) if v is None else v
    table, num = ku.random_tables(rng, [a + n for a, n in zip(t0, lens)], R)
    pool = rng.integers(0, 256, (num, Hkv, R // 64, ko.tile_bytes(D)), dtype=np.uint8)
    want = pool.copy()
    ko.append(ku.f64(k), ku.f64(v), want, table, cu, t0, s, base)
    got = torch.from_numpy(pool).cuda()
    dca.dca_kv4_append_paged(k.cuda(), v.cuda(), got, ku.ints(table), ku.ints(cu), ku.ints(t0), s,
                             s + 5, base)
    dca.dca_sync_status()
    return got, want, table, cu, k, v


@pytest.mark.parametrize("D,Hkv,R,lens,t0,s", [
    (128, 1, 64, [1], [0], 5), (64, 1, 64, [1], [0], 5),
    (128, 2, 64, [3, 0, 70], [0, 9, 61], 100), (64, 2, 64, [3, 0, 70], [0, 9, 61], 100),
    (128, 3, 192, [1, 1, 1, 1, 1], [0, 63, 64, 191, 192], 50),
    (64, 5, 128, [1, 1, 1, 1, 1], [0, 63, 64, 127, 128], 50),
    (128, 8, 128, [130, 17], [5, 100], 33), (64, 8, 128, [130, 17], [5, 100], 33),
    (128, 4, 256, [65], [1000], 1), (128, 1, 64, [200], [37], 7),
])
def test_append_stores_what_the_oracle_stores(D, Hkv, R, lens, t0, s):
    got, want, *_ = _append_case(1, lens, t0, Hkv, D, R, s)
    assert ku.same_pool(got, want) is None


@pytest.mark.parametrize("D", [64, 128])
def test_append_at_far_positions_and_other_bases(D):
    # positions up to 3e6 inside one chunk: the angle carries the whole error
    for seed, t0, s, base in ((2, 2_999_900, 4_000_000, 10000.0), (3, 70_000, 100_000, 5e5),
                              (4, 123, 1000, 2.0)):
        rng = np.random.default_rng(seed)
        gen = torch.Generator().manual_seed(seed)
        R, n, Hkv = 64, 90, 2
        k, v = ku.bf16_rows(gen, n, Hkv, D), ku.bf16_rows(gen, n, Hkv, D)
        blocks = -(-(t0 + n) // R)
        table = np.zeros((1, blocks), np.int32)
        table[0, t0 // R:] = rng.permutation(4)[:blocks - t0 // R]
        want = np.zeros((4, Hkv, 1, ko.tile_bytes(D)), np.uint8)
        ko.append(ku.f64(k), ku.f64(v), want, table, [0, n], [t0], s, base)
        got = torch.zeros(want.shape, dtype=torch.uint8, device="cuda")
        dca.dca_kv4_append_paged(k.cuda(), v.cuda(), got, ku.ints(table), ku.ints([0, n]),
                                 ku.ints([t0]), s, s, base)
        dca.dca_sync_status()
        assert ku.same_pool(got, want) is None


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_unusual_values(D):
    gen = torch.Generator().manual_seed(5)
    n, Hkv = 26, 2
    v = torch.randn(n, Hkv, D, generator=gen)
    v[0] = 0.0
    v[1] = -0.0
    v[2] = 0.3333
    v[3] *= 1e-38
    v[4] *= 1e-40          # subnormals
    v[5] = torch.where(v[5] > 0, 3.3e38, -3.3e38)
    v[6] *= 1e37
    v[7, :, 3] = float("inf")
    v[8, :, D - 1] = float("-inf")
    v[9, 1, 5] = float("nan")
    v[10] = 1000.0 + v[10]                          # an offset many steps away
    v[11] = torch.arange(D) % 16 * 2.0 - 15         # every code exactly
    v[12] = (torch.arange(D) % 31 - 15.0).clamp(-15, 15)   # ties half way
    v[13] = torch.where(torch.arange(D) % 2 == 0, 1e-30, 1.0)
    v[14] = torch.where(torch.arange(D) % 2 == 0, 1.0, 1.0078125)
    v[15, :, 0] = 1e30
    v[16] = torch.tensor([-15.0, 15.0] + [1e-30, -1e-30, 0.0, 2.0] * ((D - 2) // 4) + [0.0] * 2)[:D]
    v[17:] = (v[17:] * 4).round() / 4               # coarse values: many ties
    v = v.to(torch.bfloat16)
    # keys at position 0 (s = 1): the rotation is the identity, so they are the
    # same numbers, and the last element's infinity reaches its partner's group
    got, want, *_ = _append_case(5, [n], [3], Hkv, D, 64, 1, k=v.clone(), v=v)
    assert ku.same_pool(got, want) is None


@pytest.mark.parametrize("D", [64, 128])
def test_append_of_keys_that_cancel_or_leave_the_normal_range(D):
    # pairs whose rotation nearly vanishes: p = q tan(angle) rounded to bf16 leaves
    # 2^-9 of the operands at most, and now and then 2^-13 and far less
    gen = torch.Generator().manual_seed(15)
    n, Hkv, t0, s = 700, 2, 40, 5000
    k = ku.bf16_rows(gen, n, Hkv, D)
    pos = torch.arange(t0, t0 + n, dtype=torch.float64)[:, None]
    theta = 10000.0 ** (-2.0 * torch.arange(D // 2, dtype=torch.float64) / D)
    tan = torch.tan(pos * theta)[:, None, :]
    q = k[..., D // 2:].double()
    p = torch.where(tan.abs() < 1e4, q * tan, q)
    k[..., :D // 2] = p.to(torch.bfloat16)
    got, want, *_ = _append_case(15, [n], [t0], Hkv, D, 64, s, k=k)
    assert ku.same_pool(got, want) is None
    # subnormals, sums next to them and next to the largest bf16
    k = torch.randn(120, Hkv, D, generator=gen)
    for i, size in enumerate((1e-30, 1e-36, 1e-37, 1e-38, 3e-39, 1e-39, 1e-40, 6e-41, 1e37, 5e37,
                              1e38, 1.7e38)):
        k[i * 10:i * 10 + 10] *= size
    k = k.clamp(-3.38e38, 3.38e38).to(torch.bfloat16)
    got, want, *_ = _append_case(16, [120], [t0], Hkv, D, 64, s, k=k, v=k.clone())
    assert ku.same_pool(got, want) is None


def test_append_ignores_rows_of_no_sequence_and_keeps_the_rest():
    # _append_case compares whole pools, random bytes elsewhere included
    got, want, *_ = _append_case(6, [9, 20], [60, 1], 2, 128, 64, 10, pad=77)
    assert ku.same_pool(got, want) is None


def test_append_split_into_calls_is_the_same_cache():
    got, want, table, cu, k, v = _append_case(7, [150], [20], 3, 128, 64, 40)
    again = torch.zeros_like(got)
    at = 0
    for n in (1, 1, 15, 64, 2, 67):
        dca.dca_kv4_append_paged(k[at:at + n].contiguous().cuda(), v[at:at + n].contiguous().cuda(),
                                 again, ku.ints(table), ku.ints([0, n]), ku.ints([20 + at]), 40, 45)
        at += n
    dca.dca_sync_status()
    a = dca.dca_kv4_read_paged(got, ku.ints(table), ku.ints([0, 150]), ku.ints([20]), 150, 128)
    b = dca.dca_kv4_read_paged(again, ku.ints(table), ku.ints([0, 150]), ku.ints([20]), 150, 128)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_append_skips_and_reports_what_does_not_fit():
    D, Hkv, R = 128, 2, 64
    gen = torch.Generator().manual_seed(8)
    k, v = ku.bf16_rows(gen, 12, Hkv, D), ku.bf16_rows(gen, 12, Hkv, D)
    cases = [
        ([0, 4, 8, 12], [0, 126, 0], [[0, 1], [2, 3], [4, 5]]),   # past the cache
        ([0, 4, 8, 12], [0, -1, 0], [[0, 1], [2, 3], [4, 5]]),    # before it
        ([0, 4, 8, 12], [0, 0, 0], [[0, 1], [9, 3], [4, 5]]),     # no such page
        ([0, 4, 8, 12], [0, 0, 0], [[0, 1], [-1, 3], [4, 5]]),
    ]
    for cu, t0, table in cases:
        got = torch.zeros((6, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
        want = np.zeros(got.shape, np.uint8)
        for b in (0, 2):
            ko.append(ku.f64(k[cu[b]:cu[b + 1]]), ku.f64(v[cu[b]:cu[b + 1]]), want,
                      np.array(table[b:b + 1]), [0, 4], [t0[b]], 10)
        dca.dca_kv4_append_paged(k.cuda(), v.cuda(), got, ku.ints(table), ku.ints(cu), ku.ints(t0),
                                 10, 12)
        with pytest.raises(dca.DcaError) as ei:
            dca.dca_sync_status()
        assert ei.value.status == 1
        assert ku.same_pool(got, want) is None
        dca.dca_sync_status()
    # offsets past the rows: only the sequence inside [0, T) is stored
    got = torch.zeros((6, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
    dca.dca_kv4_append_paged(k.cuda(), v.cuda(), got, ku.ints([[0, 1], [2, 3]]),
                             ku.ints([0, 4, 30]), ku.ints([0, 0]), 10, 12)
    with pytest.raises(dca.DcaError):
        dca.dca_sync_status()
    assert got[0].any() and not got[1:].any()


@pytest.mark.parametrize("D", [64, 128])
def test_read_gives_the_stored_values_packed_and_as_a_cache(D):
    rng = np.random.default_rng(9)
    Hkv, R, lens, t0 = 3, 64, [5, 0, 90, 1], [60, 3, 0, 127]
    table, num = ku.random_tables(rng, [a + n for a, n in zip(t0, lens)], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    cu = _cu(lens)
    T = int(cu[-1])
    dev = (torch.from_numpy(pool).cuda(), ku.ints(table), ku.ints(cu), ku.ints(t0))
    K, V = dca.dca_kv4_read_paged(*dev, T, D)
    Kc = torch.full((4, 130, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    Vc = Kc.clone()
    dca.dca_kv4_read_paged(*dev, T, D, Kc, Vc)
    dca.dca_sync_status()
    for b, n in enumerate(lens):
        if n:
            got = ko.cache(pool, table, b, t0[b] + n, D)
            for what, packed, cache in (("k", K, Kc), ("v", V, Vc)):
                want = ko.bf16(ko.values(*got[what])[t0[b]:])
                assert np.array_equal(ku.f64(packed[cu[b]:cu[b + 1]]), want)
                assert np.array_equal(ku.f64(cache[b, t0[b]:t0[b] + n]), want)
                assert (cache[b, :t0[b]] == 7).all() and (cache[b, t0[b] + n:] == 7).all()
    # a cache too short for a sequence: that one is skipped and reported
    short = torch.full((4, 100, Hkv, D), 7.0, dtype=torch.bfloat16, device="cuda")
    dca.dca_kv4_read_paged(*dev, T, D, short, short.clone())
    with pytest.raises(dca.DcaError):
        dca.dca_sync_status()
    assert (short[3] == 7).all() and not (short[0, 60:65] == 7).all()


def _with_room(table, rows, R):
    """The table with room for that many more rows, named by no page."""
    return np.pad(table, ((0, 0), (0, -(-rows // R))), constant_values=-1)


def _decode_case(seed, D, Hq, Hkv, R, t, s, c, base=10000.0, scale=0.0, q=None, pool=None,
                 table=None, rows=0):
    rng = np.random.default_rng(seed)
    gen = torch.Generator().manual_seed(seed)
    if table is None:
        table, num = ku.random_tables(rng, [x + 1 for x in t], R)
        pool = ku.random_pool(rng, num, Hkv, R, D)
        for b, x in enumerate(t):  # NaN parameters in every row past the last
            page, r0 = table[b, x // R], x % R + 1
            for r in range(r0, R):
                tile = pool[page]
                for h in range(Hkv):
                    for what in ("k", "v"):
                        ko.write_row(tile[h, r // 64], what, r % 64, np.full(D, 15, np.uint8),
                                     np.full(D // 64, np.nan), np.full(D // 64, np.nan))
    q = ku.bf16_rows(gen, len(t), Hq, D) if q is None else q
    table = _with_room(table, rows, R)
    got = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(), ku.ints(table),
                                        ku.ints(t), s, c, base, scale)
    dca.dca_sync_status()
    want = ko.decode(ku.f64(q), pool, table, t, s, c, base, scale)
    return got, want


def _close(got, want, what=""):
    (O, LSE), (Ow, Lw, bO, bL) = got, want
    eo, el = np.abs(ku.f64(O) - Ow), np.abs(ku.f64(LSE) - Lw)
    assert (eo <= bO).all(), (what, float((eo / bO).max()))
    assert (el <= bL).all(), (what, float((el / bL).max()))


@pytest.mark.parametrize("D,Hq,Hkv,R,t,s,c", [
    (128, 1, 1, 64, [0], 4, 6), (64, 1, 1, 64, [0], 4, 6),
    (128, 8, 1, 64, [1, 63, 64, 65], 100, 130), (64, 8, 1, 64, [1, 63, 64, 65], 100, 130),
    (128, 16, 2, 128, [300, 0, 511, 127], 64, 100), (64, 16, 2, 192, [300, 0, 511, 127], 64, 100),
    (128, 12, 1, 64, [200, 31], 50, 50), (64, 20, 2, 64, [129], 7, 11),
    (128, 3, 3, 256, [255, 256], 1, 1), (64, 5, 5, 64, [400], 333, 500),
    (128, 6, 2, 64, [1000, 5], 16, 40), (128, 8, 8, 64, [777], 256, 384),
])
def test_decode_matches_the_oracle(D, Hq, Hkv, R, t, s, c):
    _close(*_decode_case(10, D, Hq, Hkv, R, t, s, c))


@pytest.mark.parametrize("D,Hq,Hkv,R,t,s,c", [
    (128, 1, 1, 64, [0], 4, 6), (64, 8, 1, 64, [1, 63, 64, 65], 100, 130),
    (128, 16, 2, 128, [300, 0, 511, 127], 64, 100), (64, 20, 2, 64, [129], 7, 11),
    (128, 3, 3, 256, [255, 256], 1, 1), (64, 5, 5, 64, [400], 333, 500),
    (128, 24, 24, 64, [700, 9, 40], 256, 384), (64, 90, 30, 64, [1, 2, 63, 64, 2047, 900], 99, 120),
    (128, 99, 33, 128, [2047, 5, 128, 0, 640], 500, 600),
])
def test_decode_of_short_sequences_in_caches_of_any_size(D, Hq, Hkv, R, t, s, c):
    # a CTA a unit where the cache is short, shares where it has room for more
    for rows in (0, 4096):
        _close(*_decode_case(12, D, Hq, Hkv, R, t, s, c, rows=rows), rows)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("G", [1, 4, 5, 8, 12])
def test_decode_of_a_few_keys_keeps_fp32_scores(D, G):
    # With one to four keys LSE is a score or nearly one, of size about 1 for normal
    # q and k.  Its roundings, each of 2^-24 / sqrt(3) rms of what it rounds, are:
    # three for every rotated element (6e-8 of the score in all); 64 in each of the
    # six levels of a group's sum of q, of 64 / 2^n elements of size sqrt(2^n) (8 * sqrt(6)
    # * 3.4e-8 = 7e-7, times an offset of 2.5 over sqrt(128): 1.5e-7, sqrt(2) of that
    # for two groups); some six of the products scale * sum(q c) and offset * sum(q), of
    # size 2 each (2e-7).  The integer parts of the query sum exactly and their
    # remainders are 2^-11 of them.  Together 3.5e-7 rms; 1e-6 is allowed.
    rng, gen = np.random.default_rng(31), torch.Generator().manual_seed(31)
    B, Hkv, R, s = 24, 4, 64, 3
    t = [b % 4 for b in range(B)]
    lens = [x + 1 for x in t]
    k, v = (torch.randn(sum(lens), Hkv, D, generator=gen).bfloat16() for _ in range(2))
    table, num = ku.random_tables(rng, lens, R)
    pool = np.zeros((num, Hkv, 1, ko.tile_bytes(D)), np.uint8)
    ko.append(ku.f64(k), ku.f64(v), pool, table, _cu(lens), [0] * B, s)
    q = torch.randn(B, Hkv * G, D, generator=gen).bfloat16()
    (O, LSE), want = _decode_case(31, D, Hkv * G, Hkv, R, t, s, 5, q=q, pool=pool, table=table)
    _close((O, LSE), want)
    off = ku.f64(LSE) - want[1]
    assert np.sqrt((off ** 2).mean()) <= 1e-6 * np.sqrt((want[1] ** 2).mean())


@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_long_caches_in_many_shares(D):
    # more tiles than shares, a ragged batch, and a capacity far past every t
    rng = np.random.default_rng(11)
    t, R, Hkv = [9000, 4095, 20], 128, 2
    table, num = ku.random_tables(rng, [x + 1 for x in t], R, most=400)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    _close(*_decode_case(11, D, 16, Hkv, R, t, 1000, 1500, table=table, pool=pool))


def test_decode_with_other_bases_scales_and_large_queries():
    for seed, base, scale, mult in ((12, 5e5, 0.0, 1.0), (13, 10000.0, 0.3, 0.2),
                                    (14, 10000.0, -0.1, 1.0), (15, 10000.0, 0.0, 1e-20),
                                    (16, 10000.0, 1e-30, 1e30), (17, 10000.0, 0.0, 0.0)):
        gen = torch.Generator().manual_seed(seed)
        q = (torch.randn(2, 8, 128, generator=gen) * mult).to(torch.bfloat16)
        _close(*_decode_case(seed, 128, 8, 2, 64, [150, 70], 40, 60, base, scale, q=q), seed)


def test_decode_of_values_whose_scales_span_many_decades():
    rng = np.random.default_rng(18)
    t, R, D, Hkv = [300], 64, 128, 2
    table, num = ku.random_tables(rng, [301], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    for j in range(301):
        for h in range(Hkv):
            x = ko.bf16(rng.standard_normal(D) * 10.0 ** rng.uniform(-12, 12))
            ko.write_row(ko._tile(pool, table, 0, j, h), "v", j % 64, *ko.quantise(x))
    _close(*_decode_case(18, D, 8, Hkv, R, t, 100, 150, table=table, pool=pool))


@pytest.mark.parametrize("rows", [0, 4096])
def test_decode_reads_nan_rows_as_nan_and_only_there(rows):
    rng = np.random.default_rng(19)
    D, Hkv, R, t = 128, 2, 64, [100, 100]
    table, num = ku.random_tables(rng, [101, 101], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    nan = (np.zeros(D, np.uint8), np.full(2, np.nan), np.full(2, np.nan))
    ko.write_row(ko._tile(pool, table, 0, 70, 0), "k", 70 % 64, *nan)           # key: all of head 0
    ko.write_row(ko._tile(pool, table, 1, 3, 1), "v", 3, nan[0],
                 np.array([0.1, np.nan]), np.array([0.0, np.nan]))               # one value group
    gen = torch.Generator().manual_seed(19)
    q = ku.bf16_rows(gen, 2, 4, D)
    O, LSE = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(),
                                           ku.ints(_with_room(table, rows, R)), ku.ints(t), 30, 40)
    dca.dca_sync_status()
    bad = torch.isnan(O.cpu())
    want = torch.zeros_like(bad)
    want[0, :2] = True
    want[1, 2:, 64:] = True
    assert torch.equal(bad, want)
    assert torch.equal(torch.isnan(LSE.cpu()), torch.tensor([[True, True, False, False],
                                                            [False] * 4]))


@pytest.mark.parametrize("rows", [0, 4096])
def test_decode_reports_bad_positions_and_pages(rows):
    rng = np.random.default_rng(20)
    D, Hkv, R = 128, 2, 64
    table, num = ku.random_tables(rng, [128, 128, 128], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    gen = torch.Generator().manual_seed(20)
    q = ku.bf16_rows(gen, 3, 4, D)
    want = ko.decode(ku.f64(q), pool, table, [127, 127, 127], 30, 40)
    for t, entry in (([127, 128, 127], None), ([127, -1, 127], None), ([127, 127, 127], num),
                     ([127, 127, 127], -1)):
        tab = _with_room(table, rows, R)
        if entry is not None:
            tab[1, 1] = entry
        O, LSE = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(),
                                               ku.ints(tab), ku.ints(t), 30, 40)
        with pytest.raises(dca.DcaError) as ei:
            dca.dca_sync_status()
        assert ei.value.status == 1
        assert torch.isnan(O[1]).all() and torch.isnan(LSE[1]).all()
        keep = [0, 2]
        _close((O[keep], LSE[keep]), tuple(x[keep] for x in want))
    # an entry past the sequence's last page is not read
    tab = np.concatenate([table, np.full((3, 2), 1 << 30, np.int32)], 1)
    got = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(), ku.ints(tab),
                                        ku.ints([127] * 3), 30, 40)
    dca.dca_sync_status()
    _close(got, want)


def test_decode_with_an_empty_batch_and_given_outputs():
    rng = np.random.default_rng(21)
    table, num = ku.random_tables(rng, [90], 64)
    pool = torch.from_numpy(ku.random_pool(rng, num, 1, 64, 64)).cuda()
    q = torch.randn(1, 4, 64).to(torch.bfloat16).cuda()
    O, LSE = dca.dca_attn_decode_kv4_paged(q[:0].contiguous(), pool, ku.ints(table[:0]),
                                           ku.ints([]), 30, 40)
    assert O.shape == (0, 4, 64) and LSE.shape == (0, 4)
    ws = torch.empty(dca.dca_attn_decode_kv4_workspace(1, 4, 1, 64, 128), dtype=torch.uint8,
                     device="cuda")
    ws.fill_(0xFF)  # nothing in it needs to start at any value
    a = dca.dca_attn_decode_kv4_paged(q, pool, ku.ints(table), ku.ints([89]), 30, 40)
    Og, Lg = torch.empty_like(q), torch.empty(1, 4, device="cuda")
    b = dca.dca_attn_decode_kv4_paged(q, pool, ku.ints(table), ku.ints([89]), 30, 40,
                                      workspace=ws, O=Og, LSE=Lg)
    dca.dca_sync_status()
    assert b[0] is Og and torch.equal(a[0], Og) and torch.equal(a[1], Lg)
    with pytest.raises(dca.DcaError) as ei:
        dca.dca_attn_decode_kv4_paged(q, pool, ku.ints(table), ku.ints([89]), 30, 40,
                                      workspace=ws[:16])
    assert ei.value.status == 5


def test_append_and_decode_on_a_stream_and_in_a_graph():
    rng = np.random.default_rng(22)
    gen = torch.Generator().manual_seed(22)
    D, Hq, Hkv, R, s, c, n = 128, 8, 2, 64, 50, 70, 140
    k, v = ku.bf16_rows(gen, n, Hkv, D).cuda(), ku.bf16_rows(gen, n, Hkv, D).cuda()
    q = ku.bf16_rows(gen, n, Hq, D).cuda()
    table, num = ku.random_tables(rng, [n], R)
    table = ku.ints(table)
    one = ku.ints([0, 1])
    # the plain loop
    pool = torch.zeros((num, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
    want = []
    for j in range(n):
        t = ku.ints([j])
        dca.dca_kv4_append_paged(k[j:j + 1], v[j:j + 1], pool, table, one, t, s, c)
        O, _ = dca.dca_attn_decode_kv4_paged(q[j:j + 1], pool, table, t, s, c)
        want.append(O.clone())
    # the same step captured once and replayed with new inputs, on another stream
    pool2 = torch.zeros_like(pool)
    kb, vb, qb, tb = k[:1].clone(), v[:1].clone(), q[:1].clone(), ku.ints([0])
    ws = torch.empty(dca.dca_attn_decode_kv4_workspace(1, Hq, Hkv, D, table.shape[1] * R),
                     dtype=torch.uint8, device="cuda")
    Ob, Lb = torch.empty_like(qb), torch.empty(1, Hq, device="cuda")
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())

    def step():
        dca.dca_kv4_append_paged(kb, vb, pool2, table, one, tb, s, c)
        dca.dca_attn_decode_kv4_paged(qb, pool2, table, tb, s, c, workspace=ws, O=Ob, LSE=Lb)

    with torch.cuda.stream(side):
        step()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        for j in range(n):
            kb.copy_(k[j:j + 1])
            vb.copy_(v[j:j + 1])
            qb.copy_(q[j:j + 1])
            tb.fill_(j)
            graph.replay()
            assert torch.equal(Ob, want[j]), j
    torch.cuda.current_stream().wait_stream(side)
    dca.dca_sync_status()
    a = dca.dca_kv4_read_paged(pool, table, ku.ints([0, n]), ku.ints([0]), n, D)
    b = dca.dca_kv4_read_paged(pool2, table, ku.ints([0, n]), ku.ints([0]), n, D)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_prompt_then_chunk_then_tokens_over_a_4bit_cache():
    """A conversation: the prompt's prefill goes to the 4-bit cache; its next
    turn reads the prefix into a bf16 cache, runs a packed chunk over it and
    appends the chunk; decode goes on over the 4-bit cache.  Each step against
    the bf16 calls on the values that the 4-bit cache stands for."""
    gen = torch.Generator().manual_seed(23)
    rng = np.random.default_rng(23)
    D, Hq, Hkv, R, s, c = 128, 8, 2, 64, 256, 384
    n0, n1 = 300, 45
    n = n0 + n1
    Q, K, V = (ku.bf16_rows(gen, n, h, D).cuda() for h in (Hq, Hkv, Hkv))
    table_np, num = ku.random_tables(rng, [n + 1], R)
    table = ku.ints(table_np)
    pool = torch.zeros((num, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
    cu0, zero = ku.ints([0, n0]), ku.ints([0])
    first = lambda x: x[:n0].contiguous()  # noqa: E731
    dca.dca_attn_prefill_varlen(first(Q), first(K), first(V), cu0, n0, s, c)
    dca.dca_kv4_append_paged(first(K), first(V), pool, table, cu0, zero, s, c)
    # next turn
    Tcap = 512
    Kc = torch.zeros((1, Tcap, Hkv, D), dtype=torch.bfloat16, device="cuda")
    Vc = torch.zeros_like(Kc)
    dca.dca_kv4_read_paged(pool, table, cu0, zero, n0, D, Kc, Vc)
    Kp, Vp = Kc[0, :n0].clone(), Vc[0, :n0].clone()
    rest = lambda x: x[n0:].contiguous()  # noqa: E731
    cu1, t0 = ku.ints([0, n1]), ku.ints([n0])
    O1, _ = dca.dca_attn_prefill_varlen_chunk(rest(Q), rest(K), rest(V), Kc, Vc, cu1, t0, n1, n, s,
                                              c)
    dca.dca_kv4_append_paged(rest(K), rest(V), pool, table, cu1, t0, s, c)
    dca.dca_sync_status()
    ref = orc.dca_prefill_varlen_chunk_rows(ku.f64(rest(Q)), ku.f64(rest(K)), ku.f64(rest(V)),
                                            [0, n1], [n0], ku.f64(Kp)[None], ku.f64(Vp)[None], s, c,
                                            rows=[0, n1 - 1])
    # P and the output are rounded to bf16 (half a step is 2^-8 of the value, and
    # sum p |v| <= max |v|); query and key are each rounded to fp16, 2^-11 of a
    # score's size together, which moves every weight by twice that at most
    qk = float(Q[n0:].float().abs().sum(-1).max() * Kc.float().abs().max()) / np.sqrt(D)
    most = (2.0 ** -7 + 2 * 2.0 ** -11 * qk) * float(Vc.float().abs().max())
    for (h, r), (o, _) in ref.items():
        assert np.abs(ku.f64(O1[r, h]) - o).max() < most
    # decode at the last token, against the bf16 decode of the read-back cache
    Kall, Vall = dca.dca_kv4_read_paged(pool, table, ku.ints([0, n]), zero, n, D)
    t = ku.ints([n - 1])
    q = Q[n - 1:].contiguous()
    O4, L4 = dca.dca_attn_decode_kv4_paged(q, pool, table, t, s, c)
    dca.dca_sync_status()
    Ob, Lb = dca.dca_attn_decode(q, Kall[None].contiguous(), Vall[None].contiguous(), t, s, c)
    dca.dca_sync_status()
    _close((O4, L4), ko.decode(ku.f64(q), pool.cpu().numpy(), table_np, [n - 1], s, c))
    # the bf16 cache rounds every stored value once more: 2^-8 of |k| in each
    # product and of |v| in each term
    wide = float((Q[n - 1].float().abs().sum(-1).max() * Kall.float().abs().max()) / np.sqrt(D))
    assert (L4 - Lb).abs().max() <= 2.0 ** -8 * wide
    assert (O4.float() - Ob.float()).abs().max() <= (2.0 ** -7 + 2 * 2.0 ** -8 * wide) * float(
        Vall.float().abs().max())


@pytest.mark.parametrize("D,Hq,Hkv", [(128, 6, 3), (64, 24, 2), (128, 4, 4)])
def test_decode_of_many_short_sequences(D, Hq, Hkv):
    # a CTA's share holds several (sequence, head) pieces; one bad page among them
    # makes that sequence NaN and no other
    rng = np.random.default_rng(24)
    B, R = 150, 64
    t = [int(x) for x in rng.integers(0, 150, B)]
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    gen = torch.Generator().manual_seed(24)
    q = ku.bf16_rows(gen, B, Hq, D)
    want = ko.decode(ku.f64(q), pool, table, t, 37, 60)
    dev = (q.cuda(), torch.from_numpy(pool).cuda())
    _close(dca.dca_attn_decode_kv4_paged(*dev, ku.ints(table), ku.ints(t), 37, 60), want)
    dca.dca_sync_status()
    bad = 71
    table[bad, 0] = num + 5
    O, LSE = dca.dca_attn_decode_kv4_paged(*dev, ku.ints(table), ku.ints(t), 37, 60)
    with pytest.raises(dca.DcaError):
        dca.dca_sync_status()
    assert torch.isnan(O[bad]).all() and torch.isnan(LSE[bad]).all()
    keep = [b for b in range(B) if b != bad]
    _close((O[keep], LSE[keep]), tuple(x[keep] for x in want))


def test_decode_with_sequences_outside_the_cache_among_others():
    # positions outside the cache anywhere in the batch, first and last too
    rng = np.random.default_rng(25)
    D, Hq, Hkv, R, B = 64, 8, 1, 64, 40
    t = [int(x) for x in rng.integers(0, 300, B)]
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    gen = torch.Generator().manual_seed(25)
    q = ku.bf16_rows(gen, B, Hq, D)
    want = ko.decode(ku.f64(q), pool, table, t, 50, 70)
    out = [0, 1, 17, 18, 39]
    tt = list(t)
    for b, x in zip(out, (-1, 100000, table.shape[1] * R, -2 ** 31, 2 ** 31 - 1)):
        tt[b] = x
    O, LSE = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(),
                                           ku.ints(table), ku.ints(tt), 50, 70)
    with pytest.raises(dca.DcaError):
        dca.dca_sync_status()
    assert torch.isnan(O[out]).all() and torch.isnan(LSE[out]).all()
    keep = [b for b in range(B) if b not in out]
    _close((O[keep], LSE[keep]), tuple(x[keep] for x in want))
    # none inside
    O, LSE = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(),
                                           ku.ints(table), ku.ints([-1] * B), 50, 70)
    with pytest.raises(dca.DcaError):
        dca.dca_sync_status()
    assert torch.isnan(O).all() and torch.isnan(LSE).all()


def test_decode_in_two_graphs_with_a_workspace_each():
    rng = np.random.default_rng(26)
    gen = torch.Generator().manual_seed(26)
    D, Hq, Hkv, R, s, c = 128, 8, 2, 64, 50, 70
    graphs = []
    for n in (300, 1100):
        table, num = ku.random_tables(rng, [n], R)
        pool = ku.random_pool(rng, num, Hkv, R, D)
        q = ku.bf16_rows(gen, 1, Hq, D)
        dev = (q.cuda(), torch.from_numpy(pool).cuda(), ku.ints(table), ku.ints([n - 1]))
        ws = torch.empty(dca.dca_attn_decode_kv4_workspace(1, Hq, Hkv, D, table.shape[1] * R),
                         dtype=torch.uint8, device="cuda")
        O, LSE = torch.empty_like(dev[0]), torch.empty(1, Hq, device="cuda")
        call = lambda: dca.dca_attn_decode_kv4_paged(  # noqa: E731
            *dev, s, c, workspace=ws, O=O, LSE=LSE)
        call()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        want = ko.decode(ku.f64(q), pool, table, [n - 1], s, c)
        graphs.append((graph, O, LSE, want, dev, ws))
    streams = [torch.cuda.Stream() for _ in graphs]
    for _ in range(20):  # both at once
        for stream, (graph, O, LSE, *_) in zip(streams, graphs):
            O.zero_()
            LSE.zero_()
        torch.cuda.synchronize()
        for stream, (graph, *_) in zip(streams, graphs):
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, O, LSE, want, *_ in graphs:
            _close((O, LSE), want)
    dca.dca_sync_status()


def test_pools_past_four_gigabytes():
    # the pages in use lie at the end of a pool of 4.7 GB, and pages are moved there
    D, Hq, Hkv, R = 128, 4, 8, 256
    num = 16000
    rng = np.random.default_rng(27)
    gen = torch.Generator().manual_seed(27)
    small, t = 5, [600]
    table = np.array([[num - 1, num - 3, num - 2]], np.int32)
    part = ku.random_pool(rng, small, Hkv, R, D)
    pool = torch.zeros((num, Hkv, R // 64, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
    assert pool.numel() > 2 ** 32
    pool[-small:] = torch.from_numpy(part).cuda()
    q = ku.bf16_rows(gen, 1, Hkv * Hq, D)
    at = table - (num - small)
    want = ko.decode(ku.f64(q), part, at, t, 300, 400)
    _close(dca.dca_attn_decode_kv4_paged(q.cuda(), pool, ku.ints(table), ku.ints(t), 300, 400),
           want)
    k, v = ku.bf16_rows(gen, 30, Hkv, D), ku.bf16_rows(gen, 30, Hkv, D)
    ko.append(ku.f64(k), ku.f64(v), part, at, [0, 30], [601], 300)
    dca.dca_kv4_append_paged(k.cuda(), v.cuda(), pool, ku.ints(table), ku.ints([0, 30]),
                             ku.ints([601]), 300, 400)
    dca.dca_sync_status()
    assert ku.same_pool(pool[-small:], part) is None
    K, V = dca.dca_kv4_read_paged(pool, ku.ints(table), ku.ints([0, 30]), ku.ints([601]), 30, D)
    got = ko.cache(part, at, 0, 631, D)
    assert np.array_equal(ku.f64(K), ko.bf16(ko.values(*got["k"])[601:]))
    assert np.array_equal(ku.f64(V), ko.bf16(ko.values(*got["v"])[601:]))
    # all pages but the last ones held besides, so that a fork's copy goes to num - 4
    refs = torch.ones(num, dtype=torch.int32, device="cuda")
    refs[num - 4] = 0
    both = torch.cat([ku.ints(table), torch.full_like(ku.ints(table), -1)])
    out, counts, info = dca.dca_pages_remap(ku.ints([0, 0]), ku.ints([631, 0]),
                                            ku.ints([631, 631]), both, refs, [pool], R)
    assert info.tolist() == [0, 1] and out.tolist()[1] == [num - 1, num - 3, num - 4]
    tiles = -(-(631 % R) // 64)
    assert torch.equal(pool[num - 4, :, :tiles], pool[num - 2, :, :tiles])
    assert torch.equal(pool[num - 4, :, tiles:].cpu(), torch.from_numpy(part[1, :, tiles:]))
    # and compaction moves the last page to a hole at the front
    refs = torch.ones(num, dtype=torch.int32, device="cuda")
    refs[7] = 0
    last = pool[-1].clone()
    out, counts, moved, info = dca.dca_pages_compact(ku.ints([631]), ku.ints(table), refs, [pool],
                                                     R)
    assert info.tolist() == [num - 1, 1] and out.tolist() == [[7, num - 3, num - 2]]
    assert torch.equal(pool[7], last) and int(moved[num - 1]) == 7
    dca.dca_sync_status()

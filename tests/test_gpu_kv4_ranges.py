"""Decode over the 4-bit cache at the ends of the number ranges: values, keys
and queries as large and as small as append and bf16 take them."""

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
from oracle import kv4_oracle as ko
from tests import kv4_util as ku
from tests.test_gpu_kv4 import _close, _with_room

pytestmark = pytest.mark.gpu

# A table as long as its sequences (a block a unit) and a longer one (shares).
ROWS = [0, 4096]


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_attention_dca_b200 import build
    build.build()
    dca.lib()
    yield
    dca.dca_sync_status()


def _decode(q, pool, table, t, s, c, rows, scale=0.0):
    out = dca.dca_attn_decode_kv4_paged(q.cuda(), torch.from_numpy(pool).cuda(),
                                        ku.ints(_with_room(table, rows, pool.shape[2] * 64)),
                                        ku.ints(t), s, c, scale=scale)
    dca.dca_sync_status()
    return out


def _forget_the_rest(pool, table, t, D):
    """NaN parameters in every row past a sequence's last one."""
    R = pool.shape[2] * 64
    for b, x in enumerate(t):
        for r in range(x % R + 1, R):
            for h in range(pool.shape[1]):
                for what in ("k", "v"):
                    ko.write_row(pool[table[b, x // R], h, r // 64], what, r % 64,
                                 np.full(D, 15, np.uint8), np.full(D // 64, np.nan),
                                 np.full(D // 64, np.nan))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_large_values_beside_constant_ones(D, G, rows):
    # Every tile, a partly filled last one too, has a row of the stated scale, rows of
    # equal values (their scale is 0, as append stores them) and ordinary rows.
    rng, gen = np.random.default_rng(41), torch.Generator().manual_seed(41)
    Hkv, R, s, c = 2, 64, 40, 60
    t = [100, 68, 30]
    q = ku.bf16_rows(gen, len(t), Hkv * G, D)
    for power in (13, 14, 15, 16, 17, 20, 100, 118):
        table, num = ku.random_tables(rng, [x + 1 for x in t], R)
        pool = ku.random_pool(rng, num, Hkv, R, D)
        _forget_the_rest(pool, table, t, D)
        gr = D // 64
        for b, x in enumerate(t):
            for first in range(0, x + 1, 64):
                for h in range(Hkv):
                    tile = ko._tile(pool, table, b, first, h)
                    big = np.full(gr, 1.5 * 2.0 ** power)
                    ko.write_row(tile, "v", 1, rng.integers(0, 16, D).astype(np.uint8), big,
                                 -7 * big)
                    zero = np.zeros(D, np.uint8)
                    ko.write_row(tile, "v", 0, zero, np.zeros(gr), np.zeros(gr))
                    ko.write_row(tile, "v", 3, zero, np.zeros(gr), big)
        got = _decode(q, pool, table, t, s, c, rows)
        _close(got, ko.decode(ku.f64(q), pool, table, t, s, c), (power, rows))


def _params(pool, D, what):
    """The bf16 parameters of all keys or values, uint16, as a view."""
    gr, nb = D // 64, 32 * D
    first = nb if what == "k" else 2 * nb + 256 * gr
    return pool[..., first:first + 256 * gr].view(np.uint16)


def _scaled(pool, D, what, power):
    """The pool with all scales and offsets of the keys or values times 2^power."""
    out = pool.copy()
    words = _params(out, D, what)
    words += np.array(power << 7).astype(np.uint16)  # to the exponent, modulo 2^16
    return out


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_scales_with_its_values(D, G, rows):
    # Every step up to the output's rounding commutes with a power of two as long as
    # nothing leaves the normal range, so the outputs are the same bits, moved.
    rng, gen = np.random.default_rng(42), torch.Generator().manual_seed(42)
    Hkv, R, s, c, t = 2, 64, 40, 60, [100, 68, 30]
    q = ku.bf16_rows(gen, len(t), Hkv * G, D)
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    O, LSE = _decode(q, pool, table, t, s, c, rows)
    _close((O, LSE), ko.decode(ku.f64(q), pool, table, t, s, c))
    for power in (-100, -85, -40, 14, 17, 40, 115):
        Ok, Lk = _decode(q, _scaled(pool, D, "v", power), table, t, s, c, rows)
        assert torch.equal(Lk, LSE), power
        assert torch.equal(Ok.double(), O.double() * 2.0 ** power), power


def _signed_rows(gen, *shape):
    """bf16 values of size 1 to 2, which any power of two keeps exact."""
    x = 1 + torch.randint(0, 128, shape, generator=gen) / 128.0
    return torch.where(torch.rand(shape, generator=gen) < 0.5, -x, x).to(torch.bfloat16)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_small_queries_over_large_keys(D, G, rows):
    # scores of a query times 2^-p over keys times 2^p are the same bits
    rng, gen = np.random.default_rng(43), torch.Generator().manual_seed(43)
    Hkv, R, s, c, t = 2, 64, 40, 60, [100, 68, 30]
    q = _signed_rows(gen, len(t), Hkv * G, D)
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    O, LSE = _decode(q, pool, table, t, s, c, rows)
    _close((O, LSE), ko.decode(ku.f64(q), pool, table, t, s, c))
    for power in (60, 100, 110, 114, 118, 122):
        got = _decode(q * 2.0 ** -power, _scaled(pool, D, "k", power), table, t, s, c, rows)
        assert torch.equal(got[1], LSE) and torch.equal(got[0], O), power


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8), (128, 1), (64, 12)])
def test_decode_of_queries_and_scales_next_to_nothing(D, G, rows):
    rng, gen = np.random.default_rng(44), torch.Generator().manual_seed(44)
    Hkv, R, s, c, t = 2, 64, 40, 60, [100, 68, 0]
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    for size, scale in ((4e-35, 0.0), (1e-35, 0.0), (1e-38, 0.0), (1e-40, 0.0), (1.0, 1e-36),
                        (1e-30, 1e-20), (1.0, -1e-37), (1e-36, 1e37)):
        q = (torch.randn(len(t), Hkv * G, D, generator=gen) * size).to(torch.bfloat16)
        q[0, 0] = 0.0
        got = _decode(q, pool, table, t, s, c, rows, scale)
        _close(got, ko.decode(ku.f64(q), pool, table, t, s, c, scale=scale), (size, scale))


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("G", [2, 8])
@pytest.mark.parametrize("D", [64, 128])
def test_decode_of_large_queries_over_small_keys(D, G, rows):
    # The same scores as of the unscaled query and keys, but a score's sums leave
    # fp32's normal range: five roundings of 2^-150 each.  In the units of the largest
    # query element, below 4 * 2^power / sqrt(D) * log2(e) = 2^(power + .03 or .53), which
    # is kept below 2^11 with codes in units of 2^-24, that is 5 * 2^-150 *
    # 2^(power + 1 - 11 + 24) of a score, twice that of a weight.
    rng, gen = np.random.default_rng(45), torch.Generator().manual_seed(45)
    Hkv, R, s, c, t = 2, 64, 40, 60, [100, 68, 30]
    q = _signed_rows(gen, len(t), Hkv * G, D)
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    O, LSE, bO, bL = ko.decode(ku.f64(q), pool, table, t, s, c)
    for power in (100, 112, 115, 118):
        got = _decode(q * 2.0 ** power, _scaled(pool, D, "k", -power), table, t, s, c, rows)
        more = 5 * 2.0 ** (power + 14 - 150)
        # a value is at most 15 * 0.6 + 7.5 * 0.6 here
        _close(got, (O, LSE, bO + 2 * more * 13.5, bL + more), power)


@pytest.mark.parametrize("rows", ROWS)
@pytest.mark.parametrize("D,G", [(64, 2), (128, 8)])
def test_decode_of_the_largest_queries_over_keys_of_zero(D, G, rows):
    # every score is 0: LSE is ln of the number of keys, the output their mean value
    rng, gen = np.random.default_rng(46), torch.Generator().manual_seed(46)
    Hkv, R, s, c, t = 2, 64, 40, 60, [100, 68, 30]
    q = (torch.randn(len(t), Hkv * G, D, generator=gen) * 1e38).clamp(-3.3e38, 3.3e38)
    q = q.to(torch.bfloat16)
    table, num = ku.random_tables(rng, [x + 1 for x in t], R)
    pool = ku.random_pool(rng, num, Hkv, R, D)
    pool[..., :32 * D + 256 * (D // 64)] = 0  # codes and parameters of the keys
    got = _decode(q, pool, table, t, s, c, rows)
    _close(got, ko.decode(ku.f64(q), pool, table, t, s, c))


@pytest.mark.parametrize("rows", ROWS)
def test_decode_of_very_many_query_heads(rows):
    # more groups of eight heads on a kv head than a launch's second dimension counts
    rng, gen = np.random.default_rng(47), torch.Generator().manual_seed(47)
    D, R, s, c, Hq, part = 64, 64, 40, 60, 70001 * 8, 2000 * 8
    table, num = ku.random_tables(rng, [41], R)
    pool = ku.random_pool(rng, num, 1, R, D)
    q = torch.randn(1, Hq, D, generator=gen).to(torch.bfloat16)
    O, LSE = _decode(q, pool, table, [40], s, c, rows)
    for h in (0, 30000 * 8, 65535 * 8 - 1000, Hq - part):  # every unit of a call is worked alike
        a, b = _decode(q[:, h:h + part].contiguous(), pool, table, [40], s, c, rows)
        assert torch.equal(O[:, h:h + part], a) and torch.equal(LSE[:, h:h + part], b), h
    for h in (0, Hq - 24):
        few = slice(h, h + 24)
        _close((O[:, few], LSE[:, few]),
               ko.decode(ku.f64(q[:, few]), pool, table, [40], s, c), h)

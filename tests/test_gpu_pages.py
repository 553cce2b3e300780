"""The page operations on the GPU against the step-by-step restatement: tables,
counts and page contents have to be equal, byte for byte."""

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
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


def _pools(num, R, seed, kinds=("bf16", "kv4")):
    """Pools with pages of R rows and known contents, on the GPU."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for kind in kinds:
        if kind == "bf16":
            x = torch.randn(num, R, 2, 64, generator=gen, device="cuda").to(torch.bfloat16)
        else:
            x = torch.randint(0, 256, (num, 3, R // 64, 4608), generator=gen, device="cuda",
                              dtype=torch.uint8)
        out.append(x)
    return out


def _moved(pools, copies):
    """The pools after the copies, each in its units (rows, or tiles of 64 rows)."""
    out = []
    for p in pools:
        x = p.clone()
        for a, z, rows in copies:
            if p.dtype == torch.uint8:
                x[z, :, :-(-rows // 64)] = p[a, :, :-(-rows // 64)]
            else:
                x[z, :rows] = p[a, :rows]
        out.append(x)
    return out


def _remap(src, lens, new, table, refs, pools, R, alias=False, **kw):
    dev = [ku.ints(x) for x in (src, lens, new)]
    t, r = ku.ints(table), ku.ints(refs)
    if alias:
        kw.update(block_table_out=t, refs_out=r)
    t2, r2, info = dca.dca_pages_remap(*dev, t, r, pools, R, **kw)
    return t2.tolist(), r2.tolist(), info.tolist()


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("k", range(14))
def test_remap_matches_the_oracle(k, alias):
    rng = np.random.default_rng(300 + k)
    R, most = int(rng.choice([64, 128, 192])), int(rng.integers(1, 9))
    B = int(rng.choice([1, 2, 7, 33]))
    lens, table, refs, num = ku.random_slots(rng, B, most, R, extra=int(rng.integers(0, 3 * B + 2)),
                                             pins=k % 4)
    src = [int(x) for x in rng.integers(-1, B, B)]
    if k % 3 == 0:  # a beam search: few parents, one row more each
        src = [int(rng.integers(0, 1 + B // 3)) for _ in range(B)]
    new = [int(rng.integers(0, most * R + 1)) for _ in range(B)]
    if k % 2:
        new = [min(most * R, lens[f] + 1) if f >= 0 else 0 for f in src]
    pools = _pools(num, R, k)
    want = ko.remap(src, lens, new, table, refs, R)
    expect = _moved(pools, want[3])
    got = _remap(src, lens, new, table, refs, pools, R, alias)
    dca.dca_sync_status()
    assert got == tuple(want[:3])
    for a, b in zip(pools, expect):
        assert torch.equal(a, b)


def test_remap_small_pages_and_pools_of_rows():
    # pages of one and of five rows hold bf16 rows only
    for R in (1, 5):
        rng = np.random.default_rng(400 + R)
        lens, table, refs, num = ku.random_slots(rng, 9, 7, R, extra=60)
        src = [int(x) for x in rng.integers(-1, 9, 9)]
        new = [int(rng.integers(0, 7 * R + 1)) for _ in range(9)]
        pools = _pools(num, R, 3, ("bf16", "bf16"))
        want = ko.remap(src, lens, new, table, refs, R)
        expect = _moved(pools, want[3])
        assert _remap(src, lens, new, table, refs, pools, R) == tuple(want[:3])
        dca.dca_sync_status()
        assert all(torch.equal(a, b) for a, b in zip(pools, expect))


def test_remap_many_slots_and_pages():
    rng = np.random.default_rng(500)
    R, B, most = 64, 2500, 12
    lens, table, refs, num = ku.random_slots(rng, B, most, R, extra=9000, pins=50)
    src = [int(x) for x in rng.integers(-1, B, B)]
    new = [int(rng.integers(0, most * R + 1)) for _ in range(B)]
    want = ko.remap(src, lens, new, table, refs, R)
    assert want[2][1] > 500
    got = _remap(src, lens, new, table, refs, [], R)
    dca.dca_sync_status()
    assert got == tuple(want[:3])


@pytest.mark.parametrize("B,most", [(2, 9500), (1, 1), (5000, 1), (3, 1024), (9, 1023), (5, 4097),
                                    (1, 30000), (40, 1025)])
def test_long_rows_and_many_short_ones(B, most):
    # rows as long as, longer and shorter than the threads that share the entries
    rng = np.random.default_rng(B)
    lens, table, refs, num = ku.random_slots(rng, B, most, 1, extra=most + 3 * B, pins=5)
    src = [int(x) for x in rng.integers(-1, B, B)]
    new = [int(rng.integers(0, most + 1)) for _ in range(B)]
    want = ko.remap(src, lens, new, table, refs, 1)
    assert _remap(src, lens, new, table, refs, [], 1) == tuple(want[:3])
    want = ko.compact(lens, table, refs, 1)
    got = dca.dca_pages_compact(ku.ints(lens), ku.ints(table), ku.ints(refs), [], 1)
    assert tuple(x.tolist() for x in got) == tuple(want[:4])
    dca.dca_sync_status()


def test_remap_with_missing_pages_changes_nothing():
    lens, table = [70, 64], [[2, 0, -1], [1, -1, -1]]
    pools = _pools(4, 64, 5)
    before = [p.clone() for p in pools]
    # the fork needs a copy and two pages more than are left
    for alias in (False, True):
        got = _remap([0, 0], lens, [192, 192], table, [2, 1, 2, 1], pools, 64, alias)
        assert got[0] == table and got[1] == [2, 1, 2, 1] and got[2][0] < 0
        assert got[2] == ko.remap([0, 0], lens, [192, 192], table, [2, 1, 2, 1], 64)[2]
    dca.dca_sync_status()
    assert all(torch.equal(a, b) for a, b in zip(pools, before))


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("change", ["src", "src_low", "new", "new_low", "old", "entry", "entry_low",
                                    "count", "negative"])
def test_remap_refuses_bad_states(change, alias):
    src, lens, new = [0, 0], [70, 64], [71, 66]
    table, refs = [[2, 0, -1], [1, -1, -1]], [1, 1, 1, 0, 0, 0]
    if change == "src":
        src[1] = 2
    elif change == "src_low":
        src[1] = -2
    elif change == "new":
        new[0] = 193
    elif change == "new_low":
        new[0] = -1
    elif change == "old":
        lens[1] = 193
    elif change == "entry":
        table[0][1] = 6
    elif change == "entry_low":
        table[0][1] = -1
    elif change == "count":
        refs[1] = 0
    elif change == "negative":
        refs[5] = -1
    pools = _pools(6, 64, 6)
    before = [p.clone() for p in pools]
    got = _remap(src, lens, new, table, refs, pools, 64, alias)
    with pytest.raises(dca.DcaError) as ei:
        dca.dca_sync_status()
    assert ei.value.status == 1
    assert got == (table, refs, [2 ** 31 - 1, 0])
    assert all(torch.equal(a, b) for a, b in zip(pools, before))
    dca.dca_sync_status()


def test_remap_of_a_tail_that_came_shared():
    # two slots came with the same partial page: the lower keeps it
    got = _remap([0, 1], [70, 70], [70, 70], [[2, 0], [2, 0]], [2, 0, 2, 0, 0], [], 64)
    assert got == ([[2, 0], [2, 1]], [1, 1, 2, 0, 0], [2, 1])
    # cut inside a full page that another slot goes on sharing: a copy
    got = _remap([0, 1], [128, 128], [128, 100], [[2, 0], [2, 0]], [2, 0, 2, 0, 0], [], 64)
    assert got == ([[2, 0], [2, 1]], [1, 1, 2, 0, 0], [2, 1])
    dca.dca_sync_status()


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("k", range(10))
def test_compact_matches_the_oracle(k, alias):
    rng = np.random.default_rng(600 + k)
    R = int(rng.choice([64, 128]))
    B, most = int(rng.choice([0, 1, 6, 40])), int(rng.integers(1, 7))
    lens, table, refs, num = ku.random_slots(rng, B, most, R, pins=k % 5,
                                             extra=int(rng.choice([0, 1, 20, 200])))
    if num == 0:
        refs, num = [0], 1
    pools = _pools(num, R, k)
    want = ko.compact(lens, table, refs, R)
    expect = _moved(pools, want[4])
    t = ku.ints(table).view(B, most)
    r = ku.ints(refs)
    kw = dict(block_table_out=t, refs_out=r) if alias else {}
    got = dca.dca_pages_compact(ku.ints(lens), t, r, pools, R, **kw)
    dca.dca_sync_status()
    assert tuple(x.tolist() for x in got) == tuple(want[:4])
    for a, b in zip(pools, expect):
        assert torch.equal(a, b)


def test_compact_many_pages():
    rng = np.random.default_rng(700)
    lens, table, refs, num = ku.random_slots(rng, 3000, 10, 64, extra=30000, pins=77)
    want = ko.compact(lens, table, refs, 64)
    got = dca.dca_pages_compact(ku.ints(lens), ku.ints(table), ku.ints(refs), [], 64)
    dca.dca_sync_status()
    assert tuple(x.tolist() for x in got) == tuple(want[:4])


@pytest.mark.parametrize("alias", [False, True])
@pytest.mark.parametrize("change", ["len", "len_low", "entry", "entry_low", "free", "negative"])
def test_compact_refuses_bad_states(change, alias):
    lens, table, refs = [70, 64], [[5, 0, -1], [1, -1, -1]], [1, 1, 0, 0, 0, 1]
    if change == "len":
        lens[0] = 193
    elif change == "len_low":
        lens[1] = -1
    elif change == "entry":
        table[1][0] = 6
    elif change == "entry_low":
        table[1][0] = -7
    elif change == "free":
        refs[5] = 0
    elif change == "negative":
        refs[2] = -1
    pools = _pools(6, 64, 8)
    before = [p.clone() for p in pools]
    t, r = ku.ints(table), ku.ints(refs)
    kw = dict(block_table_out=t, refs_out=r) if alias else {}
    got = dca.dca_pages_compact(ku.ints(lens), t, r, pools, 64, **kw)
    with pytest.raises(dca.DcaError) as ei:
        dca.dca_sync_status()
    assert ei.value.status == 1
    assert tuple(x.tolist() for x in got) == (table, refs, list(range(6)), [2 ** 31 - 1, 0])
    assert all(torch.equal(a, b) for a, b in zip(pools, before))
    dca.dca_sync_status()


def test_stacked_pools_and_refused_pools():
    R, num = 64, 9
    stacked = torch.stack(_pools(num, R, 9, ("kv4", "kv4", "kv4")))
    apart = [x.clone() for x in stacked]
    state = ([1, 1], [10, 70], [11, 75], [[3, -1], [8, 5]], [0, 0, 0, 1, 0, 1, 0, 0, 1])
    a = _remap(*state, stacked, R)
    b = _remap(*state, apart, R)
    dca.dca_sync_status()
    assert a == b and a[2][1] == 1
    assert all(torch.equal(x, y) for x, y in zip(stacked, apart))
    for pools in ([apart[0][:5]], [apart[0].float()], [apart[0].cpu()], [apart[0].transpose(1, 3)],
                  [torch.zeros(num, 65, 2, 64, dtype=torch.bfloat16, device="cuda")], [3],
                  torch.zeros(num, 4, dtype=torch.uint8, device="cuda")):
        with pytest.raises(dca.DcaError):
            _remap(*state, pools, R)


def test_page_operations_in_a_graph_on_a_stream():
    rng = np.random.default_rng(800)
    R, B = 64, 6
    lens, table, refs, num = ku.random_slots(rng, B, 5, R, extra=40)
    pools = _pools(num, R, 10)
    t, r, n = ku.ints(table), ku.ints(refs), ku.ints(lens)
    src, new = ku.ints([0] * B), ku.ints([0] * B)
    info, moved = ku.ints([0, 0]), ku.ints([0] * num)
    ws = torch.empty(dca.dca_pages_workspace(B, 5, num), dtype=torch.uint8, device="cuda")

    def step():
        dca.dca_pages_remap(src, n, new, t, r, pools, R, workspace=ws, block_table_out=t,
                            refs_out=r, info=info)
        n.copy_(new)
        dca.dca_pages_compact(n, t, r, pools, R, workspace=ws, block_table_out=t, refs_out=r,
                              moved=moved, info=info)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        keep = [x.clone() for x in (t, r, n, *pools)]
        step()
        for x, y in zip((t, r, n, *pools), keep):
            x.copy_(y)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            step()
        host = [p.clone() for p in pools]
        for _ in range(6):
            f = [int(x) for x in rng.integers(-1, B, B)]
            m = [int(rng.integers(0, 5 * R + 1)) for _ in range(B)]
            src.copy_(ku.ints(f))
            new.copy_(ku.ints(m))
            graph.replay()
            table, refs, got, copies = ko.remap(f, lens, m, table, refs, R)
            assert got[0] >= 0
            host, lens = _moved(host, copies), m
            table, refs, want, got, copies = ko.compact(lens, table, refs, R)
            host = _moved(host, copies)
            assert t.tolist() == table and r.tolist() == refs
            assert moved.tolist() == want and info.tolist() == got
            assert all(torch.equal(a, b) for a, b in zip(pools, host))
    torch.cuda.current_stream().wait_stream(side)
    dca.dca_sync_status()


def test_beam_search_over_4bit_pages():
    """The operators together: prompts in, beams forked, reordered and freed,
    tokens appended, pages compacted, attention after every step; against
    caches that are simply copied."""
    rng = np.random.default_rng(900)
    gen = torch.Generator().manual_seed(900)
    D, Hq, Hkv, R, s, c, B, most = 64, 4, 2, 64, 40, 60, 5, 4
    num = 24
    pool = torch.zeros((num, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    lens = [0] * B
    flat_table = torch.arange(B * most, dtype=torch.int32, device="cuda").view(B, most)
    flat = torch.zeros((B * most, Hkv, 1, ko.tile_bytes(D)), dtype=torch.uint8, device="cuda")

    def move(src, new):
        nonlocal table, refs, flat, lens
        table, refs, info = dca.dca_pages_remap(ku.ints(src), ku.ints(lens), ku.ints(new), table,
                                                refs, [pool], R)
        assert info.tolist()[0] >= 0
        f = flat.view(B, most, *flat.shape[1:])
        flat = torch.stack([f[max(x, 0)] for x in src]).reshape(flat.shape).contiguous()
        lens = list(new)

    def put(t0, n):
        nonlocal pool, flat
        cu = np.concatenate(([0], np.cumsum(n)))
        k, v = (ku.bf16_rows(gen, int(cu[-1]), Hkv, D).cuda() for _ in range(2))
        for p, tab in ((pool, table), (flat, flat_table)):
            dca.dca_kv4_append_paged(k, v, p, tab, ku.ints(cu), ku.ints(t0), s, c)

    def check():
        q = ku.bf16_rows(gen, B, Hq, D).cuda()
        live = [b for b in range(B) if lens[b]]
        pick = torch.tensor(live, device="cuda")
        t = ku.ints([lens[b] - 1 for b in live])
        a = dca.dca_attn_decode_kv4_paged(q[pick], pool, table[pick], t, s, c)
        b = dca.dca_attn_decode_kv4_paged(q[pick], flat, flat_table[pick], t, s, c)
        dca.dca_sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    move([-1] * B, [90, 0, 0, 30, 0])            # two prompts
    put([0] * B, [90, 0, 0, 30, 0])
    check()
    move([0, 0, 0, 3, 3], [91, 91, 91, 31, 31])  # beams, room for a token each
    put([90, 90, 90, 30, 30], [1] * B)
    check()
    for step in range(60):
        src = [int(rng.integers(0, 3)) for _ in range(3)] + [3 + int(rng.integers(0, 2))
                                                             for _ in range(2)]
        new = [lens[f] + 1 for f in src]
        old = [lens[f] for f in src]
        move(src, new)
        put(old, [1] * B)
        if step % 9 == 4:
            table, refs, moved, info = dca.dca_pages_compact(ku.ints(lens), table, refs, [pool], R)
            assert refs.tolist()[info.tolist()[0]:] == [0] * (num - info.tolist()[0])
        check()
    move([0, -1, 2, -1, -1], [lens[0], 0, 65, 0, 0])   # one beam ends, one is cut
    check()
    assert int((refs > 0).sum()) <= -(-lens[0] // R) + 2

"""The bf16 paged calls on tables that the page operations make: packed chunks,
appends and decode over pages that slots share, take over and copy, against the
contiguous calls over caches that are simply copied."""

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
from tests import kv4_util as ku

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_attention_dca_b200 import build
    build.build()
    dca.lib()
    yield
    dca.dca_sync_status()


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 6, 1)])
def test_beams_over_bf16_pages(D, Hq, Hkv):
    rng, gen = np.random.default_rng(61), torch.Generator().manual_seed(61)
    R, most, num, B, s, c = 128, 4, 20, 4, 100, 150
    Tcap = most * R
    bf16 = lambda *shape: ku.bf16_rows(gen, *shape).cuda()  # noqa: E731
    # NaN wherever nothing was written: a row that is read by mistake shows
    Kp, Vp = (torch.full((num, R, Hkv, D), float("nan"), dtype=torch.bfloat16, device="cuda")
              for _ in range(2))
    Kc, Vc = (torch.zeros(B, Tcap, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    table = torch.full((B, most), -1, dtype=torch.int32, device="cuda")
    refs = torch.zeros(num, dtype=torch.int32, device="cuda")
    lens = [0] * B

    def move(src, new):
        nonlocal table, refs, Kc, Vc, lens
        table, refs, info = dca.dca_pages_remap(ku.ints(src), ku.ints(lens), ku.ints(new), table,
                                                refs, [Kp, Vp], R)
        assert info.tolist()[0] >= 0
        pick = torch.tensor([max(f, 0) for f in src], device="cuda")
        Kc, Vc, lens = Kc[pick].contiguous(), Vc[pick].contiguous(), list(new)

    def chunk(t0, n):
        cu = ku.ints(np.concatenate(([0], np.cumsum(n))))
        T = sum(n)
        x = (bf16(T, Hq, D), bf16(T, Hkv, D), bf16(T, Hkv, D))
        rest = (cu, ku.ints(t0), max(n), Tcap, s, c)
        a = dca.dca_attn_prefill_varlen_chunk_paged(*x, Kp, Vp, table, *rest)
        b = dca.dca_attn_prefill_varlen_chunk(*x, Kc, Vc, *rest)
        dca.dca_sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    def token(live):
        """A token for every live slot, whose page it already has, and its attention."""
        pick = torch.tensor(live, device="cuda")
        k, v, q = bf16(len(live), Hkv, D), bf16(len(live), Hkv, D), bf16(len(live), Hq, D)
        t = ku.ints([lens[b] - 1 for b in live])
        rows = table[pick].contiguous()
        dca.dca_kv_append_paged(k, v, Kp, Vp, rows, t, s, c)
        Ks, Vs = Kc[pick].contiguous(), Vc[pick].contiguous()
        dca.dca_kv_append(k, v, Ks, Vs, t, s, c)
        Kc[pick], Vc[pick] = Ks, Vs
        a = dca.dca_attn_decode_paged(q, Kp, Vp, rows, t, s, c)
        b = dca.dca_attn_decode(q, Ks, Vs, t, s, c)
        dca.dca_sync_status()
        assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])

    move([-1] * B, [200, 0, 130, 0])
    chunk([0] * B, [200, 0, 130, 0])           # two prompts
    move([0, 0, 2, 2], [230, 240, 140, 131])   # forked, then chunks of their own
    chunk([200, 200, 130, 130], [30, 40, 10, 1])
    for step in range(40):                     # over a page's end
        src = [int(rng.integers(0, 2)), int(rng.integers(0, 2)), 2, 3]
        move(src, [lens[f] + 1 for f in src])
        if step % 13 == 5:
            table, refs, _, _ = dca.dca_pages_compact(ku.ints(lens), table, refs, [Kp, Vp], R)
        token([0, 1, 2, 3])
    move([-1, 1, 2, -1], [0, lens[1] + 1, 90, 0])  # one freed, one cut inside a page it shared
    chunk([0, lens[1] - 1, 77, 0], [0, 1, 13, 0])
    move([0, 1, 2, -1], [0, lens[1] + 1, 91, 0])
    token([1, 2])

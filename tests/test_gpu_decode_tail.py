"""Decode over bf16 caches whose rows past the sequence hold anything: a new
page or a new cache is not cleared, and its old bits can be NaN."""

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


@pytest.mark.parametrize("D,Hq,Hkv", [(64, 4, 2), (128, 9, 1), (128, 3, 3)])
@pytest.mark.parametrize("rest", [float("nan"), float("inf"), -3e38])
def test_rows_past_the_sequence_do_not_show(D, Hq, Hkv, rest):
    gen = torch.Generator().manual_seed(71)
    t = [0, 1, 15, 16, 40, 63, 64, 1000, 1023, 1024, 1500]
    B, Tcap, R, s, c = len(t), 1536, 64, 300, 400
    K, V = (ku.bf16_rows(gen, B, Tcap, Hkv, D).cuda() for _ in range(2))
    q = ku.bf16_rows(gen, B, Hq, D).cuda()
    past = (torch.arange(Tcap, device="cuda")[None] > torch.tensor(t, device="cuda")[:, None])
    Kz, Vz = (x.masked_fill(past[..., None, None], 0.0) for x in (K, V))
    Kr, Vr = (x.masked_fill(past[..., None, None], rest) for x in (K, V))
    t = ku.ints(t)
    want = dca.dca_attn_decode(q, Kz, Vz, t, s, c)
    assert not torch.isnan(want[0]).any()
    table = torch.randperm(B * (Tcap // R), generator=gen).to(torch.int32).cuda()
    pages = [torch.empty(B * (Tcap // R), R, Hkv, D, dtype=torch.bfloat16, device="cuda")
             for _ in range(2)]
    for pool, x in zip(pages, (Kr, Vr)):
        pool[table.long()] = x.view(-1, R, Hkv, D)
    for O, LSE in (dca.dca_attn_decode(q, Kr, Vr, t, s, c),
                   dca.dca_attn_decode_noalloc(q, Kr, Vr, t, s, c),
                   dca.dca_attn_decode_paged(q, *pages, table.view(B, -1), t, s, c)):
        assert torch.equal(O, want[0]) and torch.equal(LSE, want[1])
    dca.dca_sync_status()

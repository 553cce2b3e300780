"""The page operations at the sizes where their launches change."""

import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import long_context_attention_dca_b200 as dca
from oracle import kv4_oracle as ko
from tests import kv4_util as ku
from tests.test_gpu_pages import _moved, _remap

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module", autouse=True)
def _built():
    from long_context_attention_dca_b200 import build
    build.build()
    dca.lib()
    yield
    dca.dca_sync_status()


_GROWING = """
import numpy as np
import long_context_attention_dca_b200 as dca
from oracle import kv4_oracle as ko
from tests import kv4_util as ku

num = 3000
for most in range({first}, {last}):  # a page list of one entry more each time
    rng = np.random.default_rng(most)
    order = rng.permutation(num).tolist()
    lens, table = [1000], [order[:1000] + [-1] * (most - 1000)]
    refs = [0] * num
    for p in order[:1000]:
        refs[p] = 1
    src, new = [0], [1500]
    want = ko.remap(src, lens, new, table, refs, 1)
    got = dca.dca_pages_remap(*(ku.ints(x) for x in (src, lens, new, table, refs)), [], 1)
    assert tuple(x.tolist() for x in got) == tuple(want[:3]), most
    want = ko.compact(lens, table, refs, 1)
    got = dca.dca_pages_compact(*(ku.ints(x) for x in (lens, table, refs)), [], 1)
    assert tuple(x.tolist() for x in got) == tuple(want[:4]), most
dca.dca_sync_status()
"""


def test_plans_that_just_pass_the_default_shared_memory():
    # A plan takes 64 + 3 pages + table entries + 6 slots ints of shared memory, here
    # 9070 and the table's width: from below the 48 KB that a kernel has without asking
    # (its own 256 bytes included) to above 48 KB.  A process of its own, since
    # a kernel that has once asked for more keeps it.
    code = _GROWING.format(first=12224 - 9070 - 2, last=12289 - 9070 + 2)
    res = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True,
                         timeout=600)
    assert res.returncode == 0, res.stderr[-2000:]


def _pools(num, R, n, seed):
    """n pools of three kinds, whose pages are 8 KB, 128 KB and 2 x 4.5 KB."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    out = []
    for j in range(n):
        if j % 3 == 2:
            out.append(torch.randint(0, 256, (num, 2, R // 64, 4608), generator=gen, device="cuda",
                                     dtype=torch.uint8))
        else:
            shape = (num, R, 1, 64) if j % 3 == 0 else (num, R, 8, 128)
            out.append(torch.randn(shape, generator=gen, device="cuda").to(torch.bfloat16))
    return out


@pytest.mark.parametrize("n", [1, 15, 16, 17, 64, 255, 256])
def test_pools_of_many_layers(n):
    rng = np.random.default_rng(n)
    R, B = 64, 5
    lens, table, refs, num = ku.random_slots(rng, B, 4, R, extra=12)
    src = [0, 0, 2, 2, -1]
    new = [min(4 * R, lens[f] + 1) if f >= 0 else 70 for f in src]
    pools = _pools(num, R, n, n)
    want = ko.remap(src, lens, new, table, refs, R)
    assert want[2][1] > 0
    expect = _moved(pools, want[3])
    got = _remap(src, lens, new, table, refs, pools, R)
    dca.dca_sync_status()
    assert got == tuple(want[:3])
    assert all(torch.equal(a, b) for a, b in zip(pools, expect))
    table, refs = want[:2]
    want = ko.compact(new, table, refs, R)
    assert want[3][1] > 0
    expect = _moved(pools, want[4])
    got = dca.dca_pages_compact(ku.ints(new), ku.ints(table), ku.ints(refs), pools, R)
    dca.dca_sync_status()
    assert tuple(x.tolist() for x in got) == tuple(want[:4])
    assert all(torch.equal(a, b) for a, b in zip(pools, expect))


def test_more_pools_than_a_call_takes_are_refused():
    stacked = torch.zeros(257, 3, 64, 1, 64, dtype=torch.bfloat16, device="cuda")
    state = ([0], [10], [11], [[2]], [0, 0, 1])
    with pytest.raises(dca.DcaError, match="256"):
        _remap(*state, stacked, 64)
    with pytest.raises(dca.DcaError, match="256"):
        dca.dca_pages_compact(ku.ints([10]), ku.ints([[2]]), ku.ints([0, 0, 1]), stacked, 64)
    assert _remap(*state, stacked[1:], 64) == ([[2]], [0, 0, 1], [2, 0])
    dca.dca_sync_status()

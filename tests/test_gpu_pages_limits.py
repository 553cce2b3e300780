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

"""What the 4-bit decode takes and refuses by size alone, before it touches the
device."""

import ctypes

import pytest

import long_context_attention_dca_b200 as dca

FAKE = ctypes.c_void_p(0x10000)  # never dereferenced


@pytest.fixture(scope="module")
def lib():
    from long_context_attention_dca_b200 import build
    build.build()
    return dca.lib()


@pytest.mark.parametrize("want,B,Hq,Hkv,D,mb,br", [
    # taken, as far as the workspace, which is too small
    (5, 1, 8 * 65536, 1, 128, 4, 64), (5, 1, 8 * 70001, 1, 64, 4, 64),
    (5, 3, 4 * 65535, 65535, 64, 4, 64), (5, 65535, 8, 1, 128, 1 << 14, 64),
    # a sequence's query elements, all units, all shares
    (2, 1, (1 << 23) + 8, 1, 128, 4, 64), (2, 65535, 65535, 65535, 64, 4, 64),
    (2, 30000, 65535, 65535, 64, 1 << 24, 64),
])
def test_decode_sizes(lib, want, B, Hq, Hkv, D, mb, br):
    got = lib.dca_attn_decode_kv4_paged(FAKE, FAKE, FAKE, mb, br, 8, FAKE, FAKE, FAKE, B, Hq, Hkv,
                                        D, 8, 12, 1e4, 0.0, FAKE, 16, None)
    assert int(got) == want, dca.dca_last_error_string()
    need = dca.dca_attn_decode_kv4_workspace(B, Hq, Hkv, D, mb * br)
    assert (need > 16) == (want == 5)

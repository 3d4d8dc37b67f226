"""Attention in place is refused on the host: warps that share a row's query would read it after its output was
written (no GPU needed)."""
import ctypes

import paged_kv_cache_420_b200 as pkv
from paged_kv_cache_420_b200 import _Pool

EALIAS = 3
FAKE = ctypes.c_void_p(0x10000)  # aligned, never dereferenced


def test_dense_decode_refuses_its_query_as_output():
    f = pkv.load_library().paged_attn_decode_fp8_block
    assert f(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, 4, FAKE, 2, 4, 0.1, 2, FAKE, _Pool(8, 2, 16, 128, 1), 64, FAKE, 1 << 30,
             None) == EALIAS


def test_sparse_decode_refuses_its_query_as_output():
    f = pkv.load_library().paged_attn_decode_sparse
    for scales, dtype in ((FAKE, 1), (None, 0)):
        assert f(FAKE, FAKE, FAKE, scales, scales, FAKE, 4, FAKE, FAKE, 4, 2, 4, 0.1, 2, FAKE, _Pool(8, 2, 16, 128, dtype),
                 FAKE, 1 << 30, None) == EALIAS

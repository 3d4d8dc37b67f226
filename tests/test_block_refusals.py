"""Host checks of the block-scaled cache and of block-sparse decode: what they refuse, before any CUDA work (no GPU
needed)."""
import ctypes

import numpy as np
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from paged_kv_cache_420_b200 import _Pool

EINVAL, ERANGE, EALIAS, EUNSUP = 1, 2, 3, 6
FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced
ODD16 = ctypes.c_void_p(0x10008)     # not 16-byte aligned
ODD4 = ctypes.c_void_p(0x10002)      # not 4-byte aligned


def pool(nb=8, hkv=2, bs=16, d=128, dtype=1):
    return _Pool(nb, hkv, bs, d, dtype)


def write(**kw):
    a = dict(k=FAKE, v=FAKE, tables=FAKE, mbs=4, ctx=FAKE, start=FAKE, B=2, T=8, max_new=4, ks=FAKE, vs=FAKE, kc=FAKE,
             vc=FAKE, pool=pool())
    a.update(kw)
    return pkv.load_library().pkv_write_fp8_block(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, 0), ({"T": 0}, 0), ({"max_new": 0}, 0),
    ({"B": -1}, EINVAL), ({"T": -1}, EINVAL), ({"max_new": -1}, EINVAL), ({"mbs": 0}, EINVAL),
    ({"pool": pool(dtype=0)}, EINVAL), ({"pool": pool(dtype=2)}, EINVAL), ({"pool": pool(nb=0)}, EINVAL),
    ({"pool": pool(d=96)}, EUNSUP), ({"pool": pool(bs=24)}, EUNSUP), ({"pool": pool(bs=1040)}, EUNSUP),
    ({"pool": pool(nb=1 << 20, hkv=128)}, EUNSUP), ({"B": 1 << 30, "max_new": 64, "pool": pool(bs=64)}, EUNSUP),
    *[({n: None}, EINVAL) for n in ("k", "v", "tables", "ctx", "start", "ks", "vs", "kc", "vc")],
    *[({n: ODD16}, EINVAL) for n in ("k", "v", "kc", "vc")],
    *[({n: ODD4}, EINVAL) for n in ("tables", "ctx", "start", "ks", "vs")],
])
def test_write_refuses(change, status):
    assert write(**change) == status


def bounds(**kw):
    a = dict(kc=FAKE, ks=FAKE, tables=FAKE, mbs=4, ctx=FAKE, start=FAKE, B=2, max_new=4, bounds=FAKE, pool=pool())
    a.update(kw)
    return pkv.load_library().pkv_key_bounds(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, 0), ({"max_new": 0}, 0),
    ({"B": -1}, EINVAL), ({"max_new": -1}, EINVAL), ({"mbs": 0}, EINVAL),
    ({"ks": None}, EINVAL), ({"pool": pool(dtype=0)}, EINVAL),  # scales with an e4m3 pool, and only there
    ({"pool": pool(d=256)}, EUNSUP), ({"pool": pool(bs=8)}, EUNSUP),
    *[({n: None}, EINVAL) for n in ("kc", "tables", "ctx", "start", "bounds")],
    *[({n: ODD16}, EINVAL) for n in ("kc", "bounds")],
    *[({n: ODD4}, EINVAL) for n in ("ks", "tables", "ctx", "start")],
])
def test_key_bounds_refuses(change, status):
    assert bounds(**change) == status


def decode8(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, tables=FAKE, mbs=4, ctx=FAKE, B=2, Hq=4, scale=0.1, Hkv=2,
             out=FAKE, pool=pool(), max_ctx=64, ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return pkv.load_library().paged_attn_decode_fp8_block(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, 0), ({"B": -1}, EINVAL), ({"Hq": 5}, EINVAL), ({"Hq": 34}, EUNSUP), ({"Hkv": 4, "Hq": 8}, EINVAL),
    ({"pool": pool(dtype=0)}, EINVAL), ({"pool": pool(d=256)}, EUNSUP), ({"max_ctx": -1}, EINVAL), ({"mbs": 0}, EINVAL),
    ({"ws_bytes": 16}, EINVAL), ({"ws": ODD16}, EINVAL),
    *[({n: None}, EINVAL) for n in ("q", "kc", "vc", "ks", "vs", "tables", "ctx", "out", "ws")],
    *[({n: ODD16}, EINVAL) for n in ("q", "kc", "vc", "out")],
    *[({n: ODD4}, EINVAL) for n in ("ks", "vs", "tables", "ctx")],
])
def test_decode_refuses(change, status):
    assert decode8(**change) == status


def test_copy_scales_refuses():
    lib = pkv.load_library()

    def copy(p, n=None, ks=FAKE, vs=FAKE, nb=8, h=2):
        a = np.ascontiguousarray(np.asarray(p, np.int32).reshape(-1, 2))
        return lib.pkv_copy_scales(a.ctypes.data_as(ctypes.c_void_p), len(a) if n is None else n, ks, vs, nb, h, None)

    assert copy([[0, 1]], n=0) == 0
    for p, status in [([[0, 8]], ERANGE), ([[-1, 2]], ERANGE), ([[0, 1], [2, 1]], EALIAS), ([[0, 1], [1, 2]], EALIAS),
                      ([[3, 3]], EALIAS)]:
        assert copy(p) == status
    assert copy([[0, 1]], n=-1) == EINVAL
    assert copy([[0, 1]], ks=None) == EINVAL and copy([[0, 1]], vs=ODD4) == EINVAL
    assert copy([[0, 1]], nb=0) == EINVAL and copy([[0, 1]], h=0) == EINVAL and copy([[0, 1]], h=1 << 21) == EUNSUP
    dev = lib.pkv_copy_scales_dev
    assert dev(FAKE, FAKE, 0, FAKE, FAKE, 8, 2, None) == 0
    assert dev(FAKE, FAKE, -1, FAKE, FAKE, 8, 2, None) == EINVAL
    assert dev(None, FAKE, 4, FAKE, FAKE, 8, 2, None) == EINVAL
    assert dev(FAKE, ODD4, 4, FAKE, FAKE, 8, 2, None) == EINVAL
    assert dev(FAKE, FAKE, 4, FAKE, FAKE, 0, 2, None) == EINVAL


def test_binding_refuses_wrong_tensors():
    """Types, layouts and shapes that the binding refuses before the library sees them (CPU tensors)."""
    i32, bf16, u8 = torch.int32, torch.bfloat16, torch.uint8
    k = torch.zeros((3, 2, 64), dtype=bf16)
    with pytest.raises(TypeError):  # fp32 rows
        pkv.pkv_write_fp8_block(k.float(), k, *[torch.zeros(1, dtype=i32)] * 3, *[torch.zeros((4, 2))] * 2,
                                *[torch.zeros((4, 2, 16, 64), dtype=u8)] * 2, 1)
    with pytest.raises(ValueError):  # host memory
        pkv.pkv_write_fp8_block(k, k, *[torch.zeros(1, dtype=i32)] * 3, *[torch.zeros((4, 2))] * 2,
                                *[torch.zeros((4, 2, 16, 64), dtype=u8)] * 2, 1)
    with pytest.raises(ValueError):  # a transposed view
        pkv.pkv_write_fp8_block(k.transpose(0, 1), k, *[torch.zeros(1, dtype=i32)] * 3, *[torch.zeros((4, 2))] * 2,
                                *[torch.zeros((4, 2, 16, 64), dtype=u8)] * 2, 1)


def select(**kw):
    a = dict(q=FAKE, bounds=FAKE, tables=FAKE, mbs=4, ctx=FAKE, B=2, Hq=4, Hkv=2, pool=pool(), sel=FAKE, K=4, max_ctx=64,
             ws=FAKE, ws_bytes=1 << 20)
    a.update(kw)
    return pkv.load_library().pkv_select_blocks(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, 0), ({"B": -1}, EINVAL), ({"Hq": 5}, EINVAL), ({"Hq": 34}, EUNSUP), ({"Hkv": 4, "Hq": 8}, EINVAL),
    ({"K": 1}, EINVAL), ({"K": 0}, EINVAL), ({"max_ctx": -1}, EINVAL), ({"mbs": 0}, EINVAL),
    ({"pool": pool(d=96)}, EUNSUP), ({"pool": pool(bs=20)}, EUNSUP), ({"pool": pool(dtype=7)}, EINVAL),
    ({"ws_bytes": 16}, EINVAL), ({"ws": ODD16}, EINVAL),
    *[({n: None}, EINVAL) for n in ("q", "bounds", "tables", "ctx", "sel", "ws")],
    *[({n: ODD16}, EINVAL) for n in ("q", "bounds")],
    *[({n: ODD4}, EINVAL) for n in ("tables", "ctx", "sel")],
])
def test_select_refuses(change, status):
    assert select(**change) == status


def sparse(**kw):
    a = dict(q=FAKE, kc=FAKE, vc=FAKE, ks=FAKE, vs=FAKE, tables=FAKE, mbs=4, ctx=FAKE, sel=FAKE, K=4, B=2, Hq=4,
             scale=0.1, Hkv=2, out=FAKE, pool=pool(), ws=FAKE, ws_bytes=1 << 30)
    a.update(kw)
    return pkv.load_library().paged_attn_decode_sparse(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    ({"B": 0}, 0), ({"B": -1}, EINVAL), ({"Hq": 5}, EINVAL), ({"Hq": 34}, EUNSUP), ({"Hkv": 4, "Hq": 8}, EINVAL),
    ({"K": 0}, EINVAL), ({"K": 1 << 27}, EUNSUP), ({"mbs": 0}, EINVAL), ({"pool": pool(d=256)}, EUNSUP),
    ({"ks": None}, EINVAL), ({"vs": None}, EINVAL), ({"pool": pool(dtype=0)}, EINVAL),  # scales go with an e4m3 pool
    ({"ks": None, "pool": pool(dtype=0)}, EINVAL), ({"pool": pool(dtype=3)}, EINVAL),
    *[({n: None}, EINVAL) for n in ("q", "kc", "vc", "tables", "ctx", "sel", "out", "ws")],
    ({"ws_bytes": 16}, EINVAL), ({"ws": ODD16}, EINVAL),
    *[({n: ODD16}, EINVAL) for n in ("q", "kc", "vc", "out")],
    *[({n: ODD4}, EINVAL) for n in ("ks", "vs", "tables", "ctx", "sel")],
])
def test_sparse_decode_refuses(change, status):
    assert sparse(**change) == status

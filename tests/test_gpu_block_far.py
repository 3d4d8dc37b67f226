"""Appends whose last positions lie just under 2^31."""
import numpy as np
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def test_append_and_bounds_at_the_last_positions():
    """A table longer than 2^31 positions, and a bound of the new tokens that reaches behind the context: only the blocks
    that receive tokens change."""
    H, D, bs, NB, n = 2, 64, 16, 8, 21
    blocks = 2 ** 31 // bs
    tables = torch.full((1, blocks + 70000), 7, dtype=torch.int32, device="cuda")  # block 7: not to be touched
    ctx = 2 ** 31 - 5
    tables[0, blocks - 1], tables[0, blocks - 2] = 3, 5
    r = np.random.default_rng(1)
    codes = [r.integers(0, 0x7F, (NB, H, bs, D)).astype(np.uint8) for _ in "kv"]
    gen = torch.Generator().manual_seed(1)
    x = [torch.randn((n, H, D), generator=gen).to(torch.bfloat16) for _ in "kv"]
    kc, vc = (torch.from_numpy(c.copy()).cuda() for c in codes)
    ks, vs = (torch.full((NB, H), 2.0 ** -6, device="cuda") for _ in "kv")
    bounds = torch.zeros((NB, H, 2, D), dtype=torch.bfloat16, device="cuda")
    cx = torch.tensor([ctx], dtype=torch.int32, device="cuda")
    start = torch.tensor([0, n], dtype=torch.int32, device="cuda")
    pkv.pkv_write_fp8_block(x[0].cuda(), x[1].cuda(), tables, cx, start, ks, vs, kc, vc, 2 ** 20)
    pkv.pkv_key_bounds(kc, tables, cx, start, bounds, 2 ** 20, k_scales=ks)
    # the same append at the same places in blocks of a short table
    near = np.array([[5, 3]], np.int32)
    end = np.array([32 - 5], np.int32)
    at = np.array([0, n])
    was = np.full((NB, H), 2.0 ** -6)
    for got, scale, c, rows in ((kc, ks, codes[0], x[0]), (vc, vs, codes[1], x[1])):
        want, scales = ref.write(c, was, ref.f64(rows), near, end, at, bs)
        assert ref.same_codes(got.cpu().numpy(), want) and np.array_equal(scale.cpu().numpy(), scales)
    keys = ref.values(kc.cpu().numpy(), ks.cpu().numpy())
    assert np.array_equal(ref.f64(bounds), ref.key_bounds(np.zeros(bounds.shape), keys, near, end, at, bs))
    no_device_error()

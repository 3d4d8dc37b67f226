"""Swap of blocks whose scales and bounds are kept by block id: saved and put back beside K and V they give the same
attention from other blocks of the pool."""
import numpy as np
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


@pytest.mark.parametrize("fp8", [True, False])
def test_a_swapped_sequence_attends_as_before(fp8):
    H, g, D, bs, K = 2, 4, 128, 16, 9
    b = ref.Batch([500, 333], [500, 333], H, D, bs, seed=41, g=g)
    n = 32
    old, free = b.tables[0, :n].copy(), np.arange(b.NB, b.NB + n, dtype=np.int32)
    k, v = (cuda(x) for x in ((b.kc, b.vc) if fp8 else b.bf16_pool()))
    k, v = (torch.cat([x, x[:n].clone()]).contiguous() for x in (k, v))  # the free blocks hold others' rows
    ks, vs = (cuda(np.concatenate([x, 3 * x[:n]])) if fp8 else None for x in (b.ks, b.vs))
    bounds = torch.zeros((b.NB + n, H, 2, D), dtype=torch.bfloat16, device="cuda")
    ctx, start, q = cuda(b.ctx), cuda(b.start), cuda(b.q)

    def attention(tables):
        sel = torch.empty((2, H, K), dtype=torch.int32, device="cuda")
        out, dense = torch.empty_like(q), torch.zeros_like(q)
        pkv.pkv_select_blocks(q, bounds, tables, ctx, H, bs, sel, 500)
        pkv.paged_attn_decode_sparse(q, k, v, tables, ctx, sel, b.scale, H, out, k_scales=ks, v_scales=vs)
        if fp8:
            pkv.paged_attn_decode_fp8_block(q, k, v, ks, vs, tables, ctx, b.scale, H, dense, 500)
        return sel, out, dense

    pkv.pkv_key_bounds(k, cuda(b.tables), ctx, start, bounds, 500, k_scales=ks)
    before = attention(cuda(b.tables))

    host_k, host_v = (torch.empty((n, H, bs, D), dtype=k.dtype).pin_memory() for _ in "kv")
    at = torch.from_numpy(old).long().cuda()
    pkv.pkv_swap_out(k, v, old, host_k, host_v)
    saved = [x[at].cpu() for x in ((ks, vs, bounds) if fp8 else (bounds,))]
    torch.cuda.synchronize()
    for x in (k, v):  # the blocks' next owner
        x[at] = 0x7F if fp8 else float("nan")
    for x in (ks, vs) if fp8 else ():
        x[at] = float("nan")
    bounds[at] = float("nan")
    pkv.pkv_swap_in(host_k, host_v, free, k, v)
    to = torch.from_numpy(free).long().cuda()
    for x, rows in zip((ks, vs, bounds) if fp8 else (bounds,), saved):
        x[to] = rows.cuda()
    b.tables[0, :n] = free
    for x, y in zip(before, attention(cuda(b.tables))):
        assert torch.equal(x, y)
    # the bounds again from the keys, the whole sequence as new tokens
    bounds[to] = 0
    pkv.pkv_key_bounds(k, cuda(b.tables), ctx, start, bounds, 500, k_scales=ks)
    for x, y in zip(before, attention(cuda(b.tables))):
        assert torch.equal(x, y)
    no_device_error()

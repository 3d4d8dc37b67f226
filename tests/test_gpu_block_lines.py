"""Every way in which the stream kernel cuts its work, at sizes that take several CTAs: selected blocks as a line that
is cut anywhere (merged by CTA and by unit), dense contexts whose units stay whole, and calls that overlap."""
import numpy as np
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


def repeated(ctx, times, H, g, D, bs, seed):
    """len(ctx) sequences' blocks, read by `times` as many sequences with queries of their own; the contexts of the
    repeats are shorter by up to a block and a half."""
    b = ref.Batch(ctx, [min(c, 1) for c in ctx], H, D, bs, seed=seed, g=g)
    r = np.random.default_rng(seed)
    b.tables = np.ascontiguousarray(np.tile(b.tables, (times, 1)))
    less = r.integers(0, 3 * bs // 2 + 1, len(ctx) * times) * (np.arange(len(ctx) * times) >= len(ctx))
    b.ctx = np.maximum(np.tile(b.ctx, times) - less, 0).astype(np.int32)
    b.q = torch.randn((len(b.ctx), H * g, D), generator=torch.Generator().manual_seed(seed)).to(torch.bfloat16)
    return b


def twice(b, nbytes, call):
    """call(out, workspace) with two different fillings of the workspace and the output: the same rows bit for bit."""
    outs = []
    for byte in (0xFF, 0x7F):
        ws = torch.full((nbytes,), byte, dtype=torch.uint8, device="cuda")
        outs.append(torch.full((len(b.ctx), b.H * b.g, b.D), float("nan"), dtype=torch.bfloat16, device="cuda"))
        call(outs[-1], ws)
    torch.cuda.synchronize()
    assert torch.equal(outs[0].view(torch.int16), outs[1].view(torch.int16))
    return outs[0]


def check_sparse(b, sel, fp8):
    k, v = (b.kc, b.vc) if fp8 else b.bf16_pool()
    t = [cuda(x) for x in (b.q, k, v, b.tables, b.ctx, sel)]
    scales = {"k_scales": cuda(b.ks), "v_scales": cuda(b.vs)} if fp8 else {}
    K = sel.shape[2]
    out = twice(b, pkv.decode_sparse_workspace_bytes(len(b.ctx), b.H * b.g, b.H, b.D, b.bs, K),
                lambda o, ws: pkv.paged_attn_decode_sparse(*t, b.scale, b.H, o, workspace=ws, **scales))
    want = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx, b.scale, b.bs, sel,
                      b.vs if fp8 else None)
    ref.assert_attention(out, want, 2.0 ** -11 if fp8 else 2.0 ** -16)
    empty = torch.from_numpy(np.repeat((sel < 0).all(2), b.g, 1) | (b.ctx <= 0)[:, None])
    assert (out.cpu()[empty] == 0).all()
    no_device_error()


def selection(b, K, seed):
    """Valid blocks in any order, -1 between them and at both ends, some heads without an entry."""
    r = np.random.default_rng(seed)
    sel = np.full((len(b.ctx), b.H, K), -1, np.int32)
    for s, c in enumerate(b.ctx):
        n = -(-int(c) // b.bs)
        for h in range(b.H):
            m = int(r.integers(0, min(n, K) + 1)) if (s + h) % 11 else 0
            sel[s, h, r.permutation(K)[:m]] = r.permutation(n)[:m]
    return sel


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g,D", [(1, 64), (4, 128), (11, 64)])
def test_selected_line_merged_by_cta(fp8, g, D):
    """Over 32,000 stages of 512 units: more than clusters take a unit each for."""
    b = repeated([1500, 900, 37, 1031, 0, 1024, 700, 16], 8, 8, g, D, 16, seed=21)
    sel = selection(b, 64, 1)
    assert sel[..., 0].size * 64 > 32000
    check_sparse(b, sel, fp8)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("H,g,D,bs,K", [(8, 2, 64, 16, 500), (4, 8, 128, 64, 250), (8, 16, 64, 16, 500)])
def test_selected_line_merged_by_unit(fp8, H, g, D, bs, K):
    """At most 64 units of 500 stages or more, each of which goes on over several CTAs, those of a head without an
    entry too."""
    b = repeated([8000, 7000, 16 * 500, 400], 2, H, g, D, bs, seed=22)
    sel = selection(b, K, 2)
    n = -(-b.ctx[0] // bs)
    sel[0, 0] = np.arange(K) % n                        # all of them, none missing
    sel[1, 1], sel[1, 1, -1] = -1, 3                    # the last one alone
    sel[2, 1], sel[2, 1, 0] = -1, 0                     # the first one alone
    assert (sel < 0).all(2).any() and sel[..., 0].size <= 64 and sel[..., 0].size * K * bs // 16 > 30000
    check_sparse(b, sel, fp8)


def check_dense(b, bound):
    t = [cuda(x) for x in (b.q, b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx)]
    out = twice(b, pkv.decode_fp8_block_workspace_bytes(len(b.ctx), b.H * b.g, b.H, b.D, bound),
                lambda o, ws: pkv.paged_attn_decode_fp8_block(*t, b.scale, b.H, o, bound, workspace=ws))
    want = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx, b.scale, b.bs,
                      v_scales=b.vs)
    ref.assert_attention(out, want, 2.0 ** -11)
    assert (out.cpu()[torch.from_numpy(b.ctx <= 0)] == 0).all()
    no_device_error()


@pytest.mark.parametrize("H,g,D", [(3, 1, 64), (2, 4, 128), (2, 12, 64), (1, 16, 128)])
def test_whole_units_of_short_contexts(H, g, D):
    """200 sequences of 0 to 64 tokens: no unit is cut, nothing is merged."""
    ctx = [0, 1, 15, 16, 17, 31, 32, 33, 48, 63, 64, 0, 64] + [(i * 37) % 65 for i in range(37)]
    check_dense(repeated(ctx, 4, H, g, D, 16, seed=23), 64)


@pytest.mark.parametrize("g,D", [(1, 64), (1, 128), (9, 64), (16, 128)])
def test_whole_units_of_many_heads(g, D):
    """2400 units of 0 to 256 tokens."""
    ctx = [256, 1, 16, 15, 17, 240, 241, 255, 0, 128, 127, 129] + [1 + (i * 71) % 256 for i in range(13)]
    check_dense(repeated(ctx, 4, 24, g, D, 16, seed=24), 256)


@pytest.mark.parametrize("bound", [64, 65, 256, 257, 4096])
def test_any_bound_of_the_contexts(bound):
    """The same short batch under bounds that make the units whole or cut."""
    ctx = [64, 1, 16, 63, 17, 0, 33, 48] + [1 + (i * 29) % 64 for i in range(17)]
    check_dense(repeated(ctx, 4, 24, 2, 64, 16, seed=25), bound)


def test_overlapping_dense_calls_give_what_each_gives_alone():
    args, want, got = [], [], []
    for ctx, H, g, D, seed in (([16 * 900], 2, 4, 128, 31), ([16 * 700, 500, 0], 1, 2, 64, 32)):
        b = ref.Batch(ctx, [min(c, 1) for c in ctx], H, D, 16, seed=seed, g=g)
        t = [cuda(x) for x in (b.q, b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx)]
        args.append((t, b.scale, H, max(ctx)))
        alone = torch.empty_like(t[0])
        pkv.paged_attn_decode_fp8_block(*t, b.scale, H, alone, max(ctx))
        torch.cuda.synchronize()
        ref.assert_attention(alone, ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx,
                                               b.scale, 16, v_scales=b.vs), 2.0 ** -11)
        want.append(alone)
        got.append([torch.full_like(alone, float("nan")) for _ in range(8)])
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    torch.cuda.synchronize()
    for i in range(8):
        for (t, scale, H, bound), outs, stream in zip(args, got, streams):
            pkv.paged_attn_decode_fp8_block(*t, scale, H, outs[i], bound, stream=stream)
    torch.cuda.synchronize()
    for outs, alone in zip(got, want):
        for o in outs:
            assert torch.equal(o, alone)
    no_device_error()

"""Block-sparse decode: the selected blocks equal those of fp64 scores, ties, borders and special values included;
attention over them within the kernel's roundings; and the whole step, from the block manager's append to the
attention, eager and as a graph."""
import numpy as np
import pytest
import torch

import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


def batch(ctx, H, g, D, bs, seed):
    return ref.Batch(ctx, [min(c, 1) for c in ctx], H, D, bs, seed=seed, g=g)


def random_bounds(b, seed, spread=1.0):
    gen = torch.Generator().manual_seed(seed)
    x = torch.randn((2, b.NB, b.H, b.D), generator=gen) * spread
    x *= 1 + 6 * (torch.rand((1, 1, b.H, b.D), generator=gen) < 0.05)  # a few large channels
    return torch.stack([torch.minimum(x[0], x[1]), torch.maximum(x[0], x[1])], 2).to(torch.bfloat16).contiguous()


def run_select(b, bounds, K, max_ctx=None, q=None, stream=None):
    sel = torch.full((len(b.ctx), b.H, K), -7, dtype=torch.int32, device="cuda")
    pkv.pkv_select_blocks(cuda(b.q if q is None else q), cuda(bounds), cuda(b.tables), cuda(b.ctx), b.H, b.bs, sel,
                          int(max(b.ctx)) if max_ctx is None else max_ctx, stream=stream)
    torch.cuda.synchronize()
    return sel.cpu().numpy()


def check_select(b, bounds, K, q=None):
    got = run_select(b, bounds, K, q=q)
    want = ref.select(ref.f64(b.q if q is None else q), ref.f64(bounds), b.tables, b.ctx, K, b.bs)
    assert np.array_equal(got, want)
    no_device_error()


SELECTS = [
    # contexts, kv heads, group, head dim, block size, K
    ([0, 1, 16, 33, 64, 65, 1000], 2, 4, 128, 16, 4),
    ([1000, 777, 3000], 3, 1, 64, 16, 2),        # K = 2: the first and the last block only
    ([1000, 777, 3000], 3, 1, 64, 16, 3),
    ([16 * 130, 16 * 1100 + 5], 1, 8, 128, 16, 33), 
    ([16 * 2000, 16 * 1999 + 1], 1, 3, 64, 16, 700),
    ([16 * 2000], 1, 16, 128, 16, 128),
    ([48 * 300 + 7, 48 * 10], 2, 11, 64, 48, 16),
    ([128 * 200], 1, 5, 128, 128, 199),          # all but one
    ([1024 * 70, 1024 * 3], 1, 2, 128, 1024, 8),
    ([300 + 13 * i for i in range(80)], 4, 2, 64, 16, 8),
    ([16 * 9001 + 3, 16 * 8200, 40], 1, 2, 64, 16, 300),  # more scores than a CTA keeps in registers
]


@pytest.mark.parametrize("ctx,H,g,D,bs,K", SELECTS)
def test_select(ctx, H, g, D, bs, K):
    b = batch(ctx, H, g, D, bs, seed=sum(ctx) + K)
    check_select(b, random_bounds(b, sum(ctx)), K)


@pytest.mark.parametrize("ctx,H,K", [
    ([16 * 2100 + 37 * i for i in range(5)], 32, 8),                # 160 heads of over 2048 blocks
    ([40 + 13 * i % 1900 for i in range(155)], 8, 5),               # 1240 heads of up to 122 blocks
])
def test_select_of_many_heads(ctx, H, K):
    """Where there are more heads than an SM takes at once, smaller CTAs select: the same blocks, ties included."""
    b = batch(ctx, H, 1, 64, 16, seed=len(ctx))
    bounds = random_bounds(b, H)
    check_select(b, bounds, K)
    check_select(b, bounds[:3][torch.arange(b.NB) % 3].contiguous(), K)


@pytest.mark.parametrize("n,K", [(40, 9), (600, 100), (3000, 1500), (8500, 700)])
def test_select_ties(n, K):
    """Equal scores go to the lower index: all bounds alike (more undecided blocks than are compared one by one),
    a zero query, and a few kinds of blocks repeated over the context."""
    b = batch([16 * n - 3, 16 * n], 1, 2, 64, 16, seed=n)
    same = torch.zeros((b.NB, 1, 2, 64), dtype=torch.bfloat16)
    same[:, :, 0], same[:, :, 1] = -1.5, 2.25
    check_select(b, same, K)
    check_select(b, random_bounds(b, n), K, q=torch.zeros_like(b.q))
    kinds = random_bounds(b, n + 1)[:5]
    check_select(b, kinds[torch.arange(b.NB) % 5].contiguous(), K)


def test_select_close_scores():
    """Terms of +2^16 and -2^16 leave differences that an fp32 sum cannot see; whole steps of bf16's last bit in one
    column, so that neighbours differ by less than the error of the first scores."""
    b = batch([16 * 1500], 1, 1, 64, 16, seed=3)
    bounds = torch.zeros((b.NB, 1, 2, 64), dtype=torch.bfloat16)
    q = torch.ones_like(b.q)
    q[:, :, 1] = -1
    bounds[:, :, :, 0] = 2.0 ** 16
    bounds[:, :, :, 1] = 2.0 ** 16
    gen = torch.Generator().manual_seed(0)
    bounds[:, :, :, 2] = (torch.randint(0, 9, (b.NB, 1, 1), generator=gen) * 2.0 ** -12).to(torch.bfloat16)
    bounds[:, :, :, 3] = (torch.randint(0, 99, (b.NB, 1, 1), generator=gen) * 2.0 ** -20).to(torch.bfloat16)
    for K in (20, 333, 1400):
        check_select(b, bounds, K, q=q)


@pytest.mark.parametrize("spread", [1e-30, 1e-19, 1e18, 1e37])
def test_select_extreme_magnitudes(spread):
    b = batch([16 * 300], 2, 4, 128, 16, seed=5)
    check_select(b, random_bounds(b, 1, spread), 40)
    check_select(b, random_bounds(b, 1), 40, q=(b.q.float() * spread).to(torch.bfloat16))


def test_select_special_values():
    b = batch([16 * 300, 16 * 50], 2, 4, 128, 16, seed=6)
    bounds = random_bounds(b, 2)
    t = b.tables[0]
    bounds[t[7], 0, 1, 3] = float("nan")      # a NaN score counts as +infinity
    bounds[t[9], 0, 1, :] = float("inf")
    bounds[t[9], 0, 0, :] = float("-inf")
    bounds[t[11], 1, 0, 5] = float("-inf")
    bounds[t[12], 1, 1, 6] = float("inf")
    check_select(b, bounds, 20)
    got = run_select(b, bounds, 20)
    assert 7 in got[0, 0] and 9 in got[0, 0]


def test_select_ignores_what_no_context_covers():
    """Blocks behind the context and other sequences' bounds may hold anything."""
    b = batch([16 * 200 - 8, 16 * 90], 1, 2, 128, 16, seed=7)
    bounds = random_bounds(b, 3)
    used = np.concatenate([b.tables[0, :200], b.tables[1, :90]])
    free = np.setdiff1d(np.arange(b.NB), used)
    bounds[free] = float("nan")
    b.tables[0, 200:] = free[0]
    check_select(b, bounds, 17)


def test_select_reports_bad_blocks_and_contexts():
    b = batch([16 * 100, 16 * 60], 2, 2, 64, 16, seed=8)
    bounds = random_bounds(b, 4)
    want = ref.select(ref.f64(b.q), ref.f64(bounds), b.tables, b.ctx, 10, 16)
    skip = next(j for j in range(1, 99) if j not in want[0, 0] and j not in want[0, 1])
    b.tables[0, skip] = b.NB                      # a block that was not selected anyway
    assert np.array_equal(run_select(b, bounds, 10), want)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    run_select(b, bounds, 10, max_ctx=16 * 60)    # the first context is above the bound: clamped
    assert pkv.get_device_error() & pkv.DEVERR_CONTEXT
    b.ctx[1] = -5
    assert (run_select(b, bounds, 10)[1] == -1).all()
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK


# ------------------------------------------------------------- attention ----


def random_selection(b, K, seed):
    """Distinct valid blocks in any order, -1 between them; at most K."""
    r = np.random.default_rng(seed)
    sel = np.full((len(b.ctx), b.H, K), -1, np.int32)
    for s, c in enumerate(b.ctx):
        n = -(-int(c) // b.bs)
        for h in range(b.H):
            m = r.integers(0, min(n, K) + 1)
            sel[s, h, r.permutation(K)[:m]] = r.permutation(n)[:m]
    return sel


def run_sparse(b, sel, fp8, q=None, stream=None):
    out = torch.full((len(b.ctx), b.H * b.g, b.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    k, v = (b.kc, b.vc) if fp8 else b.bf16_pool()
    scales = {"k_scales": cuda(b.ks), "v_scales": cuda(b.vs)} if fp8 else {}
    pkv.paged_attn_decode_sparse(cuda(b.q if q is None else q), cuda(k), cuda(v), cuda(b.tables), cuda(b.ctx), cuda(sel),
                                 b.scale, b.H, out, stream=stream, **scales)
    torch.cuda.synchronize()
    return out


def check_sparse(b, sel, fp8, what=""):
    out = run_sparse(b, sel, fp8)
    want = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx, b.scale, b.bs, sel,
                      b.vs if fp8 else None)
    # weights: f16 over codes, two bf16 over a bf16 pool
    ref.assert_attention(out, want, 2.0 ** -11 if fp8 else 2.0 ** -16, what)
    empty = torch.from_numpy(np.repeat((sel < 0).all(2), b.g, 1) | (b.ctx <= 0)[:, None])
    assert (out.cpu()[empty] == 0).all()
    return out


SPARSE = [
    # contexts, kv heads, group, head dim, block size, K
    ([0, 1, 15, 16, 17, 100, 1000], 2, 1, 128, 16, 5),
    ([0, 1, 15, 16, 17, 100, 1000], 2, 4, 128, 16, 5),
    ([1000, 1], 1, 1, 64, 16, 64),
    ([5000, 70, 0], 1, 8, 128, 16, 300),  
    ([5000, 4999], 1, 3, 64, 16, 301),
    ([3000, 17], 1, 16, 128, 48, 40),
    ([3000, 1030], 2, 11, 64, 1024, 3),
    ([2000, 129], 1, 2, 128, 128, 1),
    ([200 + 7 * i for i in range(60)], 9, 2, 64, 32, 4),
]


@pytest.mark.parametrize("ctx,H,g,D,bs,K", SPARSE)
@pytest.mark.parametrize("fp8", [False, True])
def test_sparse_decode(ctx, H, g, D, bs, K, fp8):
    b = batch(ctx, H, g, D, bs, seed=sum(ctx) + K).poison()
    check_sparse(b, random_selection(b, K, 1), fp8, f"{ctx} g={g} D={D} bs={bs}")
    no_device_error()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("g", [1, 4])
def test_sparse_reads_only_what_is_selected(fp8, g):
    """NaN everywhere else, a block twice, negative entries of every kind, nothing selected for one head."""
    b = batch([16 * 40 - 5, 100], 2, g, 128, 16, seed=3)
    sel = np.full((2, 2, 12), -1, np.int32)
    sel[0, 0] = [39, 3, -1, 3, 17, -5, 0, 8, -2 ** 31, 25, 4, 5]
    sel[0, 1, 7] = 39
    sel[1, 1, :3] = [6, 0, 6]
    for s in range(2):
        for h in range(2):
            for j in range(-(-int(b.ctx[s]) // 16)):
                if j not in sel[s, h]:
                    b.kc[b.tables[s, j], h] = b.vc[b.tables[s, j], h] = 0x7F
    check_sparse(b, sel, fp8)
    assert (run_sparse(b, sel, fp8)[1, :g] == 0).all()
    no_device_error()


@pytest.mark.parametrize("g,K", [(1, 40), (4, 40), (16, 40), (8, 2)])
def test_sparse_scores_of_minus_infinity(g, K):
    """Keys that lead to scores of -infinity (or below fp32's range) weigh nothing, wherever they come in a warp's
    stretch; a row of nothing else is zero."""
    b = batch([16 * 50, 16 * 3 + 5], 2, g, 128, 16, seed=8)
    b.q[..., 0] = b.q[..., 0].abs() + 0.5
    sel = np.full((2, 2, K), -1, np.int32)
    sel[0] = np.random.default_rng(8).permutation(50)[:K]
    sel[1, :, 0] = 3
    k, v = b.bf16_pool()
    left = sel.copy()
    low = [(0, j) for j in (sel[0, 0, 0], sel[0, 0, K // 2], sel[0, 0, K - 1])[:K // 2]] + [(1, 3)]
    for i, (s, j) in enumerate(low):
        k[b.tables[s, j], :, :, 0] = float("-inf")
        if i == 1:  # finite keys, whose scores overflow
            k[b.tables[s, j], :, :, 0] = torch.finfo(torch.bfloat16).min
            b.q[s, :, 0] = 8.0
        left[s][left[s] == j] = -1
    out = torch.empty((2, 2 * g, 128), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_sparse(cuda(b.q), cuda(k), cuda(v), cuda(b.tables), cuda(b.ctx), cuda(sel), b.scale, 2, out)
    want = ref.attend(ref.f64(b.q), ref.f64(k), ref.f64(v), b.tables, b.ctx, b.scale, 16, left)
    ref.assert_attention(out, want, 2.0 ** -16)
    assert (out[1] == 0).all()
    no_device_error()


def test_sparse_reports_bad_entries():
    b = batch([100, 64], 1, 2, 64, 16, seed=4)
    sel = np.array([[[0, 6, 7, 2]], [[0, 4, 1, 2 ** 31 - 1]]], np.int32)  # 7 and 4 lie behind the contexts
    check_sparse(b, sel, True)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    b.tables[0, 2] = -1
    assert torch.isfinite(run_sparse(b, sel, True).float()).all()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    b.ctx[1] = 1 << 20
    run_sparse(b, sel, False)
    assert pkv.get_device_error() & pkv.DEVERR_CONTEXT


@pytest.mark.parametrize("g", [1, 8])
def test_all_blocks_selected_is_dense_decode(g):
    b = batch([1500, 31], 2, g, 128, 16, seed=5)
    sel = np.full((2, 2, 94), -1, np.int32)
    sel[0], sel[1, :, :2] = np.arange(94), [0, 1]
    out = check_sparse(b, sel, True)
    dense = torch.empty_like(out)
    pkv.paged_attn_decode_fp8_block(cuda(b.q), cuda(b.kc), cuda(b.vc), cuda(b.ks), cuda(b.vs), cuda(b.tables), cuda(b.ctx),
                                    b.scale, 2, dense, 1500)
    want = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx, b.scale, 16,
                      v_scales=b.vs)
    ref.assert_attention(dense, want, 2.0 ** -11)
    no_device_error()


@pytest.mark.parametrize("scale", [-0.25, 0.0])
def test_any_scale(scale):
    b = batch([900, 31], 2, 4, 128, 16, seed=15)
    b.scale = scale
    for fp8 in (False, True):
        check_sparse(b, random_selection(b, 30, 2), fp8)


def test_empty_batch():
    """No sequences: every call returns, with a workspace of its own making too."""
    i32 = dict(dtype=torch.int32, device="cuda")
    ctx, tables, start = torch.zeros(0, **i32), torch.zeros((0, 4), **i32), torch.zeros(1, **i32)
    q = torch.zeros((0, 4, 64), dtype=torch.bfloat16, device="cuda")
    codes = torch.zeros((4, 2, 16, 64), dtype=torch.uint8, device="cuda")
    scales = torch.ones((4, 2), device="cuda")
    bounds = torch.zeros((4, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    sel, rows = torch.zeros((0, 2, 3), **i32), q[:, :2].contiguous()
    pkv.pkv_write_fp8_block(rows, rows, tables, ctx, start, scales, scales, codes, codes, 1)
    pkv.pkv_key_bounds(codes, tables, ctx, start, bounds, 1, scales)
    pkv.pkv_select_blocks(q, bounds, tables, ctx, 2, 16, sel, 64)
    pkv.paged_attn_decode_sparse(q, codes, codes, tables, ctx, sel, 1.0, 2, q, scales, scales)
    pkv.paged_attn_decode_fp8_block(q, codes, codes, scales, scales, tables, ctx, 1.0, 2, q, 64)
    torch.cuda.synchronize()
    assert (codes == 0).all() and (bounds == 0).all()
    no_device_error()


def test_workspace_for_another_stream_is_that_streams_memory():
    """What the current stream has let go of may still be in use there, so a call for another stream takes none of
    it."""
    torch.cuda.empty_cache()
    stream, n = torch.cuda.Stream(), 24 << 20
    device = torch.cuda.current_device()
    for other in (stream, stream.cuda_stream):
        held = torch.empty(n, dtype=torch.uint8, device="cuda")
        at = held.data_ptr()
        del held
        assert pkv._scratch(None, n, device, None)[0] == at
        assert pkv._scratch(None, n, device, other)[0] != at


@pytest.mark.parametrize("fp8", [True, False])
def test_blocks_past_4_gib_of_the_pool(fp8):
    """The same step at the lowest and at the highest block ids of pools of more than 2^32 bytes: every result repeats
    bit for bit."""
    H, g, D, bs, n = 8, 2, 128, 16, 40
    NB = (2 ** 32 // (H * bs * D)) // (1 if fp8 else 2) + 64
    keys, vals = (torch.empty((NB, H, bs, D), dtype=torch.uint8 if fp8 else torch.bfloat16, device="cuda") for _ in "kv")
    ks, vs = (torch.ones((NB, H), device="cuda") if fp8 else None for _ in "kv")
    bounds = torch.empty((NB, H, 2, D), dtype=torch.bfloat16, device="cuda")
    gen = torch.Generator().manual_seed(21)
    x = cuda(torch.randn((bs * n, H, D), generator=gen).to(torch.bfloat16))
    q = cuda(torch.randn((1, H * g, D), generator=gen).to(torch.bfloat16))
    ctx, start = cuda(np.array([bs * n], np.int32)), cuda(np.array([0, bs * n], np.int32))
    got = []
    for first in (0, NB - n):
        tables = cuda(np.arange(first, first + n, dtype=np.int32)[None])
        if fp8:
            pkv.pkv_write_fp8_block(x, x, tables, ctx, start, ks, vs, keys, vals, bs * n)
        else:
            keys[first:first + n] = vals[first:first + n] = x.view(n, bs, H, D).transpose(1, 2)
        pkv.pkv_key_bounds(keys, tables, ctx, start, bounds, bs * n, ks)
        sel = torch.empty((1, H, 9), dtype=torch.int32, device="cuda")
        pkv.pkv_select_blocks(q, bounds, tables, ctx, H, bs, sel, bs * n)
        out = [torch.zeros_like(q), torch.zeros_like(q)]
        pkv.paged_attn_decode_sparse(q, keys, vals, tables, ctx, sel, 0.1, H, out[0], ks, vs)
        if fp8:
            pkv.paged_attn_decode_fp8_block(q, keys, vals, ks, vs, tables, ctx, 0.1, H, out[1], bs * n)
        # a code is half a step off at most: 2^-4 of its value, or 2^-10 of a scale that is 2^-6 at most here
        top, most = bounds[first:first + n, :, 1].float(), x.view(n, bs, H, D).amax(1).float()
        assert ((top - most).abs() <= (most.abs() / 16 + 2.0 ** -16 if fp8 else 0)).all()
        got.append((keys[first:first + n].clone(), vals[first:first + n].clone(), bounds[first:first + n].clone(), sel, *out))
    for a, b in zip(*got):
        assert torch.equal(a, b)
    no_device_error()


def test_two_calls_at_once_give_the_same_results():
    """No state outside a call's arguments: calls that overlap on two streams repeat bit for bit what each gives
    alone."""
    one, two = batch([16 * 900], 2, 4, 128, 16, seed=11), batch([16 * 700, 500], 1, 2, 64, 16, seed=12)
    want = []
    for b in (one, two):
        bounds = random_bounds(b, 9)
        want.append((bounds, run_select(b, bounds, 50), run_sparse(b, run_select(b, bounds, 50), True)))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    calls = []
    for b, (bounds, sel, out), st in zip((one, two), want, streams):
        t = {n: cuda(x) for n, x in (("q", b.q), ("k", b.kc), ("v", b.vc), ("ks", b.ks), ("vs", b.vs), ("bounds", bounds),
                                     ("tables", b.tables), ("ctx", b.ctx))}
        got = [(torch.empty(sel.shape, dtype=torch.int32, device="cuda"), torch.empty_like(out), torch.empty_like(out))
               for _ in range(6)]
        calls.append((b, t, got, st))
    torch.cuda.synchronize()
    for i in range(6):
        for b, t, got, st in calls:
            s, o, dense = got[i]
            pkv.pkv_select_blocks(t["q"], t["bounds"], t["tables"], t["ctx"], b.H, b.bs, s, int(b.ctx.max()), stream=st)
            pkv.paged_attn_decode_sparse(t["q"], t["k"], t["v"], t["tables"], t["ctx"], s, b.scale, b.H, o, k_scales=t["ks"],
                                         v_scales=t["vs"], stream=st)
            pkv.paged_attn_decode_fp8_block(t["q"], t["k"], t["v"], t["ks"], t["vs"], t["tables"], t["ctx"], b.scale, b.H,
                                            dense, int(b.ctx.max()), stream=st)
    torch.cuda.synchronize()
    for (b, t, got, st), (bounds, sel, out) in zip(calls, want):
        for s, o, dense in got:
            assert np.array_equal(s.cpu().numpy(), sel) and torch.equal(o, out) and torch.equal(dense, got[0][2])
    no_device_error()


# ------------------------------------------------------------ whole steps ----


@pytest.mark.parametrize("fp8", [True, False])
def test_serving_steps(fp8):
    """Prompts, a fork, and decode steps: append (block manager), copy-on-write of blocks and scales, write, bounds,
    selection, attention.  The pool is checked against the plain forms after each step, the selection and the
    attention too; the decode step runs as one captured graph that is replayed."""
    H, g, D, bs, NB, K = 2, 4, 128, 16, 200, 6
    B, MBS = 3, 40
    gen = torch.Generator().manual_seed(2)
    bm = pkv.BlockManager(NB)
    tables = torch.full((B, MBS), -1, dtype=torch.int32, device="cuda")
    ctx = torch.zeros(B, dtype=torch.int32, device="cuda")
    dtype = torch.uint8 if fp8 else torch.bfloat16
    kc, vc = (torch.zeros((NB, H, bs, D), dtype=dtype, device="cuda") for _ in range(2))
    ks, vs = (torch.zeros((NB, H), device="cuda") for _ in range(2))
    bounds = torch.zeros((NB, H, 2, D), dtype=torch.bfloat16, device="cuda")
    sel = torch.empty((B, H, K), dtype=torch.int32, device="cuda")
    out = torch.empty((B, H * g, D), dtype=torch.bfloat16, device="cuda")
    scale = D ** -0.5
    wk, wv = np.zeros((NB, H, bs, D), np.uint8 if fp8 else np.float64), np.zeros((NB, H, bs, D), np.uint8 if fp8 else np.float64)
    wks, wvs = np.zeros((NB, H)), np.zeros((NB, H))
    wb = np.zeros((NB, H, 2, D))

    def step(k, v, q, new, num_new, start):
        slots, pairs, npairs = bm.append_slots(tables, ctx, num_new, bs, k.shape[0])
        pkv.copy_blocks_dev(pairs, npairs, kc, vc)
        if fp8:
            pkv.copy_scales_dev(pairs, npairs, ks, vs)
            pkv.pkv_write_fp8_block(k, v, tables, ctx, start, ks, vs, kc, vc, new)
        else:
            pkv.pkv_write(k, v, slots, kc, vc)
        pkv.pkv_key_bounds(kc, tables, ctx, start, bounds, new, k_scales=ks if fp8 else None)
        pkv.pkv_select_blocks(q, bounds, tables, ctx, H, bs, sel, MBS * bs)
        pkv.paged_attn_decode_sparse(q, kc, vc, tables, ctx, sel, scale, H, out, **({"k_scales": ks, "v_scales": vs} if fp8 else {}))
        return pairs, npairs

    def check(k, v, q, num_new, pairs, npairs):
        nonlocal wk, wv, wks, wvs, wb
        torch.cuda.synchronize()
        t, c = tables.cpu().numpy(), ctx.cpu().numpy()
        start = np.concatenate([[0], np.cumsum(num_new)])
        for src, dst in pairs.cpu().numpy()[:int(npairs.item())]:
            wk[dst], wv[dst], wks[dst], wvs[dst] = wk[src], wv[src], wks[src], wvs[src]
        if fp8:
            wk, wks = ref.write(wk, wks, ref.f64(k), t, c, start, bs)
            wv, wvs = ref.write(wv, wvs, ref.f64(v), t, c, start, bs)
            assert ref.same_codes(kc.cpu().numpy(), wk) and ref.same_codes(vc.cpu().numpy(), wv)
            assert np.array_equal(ks.cpu().numpy(), wks) and np.array_equal(vs.cpu().numpy(), wvs)
            keys, vals = ref.values(wk, wks), ref.values(wv, wvs)
        else:
            for s in range(B):
                for i in range(int(num_new[s])):
                    p = c[s] - num_new[s] + i
                    wk[t[s, p // bs], :, p % bs] = ref.f64(k)[start[s] + i]
                    wv[t[s, p // bs], :, p % bs] = ref.f64(v)[start[s] + i]
            keys, vals = wk, wv
        wb = ref.key_bounds(wb, keys, t, c, start, bs)
        assert np.array_equal(ref.f64(bounds), wb)
        want = ref.select(ref.f64(q), wb, t, c, K, bs)
        assert np.array_equal(sel.cpu().numpy(), want)
        o = ref.attend(ref.f64(q), keys, vals, t, c, scale, bs, want, wvs if fp8 else None)
        ref.assert_attention(out, o, 2.0 ** -11 if fp8 else 2.0 ** -16)

    def rows(T):
        mag = torch.exp(torch.randn((T, H, 1), generator=gen))
        return [(torch.randn((T, H, D), generator=gen) * mag).to(torch.bfloat16).cuda() for _ in range(2)]

    def query():
        return torch.randn((B, H * g, D), generator=gen).to(torch.bfloat16).cuda()

    # prompts of 300 and 70 tokens; the third sequence starts as a fork of the first
    num = np.array([300, 70, 0])
    k, v = rows(370)
    q = query()
    pairs = step(k, v, q, 300, torch.tensor([300, 70, 0], dtype=torch.int32, device="cuda"),
                 torch.tensor([0, 300, 370, 370], dtype=torch.int32, device="cuda"))
    check(k, v, q, num, *pairs)
    tables[2], ctx[2] = tables[0], ctx[0]
    bm.share(tables[0, :19].contiguous())
    # decode steps: the graph is captured once, its inputs change
    k, v = rows(B)
    q = query()
    ones = torch.ones(B, dtype=torch.int32, device="cuda")
    start = torch.arange(B + 1, dtype=torch.int32, device="cuda")
    pairs = step(k, v, q, 1, ones, start)  # eager: both sharers of the last block append, one copies it
    check(k, v, q, np.array([1, 1, 1]), *pairs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        captured = step(k, v, q, 1, ones, start)
    for _ in range(18):
        nk, nv = rows(B)
        k.copy_(nk)
        v.copy_(nv)
        q.copy_(query())
        graph.replay()
        check(k, v, q, np.array([1, 1, 1]), *captured)
    assert bm.error() == 0
    no_device_error()

"""The 8-bit cache with a scale for each block: the quantising append and the key bounds bit for bit against plain
fp64 forms, the copies of the scales, and decode attention within the roundings that the kernel makes."""
import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


def run_write(b, max_new=None, k=None, v=None, stream=None):
    kc, vc, ks, vs = (cuda(x.copy()) for x in (b.kc, b.vc, b.ks, b.vs))
    pkv.pkv_write_fp8_block(cuda(b.k if k is None else k), cuda(b.v if v is None else v), cuda(b.tables), cuda(b.ctx),
                            cuda(b.start), ks, vs, kc, vc, int(b.new.max()) if max_new is None else max_new, stream)
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in (kc, vc, ks, vs)]


def check_write(b, got, k=None, v=None):
    for c, s, gc, gs, x in ((b.kc, b.ks, got[0], got[2], b.k if k is None else k),
                            (b.vc, b.vs, got[1], got[3], b.v if v is None else v)):
        wc, ws = ref.write(c, s, ref.f64(x), b.tables, b.ctx, b.start, b.bs)
        assert np.array_equal(gs.astype(np.float64), ws)
        assert ref.same_codes(gc, wc)


WRITES = [
    # contexts, new tokens, kv heads, head dim, block size
    ([1], [1], 1, 64, 16),
    ([17, 16, 15, 33, 1], [1, 1, 1, 1, 1], 3, 128, 16),          # a decode step: block ends, fresh blocks
    ([40, 100, 7, 64], [40, 37, 0, 64], 2, 64, 16),               # prompts, a chunk, an idle sequence
    ([130, 95, 48], [130, 50, 1], 4, 128, 48),                    # teams of 3 warps
    ([300, 129, 128], [299, 1, 128], 2, 64, 128),                 # teams of 8
    ([1500, 1024, 700], [1500, 5, 650], 2, 128, 1024),            # several groups of rows a warp
    ([0, 5], [0, 5], 40, 128, 32),
]


@pytest.mark.parametrize("ctx,new,H,D,bs", WRITES)
def test_write_bit_exact(ctx, new, H, D, bs):
    b = ref.Batch(ctx, new, H, D, bs, seed=sum(ctx) + bs)
    check_write(b, run_write(b))
    no_device_error()


@pytest.mark.parametrize("D", [64, 128])
def test_write_growth_and_special_values(D):
    """Scales that grow by many powers of two, zeros, infinities, NaN, bf16's least and largest values, and
    magnitudes at the border 448 * 2^k."""
    b = ref.Batch([9, 20, 33, 18, 30, 16, 5, 21], [1, 3, 17, 1, 13, 16, 5, 2], 2, D, 16, seed=3)
    k = b.k.clone()
    t = b.start
    k[t[0]:t[1]] = 1e30
    k[t[1]:t[2]] = 0
    k[t[2], 0, 0], k[t[2] + 1, 0, 1], k[t[2] + 2, 1, 5] = float("inf"), float("-inf"), float("nan")
    k[t[3]:t[4]] = float("inf")  # nothing finite: no growth
    k[t[4]:t[5]] = torch.finfo(torch.bfloat16).max
    k[t[4], 0, :4] = torch.tensor([1e-40, -1e-38, 448.0, 0.0]).to(torch.bfloat16)
    k[t[5]:t[6]] = 1e-39  # below every scale
    k[t[6]:t[7], 0] = 448.0 * 4
    k[t[6]:t[7], 1] = 452.0 * 4  # the next bf16 up
    k[t[7]:t[8]] = 1e-3
    b.ks[:] = 2.0 ** -120
    b.kc[:, 1] = 0x01  # the least code: growth rounds it away
    check_write(b, run_write(b, k=k), k=k)
    no_device_error()


def test_write_grows_a_block_whole():
    """Rows past the context keep their values too when the scale of their block grows, NaN among them."""
    b = ref.Batch([20, 35], [1, 2], 2, 128, 16, seed=15)
    b.ks[:], b.vs[:] = 2.0 ** -9, 2.0 ** -5
    b.kc[b.tables[0, 1], :, 9] = 0x7F
    got = run_write(b, k=b.k * 50, v=b.v * 1e4)
    check_write(b, got, k=b.k * 50, v=b.v * 1e4)
    assert (got[2] > b.ks).sum() == 4 and (got[0][b.tables[0, 1], :, 10:] != b.kc[b.tables[0, 1], :, 10:]).any()
    no_device_error()


def test_write_again_changes_nothing():
    """The same append on its own result: scales and codes stay (it is what a replayed graph does)."""
    b = ref.Batch([40, 9, 100], [5, 1, 100], 3, 128, 16, seed=8)
    first = run_write(b)
    b.kc, b.vc, b.ks, b.vs = first
    again = run_write(b)
    for x, y in zip(first, again):
        assert np.array_equal(x, y)
    no_device_error()


def test_write_leaves_faulty_sequences_out():
    b = ref.Batch([40, 30, 20, 50], [10, 30, 20, 3], 2, 64, 16, seed=4)
    want = ref.Batch([40, 30, 20, 50], [10, 30, 20, 3], 2, 64, 16, seed=4)
    b.tables[1, 1] = b.NB + 7                      # its second block lies outside the pool
    got = run_write(b, max_new=20)                  # and it has more tokens than the bound
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT
    want.start = b.start
    keep = want.tables[1, :2]
    check = [x.copy() for x in (b.kc, b.ks)]
    wc, ws = ref.write(b.kc, b.ks, ref.f64(b.k), want.tables, want.ctx, want.start, 16)
    wc[keep], ws[keep] = check[0][keep], check[1][keep]
    assert ref.same_codes(got[0], wc) and np.array_equal(got[2].astype(np.float64), ws)
    got = run_write(b)                              # within the bound: only the bad block is left out
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    wc, ws = ref.write(b.kc, b.ks, ref.f64(b.k), want.tables, want.ctx, want.start, 16)
    wc[keep[1]], ws[keep[1]] = check[0][keep[1]], check[1][keep[1]]
    assert ref.same_codes(got[0], wc) and np.array_equal(got[2].astype(np.float64), ws)
    b.ctx[3] = 2                                    # fewer positions than new tokens
    run_write(b)
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK


def test_write_ignores_rows_behind_the_last_sequence():
    b = ref.Batch([20, 11], [20, 11], 2, 128, 16, seed=6)
    tail = torch.full((5, 2, 128), float("nan"), dtype=torch.bfloat16)
    got = run_write(b, k=torch.cat([b.k, tail]), v=torch.cat([b.v, tail]))
    check_write(b, got)
    no_device_error()


def test_copy_scales_host_and_device():
    g = torch.Generator().manual_seed(0)
    NB, H = 900, 5
    ks, vs = torch.rand((NB, H), generator=g).cuda(), torch.rand((NB, H), generator=g).cuda()
    wk, wv = ks.clone(), vs.clone()
    perm = torch.randperm(NB, generator=g).numpy().astype(np.int32)
    pairs = np.stack([perm[:420], perm[420:840]], 1)  # more than one launch's
    wk[pairs[:, 1]], wv[pairs[:, 1]] = wk[pairs[:, 0]], wv[pairs[:, 0]]
    pkv.pkv_copy_scales(pairs, ks, vs)
    assert torch.equal(ks, wk) and torch.equal(vs, wv)
    dev = torch.tensor([[0, 890], [3, 891], [NB, 892], [5, -1], [7, 893]], dtype=torch.int32, device="cuda")
    ids = torch.tensor([0, 3], device="cuda")
    pkv.copy_scales_dev(dev, torch.tensor([4], dtype=torch.int32, device="cuda"), ks, vs)
    wk[890:892], wv[890:892] = wk[ids], wv[ids]
    assert torch.equal(ks, wk) and torch.equal(vs, wv)
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK


@pytest.mark.parametrize("ctx,new,H,D,bs", WRITES)
@pytest.mark.parametrize("fp8", [False, True])
def test_key_bounds(ctx, new, H, D, bs, fp8):
    b = ref.Batch(ctx, new, H, D, bs, seed=sum(ctx) + bs + 1).poison()
    gen = torch.Generator().manual_seed(1)
    bounds = torch.randn((b.NB, H, 2, D), generator=gen).to(torch.bfloat16)
    got = bounds.cuda()
    if fp8:
        keys = ref.values(b.kc, b.ks)
        pkv.pkv_key_bounds(cuda(b.kc), cuda(b.tables), cuda(b.ctx), cuda(b.start), got, int(b.new.max()),
                           k_scales=cuda(b.ks))
    else:
        pool = b.bf16_pool()[0]
        keys = ref.f64(pool)
        pkv.pkv_key_bounds(cuda(pool), cuda(b.tables), cuda(b.ctx), cuda(b.start), got, int(b.new.max()))
    want = ref.key_bounds(ref.f64(bounds), keys, b.tables, b.ctx, b.start, bs)
    assert torch.equal(got.cpu().float(), torch.from_numpy(want).to(torch.bfloat16).float())
    no_device_error()


def test_key_bounds_of_nan_and_infinite_keys():
    b = ref.Batch([20], [20], 2, 64, 16, seed=2)
    pool = b.bf16_pool()[0]
    blk = int(b.tables[0, 0])
    pool[blk, 0, 3, 5], pool[blk, 1, 0, 7], pool[blk, 1, 2, 8] = float("nan"), float("inf"), float("-inf")
    got = torch.zeros((b.NB, 2, 2, 64), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_key_bounds(cuda(pool), cuda(b.tables), cuda(b.ctx), cuda(b.start), got, 20)
    got = got.cpu().float()
    assert got[blk, 0, :, 5].isnan().all() and got.isnan().sum() == 2
    assert got[blk, 1, 1, 7] == float("inf") and got[blk, 1, 0, 8] == float("-inf")
    no_device_error()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 48])
def test_key_bounds_of_every_code(D, bs):
    """Any code beside any other: columns of one sign, of zeros of both signs, of the largest codes, with a NaN of
    either sign."""
    r = np.random.default_rng(17)
    b = ref.Batch([bs * 5 - 3, 2], [bs * 5 - 3, 2], 3, D, bs, seed=16)
    kinds = [np.arange(256), np.arange(0x7F), 0x80 + np.arange(0x7F), [0, 0x80], [0x7C, 0x7D, 0x7E], [0xFC, 0xFD, 0xFE],
             [0x7E, 0xFE, 0x7F], [0xFE, 0xFF], [0x01, 0x81, 0x00]]
    for blk in range(b.NB):
        for h in range(3):
            for d in range(D):
                b.kc[blk, h, :, d] = r.choice(np.asarray(kinds[r.integers(len(kinds))], np.uint8), bs)
    got = torch.zeros((b.NB, 3, 2, D), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_key_bounds(cuda(b.kc), cuda(b.tables), cuda(b.ctx), cuda(b.start), got, bs * 5, k_scales=cuda(b.ks))
    want = ref.key_bounds(np.zeros(got.shape), ref.values(b.kc, b.ks), b.tables, b.ctx, b.start, bs)
    assert np.array_equal(ref.f64(got), want, equal_nan=True)
    no_device_error()


def run_decode(b, q=None, stream=None, workspace=None):
    out = torch.full((len(b.ctx), b.H * b.g, b.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_fp8_block(cuda(b.q if q is None else q), cuda(b.kc), cuda(b.vc), cuda(b.ks), cuda(b.vs),
                                    cuda(b.tables), cuda(b.ctx), b.scale, b.H, out, int(b.ctx.max()), workspace=workspace,
                                    stream=stream)
    torch.cuda.synchronize()
    return out


def attend(b, q=None):
    return ref.attend(ref.f64(b.q if q is None else q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx,
                      b.scale, b.bs, v_scales=b.vs)


DECODES = [
    # contexts, kv heads, group, head dim, block size
    ([1, 15, 16, 17, 31, 100, 0], 3, 1, 128, 16),
    ([1, 15, 16, 17, 31, 100, 0], 3, 1, 64, 16),
    ([0, 0, 0], 2, 4, 128, 16),                        # nothing to attend to
    ([700, 33, 2049], 2, 1, 64, 32),
    ([700, 33, 2049], 2, 1, 128, 48),
    ([5, 200, 513, 0], 2, 2, 128, 16),
    ([5, 200, 513, 1537], 4, 3, 64, 64),
    ([2048, 2047, 2576], 2, 4, 128, 16),
    ([6000], 1, 8, 128, 16),                           # one head over many CTAs
    ([2048, 1000, 2576], 1, 8, 64, 128),
    ([1000, 3000, 77], 1, 16, 128, 16),
    ([1000, 3000, 77], 2, 11, 64, 1024),
    ([0, 40, 0, 16, 0, 7] + [i % 90 for i in range(400)] + [0, 0], 2, 2, 64, 16),   # more sequences than threads
    ([17 + 37 * i % 400 for i in range(90)], 24, 1, 128, 16),                       # units within a warp's stretch
]


@pytest.mark.parametrize("ctx,H,g,D,bs", DECODES)
@pytest.mark.parametrize("poison", [False, True])
def test_decode(ctx, H, g, D, bs, poison):
    b = ref.Batch(ctx, [min(c, 1) for c in ctx], H, D, bs, seed=sum(ctx) + g, g=g)
    if poison:
        b.poison()
    out = run_decode(b)
    ref.assert_attention(out, attend(b), 2.0 ** -11, f"{ctx} g={g} D={D}")
    assert (out.cpu()[torch.tensor(ctx) == 0] == 0).all()
    no_device_error()


@pytest.mark.parametrize("g,D", [(1, 128), (1, 64), (4, 128), (16, 64)])
def test_decode_scales_far_apart(g, D):
    """V scales from 2^-100 to 2^90 and K scales over 2^20, with q as small as 2^-40 and as large as 2^30: the
    weighted sum is taken relative to the largest product, so no block's share is lost."""
    r = np.random.default_rng(g + D)
    b = ref.Batch([400, 129, 64], [1, 1, 1], 2, D, 16, seed=11, g=g)
    b.vs = (2.0 ** r.integers(-100, 91, b.vs.shape)).astype(np.float32)
    b.ks = (2.0 ** r.integers(-24, -4, b.ks.shape)).astype(np.float32)
    ref.assert_attention(run_decode(b), attend(b), 2.0 ** -11, "V scales")
    # one sequence of blocks that get larger values and smaller weights, the other way round in the second
    b = ref.Batch([256, 256], [1, 1], 1, D, 16, seed=12, g=g)
    for s in range(2):
        for j in range(16):
            up = j if s == 0 else 15 - j
            b.vs[b.tables[s, j]] = 2.0 ** (4 * up)
            b.ks[b.tables[s, j]] = 2.0 ** (-8 - up / 2 // 1)
    for shift in (-40, 30):
        q = (b.q.float() * 2.0 ** shift).to(torch.bfloat16)
        b.scale = 2.0 ** -shift / 8
        ref.assert_attention(run_decode(b, q=q), attend(b, q), 2.0 ** -11, f"q 2^{shift}")
    no_device_error()


def test_decode_zero_values_and_least_scales():
    """Blocks whose values are all zero have the least scale, and still take their share of the softmax."""
    for g in (1, 4):
        b = ref.Batch([64], [1], 1, 128, 16, seed=5, g=g)
        for j in (0, 2):
            b.vc[b.tables[0, j]], b.vs[b.tables[0, j]] = 0, 2.0 ** -126
        ref.assert_attention(run_decode(b), attend(b), 2.0 ** -11, "zero blocks")
        b.vc[:], b.vs[:] = 0, 2.0 ** -126
        assert (run_decode(b) == 0).all()
    no_device_error()


def test_decode_matches_the_bf16_pool():
    """The same values in a bf16 pool, through paged_attn_decode, within both kernels' roundings."""
    b = ref.Batch([37, 500, 1025], [1, 1, 1], 2, 128, 16, seed=5, g=4, spread=0.5)
    k, v = b.bf16_pool()
    out = torch.empty((3, 8, 128), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode(b.q.cuda(), k.cuda(), v.cuda(), cuda(b.tables), cuda(b.ctx), b.scale, 2, out, 1025)
    want = attend(b)
    ref.assert_attention(out, want, 2.0 ** -8, "bf16 pool")
    ref.assert_attention(run_decode(b), want, 2.0 ** -11, "block-scaled pool")


def test_decode_on_a_stream_and_in_a_graph():
    b = ref.Batch([300, 40, 1200], [1, 1, 1], 2, 128, 16, seed=9, g=4)
    want = run_decode(b)
    stream = torch.cuda.Stream()
    assert torch.equal(run_decode(b, stream=stream), want)
    assert torch.equal(run_decode(b, stream=stream.cuda_stream), want)
    args = [cuda(x) for x in (b.q, b.kc, b.vc, b.ks, b.vs, b.tables, b.ctx)]
    out = torch.zeros_like(want)
    ws = torch.empty(pkv.decode_fp8_block_workspace_bytes(3, 8, 2, 128, 1200), dtype=torch.uint8, device="cuda")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        pkv.paged_attn_decode_fp8_block(*args, b.scale, 2, out, 1200, workspace=ws)
    for _ in range(3):
        out.zero_()
        ws.fill_(0xFF)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    no_device_error()


def test_decode_reports_bad_blocks_and_contexts():
    b = ref.Batch([100, 50], [1, 1], 2, 128, 16, seed=10, g=2)
    b.tables[0, 2] = b.NB
    out = run_decode(b)
    assert torch.isfinite(out.float()).all()
    assert pkv.get_device_error() == pkv.DEVERR_BLOCK
    b.tables[0, 2] = b.unused[0]
    b.ctx[1] = 4096  # past its table: clamped to it, whose last entries hold no block
    run_decode(b)
    assert pkv.get_device_error() == pkv.DEVERR_CONTEXT | pkv.DEVERR_BLOCK

"""The block-scaled cache and block-sparse decode at the ends of their types' ranges: small weights beside a large
one, queries with one large element, the least V scales, infinite values, old scales that are no powers of two."""
import math

import numpy as np
import pytest
import torch

import oracle
import paged_kv_cache_420_b200 as pkv
from tests import _block_ref as ref
from tests._gpu_util import no_device_error

pytestmark = pytest.mark.gpu

ONE = 0x38  # the e4m3 code of 1


def cuda(x):
    return (torch.from_numpy(x) if isinstance(x, np.ndarray) else x).cuda()


def one_warp(ctx, H, g, D, seed):
    """Contexts of at most 64 tokens, which one warp takes alone; no key differs from another yet."""
    b = ref.Batch(ctx, [1] * len(ctx), H, D, 16, seed=seed, g=g)
    b.kc[:], b.ks[:] = 0, 1.0
    return b


def decode(b, sel=None):
    out = torch.full((len(b.ctx), b.H * b.g, b.D), float("nan"), dtype=torch.bfloat16, device="cuda")
    pool = [cuda(x) for x in (b.kc, b.vc, b.ks, b.vs)]
    if sel is None:
        pkv.paged_attn_decode_fp8_block(cuda(b.q), *pool, cuda(b.tables), cuda(b.ctx), b.scale, b.H, out, int(b.ctx.max()))
    else:
        pkv.paged_attn_decode_sparse(cuda(b.q), *pool[:2], cuda(b.tables), cuda(b.ctx), cuda(sel), b.scale, b.H, out,
                                     k_scales=pool[2], v_scales=pool[3])
    torch.cuda.synchronize()
    return out


def check(b, what, zmag=None):
    """Dense, and with every block selected.  |got - out| within `_block_ref.assert_attention`'s roundings, but an f16
    product is at most 2^15 where the reference of its column is 1 * 2^7, so its spacing of 2^-24 below 2^-14 is 2^-31
    of the largest product, and half of that is what a product is off by at most; and bf16's own spacing below its
    normal range, 2^-133, in place of an absolute term.  zmag: the largest sum |q k| scale, for scores without rounding."""
    n = b.tables.shape[1]
    every = np.where(np.arange(n) * b.bs < b.ctx[:, None], np.arange(n), -1)
    sel = np.ascontiguousarray(np.broadcast_to(every[:, None], (len(b.ctx), b.H, n)).astype(np.int32))
    out, weight, most, unit = ref.attend(ref.f64(b.q), ref.values(b.kc, b.ks), ref.values(b.vc, b.vs), b.tables, b.ctx,
                                         b.scale, b.bs, v_scales=b.vs)
    dz = 2 * (2 * 132 * 2.0 ** -24 * (most if zmag is None else most * zmag) + 2.0 ** -20)[..., None]
    tol = 2.0 ** -8 * np.abs(out) + weight * (2.0 ** -11 + dz + 2.0 ** -11) + 2.0 ** -32 * unit + 2.0 ** -133
    for form, s in (("dense", None), ("selected", sel)):
        got = ref.f64(decode(b, s))
        assert np.isfinite(got).all()
        worst = (np.abs(got - out) / tol).max()
        assert worst <= 1.0, f"{what}, {form}: {worst:.3f} of the tolerance"
    no_device_error()


@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (16, 128), (11, 64)])
@pytest.mark.parametrize("below", [14.5, 20.4, 26.3])
def test_weights_far_below_the_largest(g, D, below):
    """One token outweighs the others by 2^below and has no value in half of the columns, where the row is made of the
    others alone."""
    b = one_warp([64, 41], 2, g, D, seed=int(below))
    gen = torch.Generator().manual_seed(g)
    b.q = (torch.randn(b.q.shape, generator=gen) * 0.002).to(torch.bfloat16)
    b.q[..., 0] = 1.0
    b.scale = below * math.log(2)
    r = np.random.default_rng(D)
    b.kc[..., 1:] = r.choice(np.array([0x30, 0x38, 0xB0, 0xB8], np.uint8), b.kc[..., 1:].shape)
    b.vs = (2.0 ** r.integers(-2, 3, b.vs.shape)).astype(np.float32)
    for s in range(2):
        blk = b.tables[s, 0]
        b.kc[blk, :, 5, 0] = ONE
        b.vc[blk, :, 5, ::2] = 0
    check(b, f"2^-{below}")


@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (16, 128), (11, 64)])
@pytest.mark.parametrize("shift", [0, -100, 100])
def test_query_with_one_large_element(g, D, shift):
    """The scores come from the elements at 2^-22 of the largest one, which meets keys of zero."""
    b = one_warp([64, 30], 2, g, D, seed=7)
    gen = torch.Generator().manual_seed(g)
    b.q = (torch.randn(b.q.shape, generator=gen) * 2.0 ** (shift - 22)).to(torch.bfloat16)
    b.q[..., 0] = 2.0 ** shift
    b.scale = 2.0 ** -shift
    r = np.random.default_rng(D)
    b.kc[..., 1:] = r.integers(0, 0x60, b.kc[..., 1:].shape) | r.choice(np.array([0, 0x80]), b.kc[..., 1:].shape)
    b.ks[:] = 2.0 ** 16
    check(b, f"2^{shift}")


@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (16, 128)])
@pytest.mark.parametrize("power", [17, 22, 25, 40])
def test_equal_scores_of_any_size(g, D, power):
    """All keys alike: the row is the mean of the values, whatever the score that they share."""
    b = one_warp([64, 33, 5], 2, g, D, seed=power)
    b.kc[..., 0] = ONE
    b.q[:] = 0
    b.q[..., 0] = 1.25
    b.scale = 2.0 ** power
    b.vs = (2.0 ** np.random.default_rng(power).integers(-9, 9, b.vs.shape)).astype(np.float32)
    for scale in (b.scale, -b.scale):
        b.scale = scale
        check(b, f"2^{power}", zmag=0.0)


@pytest.mark.parametrize("g", [1, 8, 16])
@pytest.mark.parametrize("up", [7.5, 8.5, 9.0])
def test_least_v_scales(g, up):
    """Values of 2^-126 * code, which bf16 holds, next to a block of larger ones that weighs 2^-up of theirs."""
    b = one_warp([32], 2, g, 128, seed=9)
    b.q[:] = 0
    b.q[..., 0] = 1.0
    b.scale = up * math.log(2)
    first, second = b.tables[0, :2]
    b.kc[second, :, :, 0] = ONE
    b.vs[first], b.vs[second] = 2.0 ** -119, 2.0 ** -126
    b.vc[first] = 0x08  # 2^-6
    check(b, f"2^-{up}")
    # nothing but the least scale
    b.vs[first] = 2.0 ** -126
    check(b, "one scale")


@pytest.mark.parametrize("g,D", [(1, 128), (4, 64), (16, 128), (8, 128)])
@pytest.mark.parametrize("blocks", [2, 40])
def test_infinite_values_of_a_bf16_pool(g, D, blocks):
    """A value of infinity gives an infinite sum in its column alone, and NaN only where both signs meet."""
    b = ref.Batch([16 * blocks - 3], [1], 2, D, 16, seed=blocks, g=g)
    b.ks[:] = 2.0 ** -9  # scores of some units: no weight is below 2^-100
    k, v = b.bf16_pool()
    for h in range(2):
        for i, col in enumerate(range(0, D, 5)):
            v[b.tables[0, i % blocks], h, i % 13, col] = float("inf") if i % 2 else float("-inf")
        v[b.tables[0, 0], h, 3, 7], v[b.tables[0, 1], h, 2, 7] = float("inf"), float("-inf")
        # the largest score: its weight is 1 exactly
        v[b.tables[0, 0], h, 0, 11] = float("inf")
        k[b.tables[0, 0], h, 0] = 6 * b.q[0, h * g] / b.q[0, h * g].float().norm()
    sel = np.ascontiguousarray(np.broadcast_to(np.arange(blocks, dtype=np.int32), (1, 2, blocks)))
    out = torch.empty((1, 2 * g, D), dtype=torch.bfloat16, device="cuda")
    pkv.paged_attn_decode_sparse(cuda(b.q), cuda(k), cuda(v), cuda(b.tables), cuda(b.ctx), cuda(sel), b.scale, 2, out)
    with np.errstate(invalid="ignore"):
        want = ref.attend(ref.f64(b.q), ref.f64(k), ref.f64(v), b.tables, b.ctx, b.scale, 16, sel)
    got, finite = ref.f64(out), np.isfinite(want[0])
    assert np.array_equal(got[~finite], want[0][~finite], equal_nan=True)
    assert np.isnan(got[..., 7]).all() and (got[..., 11] == np.inf).all()
    dz = 2 * (2 * 132 * 2.0 ** -24 * want[2] + 2.0 ** -20)[..., None]
    with np.errstate(invalid="ignore"):
        tol = 2.0 ** -8 * np.abs(want[0]) + want[1] * (2.0 ** -16 + dz + 2.0 ** -11)
    assert (np.abs(got[finite] - want[0][finite]) <= tol[finite]).all()
    no_device_error()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new,bs", [(1, 16), (7, 16), (1, 48), (40, 64)])
def test_write_under_an_old_scale_that_is_no_power_of_two(D, new, bs):
    """The quotient x / scale rounded to fp32 once, then to e4m3: quotients that are ties, and scales whose reciprocal
    is below fp32's normal range."""
    r = np.random.default_rng(D + new)
    scales = [7.0, 3.0, 49.0, 2.0 ** 126 * 1.5, 3e38, 1e-30] + [float(x) for x in np.exp(r.uniform(-60, 60, 26))]
    n = len(scales)
    b = ref.Batch([9 + new] * n, [new] * n, 2, D, bs, seed=1)
    b.ks[b.tables[:, 0]] = b.vs[b.tables[:, 0]] = np.asarray(scales, np.float32)[:, None]
    t = np.repeat(np.arange(n), new)
    s = np.asarray(scales, np.float64)[t, None, None]
    # values whose quotients are ties or near them, and any; below 224 scales, so that none of them grows
    odd = r.integers(16, 32, (len(t), 2, D)) * 2.0 ** r.integers(-6, 3, (len(t), 2, D))
    k = torch.from_numpy(np.clip(odd * s, -3e38, 3e38)).to(torch.bfloat16)
    v = torch.from_numpy(np.clip(s * 60 * r.standard_normal((len(t), 2, D)).clip(-3.5, 3.5), -3e38, 3e38)).to(torch.bfloat16)
    kc, vc, ks, vs = (cuda(x.copy()) for x in (b.kc, b.vc, b.ks, b.vs))
    pkv.pkv_write_fp8_block(cuda(k), cuda(v), cuda(b.tables), cuda(b.ctx), cuda(b.start), ks, vs, kc, vc, new)
    assert np.array_equal(ks.cpu().numpy(), b.ks) and np.array_equal(vs.cpu().numpy(), b.vs)
    for got, was, x in ((kc, b.kc, k), (vc, b.vc, v)):
        want = was.copy()
        quotient = x.float().numpy() / np.asarray(scales, np.float32)[t, None, None]
        for i in range(len(t)):
            want[b.tables[t[i], 0], :, 9 + i % new] = oracle.e4m3_encode(quotient[i].astype(np.float64))
        assert ref.same_codes(got.cpu().numpy(), want)
    no_device_error()


def outward(x, up):
    """fp64 values as the nearest bf16 that is not below them (up), or not above."""
    sign = 1.0 if up else -1.0
    y = torch.from_numpy(x * sign).to(torch.bfloat16)
    y = torch.where(y.double() < torch.from_numpy(x * sign), torch.nextafter(y, torch.full_like(y, float("inf"))), y)
    return y.double().numpy() * sign


@pytest.mark.parametrize("D,bs", [(64, 16), (128, 48)])
def test_bounds_hold_the_keys_under_any_scale(D, bs):
    """Scales that are no powers of two, and powers of two whose products leave bf16's normal range: the least key is
    rounded down, the largest up."""
    scales = [0.1, 7.0, 1e-38, 3e35, 2.0 ** -126, 2.0 ** -125, 2.0 ** -124, 2.0 ** 119, 2.0 ** 120, 3e38]
    r = np.random.default_rng(D)
    scales += [float(x) for x in np.exp(r.uniform(-80, 80, 20))]
    b = ref.Batch([bs] * len(scales), [bs] * len(scales), 2, D, bs, seed=3)
    b.ks[b.tables[:, 0]] = np.asarray(scales, np.float32)[:, None]
    b.kc[b.tables[:5, 0], :, :, :5] = np.array([0x00, 0x01, 0x81, 0x80, 0x7E], np.uint8)  # whole columns
    got = torch.zeros((b.NB, 2, 2, D), dtype=torch.bfloat16, device="cuda")
    pkv.pkv_key_bounds(cuda(b.kc), cuda(b.tables), cuda(b.ctx), cuda(b.start), got, bs, k_scales=cuda(b.ks))
    at = b.tables[:, 0]
    keys, got = ref.values(b.kc, b.ks)[at], ref.f64(got)[at]
    assert (got[:, :, 0] <= keys.min(2)).all() and (got[:, :, 1] >= keys.max(2)).all()
    big = torch.finfo(torch.bfloat16).max
    assert np.array_equal(got[:, :, 0], np.minimum(outward(keys.min(2), False), big))
    assert np.array_equal(got[:, :, 1], np.maximum(outward(keys.max(2), True), -big))
    no_device_error()

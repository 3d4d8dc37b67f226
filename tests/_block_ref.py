"""Plain fp64 forms of the block-scaled cache and of block-sparse decode, and inputs for their tests (not
collected as tests).  Loops over blocks and sequences, in numpy, from the definitions."""
import functools
import math

import numpy as np
import torch

import oracle

E4M3_MAX = 448.0


@functools.lru_cache(maxsize=None)
def _table():
    return oracle.e4m3_decode(np.arange(256, dtype=np.uint8))


def decode(codes) -> np.ndarray:
    """The values of e4m3 codes."""
    return _table()[codes]


def f64(t) -> np.ndarray:
    """A bf16 or fp32 tensor's values."""
    return t.detach().cpu().to(torch.float64).numpy()


def pow2_scale(amax: float) -> float:
    """The least power of two >= 2^-126 with amax <= 448 s, by trying them in turn."""
    for e in range(-126, 128):
        if amax <= E4M3_MAX * 2.0 ** e:
            return 2.0 ** e
    raise AssertionError(amax)


def write(codes, scales, x, tables, ctx, start, bs):
    """pkv_write_fp8_block for one of K and V: codes uint8 [NB, H, bs, D], scales [NB, H], x float64 [T, H, D]."""
    codes, scales = codes.copy(), scales.astype(np.float64)
    H = codes.shape[1]
    for s in range(len(ctx)):
        n = start[s + 1] - start[s]
        p0, j = ctx[s] - n, (ctx[s] - n) // bs
        while n > 0 and j * bs < ctx[s]:
            blk, old = tables[s, j], max(p0 - j * bs, 0)
            held = min(ctx[s] - j * bs, bs)
            t0 = start[s] + j * bs + old - p0
            for h in range(H):
                rows = x[t0:t0 + held - old, h]
                finite = np.abs(rows[np.isfinite(rows)])
                need = pow2_scale(finite.max() if finite.size else 0.0)
                if old:
                    was = scales[blk, h]
                    need = max(was, need)
                    if need > was:
                        codes[blk, h] = oracle.e4m3_encode(decode(codes[blk, h]) * (was / need))
                codes[blk, h, old:held] = oracle.e4m3_encode(rows / need)
                scales[blk, h] = need
            j += 1
    return codes, scales


def values(codes, scales):
    """The pool's values [NB, H, bs, D]."""
    return decode(codes) * np.asarray(scales, np.float64)[:, :, None, None]


def same_codes(a, b):
    """Codes that stand for the same values (either NaN code is NaN, either zero is zero)."""
    x, y = decode(a), decode(b)
    return np.array_equal(x, y, equal_nan=True)


def key_bounds(bounds, keys, tables, ctx, start, bs):
    """pkv_key_bounds over the values `keys` [NB, H, bs, D], before rounding to bf16."""
    bounds = bounds.copy()
    for s in range(len(ctx)):
        n = start[s + 1] - start[s]
        if n <= 0:
            continue
        for j in range((ctx[s] - n) // bs, (ctx[s] - 1) // bs + 1):
            rows = keys[tables[s, j], :, :min(ctx[s] - j * bs, bs)]
            bounds[tables[s, j], :, 0] = rows.min(1)
            bounds[tables[s, j], :, 1] = rows.max(1)
    return bounds


def block_scores(q, bounds, table, n):
    """Upper bounds [H, n] of q.k over the first n blocks of a table row; q [Hq, D], bounds [NB, H, 2, D]."""
    H, D = bounds.shape[1], bounds.shape[3]
    b = bounds[table[:n]]  # [n, H, 2, D]
    qg = q.reshape(H, -1, D)
    with np.errstate(invalid="ignore"):
        both = qg[None, :, :, None, :] * b[:, :, None, :, :]  # [n, H, g, 2, D]
        return np.maximum(both[..., 0, :], both[..., 1, :]).sum(-1).max(-1).T


def select(q, bounds, tables, ctx, K, bs):
    """[B, H, K]: the first and the last block, then the best by (score, lower index), in ascending order."""
    B, H = q.shape[0], bounds.shape[1]
    out = np.full((B, H, K), -1, np.int32)
    for s in range(B):
        n = -(-int(ctx[s]) // bs)
        if n == 0:
            continue
        score = block_scores(q[s], bounds, tables[s], n)
        score = np.where(np.isnan(score), np.inf, score)
        for h in range(H):
            order = sorted(range(n), key=lambda b: (b not in (0, n - 1), -score[h, b], b))
            keep = sorted(order[:K])
            out[s, h, :len(keep)] = keep
    return out


def attend(q, keys, vals, tables, ctx, scale, bs, sel=None, v_scales=None):
    """Decode attention over the values keys / vals [NB, H, bs, D]: over all rows under a context, or over those of
    the logical blocks sel [B, H, K] (negative: none; a block listed twice counts twice).  Returns out and, for
    the tolerances, sum p |v| [B, Hq, D], the largest sum |q k| scale of a row [B, Hq], and, given the v_scales of
    an e4m3 pool, (max p v_scale) sum |code| [B, Hq, D] (0 without)."""
    B, Hq, D = q.shape
    H = keys.shape[1]
    g = Hq // H
    out, weight, zmag, unit = np.zeros((B, Hq, D)), np.zeros((B, Hq, D)), np.zeros((B, Hq)), np.zeros((B, Hq, D))
    for s in range(B):
        n = -(-int(ctx[s]) // bs)
        for h in range(H):
            js = range(n) if sel is None else [j for j in sel[s, h] if 0 <= j < n]
            k = [keys[tables[s, j], h, :min(ctx[s] - j * bs, bs)] for j in js]
            if not k:
                continue
            k = np.concatenate(k)
            v = np.concatenate([vals[tables[s, j], h, :min(ctx[s] - j * bs, bs)] for j in js])
            heads = slice(h * g, (h + 1) * g)
            z = q[s, heads] @ k.T * scale
            p = np.exp(z - z.max(1, keepdims=True))
            p /= p.sum(1, keepdims=True)
            out[s, heads] = p @ v
            weight[s, heads] = p @ np.abs(v)
            zmag[s, heads] = (np.abs(q[s, heads]) @ np.abs(k).T * abs(scale)).max(1)
            if v_scales is not None:
                rows = np.concatenate([np.full(min(ctx[s] - j * bs, bs), v_scales[tables[s, j], h], np.float64) for j in js])
                unit[s, heads] = (p * rows).max(1)[:, None] * (np.abs(v) / rows[:, None]).sum(0)
    return out, weight, zmag, unit


def assert_attention(got, ref, weight_step, what=""):
    """|got - out| within what the kernel may round:
    the result to bf16: 2^-8 of it;
    every weight to a 16-bit type, `weight_step` of it (bf16 2^-8, f16 2^-11, none in fp32): so much of sum p |v|;
    a score's sum of D <= 128 products in fp32, and the exponential's argument and value: they change a weight by a
    factor within 2 (128 + 4) 2^-24 sum |q k| scale + 2^-20, in the numerator and in the denominator;
    the sums over the rows in fp32 (at most 2^13 rows of a warp in these tests, and the merges): 2^-11;
    over an e4m3 pool, a weight times its block's V scale as f16 relative to a reference that is the
    largest product at most: below 2^-14 f16 is spaced 2^-24, so each of them is off by 2^-25 of the largest product
    at most, and that many codes' magnitudes are added up."""
    out, weight, zmag, unit = ref
    got = f64(got)
    dz = 2 * (2 * 132 * 2.0 ** -24 * zmag + 2.0 ** -20)[..., None]
    tol = 2.0 ** -8 * np.abs(out) + weight * (weight_step + dz + 2.0 ** -11) + 2.0 ** -25 * unit + 1e-30
    assert np.isfinite(got).all(), f"{what}: not finite"
    worst = (np.abs(got - out) / tol).max() if out.size else 0.0
    assert worst <= 1.0, f"{what}: {worst:.3f} of the tolerance"


class Batch:
    """Ragged sequences on one pool: tables, contexts and the appended tokens of a call."""

    def __init__(self, ctx, new, H, D, bs, seed, g=1, spread=1.0):
        r = np.random.default_rng(seed)
        self.bs, self.H, self.D, self.g = bs, H, D, g
        self.ctx = np.asarray(ctx, np.int32)
        self.new = np.asarray(new, np.int32)
        self.start = np.concatenate([[0], np.cumsum(self.new)]).astype(np.int32)
        need = [-(-c // bs) for c in ctx]
        self.NB = sum(need) + 3
        ids = r.permutation(self.NB).astype(np.int32)
        self.tables = np.full((len(ctx), max(need + [1]) + 1), -1, np.int32)
        at = 0
        for s, n in enumerate(need):
            self.tables[s, :n] = ids[at:at + n]
            at += n
        self.unused = ids[at:]
        T = int(self.start[-1])
        gen = torch.Generator().manual_seed(seed)
        mag = torch.exp(spread * torch.randn((T, H, 1), generator=gen))
        self.k = (torch.randn((T, H, D), generator=gen) * mag).to(torch.bfloat16)
        self.v = (torch.randn((T, H, D), generator=gen) * mag.flip(0)).to(torch.bfloat16)
        self.q = torch.randn((len(ctx), H * g, D), generator=gen).to(torch.bfloat16)
        self.scale = 1 / math.sqrt(D)
        # the pool: codes of an older life everywhere, scales as the write makes them
        self.kc = r.integers(0, 256, (self.NB, H, bs, D)).astype(np.uint8)
        self.vc = r.integers(0, 256, (self.NB, H, bs, D)).astype(np.uint8)
        for c in (self.kc, self.vc):
            c[(c & 0x7F) == 0x7F] = 0x5A  # no NaN
        self.ks = (2.0 ** np.round(spread * 2 * r.standard_normal((self.NB, H)) - 7)).astype(np.float32)
        self.vs = (2.0 ** np.round(spread * 2 * r.standard_normal((self.NB, H)) - 7)).astype(np.float32)

    def poison(self):
        """NaN codes in every row that no context covers, NaN scales for the blocks without one."""
        covered = np.zeros((self.NB, self.bs), bool)
        for s, c in enumerate(self.ctx):
            for j in range(-(-int(c) // self.bs)):
                covered[self.tables[s, j], :min(c - j * self.bs, self.bs)] = True
        for c in (self.kc, self.vc):
            c[np.broadcast_to(~covered[:, None, :, None], c.shape)] = 0x7F
        for x in (self.ks, self.vs):
            x[~covered.any(1)] = np.nan
        return self

    def bf16_pool(self):
        """The pool's values as bf16 (exact: four bits and a power of two); NaN stays NaN."""
        with np.errstate(invalid="ignore"):
            return [torch.from_numpy(values(c, s)).to(torch.bfloat16) for c, s in ((self.kc, self.ks), (self.vc, self.vs))]

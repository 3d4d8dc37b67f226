// block_cache.cuh -- per-block state of the cache, kept up to date as tokens
// arrive: the quantising write into an 8-bit (e4m3) pool with a scale for
// each (block, kv head), the copies of those scales, and the key bounds of
// every (block, kv head) that block selection scores.
//
// A call appends query_start[s+1] - query_start[s] tokens to sequence s, whose
// context_lens[s] counts them already: they are its last positions.  The work
// unit is one touched block of one head: the blocks from the first new
// token's to the context's last.
#pragma once

#include "ptx.cuh"

namespace pkv {

struct TouchParams {
    const int32_t *tables;  // [B][MBS]
    const int32_t *ctx;     // [B], new tokens included
    const int32_t *start;   // [B + 1]
    int B, MBS, bs, NB, H;
    int T;                  // rows of k and v that exist
    int max_new;            // host bound of the new tokens of a sequence
    int J;                  // touched blocks of max_new tokens at most
};

// Block i of those that sequence s touches.
struct TouchedBlock {
    int block;  // physical id
    int old;    // rows before the first new one
    int held;   // rows under the context
    int token;  // row of k / v that holds row `old`
};

// False: nothing to do (no such block, or a fault, which the unit with
// `report` records).  A sequence whose new tokens are negative in number,
// more than max_new or its context, outside [0, T] or past its table is left
// out whole.
__device__ __forceinline__ bool touched_block(const TouchParams &p, int s, int i, bool report, TouchedBlock *t) {
    const int a = __ldg(p.start + s), b = __ldg(p.start + s + 1), c = __ldg(p.ctx + s);
    const long long n = (long long)b - a;
    if (n == 0) return false;
    if (n < 0 || n > p.max_new || n > c || a < 0 || b > p.T || c > (long long)p.MBS * p.bs) {
        if (report && i == 0) raise_error(PKV_DEVERR_CONTEXT);
        return false;
    }
    const int p0 = c - (int)n;  // the first new token's position
    const int first = p0 / p.bs;
    // behind the context (told before a position is formed, which can pass 2^31 there)
    if ((uint32_t)i * (uint32_t)p.bs >= (uint32_t)(p0 - first * p.bs) + (uint32_t)n) return false;
    const int j = first + i, j0 = j * p.bs;
    const int blk = __ldg(p.tables + (size_t)s * p.MBS + j);
    if (blk < 0 || blk >= p.NB) {
        if (report) raise_error(PKV_DEVERR_BLOCK);
        return false;
    }
    t->block = blk;
    t->old = max(p0 - j0, 0);
    t->held = min(c - j0, p.bs);
    t->token = a + max(j0 - p0, 0);
    return true;
}

// A warp takes groups of rows, 16 bytes of bf16 a lane: 2 rows at a time at
// head dim 128, 4 at 64, and 16 rows in flight.  A team of W = min(bs / 16, 8)
// warps shares a unit, one group each up to blocks of 128 tokens.  A unit's
// chain of loads (query_start and context, table, rows) is 2 us long whatever it
// moves, so the warps of an SM set the rate: two or four blocks of 16 a warp
// measured 1.5 us slower than one (8 prompts of up to 2048 tokens, 11.8 against
// 10.2 us), for their registers halve the warps.
constexpr int kTouchRows = 16;
constexpr int kTouchMaxWarps = 8;
constexpr int kTouchTeams = 4;  // teams of one warp in a CTA

// ---------------------------------------------------- quantising write ----
// For one (block, head) of K or V:
//   a    = the largest finite |x| of the new rows
//   need = the least power of two s >= 2^-126 with a <= 448 s
//   s'   = need if no older row is held, else max(s, need)
//   new rows:   code  = e4m3(x / s')
//   all others: code' = e4m3(e4m3(code) s / s'), only when s' > s > 0
// A power of two makes both products exact in fp32 (so each element is rounded
// once, ties to even, saturating; fp32 underflow rounds to a zero code), and
// growing a scale exact for every code that stays a normal e4m3 number.  Another
// old scale that is large enough stays, and x is divided by it: the product with
// its reciprocal would be rounded twice, and miss ties (175 / 7 = 25).
struct WriteBlockParams {
    TouchParams t;
    const uint4 *k;  // [T][H][D] bf16 as 16-byte vectors
    const uint4 *v;
    uint2 *k_cache;  // [NB][H][bs][D] codes as 8-byte vectors
    uint2 *v_cache;
    float *k_scales;  // [NB][H]
    float *v_scales;
    uint32_t units;   // B * J * H * 2
    int W;            // warps of a team
};

// The least power of two >= 2^-126 with a <= 448 * 2^k (448 = 1.75 * 2^8).
__device__ __forceinline__ float pow2_scale(float a) {
    const uint32_t u = __float_as_uint(a);
    const int e = (int)(u >> 23) - 8 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
    return __uint_as_float((uint32_t)max(e, 1) << 23);
}

__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));  // a NaN loses against a number
    return r;
}

// 8 bf16 elements times `inv` as 8 codes.
__device__ __forceinline__ uint2 codes_from_bf16(const uint4 &x, float inv) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[2];
#pragma unroll
    for (int u = 0; u < 2; ++u)
        c[u] = e4m3x2_from_f32(bf16lo_to_f32(w[2 * u]) * inv, bf16hi_to_f32(w[2 * u]) * inv) |
               (e4m3x2_from_f32(bf16lo_to_f32(w[2 * u + 1]) * inv, bf16hi_to_f32(w[2 * u + 1]) * inv) << 16);
    return make_uint2(c[0], c[1]);
}

// Two e4m3 codes (the low half of `w`) as an f16 pair, exactly.
__device__ __forceinline__ uint32_t f16x2_from_e4m3x2(uint32_t w) {
    uint32_t r;
    asm("{\n\t.reg .b16 l;\n\tcvt.u16.u32 l, %1;\n\tcvt.rn.f16x2.e4m3x2 %0, l;\n\t}" : "=r"(r) : "r"(w));
    return r;
}

__device__ __forceinline__ float2 f32x2_from_f16x2(uint32_t h) {
    float2 r;
    asm("{\n\t.reg .b16 l, u;\n\tmov.b32 {l, u}, %2;\n\tcvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, u;\n\t}"
        : "=f"(r.x), "=f"(r.y) : "r"(h));
    return r;
}

__device__ __forceinline__ uint32_t rescale_codes(uint32_t w, float ratio) {
    const float2 a = f32x2_from_f16x2(f16x2_from_e4m3x2(w & 0xffffu));
    const float2 b = f32x2_from_f16x2(f16x2_from_e4m3x2(w >> 16));
    return e4m3x2_from_f32(a.x * ratio, a.y * ratio) | (e4m3x2_from_f32(b.x * ratio, b.y * ratio) << 16);
}

// 8 bf16 elements divided by `s` as 8 codes.  In line: as a function of its own it
// cost the other path more (32 prompts of up to 2048 tokens at head dim 64: 29.7
// us, 27.7 in line).
__device__ __forceinline__ uint2 codes_divided(const uint4 &x, float s) {
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
    uint32_t c[4];
#pragma unroll
    for (int u = 0; u < 4; ++u)
        c[u] = e4m3x2_from_f32(__fdiv_rn(bf16lo_to_f32(w[u]), s), __fdiv_rn(bf16hi_to_f32(w[u]), s));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

// PASSES: rows of a group / rows of a pass (fewer for short appends, whose
// blocks receive at most that many).
template <int D, int PASSES>
__global__ void __launch_bounds__(kTouchMaxWarps * 32) write_fp8_block_kernel(const WriteBlockParams p) {
    constexpr int VPR = D / 8;          // lanes of a row
    constexpr int RPP = 32 / VPR;       // rows of a pass
    constexpr int GROUP = PASSES * RPP;
    __shared__ float s_amax[kTouchMaxWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wt = p.W > 1 ? warp : 0;  // warp of the team; several teams share a CTA only when W is 1
    grid_dependency_wait();
    const uint32_t u = p.W > 1 ? blockIdx.x : blockIdx.x * kTouchTeams + warp;
    if (u >= p.units) return;
    const int kv = (int)(u & 1);
    const uint32_t r = (u >> 1) / (uint32_t)p.t.H;
    const int h = (int)((u >> 1) - r * p.t.H), s = (int)(r / (uint32_t)p.t.J), i = (int)(r - (uint32_t)s * p.t.J);
    TouchedBlock t;
    if (!touched_block(p.t, s, i, h == 0 && kv == 0 && wt == 0 && lane == 0, &t)) return;  // (the whole team)
    const size_t stride = (size_t)p.t.H * VPR;  // vectors between tokens
    const int sub = lane / VPR, c = lane % VPR;

    const int fresh = t.held - t.old;  // new rows
    const uint4 *x = (kv ? p.v : p.k) + ((size_t)t.token * p.t.H + h) * VPR;
    uint2 *cache = (kv ? p.v_cache : p.k_cache) + ((size_t)t.block * p.t.H + h) * p.t.bs * VPR;
    float *scale = (kv ? p.v_scales : p.k_scales) + (size_t)t.block * p.t.H + h;
    const float s_old = t.old > 0 ? *scale : 0.f;
    uint4 in[PASSES];
    auto load = [&](int grp) {  // group `grp` of the new rows
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int row = grp * GROUP + q * RPP + sub;
            in[q] = row < fresh ? __ldg(x + (size_t)row * stride + c) : make_uint4(0, 0, 0, 0);
        }
    };
    int loaded = -1;
    uint32_t m = 0;
    for (int grp = wt; grp * GROUP < fresh; grp += p.W) {
        load(grp);
        loaded = grp;
        uint32_t mg = 0;
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            mg = max_bf16x2(mg, in[q].x & 0x7fff7fffu);
            mg = max_bf16x2(mg, in[q].y & 0x7fff7fffu);
            mg = max_bf16x2(mg, in[q].z & 0x7fff7fffu);
            mg = max_bf16x2(mg, in[q].w & 0x7fff7fffu);
        }
        if ((mg & 0xffffu) >= 0x7f80u || (mg >> 16) >= 0x7f80u) {
            // infinities do not count: once more, element by element
            mg = 0;
#pragma unroll
            for (int q = 0; q < PASSES; ++q) {
                const uint32_t w[4] = {in[q].x, in[q].y, in[q].z, in[q].w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t lo = w[e] & 0x7fffu, hi = (w[e] >> 16) & 0x7fffu;
                    if (lo < 0x7f80u) mg = max(mg, lo);
                    if (hi < 0x7f80u) mg = max(mg, hi);
                }
            }
        }
        m = max_bf16x2(m, mg);
    }
    // magnitudes as integers keep their order
    m = max(m & 0xffffu, m >> 16);
    float amax = __uint_as_float(__reduce_max_sync(0xffffffffu, m) << 16);
    if (p.W > 1) {
        if (lane == 0) s_amax[wt] = amax;
        __syncthreads();
        for (int w = 0; w < p.W; ++w) amax = fmaxf(amax, s_amax[w]);
    }
    const float grown = fmaxf(s_old, pow2_scale(amax));
    const float inv = __frcp_rn(grown);  // exact for a power of two
    if ((__float_as_uint(grown) & 0x7fffffu) != 0) {  // no power of two
        for (int row = wt * RPP + sub; row < fresh; row += p.W * RPP)
            cache[(size_t)(t.old + row) * VPR + c] = codes_divided(__ldg(x + (size_t)row * stride + c), grown);
    } else for (int grp = wt; grp * GROUP < fresh; grp += p.W) {
        if (grp != loaded) load(grp);
        loaded = grp;
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            const int row = grp * GROUP + q * RPP + sub;
            if (row < fresh) cache[(size_t)(t.old + row) * VPR + c] = codes_from_bf16(in[q], inv);
        }
    }
    if (t.old > 0 && grown > s_old) {
        const float ratio = s_old * inv;
        for (int row = wt * RPP + sub; row < p.t.bs; row += p.W * RPP) {
            if (row >= t.old && row < t.held) continue;
            uint2 w = cache[(size_t)row * VPR + c];
            w.x = rescale_codes(w.x, ratio);
            w.y = rescale_codes(w.y, ratio);
            cache[(size_t)row * VPR + c] = w;
        }
    }
    if (p.W == 1) __syncwarp();  // every lane has read the old scale
    if (wt == 0 && lane == 0 && grown != s_old) *scale = grown;
}

// ------------------------------------------------------- scale copies ----
// Row src -> row dst of both scale arrays, for the block pairs of a
// copy-on-write.  Pairs by value (host list, validated there) or from the
// device list that the block manager leaves.
constexpr int kScalePairs = 256;

struct CopyScalesParams {
    float *k_scales;
    float *v_scales;
    int H, n;
    int2 pairs[kScalePairs];
};

__global__ void __launch_bounds__(256) copy_scales_kernel(const __grid_constant__ CopyScalesParams p) {
    const int i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= p.n * p.H) return;
    const int e = i / p.H, h = i - e * p.H;
    const size_t src = (size_t)p.pairs[e].x * p.H + h, dst = (size_t)p.pairs[e].y * p.H + h;
    p.k_scales[dst] = p.k_scales[src];
    p.v_scales[dst] = p.v_scales[src];
}

__global__ void __launch_bounds__(256) copy_scales_dev_kernel(float *k_scales, float *v_scales, const int32_t *pairs,
                                                              const int32_t *num_pairs, int max_pairs, int NB, int H) {
    const long long n = (long long)max(0, min(__ldg(num_pairs), max_pairs)) * H;
    for (long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x; i < n; i += (long long)gridDim.x * blockDim.x) {
        const int e = (int)(i / H), h = (int)(i - (long long)e * H);
        const int src = __ldg(pairs + 2 * e), dst = __ldg(pairs + 2 * e + 1);
        if (src < 0 || src >= NB || dst < 0 || dst >= NB) {
            if (h == 0) raise_error(PKV_DEVERR_BLOCK);
            continue;
        }
        k_scales[(size_t)dst * H + h] = k_scales[(size_t)src * H + h];
        v_scales[(size_t)dst * H + h] = v_scales[(size_t)src * H + h];
    }
}

// ---------------------------------------------------------- key bounds ----
// lo[d] = min, hi[d] = max over the held rows of a (block, head), NaN if one
// of them is NaN; [NB][H][2][D] bf16, lo first.  Every held row is read, not
// only the new ones: a block that was copied or whose scale has grown needs no
// other care.  Over an 8-bit pool the least and largest CODE are found and
// scaled once (the scale is positive).  The product is exact in bf16 where the scale
// is a power of two and nothing leaves bf16's normal range; otherwise the least is
// rounded down and the largest up, so that every key lies between them.
// Sign-magnitude numbers order alike whatever their fields, so a code is
// compared as the upper byte of a bf16: what lies in the lower one decides
// between equal codes only, and 0x7f and 0xff, the NaN codes, stay at an end or
// become a bf16 NaN, whose upper byte is 0x7f.  8 prompts of 2048 to 8192
// tokens, 8 heads: 9.1 us, 9.7 with codes converted to f16 first, 10.5 as integers
// (which take a third extreme).
struct KeyBoundsParams {
    TouchParams t;
    const void *k_cache;   // [NB][H][bs][D] bf16, or e4m3 codes
    const float *k_scales;  // [NB][H], e4m3 only
    uint4 *bounds;
    uint32_t units;  // B * J * H
    int W;
};

__device__ __forceinline__ void min_max_bf16x2(uint32_t &lo, uint32_t &hi, uint32_t l, uint32_t h) {
    asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(lo) : "r"(l));
    asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(hi) : "r"(h));
}

// code * s as the next bf16 below it, or above.
__device__ __forceinline__ float scaled_down(float code, float s) {
    const uint32_t u = __float_as_uint(__fmul_rd(code, s));
    return __uint_as_float(((u & 0xffffu) != 0 && (u >> 31) ? u + 0x10000u : u) & 0xffff0000u);
}
__device__ __forceinline__ float scaled_up(float code, float s) { return -scaled_down(-code, s); }

// The upper bytes of `even` and `odd`, codes of columns 0, 2 and 1, 3, as values.
__device__ __forceinline__ void values_of_codes(uint32_t even, uint32_t odd, float (&x)[4]) {
    const float2 a = f32x2_from_f16x2(f16x2_from_e4m3x2(__byte_perm(even, odd, 0x4451)));
    const float2 b = f32x2_from_f16x2(f16x2_from_e4m3x2(__byte_perm(even, odd, 0x4473)));
    x[0] = a.x; x[1] = a.y; x[2] = b.x; x[3] = b.y;
}

template <int D, bool KV8>
__global__ void __launch_bounds__(kTouchMaxWarps * 32) key_bounds_kernel(const KeyBoundsParams p) {
    constexpr int VPR = D / 8, RPP = 32 / VPR, PASSES = kTouchRows / RPP;
    constexpr uint32_t kPosInf = 0x7f807f80u, kNegInf = 0xff80ff80u;
    using Vec = typename std::conditional<KV8, uint2, uint4>::type;
    __shared__ uint4 s_lo[kTouchMaxWarps][VPR], s_hi[kTouchMaxWarps][VPR];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int wt = p.W > 1 ? warp : 0;
    grid_dependency_wait();
    const uint32_t u = p.W > 1 ? blockIdx.x : blockIdx.x * kTouchTeams + warp;
    if (u >= p.units) return;
    const uint32_t r = u / (uint32_t)p.t.H;
    const int h = (int)(u - r * p.t.H), s = (int)(r / (uint32_t)p.t.J), i = (int)(r - (uint32_t)s * p.t.J);
    TouchedBlock t;
    if (!touched_block(p.t, s, i, h == 0 && wt == 0 && lane == 0, &t)) return;  // (the whole team)
    const int sub = lane / VPR, c = lane % VPR;
    const size_t head = (size_t)t.block * p.t.H + h;
    const Vec *x = static_cast<const Vec *>(p.k_cache) + head * p.t.bs * VPR;
    const float ks = KV8 ? __ldg(p.k_scales + head) : 1.f;
    uint32_t lo[4] = {kPosInf, kPosInf, kPosInf, kPosInf}, hi[4] = {kNegInf, kNegInf, kNegInf, kNegInf};
    for (int grp = wt; grp * kTouchRows < t.held; grp += p.W) {
        Vec in[PASSES];
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            // a row past the held ones repeats the last held row
            const int row = min(grp * kTouchRows + q * RPP + sub, t.held - 1);
            in[q] = __ldg(x + (size_t)row * VPR + c);
        }
#pragma unroll
        for (int q = 0; q < PASSES; ++q) {
            uint32_t w[4];
            if constexpr (KV8) {
                w[0] = in[q].x << 8; w[1] = in[q].x; w[2] = in[q].y << 8; w[3] = in[q].y;
            } else {
                w[0] = in[q].x; w[1] = in[q].y; w[2] = in[q].z; w[3] = in[q].w;
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) min_max_bf16x2(lo[e], hi[e], w[e], w[e]);
        }
    }
#pragma unroll
    for (int o = VPR; o < 32; o <<= 1) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
            const uint32_t l = __shfl_xor_sync(0xffffffffu, lo[e], o), g = __shfl_xor_sync(0xffffffffu, hi[e], o);
            min_max_bf16x2(lo[e], hi[e], l, g);
        }
    }
    if (p.W > 1) {
        if (lane < VPR) {
            s_lo[wt][c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            s_hi[wt][c] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
        }
        __syncthreads();
        if (wt != 0) return;
        for (int w = 1; w < p.W; ++w) {
            const uint4 l = s_lo[w][c], g = s_hi[w][c];
            min_max_bf16x2(lo[0], hi[0], l.x, g.x);
            min_max_bf16x2(lo[1], hi[1], l.y, g.y);
            min_max_bf16x2(lo[2], hi[2], l.z, g.z);
            min_max_bf16x2(lo[3], hi[3], l.w, g.w);
        }
    }
    if constexpr (KV8) {
        // a code is 2^-9 at least and 448 at most, bf16 2^-133 and below 2^128
        const uint32_t sb = __float_as_uint(ks), se = sb >> 23;
        const bool exact = (sb & 0x7fffffu) == 0 && se >= 127 - 124 && se <= 127 + 119;
        auto scale = [&](auto &&down, auto &&up) {
#pragma unroll
            for (int v = 0; v < 4; v += 2) {  // word v / 2 of the row's codes
                float l[4], g[4];
                values_of_codes(lo[v], lo[v + 1], l);
                values_of_codes(hi[v], hi[v + 1], g);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const bool nan = l[e] != l[e] || g[e] != g[e];
                    l[e] = nan ? __int_as_float(0x7fffffff) : down(l[e], ks);
                    g[e] = nan ? __int_as_float(0x7fffffff) : up(g[e], ks);
                }
                lo[v] = pack_bf16x2(l[0], l[1]);
                lo[v + 1] = pack_bf16x2(l[2], l[3]);
                hi[v] = pack_bf16x2(g[0], g[1]);
                hi[v + 1] = pack_bf16x2(g[2], g[3]);
            }
        };
        auto product = [](float x, float y) { return x * y; };
        if (exact) scale(product, product);
        else scale(scaled_down, scaled_up);
    }
    if (lane < VPR) {
        uint4 *out = p.bounds + head * 2 * VPR;
        out[c] = make_uint4(lo[0], lo[1], lo[2], lo[3]);
        out[VPR + c] = make_uint4(hi[0], hi[1], hi[2], hi[3]);
    }
}

}  // namespace pkv

// block_select.cuh -- the blocks that a query's attention keeps.
//
// For sequence s and kv head h with the g query heads q_j and the key bounds
// lo_b, hi_b of every block b under the context,
//   score(b) = max_j sum_d max(q_jd lo_bd, q_jd hi_bd)
// bounds q_j.k from above for every key k of the block.  The first and the
// last block are kept, and the best others up to K in all, by (score, lower
// index); a NaN score counts as +infinity.
//
// max(q lo, q hi) = max(q, 0) hi + min(q, 0) lo, so the scores of 8 blocks are
// one product of [g heads][2 D] and [2 D][8 blocks] on the tensor cores.  bf16
// products are exact in fp32 and their sums are not, so these scores only
// narrow the choice: with an error of at most e, a block whose score is more
// than 2 e above the K-th largest is in, one more than 2 e below is out, and
// the few between them are scored again in fp64.
//
// Two kernels.  Scoring is bound by the bounds' bytes (512 for a block and
// head at head dim 128, against 8 D g operations): all tiles of 8 blocks of all
// sequences and groups of heads form one line, of which every group of warps of
// the grid takes an equal stretch, a head a warp (the heads of a block lie side
// by side in memory), through a ring of bulk copies of each warp.  Selection is a CTA for each (s, h)
// over the scores that the first kernel left in the workspace (in L2).
#pragma once

#include "ptx.cuh"

namespace pkv {

// Bound of a score's fp32 error relative to the sum of its terms' magnitudes:
// at most 8 products of k = 16 follow one another in a chain and two chains are
// added; each product adds 17 numbers and rounds the sum, and each of those
// steps loses at most 2^-23 of the largest magnitude: (8 * 18 + 1) 2^-23 =
// 1.73e-5.  The terms min(q, 0) lo and max(q, 0) hi are negative only where lo
// > 0 or hi < 0, so the magnitudes add up to the score and twice the negative
// terms, at most 2 sum |q_d| w with the largest lo or -hi above zero as w.
constexpr float kSelError = 2e-5f;

struct SelectParams {
    const __nv_bfloat16 *q;       // [B][Hq][D]
    const __nv_bfloat16 *bounds;  // [NB][H][2][D]
    const int32_t *block_tables;  // [B][MBS]
    const int32_t *context_lens;  // [B]
    int32_t *selected;            // [B][H][K]
    float2 *scores;               // workspace: [B][H][stride], a score and the bound of its error
    uint64_t *keys;               // workspace: [B][H][stride], fp64 scores when many are undecided
    int B, H, g, MBS, bs, NB, K, max_ctx;
    int stride;  // blocks of a (s, h) at most, rounded up to 32
};

__device__ __forceinline__ int select_blocks_of(const SelectParams &p, int s, bool report) {
    int n = __ldg(p.context_lens + s);
    const int cap = (int)min((long long)p.MBS * p.bs, (long long)p.max_ctx);
    if (n < 0 || n > cap) {
        if (report) raise_error(PKV_DEVERR_CONTEXT);
        n = n < 0 ? 0 : cap;
    }
    return (int)(((long long)n + p.bs - 1) / p.bs);
}

// ----------------------------------------------------------- scoring ----
constexpr int kScoreWarps = 4;
constexpr int kScoreThreads = kScoreWarps * 32;
constexpr int kScoreRing = 3;      // tiles of a warp in flight
constexpr int kScoreMinTiles = 2;  // of a warp, while there are fewer than fill the grid
constexpr uint64_t kScoreWaitNs = 2000000000ull;

template <int D>
struct ScoreSmem {
    static constexpr int kBytes = 4 * D;          // a block's bounds
    static constexpr int kStride = kBytes + 64;   // two blocks' rows of 64 bytes lie in different halves of the banks
    static constexpr int kWarp = kScoreRing * 8 * kStride;
    static constexpr int oScan = kScoreWarps * kWarp;              // long long [threads]
    static constexpr int oSum = oScan + kScoreThreads * 8;         // long long [warps]
    static constexpr int oBars = oSum + kScoreWarps * 8;
    static constexpr int kAlloc = oBars + kScoreWarps * kScoreRing * 8;
};

__device__ __forceinline__ float max_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

template <int D, bool TALL>  // TALL: more than 8 query heads
__global__ void __launch_bounds__(kScoreThreads, 3) score_blocks_kernel(const SelectParams p) {
    using L = ScoreSmem<D>;
    constexpr int VE = 2 * D;    // elements of a block's bounds
    constexpr int CH = VE / 32;  // 16-byte loads of a lane per block
    constexpr int R = kScoreRing;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    uint8_t *ring = smem_raw + warp * L::kWarp;
    long long *scan = reinterpret_cast<long long *>(smem_raw + L::oScan);
    long long *warp_sum = reinterpret_cast<long long *>(smem_raw + L::oSum);
    uint64_t *bars = reinterpret_cast<uint64_t *>(smem_raw + L::oBars) + warp * R;
    if (lane == 0) {
        for (int t = 0; t < R; ++t) mbar_init(&bars[t], 1);
        fence_mbar_init();
    }
    grid_dependency_wait();
    // The line: sequences with something to choose, their groups of `heads`
    // heads, tiles of 8 blocks.
    const int heads = p.H % 4 == 0 ? 4 : p.H % 2 == 0 ? 2 : 1, hgroups = p.H / heads;
    static_assert(kScoreWarps == 4, "a group of 4, 2 or 1 heads");
    auto tiles_of = [&](int s, int &n) {
        n = select_blocks_of(p, s, false);
        return n > p.K ? (n + 7) / 8 : 0;
    };
    const int per = (p.B + kScoreThreads - 1) / kScoreThreads;
    long long sum = 0, total = 0, before = 0;
    for (int s = tid * per, n; s < min(p.B, (tid + 1) * per); ++s) sum += tiles_of(s, n);
    sum *= hgroups;
    long long incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) warp_sum[warp] = incl;
    __syncthreads();
    for (int w = 0; w < kScoreWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    scan[tid] = before + incl - sum;  // the tiles before this thread's sequences
    __syncthreads();
    const long long parts = max(1ll, min((long long)gridDim.x * (kScoreWarps / heads), total / kScoreMinTiles));
    const long long me = (long long)blockIdx.x * (kScoreWarps / heads) + warp / heads;
    if (me >= parts || total == 0) return;
    const long long a = (total / parts) * me + (total % parts) * me / parts;
    const int len = (int)((total / parts) * (me + 1) + (total % parts) * (me + 1) / parts - a);
    if (len == 0) return;

    // Lane l looks up block l % 8 of tile 4 G + l / 8 of the stretch.
    int cs, nt, n;
    long long base;
    {
        int lo = 0, hi = kScoreThreads - 1;  // the last thread whose sequences begin at or before a
        while (lo < hi) {
            const int mid = (lo + hi + 1) >> 1;
            if (scan[mid] <= a) lo = mid; else hi = mid - 1;
        }
        cs = min(lo * per, p.B - 1);
        base = scan[lo];
        nt = tiles_of(cs, n);
    }
    struct Look {
        int unit, b, row;  // (s, h), logical block, row of its bounds (-1: none)
    };
    auto look_up = [&](int G) -> Look {
        const int k = 4 * G + (lane >> 3);
        Look r = {-1, 0, -1};
        if (k >= len) return r;
        const long long x = a + k;
        while (x >= base + (long long)nt * hgroups) {
            base += (long long)nt * hgroups;
            nt = tiles_of(++cs, n);
        }
        const uint32_t off = (uint32_t)(x - base);  // below H * blocks / 8, and that below 2^31
        const int hg = (int)(off / (uint32_t)nt), h = hg * heads + warp % heads;
        r.unit = cs * p.H + h;
        r.b = (int)(off - (uint32_t)hg * nt) * 8 + (lane & 7);
        if (r.b < n) {
            const int id = __ldg(p.block_tables + (size_t)cs * p.MBS + r.b);
            if (id >= 0 && id < p.NB) r.row = id * p.H + h;
            else if (h == 0) raise_error(PKV_DEVERR_BLOCK);
        }
        return r;
    };
    // Copies tile k, which the lanes l / 8 = k % 4 of `t` know.
    auto issue = [&](int k, const Look &t) {
        const bool mine = (lane >> 3) == (k & 3) && t.row >= 0;
        const uint32_t who = __ballot_sync(0xffffffffu, mine);
        const int slot = k % R;
        if (lane == 0) mbar_arrive_expect_tx(&bars[slot], __popc(who) * L::kBytes);
        __syncwarp();
        if (mine)
            bulk_load(ring + (slot * 8 + (lane & 7)) * L::kStride, p.bounds + (size_t)t.row * VE, L::kBytes, &bars[slot]);
    };
    Look cur = look_up(0), next = look_up(1);
    for (int k = 0; k < min(R, len); ++k) issue(k, cur);

    // A fragments of the heads' min(q, 0) and max(q, 0): lane (r = lane / 4,
    // j = lane % 4) holds rows r and r + 8.  Chunk i of a block's bounds is its
    // elements 32 i .. 32 i + 31; lane j reads 8 of them, 32 i + 8 j .. + 7,
    // which are the operands of two k-steps (the order of k is free).  The
    // first half of the chunks are least elements, the second largest ones.
    uint32_t a0[CH][4], a1[TALL ? CH : 1][4];
    float qsum = 0.f;  // the largest sum |q_jd| of a head
    auto load_q = [&](int unit) {
        auto row = [&](int head, uint32_t (&f)[CH][4]) {
            const __nv_bfloat16 *q = p.q + ((size_t)unit * p.g + head) * D + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                const uint4 v = head < p.g ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * i)) : make_uint4(0, 0, 0, 0);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t neg = (w[u] & 0x8000u ? 0xffffu : 0u) | (w[u] & 0x80000000u ? 0xffff0000u : 0u);
                    f[i][u] = w[u] & neg;
                    f[i + CH / 2][u] = w[u] & ~neg;
                }
            }
        };
        row(lane >> 2, a0);
        if constexpr (TALL) row((lane >> 2) + 8, a1);
        float s0 = 0.f, s1 = 0.f;
#pragma unroll
        for (int i = 0; i < CH; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                s0 += fabsf(bf16lo_to_f32(a0[i][u])) + fabsf(bf16hi_to_f32(a0[i][u]));
                if constexpr (TALL) s1 += fabsf(bf16lo_to_f32(a1[i][u])) + fabsf(bf16hi_to_f32(a1[i][u]));
            }
        s0 += __shfl_xor_sync(0xffffffffu, s0, 1);
        s0 += __shfl_xor_sync(0xffffffffu, s0, 2);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 1);
        s1 += __shfl_xor_sync(0xffffffffu, s1, 2);
        qsum = warp_max_f32(fmaxf(s0, s1));
    };
    const float inf = __int_as_float(0x7f800000);
    int unit = -1;
    for (int k = 0; k < len; ++k) {
        const int src_lane = 8 * (k & 3);
        const int u = __shfl_sync(0xffffffffu, cur.unit, src_lane), b0 = __shfl_sync(0xffffffffu, cur.b, src_lane);
        if (u != unit) {
            unit = u;
            load_q(unit);
        }
        const int slot = k % R;
        bool ok = mbar_wait_bounded(&bars[slot], (k / R) & 1, kScoreWaitNs);
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) {  // copies in flight have to land before the warp ends
            for (int t = k + 1; t < min(len, k + R); ++t) mbar_wait_bounded(&bars[t % R], (t / R) & 1, kScoreWaitNs);
            return;
        }
        // (a block without a row leaves old bytes here, and garbage in its own column only)
        const bool good = __shfl_sync(0xffffffffu, cur.row, src_lane + (lane >> 2)) >= 0;
        const uint32_t src = smem_u32(ring) + (slot * 8 + (lane >> 2)) * L::kStride + 16 * (lane & 3);
        float d[2][4];
        uint32_t w_lo = 0, w_hi = 0;  // the largest least element above 0, the smallest largest one below
#pragma unroll
        for (int c = 0; c < 4; ++c) d[0][c] = d[1][c] = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            uint4 x;
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x.x), "=r"(x.y), "=r"(x.z), "=r"(x.w)
                         : "r"(src + 64 * c));
            float(&e)[4] = d[c & 1];
            const uint32_t z0 = TALL ? a1[TALL ? c : 0][0] : 0u, z1 = TALL ? a1[TALL ? c : 0][1] : 0u;
            const uint32_t z2 = TALL ? a1[TALL ? c : 0][2] : 0u, z3 = TALL ? a1[TALL ? c : 0][3] : 0u;
            mma_bf16_16816(e[0], e[1], e[2], e[3], a0[c][0], z0, a0[c][1], z1, x.x, x.y);
            mma_bf16_16816(e[0], e[1], e[2], e[3], a0[c][2], z2, a0[c][3], z3, x.z, x.w);
            const uint32_t y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int u = 0; u < 4; ++u) {
                if (c < CH / 2) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w_lo) : "r"(y[u]));
                else asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(w_hi) : "r"(y[u]));
            }
        }
        __syncwarp();
        if (k + R < len) issue(k + R, ((k + R) >> 2) == (k >> 2) ? cur : next);  // the slot is read
        // w of the tile, as bits: a NaN is above every number
        w_hi &= 0x7fff7fffu;
        uint32_t wb = max(max(w_lo & 0xffffu, w_lo >> 16), max(w_hi & 0xffffu, w_hi >> 16));
        wb = __reduce_max_sync(0xffffffffu, good ? wb : 0u);
        // rows r and r + 8 of columns 2 j and 2 j + 1: the max over the heads,
        // NaN if one is
        const int r = lane >> 2;
        float s0 = -inf, s1 = -inf;
        if (r < p.g) {
            s0 = d[0][0] + d[1][0];
            s1 = d[0][1] + d[1][1];
        }
        if (TALL && r + 8 < p.g) {
            s0 = max_nan(s0, d[0][2] + d[1][2]);
            s1 = max_nan(s1, d[0][3] + d[1][3]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            s0 = max_nan(s0, __shfl_xor_sync(0xffffffffu, s0, o));
            s1 = max_nan(s1, __shfl_xor_sync(0xffffffffu, s1, o));
        }
        // Room for products below fp32's normal range.  Where a sum of
        // magnitudes is not finite, or so large that the sums may not be,
        // nothing is known of the score.
        const float neg = 2.f * qsum * __uint_as_float(wb << 16);
        float e0 = fmaxf(s0, 0.f) + neg, e1 = fmaxf(s1, 0.f) + neg;
        e0 = e0 < 1e37f && s0 == s0 ? fmaf(e0, kSelError, 1e-33f) : inf;
        e1 = e1 < 1e37f && s1 == s1 ? fmaf(e1, kSelError, 1e-33f) : inf;
        const uint32_t bad = __ballot_sync(0xffffffffu, !good);  // of block c: bit 4 c
        if (lane < 4)
            *reinterpret_cast<float4 *>(p.scores + (size_t)unit * p.stride + b0 + 2 * lane) =
                make_float4((bad >> (8 * lane)) & 1u ? -inf : s0, (bad >> (8 * lane)) & 1u ? 0.f : e0,
                            (bad >> (8 * lane + 4)) & 1u ? -inf : s1, (bad >> (8 * lane + 4)) & 1u ? 0.f : e1);
        if ((k & 3) == 3) {
            cur = next;
            next = look_up((k >> 2) + 2);
        }
    }
    grid_launch_dependents();
}

// ---------------------------------------------------------- selection ----
// A CTA of T threads for each (s, h).  Up to PER scores a thread stay in
// registers; PER = 0 reads them again (from L2) in each pass.  The search for
// the K-th score counts keys in 2048 equal bins between the least and the
// largest (scores of one query lie close together: bins by leading bits would
// send them all to a few counters), and again within a bin that holds more
// keys than there are warps to score them again, until it is as narrow as the
// scores' error.
constexpr int kSelBins = 2048;
constexpr int kSelPairMax = 512;  // undecided blocks up to which each is compared with each

template <int T>
struct SelectSmem {
    uint32_t hist[kSelBins];
    uint64_t key[kSelPairMax];  // undecided blocks, while they are few
    int idx[kSelPairMax];
    uint32_t scan[T / 32], lo[T / 32], hi[T / 32];
    float emax[T / 32];
    uint32_t found[3];
    uint32_t undecided;
};

// Order-preserving integers; -0 as +0, NaN as +infinity.
__device__ __forceinline__ uint32_t order_key(float x) {
    if (x != x) x = __int_as_float(0x7f800000);
    const uint32_t u = __float_as_uint(x + 0.f);
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float order_value(uint32_t k) {
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ uint64_t order_key(double x) {
    if (x != x) x = __longlong_as_double(0x7ff0000000000000ll);
    const uint64_t u = (uint64_t)__double_as_longlong(x + 0.0);
    return (u >> 63) ? ~u : u | 0x8000000000000000ull;
}

// Exclusive prefix sum of a value of each thread, and the total (all threads).
template <int T>
__device__ __forceinline__ uint32_t block_scan(SelectSmem<T> *sm, uint32_t x, uint32_t &total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    uint32_t incl = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    __syncthreads();  // scan[] is free
    if (lane == 31) sm->scan[warp] = incl;
    __syncthreads();
    uint32_t w = lane < T / 32 ? sm->scan[lane] : 0;
#pragma unroll
    for (int o = 1; o < T / 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    total = __shfl_sync(0xffffffffu, w, T / 32 - 1);
    const uint32_t before = __shfl_sync(0xffffffffu, w, max(warp - 1, 0));
    return incl - x + (warp > 0 ? before : 0);
}

// The bin of the histogram that holds the m-th largest key (m >= 1, at most
// the number of keys), the number of keys in the bins above it, and in it.
template <int BINS, int T>
__device__ __forceinline__ void find_bin(SelectSmem<T> *sm, uint32_t m, uint32_t &bin, uint32_t &above, uint32_t &inside) {
    constexpr int PER = BINS >= T ? BINS / T : 1;  // bins of a thread, from the top
    const int b0 = BINS - 1 - (int)threadIdx.x * PER;
    uint32_t sum = 0, total;
    __syncthreads();  // the histogram is complete
#pragma unroll
    for (int i = 0; i < PER; ++i) sum += b0 - i >= 0 ? sm->hist[b0 - i] : 0;
    uint32_t a = block_scan<T>(sm, sum, total);
    if (a < m && a + sum >= m) {
        for (int i = 0; i < PER; ++i) {
            const uint32_t c = sm->hist[b0 - i];
            if (a + c >= m) {
                sm->found[0] = (uint32_t)(b0 - i);
                sm->found[1] = a;
                sm->found[2] = c;
                break;
            }
            a += c;
        }
    }
    __syncthreads();
    bin = sm->found[0];
    above = sm->found[1];
    inside = sm->found[2];
}

// A block's score in fp64, as an ordered key.  Eight lanes take a head, each D /
// 8 of its elements; all lanes return the key.
template <int D>
__device__ __forceinline__ uint64_t exact_key(const SelectParams &p, const __nv_bfloat16 *q, int blk, int h) {
    constexpr int E = D / 8;
    const double inf = __longlong_as_double(0x7ff0000000000000ll);
    if (blk < 0 || blk >= p.NB) return order_key(-inf);
    const int lane = threadIdx.x & 31, d0 = (lane & 7) * E;
    auto load = [&](const __nv_bfloat16 *src, float (&x)[E]) {
#pragma unroll
        for (int i = 0; i < E; i += 8) {
            const uint4 v = __ldg(reinterpret_cast<const uint4 *>(src + d0 + i));
            const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
            for (int c = 0; c < 4; ++c) {
                x[i + 2 * c] = bf16lo_to_f32(w[c]);
                x[i + 2 * c + 1] = bf16hi_to_f32(w[c]);
            }
        }
    };
    const __nv_bfloat16 *b = p.bounds + ((size_t)blk * p.H + h) * 2 * D;
    float lo[E], hi[E];
    load(b, lo);
    load(b + D, hi);
    double best = -inf;
    bool nan = false;
    for (int j0 = 0; j0 < p.g; j0 += 4) {
        const int j = j0 + (lane >> 3);
        double sum[2] = {0.0, 0.0};
        if (j < p.g) {
            float x[E];
            load(q + (size_t)j * D, x);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const double y = (double)x[i] * (double)lo[i], z = (double)x[i] * (double)hi[i];
                sum[i & 1] += (y != y || z != z) ? y + z : (y > z ? y : z);
            }
        }
        double t = sum[0] + sum[1];
#pragma unroll
        for (int o = 4; o >= 1; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (j < p.g) {
            nan |= t != t;
            best = t > best ? t : best;
        }
    }
#pragma unroll
    for (int o = 8; o < 32; o <<= 1) {
        const double t = __shfl_xor_sync(0xffffffffu, best, o);
        best = t > best ? t : best;
    }
    return order_key(__any_sync(0xffffffffu, nan) ? inf : best);
}

template <int D, int T, int PER>
__global__ void __launch_bounds__(T) select_blocks_kernel(const SelectParams p) {
    constexpr int WARPS = T / 32;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    SelectSmem<T> *sm = reinterpret_cast<SelectSmem<T> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = blockIdx.x;
    const int s = (int)(unit / p.H), h = (int)(unit % p.H);
    for (int i = tid; i < kSelBins; i += T) sm->hist[i] = 0;
    if (tid == 0) sm->undecided = 0;
    grid_dependency_wait();
    const int n = select_blocks_of(p, s, h == 0 && tid == 0);
    int32_t *out = p.selected + unit * p.K;
    if (n <= p.K) {
        for (int i = tid; i < p.K; i += T) out[i] = i < n ? i : -1;
        return;
    }
    // a bit for each block: kept, and undecided
    const int words = (n + 31) / 32;
    uint32_t *kept = reinterpret_cast<uint32_t *>(smem_raw + sizeof(SelectSmem<T>)), *open = kept + words;
    const float2 *score = p.scores + unit * p.stride;
    const int32_t *table = p.block_tables + (size_t)s * p.MBS;
    const float inf = __int_as_float(0x7f800000);
    // Thread t's scores are blocks t, t + T, ...
    float a[PER > 0 ? PER : 1], e = 0.f;  // e: the largest error bound
    if constexpr (PER > 0) {
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            const float2 x = tid + i * T < n ? score[tid + i * T] : make_float2(0.f, 0.f);
            a[i] = x.x;
            e = fmaxf(e, x.y);
        }
    } else {
#pragma unroll 4
        for (int i = tid; i < n; i += T) e = fmaxf(e, score[i].y);
    }
    auto each = [&](auto &&f) {  // f(block, score), all threads of a warp together
        if constexpr (PER > 0) {
#pragma unroll
            for (int i = 0; i < PER; ++i)
                if (warp * 32 + i * T < n) f(tid + i * T, a[i]);
        } else {
#pragma unroll 4
            for (int i = tid; i - lane < n; i += T) f(i, i < n ? score[i].x : 0.f);
        }
    };
    auto ranked = [&](int i) { return i > 0 && i < n - 1; };
    uint32_t lo = 0xffffffffu, hi = 0;
    each([&](int i, float x) {
        if (ranked(i)) {
            const uint32_t k = order_key(x);
            lo = min(lo, k);
            hi = max(hi, k);
        }
    });
    e = warp_max_f32(e);
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (lane == 0) { sm->emax[warp] = e; sm->lo[warp] = lo; sm->hi[warp] = hi; }
    __syncthreads();
    for (int w = 0; w < WARPS; ++w) {
        e = fmaxf(e, sm->emax[w]);
        lo = min(lo, sm->lo[w]);
        hi = max(hi, sm->hi[w]);
    }

    // The K-th largest of the blocks between the first and the last lies in
    // t_lo .. t_hi.
    const uint32_t want = (uint32_t)(p.K - 2);
    float t_lo = -inf, t_hi = inf;
    if (want > 0 && e < inf) {
        uint32_t left = want, base = lo, width = hi - lo;  // the keys base .. base + width
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = max(0, 32 - __clz(width) - 11);
            each([&](int i, float x) {
                const uint32_t k = order_key(x) - base;
                if (ranked(i) && k <= width) atomicAdd(&sm->hist[k >> shift], 1u);
            });
            uint32_t bin, above, inside;
            find_bin<kSelBins, T>(sm, left, bin, above, inside);
            left -= above;
            base += bin << shift;
            width = min(width - (bin << shift), (1u << shift) - 1);
            t_lo = order_value(base);
            t_hi = order_value(base + width);
            if (inside <= WARPS || t_hi - t_lo <= e || width == 0) break;
            if (pass < 2) {
                for (int i = tid; i < kSelBins; i += T) sm->hist[i] = 0;
                __syncthreads();
            }
        }
    }
    // In, out or undecided.  With an unbounded error every block is undecided.
    const float in_above = t_hi + 2.f * e, out_below = t_lo - 2.f * e;
    uint32_t n_in = 0;
    each([&](int i, float x) {
        const bool in = i < n && (!ranked(i) || (want > 0 && x > in_above));
        const bool maybe = i < n && !in && want > 0 && !(x < out_below);
        const uint32_t mi = __ballot_sync(0xffffffffu, in), mu = __ballot_sync(0xffffffffu, maybe);
        n_in += __popc(mi);
        if (lane == 0) {
            kept[i >> 5] = mi;
            open[i >> 5] = mu;
        }
        if (mu != 0) {
            uint32_t at = 0;
            if (lane == 0) at = atomicAdd(&sm->undecided, __popc(mu));
            at = __shfl_sync(0xffffffffu, at, 0) + __popc(mu & ((1u << lane) - 1));
            if (maybe && at < (uint32_t)kSelPairMax) sm->idx[at] = i;
        }
    });
    uint32_t all_in;
    block_scan<T>(sm, lane == 0 ? n_in : 0, all_in);
    const uint32_t left = p.K - all_in;  // how many of the undecided are kept
    const uint32_t und = sm->undecided;
    const __nv_bfloat16 *q = p.q + unit * p.g * D;
    if (und <= (uint32_t)kSelPairMax) {
        // few: each against each, one is kept if fewer than `left` are ahead
        for (uint32_t u = warp; u < und; u += WARPS) {
            const uint64_t k = exact_key<D>(p, q, __ldg(table + sm->idx[u]), h);
            if (lane == 0) sm->key[u] = k;
        }
        __syncthreads();
        for (uint32_t u = warp; u < und; u += WARPS) {
            const uint64_t k = sm->key[u];
            const int i = sm->idx[u];
            uint32_t ahead = 0;
            for (uint32_t v = lane; v < und; v += 32) {
                const uint64_t kv = sm->key[v];
                ahead += kv > k || (kv == k && sm->idx[v] < i);
            }
            ahead = __reduce_add_sync(0xffffffffu, ahead);
            if (lane == 0 && ahead < left) atomicOr(&kept[i >> 5], 1u << (i & 31));
        }
        __syncthreads();
    } else {
        // many: the left-th largest key by radix, 8 bits a pass, then as many
        // of the blocks that equal it as are missing, the lowest indexes first
        uint64_t *key = p.keys + unit * p.stride;
        for (int w = warp; w < words; w += WARPS)
            for (uint32_t m = open[w]; m != 0; m &= m - 1) {
                const int i = w * 32 + __ffs(m) - 1;
                const uint64_t k = exact_key<D>(p, q, __ldg(table + i), h);
                if (lane == 0) key[i] = k;
            }
        uint64_t prefix = 0;
        uint32_t rest = left;  // 1 <= left <= und: all but `und` blocks are in or out
        for (int shift = 56; shift >= 0; shift -= 8) {
            __syncthreads();  // keys written; the last pass's histogram read
            for (int i = tid; i < 256; i += T) sm->hist[i] = 0;
            __syncthreads();
            for (int i = tid; i < n; i += T)
                if ((open[i >> 5] >> (i & 31)) & 1u) {
                    const uint64_t k = key[i];
                    if (shift == 56 || (k >> (shift + 8)) == prefix) atomicAdd(&sm->hist[(k >> shift) & 255u], 1u);
                }
            uint32_t digit, ab, inside;
            find_bin<256, T>(sm, rest, digit, ab, inside);
            prefix = (prefix << 8) | digit;
            rest -= ab;
        }
        uint32_t seen = 0;  // blocks equal to the border so far
        for (int base = 0; base < n; base += T) {
            const int i = base + tid;
            const bool und_i = i < n && ((open[i >> 5] >> (i & 31)) & 1u);
            const uint64_t k = und_i ? key[i] : 0;
            const bool eq = und_i && k == prefix;
            uint32_t total;
            const uint32_t before = seen + block_scan<T>(sm, eq, total);
            seen += total;
            const uint32_t add = __ballot_sync(0xffffffffu, und_i && (k > prefix || (eq && before < rest)));
            if (lane == 0 && add != 0) kept[i >> 5] |= add;  // the warp's word
        }
        __syncthreads();
    }
    // the list, in ascending order
    uint32_t at = 0;
    for (int base = 0; base < words; base += T) {
        const int w = base + tid;
        uint32_t m = w < words ? kept[w] : 0, total;
        uint32_t pos = at + block_scan<T>(sm, __popc(m), total);
        at += total;
        for (; m != 0; m &= m - 1, ++pos)
            if (pos < (uint32_t)p.K) out[pos] = w * 32 + __ffs(m) - 1;
    }
}

}  // namespace pkv

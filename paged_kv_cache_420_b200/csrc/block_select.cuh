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
// one product of [g heads][2 D] and [2 D][8 blocks] on the tensor cores, whose
// operand is read straight from global memory in fragment order: the kernel is
// bound by the bounds' bytes.  bf16 products are exact in fp32 and their sums
// are not, so these scores only narrow the choice: with an error of at most e,
// a block whose score is more than 2 e above the K-th largest is in, one more
// than 2 e below is out, and the few between them are scored again in fp64.
//
// A cluster of CTAs takes one (s, h), each a contiguous range of its blocks;
// scores stay in shared memory, counts are added up over distributed shared
// memory, and the list is written in ascending order.  One launch, no
// workspace.
#pragma once

#include "ptx.cuh"

namespace pkv {

constexpr int kSelThreads = 256;
constexpr int kSelWarps = kSelThreads / 32;
constexpr int kSelBins = 2048;       // two passes of 11 bits find the K-th score to 22 of its 32
constexpr int kSelPairMax = 512;     // undecided blocks up to which each is compared with each
constexpr int kSelMaxCluster = 8;
// Bound of a score's fp32 error relative to sum |q_d| max |bound|: at most 16
// products of k = 16 follow one another; each adds 17 numbers, and each
// addition loses at most 2^-23 of the largest: 16 * 17 * 2^-23 < 2^-14.9.
constexpr float kSelError = 1.220703125e-4f;  // 2^-13

struct SelectParams {
    const __nv_bfloat16 *q;       // [B][Hq][D]
    const __nv_bfloat16 *bounds;  // [NB][H][2][D]
    const int32_t *block_tables;  // [B][MBS]
    const int32_t *context_lens;  // [B]
    int32_t *selected;            // [B][H][K]
    int H, g, MBS, bs, NB, K, max_ctx;
    int splits;  // CTAs of a cluster
    int cap;     // blocks of a CTA at most
};

struct SelectSmem {
    uint32_t hist[2][kSelBins];
    uint64_t pair_key[kSelPairMax];  // the undecided blocks of the whole cluster
    int pair_idx[kSelPairMax];
    uint32_t scan[kSelWarps];
    uint32_t counts[4];  // read by peers: undecided, in, selected, equal to the border
    uint32_t found[4];   // threshold search: bin, count above it
    float qsum, bmax[kSelWarps];
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

// Finds, in the cluster's summed histogram of `bins` bins, the bin that holds
// the m-th largest key (m >= 1; fewer than m keys: bin 0) and the number of
// keys in the bins above it.  The histograms are complete (a cluster barrier
// has passed).  All threads return the same values.
__device__ __forceinline__ void find_bin(SelectSmem *sm, const uint32_t *hist, int bins, int splits, uint32_t m,
                                         uint32_t &bin, uint32_t &above) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = bins / kSelThreads;  // 8 or 1 bins of a thread, from the top
    uint32_t c[8], sum = 0;
    if (per == 8) {
        const int b0 = bins - (tid + 1) * 8;
#pragma unroll
        for (int i = 0; i < 8; ++i) c[i] = 0;
        for (int u = 0; u < splits; ++u) {
            const uint4 x = cluster_ld_v4(cluster_addr(hist + b0, u)), y = cluster_ld_v4(cluster_addr(hist + b0 + 4, u));
            c[7] += x.x; c[6] += x.y; c[5] += x.z; c[4] += x.w;
            c[3] += y.x; c[2] += y.y; c[1] += y.z; c[0] += y.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) sum += c[i];
    } else {
        c[0] = 0;
        for (int u = 0; u < splits; ++u) c[0] += cluster_ld_u32(cluster_addr(hist + bins - 1 - tid, u));
        sum = c[0];
    }
    uint32_t incl = sum;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const uint32_t y = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += y;
    }
    if (lane == 31) sm->scan[warp] = incl;
    if (tid == 0) { sm->found[0] = 0; sm->found[1] = 0; }
    __syncthreads();
    uint32_t before = incl - sum;
    for (int w = 0; w < warp; ++w) before += sm->scan[w];
    if (before < m && before + sum >= m) {
        uint32_t a = before;
        for (int i = 0; i < per; ++i) {
            if (a + c[i] >= m) {
                sm->found[0] = (uint32_t)(bins - 1 - (tid * per + i));
                sm->found[1] = a;
                break;
            }
            a += c[i];
        }
    }
    __syncthreads();
    bin = sm->found[0];
    above = sm->found[1];
    __syncthreads();
}

template <int D, bool TALL>  // TALL: more than 8 query heads
__global__ void __launch_bounds__(kSelThreads) select_blocks_kernel(const SelectParams p) {
    constexpr int VE = 2 * D;          // elements of a block's bounds
    constexpr int CH = VE / 32;        // 16-byte loads of a lane per block
    extern __shared__ __align__(16) uint8_t select_smem_raw[];
    SelectSmem *sm = reinterpret_cast<SelectSmem *>(select_smem_raw);
    // per block of this CTA: its score (later whether it is selected), and the
    // undecided ones' fp64 keys and indexes
    float *score = reinterpret_cast<float *>(select_smem_raw + (sizeof(SelectSmem) + 15) / 16 * 16);
    uint64_t *ukey = reinterpret_cast<uint64_t *>(score + (p.cap + 3) / 4 * 4);
    int *uidx = reinterpret_cast<int *>(ukey + p.cap);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x / p.splits, rank = blockIdx.x - unit * p.splits;
    const int s = unit / p.H, h = unit - s * p.H;
    grid_dependency_wait();
    int n_ctx = __ldg(p.context_lens + s);
    const int cap_ctx = (int)min((long long)p.MBS * p.bs, (long long)p.max_ctx);
    if (n_ctx < 0 || n_ctx > cap_ctx) {
        if (h == 0 && rank == 0 && tid == 0) raise_error(PKV_DEVERR_CONTEXT);
        n_ctx = n_ctx < 0 ? 0 : cap_ctx;
    }
    const int n = (n_ctx + p.bs - 1) / p.bs;
    int32_t *out = p.selected + (size_t)unit * p.K;
    if (n <= p.K) {  // nothing to choose (the whole cluster leaves here)
        for (int i = rank * kSelThreads + tid; i < p.K; i += p.splits * kSelThreads) out[i] = i < n ? i : -1;
        return;
    }
    const int32_t *table = p.block_tables + (size_t)s * p.MBS;
    const int per = (n + p.splits - 1) / p.splits;
    const int lo = min(n, rank * per), cnt = min(n, lo + per) - lo;  // this CTA's blocks
    for (int i = tid; i < 2 * kSelBins; i += kSelThreads) (&sm->hist[0][0])[i] = 0;
    if (tid == 0) sm->counts[0] = 0;

    // ------------------------------------------------------------ scores ----
    // A fragments of the heads' max(q, 0) and min(q, 0): lane (r = lane / 4,
    // j = lane % 4) holds rows r and r + 8.  Chunk i of a block's bounds is its
    // elements 32 i .. 32 i + 31; lane j loads 8 of them, 32 i + 8 j .. + 7,
    // which are the operands of two k-steps (the order of k is free).
    const __nv_bfloat16 *q = p.q + ((size_t)unit * p.g) * D;
    uint32_t a0[CH][4], a1[TALL ? CH : 1][4];
    auto q_pair = [&](int head, int e) -> uint32_t {  // elements e, e + 1 of [min(q, 0) | max(q, 0)]
        if (head >= p.g) return 0u;
        uint32_t x = *reinterpret_cast<const uint32_t *>(q + (size_t)head * D + (e >= D ? e - D : e));
        const uint32_t neg = (x & 0x8000u ? 0xffffu : 0u) | (x & 0x80000000u ? 0xffff0000u : 0u);
        return e >= D ? x & ~neg : x & neg;
    };
#pragma unroll
    for (int i = 0; i < CH; ++i)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            a0[i][u] = q_pair(lane >> 2, 32 * i + 8 * (lane & 3) + 2 * u);
            if constexpr (TALL) a1[i][u] = q_pair((lane >> 2) + 8, 32 * i + 8 * (lane & 3) + 2 * u);
        }
    {   // the largest sum |q_jd| of a head
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
        float m = fmaxf(s0, s1);
        if (s0 != s0 || s1 != s1) m = __int_as_float(0x7f800000);
        m = warp_max_f32(m);
        if (tid == 0) sm->qsum = m;
    }
    __syncthreads();
    uint32_t bmax = 0;  // the largest |bound|, NaN if there is one
    const float inf = __int_as_float(0x7f800000);
    for (int t = warp * 8; t < cnt; t += kSelWarps * 8) {
        const int i = t + (lane >> 2);  // this lane loads for block lo + i
        int blk = -1;
        if (i < cnt) {
            blk = __ldg(table + lo + i);
            if (blk < 0 || blk >= p.NB) {
                if (h == 0 && (lane & 3) == 0) raise_error(PKV_DEVERR_BLOCK);
                blk = -1;
            }
        }
        uint4 x[CH];
        const uint4 *src = reinterpret_cast<const uint4 *>(p.bounds + ((size_t)max(blk, 0) * p.H + h) * VE) + (lane & 3);
#pragma unroll
        for (int c = 0; c < CH; ++c) x[c] = blk >= 0 ? __ldg(src + 4 * c) : make_uint4(0, 0, 0, 0);
        float d0 = 0.f, d1 = 0.f, d2 = 0.f, d3 = 0.f;
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            const uint32_t h1 = TALL ? 1u : 0u;
            mma_bf16_16816(d0, d1, d2, d3, a0[c][0], h1 ? a1[TALL ? c : 0][0] : 0u, a0[c][1], h1 ? a1[TALL ? c : 0][1] : 0u,
                           x[c].x, x[c].y);
            mma_bf16_16816(d0, d1, d2, d3, a0[c][2], h1 ? a1[TALL ? c : 0][2] : 0u, a0[c][3], h1 ? a1[TALL ? c : 0][3] : 0u,
                           x[c].z, x[c].w);
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(bmax) : "r"(x[c].x & 0x7fff7fffu));
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(bmax) : "r"(x[c].y & 0x7fff7fffu));
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(bmax) : "r"(x[c].z & 0x7fff7fffu));
            asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(bmax) : "r"(x[c].w & 0x7fff7fffu));
        }
        // rows r and r + 8 of columns 2 j and 2 j + 1: the max over the heads
        const int r = lane >> 2;
        float m0 = r < p.g ? d0 : -inf, m1 = r < p.g ? d1 : -inf;
        if (TALL && r + 8 < p.g) {
            m0 = fmaxf(m0, d2);
            m1 = fmaxf(m1, d3);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1) {
            m0 = fmaxf(m0, __shfl_xor_sync(0xffffffffu, m0, o));
            m1 = fmaxf(m1, __shfl_xor_sync(0xffffffffu, m1, o));
        }
        const uint32_t bad = __ballot_sync(0xffffffffu, blk < 0);  // of block c: bit 4 c
        if (lane < 4) {
            const int c0 = t + 2 * lane, c1 = c0 + 1;
            if (c0 < cnt) score[c0] = (bad >> (8 * lane)) & 1u ? -inf : m0;
            if (c1 < cnt) score[c1] = (bad >> (8 * lane + 4)) & 1u ? -inf : m1;
        }
    }
    {
        const float b0 = bf16lo_to_f32(bmax), b1 = bf16hi_to_f32(bmax);
        float b = fmaxf(b0, b1);
        if (b0 != b0 || b1 != b1) b = inf;
        b = warp_max_f32(b);
        if (lane == 0) sm->bmax[warp] = b;
    }
    __syncthreads();
    float bm = 0.f;
    for (int w = 0; w < kSelWarps; ++w) bm = fmaxf(bm, sm->bmax[w]);
    // The bound of this CTA's errors, with room for products below fp32's
    // normal range.  Not finite (or so large that the sums may not be): every
    // block of the cluster is undecided.
    float err = fmaf(sm->qsum * bm, kSelError, 1e-33f);
    if (!(sm->qsum * bm < 1e37f)) err = inf;

    // --------------------------------------------------- the K-th largest ----
    // of the blocks between the first and the last, to 22 bits.
    const uint32_t want = (uint32_t)(p.K - 2);
    auto ranked = [&](int i) { return lo + i > 0 && lo + i < n - 1; };
    uint32_t k0 = 0, k1 = 0, above = 0;
    float t_lo = -inf, t_hi = inf, e2 = inf;
    // the largest error bound of the cluster is needed with the counts
    if (tid == 0) sm->counts[1] = __float_as_uint(err);
    for (int i = tid; i < cnt; i += kSelThreads)
        if (ranked(i)) atomicAdd(&sm->hist[0][order_key(score[i]) >> 21], 1u);
    cluster_arrive();
    cluster_wait();
    float emax = 0.f;
    for (int u = 0; u < p.splits; ++u) emax = fmaxf(emax, __uint_as_float(cluster_ld_u32(cluster_addr(&sm->counts[1], u))));
    if (want > 0 && emax < inf) {
        find_bin(sm, sm->hist[0], kSelBins, p.splits, want, k0, above);
        for (int i = tid; i < cnt; i += kSelThreads) {
            const uint32_t k = order_key(score[i]);
            if (ranked(i) && (k >> 21) == k0) atomicAdd(&sm->hist[1][(k >> 10) & (kSelBins - 1)], 1u);
        }
    }
    cluster_arrive();
    cluster_wait();
    if (want > 0 && emax < inf) {
        uint32_t above1;
        find_bin(sm, sm->hist[1], kSelBins, p.splits, want - above, k1, above1);
        const uint32_t key = (k0 << 21) | (k1 << 10);
        t_lo = order_value(key);
        t_hi = order_value(key | 1023u);
        e2 = 2.f * emax;
    }
    // in, out or undecided
    uint32_t n_in = 0;
    for (int i = tid; i < cnt; i += kSelThreads) {
        float verdict = 0.f;
        if (!ranked(i)) {
            verdict = 1.f;  // kept whatever its score
        } else if (want > 0) {
            const float a = score[i];
            if (a > t_hi + e2) {
                verdict = 1.f;
                ++n_in;
            } else if (!(a < t_lo - e2)) {
                verdict = 0.f;
                uidx[atomicAdd(&sm->counts[0], 1u)] = i;
            }
        }
        score[i] = verdict;
    }
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) n_in += __shfl_xor_sync(0xffffffffu, n_in, o);
    if (lane == 0) sm->scan[warp] = n_in;
    __syncthreads();
    n_in = 0;
    for (int w = 0; w < kSelWarps; ++w) n_in += sm->scan[w];
    const int und = (int)sm->counts[0];
    // their scores in fp64: a warp a block
    for (int u = warp; u < und; u += kSelWarps) {
        const int i = uidx[u];
        const int blk = __ldg(table + lo + i);
        double best = -__longlong_as_double(0x7ff0000000000000ll);
        if (blk >= 0 && blk < p.NB) {
            const __nv_bfloat16 *b = p.bounds + ((size_t)blk * p.H + h) * VE;
            bool nan = false;
            for (int j = 0; j < p.g; ++j) {
                double sum = 0.0;
#pragma unroll
                for (int e = 0; e < D / 32; ++e) {
                    const int d = e * 32 + lane;
                    const double x = (double)__bfloat162float(q[(size_t)j * D + d]);
                    const double y = x * (double)__bfloat162float(b[d]), z = x * (double)__bfloat162float(b[D + d]);
                    sum += (y != y || z != z) ? y + z : (y > z ? y : z);
                }
#pragma unroll
                for (int o = 16; o >= 1; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
                nan |= sum != sum;
                best = sum > best ? sum : best;
            }
            if (nan) best = __longlong_as_double(0x7ff0000000000000ll);
        }
        if (lane == 0) ukey[u] = order_key(best);
    }
    if (tid == 0) sm->counts[1] = n_in;
    cluster_arrive();
    cluster_wait();
    uint32_t all_in = 0, all_und = 0, und_before = 0;
    for (int u = 0; u < p.splits; ++u) {
        all_in += cluster_ld_u32(cluster_addr(&sm->counts[1], u));
        const uint32_t c = cluster_ld_u32(cluster_addr(&sm->counts[0], u));
        und_before += u < rank ? c : 0;
        all_und += c;
    }
    const uint32_t m = want - all_in;  // how many of the undecided are kept
    if (all_und <= (uint32_t)kSelPairMax) {
        // each against each: one is kept if fewer than m are ahead of it
        uint32_t off = 0;
        for (int u = 0; u < p.splits; ++u) {
            const int c = (int)cluster_ld_u32(cluster_addr(&sm->counts[0], u));
            for (int i = tid; i < c; i += kSelThreads) {
                sm->pair_key[off + i] = cluster_ld_u64(cluster_addr(ukey + i, u));
                sm->pair_idx[off + i] = u * per + (int)cluster_ld_u32(cluster_addr(uidx + i, u));
            }
            off += c;
        }
        __syncthreads();
        for (int u = warp; u < und; u += kSelWarps) {
            const uint64_t k = ukey[u];
            const int idx = lo + uidx[u];
            uint32_t ahead = 0;
            for (uint32_t v = lane; v < all_und; v += 32) {
                const uint64_t kv = sm->pair_key[v];
                ahead += kv > k || (kv == k && sm->pair_idx[v] < idx);
            }
#pragma unroll
            for (int o = 16; o >= 1; o >>= 1) ahead += __shfl_xor_sync(0xffffffffu, ahead, o);
            if (lane == 0 && ahead < m) score[uidx[u]] = 1.f;
        }
    } else {
        // many: the m-th largest key by radix, 8 bits a pass, then as many of
        // the blocks that equal it as are missing, lowest indexes first
        uint64_t prefix = 0;
        uint32_t left = m;  // 1 <= m <= all_und here: want of the ranked blocks are in or undecided
        for (int pass = 0; pass < 8; ++pass) {
            uint32_t *hist = sm->hist[pass & 1];
            const int shift = 56 - 8 * pass;
            if (tid < 256) hist[tid] = 0;
            __syncthreads();
            for (int u = tid; u < und; u += kSelThreads)
                if (pass == 0 || (ukey[u] >> (shift + 8)) == prefix) atomicAdd(&hist[(ukey[u] >> shift) & 255u], 1u);
            cluster_arrive();
            cluster_wait();
            uint32_t digit, ab;
            find_bin(sm, hist, 256, p.splits, left, digit, ab);
            prefix = (prefix << 8) | digit;
            left -= ab;
        }
        // score: 1 kept, 2 equal to the border
        uint32_t eq = 0;
        for (int u = tid; u < und; u += kSelThreads) {
            if (ukey[u] > prefix) score[uidx[u]] = m > 0 ? 1.f : 0.f;
            else if (ukey[u] == prefix) {
                score[uidx[u]] = 2.f;
                ++eq;
            }
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) eq += __shfl_xor_sync(0xffffffffu, eq, o);
        if (lane == 0) sm->scan[warp] = eq;
        __syncthreads();
        if (tid == 0) {
            uint32_t e = 0;
            for (int w = 0; w < kSelWarps; ++w) e += sm->scan[w];
            sm->counts[3] = e;
        }
        cluster_arrive();
        cluster_wait();
        uint32_t eq_before = 0;
        for (int u = 0; u < rank; ++u) eq_before += cluster_ld_u32(cluster_addr(&sm->counts[3], u));
        // in index order: the first `left` of the cluster's equal ones are kept
        for (int base = 0; base < cnt; base += kSelThreads) {
            const int i = base + tid;
            const bool is = i < cnt && score[i] == 2.f;
            const uint32_t mask = __ballot_sync(0xffffffffu, is);
            __syncthreads();
            if (lane == 0) sm->scan[warp] = __popc(mask);
            __syncthreads();
            uint32_t before = eq_before + __popc(mask & ((1u << lane) - 1)), chunk = 0;
            for (int w = 0; w < kSelWarps; ++w) {
                if (w < warp) before += sm->scan[w];
                chunk += sm->scan[w];
            }
            if (is) score[i] = before < left && m > 0 ? 1.f : 0.f;
            eq_before += chunk;
        }
    }
    __syncthreads();

    // -------------------------------------------------------------- list ----
    uint32_t kept = 0;
    for (int i = tid; i < cnt; i += kSelThreads) kept += score[i] == 1.f;
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) kept += __shfl_xor_sync(0xffffffffu, kept, o);
    if (lane == 0) sm->scan[warp] = kept;
    __syncthreads();
    if (tid == 0) {
        uint32_t e = 0;
        for (int w = 0; w < kSelWarps; ++w) e += sm->scan[w];
        sm->counts[2] = e;
    }
    cluster_arrive();
    cluster_wait();
    grid_launch_dependents();
    uint32_t at = 0;
    for (int u = 0; u < rank; ++u) at += cluster_ld_u32(cluster_addr(&sm->counts[2], u));
    cluster_arrive();  // the last reads of the peers' shared memory
    for (int base = 0; base < cnt; base += kSelThreads) {
        const int i = base + tid;
        const bool is = i < cnt && score[i] == 1.f;
        const uint32_t mask = __ballot_sync(0xffffffffu, is);
        __syncthreads();
        if (lane == 0) sm->scan[warp] = __popc(mask);
        __syncthreads();
        uint32_t before = at + __popc(mask & ((1u << lane) - 1));
        for (int w = 0; w < kSelWarps; ++w) {
            if (w < warp) before += sm->scan[w];
            at += sm->scan[w];
        }
        if (is && before < (uint32_t)p.K) out[before] = lo + i;
    }
    cluster_wait();
}

}  // namespace pkv

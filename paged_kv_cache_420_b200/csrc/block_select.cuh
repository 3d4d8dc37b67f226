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
// head at head dim 128, against 8 D g operations).  All tiles of 8 blocks of all
// sequences and groups of 4 heads form one line, of which every CTA takes an
// equal stretch, a head a warp; a fifth warp looks the blocks up and copies a
// block's 4 heads, which lie side by side, at once (2 KB: a bulk copy takes its
// lane 70 cycles to issue, and copies of single heads kept their warps from
// computing: 64 sequences of 1025 to 8192 tokens, selection included, 25.9 us
// against 22.0; loads straight into the operand registers 25.6).  Selection is a CTA for each
// (s, h) over the scores that the first kernel left in the workspace (in L2).
#pragma once

#include "decode.cuh"
#include "even_cut.cuh"

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
    return (int)(((uint32_t)n + p.bs - 1) / (uint32_t)p.bs);
}

// ----------------------------------------------------------- scoring ----
constexpr int kScoreWarps = 4;  // that compute; one more copies
constexpr int kScoreThreads = (kScoreWarps + 1) * 32;
constexpr int kScoreTile = 8;   // blocks of a tile
constexpr int kScoreRing = 4;   // tiles of a warp in flight

// What the computing warps have to know of a tile.
struct __align__(16) ScoreTile {
    int unit;  // (s, first head of the group)
    int b0;    // its first logical block
    int good;  // a bit for each block that has a row
    int none;
};

template <int D>
struct ScoreSmem {
    static constexpr int kBytes = 4 * D;  // a block's bounds, of one head
    // a ring slot of one head's tile at most: the blocks of a tile are `heads`
    // rows and 64 bytes apart, so that two of them lie in different halves of
    // the banks
    static constexpr int kSlot = kScoreTile * (kBytes + 64);
    static constexpr int oInfo = kScoreWarps * kScoreRing * kSlot;             // ScoreTile [streams][ring]
    static constexpr int oScan = oInfo + kScoreWarps * kScoreRing * 16;        // long long [threads]
    static constexpr int oSum = oScan + kScoreThreads * 8;                     // long long [warps]
    static constexpr int oBars = oSum + (kScoreWarps + 1) * 8;
    static constexpr int oAbort = oBars + 2 * kScoreWarps * kScoreRing * 8;
    static constexpr int kAlloc = oAbort + 16;
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
    constexpr int R = kScoreRing, TB = kScoreTile;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    ScoreTile *info = reinterpret_cast<ScoreTile *>(smem_raw + L::oInfo);
    long long *scan = reinterpret_cast<long long *>(smem_raw + L::oScan);
    long long *warp_sum = reinterpret_cast<long long *>(smem_raw + L::oSum);
    uint64_t *full = reinterpret_cast<uint64_t *>(smem_raw + L::oBars), *empty = full + kScoreWarps * R;
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem_raw + L::oAbort);
    // groups of 4, 2 or 1 heads: as many warps share a stretch
    const int heads = p.H % 4 == 0 ? 4 : p.H % 2 == 0 ? 2 : 1, hgroups = p.H / heads, streams = kScoreWarps / heads;
    if (tid == 0) {
        for (int i = 0; i < streams * R; ++i) { mbar_init(&full[i], 1); mbar_init(&empty[i], heads); }
        *abort_flag = 0;
        fence_mbar_init();
    }
    grid_dependency_wait();
    // The line: sequences with something to choose, their groups of `heads`
    // heads, tiles of 8 blocks.
    auto tiles_of = [&](int s, int &n) {
        n = select_blocks_of(p, s, false);
        return n > p.K ? (n + kScoreTile - 1) / kScoreTile : 0;
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
    for (int w = 0; w <= kScoreWarps; ++w) {
        if (w < warp) before += warp_sum[w];
        total += warp_sum[w];
    }
    scan[tid] = before + incl - sum;  // the tiles before this thread's sequences
    __syncthreads();
    const int parts = (int)max(1ll, min((long long)gridDim.x * streams, total));
    const EvenCut line(total, parts);
    // Stream j of the CTA: its stretch of the line.
    auto stretch = [&](int j, long long &a) -> int {
        const int me = (int)blockIdx.x * streams + j;
        if (me >= parts || total == 0) return 0;
        a = line.begin(me);
        return (int)(line.begin(me + 1) - a);
    };

    if (warp == kScoreWarps) {
        // ------------------------------------------------------ producer --
        // 32 / streams lanes for a stream: they look up as many blocks at once.
        const int lanes = 32 / streams, j = lane / lanes, sub = lane % lanes, ahead = lanes / TB;  // tiles
        long long a = 0;
        const int len = stretch(j, a);
        int longest = len;
#pragma unroll
        for (int o = 8; o < 32; o <<= 1) longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, o));
        int cs = 0, nt = 0, n = 0;
        long long base = 0;
        if (len > 0) {
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
            int unit, b, id;  // (s, first head), logical block, physical block as the table has it
            bool under;       // the context reaches the block
        };
        auto look_up = [&](int G) -> Look {  // this lane's block of tile G * ahead + sub / TB
            const int k = G * ahead + sub / TB;
            Look r = {-1, 0, -1, false};
            if (k >= len) return r;
            const long long x = a + k;
            while (x >= base + (long long)nt * hgroups) {
                base += (long long)nt * hgroups;
                nt = tiles_of(++cs, n);
            }
            const uint32_t off = (uint32_t)(x - base);  // below H * blocks / 8, and that below 2^31
            const int hg = (int)(off / (uint32_t)nt);
            r.unit = cs * p.H + hg * heads;
            r.b = (int)(off - (uint32_t)hg * nt) * TB + sub % TB;
            r.under = r.b < n;
            if (r.under) r.id = __ldg(p.block_tables + (size_t)cs * p.MBS + r.b);
            return r;
        };
        const int slot_bytes = heads * L::kSlot, row_bytes = heads * L::kBytes;
        bool ok = true;
        int issued = 0;
        Look next = look_up(0);
        for (int G = 0; G * ahead < longest && ok; ++G) {
            const Look cur = next;
            next = look_up(G + 1);
            const bool have = cur.id >= 0 && cur.id < p.NB;
            if (cur.under && !have && cur.unit % p.H == 0) raise_error(PKV_DEVERR_BLOCK);
            const uint32_t good = __ballot_sync(0xffffffffu, have);
            for (int t = 0; t < ahead && ok; ++t) {
                const int k = G * ahead + t, slot = j * R + k % R;
                const bool mine = sub / TB == t && k < len;
                bool lane_ok = true;
                if (mine) {
                    lane_ok = wait_slot(&empty[slot], ((k / R) & 1) ^ 1, abort_flag);
                    if (lane_ok && sub % TB == 0) {
                        ScoreTile ti;
                        ti.unit = cur.unit;
                        ti.b0 = cur.b;
                        ti.good = (int)((good >> lane) & ((1u << TB) - 1));
                        ti.none = 0;
                        info[slot] = ti;
                        mbar_arrive_expect_tx(&full[slot], (uint32_t)(__popc(ti.good) * row_bytes));
                    }
                }
                ok = __all_sync(0xffffffffu, lane_ok);
                if (mine && ok && have)
                    bulk_load(smem_raw + j * R * slot_bytes + (k % R) * slot_bytes + (sub % TB) * (row_bytes + 64),
                              p.bounds + ((size_t)cur.id * p.H + cur.unit % p.H) * VE, row_bytes, &full[slot]);
                if (k < len) issued = k + 1;
            }
        }
        __syncthreads();  // the consumers are through
        // After a wait that gave up, what is in flight still has to land.
        if (*abort_flag && sub == 0)
            for (int k = max(0, issued - R); k < issued; ++k) mbar_wait_bounded(&full[j * R + k % R], (k / R) & 1, kWaitLimitNs);
        return;
    }
    // -------------------------------------------------------- consumer --
    const int j = warp / heads, hd = warp % heads;  // its stream, its head of the group
    long long a = 0;
    const int len = stretch(j, a);
    // A fragments of the heads' min(q, 0) and max(q, 0): lane (r = lane / 4,
    // j = lane % 4) holds rows r and r + 8.  Chunk i of a block's bounds is its
    // elements 32 i .. 32 i + 31; lane j reads 8 of them, 32 i + 8 j .. + 7,
    // which are the operands of two k-steps (the order of k is free).  The
    // first half of the chunks are least elements, the second largest ones.
    const float inf = __int_as_float(0x7f800000);
    uint32_t a0[CH][4], a1[TALL ? CH : 1][4];
    float qsum = 0.f;  // the largest sum |q_jd| of a head
    auto load_q = [&](int unit) {
        float sum[2] = {0.f, 0.f};
        auto row = [&](int head, uint32_t (&f)[CH][4], float &sum) {
            const __nv_bfloat16 *q = p.q + ((size_t)unit * p.g + head) * D + 8 * (lane & 3);
#pragma unroll
            for (int i = 0; i < CH / 2; ++i) {
                const uint4 v = head < p.g ? __ldg(reinterpret_cast<const uint4 *>(q + 32 * i)) : make_uint4(0, 0, 0, 0);
                f[i][0] = v.x; f[i][1] = v.y; f[i][2] = v.z; f[i][3] = v.w;
            }
            float t = 0.f;
#pragma unroll
            for (int i = 0; i < CH / 2; ++i)
#pragma unroll
                for (int u = 0; u < 4; ++u) {
                    const uint32_t w = f[i][u];
                    sum += fabsf(bf16lo_to_f32(w));
                    t += fabsf(bf16hi_to_f32(w));
                    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(f[i][u]) : "r"(w), "r"(0u));
                    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(f[i + CH / 2][u]) : "r"(w), "r"(0u));
                }
            sum += t;
            sum += __shfl_xor_sync(0xffffffffu, sum, 1);
            sum += __shfl_xor_sync(0xffffffffu, sum, 2);
            if (sum != sum) sum = inf;
        };
        row(lane >> 2, a0, sum[0]);
        if constexpr (TALL) row((lane >> 2) + 8, a1, sum[1]);
        qsum = warp_max_f32(fmaxf(sum[0], sum[1]));
    };
    int unit = -1;
    const int slot_bytes = heads * L::kSlot, block_stride = heads * L::kBytes + 64;
    for (int k = 0; k < len; ++k) {
        const int slot = j * R + k % R;
        if (!wait_or_abort(&full[slot], (k / R) & 1, abort_flag)) break;
        const ScoreTile ti = info[slot];
        if (ti.unit + hd != unit) {
            unit = ti.unit + hd;
            load_q(unit);
        }
        // (a block without a row leaves old bytes here, and garbage in its own column only)
        const uint32_t src = smem_u32(smem_raw) + slot * slot_bytes + (lane >> 2) * block_stride + hd * L::kBytes + 16 * (lane & 3);
        const uint32_t good = (uint32_t)ti.good;
        float d[2][4];
        uint32_t w_lo = 0, w_hi = 0;  // the largest least element above 0, the smallest largest one below
#pragma unroll
        for (int c = 0; c < 4; ++c) d[0][c] = d[1][c] = 0.f;
        uint4 x[CH];
#pragma unroll
        for (int c = 0; c < CH; ++c)
            asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
                         : "=r"(x[c].x), "=r"(x[c].y), "=r"(x[c].z), "=r"(x[c].w)
                         : "r"(src + 64 * c));
#pragma unroll
        for (int c = 0; c < CH; ++c) {
            float(&e)[4] = d[c & 1];
            const uint32_t z0 = TALL ? a1[TALL ? c : 0][0] : 0u, z1 = TALL ? a1[TALL ? c : 0][1] : 0u;
            const uint32_t z2 = TALL ? a1[TALL ? c : 0][2] : 0u, z3 = TALL ? a1[TALL ? c : 0][3] : 0u;
            mma_bf16_16816(e[0], e[1], e[2], e[3], a0[c][0], z0, a0[c][1], z1, x[c].x, x[c].y);
            mma_bf16_16816(e[0], e[1], e[2], e[3], a0[c][2], z2, a0[c][3], z3, x[c].z, x[c].w);
            const uint32_t v[4] = {x[c].x, x[c].y, x[c].z, x[c].w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                if (c < CH / 2) asm("max.NaN.bf16x2 %0, %0, %1;" : "+r"(w_lo) : "r"(v[i]));
                else asm("min.NaN.bf16x2 %0, %0, %1;" : "+r"(w_hi) : "r"(v[i]));
            }
        }
        __syncwarp();
        if (lane == 0) mbar_arrive(&empty[slot]);  // the slot is read
        // w of the tile, as bits: a NaN is above every number
        w_hi &= 0x7fff7fffu;
        uint32_t wb = max(max(w_lo & 0xffffu, w_lo >> 16), max(w_hi & 0xffffu, w_hi >> 16));
        wb = __reduce_max_sync(0xffffffffu, (good >> (lane >> 2)) & 1u ? wb : 0u);
        // rows r and r + 8 of columns 2 j and 2 j + 1: the max over the heads,
        // NaN if one is
        const int r = lane >> 2;
        float sc[2];
#pragma unroll
        for (int c = 0; c < 2; ++c) {
            sc[c] = r < p.g ? d[0][c] + d[1][c] : -inf;
            if (TALL && r + 8 < p.g) sc[c] = max_nan(sc[c], d[0][c + 2] + d[1][c + 2]);
        }
#pragma unroll
        for (int o = 4; o < 32; o <<= 1)
#pragma unroll
            for (int c = 0; c < 2; ++c) sc[c] = max_nan(sc[c], __shfl_xor_sync(0xffffffffu, sc[c], o));
        // Room for products below fp32's normal range.  Where a sum of
        // magnitudes is not finite, or so large that the sums may not be,
        // nothing is known of the score.
        const float neg = 2.f * qsum * __uint_as_float(wb << 16);
        auto bound = [&](float y) {
            const float m = fmaxf(y, 0.f) + neg;
            return m < 1e37f && y == y ? fmaf(m, kSelError, 1e-33f) : inf;
        };
        if (lane < 4) {
            const bool g0 = (good >> (2 * lane)) & 1u, g1 = (good >> (2 * lane + 1)) & 1u;
            *reinterpret_cast<float4 *>(p.scores + (size_t)unit * p.stride + ti.b0 + 2 * lane) =
                make_float4(g0 ? sc[0] : -inf, g0 ? bound(sc[0]) : 0.f, g1 ? sc[1] : -inf, g1 ? bound(sc[1]) : 0.f);
        }
    }
    __syncthreads();
}

// ---------------------------------------------------------- selection ----
// A CTA of T threads for each (s, h).  Up to PER scores a thread stay in
// registers; PER = 0 reads them again (from L2) in each pass.  The search for
// the K-th score counts keys in 4 T equal bins between the least and the
// largest (scores of one query lie close together: bins by leading bits would
// send them all to a few counters), and again within a bin that holds more
// keys than there are warps to score them again, until it is as narrow as the
// scores' error.
constexpr int kSelPairMax = 512;  // undecided blocks up to which each is compared with each

template <int T>
struct SelectSmem {
    uint32_t hist[4 * T];
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
// Thread t takes bins 4 (T - 1 - t) .. + 3, the topmost first.
template <int T>
__device__ __forceinline__ void find_bin(SelectSmem<T> *sm, uint32_t m, uint32_t &bin, uint32_t &above, uint32_t &inside) {
    const int b0 = 4 * (T - 1 - (int)threadIdx.x);
    __syncthreads();  // the histogram is complete
    const uint4 v = *reinterpret_cast<const uint4 *>(&sm->hist[b0]);
    const uint32_t c[4] = {v.w, v.z, v.y, v.x};
    uint32_t total;
    uint32_t a = block_scan<T>(sm, v.x + v.y + v.z + v.w, total);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if (a < m && a + c[i] >= m) {
            sm->found[0] = (uint32_t)(b0 + 3 - i);
            sm->found[1] = a;
            sm->found[2] = c[i];
        }
        a += c[i];
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
            // the larger product is hi's where q is positive; both of them have
            // to be numbers (an fp32 product is NaN where the exact one is)
            float x[E];
            load(q + (size_t)j * D, x);
#pragma unroll
            for (int i = 0; i < E; ++i) {
                const float y = x[i] * lo[i], z = x[i] * hi[i];
                nan |= y != y || z != z;
                sum[i & 1] = fma((double)x[i], (double)(x[i] > 0.f ? hi[i] : lo[i]), sum[i & 1]);
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
    constexpr int kBits = T == 512 ? 11 : T == 256 ? 10 : T == 128 ? 9 : 8;  // of 4 T bins
    static_assert(4 * T == 1 << kBits, "bins");
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    SelectSmem<T> *sm = reinterpret_cast<SelectSmem<T> *>(smem_raw);
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const size_t unit = blockIdx.x;
    const int s = (int)(unit / p.H), h = (int)(unit % p.H);
    *reinterpret_cast<uint4 *>(&sm->hist[4 * tid]) = make_uint4(0, 0, 0, 0);
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
        for (int pass = 0; pass < (31 + kBits) / kBits; ++pass) {
            const int shift = max(0, 32 - __clz(width) - kBits);
            each([&](int i, float x) {
                const uint32_t k = order_key(x) - base;
                if (ranked(i) && k <= width) atomicAdd(&sm->hist[k >> shift], 1u);
            });
            uint32_t bin, above, inside;
            find_bin<T>(sm, left, bin, above, inside);
            left -= above;
            base += bin << shift;
            width = min(width - (bin << shift), (1u << shift) - 1);
            t_lo = order_value(base);
            t_hi = order_value(base + width);
            if (inside <= WARPS || t_hi - t_lo <= e || width == 0) break;
            *reinterpret_cast<uint4 *>(&sm->hist[4 * tid]) = make_uint4(0, 0, 0, 0);
            __syncthreads();
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
            *reinterpret_cast<uint4 *>(&sm->hist[4 * tid]) = make_uint4(0, 0, 0, 0);
            __syncthreads();
            for (int i = tid; i < n; i += T)
                if ((open[i >> 5] >> (i & 31)) & 1u) {
                    const uint64_t k = key[i];
                    if (shift == 56 || (k >> (shift + 8)) == prefix) atomicAdd(&sm->hist[(k >> shift) & 255u], 1u);
                }
            uint32_t digit, ab, inside;
            find_bin<T>(sm, rest, digit, ab, inside);
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
    // the list, in ascending order: where each word's blocks begin, then a warp a
    // word
    uint32_t at = 0;
    for (int base = 0; base < words; base += T) {
        const int w = base + tid;
        uint32_t total;
        const uint32_t pos = at + block_scan<T>(sm, w < words ? __popc(kept[w]) : 0, total);
        at += total;
        if (w < words) open[w] = pos;
    }
    __syncthreads();
    for (int w = warp; w < words; w += WARPS) {
        const uint32_t m = kept[w], pos = open[w] + __popc(m & ((1u << lane) - 1));
        if (((m >> lane) & 1u) && pos < (uint32_t)p.K) out[pos] = w * 32 + lane;
    }
}

}  // namespace pkv

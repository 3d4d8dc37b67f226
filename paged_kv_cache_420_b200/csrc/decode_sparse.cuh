// decode_sparse.cuh -- decode attention over selected blocks for sm_100a.
//
// For sequence s and kv head h only the rows of the logical blocks
// selected[s][h][0 .. K) under the context take part in the softmax.  The
// arithmetic is decode.cuh's (the same consumer states over 16-token stages,
// bf16 or block-scaled e4m3); the work is not: every (s, h) has at most K
// blocks, known on the host, so there is no plan and no persistent loop.  A
// cluster of `splits` CTAs takes one (s, h).  Each CTA compacts the valid
// entries of the list, takes its share of their stages through a ring of TMA
// loads, and merges its warps' partial (m, l, acc); then the cluster merges
// the CTAs' partials through distributed shared memory and writes out: one
// launch, no workspace.
#pragma once

#include "decode.cuh"

namespace pkv {

struct SparseParams {
    const __nv_bfloat16 *q;       // [B][Hq][D]
    __nv_bfloat16 *out;           // [B][Hq][D]
    const int32_t *block_tables;  // [B][MBS]
    const int32_t *context_lens;  // [B]
    const int32_t *selected;      // [B][Hkv][K]
    const float *k_scales;        // [NB][Hkv] (e4m3 pool)
    const float *v_scales;
    int Hq, Hkv, g, MBS, bs, NB, K;
    int splits;  // CTAs of a cluster
    int share;   // entries that a CTA's stages can come from (sizes its list)
    int pool_rows;
    float scale_log2;
};

template <int D, int GP, int NS, bool KV8>
struct SparseSmem {
    using R = DecodeSmem<D, GP, NS, KV8, KV8>;
    static constexpr int kW = kConsumerWarps;
    static constexpr int oTiles = 0;
    static constexpr int oMergeO = oTiles + NS * R::kStage;            // [W][GP][stride], the warps' partials
    static constexpr int oMergeM = oMergeO + kW * GP * R::kMergeStride * 4;
    static constexpr int oMergeL = oMergeM + kW * GP * 4;
    static constexpr int oCtaO = oMergeL + kW * GP * 4;                // [GP][D], this CTA's partial
    static constexpr int oCtaM = oCtaO + GP * D * 4;
    static constexpr int oCtaL = oCtaM + GP * 4;
    static constexpr int oBars = (oCtaL + GP * 4 + 7) / 8 * 8;
    static constexpr int oScales = oBars + 2 * NS * 8;
    static constexpr int oCount = oScales + (KV8 ? NS * 8 : 0);        // valid entries of each warp's part of the list
    static constexpr int oAbort = oCount + (kW + 1) * 4;
    static constexpr int oList = (oAbort + 4 + 7) / 8 * 8;             // int2 [share]: (first pool row, rows under the context)
    static int bytes(int share) { return oList + share * 8; }
};

template <int D, int PATH, int GPAD, int NS, bool KV8>
__global__ void __launch_bounds__(kDecodeThreads, decode_min_ctas(PATH, GPAD, KV8))
    sparse_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const SparseParams p) {
    constexpr int W = kConsumerWarps;
    constexpr int GP = GPAD;
    constexpr int NT = (GPAD + 7) / 8;
    constexpr int kFullArrivals = KV8 ? 2 : 1;
    using L = SparseSmem<D, GP, NS, KV8>;
    using R = typename L::R;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::oBars);
    uint64_t *empty = full + NS;
    float2 *slot_scales = reinterpret_cast<float2 *>(smem + L::oScales);
    int *count = reinterpret_cast<int *>(smem + L::oCount);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::oAbort);
    int2 *list = reinterpret_cast<int2 *>(smem + L::oList);
    const uint32_t tiles = smem_u32(smem + L::oTiles);
    float *mO = reinterpret_cast<float *>(smem + L::oMergeO);
    float *mM = reinterpret_cast<float *>(smem + L::oMergeM);
    float *mL = reinterpret_cast<float *>(smem + L::oMergeL);
    float *cO = reinterpret_cast<float *>(smem + L::oCtaO);
    float *cM = reinterpret_cast<float *>(smem + L::oCtaM);
    float *cL = reinterpret_cast<float *>(smem + L::oCtaL);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int unit = blockIdx.x / p.splits, rank = blockIdx.x - unit * p.splits;
    const int s = unit / p.Hkv, h = unit - s * p.Hkv;
    const bool aligned_window = (smem_u32(smem_raw) & 1023u) == 0;  // the swizzle pattern repeats every 1 KB
    if (threadIdx.x == 0) {
        for (int i = 0; i < NS; ++i) { mbar_init(&full[i], kFullArrivals); mbar_init(&empty[i], 1); }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        if (!aligned_window) raise_error(PKV_DEVERR_LAYOUT);
    }
    grid_dependency_wait();

    // The list of valid entries, in order: warp w counts those of its part,
    // then writes the ones that this CTA's stages come from.
    int n = __ldg(p.context_lens + s);
    const long long cap = (long long)p.MBS * p.bs;
    if (n < 0 || n > cap) {
        if (h == 0 && rank == 0 && threadIdx.x == 0) raise_error(PKV_DEVERR_CONTEXT);
        n = n < 0 ? 0 : (int)cap;
    }
    const int nblk = (n + p.bs - 1) / p.bs;
    const int spe = p.bs / kStageTok;  // stages of an entry
    const int32_t *sel = p.selected + (size_t)unit * p.K;
    const int part = (p.K + (W + 1) * 32 - 1) / ((W + 1) * 32) * 32;
    const int i0 = warp * part, i1 = min(p.K, i0 + part);
    int mine = 0;
    for (int i = i0; i < i1; i += 32) {
        const int j = i + lane < i1 ? __ldg(sel + i + lane) : -1;
        if (j >= nblk && rank == 0) raise_error(PKV_DEVERR_BLOCK);  // behind the context
        mine += __popc(__ballot_sync(0xffffffffu, j >= 0 && j < nblk));
    }
    if (lane == 0) count[warp] = mine;
    __syncthreads();
    int before = 0, total = 0;
    for (int w = 0; w <= W; ++w) {
        before += w < warp ? count[w] : 0;
        total += count[w];
    }
    const long long stages = (long long)total * spe;
    const int st0 = (int)(stages * rank / p.splits), st1n = (int)(stages * (rank + 1) / p.splits);
    const int e0 = st0 / spe, e1 = (st1n + spe - 1) / spe;  // entries of this CTA
    const int nst = aligned_window ? st1n - st0 : 0;
    for (int i = i0; i < i1 && before < e1; i += 32) {
        const int j = i + lane < i1 ? __ldg(sel + i + lane) : -1;
        const bool ok = j >= 0 && j < nblk;
        const uint32_t mask = __ballot_sync(0xffffffffu, ok);
        const int r = before + __popc(mask & ((1u << lane) - 1));
        if (ok && r >= e0 && r < e1) {
            const int blk = __ldg(p.block_tables + (size_t)s * p.MBS + j);
            int row = p.pool_rows;  // an id outside the pool reads the zero fill
            if (blk < 0 || blk >= p.NB) raise_error(PKV_DEVERR_BLOCK);
            else row = (blk * p.Hkv + h) * p.bs;
            list[r - e0] = make_int2(row, min(p.bs, n - j * p.bs));
        }
        before += __popc(mask);
    }
    __syncthreads();
    auto stage_valid = [&](int k, int &row) {  // stage k of this CTA: its first pool row and rows under the context
        const int t = st0 + k, e = t / spe, sub = t - e * spe;
        const int2 x = list[e - e0];
        row = min(x.x + sub * kStageTok, p.pool_rows);
        return min(kStageTok, x.y - sub * kStageTok);
    };

    if (warp == W) {
        // ------------------------------------------------------ producer --
        bool ok = true;
        int issued = 0;
        for (int k0 = 0; k0 < nst && ok; k0 += W) {
            bool lane_ok = true;
            const int k = k0 + lane;
            if (lane < W && k < nst) {
                const int slot = k % NS;
                lane_ok = wait_slot(&empty[slot], ((k / NS) & 1) ^ 1, abort_flag);
                if (lane_ok) {
                    int row;
                    const int valid = stage_valid(k, row);
                    if (valid > 0) {
                        const uint32_t kt = tiles + slot * R::kStage;
                        if constexpr (KV8) {
                            if (row < p.pool_rows) {
                                const int e = row / p.bs;  // block * Hkv + head
                                cp_async4(&slot_scales[slot].x, p.k_scales + e);
                                cp_async4(&slot_scales[slot].y, p.v_scales + e);
                                cp_async_mbar_arrive(&full[slot]);
                            } else {
                                slot_scales[slot] = make_float2(1.f, 1.f);
                                mbar_arrive(&full[slot]);
                            }
                        }
                        mbar_arrive_expect_tx(&full[slot], (uint32_t)R::kStage);
#pragma unroll
                        for (int hf = 0; hf < R::kBoxes; ++hf) {
                            const int x = hf * (R::kBoxRow / R::kElem);
                            tma_load_2d_u32(kt + hf * R::kHalfTile, &tmap_k, &full[slot], x, row);
                            tma_load_2d_u32(kt + R::kTile + hf * R::kHalfTile, &tmap_v, &full[slot], x, row);
                        }
                    } else {
                        mbar_arrive_count(&full[slot], kFullArrivals);
                    }
                }
            }
            ok = __all_sync(0xffffffffu, lane_ok);
            issued = min(nst, k0 + W);
        }
        // After a wait that gave up, what is in flight still has to land.
        if (!ok && lane == 0) {
            for (int c = max(0, issued - NS); c < issued; ++c)
                mbar_wait_bounded(&full[c % NS], (c / NS) & 1, kWaitLimitNs);
        }
    } else {
        // ------------------------------------------------------ consumer --
        const __nv_bfloat16 *qs = p.q + ((size_t)s * p.Hq + (size_t)h * p.g) * D;
        SimtState<D, KV8, KV8> st0s;
        MmaState<D, (PATH == 1 ? NT : 1), KV8, KV8> st1s;
        if constexpr (PATH == 0) {
            st0s.reset();
            st0s.load_q(qs, lane, p.scale_log2);
        } else {
            st1s.reset();
            st1s.load_q(qs, lane, p.g);
        }
        for (int k = warp; k < nst; k += W) {
            const int slot = k % NS;
            int row;
            const int valid = stage_valid(k, row);
            if (!wait_or_abort(&full[slot], (k / NS) & 1, abort_flag)) break;
            if (valid > 0) {
                const uint32_t kt = tiles + slot * R::kStage;
                const bool partial = valid < kStageTok;
                float ks = 1.f, vs = 1.f;
                if constexpr (KV8) {
                    const float2 sc = slot_scales[slot];
                    ks = sc.x;
                    vs = sc.y;
                }
                if constexpr (PATH == 0) {
                    if (partial) st0s.template stage<true>(kt, kt + R::kTile, valid, lane, ks, vs);
                    else st0s.template stage<false>(kt, kt + R::kTile, valid, lane, ks, vs);
                } else {
                    if (partial) st1s.template stage<true>(kt, kt + R::kTile, valid, lane, p.scale_log2 * ks, vs);
                    else st1s.template stage<false>(kt, kt + R::kTile, valid, lane, p.scale_log2 * ks, vs);
                }
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
        }
        if constexpr (PATH == 0) st0s.store_partial(mO, mM, mL, warp, lane, R::kMergeStride);
        else st1s.store_partial(mO, mM, mL, warp, lane, R::kMergeStride, GP, p.g);
    }
    __syncthreads();
    grid_launch_dependents();

    // The CTA's partial: element i of the g heads' rows.
    __nv_bfloat16 *out = p.out + ((size_t)s * p.Hq + (size_t)h * p.g) * D;
    for (int i = threadIdx.x; i < p.g * D; i += kDecodeThreads) {
        const int j = i / D, d = i - j * D;
        float M = PKV_NEG_INF, Ls = 0.f, O = 0.f;
#pragma unroll
        for (int u = 0; u < W; ++u) M = fmaxf(M, mM[u * GP + j]);
#pragma unroll
        for (int u = 0; u < W; ++u) {
            const float mu = mM[u * GP + j];
            const float f = mu == PKV_NEG_INF ? 0.f : exp2f(mu - M);
            Ls = fmaf(mL[u * GP + j], f, Ls);
            O = fmaf(mO[(u * GP + j) * R::kMergeStride + d], f, O);
        }
        if (p.splits == 1) {
            out[i] = __float2bfloat16_rn(Ls > 0.f || Ls != Ls ? O / Ls : 0.f);
        } else {
            cO[i] = O;
            if (d == 0) { cM[j] = M; cL[j] = Ls; }
        }
    }
    if (p.splits == 1) return;
    cluster_arrive();
    cluster_wait();
    for (int i = rank * kDecodeThreads + threadIdx.x; i < p.g * D; i += p.splits * kDecodeThreads) {
        const int j = i / D;
        float M = PKV_NEG_INF, Ls = 0.f, O = 0.f;
        for (int u = 0; u < p.splits; ++u) M = fmaxf(M, cluster_ld_f32(cluster_addr(cM + j, u)));
        for (int u = 0; u < p.splits; ++u) {
            const float mu = cluster_ld_f32(cluster_addr(cM + j, u));
            const float f = mu == PKV_NEG_INF ? 0.f : exp2f(mu - M);
            Ls = fmaf(cluster_ld_f32(cluster_addr(cL + j, u)), f, Ls);
            O = fmaf(cluster_ld_f32(cluster_addr(cO + i, u)), f, O);
        }
        out[i] = __float2bfloat16_rn(Ls > 0.f || Ls != Ls ? O / Ls : 0.f);
    }
    // a CTA's shared memory stays until its peers have read it
    cluster_arrive();
    cluster_wait();
}

}  // namespace pkv

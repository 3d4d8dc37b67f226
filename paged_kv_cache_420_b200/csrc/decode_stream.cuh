// decode_stream.cuh -- decode attention over a block-scaled 8-bit pool, and
// over selected blocks (bf16 or block-scaled 8-bit), for sm_100a.
//
// All 16-token stages of all (sequence, kv head) units form one line,
// sequence-major, and every consumer warp of the grid takes one contiguous
// stretch of it, all of the same cost (a stage counts 1, a unit kUnitCost more
// for its q, its first maxima and its output): no plan kernel, no work counter
// and no partition size, however the lengths are spread, from one long
// sequence to thousands of short ones.  A warp runs through the units of its
// stretch with one softmax state.  A unit that lies within a stretch is written
// out by its warp; the parts of a unit that stretches cut are merged in two
// steps, within the CTA (whose four stretches are neighbours), then, where a
// unit goes on over CTAs, through at most two records of each CTA that a second
// kernel merges.  Where all units are short, the stretches end between units,
// and there is nothing to merge; where units of equal length (selected blocks)
// are few, a cluster of CTAs takes each and merges its parts through
// distributed shared memory.
//
// Bound by HBM on long lines: 8 sequences of 32768 to 131072 tokens, 64 query
// heads on 8 (1.23 GB of codes), 199 to 205 us, 0.91 to 0.94 of the measured
// copy rate; the warps of a fast CTA end 25% before those of the slowest, since
// the stretches are fixed.  128 MHA sequences of 16 to 2048 tokens (0.53 GB) 101
// us, 0.80.  Short lines are bound by the chain of loads before the first stage
// (context, table, tiles: 4 us) and the merge.
//
//   dense:    unit (s, h) has ceil(context / 16) stages; each CTA adds up the
//             contexts itself (they are few, and in L2)
//   selected: unit (s, h) has K entries of block_size / 16 stages each
//
// In a CTA one producer warp feeds four rings, one for each consumer warp: 8
// of its lanes look up the next 8 stages of each stretch (table entries, and
// the selection before them) a group ahead, and issue their TMA loads, the
// scales of the stage's block (cp.async) and, where a unit begins, a prefetch
// of its q.
#pragma once

#include "decode.cuh"
#include "even_cut.cuh"

namespace pkv {

// ----------------------------------------------------------- instructions ----

// A 4-byte asynchronous copy global -> shared, and an arrival on `bar` once the
// calling thread's earlier ones have landed (one of the barrier's expected
// arrivals).
__device__ __forceinline__ void cp_async4(void *smem_dst, const void *gmem_src) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4;" ::"r"(smem_u32(smem_dst)), "l"(gmem_src) : "memory");
}
__device__ __forceinline__ void cp_async_mbar_arrive(uint64_t *bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Barrier of all threads of the cluster; what one wrote before it (its shared
// memory included) the others see after it.
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// Address of the same shared variable in CTA `rank` of the cluster, and loads
// from there.
__device__ __forceinline__ uint32_t cluster_addr(const void *p, uint32_t rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}
__device__ __forceinline__ float cluster_ld_f32(uint32_t addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(addr) : "memory");
    return v;
}
__device__ __forceinline__ float4 cluster_ld_f32x4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
                 : "r"(addr)
                 : "memory");
    return v;
}

// ------------------------------------------------------------- arithmetic ----

// Where the references begin: the least finite number, so that a score of
// -infinity weighs 0 from the first stage on (-infinity would leave NaN there).
constexpr float kNoScore = -3.402823466e38f;

// e4m3 pool: a weight times its V scale is at most 2^kRescaleSlack of its
// reference and enters the weighted sum as f16 times 2^kWeightUp, at most 2^15.
// f16's normal range ends at 2^-14 and its spacing below is 2^-24: a product keeps
// 11 bits down to 2^-21 of the reference and is dropped below 2^-32 of it only, so
// 2^20 rows that are dropped next to one that is not are 2^-12 of the sum.
// Without the factor they were dropped below 2^-25, 131072 rows of them 2^-8.
constexpr float kWeightUp = 7.0f;
static_assert(kRescaleSlack + kWeightUp < 16.f, "f16 holds the largest product");

// The power of two that brings a largest magnitude into [2^14, 2^15) (below that
// for less than 2^-112): q is converted to f16 with it, so that an element keeps
// its 8 bits down to 2^-31 of the head's largest whatever their size.  The inverse,
// for the scores, is exact too.
__device__ __forceinline__ void unit_power(float amax, float &down, float &up) {
    const int e = min(max((int)(__float_as_uint(amax) >> 23), 15), 254);
    down = __uint_as_float((uint32_t)(268 - e) << 23);
    up = __uint_as_float((uint32_t)(e - 14) << 23);
}

__device__ __forceinline__ float ex2(float x) {  // 2^x; results below 2^-126 are 0
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Byte address of e4m3 element (row r, column c) of a stage tile: one 128-byte
// line per row at head dim 128, 16-byte chunks XOR-swizzled with (r & 7); two
// 64-byte rows per line at 64, chunks XOR-swizzled with the line's number.
template <int D>
__device__ __forceinline__ uint32_t tile_addr_e4m3(uint32_t tile, int r, int c) {
    if constexpr (D == 64) return tile + r * 64 + ((((c >> 4) ^ ((r >> 1) & 3))) << 4) + (c & 15);
    return tile_addr8(tile, r, c);
}

// The attention of one warp over stages of 16 tokens, for the g <= 8 NT query
// heads of a kv head, on the tensor cores (a single head as well: the products
// of the unused columns are free, and the CUDA-core form takes twice the
// instructions):
//   S^T[16 tokens][8 heads] = K Q^T,  O^T[D][8 heads] += V^T P^T
// in the fragment layouts of MmaState.  Beside HBM its instructions bound it, not
// the tensor cores (issue 50%, tensor pipe 19% on long lines; a warp can issue one
// in four cycles at best), so what is done for each stage beside the products and
// conversions is kept small.
//
// bf16 pool: the weights enter the second product as a sum of two bf16 (16
// bits): twice the products, which are free.  Both are above zero, the first cut
// off instead of rounded and the last bit of the weight set, so that an infinite
// V gives an infinite sum: beside a negative or a zero second one it gave NaN.
//
// e4m3 pool, scales ks and vs of the stage's block: the codes are exact as
// f16, and a stage's tokens are taken in perm16 order.  ks multiplies the
// summed scores.  vs is a part of a token's weight, 2^(z - m) vs, and blocks
// may differ in it by any power of two, while the weight is used as f16: so O
// has references of its own, m2 ~ max(z + log2 vs), and holds
// sum 2^(z + log2 vs - m2 + kWeightUp) code, beside m and l of the softmax.  m2 is
// kept as r = m2 - m, and a score used by its distance from m, which is exact near
// m: with scores of 2^23 and more a sum z + log2 vs would lose the scale, and O a
// power of two against l.
//
// Both references are raised only when a value exceeds them by kRescaleSlack
// (weights stay below 2^8), so a stage compares its values with one threshold
// for each head and votes; the maxima are worked out only in the stages that
// raise one.
template <int D, int NT, bool KV8>
struct TileState {
    static constexpr int KS = D / 16;  // k-steps of K Q^T
    static constexpr int MT = D / 16;  // m-tiles of O^T
    static constexpr int KL = KV8 ? KS / 2 : KS;  // matrix loads of a K tile
    uint32_t qb[NT][KS][2];  // B fragments of Q^T
    float o[NT][MT][4];      // O^T accumulators
    float m[NT][2];          // reference of the scores of heads nt*8 + 2*(lane%4) + {0,1}
    float r[NT][2];          // e4m3: of the columns of O^T, less m
    float l[NT][2];          // this thread's share of the sums
    float sc[NT][2];         // e4m3: scale * log2 e times the power of two that a head's q was divided by

    __device__ __forceinline__ void reset() {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) { m[nt][c] = kNoScore; r[nt][c] = 0.f; l[nt][c] = 0.f; }
#pragma unroll
            for (int mt = 0; mt < MT; ++mt)
#pragma unroll
                for (int c = 0; c < 4; ++c) o[nt][mt][c] = 0.f;
        }
    }

    // B fragment of Q^T (k = head dim, n = head); heads >= g are zero.  e4m3:
    // k slots 2j, 2j+1, 2j+8, 2j+9 hold columns 4j .. 4j+3.
    __device__ __forceinline__ void load_q(const __nv_bfloat16 *q, int lane, int g, float scale_log2) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            const int head = nt * 8 + (lane >> 2);
            const __nv_bfloat16 *row = q + head * D + (KV8 ? 4 : 2) * (lane & 3);
#pragma unroll
            for (int kk = 0; kk < KS; ++kk) {
                qb[nt][kk][0] = qb[nt][kk][1] = 0u;
                if (head < g) {
                    if constexpr (KV8) {
                        const uint2 x = __ldg(reinterpret_cast<const uint2 *>(row + kk * 16));
                        qb[nt][kk][0] = x.x;
                        qb[nt][kk][1] = x.y;
                    } else {
                        qb[nt][kk][0] = __ldg(reinterpret_cast<const uint32_t *>(row + kk * 16));
                        qb[nt][kk][1] = __ldg(reinterpret_cast<const uint32_t *>(row + kk * 16 + 8));
                    }
                }
            }
            if constexpr (KV8) {
                float amax = 0.f;
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        amax = fmaxf(amax, fmaxf(fabsf(bf16lo_to_f32(qb[nt][kk][c])), fabsf(bf16hi_to_f32(qb[nt][kk][c]))));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
                amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
                float down, up;
                unit_power(amax, down, up);
#pragma unroll
                for (int kk = 0; kk < KS; ++kk)
#pragma unroll
                    for (int c = 0; c < 2; ++c)
                        qb[nt][kk][c] = f16x2_from_f32(bf16lo_to_f32(qb[nt][kk][c]) * down,
                                                       bf16hi_to_f32(qb[nt][kk][c]) * down);
                // this lane's columns of S^T are heads 2 (lane % 4) + c
#pragma unroll
                for (int c = 0; c < 2; ++c)
                    sc[nt][c] = scale_log2 * __shfl_sync(0xffffffffu, up, (2 * (lane & 3) + c) * 4);
            }
        }
    }

    // Raises the references that a stage's values exceed (all lanes).
    __device__ __forceinline__ void raise(const float (&z)[NT][4], float lv) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float mx = fmaxf(z[nt][c], z[nt][c + 2]);
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 4));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 8));
                mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 16));
                float fo = 1.f, d = mx - m[nt][c];
                if (d > kRescaleSlack) {
                    const float f = ex2(-d);
                    m[nt][c] = mx;
                    r[nt][c] -= d;
                    d = 0.f;
                    l[nt][c] *= f;
                    if constexpr (!KV8) fo = f;
                }
                if constexpr (KV8) {
                    if (d + lv - r[nt][c] > kRescaleSlack) {
                        fo = ex2(r[nt][c] - (d + lv));
                        r[nt][c] = d + lv;
                    }
                }
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    o[nt][mt][c] *= fo;
                    o[nt][mt][c + 2] *= fo;
                }
            }
        }
    }

    // PARTIAL: fewer than 16 valid tokens; only then are scores past `valid`
    // masked and the V operand's rows of those tokens zeroed.  scale: scale *
    // log2 e (bf16).  The tiles are 1 KB-aligned, so a lane's addresses in
    // them differ by an exclusive or.
    template <bool PARTIAL>
    __device__ __forceinline__ void stage(uint32_t ktile, uint32_t vtile, int valid, int lane, float scale, float ks,
                                          float vs) {
        const int mi = lane >> 3, ri = lane & 7;
        uint32_t ka[KL][4], va[MT][KV8 ? 2 : 4];
        {
            const uint32_t at = KV8 ? tile_addr_e4m3<D>(ktile, perm16(ri + 8 * (mi & 1)), 16 * (mi >> 1))
                                    : tile_addr(ktile, ri + 8 * (mi & 1), 8 * (mi >> 1));
#pragma unroll
            for (int i = 0; i < KL; ++i)
                ldmatrix_x4(KV8 ? at ^ (32 * i) : (at ^ (32 * (i & 3))) + (i >> 2) * (kStageTok * 128), ka[i][0], ka[i][1],
                            ka[i][2], ka[i][3]);
        }
        // two chains of products (even / odd k-steps), added after
        float s[NT][4], s2[NT][4];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 4; ++c) { s[nt][c] = 0.f; s2[nt][c] = 0.f; }
#pragma unroll
        for (int kk = 0; kk < KS; ++kk) {
            uint32_t a0, a1, a2, a3;
            if constexpr (KV8) {
                f16x2_from_e4m3x4(ka[kk / 2][2 * (kk & 1)], a0, a2);
                f16x2_from_e4m3x4(ka[kk / 2][2 * (kk & 1) + 1], a1, a3);
            } else {
                a0 = ka[kk][0]; a1 = ka[kk][1]; a2 = ka[kk][2]; a3 = ka[kk][3];
            }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float(&acc)[4] = (kk & 1) ? s2[nt] : s[nt];
                if constexpr (KV8) mma_f16_16816(acc[0], acc[1], acc[2], acc[3], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
                else mma_bf16_16816(acc[0], acc[1], acc[2], acc[3], a0, a1, a2, a3, qb[nt][kk][0], qb[nt][kk][1]);
            }
        }
        // the V operands are on their way while the weights are worked out
        {
            const uint32_t at = KV8 ? tile_addr_e4m3<D>(vtile, lane & 15, 0)
                                    : tile_addr(vtile, ri + 8 * (mi >> 1), 8 * (mi & 1));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                if constexpr (KV8) ldmatrix_b8_trans(at ^ (16 * mt), va[mt][0], va[mt][1]);
                else ldmatrix_x4_trans((at ^ (32 * (mt & 3))) + (mt >> 2) * (kStageTok * 128), va[mt][0], va[mt][1], va[mt][2],
                                       va[mt][3]);
            }
        }
        const int t0 = lane >> 2;  // rows t0 and t0 + 8 of S^T
        const bool ok0 = !PARTIAL || (KV8 ? perm16(t0) : t0) < valid;
        const bool ok1 = !PARTIAL || (KV8 ? perm16(t0 + 8) : t0 + 8) < valid;
        float lv = 0.f;
        if constexpr (KV8) lv = vs > 0.f ? __log2f(vs) : -1000.f;  // a scale that is not above zero holds no value
        float z[NT][4];
        bool over = false;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float f = KV8 ? sc[nt][c] * ks : scale;
                z[nt][c] = ok0 ? (s[nt][c] + s2[nt][c]) * f : PKV_NEG_INF;
                z[nt][c + 2] = ok1 ? (s[nt][c + 2] + s2[nt][c + 2]) * f : PKV_NEG_INF;
                const float top = (KV8 ? fminf(0.f, r[nt][c] - lv) : 0.f) + kRescaleSlack;
                over |= fmaxf(z[nt][c], z[nt][c + 2]) - m[nt][c] > top;
            }
        if (__any_sync(0xffffffffu, over)) raise(z, lv);
        uint32_t pb[NT][2], pc[KV8 ? 1 : NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float p[4];
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                const float d0 = z[nt][c] - m[nt][c], d1 = z[nt][c + 2] - m[nt][c];
                p[c] = ex2(d0);
                p[c + 2] = ex2(d1);
                l[nt][c] += p[c] + p[c + 2];
                if constexpr (KV8) {
                    const float up = lv - r[nt][c] + kWeightUp;
                    p[c] = ex2(d0 + up);
                    p[c + 2] = ex2(d1 + up);
                }
            }
            // accumulator layout (token row, head pair) -> operand layout of P^T
            if constexpr (KV8) {
                pb[nt][0] = movmatrix_trans(f16x2_from_f32(p[0], p[1]));
                pb[nt][1] = movmatrix_trans(f16x2_from_f32(p[2], p[3]));
            } else {
#pragma unroll
                for (int c = 0; c < 4; ++c) p[c] = __uint_as_float(__float_as_uint(p[c]) | 1u);
                const uint32_t h0 = __byte_perm(__float_as_uint(p[0]), __float_as_uint(p[1]), 0x7632);
                const uint32_t h1 = __byte_perm(__float_as_uint(p[2]), __float_as_uint(p[3]), 0x7632);
                pb[nt][0] = movmatrix_trans(h0);
                pb[nt][1] = movmatrix_trans(h1);
                pc[nt][0] = movmatrix_trans(pack_bf16x2(p[0] - bf16lo_to_f32(h0), p[1] - bf16hi_to_f32(h0)));
                pc[nt][1] = movmatrix_trans(pack_bf16x2(p[2] - bf16lo_to_f32(h1), p[3] - bf16hi_to_f32(h1)));
            }
        }
        // token masks of this thread's V^T operand halves
        uint32_t mask01 = 0xffffffffu, mask23 = 0xffffffffu;
        if constexpr (PARTIAL) {
            const int j0 = KV8 ? 4 * (lane & 3) : 2 * (lane & 3);
            const int j2 = KV8 ? j0 + 2 : j0 + 8;
            mask01 = (j0 < valid ? 0x0000ffffu : 0u) | (j0 + 1 < valid ? 0xffff0000u : 0u);
            mask23 = (j2 < valid ? 0x0000ffffu : 0u) | (j2 + 1 < valid ? 0xffff0000u : 0u);
        }
#pragma unroll
        for (int mt = 0; mt < MT; ++mt) {
            uint32_t a0, a1, a2, a3;
            if constexpr (KV8) {
                f16x2_from_e4m3x4(va[mt][0], a0, a2);  // d = l/4: tokens 4j, 4j+1 and 4j+2, 4j+3
                f16x2_from_e4m3x4(va[mt][1], a1, a3);  // d = l/4 + 8
            } else {
                a0 = va[mt][0]; a1 = va[mt][1]; a2 = va[mt][2]; a3 = va[mt][3];
            }
            if constexpr (PARTIAL) { a0 &= mask01; a1 &= mask01; a2 &= mask23; a3 &= mask23; }
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
                float(&acc)[4] = o[nt][mt];
                if constexpr (KV8) {
                    mma_f16_16816(acc[0], acc[1], acc[2], acc[3], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                } else {
                    mma_bf16_16816(acc[0], acc[1], acc[2], acc[3], a0, a1, a2, a3, pb[nt][0], pb[nt][1]);
                    mma_bf16_16816(acc[0], acc[1], acc[2], acc[3], a0, a1, a2, a3, pc[nt][0], pc[nt][1]);
                }
            }
        }
    }

    // l summed over its lanes, and what brings a column of O^T to reference m:
    // f twice, each half of the exponent, since the whole leaves fp32's range where
    // V's scales lie at its ends (2^-126 is a block's of zeros).
    __device__ __forceinline__ void finish(int nt, int c, float &lsum, float &f) {
        lsum = l[nt][c];
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 4);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 8);
        lsum += __shfl_xor_sync(0xffffffffu, lsum, 16);
        f = KV8 ? ex2(0.5f * (r[nt][c] - kWeightUp)) : 1.f;
    }

    // This warp's part (m, l, O) of a unit: rows of `stride` floats.
    __device__ __forceinline__ void store_part(float *acc, int stride, float *pm, float *pl, int lane, int g) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float lsum, f;
                finish(nt, c, lsum, f);
                const int head = nt * 8 + 2 * (lane & 3) + c;
                if (head >= g) continue;
                if (lane < 4) { pm[head] = m[nt][c]; pl[head] = lsum; }
                float *row = acc + head * stride + (lane >> 2);
#pragma unroll
                for (int mt = 0; mt < MT; ++mt) {
                    row[mt * 16] = KV8 ? o[nt][mt][c] * f * f : o[nt][mt][c];
                    row[mt * 16 + 8] = KV8 ? o[nt][mt][c + 2] * f * f : o[nt][mt][c + 2];
                }
            }
    }

    // The normalised rows of a unit that this warp took alone.
    __device__ __forceinline__ void write_out(__nv_bfloat16 *out, int lane, int g) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
            float f[2], fl[2];  // O f fl is the row
#pragma unroll
            for (int c = 0; c < 2; ++c) {
                float lsum;
                finish(nt, c, lsum, f[c]);
                fl[c] = lsum > 0.f || lsum != lsum ? __fdividef(f[c], lsum) : 0.f;
            }
            auto value = [&](float x, int c) { return KV8 ? x * f[c] * fl[c] : x * fl[c]; };
            const int head = nt * 8 + (lane >> 2);  // after the transpose
            uint32_t *row = reinterpret_cast<uint32_t *>(out + head * D + 2 * (lane & 3));
#pragma unroll
            for (int mt = 0; mt < MT; ++mt) {
                const uint32_t x = movmatrix_trans(pack_bf16x2(value(o[nt][mt][0], 0), value(o[nt][mt][1], 1)));
                const uint32_t y = movmatrix_trans(pack_bf16x2(value(o[nt][mt][2], 0), value(o[nt][mt][3], 1)));
                if (head < g) {
                    row[mt * 8] = x;
                    row[mt * 8 + 4] = y;
                }
            }
        }
    }
};

// ------------------------------------------------------------------- work ----

constexpr int kUnitCost = 2;     // of a unit, in stages
constexpr int kMinCost = 4;      // of a stretch, while there is less work than fills the grid
constexpr int kStreamMaxSplit = 8;
constexpr int kStreamGroup = 8;  // stages that a stretch's lanes look up at once
static_assert(kConsumerWarps * kStreamGroup == 32, "a lane of the producer for each stage of a group");

struct StreamParams {
    const __nv_bfloat16 *q;       // [B][Hq][D]
    __nv_bfloat16 *out;           // [B][Hq][D]
    const int32_t *block_tables;  // [B][MBS]
    const int32_t *context_lens;  // [B]
    const int32_t *selected;      // [B][Hkv][K] (selected blocks only)
    const float *k_scales;        // [NB][Hkv] (e4m3 pool)
    const float *v_scales;
    float *cut;                   // workspace: [CTAs][W][g][D], the parts at the beginnings of warps' stretches
    int2 *meta;                   // workspace: [CTAs] (a unit that ends in the CTA and began in another, or -1; that CTA)
    float2 *rec_ml;               // workspace: [CTAs][2][g] = (m, l)
    float *rec_acc;               // workspace: [CTAs][2][g][D]
    int B, Hq, Hkv, g, MBS, bs, NB, K, max_ctx;
    int pool_rows;
    int whole;       // stretches end between units
    int split;       // selected: CTAs of a cluster that take a unit; 0: the line is cut anywhere
    float scale_log2;
};

// A part of a unit that a warp leaves behind.
struct StreamPart {
    int unit;
    int from;  // the CTA in which the unit began, if it ends in this part; else -1
    int begins;  // whether the unit begins in this part
};

// Where a stretch begins: a stage of the line, the sequence it lies in, and the
// stages and the cost of the line before that sequence.
struct StreamBound {
    long long x, base, cost_base;
    int seq;
};

// What a consumer has to know of a stage.
struct __align__(16) StreamStage {
    int unit;
    int valid;  // tokens; 0: none (nothing was loaded)
    int first;  // the first of its unit in this stretch: fresh state and q
    // The last of its unit in this stretch: 0 no, 1 the unit is complete, 2 its
    // beginning was cut off, 4 its end is cut off, 8 + c: it began in CTA c and
    // ends here.
    int last;
};

template <int D, int GP, int NS, bool KV8>
struct StreamSmem {
    static constexpr int kW = kConsumerWarps;
    static constexpr int kElem = KV8 ? 1 : 2;                           // bytes per K/V element
    static constexpr int kBoxRow = D * kElem < 128 ? D * kElem : 128;   // bytes of a TMA box's row
    static constexpr int kBox = kStageTok * kBoxRow;
    static constexpr int kBoxes = D * kElem / kBoxRow;
    static constexpr int kTile = kStageTok * D * kElem;                 // a K (or V) tile
    static constexpr int kStage = 2 * kTile;
    static constexpr int kStride = D + 4;                               // floats of a part's row, padded against bank conflicts
    static constexpr int kPart = GP * kStride * 4;
    static constexpr int oTiles = 0;                                    // the rings; the parts at the stretches' ends reuse them
    static constexpr int oM = oTiles + NS * kStage;                     // [2 W][GP]: of the parts at the beginnings, then the ends
    static constexpr int oL = oM + 2 * kW * GP * 4;
    static constexpr int oFactor = oL + 2 * kW * GP * 4;
    static constexpr int oPartInfo = oFactor + 2 * kW * GP * 4;         // StreamPart [2 W]
    static constexpr int oGroups = oPartInfo + 2 * kW * (int)sizeof(StreamPart);  // int [1 + 2 W]: neighbouring parts of one unit
    static constexpr int oBars = (oGroups + (1 + 2 * kW) * 4 + 7) / 8 * 8;
    static constexpr int oScales = oBars + 2 * NS * 8;
    static constexpr int oInfo = (oScales + (KV8 ? NS * 8 : 0) + 15) / 16 * 16;
    static constexpr int oScan = oInfo + NS * 16;                       // long long [threads][2]: stages, cost
    static constexpr int oWarpSum = oScan + kDecodeThreads * 16;
    static constexpr int oBounds = oWarpSum + (kW + 1) * 16;            // StreamBound [W + 1]
    static constexpr int oAbort = oBounds + (kW + 1) * (int)sizeof(StreamBound);
    static constexpr int kBytes = oAbort + 16;
    static constexpr int oOwn = kW * kPart;  // split: the CTA's partial, behind the parts in the rings
    static_assert(oOwn % 16 == 0 && oOwn + GP * (D + 2) * 4 <= NS * kStage,
                  "the parts at the stretches' ends and the CTA's partial fit into the rings");
};

// CTAs of an SM that the registers must allow.
constexpr int stream_min_ctas(int D, int GPAD, bool KV8) { return GPAD > 8 ? (D == 64 ? 3 : 2) : KV8 ? 4 : 3; }

template <int D, int GPAD, int NS, bool KV8, bool SEL>
__global__ void __launch_bounds__(kDecodeThreads, stream_min_ctas(D, GPAD, KV8))
    stream_decode_kernel(const __grid_constant__ CUtensorMap tmap_k, const __grid_constant__ CUtensorMap tmap_v,
                         const StreamParams p) {
    constexpr int W = kConsumerWarps;
    constexpr int GP = GPAD;
    constexpr int NT = (GPAD + 7) / 8;
    constexpr int DEPTH = NS / W;  // slots of a ring
    constexpr int kFullArrivals = KV8 ? 2 : 1;
    using L = StreamSmem<D, GP, NS, KV8>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *smem = smem_raw;
    uint64_t *full = reinterpret_cast<uint64_t *>(smem + L::oBars);
    uint64_t *empty = full + NS;
    float2 *slot_scales = reinterpret_cast<float2 *>(smem + L::oScales);
    StreamStage *info = reinterpret_cast<StreamStage *>(smem + L::oInfo);
    StreamPart *part_info = reinterpret_cast<StreamPart *>(smem + L::oPartInfo);
    float *mM = reinterpret_cast<float *>(smem + L::oM);
    float *mL = reinterpret_cast<float *>(smem + L::oL);
    int *groups = reinterpret_cast<int *>(smem + L::oGroups);
    longlong2 *scan = reinterpret_cast<longlong2 *>(smem + L::oScan);
    longlong2 *warp_sum = reinterpret_cast<longlong2 *>(smem + L::oWarpSum);
    StreamBound *bounds = reinterpret_cast<StreamBound *>(smem + L::oBounds);
    volatile int *abort_flag = reinterpret_cast<volatile int *>(smem + L::oAbort);
    const uint32_t tiles = smem_u32(smem + L::oTiles);
    float *factor = reinterpret_cast<float *>(smem + L::oFactor);
    // Part i of the CTA: 0 .. W - 1 at a stretch's beginning, which is put into
    // the workspace while the warp goes on, W .. 2 W - 1 at its end.
    float *cut = p.cut + (size_t)blockIdx.x * W * p.g * D;
    float *ends = reinterpret_cast<float *>(smem + L::oTiles);

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int i = 0; i < NS; ++i) { mbar_init(&full[i], kFullArrivals); mbar_init(&empty[i], 1); }
        *abort_flag = 0;
        fence_mbar_init();
        tma_prefetch_desc(&tmap_k);
        tma_prefetch_desc(&tmap_v);
        if ((smem_u32(smem_raw) & 1023u) != 0) {  // the swizzle pattern repeats every 1 KB
            raise_error(PKV_DEVERR_LAYOUT);
            *abort_flag = 1;
        }
    }
    if (tid < 2 * W) part_info[tid].unit = -1;
    grid_dependency_wait();

    const long long ctx_cap = min((long long)p.MBS * p.bs, (long long)p.max_ctx);
    auto context = [&](int s, bool report) -> int {
        const int n = __ldg(p.context_lens + s);
        if (n < 0 || n > ctx_cap) {
            if (report) raise_error(PKV_DEVERR_CONTEXT);
            return n < 0 ? 0 : (int)ctx_cap;
        }
        return n;
    };
    const int spe = p.bs / kStageTok;  // stages of a block
    const int per = (p.B + kDecodeThreads - 1) / kDecodeThreads;  // sequences whose stages a thread adds up
    auto stages_of = [&](int n) { return n / kStageTok + (n % kStageTok != 0); };
    longlong2 total;  // stages, cost
    if constexpr (SEL) {
        total.x = total.y = (long long)p.B * p.Hkv * p.K * spe;
        if (blockIdx.x == 0)
            for (int s = tid; s < p.B; s += kDecodeThreads) context(s, true);
    } else {
        longlong2 sum = make_longlong2(0, 0);
        for (int s = tid * per; s < min(p.B, (tid + 1) * per); ++s) {
            const int nst = stages_of(context(s, blockIdx.x == 0));
            sum.x += nst;
            sum.y += nst > 0 ? nst + kUnitCost : 0;
        }
        sum.x *= p.Hkv;
        sum.y *= p.Hkv;
        longlong2 incl = sum;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const long long x = __shfl_up_sync(0xffffffffu, incl.x, o), y = __shfl_up_sync(0xffffffffu, incl.y, o);
            if (lane >= o) { incl.x += x; incl.y += y; }
        }
        if (lane == 31) warp_sum[warp] = incl;
        __syncthreads();
        longlong2 before = make_longlong2(0, 0);
        total = before;
        for (int w = 0; w <= W; ++w) {
            if (w < warp) { before.x += warp_sum[w].x; before.y += warp_sum[w].y; }
            total.x += warp_sum[w].x;
            total.y += warp_sum[w].y;
        }
        // what lies before this thread's sequences
        scan[tid] = make_longlong2(before.x + incl.x - sum.x, before.y + incl.y - sum.y);
        // empty sequences get a zero row
        const int vec = p.Hq * D / 8;
        for (int s = blockIdx.x; s < p.B; s += gridDim.x)
            if (context(s, false) == 0)
                for (int i = tid; i < vec; i += kDecodeThreads)
                    reinterpret_cast<uint4 *>(p.out)[(size_t)s * vec + i] = make_uint4(0, 0, 0, 0);
    }
    const int ctas = SEL && p.split ? gridDim.x : (int)max(1ll, min((long long)gridDim.x, total.y / (W * kMinCost)));
    if ((int)blockIdx.x >= ctas || total.x == 0) {
        if (tid == 0) p.meta[blockIdx.x] = make_int2(-1, 0);
        return;
    }
    const EvenCut line(total.y, ctas);
    __syncthreads();
    // The bounds of the warps' stretches: thread t finds the stage at cost y.
    if (tid <= W) {
        const long long A = line.begin(blockIdx.x), E = line.begin(blockIdx.x + 1);
        const long long y = A + (E - A) * tid / W;
        StreamBound bd;
        if constexpr (SEL) {
            const int len_u = p.K * spe, unit = p.split ? blockIdx.x / p.split : 0, part = p.split ? blockIdx.x % p.split : 0;
            bd.x = p.split ? (long long)unit * len_u + (long long)len_u * (part * W + tid) / (p.split * W) : y;
            bd.seq = 0;
            bd.base = bd.cost_base = 0;
        } else {
            int lo = 0, hi = kDecodeThreads - 1;  // the last thread whose sequences begin at or before y
            while (lo < hi) {
                const int mid = (lo + hi + 1) >> 1;
                if (scan[mid].y <= y) lo = mid; else hi = mid - 1;
            }
            bd.seq = min(lo * per, p.B - 1);
            bd.base = scan[lo].x;
            bd.cost_base = scan[lo].y;
            bd.x = total.x;
            for (int s = bd.seq; s < p.B && y < total.y; ++s) {
                const int nst = stages_of(context(s, false)), cost = nst > 0 ? nst + kUnitCost : 0;
                const long long off = y - bd.cost_base;
                if (off < (long long)cost * p.Hkv) {
                    const int h = (int)quotient(off, cost), in = (int)(off - (long long)h * cost);
                    const int i = p.whole ? (2 * in > cost ? nst : 0) : max(0, in - kUnitCost);
                    bd.seq = s;
                    bd.x = bd.base + (long long)h * nst + i;
                    break;
                }
                bd.base += (long long)nst * p.Hkv;
                bd.cost_base += (long long)cost * p.Hkv;
            }
        }
        bounds[tid] = bd;
    }
    __syncthreads();

    if (warp == W) {
        // ------------------------------------------------------ producer --
        const int j = lane / kStreamGroup, sub = lane % kStreamGroup;
        const long long a = bounds[j].x, b = bounds[j + 1].x;
        const int len = (int)(b - a);
        int longest = len;
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, 8));
        longest = max(longest, __shfl_xor_sync(0xffffffffu, longest, 16));
        // dense: this lane's sequence, and the line before it
        int cs = bounds[j].seq, n = SEL ? 0 : context(cs, false), nst = stages_of(n);
        long long base = bounds[j].base, cost_base = bounds[j].cost_base;
        struct Stage {
            StreamStage st;
            int row;
        };
        // stage k of this lane's stretch
        auto look_up = [&](int k) -> Stage {
            Stage r;
            r.row = p.pool_rows;
            r.st.unit = 0; r.st.valid = 0; r.st.first = 0; r.st.last = 0;
            if (k >= len) return r;
            const long long x = a + k;
            int s, h, i, len_u;  // stage i of len_u of unit (s, h)
            if constexpr (SEL) {
                len_u = p.K * spe;
                const long long unit = quotient(x, len_u);
                i = (int)(x - unit * len_u);
                s = (int)(unit / p.Hkv);
                h = (int)(unit - (long long)s * p.Hkv);
            } else {
                while (x >= base + (long long)nst * p.Hkv) {
                    base += (long long)nst * p.Hkv;
                    cost_base += nst > 0 ? (long long)(nst + kUnitCost) * p.Hkv : 0;
                    n = context(++cs, false);
                    nst = stages_of(n);
                }
                s = cs;
                len_u = nst;
                const long long off = x - base;
                h = (int)quotient(off, nst);
                i = (int)(off - (long long)h * nst);
            }
            r.st.unit = s * p.Hkv + h;
            const bool begins = x - i >= a, ends = x - i + len_u <= b;
            r.st.first = i == 0 || k == 0;
            if (r.st.first)  // its q, for the consumer's loads
                for (int y = 0; y < p.g * D * 2; y += 128)
                    asm volatile("prefetch.global.L1 [%0];" ::"l"(reinterpret_cast<const uint8_t *>(p.q) + (size_t)r.st.unit * p.g * D * 2 + y));
            r.st.last = i == len_u - 1 || k == len - 1 ? (begins ? (ends ? 1 : 4) : 2) : 0;
            if (r.st.last == 2 && ends) {
                // it began in the last CTA whose bound is not behind its first stage
                const long long y0 = SEL ? x - i : cost_base + (long long)h * (len_u + kUnitCost) + kUnitCost;
                r.st.last = 8 + (SEL && p.split ? 0 : line.part_of(y0));
            }
            int blk = i / spe, off_blk = (i - blk * spe) * kStageTok;  // logical block, token in it
            if constexpr (SEL) {
                n = context(s, false);
                const int e = blk;
                blk = __ldg(p.selected + (size_t)r.st.unit * p.K + e);
                if (blk < 0) return r;
                if (blk >= n / p.bs + (n % p.bs != 0)) {  // behind the context
                    raise_error(PKV_DEVERR_BLOCK);
                    return r;
                }
            }
            r.st.valid = min(kStageTok, n - blk * p.bs - off_blk);
            if (r.st.valid <= 0) {
                r.st.valid = 0;
                return r;
            }
            const int id = __ldg(p.block_tables + (size_t)s * p.MBS + blk);
            if (id < 0 || id >= p.NB) raise_error(PKV_DEVERR_BLOCK);  // reads the zero fill
            else r.row = (id * p.Hkv + h) * p.bs + off_blk;
            return r;
        };
        bool ok = true;
        int issued = 0;
        Stage next = look_up(sub);
        for (int k0 = 0; k0 < longest && ok; k0 += kStreamGroup) {
            const Stage cur = next;
            next = look_up(k0 + kStreamGroup + sub);
            for (int t = 0; t < kStreamGroup && ok; ++t) {
                const int k = k0 + t;
                bool lane_ok = true;
                if (sub == t && k < len) {
                    const int slot = j * DEPTH + k % DEPTH;
                    lane_ok = wait_slot(&empty[slot], ((k / DEPTH) & 1) ^ 1, abort_flag);
                    if (lane_ok) {
                        info[slot] = cur.st;
                        const bool load = cur.st.valid > 0;
                        if constexpr (KV8) {
                            if (load && cur.row < p.pool_rows) {
                                const int e = cur.row / p.bs;  // block * Hkv + head
                                cp_async4(&slot_scales[slot].x, p.k_scales + e);
                                cp_async4(&slot_scales[slot].y, p.v_scales + e);
                                cp_async_mbar_arrive(&full[slot]);
                            } else {
                                slot_scales[slot] = make_float2(1.f, 1.f);
                                mbar_arrive(&full[slot]);
                            }
                        }
                        mbar_arrive_expect_tx(&full[slot], load ? (uint32_t)L::kStage : 0u);
                        if (load) {
                            const uint32_t kt = tiles + slot * L::kStage;
#pragma unroll
                            for (int hf = 0; hf < L::kBoxes; ++hf) {
                                const int x = hf * (L::kBoxRow / L::kElem);
                                tma_load_2d_u32(kt + hf * L::kBox, &tmap_k, &full[slot], x, cur.row);
                                tma_load_2d_u32(kt + L::kTile + hf * L::kBox, &tmap_v, &full[slot], x, cur.row);
                            }
                        }
                        issued = k + 1;
                    }
                }
                ok = __all_sync(0xffffffffu, lane_ok);
            }
        }
        named_barrier_sync(1, kDecodeThreads);  // the consumers are through
        // After a wait that gave up, what this lane has in flight still has to land.
        if (*abort_flag)
            for (int k = max(0, issued - kStreamGroup); k < issued; ++k)
                if (k % kStreamGroup == sub) mbar_wait_bounded(&full[j * DEPTH + k % DEPTH], (k / DEPTH) & 1, kWaitLimitNs);
    } else {
        // ------------------------------------------------------ consumer --
        const int len = (int)(bounds[warp + 1].x - bounds[warp].x);
        TileState<D, NT, KV8> state;
        auto store_part = [&](int i, float *acc, int stride, const StreamStage &st) {
            state.store_part(acc, stride, mM + i * GP, mL + i * GP, lane, p.g);
            if (lane == 0) {
                part_info[i].unit = st.unit;
                part_info[i].begins = st.last == 4;
                part_info[i].from = st.last >= 8 ? st.last - 8 : -1;
            }
        };
        StreamStage tail;
        tail.unit = -1; tail.last = 0;
        for (int k = 0; k < len; ++k) {
            const int slot = warp * DEPTH + k % DEPTH;
            if (!wait_or_abort(&full[slot], (k / DEPTH) & 1, abort_flag)) break;
            const StreamStage st = info[slot];
            if (st.first) {
                state.reset();
                state.load_q(p.q + (size_t)st.unit * p.g * D, lane, p.g, p.scale_log2);
            }
            if (st.valid > 0) {
                const uint32_t kt = tiles + slot * L::kStage;
                const bool partial = st.valid < kStageTok;
                float ks = 1.f, vs = 1.f;
                if constexpr (KV8) {
                    const float2 sc = slot_scales[slot];
                    ks = sc.x;
                    vs = sc.y;
                }
                if (partial) state.template stage<true>(kt, kt + L::kTile, st.valid, lane, p.scale_log2, ks, vs);
                else state.template stage<false>(kt, kt + L::kTile, st.valid, lane, p.scale_log2, ks, vs);
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&empty[slot]);
            if (st.last != 0 && SEL && p.split) {
                tail = st;
            } else if (st.last == 1) {
                state.write_out(p.out + (size_t)st.unit * p.g * D, lane, p.g);
            } else if (st.last == 4 || (st.last != 0 && k == len - 1)) {
                tail = st;  // the stretch ends with it: it stays in registers
            } else if (st.last != 0) {
                store_part(warp, cut + (size_t)warp * p.g * D, D, st);
            }
        }
        named_barrier_sync(1, kDecodeThreads);  // every ring has run dry
        if (tail.unit >= 0) store_part(W + warp, ends + warp * (L::kPart / 4), L::kStride, tail);
    }
    __syncthreads();
    grid_launch_dependents();

    // The parts in the line's order: warp 0's first, warp 0's last, warp 1's
    // first, ...  Neighbours of one unit form a group.  Thread (x, head) works
    // out part x's factor in its group, a warp lists the groups.
    auto part_at = [&](int x) { return (x >> 1) + (x & 1) * W; };
    if (warp == W) {
        const int x = lane & (2 * W - 1), unit = part_info[part_at(x)].unit;
        const uint32_t some = __ballot_sync(0xffffffffu, unit >= 0) & ((1u << (2 * W)) - 1);
        const uint32_t below = some & ((1u << x) - 1);
        const int prev = __shfl_sync(0xffffffffu, unit, below ? 31 - __clz(below) : 0);
        const uint32_t first = __ballot_sync(0xffffffffu, unit >= 0 && !(below && prev == unit)) & ((1u << (2 * W)) - 1);
        if (lane < 2 * W && ((first >> x) & 1u)) groups[1 + __popc(first & ((1u << x) - 1))] = x;
        if (lane == 0) groups[0] = __popc(first);
    }
    for (int i = tid; i < 2 * W * p.g; i += kDecodeThreads) {
        const int x = i / p.g, hd = i - x * p.g, unit = part_info[part_at(x)].unit;
        if (unit < 0) continue;
        float M = PKV_NEG_INF;
#pragma unroll
        for (int y = 0; y < 2 * W; ++y)
            if (part_info[y].unit == unit) M = fmaxf(M, mM[y * GP + hd]);
        factor[x * GP + hd] = ex2(mM[part_at(x) * GP + hd] - M);
    }
    if (tid == 0 && !(SEL && p.split)) p.meta[blockIdx.x] = make_int2(-1, 0);
    __syncthreads();
    if constexpr (SEL) {
        if (p.split) {
            // one unit: this CTA's partial, then the cluster's
            const int quads = p.g * D / 4;
            float *own = reinterpret_cast<float *>(smem + L::oOwn), *own_ml = own + GP * D;  // [g][D], (m, l) of a head
            for (int i = tid; i < quads; i += kDecodeThreads) {
                const int hd = i / (D / 4), d = (i - hd * (D / 4)) * 4;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                float Ls = 0.f, M = PKV_NEG_INF;
#pragma unroll
                for (int w = 0; w < W; ++w) {
                    if (part_info[W + w].unit < 0) continue;  // an empty stretch
                    const float f = factor[(2 * w + 1) * GP + hd];
                    const float4 v = *reinterpret_cast<const float4 *>(ends + w * (L::kPart / 4) + hd * L::kStride + d);
                    O.x = fmaf(v.x, f, O.x); O.y = fmaf(v.y, f, O.y); O.z = fmaf(v.z, f, O.z); O.w = fmaf(v.w, f, O.w);
                    Ls = fmaf(mL[(W + w) * GP + hd], f, Ls);
                    M = fmaxf(M, mM[(W + w) * GP + hd]);
                }
                *reinterpret_cast<float4 *>(own + hd * D + d) = O;
                if (d == 0) { own_ml[2 * hd] = M; own_ml[2 * hd + 1] = Ls; }
            }
            if (p.split > 1) {
                cluster_arrive();
                cluster_wait();
            } else {
                __syncthreads();
            }
            const int unit = blockIdx.x / p.split, rank = blockIdx.x % p.split;
            for (int i = rank * kDecodeThreads + tid; i < quads; i += p.split * kDecodeThreads) {
                const int hd = i / (D / 4), d = (i - hd * (D / 4)) * 4;
                float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
                float Ls = 0.f, M = PKV_NEG_INF, m[kStreamMaxSplit];
#pragma unroll
                for (int u = 0; u < kStreamMaxSplit; ++u) {
                    m[u] = u < p.split ? cluster_ld_f32(cluster_addr(own_ml + 2 * hd, u)) : PKV_NEG_INF;
                    M = fmaxf(M, m[u]);
                }
#pragma unroll
                for (int u = 0; u < kStreamMaxSplit; ++u) {
                    if (u >= p.split) break;
                    const float f = m[u] == PKV_NEG_INF ? 0.f : ex2(m[u] - M);
                    const float4 v = cluster_ld_f32x4(cluster_addr(own + hd * D + d, u));
                    O.x = fmaf(v.x, f, O.x); O.y = fmaf(v.y, f, O.y); O.z = fmaf(v.z, f, O.z); O.w = fmaf(v.w, f, O.w);
                    Ls = fmaf(cluster_ld_f32(cluster_addr(own_ml + 2 * hd + 1, u)), f, Ls);
                }
                const float inv = Ls > 0.f || Ls != Ls ? 1.f / Ls : 0.f;
                *reinterpret_cast<uint2 *>(p.out + (size_t)unit * p.g * D + hd * D + d) =
                    make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
            }
            if (p.split > 1) {  // a CTA's shared memory stays until its peers have read it
                cluster_arrive();
                cluster_wait();
            }
            return;
        }
    }
    const int quads = p.g * D / 4;
    for (int i = tid; i < groups[0] * quads; i += kDecodeThreads) {
        const int gr = i / quads, e = i - gr * quads;
        const int x = groups[1 + gr], end = gr + 1 < groups[0] ? groups[2 + gr] : 2 * W;
        const int hd = e / (D / 4), d = (e - hd * (D / 4)) * 4;
        const int unit = part_info[part_at(x)].unit, begins = part_info[part_at(x)].begins;
        int from = -1;
        float4 O = make_float4(0.f, 0.f, 0.f, 0.f);
        float Ls = 0.f, M = PKV_NEG_INF;
        for (int z = x; z < end; ++z) {
            const int pi = part_at(z);
            if (part_info[pi].unit < 0) continue;
            from = part_info[pi].from;
            const float f = factor[z * GP + hd];
            const float4 v = *reinterpret_cast<const float4 *>(
                pi < W ? cut + ((size_t)pi * p.g + hd) * D + d : ends + (pi - W) * (L::kPart / 4) + hd * L::kStride + d);
            O.x = fmaf(v.x, f, O.x); O.y = fmaf(v.y, f, O.y); O.z = fmaf(v.z, f, O.z); O.w = fmaf(v.w, f, O.w);
            Ls = fmaf(mL[pi * GP + hd], f, Ls);
            M = fmaxf(M, mM[pi * GP + hd]);
        }
        if (begins && from >= 0) {
            const float inv = Ls > 0.f || Ls != Ls ? 1.f / Ls : 0.f;
            *reinterpret_cast<uint2 *>(p.out + (size_t)unit * p.g * D + hd * D + d) =
                make_uint2(pack_bf16x2(O.x * inv, O.y * inv), pack_bf16x2(O.z * inv, O.w * inv));
        } else {
            // record 1: the unit begins here; 0: it began before
            const size_t r = ((size_t)blockIdx.x * 2 + begins) * p.g + hd;
            *reinterpret_cast<float4 *>(p.rec_acc + r * D + d) = O;
            if (d == 0) p.rec_ml[r] = make_float2(M, Ls);
            if (e == 0 && from >= 0) p.meta[blockIdx.x] = make_int2(unit, from);
        }
    }
}

// --------------------------------------------------------------- reduce ----
// Where a unit ends in CTA c of the attention kernel and began in an earlier
// one, that unit's records, that CTA's second one and the first ones of the CTAs
// behind it, are merged by log-sum-exp.  Block (i, head) looks at CTA i's note
// or, BY_UNIT, for unit i's among the notes of `ctas` CTAs: few units leave many
// records each, and take 16 warps to a row (one sequence of 131072 tokens, one
// kv head, 512 records: 42 us in all with 4 warps, 29 with 16).  Warp w takes records w,
// w + WARPS, ...; lanes own D / 32 elements.
template <int D, int WARPS, bool BY_UNIT>
__global__ void __launch_bounds__(WARPS * 32) stream_reduce_kernel(const StreamParams p, int ctas) {
    constexpr int EPL = D / 32;
    __shared__ float s_o[WARPS][D], s_l[WARPS], s_m[WARPS];
    __shared__ int s_c;
    const int head = blockIdx.y, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    int c = blockIdx.x;
    if (tid == 0) s_c = -1;
    grid_dependency_wait();
    if constexpr (BY_UNIT) {
        __syncthreads();
        for (int i = tid; i < ctas; i += WARPS * 32)
            if (p.meta[i].x == (int)blockIdx.x) s_c = i;  // one at most
        __syncthreads();
        c = s_c;
        if (c < 0) return;
    }
    const int2 meta = p.meta[c];
    if (meta.x < 0) return;
    const int n = c - meta.y + 1;  // records
    auto record = [&](int i) { return ((size_t)(meta.y + i) * 2 + (i == 0)) * p.g + head; };
    float M = PKV_NEG_INF, acc[EPL], lsum = 0.f;
    for (int i = warp + WARPS * lane; i < n; i += WARPS * 32) M = fmaxf(M, p.rec_ml[record(i)].x);
    M = warp_max_f32(M);
#pragma unroll
    for (int e = 0; e < EPL; ++e) acc[e] = 0.f;
#pragma unroll 8
    for (int i = warp; i < n; i += WARPS) {
        const size_t r = record(i);
        const float2 ml = p.rec_ml[r];
        const float f = ml.x == PKV_NEG_INF ? 0.f : ex2(ml.x - M);
        lsum = fmaf(ml.y, f, lsum);
        const float *a = p.rec_acc + r * D + lane * EPL;
        if constexpr (EPL == 4) {
            const float4 x = *reinterpret_cast<const float4 *>(a);
            acc[0] = fmaf(x.x, f, acc[0]); acc[1] = fmaf(x.y, f, acc[1]);
            acc[2] = fmaf(x.z, f, acc[2]); acc[3] = fmaf(x.w, f, acc[3]);
        } else {
            const float2 x = *reinterpret_cast<const float2 *>(a);
            acc[0] = fmaf(x.x, f, acc[0]); acc[1] = fmaf(x.y, f, acc[1]);
        }
    }
#pragma unroll
    for (int e = 0; e < EPL; ++e) s_o[warp][lane * EPL + e] = acc[e];
    if (lane == 0) { s_l[warp] = lsum; s_m[warp] = M; }
    __syncthreads();
    if (tid < D) {
        float T = PKV_NEG_INF, Ls = 0.f, O = 0.f;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) T = fmaxf(T, s_m[w]);
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            const float f = s_m[w] == PKV_NEG_INF ? 0.f : ex2(s_m[w] - T);
            Ls = fmaf(s_l[w], f, Ls);
            O = fmaf(s_o[w][tid], f, O);
        }
        p.out[((size_t)meta.x * p.g + head) * D + tid] = __float2bfloat16_rn(Ls > 0.f || Ls != Ls ? O / Ls : 0.f);
    }
}

}  // namespace pkv

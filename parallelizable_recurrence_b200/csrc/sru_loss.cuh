// sru_loss.cuh -- softmax cross entropy over a large vocabulary, with its
// gradients, without keeping the logits.
//
// For a row h_i of the last layer's output and the output matrix W (V, K):
//   z_i = W h_i,   lse_i = log sum_v exp z_iv,   loss_i = lse_i - z_i,t(i)
//   dz_iv = g_i (exp(z_iv - lse_i) - [v = t(i)]),   dH = dz W,   dW = dz^T H
// vocab_gemm_kernel runs z = H W^T as the pair GEMM of sru_gemm.cuh does (a
// cluster of two CTAs per 256 x 256 tile, TMA-fed ring, tcgen05.mma
// cta_group::2, two accumulators) and never stores z: a TMEM lane holds 256
// logits of one row, so each epilogue thread reduces its row alone, without
// shuffles.  Two epilogues:
//   kStats  running maximum and sum of exponentials of the row's 256 logits
//           (8 bytes per row and part; vocab_loss_kernel joins them) and, in
//           the one that holds it, the target's logit;
//   kGrad   dz of the tile from the row's lse and weight g, rounded to bf16 as
//           the operand of the two gradient products, stored by TMA.
// Four epilogue warps (a thread per row), or eight (two per row) for a short
// reduction, whose product takes less time than one warp per scheduler needs for a
// tile's exponentials.
// The gradients run over pieces of the vocabulary, so that dz takes 512 MB or 2 KB
// a row at most, whichever is more, and never V columns of them; z is recomputed there (2 M V K
// operations on top of the gradients' 4 M V K): kept, it would take 4 M V bytes (2 GB at
// M16384 V32000), and writing and reading it as long as the product at K of about 900.
// Measured, a kernel alone: M16384 V32000, kStats 702 us at K1024 (1.53 PFLOP/s) and
// 1.36 ms at K2048 (1.58); M4096 V8192 K1024, kStats 53 us (1.30), both gradient
// products 98.5 us (1.40).  In a row, long calls settle at the card's power limit.
#pragma once

#include <type_traits>

#include "sru_gemm.cuh"

namespace sru {
namespace loss {

using namespace gemm;

enum Epilogue : int { kStats = 0, kGrad = 1 };
constexpr float kLog2e = 1.4426950408889634f;

__device__ __forceinline__ float ex2_approx(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// r[i] without an indexed (hence local-memory) array.
template <int NC>
__device__ __forceinline__ float pick(const uint32_t (&r)[NC], int i) {
    uint32_t v = 0;
#pragma unroll
    for (int e = 0; e < NC; ++e)
        asm("{\n\t.reg .pred p;\n\tsetp.eq.s32 p, %1, %2;\n\t@p mov.b32 %0, %3;\n\t}" : "+r"(v) : "r"(i), "r"(e), "r"(r[e]));
    return __uint_as_float(v);
}

// Tiles in groups of kGroupM row tiles, the row tile fastest: the 74 pairs of a
// round then cover about 8 x 9 tiles, and a piece of W is read from memory once
// per group of 2048 rows instead of once per 256.
constexpr int kGroupM = 8;
__device__ __forceinline__ void unit_tile(int u, int m_tiles, int n_tiles, int& tm, int& tn) {
    const int per = kGroupM * n_tiles, g = u / per, r = u - g * per;
    const int gm = min(kGroupM, m_tiles - g * kGroupM);
    tn = r / gm;
    tm = g * kGroupM + r - tn * gm;
}

// The largest weight of a counted row (1 if there is none, or no finite one).  dz is
// held over it, and the gradients are multiplied by it in fp32: with the usual equal
// weights 1 / n, every dz of a target is then p - 1 rounded to bf16, whose error
// differs from row to row, and not -1 / n, whose error would be the same in all
// rows and scale the whole gradient by up to 2^-9.
// Here by one warp, rows 32 apart per lane; few enough rows (kInlineScaleRows) that
// the epilogue warps have it before their first tile is multiplied.
constexpr int kInlineScaleRows = 1024;
__device__ __forceinline__ float counted_weight(const float* dloss, const long long* targets, int i, long long V) {
    const long long t = targets[i];
    const float g = fabsf(dloss[i]);
    return t >= 0 && t < V && g < INFINITY ? g : 0.f;
}
__device__ __forceinline__ float weight_scale(const float* dloss, const long long* targets, int M, long long V) {
    float top = 0.f;
#pragma unroll 8
    for (int i = threadIdx.x & 31; i < M; i += 32) top = fmaxf(top, counted_weight(dloss, targets, i, V));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    return top > 0.f ? top : 1.f;
}

struct LossArgs {
    const long long* targets;  // (M): the class of each row; negative = not counted
    float2* partial;           // kStats: (parts of tiles, M) maximum and sum of exponentials
    float* target_logit;       // kStats: (M)
    const float* lse;          // kGrad: (M)
    const float* dloss;        // kGrad: (M)
    float* scale;              // kGrad: dz is taken over it; written here when inline_scale
    int inline_scale;
    long long v0, V;           // first column of this piece of the vocabulary, its whole size
};

// M rows, N columns of this piece, K the reduction.  map_w starts at row v0 of W.
// W = 4 or 8 epilogue warps.
template <int EPI, int W>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(64 + W * 32, 1)
    vocab_gemm_kernel(const __grid_constant__ CUtensorMap map_h, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_dz, LossArgs a, int M, int N, int K) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* epi = smem + P_STAGES * P_STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + P_EPI_BYTES);
    uint64_t* empty = full + P_STAGES;
    uint64_t* tfull = empty + P_STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* consumed = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair_id = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;
    const int m_tiles = (M + P_BM - 1) / P_BM, n_tiles = (N + P_BN - 1) / P_BN;
    const int kblocks = (K + BK - 1) / BK;
    const int units = m_tiles * n_tiles;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 2 * W);  // the epilogue warps of both CTAs
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *consumed = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_h);
        tma_prefetch_desc(&map_w);
        if (EPI == kGrad) tma_prefetch_desc(&map_dz);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, P_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
    const uint32_t leader_tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    pdl_launch();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------ producer (both CTAs)
            uint32_t issued = 0, phase = 0;
            int stage = 0;
            for (int u = pair_id; u < units && !*abort_flag; u += n_pairs) {
                int tm, tn;
                unit_tile(u, m_tiles, n_tiles, tm, tn);
                const int m0 = tm * P_BM + (int)rank * P_CM, n0 = tn * P_BN + (int)rank * P_CN;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(&empty[stage], phase ^ 1u, kErrTimeoutMma) || *abort_flag) {
                        *abort_flag = 1;
                        break;
                    }
                    uint8_t* a_dst = smem + stage * P_STAGE_BYTES;
                    const uint32_t bar = leader_full0 + (uint32_t)stage * 8u;
                    if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * P_STAGE_BYTES);
                    tma_load_2d_pair(a_dst, &map_h, bar, kb * BK, m0);
                    tma_load_2d_pair(a_dst + P_A_BYTES, &map_w, bar, kb * BK, n0);
                    ++issued;
                    if (++stage == P_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
            }
            if (*abort_flag && rank == 0) {
                for (uint32_t q = *consumed; q < issued; ++q)
                    mbar_wait(&full[q % P_STAGES], (q / P_STAGES) & 1u, kErrTimeoutLoad);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ------------------------------------------------------ MMA issuer (leader)
            constexpr uint32_t idesc = idesc_bf16_pair(false, false);
            int stage = 0, it = 0;
            uint32_t phase = 0, nconsumed = 0;
            for (int u = pair_id; u < units && !*abort_flag; u += n_pairs, ++it) {
                const int acc = it & 1;
                if (!mbar_wait(&tempty[acc], ((it >> 1) & 1) ^ 1u, kErrTimeoutEpilogue)) {
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + acc * P_BN;
                bool ok = true;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(&full[stage], phase, kErrTimeoutLoad)) {
                        ok = false;
                        break;
                    }
                    tc_fence_after_sync();
                    const uint32_t a_addr = smem_u32(smem + stage * P_STAGE_BYTES), b_addr = a_addr + P_A_BYTES;
#pragma unroll
                    for (int kk = 0; kk < BK / 16; ++kk)
                        tc_mma_bf16_pair(d_tmem, smem_desc_sw128(a_addr + kk * 32, 16, 1024),
                                         smem_desc_sw128(b_addr + kk * 32, 16, 1024), idesc,
                                         (kb != 0 || kk != 0) ? 1u : 0u);
                    tc_commit_pair_mc(&empty[stage], 0x3);
                    *consumed = ++nconsumed;
                    if (++stage == P_STAGES) {
                        stage = 0;
                        phase ^= 1u;
                    }
                }
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                tc_commit_pair_mc(&tfull[acc], 0x3);
            }
            tc_commit_pair_mc(drain, 0x1);
            mbar_wait(drain, 0, kErrTimeoutMma);
        }
    } else {
        // ---------------------------------------------------------- epilogue (both CTAs)
        constexpr int kParts = W / 4, kCols = P_BN / kParts;  // column parts of a tile, and their width
        constexpr int kBufs = 8 / W;                          // staging buffers per warp
        const int quarter = warp & 3, part = (warp - 2) >> 2;
        uint8_t* bufs = epi + (size_t)(warp - 2) * kBufs * P_EPI_BUF;
        int it = 0;
        uint32_t nstaged = 0;
        float scale = 1.f;
        if (EPI == kGrad) {
            scale = a.inline_scale ? weight_scale(a.dloss, a.targets, M, a.V) : *a.scale;
            if (a.inline_scale && blockIdx.x == 0 && warp == 2 && lane == 0) *a.scale = scale;
        }
        for (int u = pair_id; u < units; u += n_pairs, ++it) {
            int tm, tn;
            unit_tile(u, m_tiles, n_tiles, tm, tn);
            const int acc = it & 1;
            const int m0 = tm * P_BM + (int)rank * P_CM, n0 = tn * P_BN;
            const int row = m0 + quarter * 32 + lane;
            const bool live = row < M;
            // the row's operands, fetched while the product runs
            long long tgt = live ? a.targets[row] : -1;
            if (tgt >= a.V) tgt = -1;  // not a class: vocab_loss_kernel reports it
            // target's column in this warp's part of the tile, if inside
            const long long trel = tgt < 0 ? -1 : tgt - a.v0 - n0 - part * kCols;
            float lse2 = 0.f, g = 0.f;
            if (EPI == kGrad && tgt >= 0) {
                lse2 = a.lse[row] * kLog2e;
                g = __fdiv_rn(a.dloss[row], scale);
            }
            const bool ok = mbar_wait(&tfull[acc], (it >> 1) & 1, kErrTimeoutMma);
            if (!__all_sync(0xffffffffu, ok) || *abort_flag) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            constexpr int NC = EPI == kStats && W == 8 ? 32 : 64, NG = kCols / NC;
            const int col0 = n0 + part * kCols;
            const int ncol = max(0, min(kCols, N - col0));
            const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * P_BN + part * kCols;
            float top = -INFINITY, sum = 0.f;
            uint32_t r0[NC], r1[NC];
            tmem_ld_cols<NC>(tacc, r0);
#pragma unroll
            for (int c = 0; c < NG; ++c) {
                uint32_t(&cur)[NC] = (c & 1) ? r1 : r0;
                uint32_t(&nxt)[NC] = (c & 1) ? r0 : r1;
                tc_wait_ld();
                if (c + 1 < NG) tmem_ld_cols<NC>(tacc + (c + 1) * NC, nxt);
                const long long tc = trel - c * NC;
                const bool has_target = tc >= 0 && tc < NC;
                if (EPI == kStats) {
                    if (ncol < (c + 1) * NC) {
                        // columns behind the vocabulary hold products with zero rows
#pragma unroll
                        for (int e = 0; e < NC; ++e)
                            if (c * NC + e >= ncol) cur[e] = 0xff800000u;
                    }
                    float mx[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                    for (int e = 0; e < NC; ++e) mx[e & 3] = fmaxf(mx[e & 3], __uint_as_float(cur[e]));
                    const float nt = fmaxf(top, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])));
                    const float base = (nt == -INFINITY ? 0.f : nt) * kLog2e;
                    float s[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
                    for (int e = 0; e < NC; ++e)
                        s[e & 3] += ex2_approx(__fmaf_rn(__uint_as_float(cur[e]), kLog2e, -base));
                    sum = __fmaf_rn(sum, ex2_approx(__fmaf_rn(top, kLog2e, -base)), (s[0] + s[1]) + (s[2] + s[3]));
                    top = nt;
                    if (has_target) a.target_logit[row] = pick(cur, (int)tc);
                } else {
#pragma unroll
                    for (int e = 0; e < NC; ++e) {
                        const float p = ex2_approx(__fmaf_rn(__uint_as_float(cur[e]), kLog2e, -lse2)) * g;
                        cur[e] = g == 0.f ? 0u : __float_as_uint(p);  // rows not counted: exactly 0
                    }
                    const float pt = has_target ? pick(cur, (int)tc) : 0.f;
                    if (c * NC >= ncol) continue;  // (uniform across the warp)
                    uint8_t* stage_buf = bufs + (nstaged++ % kBufs) * P_EPI_BUF;
                    if (lane == 0) bulk_wait_group_read<kBufs - 1>();  // its last store has read it
                    __syncwarp();
                    epilogue_stage_row<kOutBF16>(smem_u32(stage_buf), lane, cur);
                    if (has_target) {
                        // (element tc of row `lane` in the staging buffer's swizzle)
                        const uint32_t off = lane * 128u + ((((uint32_t)tc >> 3) ^ (lane & 7u)) << 4) + (tc & 7) * 2u;
                        *reinterpret_cast<__nv_bfloat16*>(stage_buf + off) = __float2bfloat16_rn(pt - g);
                    }
                    fence_proxy_async_shared();
                    __syncwarp();
                    if (lane == 0) {
                        tma_store_2d(&map_dz, stage_buf, col0 + c * NC, m0 + quarter * 32);
                        bulk_commit_group();
                    }
                }
            }
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_tempty0 + (uint32_t)acc * 8u);
            if (EPI == kStats && live) a.partial[(size_t)(kParts * tn + part) * M + row] = make_float2(top, sum);
        }
        if (EPI == kGrad && lane == 0) bulk_wait_group<0>();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, P_TMEM_COLS);
    }
}

// ---------------------------------------------------------------------------
// Both gradient products of a piece in one launch: dH (+)= dz W (problem 0) and
// dW = dz^T H (problem 1), the pair GEMM's pipeline over one list of work units, so
// that neither product's last, partial round of CTA pairs is waited for, nor a launch
// between them.  A unit is an output tile and one k part of it.  (Tiles of 128
// columns for a K that fills its last 256 badly were slower: 12% at K520.)
struct GradProblem {
    int units, n_tiles, splits, kblocks, kper, slab_rows;
    int bf16, add;  // output type; add onto the output (fp32)
};
struct GradArgs {
    GradProblem p[2];
    int K, extra;        // extra: units of problem 1 that a pair without a last one of problem 0 takes first
    const float* scale;  // the outputs are multiplied by it
};
struct GradUnit {
    int prob, tm, tn, split, kb_lo, kb_hi;
};
// The i-th unit of pair q (of P): its units of problem 0 (q, q + P, ..); then, while
// the first r = units0 % P pairs are busy with one more, the others take `extra` units
// of problem 1 each; then the rest of problem 1 round-robin, the last pairs first.
__device__ __forceinline__ bool grad_unit(const GradArgs& a, int i, int q, int P, GradUnit& w) {
    const int u0 = a.p[0].units, own = (u0 - q + P - 1) / P, r = u0 % P;
    int u;
    if (i < own) {
        w.prob = 0;
        u = q + i * P;
    } else {
        w.prob = 1;
        i -= own;
        const int x = r > 0 && q >= r ? a.extra : 0;
        if (i < x) u = (q - r) + i * (P - r);
        else u = (r > 0 ? a.extra * (P - r) : 0) + (P - 1 - q) + (i - x) * P;
        if (u >= a.p[1].units) return false;
    }
    const GradProblem& p = a.p[w.prob];
    const int tile = u / p.splits;
    w.split = u - tile * p.splits;
    w.tm = tile / p.n_tiles;
    w.tn = tile - w.tm * p.n_tiles;
    w.kb_lo = w.split * p.kper;
    w.kb_hi = min(p.kblocks, w.kb_lo + p.kper);
    return true;
}

// One output tile's rows of this warp: TMEM -> scaled, rounded -> staging -> TMA.
template <int OUT>
__device__ __forceinline__ void grad_epilogue(uint32_t tacc, int ncol, float scale, uint8_t* bufs, uint32_t& nstaged,
                                              const CUtensorMap* map, bool add, int n0, int row, int lane) {
    constexpr int NC = EpiChunk<OUT>::kCols;
    const int ng = (ncol + NC - 1) / NC;
    uint32_t r0[NC], r1[NC];
    tmem_ld_cols<NC>(tacc, r0);
#pragma unroll
    for (int g = 0; g < P_BN / NC; ++g) {
        if (g >= ng) break;  // uniform across the warp
        uint32_t(&cur)[NC] = (g & 1) ? r1 : r0;
        uint32_t(&nxt)[NC] = (g & 1) ? r0 : r1;
        tc_wait_ld();
        if (g + 1 < ng) tmem_ld_cols<NC>(tacc + (g + 1) * NC, nxt);
#pragma unroll
        for (int e = 0; e < NC; ++e) cur[e] = __float_as_uint(__uint_as_float(cur[e]) * scale);
        uint8_t* buf = bufs + (nstaged & 1) * P_EPI_BUF;
        if (lane == 0) bulk_wait_group_read<1>();  // its last store has read it
        __syncwarp();
        epilogue_stage_row<OUT>(smem_u32(buf), lane, cur);
        fence_proxy_async_shared();
        __syncwarp();
        if (lane == 0) {
            if (add) tma_reduce_add_2d(map, buf, n0 + g * NC, row);
            else tma_store_2d(map, buf, n0 + g * NC, row);
            bulk_commit_group();
        }
        ++nstaged;
    }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(THREADS, 1)
    vocab_grad_kernel(const __grid_constant__ CUtensorMap map_dz_k, const __grid_constant__ CUtensorMap map_w,
                      const __grid_constant__ CUtensorMap map_dz_m, const __grid_constant__ CUtensorMap map_h,
                      const __grid_constant__ CUtensorMap map_dh, const __grid_constant__ CUtensorMap map_dw,
                      const __grid_constant__ GradArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* epi = smem + P_STAGES * P_STAGE_BYTES;
    uint64_t* full = reinterpret_cast<uint64_t*>(epi + P_EPI_BYTES);
    uint64_t* empty = full + P_STAGES;
    uint64_t* tfull = empty + P_STAGES;
    uint64_t* tempty = tfull + 2;
    uint64_t* drain = tempty + 2;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
    volatile uint32_t* consumed = reinterpret_cast<volatile uint32_t*>(tmem_slot + 2);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const int pair_id = blockIdx.x >> 1, n_pairs = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < P_STAGES; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&tfull[i], 1);
            mbar_init(&tempty[i], 8);  // 4 epilogue warps of each CTA
        }
        mbar_init(drain, 1);
        *abort_flag = 0;
        *consumed = 0;
        fence_mbar_init();
        tma_prefetch_desc(&map_dz_k);
        tma_prefetch_desc(&map_w);
        tma_prefetch_desc(&map_dz_m);
        tma_prefetch_desc(&map_h);
    }
    if (warp == 1) {
        tmem_alloc_pair(tmem_slot, P_TMEM_COLS);
        tmem_relinquish_pair();
    }
    tc_fence_before_sync();
    cluster_sync_all();
    tc_fence_after_sync();
    const uint32_t tmem_base = *tmem_slot;
    const uint32_t leader_full0 = mapa_shared(smem_u32(&full[0]), 0);
    const uint32_t leader_tempty0 = mapa_shared(smem_u32(&tempty[0]), 0);
    pdl_launch();
    pdl_wait();

    if (warp == 0) {
        if (lane == 0) {
            // ------------------------------------------------------ producer (both CTAs)
            uint32_t issued = 0, phase = 0;
            int stage = 0;
            GradUnit w;
            for (int i = 0; !*abort_flag && grad_unit(a, i, pair_id, n_pairs, w); ++i) {
                const int m0 = w.tm * P_BM + (int)rank * P_CM, n0 = w.tn * P_BN + (int)rank * P_CN;
                // (a loop per problem: with the maps chosen inside, the loads were late and a long
                // product 8% slower)
                auto kblocks = [&](auto second) {
                    constexpr bool P1 = decltype(second)::value;
                    for (int kb = w.kb_lo; kb < w.kb_hi; ++kb) {
                        if (!mbar_wait(&empty[stage], phase ^ 1u, kErrTimeoutMma) || *abort_flag) {
                            *abort_flag = 1;
                            break;
                        }
                        uint8_t* a_dst = smem + stage * P_STAGE_BYTES;
                        uint8_t* b_dst = a_dst + P_A_BYTES;
                        const uint32_t bar = leader_full0 + (uint32_t)stage * 8u;
                        if (rank == 0) mbar_arrive_expect_tx(&full[stage], 2 * P_STAGE_BYTES);
                        if (P1) {
                            tma_load_2d_pair(a_dst, &map_dz_m, bar, m0, kb * BK);
                            tma_load_2d_pair(a_dst + MN_BOX_BYTES, &map_dz_m, bar, m0 + 64, kb * BK);
                            tma_load_2d_pair(b_dst, &map_h, bar, n0, kb * BK);
                            tma_load_2d_pair(b_dst + MN_BOX_BYTES, &map_h, bar, n0 + 64, kb * BK);
                        } else {
                            tma_load_2d_pair(a_dst, &map_dz_k, bar, kb * BK, m0);
                            tma_load_2d_pair(b_dst, &map_w, bar, n0, kb * BK);
                            tma_load_2d_pair(b_dst + MN_BOX_BYTES, &map_w, bar, n0 + 64, kb * BK);
                        }
                        ++issued;
                        if (++stage == P_STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                };
                if (w.prob == 0) kblocks(std::false_type{});
                else kblocks(std::true_type{});
            }
            if (*abort_flag && rank == 0) {
                for (uint32_t q = *consumed; q < issued; ++q)
                    mbar_wait(&full[q % P_STAGES], (q / P_STAGES) & 1u, kErrTimeoutLoad);
            }
        }
    } else if (warp == 1) {
        if (lane == 0 && rank == 0) {
            // ------------------------------------------------------ MMA issuer (leader)
            int stage = 0;
            uint32_t phase = 0, nconsumed = 0;
            GradUnit w;
            for (int i = 0; !*abort_flag && grad_unit(a, i, pair_id, n_pairs, w); ++i) {
                const int acc = i & 1;
                if (!mbar_wait(&tempty[acc], ((i >> 1) & 1) ^ 1u, kErrTimeoutEpilogue)) {
                    *abort_flag = 1;
                    break;
                }
                tc_fence_after_sync();
                const uint32_t d_tmem = tmem_base + acc * P_BN;
                auto kblocks = [&](auto a_mn) {
                    constexpr bool A_MN = decltype(a_mn)::value;
                    constexpr uint32_t idesc = idesc_bf16_pair(A_MN, true);
                    for (int kb = w.kb_lo; kb < w.kb_hi; ++kb) {
                        if (!mbar_wait(&full[stage], phase, kErrTimeoutLoad)) return false;
                        tc_fence_after_sync();
                        const uint32_t a_addr = smem_u32(smem + stage * P_STAGE_BYTES), b_addr = a_addr + P_A_BYTES;
#pragma unroll
                        for (int kk = 0; kk < BK / 16; ++kk)
                            tc_mma_bf16_pair(d_tmem,
                                             A_MN ? smem_desc_sw128(a_addr + kk * 2048, MN_BOX_BYTES, 1024)
                                                  : smem_desc_sw128(a_addr + kk * 32, 16, 1024),
                                             smem_desc_sw128(b_addr + kk * 2048, MN_BOX_BYTES, 1024), idesc,
                                             (kb != w.kb_lo || kk != 0) ? 1u : 0u);
                        tc_commit_pair_mc(&empty[stage], 0x3);
                        *consumed = ++nconsumed;
                        if (++stage == P_STAGES) {
                            stage = 0;
                            phase ^= 1u;
                        }
                    }
                    return true;
                };
                const bool ok = w.prob == 0 ? kblocks(std::false_type{}) : kblocks(std::true_type{});
                if (!ok) {
                    *abort_flag = 1;
                    break;
                }
                tc_commit_pair_mc(&tfull[acc], 0x3);
            }
            tc_commit_pair_mc(drain, 0x1);
            mbar_wait(drain, 0, kErrTimeoutMma);
        }
    } else {
        // ---------------------------------------------------------- epilogue (both CTAs)
        const int quarter = warp & 3;
        const float scale = *a.scale;
        uint8_t* bufs = epi + (size_t)quarter * 2 * P_EPI_BUF;
        uint32_t nstaged = 0;
        GradUnit w;
        for (int i = 0; grad_unit(a, i, pair_id, n_pairs, w); ++i) {
            const int acc = i & 1;
            const bool ok = mbar_wait(&tfull[acc], (i >> 1) & 1, kErrTimeoutMma);
            if (!__all_sync(0xffffffffu, ok) || *abort_flag) {
                *abort_flag = 1;
                break;
            }
            tc_fence_after_sync();
            const GradProblem& p = a.p[w.prob];
            const int n0 = w.tn * P_BN, ncol = min(P_BN, a.K - n0);
            const int row = w.tm * P_BM + (int)rank * P_CM + quarter * 32 + w.split * p.slab_rows;
            const uint32_t tacc = tmem_base + ((uint32_t)(quarter * 32) << 16) + acc * P_BN;
            const CUtensorMap* map = w.prob == 0 ? &map_dh : &map_dw;
            if (p.bf16) grad_epilogue<kOutBF16>(tacc, ncol, scale, bufs, nstaged, map, false, n0, row, lane);
            else grad_epilogue<kOutF32>(tacc, ncol, scale, bufs, nstaged, map, p.add, n0, row, lane);
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) mbar_arrive_cluster(leader_tempty0 + (uint32_t)acc * 8u);
        }
        if (lane == 0) bulk_wait_group<0>();
    }
    tc_fence_before_sync();
    __syncthreads();
    cluster_sync_all();
    if (warp == 1) {
        tc_fence_after_sync();
        tmem_dealloc_pair(tmem_base, P_TMEM_COLS);
    }
}

// The same over many rows, in a launch of its own.
__global__ void __launch_bounds__(1024) loss_scale_kernel(const float* dloss, const long long* targets, float* scale,
                                                          int M, long long V) {
    __shared__ float part[32];
    pdl_launch();
    pdl_wait();
    float top = 0.f;
#pragma unroll 4
    for (int i = threadIdx.x; i < M; i += 1024) top = fmaxf(top, counted_weight(dloss, targets, i, V));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = top;
    __syncthreads();
    if (threadIdx.x >= 32) return;
    top = part[threadIdx.x];
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    if (threadIdx.x == 0) *scale = top > 0.f ? top : 1.f;
}

// Joins a row's tiles: lse = m + log sum_t s_t exp(m_t - m) with m the largest
// m_t; loss = lse - z_target, 0 for rows that are not counted.  32 rows x 32
// tile groups per CTA (consecutive threads read consecutive rows).
constexpr int kJoinRows = 32, kJoinGroups = 32;
__global__ void __launch_bounds__(kJoinRows* kJoinGroups)
    vocab_loss_kernel(const float2* partial, const float* target_logit, const long long* targets, float* loss,
                      float* lse, int M, int parts, long long V) {
    __shared__ float2 part[kJoinGroups][kJoinRows + 1];
    pdl_launch();
    pdl_wait();
    const int r = threadIdx.x % kJoinRows, q = threadIdx.x / kJoinRows;
    const int row = blockIdx.x * kJoinRows + r;
    float top = -INFINITY, sum = 0.f;
    auto join = [&](float2 b) {
        const float nt = fmaxf(top, b.x);
        const float base = nt == -INFINITY ? 0.f : nt;
        sum = sum * __expf(top - base) + b.y * __expf(b.x - base);
        top = nt;
    };
    if (row < M) {
#pragma unroll 4
        for (int t = q; t < parts; t += kJoinGroups) join(partial[(size_t)t * M + row]);
    }
    part[q][r] = make_float2(top, sum);
    __syncthreads();
    if (q != 0 || row >= M) return;
    for (int i = 1; i < kJoinGroups; ++i) join(part[i][r]);
    const float total = top + logf(sum);
    const long long t = targets[row];
    if (t >= V) record_error(kErrBadIndex);
    lse[row] = total;
    loss[row] = t >= 0 && t < V ? total - target_logit[row] : 0.f;
}

// out[r][c] = sum over s = 0, 1, .. of slabs[s * slab_rows + r][c] in that order,
// four columns per thread (C % 4 == 0).
template <typename OutT>
__global__ void __launch_bounds__(256) slab_sum_kernel(const float4* slabs, OutT* out, int R, int C4,
                                                       long long slab_rows, int splits) {
    pdl_launch();
    pdl_wait();
    const size_t n = (size_t)R * C4;
    for (size_t e = blockIdx.x * (size_t)256 + threadIdx.x; e < n; e += (size_t)gridDim.x * 256) {
        float4 acc = slabs[e];
        for (int sp = 1; sp < splits; ++sp) {
            const float4 v = slabs[(size_t)sp * slab_rows * C4 + e];
            acc.x += v.x;
            acc.y += v.y;
            acc.z += v.z;
            acc.w += v.w;
        }
        if (sizeof(OutT) == 4) {
            reinterpret_cast<float4*>(out)[e] = acc;
        } else {
            __nv_bfloat162 lo = __floats2bfloat162_rn(acc.x, acc.y), hi = __floats2bfloat162_rn(acc.z, acc.w);
            reinterpret_cast<uint2*>(out)[e] =
                make_uint2(*reinterpret_cast<uint32_t*>(&lo), *reinterpret_cast<uint32_t*>(&hi));
        }
    }
}

}  // namespace loss
}  // namespace sru

// sru_cache_attention.cuh -- attention of one new token per request over the
// paged cache of sru_cache.cuh: the single-token form of SRU++'s attention
// ("When Attention Meets Fast Recurrence", the SRU++ section), with shared
// (grouped) key/value heads.
//
//   o = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q.k_j - m)
// over the keys lo <= j < len of request b, lo = max(0, len - window).  Each key
// and value is read once and used for 2 x (heads of its group) multiplications:
// the call is bound by reading the cache.
//
// One pass with a running maximum m and sum l per head.  A step is 16 keys.  The
// steps of all (request, key head) items form one list, cut in equal contiguous
// ranges, one per team, so that ragged lengths still load every SM alike; a
// team's loads run ahead of its products across item borders.  An item that
// spans teams leaves its pieces (m, l, unnormalised o, fp32) in the workspace
// and cache_join_kernel joins them.
//
// A team is TW = ceil(D / 128) warps; warp w owns features 128 w .. of q, k, v and
// o.  It loads its part itself, by TMA: units of 32 rows x 128 features, K and V in
// turn, through a ring of its own whose barriers no other warp touches.  A page
// of ps tokens allows boxes of R rows, R the largest power of two (<= 32) that
// divides ps.  Keys are rows of the tensor-core products -- S^T = K Q^T (16 keys x
// 8 heads), O^T = V^T P^T (16 features x 8 heads) -- so a group of up to 8 heads
// costs what one does, and only the 32 x 8 partial scores cross the team's warps,
// through shared memory.  p enters its product as two bf16 parts (value and
// remainder, 16 bits together), so o is as exact as fp32 scores make it; the second
// product is free next to the loads.
#pragma once

#include "sru_ptx.cuh"

namespace sru {
namespace cache {

constexpr int kStep = 32;     // keys per step
constexpr int kSlice = 128;   // features per warp
constexpr int kMaxWarps = 8;  // per CTA
constexpr uint32_t kHalfBytes = kStep * 128;       // 64 features of a step's rows
constexpr uint32_t kRingBytes = 6 * kHalfBytes;    // per warp: 3 units, or 6 of one half when D <= 64
constexpr int kMaxUnits = 6, kMasks = 4;

struct DecodeArgs {
    const __nv_bfloat16 *q, *k, *v;
    const int *table, *lengths;
    void* out;
    float* lse;          // nullable
    float* part;         // pieces: team * 2 + (1 = starts its item, 0 = goes on with it)
    int4* jobs;          // per team: the item that it starts and does not finish
    int B, Hq, Hkv, D, ps, maxp, pages, window, out_f32;
    int group;           // query heads per key head
    int blocks;          // head blocks per key head
    int tw, teams;       // warps per team, teams per CTA
    int box_rows;        // R
    float scale_log2;    // scale * log2 e
};

// floats of one piece: o [heads][tw * kSlice], then m and l [heads]
__host__ __device__ inline size_t piece_floats(int heads, int dp) { return (size_t)heads * dp + 2 * heads; }

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void ldsm4(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldsm4_t(uint32_t addr, uint32_t (&r)[4]) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ uint32_t movm(uint32_t a) {
    uint32_t r;
    asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(a));
    return r;
}
__device__ __forceinline__ void mma_bf16(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
        "{%0, %1, %2, %3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t pack_bf16(float a, float b) {
    __nv_bfloat162 v = __floats2bfloat162_rn(a, b);
    return *reinterpret_cast<uint32_t*>(&v);
}
__device__ __forceinline__ void team_sync(int team, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(team + 1), "r"(threads) : "memory");
}

// First key, one past the last key, and first step of a request; steps() = 0 when empty.
struct Span {
    int lo, hi, s0, s1;
    __device__ int steps() const { return s1 - s0; }
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
    Span x;
    const long long width = (long long)a.maxp * a.ps;
    x.hi = (int)min((long long)max(a.lengths[b], 0), width);
    x.lo = a.window > 0 ? max(0, x.hi - a.window) : 0;
    x.s0 = x.lo / kStep;
    x.s1 = (x.hi + kStep - 1) / kStep;
    return x;
}

// A place in the list of steps: request b, head block hh (< Hkv * blocks), step s.
struct Cursor {
    int b, hh, s;
    Span sp;
    __device__ __forceinline__ void next(const DecodeArgs& a) {
        if (++s < sp.s1) return;
        if (++hh == a.Hkv * a.blocks) {
            hh = 0;
            do {
                if (++b >= a.B) return;
                sp = span_of(a, b);
            } while (sp.steps() <= 0);
        }
        s = sp.s0;
    }
};

__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    cache_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           DecodeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    __shared__ float4 exch[2][kMaxWarps][2][32];
    __shared__ uint64_t s_full[kMaxWarps][kMaxUnits];
    __shared__ uint32_t s_mask[kMaxWarps][kMasks];
    __shared__ long long s_scan[kMaxWarps], s_rem[kMaxWarps];
    __shared__ int s_b[kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
    const int HH = a.Hkv * a.blocks;

    pdl_launch();
    if (lane == 0) {
        for (int i = 0; i < kMaxUnits; ++i) mbar_init(&s_full[warp][i], 1);
        fence_mbar_init();
    }
    if (tid == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    // ---- this CTA's teams' places in the list: sums of steps over the requests
    const int per_thread = (a.B + nthreads - 1) / nthreads;
    long long mine = 0;
    for (int i = 0; i < per_thread; ++i) {
        const int b = tid * per_thread + i;
        if (b < a.B) mine += (long long)max(span_of(a, b).steps(), 0) * HH;
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    if (lane == 31) s_scan[warp] = upto;
    __syncthreads();
    long long total = 0, before = upto - mine;
    for (int w = 0; w < nthreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const long long n_teams = (long long)gridDim.x * a.teams;
    const long long per = max(1ll, (total + n_teams - 1) / n_teams);
    for (int t = 0; t < a.teams; ++t) {
        const long long g0 = ((long long)blockIdx.x * a.teams + t) * per;
        if (g0 >= before && g0 < before + mine) {
            long long at = before;
            for (int b = tid * per_thread;; ++b) {
                const long long n = (long long)max(span_of(a, b).steps(), 0) * HH;
                if (g0 < at + n) {
                    s_b[t] = b;
                    s_rem[t] = g0 - at;
                    break;
                }
                at += n;
            }
        }
    }
    // requests without keys: their output is zero
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const Span sp = span_of(a, b);
        if (tid == 0 && a.lengths[b] > sp.hi) record_error(kErrBadIndex);  // longer than the table is wide
        if (sp.steps() > 0) continue;
        for (int i = tid; i < a.Hq * a.D; i += nthreads) {
            const size_t at = (size_t)b * a.Hq * a.D + i;
            if (a.out_f32) static_cast<float*>(a.out)[at] = 0.f;
            else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(0.f);
        }
        if (a.lse != nullptr)
            for (int i = tid; i < a.Hq; i += nthreads) a.lse[(size_t)b * a.Hq + i] = -INFINITY;
    }
    __syncthreads();

    const int team = warp / a.tw, w_in = warp - team * a.tw;
    const long long my_team = (long long)blockIdx.x * a.teams + team;
    const long long g0 = my_team * per, g1 = min(total, g0 + per);
    if (g0 >= g1) {
        if (w_in == 0 && lane == 0) a.jobs[my_team] = make_int4(-1, 0, 0, 0);
        return;
    }
    Cursor cur;
    {
        cur.b = s_b[team];
        cur.sp = span_of(a, cur.b);
        const int n = cur.sp.steps();
        cur.hh = (int)(s_rem[team] / n);
        cur.s = cur.sp.s0 + (int)(s_rem[team] - (long long)cur.hh * n);
    }
    Cursor ld = cur;

    const int f0 = w_in * kSlice;                   // first feature of this warp
    const int width = min(kSlice, a.D - f0);        // its features, a multiple of 8
    const int halves = width > 64 ? 2 : 1;          // boxes of 64 features
    const int n_units = a.D > 64 ? 3 : 6;
    const uint32_t unit_bytes = a.D > 64 ? 2 * kHalfBytes : kHalfBytes;
    uint8_t* ring = smem + warp * kRingBytes;
    const int R = a.box_rows, groups = kStep / R;
    const int my_group = lane & (groups - 1), my_half = lane / groups;  // boxes of this lane: my_half, + 32 / groups

    // Table entry of this lane's box of step `ld`: read one step before its load, so
    // that its latency is not waited for.
    int next_page = 0, next_in = -1;  // next_in < 0: no key of the box is wanted
    auto fetch_page = [&]() {
        const int pos = ld.s * kStep + my_group * R;
        next_in = -1;
        if (pos + R > ld.sp.lo && pos < ld.sp.hi) {
            const int p = pos / a.ps;
            next_page = __ldg(a.table + (size_t)ld.b * a.maxp + p);
            next_in = pos - p * a.ps;
        }
    };
    int box_row = 0, box_in = -1;  // this lane's box of the step being loaded
    uint32_t step_bytes = 0;
    long long loaded = g0;         // step of the next unit to load
    int load_unit = 0, load_stage = 0, mask_at = 0;  // load_unit: 0 = K, 1 = V
    bool dead = false;             // a wait ran out: no further loads or waits
    auto load_next = [&]() {
        if (loaded >= g1 || dead) return;
        uint64_t* bar = &s_full[warp][load_stage];
        uint8_t* dst = ring + load_stage * unit_bytes;
        if (load_unit == 0) {
            box_in = next_in;
            if (box_in >= 0 && (unsigned)next_page >= (unsigned)a.pages) {
                record_error(kErrBadIndex);  // its keys are left out
                box_in = -1;
            }
            box_row = (int)((unsigned)next_page * a.Hkv + ld.hh / a.blocks);
            const unsigned there = __ballot_sync(0xffffffffu, box_in >= 0) & (groups == 32 ? ~0u : (1u << groups) - 1);
            step_bytes = __popc(there) * halves * R * 128;
            const int pos = ld.s * kStep + lane;
            const unsigned mask =
                __ballot_sync(0xffffffffu, pos >= ld.sp.lo && pos < ld.sp.hi && ((there >> (lane / R)) & 1));
            if (lane == 0) s_mask[warp][mask_at] = mask;
            mask_at = (mask_at + 1) & (kMasks - 1);
        }
        if (lane == 0) mbar_arrive_expect_tx(bar, step_bytes);
        __syncwarp();
        if (box_in >= 0)
            for (int h = my_half; h < halves; h += 32 / groups)
                tma_load_3d(dst + h * kHalfBytes + my_group * R * 128, load_unit ? &map_v : &map_k, bar, f0 + h * 64,
                            box_in, box_row);
        if (load_unit == 1 && ++loaded < g1) {
            ld.next(a);
            fetch_page();
        }
        load_unit ^= 1;
        load_stage = load_stage + 1 == n_units ? 0 : load_stage + 1;
    };
    fetch_page();
    for (int i = 0; i < n_units; ++i) load_next();

    const int g = lane >> 2, t2 = (lane & 3) * 2;
    uint32_t qf[kSlice / 16][2];
    float o[kSlice / 16][4];
    float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;  // heads t2, t2 + 1
    bool open = false, begins = false;
    int stage = 0, buf = 0, mask_use = 0;
    uint32_t phase = 0;
    // this warp's next unit has landed (false: the wait ran out)
    auto wait_unit = [&]() {
        if (!dead && !__all_sync(0xffffffffu, mbar_wait(&s_full[warp][stage], phase, kErrTimeoutLoad))) dead = true;
    };
    auto unit_done = [&]() {
        if (++stage == n_units) {
            stage = 0;
            phase ^= 1u;
        }
        __syncwarp();  // every lane has read the unit
        load_next();
    };
    for (long long step = g0; step < g1; ++step) {
        const int hblk = cur.hh % a.blocks, kv = cur.hh / a.blocks;
        const int head0 = kv * a.group + hblk * 8, heads = min(8, a.group - hblk * 8);
        if (!open) {
            open = true;
            begins = cur.s == cur.sp.s0;
            const __nv_bfloat16* q = a.q + ((size_t)cur.b * a.Hq + head0 + min(g, heads - 1)) * a.D + f0;
#pragma unroll
            for (int kk = 0; kk < kSlice / 16; ++kk) {
                const int c = kk * 16 + t2;
                qf[kk][0] = g < heads && c < width ? *reinterpret_cast<const uint32_t*>(q + c) : 0u;
                qf[kk][1] = g < heads && c + 8 < width ? *reinterpret_cast<const uint32_t*>(q + c + 8) : 0u;
#pragma unroll
                for (int e = 0; e < 4; ++e) o[kk][e] = 0.f;
            }
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
        }
        // ---- scores of 2 x 16 keys
        float sc[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        wait_unit();
        {
            const uint32_t base = smem_u32(ring) + stage * unit_bytes + (lane & 15) * 128;
            const int r7 = lane & 7, hi = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < kSlice / 16; ++kk) {
                if (kk * 16 >= width) break;
                const uint32_t at = base + (kk >> 2) * kHalfBytes + (((2 * (kk & 3) + hi) ^ r7) << 4);
                uint32_t ka[4], kb[4];
                ldsm4(at, ka);
                ldsm4(at + 16 * 128, kb);
                mma_bf16(sc[0], ka, qf[kk][0], qf[kk][1]);
                mma_bf16(sc[1], kb, qf[kk][0], qf[kk][1]);
            }
        }
        unit_done();
        if (a.tw > 1) {
#pragma unroll
            for (int i = 0; i < 2; ++i) exch[buf][warp][i][lane] = make_float4(sc[i][0], sc[i][1], sc[i][2], sc[i][3]);
            team_sync(team, a.tw * 32);
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                float4 s = exch[buf][team * a.tw][i][lane];
                for (int w = 1; w < a.tw; ++w) {
                    const float4 x = exch[buf][team * a.tw + w][i][lane];
                    s.x += x.x;
                    s.y += x.y;
                    s.z += x.z;
                    s.w += x.w;
                }
                sc[i][0] = s.x;
                sc[i][1] = s.y;
                sc[i][2] = s.z;
                sc[i][3] = s.w;
            }
            buf ^= 1;
        }
        // ---- running maximum and sum; p of keys 16 i + g and + 8, heads t2 and t2 + 1
        const uint32_t mask = s_mask[warp][mask_use];
        mask_use = (mask_use + 1) & (kMasks - 1);
        float n0 = m0, n1 = m1;
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const bool k0 = (mask >> (16 * i + g)) & 1, k1 = (mask >> (16 * i + g + 8)) & 1;
            sc[i][0] = k0 ? sc[i][0] * a.scale_log2 : -INFINITY;
            sc[i][1] = k0 ? sc[i][1] * a.scale_log2 : -INFINITY;
            sc[i][2] = k1 ? sc[i][2] * a.scale_log2 : -INFINITY;
            sc[i][3] = k1 ? sc[i][3] * a.scale_log2 : -INFINITY;
            n0 = fmaxf(n0, fmaxf(sc[i][0], sc[i][2]));
            n1 = fmaxf(n1, fmaxf(sc[i][1], sc[i][3]));
        }
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
        }
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;  // nothing seen yet
        const float f0c = ex2f(m0 - b0), f1c = ex2f(m1 - b1);
        m0 = n0;
        m1 = n1;
        l0 *= f0c;
        l1 *= f1c;
        uint32_t ph[2][2], pl[2][2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            const float p[4] = {ex2f(sc[i][0] - b0), ex2f(sc[i][1] - b1), ex2f(sc[i][2] - b0), ex2f(sc[i][3] - b1)};
            l0 += p[0] + p[2];
            l1 += p[1] + p[3];
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t h = pack_bf16(p[2 * j], p[2 * j + 1]);
                pl[i][j] = movm(pack_bf16(p[2 * j] - __uint_as_float(h << 16),
                                          p[2 * j + 1] - __uint_as_float(h & 0xffff0000u)));
                ph[i][j] = movm(h);
            }
        }
        wait_unit();
        if (mask != ~0u) {
            // rows without a key hold what the page held (or the ring, where no box was
            // loaded): p = 0 there must meet a finite value
            if (!((mask >> lane) & 1)) {
                uint8_t* row = ring + stage * unit_bytes + lane * 128;
                for (int c = 0; c < halves * 8; ++c)
                    *reinterpret_cast<uint4*>(row + (c >> 3) * kHalfBytes + (c & 7) * 16) = make_uint4(0, 0, 0, 0);
                fence_proxy_async_shared();  // before the ring's next load of these bytes
            }
            __syncwarp();
        }
        {
            const uint32_t base =
                smem_u32(ring) + stage * unit_bytes + ((lane & 7) + ((lane >> 4) << 3)) * 128;
            const int r7 = lane & 7, hi = (lane >> 3) & 1;
#pragma unroll
            for (int mt = 0; mt < kSlice / 16; ++mt) {
                if (mt * 16 >= width) break;
                const uint32_t at = base + (mt >> 2) * kHalfBytes + (((2 * (mt & 3) + hi) ^ r7) << 4);
                uint32_t va[4], vb[4];
                ldsm4_t(at, va);
                ldsm4_t(at + 16 * 128, vb);
                o[mt][0] *= f0c;
                o[mt][1] *= f1c;
                o[mt][2] *= f0c;
                o[mt][3] *= f1c;
                mma_bf16(o[mt], va, ph[0][0], ph[0][1]);
                mma_bf16(o[mt], vb, ph[1][0], ph[1][1]);
                mma_bf16(o[mt], va, pl[0][0], pl[0][1]);
                mma_bf16(o[mt], vb, pl[1][0], pl[1][1]);
            }
        }
        unit_done();
        const bool ends = cur.s + 1 == cur.sp.s1;
        if (ends || step + 1 == g1) {
            // ---- a piece, or a whole item, is done
            float t0 = l0, t1 = l1;
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                t0 += __shfl_xor_sync(0xffffffffu, t0, x);
                t1 += __shfl_xor_sync(0xffffffffu, t1, x);
            }
            const bool whole = begins && ends;
            const float r0 = whole ? (t0 > 0.f ? 1.f / t0 : 0.f) : 1.f, r1 = whole ? (t1 > 0.f ? 1.f / t1 : 0.f) : 1.f;
            const int dp = a.tw * kSlice;
            float* part = a.part + (size_t)(my_team * 2 + (begins ? 1 : 0)) * piece_floats(8, dp);
#pragma unroll
            for (int mt = 0; mt < kSlice / 16; ++mt) {
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const int head = t2 + (e & 1), c = mt * 16 + g + (e >> 1) * 8;
                    if (head >= heads || c >= width) continue;
                    const float x = o[mt][e] * ((e & 1) ? r1 : r0);
                    if (!whole) {
                        part[(size_t)head * dp + f0 + c] = x;
                    } else {
                        const size_t at = ((size_t)cur.b * a.Hq + head0 + head) * a.D + f0 + c;
                        if (a.out_f32) static_cast<float*>(a.out)[at] = x;
                        else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(x);
                    }
                }
            }
            if (w_in == 0 && g == 0) {
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int head = t2 + e;
                    if (head >= heads) continue;
                    const float mm = e ? m1 : m0, ll = e ? t1 : t0;
                    if (!whole) {
                        part[(size_t)8 * dp + head] = mm;
                        part[(size_t)8 * dp + 8 + head] = ll;
                    } else if (a.lse != nullptr) {
                        a.lse[(size_t)cur.b * a.Hq + head0 + head] =
                            ll > 0.f ? (mm + log2f(ll)) * 0.69314718055994531f : -INFINITY;
                    }
                }
            }
            if (step + 1 == g1 && w_in == 0 && lane == 0) {
                // the last team of the item that this team starts and leaves unfinished
                const long long rest = (long long)cur.sp.s1 - cur.s - 1;
                a.jobs[my_team] = begins && !ends ? make_int4(cur.b, cur.hh, (int)((step + rest) / per), 0)
                                                  : make_int4(-1, 0, 0, 0);
            }
            open = false;
        }
        if (step + 1 < g1) cur.next(a);
    }
    if (dead) {
        // leave no copy in flight (each wait is bounded again)
        for (int i = 0; i < n_units; ++i) {
            mbar_wait(&s_full[warp][stage], phase, kErrTimeoutLoad);
            if (++stage == n_units) {
                stage = 0;
                phase ^= 1u;
            }
        }
    }
}

// Joins the pieces of the items that the teams of main CTA blockIdx.x start, for one
// head (blockIdx.y) and 128 features (blockIdx.z; a lane has 4).  An item of up to
// 8 pieces is joined by the warp of its team; a longer one by all warps, which
// take pieces in turn.  The order of the sums is fixed by the sizes alone.
constexpr int kJoinWarps = kMaxWarps;
__global__ void __launch_bounds__(kJoinWarps * 32) cache_join_kernel(DecodeArgs a) {
    __shared__ float s_m[kJoinWarps], s_l[kJoinWarps];
    __shared__ float4 s_o[kJoinWarps][32];
    pdl_wait();
    const int dp = a.tw * kSlice, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const size_t pf = piece_floats(8, dp);
    const int head = blockIdx.y, c = blockIdx.z * 128 + lane * 4;
    const bool live = c < a.D;

    auto store = [&](const int4& job, float4 acc, float top, float l) {
        const float r = l > 0.f ? 1.f / l : 0.f;
        const int hblk = job.y % a.blocks, kv = job.y / a.blocks;
        const size_t row = (size_t)job.x * a.Hq + kv * a.group + hblk * 8 + head;
        if (live) {
            if (a.out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * a.D + c) =
                    make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * a.D + c) =
                    make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
        }
        if (a.lse != nullptr && blockIdx.z == 0 && lane == 0)
            a.lse[row] = l > 0.f ? (top + log2f(l)) * 0.69314718055994531f : -INFINITY;
    };
    auto add = [](float4& acc, float w, const float4& x) {
        acc.x = __fmaf_rn(w, x.x, acc.x);
        acc.y = __fmaf_rn(w, x.y, acc.y);
        acc.z = __fmaf_rn(w, x.z, acc.z);
        acc.w = __fmaf_rn(w, x.w, acc.w);
    };

    for (int t = 0; t < a.teams; ++t) {
        const int t0 = blockIdx.x * a.teams + t;
        const int4 job = a.jobs[t0];
        if (job.x < 0 || head >= min(8, a.group - job.y % a.blocks * 8)) continue;
        const int n = job.z - t0 + 1;  // pieces: (t0, starts), (t0 + 1, goes on), ...
        auto piece = [&](int i) { return a.part + ((size_t)(t0 + i) * 2 + (i == 0 ? 1 : 0)) * pf; };
        if (n <= kJoinWarps) {
            if (warp != t) continue;
            const float m = lane < n ? piece(lane)[(size_t)8 * dp + head] : -INFINITY;
            const float li = lane < n ? piece(lane)[(size_t)8 * dp + 8 + head] : 0.f;
            float4 x[kJoinWarps];
#pragma unroll
            for (int i = 0; i < kJoinWarps; ++i)
                if (i < n && live) x[i] = *reinterpret_cast<const float4*>(piece(i) + (size_t)head * dp + c);
            float top = m;
#pragma unroll
            for (int o = 4; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
            top = __shfl_sync(0xffffffffu, top, 0);
            const float w = ex2f(m - (top == -INFINITY ? 0.f : top));
            float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
            float l = 0.f;
#pragma unroll
            for (int i = 0; i < kJoinWarps; ++i) {
                if (i >= n) break;
                const float wi = __shfl_sync(0xffffffffu, w, i);
                l = __fmaf_rn(wi, __shfl_sync(0xffffffffu, li, i), l);
                if (live) add(acc, wi, x[i]);
            }
            store(job, acc, top, l);
            continue;
        }
        float top = -INFINITY;
        for (int i = threadIdx.x; i < n; i += kJoinWarps * 32) top = fmaxf(top, piece(i)[(size_t)8 * dp + head]);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
        if (lane == 0) s_m[warp] = top;
        __syncthreads();
#pragma unroll
        for (int i = 0; i < kJoinWarps; ++i) top = fmaxf(top, s_m[i]);
        const float base = top == -INFINITY ? 0.f : top;
        float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
        float l = 0.f;
#pragma unroll 8
        for (int i = warp; i < n; i += kJoinWarps) {
            const float* p = piece(i);
            const float w = ex2f(p[(size_t)8 * dp + head] - base);
            l = __fmaf_rn(w, p[(size_t)8 * dp + 8 + head], l);
            if (live) add(acc, w, *reinterpret_cast<const float4*>(p + (size_t)head * dp + c));
        }
        s_o[warp][lane] = acc;
        if (lane == 0) s_l[warp] = l;
        __syncthreads();
        if (warp == 0) {
            for (int i = 1; i < kJoinWarps; ++i) {
                add(acc, 1.f, s_o[i][lane]);
                l += s_l[i];
            }
            store(job, acc, top, l);
        }
        __syncthreads();  // the shared sums may be written again
    }
}

}  // namespace cache
}  // namespace sru

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
// A team is TW = ceil(D / 128) warps; warp w owns the feature slice w of q, k, v
// and o (at most 128 wide), loads it itself (cp.async, kStages steps of 16 x 2 rows,
// no barrier with other warps), multiplies on the tensor cores with the keys as
// rows -- S^T = K Q^T (16 keys x 8 heads), O^T = V^T P^T (16 features x 8 heads) --
// and only the 16 x 8 partial scores cross the team's warps, through shared
// memory.  p goes to the tensor cores as two bf16 parts (value and remainder, 16
// bits together), so o is as exact as fp32 scores make it; the second product is
// free next to the loads.
#pragma once

#include "sru_ptx.cuh"

namespace sru {
namespace cache {

constexpr int kStep = 16;     // keys per step
constexpr int kStages = 3;    // steps in a warp's ring
constexpr int kSlice = 128;   // features per warp
constexpr int kMaxWarps = 8;  // per CTA
constexpr uint32_t kRowBytes = kSlice * 2;
constexpr uint32_t kStageBytes = 2 * kStep * kRowBytes;  // K and V rows
constexpr uint32_t kRingBytes = kStages * kStageBytes;

struct DecodeArgs {
    const __nv_bfloat16 *q, *k, *v;
    const int *table, *lengths;
    void* out;
    float* lse;          // nullable
    float* part;         // pieces: team * 2 + (1 = starts its item, 0 = goes on with it)
    int4* jobs;          // per team: the item that it starts and does not finish
    long long* range;    // steps per team
    int B, Hq, Hkv, D, ps, maxp, pages, window, out_f32;
    int group;           // query heads per key head
    int blocks;          // head blocks per key head
    int tw, teams;       // warps per team, teams per CTA
    int slice;           // features per warp (a multiple of 16)
    float scale_log2;    // scale * log2 e
};

// floats of one piece: o [heads][tw * slice], then m and l [heads]
__host__ __device__ inline size_t piece_floats(int heads, int dp) { return (size_t)heads * dp + 2 * heads; }

__device__ __forceinline__ float ex2f(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, uint32_t bytes) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
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

__global__ void __launch_bounds__(kMaxWarps * 32, 1) cache_attention_kernel(DecodeArgs a) {
    extern __shared__ __align__(1024) uint8_t smem[];
    __shared__ float4 exch[2][kMaxWarps][32];
    __shared__ uint32_t s_mask[kMaxWarps][kStages];
    __shared__ long long s_scan[kMaxWarps];
    __shared__ int s_b[kMaxWarps];
    __shared__ long long s_rem[kMaxWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x;
    const int HH = a.Hkv * a.blocks;

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
    for (int i = tid; i < a.teams; i += nthreads) s_b[i] = a.B;
    // stale features behind D stay zero: loads never touch them
    for (uint32_t i = tid; i < (nthreads / 32) * kRingBytes / 16; i += nthreads)
        reinterpret_cast<uint4*>(smem)[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    long long total = 0, before = upto - mine;
    for (int w = 0; w < nthreads / 32; ++w) {
        if (w < warp) before += s_scan[w];
        total += s_scan[w];
    }
    const long long n_teams = (long long)gridDim.x * a.teams;
    const long long per = max(1ll, (total + n_teams - 1) / n_teams);
    if (blockIdx.x == 0 && tid == 0) *a.range = per;
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
    if (team >= a.teams) return;
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

    const uint32_t ring = smem_u32(smem) + warp * kRingBytes;
    const int f0 = w_in * a.slice;                         // first feature of this warp
    const int width = min(a.slice, a.D - f0);              // features (D % 8 == 0), may be <= 0
    const int chunks = max(0, width) / 8;                  // 16-byte chunks of a row
    const int my_chunk = lane & 15, my_row = lane >> 4;

    // table entry and row of key (lane & 15) of step `ld`: the entry is read one step
    // before its load, so that its latency is not waited for
    int next_page = 0, next_in = -1;  // next_in < 0: no such key
    auto fetch_row = [&]() {
        const int pos = ld.s * kStep + (lane & 15);
        next_in = -1;
        if (pos >= ld.sp.lo && pos < ld.sp.hi) {
            const int p = pos / a.ps;
            next_page = __ldg(a.table + (size_t)ld.b * a.maxp + p);
            next_in = pos - p * a.ps;
        }
    };
    auto load = [&](int stage) {
        const uint32_t st = ring + stage * kStageBytes;
        bool there = next_in >= 0;
        if (there && (unsigned)next_page >= (unsigned)a.pages) {
            record_error(kErrBadIndex);  // the key is left out
            there = false;
        }
        const long long next_row = ((long long)next_page * a.Hkv + ld.hh / a.blocks) * a.ps + next_in;
        const unsigned mask = __ballot_sync(0xffffffffu, there) & 0xffffu;
        if (lane == 0) s_mask[warp][stage] = mask;
#pragma unroll
        for (int j = 0; j < kStep / 2; ++j) {
            const int r = 2 * j + my_row;
            const long long row = __shfl_sync(0xffffffffu, next_row, r);
            if (my_chunk < chunks) {
                const bool live = (mask >> r) & 1;
                const size_t at = live ? (size_t)row * a.D + f0 + my_chunk * 8 : 0;
                const uint32_t dst = st + r * kRowBytes + ((my_chunk ^ (r & 7)) << 4);
                cp_async16(dst, a.k + at, live ? 16u : 0u);
                cp_async16(dst + kStep * kRowBytes, a.v + at, live ? 16u : 0u);
            }
        }
    };
    long long loaded = g0;
    fetch_row();
    auto load_next = [&](int stage) {
        if (loaded < g1) {
            load(stage);
            if (++loaded < g1) {
                ld.next(a);
                fetch_row();
            }
        }
        cp_commit();
    };
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i) load_next(i);

    const int g = lane >> 2, t2 = (lane & 3) * 2;
    uint32_t qf[kSlice / 16][2];
    float o[kSlice / 16][4];
    float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;  // heads t2, t2 + 1
    bool open = false, begins = false;
    int stage = 0, buf = 0;
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
        load_next(stage == 0 ? kStages - 1 : stage - 1);
        cp_wait<kStages - 1>();
        __syncwarp();
        const uint32_t ks = ring + stage * kStageBytes, vs = ks + kStep * kRowBytes;
        float sc[4] = {0.f, 0.f, 0.f, 0.f}, sc2[4] = {0.f, 0.f, 0.f, 0.f};
        {
            const int r = lane & 15, hi = lane >> 4;
#pragma unroll
            for (int kk = 0; kk < kSlice / 16; ++kk) {
                if (kk * 16 >= width) break;
                uint32_t kf[4];
                ldsm4(ks + r * kRowBytes + (((2 * kk + hi) ^ (r & 7)) << 4), kf);
                if (kk & 1) mma_bf16(sc2, kf, qf[kk][0], qf[kk][1]);
                else mma_bf16(sc, kf, qf[kk][0], qf[kk][1]);
            }
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[e] += sc2[e];
        }
        if (a.tw > 1) {
            exch[buf][warp][lane] = make_float4(sc[0], sc[1], sc[2], sc[3]);
            team_sync(team, a.tw * 32);
            float4 s = exch[buf][team * a.tw][lane];
            for (int w = 1; w < a.tw; ++w) {
                const float4 x = exch[buf][team * a.tw + w][lane];
                s.x += x.x;
                s.y += x.y;
                s.z += x.z;
                s.w += x.w;
            }
            sc[0] = s.x;
            sc[1] = s.y;
            sc[2] = s.z;
            sc[3] = s.w;
            buf ^= 1;
        }
        const uint32_t mask = s_mask[warp][stage];
        const bool k0 = (mask >> g) & 1, k1 = (mask >> (g + 8)) & 1;
        sc[0] = k0 ? sc[0] * a.scale_log2 : -INFINITY;
        sc[1] = k0 ? sc[1] * a.scale_log2 : -INFINITY;
        sc[2] = k1 ? sc[2] * a.scale_log2 : -INFINITY;
        sc[3] = k1 ? sc[3] * a.scale_log2 : -INFINITY;
        float n0 = fmaxf(sc[0], sc[2]), n1 = fmaxf(sc[1], sc[3]);
#pragma unroll
        for (int x = 4; x < 32; x <<= 1) {
            n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
            n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
        }
        n0 = fmaxf(n0, m0);
        n1 = fmaxf(n1, m1);
        const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;  // nothing seen yet
        const float f0c = ex2f(m0 - b0), f1c = ex2f(m1 - b1);
        m0 = n0;
        m1 = n1;
        float p[4] = {ex2f(sc[0] - b0), ex2f(sc[1] - b1), ex2f(sc[2] - b0), ex2f(sc[3] - b1)};
        l0 = __fmaf_rn(l0, f0c, p[0] + p[2]);
        l1 = __fmaf_rn(l1, f1c, p[1] + p[3]);
        uint32_t ph[2], pl[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            ph[i] = pack_bf16(p[2 * i], p[2 * i + 1]);
            const float h0 = __uint_as_float(ph[i] << 16), h1 = __uint_as_float(ph[i] & 0xffff0000u);
            pl[i] = movm(pack_bf16(p[2 * i] - h0, p[2 * i + 1] - h1));
            ph[i] = movm(ph[i]);
        }
        {
            const int r = (lane & 7) + ((lane >> 4) << 3), hi = (lane >> 3) & 1;
#pragma unroll
            for (int mt = 0; mt < kSlice / 16; ++mt) {
                if (mt * 16 >= width) break;
                uint32_t vf[4];
                ldsm4_t(vs + r * kRowBytes + (((2 * mt + hi) ^ (r & 7)) << 4), vf);
                o[mt][0] *= f0c;
                o[mt][1] *= f1c;
                o[mt][2] *= f0c;
                o[mt][3] *= f1c;
                mma_bf16(o[mt], vf, ph[0], ph[1]);
                mma_bf16(o[mt], vf, pl[0], pl[1]);
            }
        }
        __syncwarp();  // the ring's stage has been read
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
            const int dp = a.tw * a.slice;
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
        stage = stage + 1 == kStages ? 0 : stage + 1;
    }
}

// Joins the pieces of one item and head: grid (teams, heads of a block, feature
// slices of 128), 8 groups of 32 threads x 4 features that take pieces in turn.
// The order of the sums is fixed by the sizes alone.
constexpr int kJoinThreads = 256;
__global__ void __launch_bounds__(kJoinThreads) cache_join_kernel(DecodeArgs a) {
    const int4 job = a.jobs[blockIdx.x];
    if (job.x < 0) return;
    const int head = blockIdx.y, hblk = job.y % a.blocks, kv = job.y / a.blocks;
    if (head >= min(8, a.group - hblk * 8)) return;
    __shared__ float s_m[kJoinThreads / 32], s_l[kJoinThreads / 32];
    __shared__ float4 s_o[kJoinThreads];
    const int dp = a.tw * a.slice, lane = threadIdx.x & 31, grp = threadIdx.x >> 5;
    const size_t pf = piece_floats(8, dp);
    const int t0 = blockIdx.x, n = job.z - t0 + 1;  // pieces: (t0, starts), (t0 + 1, goes on), ...
    auto piece = [&](int i) { return a.part + ((size_t)(t0 + i) * 2 + (i == 0 ? 1 : 0)) * pf; };
    float top = -INFINITY;
    for (int i = threadIdx.x; i < n; i += kJoinThreads) top = fmaxf(top, piece(i)[(size_t)8 * dp + head]);
#pragma unroll
    for (int x = 16; x > 0; x >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, x));
    if (lane == 0) s_m[grp] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) top = fmaxf(top, s_m[i]);
    const float base = top == -INFINITY ? 0.f : top;
    const int c = blockIdx.z * 128 + lane * 4;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    float l = 0.f;
#pragma unroll 4
    for (int i = grp; i < n; i += kJoinThreads / 32) {
        const float* p = piece(i);
        const float w = ex2f(p[(size_t)8 * dp + head] - base);
        l = __fmaf_rn(w, p[(size_t)8 * dp + 8 + head], l);
        if (c < a.D) {
            const float4 x = *reinterpret_cast<const float4*>(p + (size_t)head * dp + c);
            acc.x = __fmaf_rn(w, x.x, acc.x);
            acc.y = __fmaf_rn(w, x.y, acc.y);
            acc.z = __fmaf_rn(w, x.z, acc.z);
            acc.w = __fmaf_rn(w, x.w, acc.w);
        }
    }
    s_o[threadIdx.x] = acc;
    if (lane == 0) s_l[grp] = l;
    __syncthreads();
    if (grp != 0) return;
    l = 0.f;
#pragma unroll
    for (int i = 0; i < kJoinThreads / 32; ++i) l += s_l[i];
    for (int i = 1; i < kJoinThreads / 32; ++i) {
        const float4 x = s_o[i * 32 + lane];
        acc.x += x.x;
        acc.y += x.y;
        acc.z += x.z;
        acc.w += x.w;
    }
    const float r = l > 0.f ? 1.f / l : 0.f;
    const size_t row = (size_t)job.x * a.Hq + kv * a.group + hblk * 8 + head;
    if (c < a.D) {
        if (a.out_f32)
            *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * a.D + c) =
                make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
        else
            *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * a.D + c) =
                make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
    }
    if (a.lse != nullptr && blockIdx.z == 0 && lane == 0)
        a.lse[row] = l > 0.f ? (top + log2f(l)) * 0.69314718055994531f : -INFINITY;
}

}  // namespace cache
}  // namespace sru

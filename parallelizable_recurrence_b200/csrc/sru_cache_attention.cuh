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
// One pass with a running maximum m and sum l per head.  A step is 32 keys.  The
// steps of all (request, key head) items form one list, cut in equal contiguous
// ranges, one per team, so that ragged lengths still load every SM alike; a
// team's loads run ahead of its products across item borders.  An item that
// spans teams is in pieces (m, l, unnormalised o, fp32): the teams of a CTA join
// theirs through shared memory, and of the CTAs that share an item the last to
// finish joins theirs through the workspace, in the order of the keys whoever that
// is.  (A second kernel for it cost 5 to 9 us.)
//
// A team is TW = ceil(D / W) warps, W = 128 (or 64) features; warp w owns features
// W w .. of q, k, v and o.  It loads its part itself, by TMA: units of 32 rows x W
// features through a ring whose barriers no other warp touches.  A page of ps tokens allows
// boxes of R rows, R the largest power of two (<= 32) that divides ps.  Keys are
// rows of the tensor-core products -- S^T = K Q^T (16 keys x 8 heads), O^T = V^T P^T
// (16 features x 8 heads) -- so a group of up to 8 heads costs what one does, and
// only the 32 x 8 partial scores cross the team's warps, through shared memory.  The
// scores of step i + 1 are taken before the values of step i, so that neither the
// exchange nor the products' latency is waited for.  p enters its product as two
// bf16 parts (value and remainder, 16 bits together), so o is as exact as fp32
// scores make it; the second product is free next to the loads.
//
// Measured: B96 len <= 8192 D1024 277-301 us (6.0-6.5 TB/s, of 6.56 copied), B24 H32/8
// D128 len <= 6007 67-72 us, B64 D512 window 2560 57 us (4.7-4.9 TB/s): reading at the
// memory's rate, plus about 12 us that a call of any size takes (5 to the first loads, 2 to
// the rate, 4-5 to join) and the spread of the warps' ends.  Of a few keys the kernel takes 11 us
// (B1 len 200 D512) or 7 (B1 len 37 D64), a chain of latencies.
#pragma once

#include <type_traits>

#include "sru_ptx.cuh"

namespace sru {
namespace cache {

constexpr int kStep = 32;     // keys per step
constexpr int kSlice = 128;   // most features per warp
constexpr int kMaxWarps = 8;  // per CTA
constexpr uint32_t kHalfBytes = kStep * 128;        // 64 features of a step's rows
constexpr int kMasks = 8;     // steps whose keys' mask is held

struct DecodeArgs {
    const __nv_bfloat16* q;      // (the caches are read through their maps)
    const int *table, *lengths;
    void* out;
    float* lse;                  // nullable
    float* part;                 // pieces: (CTA, goes on with / starts its item), then the teams' first ones
    unsigned long long* flags;   // the same index: the CTA's piece is there, if equal to
    unsigned long long tag;      // this call's number
    int B, Hq, Hkv, D, ps, maxp, pages, window, out_f32;
    int width;           // keys that the table has room for
    int group;           // query heads per key head
    int blocks;          // head blocks per key head
    int tw, teams;       // warps per team, teams per CTA
    int box_rows;        // R
    int merged;          // the maps are 4-D and one box holds both halves of a unit's rows
    int units;           // of a warp's ring
    int early_floats;    // shared floats per warp for a piece that ends before its team's range; 0: workspace
    float scale_log2;    // scale * log2 e
};

// A piece: o [tw][8 heads][kSlice], then m and l [8].
constexpr int kSliceFloats = 8 * kSlice;
__host__ __device__ inline size_t piece_floats(int tw) { return (size_t)tw * kSliceFloats + 16; }

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

// First key, one past the last key, and first step of a request; s1 <= s0 when empty.
struct Span {
    int lo, hi, s0, s1;
    __device__ int steps() const { return max(s1 - s0, 0); }
};
__device__ __forceinline__ Span span_of(const DecodeArgs& a, int b) {
    Span x;
    x.hi = min(max(a.lengths[b], 0), a.width);
    x.lo = a.window > 0 ? max(0, x.hi - a.window) : 0;
    x.s0 = x.lo / kStep;
    x.s1 = (int)(((unsigned)x.hi + kStep - 1) / kStep);
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

// log of the sum l of exponentials over their maximum m (base 2), in base e.  Only l = 0, no key that
// weighs anything, gives -inf: a NaN among scores stays one.
__device__ __forceinline__ float lse_of(float m, float l) {
    return l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
}

// An item that is in pieces: its place, and its steps in the list.
struct Item {
    int b, hh, first, last;
};
// TW, W > 0: TW warps of W features each (D = TW W, W = 64 or 128), which makes the loops
// over features and warps straight code.  TW = W = 0: any D.
template <int TW, int W>
__global__ void __launch_bounds__(kMaxWarps * 32, 1)
    cache_attention_kernel(const __grid_constant__ CUtensorMap map_k, const __grid_constant__ CUtensorMap map_v,
                           const __grid_constant__ DecodeArgs a) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    constexpr int kWidth = W > 0 ? W : kSlice;             // features per warp
    constexpr int kUnits = W == 64 || W == 0 ? 6 : 3;      // most units of a ring
    constexpr bool kExch = TW != 1;
    __shared__ float4 exch[kExch ? 2 : 1][kExch ? kMaxWarps : 1][kExch ? 2 : 1][kExch ? 32 : 1];
    __shared__ uint64_t s_full[kMaxWarps][kUnits];
    __shared__ uint32_t s_mask[kMaxWarps][kMasks];
    __shared__ long long s_sum[kMaxWarps];
    __shared__ int s_most[kMaxWarps];
    // pieces of each team: [0] goes on with an item (1: and not to its end, 2: to its end), [1] starts
    // one; s_end: [0] is the range's last step
    __shared__ int s_has[kMaxWarps][2], s_end[kMaxWarps];
    __shared__ Item s_item[kMaxWarps][2];
    __shared__ float s_ml[kMaxWarps][2][16];  // their m and l
    static_assert(sizeof(s_ml) >= kMaxWarps * 32 * sizeof(int), "also holds an int per thread");
    int* s_before = reinterpret_cast<int*>(s_ml);
    __shared__ int s_last[2];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, nthreads = blockDim.x, n_warps = nthreads >> 5;
    const int HH = a.Hkv * a.blocks;
    const int tw = TW > 0 ? TW : a.tw, teams = TW > 0 ? kMaxWarps / TW : a.teams;

    if (lane == 0) {
        for (int i = 0; i < kUnits; ++i) mbar_init(&s_full[warp][i], 1);
        fence_mbar_init();
        s_has[warp][0] = s_has[warp][1] = 0;
    }
    if (tid == 0) {
        tma_prefetch_desc(&map_k);
        tma_prefetch_desc(&map_v);
    }
    pdl_launch();
    pdl_wait();
    // ---- this CTA's teams' places in the list: sums of steps over the requests
    const int per_thread = (a.B + nthreads - 1) / nthreads;
    long long mine = 0;
    int longest = 0;
#pragma unroll 1
    for (int b = tid * per_thread; b < min(a.B, (tid + 1) * per_thread); ++b) {
        const int n = span_of(a, b).steps();
        mine += (long long)n * HH;
        longest = max(longest, n);
    }
    long long upto = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const long long u = __shfl_up_sync(0xffffffffu, upto, o);
        if (lane >= o) upto += u;
    }
    longest = __reduce_max_sync(0xffffffffu, longest);
    if (lane == 31) {
        s_sum[warp] = upto;
        s_most[warp] = longest;
    }
    __syncthreads();
    long long total64 = 0, before = upto - mine;
#pragma unroll 1
    for (int w = 0; w < n_warps; ++w) {
        if (w < warp) before += s_sum[w];
        total64 += s_sum[w];
        longest = max(longest, s_most[w]);
    }
    if (total64 >= 1 << 30) {  // (places in the list are counted in 32 bits)
        if (tid == 0) record_error(kErrBadIndex);
        return;
    }
    const int total = (int)total64;
    // Steps per team.  Few items leave few steps to each, but an item's pieces have to be joined
    // by one CTA: about 0.75 us per eight CTAs that share it and task (head and slice) of a
    // warp, against 2 us for a step more, whose sum is least at this square root.  (One step:
    // B2 H16/1 D1024 len <= 2311 takes 75 us, B3 H4/1 D768 len <= 5000 51 us.)
    const int n_teams = gridDim.x * teams;
    const float tasks_per_warp = (float)(min(8, a.group) * tw) / n_warps;
    const int least = (int)sqrtf(0.045f * fmaxf(tasks_per_warp, 1.f) * longest / teams);
    const int per = max(max((total + n_teams - 1) / n_teams, least), 1);
    s_before[tid] = (int)before;
    __syncthreads();

    auto heads_of = [&](int hh) { return min(8, a.group - hh % a.blocks * 8); };
    auto head0_of = [&](int hh) { return hh / a.blocks * a.group + hh % a.blocks * 8; };
    const int team = warp / tw, w_in = warp - team * tw;
    const int my_team = blockIdx.x * teams + team;
    const int g0 = my_team * per, g1 = min(total, g0 + per);
    const int n_steps = max(g1 - g0, 0);
    Cursor cur;
    if (n_steps > 0) {
        int t = 0;  // the last thread whose requests start at or before g0 (nthreads <= 256)
#pragma unroll
        for (int o = kMaxWarps * 16; o > 0; o >>= 1)
            if (t + o < nthreads && s_before[t + o] <= g0) t += o;
        int at = s_before[t], n;
        cur.b = t * per_thread;
        while (g0 >= at + (n = (cur.sp = span_of(a, cur.b)).steps()) * HH) {
            at += n * HH;
            ++cur.b;
        }
        cur.hh = (g0 - at) / n;
        cur.s = cur.sp.s0 + (g0 - at) - cur.hh * n;
    }
    __syncthreads();  // s_before has been read: s_ml may be written
    const int n_units = a.units;
    const uint32_t ring_bytes = n_units * (W == 64 || (W == 0 && a.D <= 64) ? kHalfBytes : 2 * kHalfBytes);
    uint8_t* ring = smem + warp * ring_bytes;
    // pieces that end within the range lie behind the rings, or in the workspace
    const int early_stride = a.early_floats > 0 ? a.early_floats : kSliceFloats;
    float* early0 = a.early_floats > 0 ? reinterpret_cast<float*>(smem + n_warps * ring_bytes)
                                       : a.part + (size_t)gridDim.x * 2 * piece_floats(tw) +
                                             (size_t)blockIdx.x * kMaxWarps * kSliceFloats;
    if (n_steps > 0) {
        const int f0 = w_in * kWidth;                                   // first feature of this warp
        const int width = W > 0 ? W : min(kSlice, a.D - f0);            // its features, a multiple of 8
        const int halves = W > 0 ? W / 64 : (a.D > 64 ? 2 : 1);         // boxes of 64 features per row group
        const uint32_t unit_bytes = halves * kHalfBytes;

        // ---- loads.  Lane l has the box of row group l; units come in the order of use: K of step
        // 0, then K of step j + 1 and V of step j, at last V of the last step.
        const int R = a.box_rows, groups = kStep / R;
        const int boxes = a.merged ? 1 : (width > 64 ? 2 : 1);
        const uint32_t box_bytes = R * 128 * (a.merged ? halves : 1);
        Cursor ld = cur;
        int next_page = 0, next_in = -1;  // table entry of this lane's box of step `ld`; < 0: no key of it is wanted
        auto fetch_page = [&]() {         // (read one step before its load, so that its latency is not waited for)
            const int pos = ld.s * kStep + lane * R;
            next_in = -1;
            if (lane < groups && pos + R > ld.sp.lo && pos < ld.sp.hi) {
                const int p = pos / a.ps;
                next_page = a.table[(size_t)ld.b * a.maxp + p];
                next_in = pos - p * a.ps;
            }
        };
        int k_row = 0, k_in = -1, v_row = 0, v_in = -1;  // this lane's box of the step whose K (V) is loaded
        uint32_t k_bytes = 0, v_bytes = 0;
        int k_next = 0, v_next = 0, load_stage = 0;      // steps whose K and V come next
        bool dead = false;                               // a wait ran out: no further loads or waits
        auto load_next = [&]() {
            if (v_next >= n_steps || dead) return;
            const bool is_k = k_next < n_steps && k_next <= v_next + 1;
            if (is_k || v_next + 1 == k_next) {  // (the last V has no K after it)
                v_row = k_row;
                v_in = k_in;
                v_bytes = k_bytes;
            }
            if (is_k) {
                k_in = next_in;
                if (k_in >= 0 && (unsigned)next_page >= (unsigned)a.pages) {
                    record_error(kErrBadIndex);  // its keys are left out
                    k_in = -1;
                }
                k_row = (int)((unsigned)next_page * a.Hkv + ld.hh / a.blocks);
                const unsigned there = __ballot_sync(0xffffffffu, k_in >= 0);
                k_bytes = __popc(there) * boxes * box_bytes;
                const int pos = ld.s * kStep + lane;
                const unsigned mask =
                    __ballot_sync(0xffffffffu, pos >= ld.sp.lo && pos < ld.sp.hi && ((there >> (lane / R)) & 1));
                if (lane == 0) s_mask[warp][k_next & (kMasks - 1)] = mask;
                if (++k_next < n_steps) {
                    ld.next(a);
                    fetch_page();
                }
            } else {
                ++v_next;
            }
            uint64_t* bar = &s_full[warp][load_stage];
            if (lane == 0) mbar_arrive_expect_tx(bar, is_k ? k_bytes : v_bytes);
            __syncwarp();
            const int in = is_k ? k_in : v_in, row = is_k ? k_row : v_row;
            if (in >= 0) {
                uint8_t* dst = ring + load_stage * unit_bytes + lane * R * 128 * halves;
                const CUtensorMap* map = is_k ? &map_k : &map_v;
                if (a.merged) {
                    tma_load_4d(dst, map, bar, 0, in, f0 / 64, row);
                } else {
                    for (int h = 0; h < boxes; ++h) tma_load_3d(dst + h * R * 128, map, bar, f0 + h * 64, in, row);
                }
            }
            load_stage = load_stage + 1 == n_units ? 0 : load_stage + 1;
        };
        fetch_page();
        for (int i = 0; i < n_units; ++i) load_next();

        // ---- units in use.  Row r of a unit lies at row_at(r), its second half R rows on; 16-byte
        // chunks are swizzled by the address's 128-byte line.
        auto row_at = [&](int r) { return (uint32_t)((r / R) * R * halves + r % R) * 128u; };
        const uint32_t half_at = R * 128, block_at = row_at(16);  // (16 rows on: a multiple of 1024 bytes)
        const int k_hi = lane >> 4, v_hi = (lane >> 3) & 1;
        const uint32_t k_at = row_at(lane & 15), v_at = row_at((lane & 7) + ((lane >> 4) << 3));
        const uint32_t k_x[2] = {(k_at >> 7) & 7, ((k_at + half_at) >> 7) & 7};
        const uint32_t v_x[2] = {(v_at >> 7) & 7, ((v_at + half_at) >> 7) & 7};
        int stage = 0;
        uint32_t phase = 0;
        auto wait_unit = [&]() {
            if (!dead && !__all_sync(0xffffffffu, mbar_wait(&s_full[warp][stage], phase, kErrTimeoutLoad))) dead = true;
            return smem_u32(ring) + stage * unit_bytes;
        };
        auto unit_done = [&]() {
            if (++stage == n_units) {
                stage = 0;
                phase ^= 1u;
            }
            __syncwarp();  // every lane has read the unit
            load_next();
        };

        const int g = lane >> 2, t2 = (lane & 3) * 2;
        uint32_t qf[kWidth / 16][2];
        float o[kWidth / 16][4];
        float m0 = 0.f, m1 = 0.f, l0 = 0.f, l1 = 0.f;  // heads t2, t2 + 1
        float sc[2][4];                                // scores: keys 16 i + g and + 8, heads t2 and t2 + 1
        uint32_t ph[2][2], pl[2][2], mask = 0;
        int buf = 0;
        bool begins = cur.s == cur.sp.s0;
        Cursor nxt = cur;
        for (int step = -1; step < n_steps; ++step) {
            // `cur` is at `step`, `nxt` at the step behind it
            const bool more = step + 1 < n_steps;
            const bool ends = step < 0 || cur.s + 1 == cur.sp.s1;  // (an item, or nothing yet)
            if (more) {
                if (step >= 0) nxt.next(a);
                if (ends) {
                    const int heads = heads_of(nxt.hh);
                    const __nv_bfloat16* q = a.q + ((size_t)nxt.b * a.Hq + head0_of(nxt.hh) + min(g, heads - 1)) * a.D + f0;
#pragma unroll
                    for (int kk = 0; kk < kWidth / 16; ++kk) {
                        const int x = kk * 16 + t2;
                        qf[kk][0] = g < heads && x < width ? *reinterpret_cast<const uint32_t*>(q + x) : 0u;
                        qf[kk][1] = g < heads && x + 8 < width ? *reinterpret_cast<const uint32_t*>(q + x + 8) : 0u;
                    }
                }
                const uint32_t base = wait_unit() + k_at;
#pragma unroll
                for (int i = 0; i < 2; ++i) sc[i][0] = sc[i][1] = sc[i][2] = sc[i][3] = 0.f;
#pragma unroll
                for (int kk = 0; kk < kWidth / 16; ++kk) {
                    if (W == 0 && kk * 16 >= width) break;
                    const uint32_t at = base + (kk >> 2) * half_at + (((2 * (kk & 3) + k_hi) ^ k_x[kk >> 2]) << 4);
                    uint32_t ka[4], kb[4];
                    ldsm4(at, ka);
                    ldsm4(at + block_at, kb);
                    mma_bf16(sc[0], ka, qf[kk][0], qf[kk][1]);
                    mma_bf16(sc[1], kb, qf[kk][0], qf[kk][1]);
                }
                unit_done();
            }
            if (step >= 0) {
                const uint32_t unit = wait_unit();
                if (mask != ~0u) {
                    // rows without a key hold what the page held (or the ring, where no box was
                    // loaded): p = 0 there must meet a finite value
                    if (!((mask >> lane) & 1)) {
                        const uint32_t row = unit + row_at(lane);
                        for (int c = 0; c < halves * 8; ++c)
                            st_shared_v4(row + (c >> 3) * half_at + (c & 7) * 16, 0, 0, 0, 0);
                        fence_proxy_async_shared();  // before the ring's next load of these bytes
                    }
                    __syncwarp();
                }
                const uint32_t base = unit + v_at;
#pragma unroll
                for (int mt = 0; mt < kWidth / 16; ++mt) {
                    if (W == 0 && mt * 16 >= width) break;
                    const uint32_t at = base + (mt >> 2) * half_at + (((2 * (mt & 3) + v_hi) ^ v_x[mt >> 2]) << 4);
                    uint32_t va[4], vb[4];
                    ldsm4_t(at, va);
                    ldsm4_t(at + block_at, vb);
                    mma_bf16(o[mt], va, ph[0][0], ph[0][1]);
                    mma_bf16(o[mt], vb, ph[1][0], ph[1][1]);
                    mma_bf16(o[mt], va, pl[0][0], pl[0][1]);
                    mma_bf16(o[mt], vb, pl[1][0], pl[1][1]);
                }
                unit_done();
                if (ends || !more) {
                    // ---- an item, or a piece of one, is done
                    float s0 = l0, s1 = l1;
#pragma unroll
                    for (int x = 4; x < 32; x <<= 1) {
                        s0 += __shfl_xor_sync(0xffffffffu, s0, x);
                        s1 += __shfl_xor_sync(0xffffffffu, s1, x);
                    }
                    const int heads = heads_of(cur.hh), head0 = head0_of(cur.hh);
                    const bool whole = begins && ends;
                    const float r0 = whole ? (s0 > 0.f ? 1.f / s0 : 0.f) : 1.f;
                    const float r1 = whole ? (s1 > 0.f ? 1.f / s1 : 0.f) : 1.f;
                    const int kind = begins ? 1 : 0;
                    // the last piece of the range may lie in the ring, which is idle then
                    float* part = !more ? reinterpret_cast<float*>(ring) : early0 + warp * early_stride;
#pragma unroll
                    for (int mt = 0; mt < kWidth / 16; ++mt) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int head = t2 + (e & 1), x = mt * 16 + g + (e >> 1) * 8;
                            if (head >= heads || x >= width) continue;
                            const float val = o[mt][e] * ((e & 1) ? r1 : r0);
                            if (!whole) {
                                part[head * kSlice + x] = val;
                            } else {
                                const size_t at = ((size_t)cur.b * a.Hq + head0 + head) * a.D + f0 + x;
                                if (a.out_f32) static_cast<float*>(a.out)[at] = val;
                                else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(val);
                            }
                        }
                    }
                    if (w_in == 0 && g == 0) {
#pragma unroll
                        for (int e = 0; e < 2; ++e) {
                            const int head = t2 + e;
                            if (head >= heads) continue;
                            const float mm = e ? m1 : m0, ll = e ? s1 : s0;
                            if (!whole) {
                                s_ml[team][kind][head] = mm;
                                s_ml[team][kind][8 + head] = ll;
                            } else if (a.lse != nullptr) {
                                a.lse[(size_t)cur.b * a.Hq + head0 + head] = lse_of(mm, ll);
                            }
                        }
                    }
                    if (!whole && w_in == 0 && lane == 0) {
                        s_has[team][kind] = ends ? 2 : 1;
                        if (kind == 0) s_end[team] = !more;
                        s_item[team][kind] =
                            Item{cur.b, cur.hh, g0 + step - (cur.s - cur.sp.s0), g0 + step + (cur.sp.s1 - 1 - cur.s)};
                    }
                    begins = true;  // (the next step, if any, starts an item)
                }
            }
            if (!more) break;
            cur = nxt;
            // ---- whole scores from the team's parts
            if (kExch && tw > 1) {
#pragma unroll
                for (int i = 0; i < 2; ++i) exch[buf][warp][i][lane] = make_float4(sc[i][0], sc[i][1], sc[i][2], sc[i][3]);
                team_sync(team, tw * 32);
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                    float4 s = exch[buf][team * tw][i][lane];
#pragma unroll
                    for (int w = 1; w < (TW > 0 ? TW : kMaxWarps); ++w) {
                        if (TW == 0 && w >= tw) break;
                        const float4 x = exch[buf][team * tw + w][i][lane];
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
            // ---- running maximum and sum; p in two bf16 parts
            if (ends) {
                m0 = m1 = -INFINITY;
                l0 = l1 = 0.f;
#pragma unroll
                for (int mt = 0; mt < kWidth / 16; ++mt) o[mt][0] = o[mt][1] = o[mt][2] = o[mt][3] = 0.f;
            }
            mask = s_mask[warp][(step + 1) & (kMasks - 1)];
            float n0 = m0, n1 = m1;
#pragma unroll
            for (int i = 0; i < 2; ++i) {
#pragma unroll
                for (int e = 0; e < 4; ++e) sc[i][e] *= a.scale_log2;
                if (mask != ~0u) {
                    const bool k0 = (mask >> (16 * i + g)) & 1, k1 = (mask >> (16 * i + g + 8)) & 1;
                    sc[i][0] = k0 ? sc[i][0] : -INFINITY;
                    sc[i][1] = k0 ? sc[i][1] : -INFINITY;
                    sc[i][2] = k1 ? sc[i][2] : -INFINITY;
                    sc[i][3] = k1 ? sc[i][3] : -INFINITY;
                }
                n0 = fmaxf(n0, fmaxf(sc[i][0], sc[i][2]));
                n1 = fmaxf(n1, fmaxf(sc[i][1], sc[i][3]));
            }
#pragma unroll
            for (int x = 4; x < 32; x <<= 1) {
                n0 = fmaxf(n0, __shfl_xor_sync(0xffffffffu, n0, x));
                n1 = fmaxf(n1, __shfl_xor_sync(0xffffffffu, n1, x));
            }
            const float b0 = n0 == -INFINITY ? 0.f : n0, b1 = n1 == -INFINITY ? 0.f : n1;  // nothing seen yet
            if (__any_sync(0xffffffffu, n0 != m0 || n1 != m1)) {  // (seldom, after the first steps)
                const float f0c = ex2f(m0 - b0), f1c = ex2f(m1 - b1);
                l0 *= f0c;
                l1 *= f1c;
#pragma unroll
                for (int mt = 0; mt < kWidth / 16; ++mt) {
                    o[mt][0] *= f0c;
                    o[mt][1] *= f1c;
                    o[mt][2] *= f0c;
                    o[mt][3] *= f1c;
                }
                m0 = n0;
                m1 = n1;
            }
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

    // requests without keys: their output is zero
#pragma unroll 1
    for (int b = blockIdx.x; b < a.B; b += gridDim.x) {
        const int len = a.lengths[b];
        if (tid == 0 && len > a.width) record_error(kErrBadIndex);  // longer than the table is wide
        if (len > 0 && a.width > 0) continue;
#pragma unroll 1
        for (int i = tid; i < a.Hq * a.D; i += nthreads) {
            const size_t at = (size_t)b * a.Hq * a.D + i;
            if (a.out_f32) static_cast<float*>(a.out)[at] = 0.f;
            else static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(0.f);
        }
        if (a.lse != nullptr)
            for (int i = tid; i < a.Hq; i += nthreads) a.lse[(size_t)b * a.Hq + i] = -INFINITY;
    }
    if (blockIdx.x * teams * per >= total) return;  // no steps for this CTA

    // ---- joining.  One head and 128 features of n pieces per warp, a lane four features:
    // unnormalised sum, m and l; load_o(i) gives piece i's four features, load_ml(i, j) its m and l.
    auto join = [&](auto ahead, int n, auto load_o, auto load_ml, float4& acc, float& top, float& l) {
        constexpr int kAhead = decltype(ahead)::value;  // pieces whose loads are in flight
        top = -INFINITY;
        l = 0.f;
        acc = make_float4(0.f, 0.f, 0.f, 0.f);
        for (int i0 = 0; i0 < n; i0 += kAhead) {
            float4 x[kAhead];
            float m[kAhead], li[kAhead], nt = top;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                if (i0 + k < n) {
                    x[k] = load_o(i0 + k);
                    m[k] = load_ml(i0 + k, 0);
                    li[k] = load_ml(i0 + k, 8);
                } else {
                    x[k] = make_float4(0.f, 0.f, 0.f, 0.f);
                    m[k] = -INFINITY;
                    li[k] = 0.f;
                }
            }
#pragma unroll
            for (int k = 0; k < kAhead; ++k) nt = fmaxf(nt, m[k]);
            const float base = nt == -INFINITY ? 0.f : nt, w0 = ex2f(top - base);
            top = nt;
            l *= w0;
            acc.x *= w0;
            acc.y *= w0;
            acc.z *= w0;
            acc.w *= w0;
#pragma unroll
            for (int k = 0; k < kAhead; ++k) {
                const float w = ex2f(m[k] - base);
                l = __fmaf_rn(w, li[k], l);
                acc.x = __fmaf_rn(w, x[k].x, acc.x);
                acc.y = __fmaf_rn(w, x[k].y, acc.y);
                acc.z = __fmaf_rn(w, x[k].z, acc.z);
                acc.w = __fmaf_rn(w, x[k].w, acc.w);
            }
        }
    };
    auto store = [&](const Item& it, int head, int slice, const float4& acc, float top, float l) {
        const float r = l > 0.f ? 1.f / l : 0.f;
        const size_t row = (size_t)it.b * a.Hq + head0_of(it.hh) + head;
        const int c = slice * kWidth + lane * 4;
        if (lane * 4 < kWidth && c < a.D) {
            if (a.out_f32)
                *reinterpret_cast<float4*>(static_cast<float*>(a.out) + row * a.D + c) =
                    make_float4(acc.x * r, acc.y * r, acc.z * r, acc.w * r);
            else
                *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(a.out) + row * a.D + c) =
                    make_uint2(pack_bf16(acc.x * r, acc.y * r), pack_bf16(acc.z * r, acc.w * r));
        }
        if (a.lse != nullptr && c == 0) a.lse[row] = lse_of(top, l);
    };
    const size_t pf = piece_floats(tw);
    __syncthreads();
    // within the CTA: the item that comes in (t = -1), and those that a team starts and does
    // not finish; the warps take (item, head, slice) in turn
    Item in_item{}, out_item{};
    bool has_in = false, has_out = false;
    int turn = 0;
    for (int t = -1; t < teams; ++t) {
        const int from = t < 0 ? 0 : t, kind = t < 0 ? 0 : 1;
        if (s_has[from][kind] == 0) continue;
        const Item it = s_item[from][kind];
        int n = 1;
        bool ended = s_has[from][kind] == 2;
        while (!ended && from + n < teams && s_has[from + n][0] != 0) {
            ended = s_has[from + n][0] == 2;
            ++n;
        }
        const bool whole = kind == 1 && ended;
        const int tasks = heads_of(it.hh) * tw;
        for (int q = (warp - turn % n_warps + n_warps) % n_warps; q < tasks; q += n_warps) {
            const int head = q / tw, slice = q - head * tw;
            // (a team's piece lies in its rings if it is the last of the team's range)
            auto load_o = [&](int i) {
                const int w = (from + i) * tw + slice;
                const bool in_ring = (i == 0 && kind == 1) || s_end[from + i];
                const float* o_p = in_ring ? reinterpret_cast<const float*>(smem + w * ring_bytes)
                                           : early0 + w * early_stride;
                return reinterpret_cast<const float4*>(o_p + head * kSlice)[lane];
            };
            auto load_ml = [&](int i, int j) { return s_ml[from + i][i == 0 ? kind : 0][j + head]; };
            float4 acc;
            float top, l;
            join(std::integral_constant<int, kMaxWarps>{}, n, load_o, load_ml, acc, top, l);
            if (whole) {
                store(it, head, slice, acc, top, l);
            } else {
                float* p = a.part + (size_t)(blockIdx.x * 2 + kind) * pf;
                reinterpret_cast<float4*>(p + (size_t)slice * kSliceFloats + head * kSlice)[lane] = acc;
                if (slice == 0 && lane == 0) {
                    p[(size_t)tw * kSliceFloats + head] = top;
                    p[(size_t)tw * kSliceFloats + 8 + head] = l;
                }
            }
        }
        turn += tasks;
        if (!whole) {
            if (kind == 0) {
                in_item = it;
                has_in = true;
            } else {
                out_item = it;
                has_out = true;
            }
        }
    }
    if (!has_in && !has_out) return;  // (uniform over the CTA)
    // across CTAs: each raises the flag of its piece, then looks at the flags of all pieces of
    // the item.  The last to raise one sees them all and joins them (so may another that
    // looks later: it writes the same), and lowers the flags for a replay of this call.
    const int cta_steps = per * teams;
    __syncthreads();
    if (tid == 0) {
        __threadfence();  // this CTA's pieces before their flags
        if (has_in) *reinterpret_cast<volatile unsigned long long*>(a.flags + blockIdx.x * 2) = a.tag;
        if (has_out) *reinterpret_cast<volatile unsigned long long*>(a.flags + blockIdx.x * 2 + 1) = a.tag;
        __threadfence();  // and the flags before the look at the others'
    }
    __syncthreads();
    // warp 0 looks at the item that goes out, warp 1 (or 0) at the one that comes in
    for (int kind = 1; kind >= 0; --kind) {
        if (warp != (kind == 1 || n_warps == 1 ? 0 : 1)) continue;
        bool all = kind ? has_out : has_in;
        const Item it = kind ? out_item : in_item;
        const int c0 = it.first / cta_steps, n = all ? it.last / cta_steps - c0 + 1 : 0;
        for (int i = lane; i < n; i += 32)
            all = all && *reinterpret_cast<volatile unsigned long long*>(
                             a.flags + (size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0)) == a.tag;
        all = __all_sync(0xffffffffu, all);
        if (lane == 0) s_last[kind] = all;
        __threadfence();  // the others' pieces after their flags
    }
    __syncthreads();
    turn = 0;
    for (int kind = 1; kind >= 0; --kind) {
        if (!s_last[kind]) continue;
        const Item it = kind ? out_item : in_item;
        const int c0 = it.first / cta_steps, n = it.last / cta_steps - c0 + 1;
        auto index = [&](int i) { return (size_t)(c0 + i) * 2 + (i == 0 ? 1 : 0); };
        const int tasks = heads_of(it.hh) * tw;
        for (int q = (warp - turn % n_warps + n_warps) % n_warps; q < tasks; q += n_warps) {
            const int head = q / tw, slice = q - head * tw;
            float4 acc;
            float top, l;
            // (written by other SMs while this kernel runs: past L1)
            join(std::integral_constant<int, 16>{}, n,
                 [&](int i) {
                     return __ldcg(reinterpret_cast<const float4*>(a.part + index(i) * pf +
                                                                   (size_t)slice * kSliceFloats + head * kSlice) + lane);
                 },
                 [&](int i, int j) { return __ldcg(a.part + index(i) * pf + (size_t)tw * kSliceFloats + j + head); },
                 acc, top, l);
            store(it, head, slice, acc, top, l);
        }
        turn += tasks;
        for (int i = tid; i < n; i += nthreads) a.flags[index(i)] = 0;
    }
}

}  // namespace cache
}  // namespace sru

// sru_cache.cuh -- the paged key/value cache of SRU++ decoding: its page
// bookkeeping for one serving step and the append of new rows.
//
// "When Attention Meets Fast Recurrence" attends, at inference, to the keys and
// values of the tokens seen so far.  Those live in pages of ps tokens,
//   k_cache, v_cache (pages, Hkv, ps, D) bf16:
// one head of one page is ps x D consecutive elements, which the attention
// reads in whole lines.  Request b's token t is row t % ps of page
// table[b][t / ps]; its slot is table[b][t / ps] * ps + t % ps.  Pages that no
// request holds lie on a stack free_pages[0 .. n_free).
#pragma once

#include "sru_ptx.cuh"

namespace sru {
namespace cache {

// ---------------------------------------------------------------- page bookkeeping
// For request b with len tokens and `add` new ones (add < 0: released):
//   held = ceil(len / ps);  a released request's pages go onto the stack, in
//   request order; then, in request order, need = ceil((len + add) / ps) - held
//   pages come off its top, as long as the running sum of the needs stays within
//   the stack's height (and the tokens within the table's width and the step's
//   rows), else the request is refused and keeps what it had.
// Two passes over the requests, a thread each: running sums of the new tokens and
// of the released pages, then of the needs.  The call is bound by latency, so one
// CTA, no wider than the requests need, does the sums and everything that a
// request's own thread or warp can write.  A step with room for many rows gets a
// second kernel over the rows for the requests of more than kExtDirect tokens; it
// learns from such a request's first slot, written here, whether it was refused.
// (A cluster of 8 CTAs that all made the sums took 47 us where this takes 16: B1024 with
// 600 thousand rows; a step of B48 takes 9, of which the kernel is 4.5 and the call the rest.)
constexpr int kExtThreads = 1024;
constexpr int kExtDirect = 4;  // tokens that a request's own thread writes

struct ExtendArgs {
    const int *lengths, *add;
    int *table, *free_pages;
    const int* n_free;
    int *lengths_out, *n_free_out, *offsets, *slots, *refused;
    int B, maxp, pages, ps, T;
    int rows_kernel;  // long runs of slots are left to cache_slots_kernel
};

// Inclusive sum over the warp's lanes.
__device__ __forceinline__ unsigned long long warp_inclusive(unsigned long long v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const unsigned long long u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
// The same over the block's threads; `total` gets the whole sum.
__device__ __forceinline__ unsigned long long block_inclusive(unsigned long long v, unsigned long long* warp_sums,
                                                              unsigned long long& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, n_warps = blockDim.x >> 5;
    v = warp_inclusive(v, lane);
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    const unsigned long long w = warp_inclusive(lane < n_warps ? warp_sums[lane] : 0ull, lane);
    total = __shfl_sync(0xffffffffu, w, 31);
    const unsigned long long before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    __syncthreads();  // warp_sums may be written again
    return v + (warp == 0 ? 0ull : before);
}

// The n (per lane) items of a warp's lanes, shared out evenly over the lanes, four at a
// time each: store(src, i, load(src, i)) for item i of lane src.
template <typename Load, typename Store>
__device__ __forceinline__ void warp_spread(int n, Load load, Store store) {
    const int lane = threadIdx.x & 31;
    const int upto = (int)warp_inclusive((unsigned long long)n, lane);
    const int total = __shfl_sync(0xffffffffu, upto, 31);
    for (int b = 0; b < total; b += 128) {
        int src[4], i[4], v[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            const int e = b + k * 32 + lane;
            src[k] = 0;  // the first lane whose running sum passes e
#pragma unroll
            for (int o = 16; o > 0; o >>= 1)
                if (__shfl_sync(0xffffffffu, upto, src[k] + o - 1) <= e) src[k] += o;
            const int before = __shfl_sync(0xffffffffu, upto - n, src[k]);
            const int items = __shfl_sync(0xffffffffu, n, src[k]);
            i[k] = e - before;
            if (e >= total || i[k] >= items) i[k] = -1;
            v[k] = load(src[k], i[k]);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) store(src[k], i[k], v[k]);
    }
}

__global__ void __launch_bounds__(kExtThreads) cache_extend_kernel(ExtendArgs a) {
    __shared__ unsigned long long sums[kExtThreads / 32];
    __shared__ int s_refused, s_taken;
    const int tid = threadIdx.x, lane = tid & 31, nt = blockDim.x;
    pdl_launch();
    pdl_wait();
    if (tid == 0) s_refused = s_taken = 0;
    const long long width = (long long)a.maxp * a.ps;
    const int n_free = max(0, min(*a.n_free, a.pages));

    int len = 0, add = 0, held = 0;
    auto read = [&](int b) {
        len = b < a.B ? max(a.lengths[b], 0) : 0;
        add = b < a.B ? a.add[b] : 0;
        held = min((int)(((long long)len + a.ps - 1) / a.ps), a.maxp);
    };
    // an entry of the stack once the released pages lie on it
    auto stack = [&](int i) { return i >= 0 && i < a.pages ? a.free_pages[i] : -1; };

    // ---- released pages onto the stack; sums: new tokens (low word), released pages (high)
    unsigned long long upto = 0, total = 0;
    int gone_before = 0;
    for (int b0 = 0; b0 < a.B; b0 += nt) {
        read(b0 + tid);
        const int gone = add < 0 ? held : 0;
        upto = block_inclusive((unsigned)max(add, 0) | (unsigned long long)gone << 32, sums, total);
        const int base = n_free + gone_before + (int)(upto >> 32) - gone;
        const int warp_b = b0 + tid - lane;
        warp_spread(
            gone, [&](int src, int i) { return i >= 0 ? a.table[(size_t)(warp_b + src) * a.maxp + i] : 0; },
            [&](int src, int i, int page) {
                const int at = __shfl_sync(0xffffffffu, base, src) + i;
                if (i >= 0 && at >= 0 && at < a.pages) a.free_pages[at] = page;
            });
        gone_before += (int)(total >> 32);
    }
    __syncthreads();
    const int avail = min(n_free + gone_before, a.pages);

    // ---- grants, table entries, slots and lengths
    unsigned first_before = 0;
    int need_before = 0;
    for (int b0 = 0; b0 < a.B; b0 += nt) {
        const int b = b0 + tid;
        if (a.B > nt) {  // (one chunk: its values are still at hand)
            read(b);
            upto = block_inclusive((unsigned)max(add, 0), sums, total);
        }
        const int grow = max(add, 0);
        const unsigned last = first_before + (unsigned)upto, first = last - grow;
        first_before += (unsigned)total;
        const long long end = (long long)len + grow;
        const bool fits = grow > 0 && end <= width && last <= (unsigned)a.T;
        const int need = fits ? (int)((end + a.ps - 1) / a.ps) - held : 0;
        const int wanted = need_before + (int)block_inclusive((unsigned)need, sums, total);
        need_before += (int)total;
        const bool ok = fits && (need == 0 || wanted <= avail);
        const int refused = __popc(__ballot_sync(0xffffffffu, grow > 0 && !ok));
        const int taken = __reduce_max_sync(0xffffffffu, ok && need > 0 ? wanted : 0);  // grants are a prefix of the needs
        if (lane == 0) {
            if (refused) atomicAdd(&s_refused, refused);
            if (taken) atomicMax(&s_taken, taken);
        }
        // page p >= held of this request is stack entry top - p
        const int top = avail - 1 - (wanted - need) + held, take = ok ? need : 0;
        int* row = a.table + (size_t)b * a.maxp;
        const int warp_b = b0 + tid - lane;
        warp_spread(
            take,
            [&](int src, int i) {
                const int p = __shfl_sync(0xffffffffu, held, src) + i, from = __shfl_sync(0xffffffffu, top, src);
                return i >= 0 ? stack(from - p) : 0;
            },
            [&](int src, int i, int page) {
                const int p = __shfl_sync(0xffffffffu, held, src) + i;
                if (i >= 0) a.table[(size_t)(warp_b + src) * a.maxp + p] = page;
            });
        // slot of token j of a request
        auto slot = [&](const int* r, int len_, int held_, int top_, int j) {
            const int pos = len_ + j, p = pos / a.ps;
            const int page = p < held_ ? r[p] : stack(top_ - p);
            return page < 0 ? -1 : page * a.ps + (pos - p * a.ps);
        };
        // (a refused request's rows may reach behind T; `first` below T is below 2^31)
        if (grow > 0 && first < (unsigned)a.T) {
            const int n = grow <= kExtDirect ? grow : (a.rows_kernel ? 1 : 0);
            for (int j = 0; j < n; ++j)
                if (first + j < (unsigned)a.T) a.slots[first + j] = ok ? slot(row, len, held, top, j) : -1;
        }
        if (!a.rows_kernel) {
            const int rows = grow > kExtDirect && first < (unsigned)a.T ? min(grow, a.T - (int)first) : 0;
            warp_spread(
                rows,
                [&](int src, int i) {
                    const int len_ = __shfl_sync(0xffffffffu, len, src), held_ = __shfl_sync(0xffffffffu, held, src);
                    const int top_ = __shfl_sync(0xffffffffu, top, src);
                    const bool ok_ = __shfl_sync(0xffffffffu, (int)ok, src) != 0;
                    return i >= 0 && ok_ ? slot(a.table + (size_t)(warp_b + src) * a.maxp, len_, held_, top_, i) : -1;
                },
                [&](int src, int i, int s) {
                    const int at = (int)__shfl_sync(0xffffffffu, first, src);
                    if (i >= 0) a.slots[at + i] = s;
                });
        }
        if (b < a.B) {
            a.lengths_out[b] = add < 0 ? 0 : (ok ? (int)end : len);
            a.offsets[b] = (int)first;
        }
    }
    __syncthreads();
    if (!a.rows_kernel)  // rows behind the last token
        for (unsigned i = first_before + tid; i < (unsigned)a.T; i += nt) a.slots[i] = -1;
    if (tid == 0) {
        a.offsets[a.B] = (int)first_before;
        *a.n_free_out = avail - s_taken;
        if (a.refused != nullptr) *a.refused = s_refused;
    }
}

// The slots that cache_extend_kernel leaves: rows of requests with more than
// kExtDirect tokens (all but the first row) and the rows behind the last token.  A
// warp takes kSlotRows consecutive rows, finds the request of its first one by
// a 33-way search of the offsets and walks on from there.
constexpr int kSlotRows = 128;
__global__ void __launch_bounds__(256) cache_slots_kernel(ExtendArgs a) {
    pdl_launch();
    pdl_wait();
    const int lane = threadIdx.x & 31;
    const long long t0 = ((long long)blockIdx.x * 8 + (threadIdx.x >> 5)) * kSlotRows;
    if (t0 >= a.T) return;
    const int total = a.offsets[a.B];
    int lo = 0, hi = a.B;  // offsets[lo] <= t0 < offsets[hi], if t0 < total
    while (hi - lo > 1) {
        const int probe = lo + (int)((long long)(hi - lo) * (lane + 1) / 33);
        const int n = __popc(__ballot_sync(0xffffffffu, a.offsets[probe] <= t0));  // (probe = lo counts)
        const int new_lo = n == 0 ? lo : lo + (int)((long long)(hi - lo) * n / 33);
        if (n < 32) hi = lo + (int)((long long)(hi - lo) * (n + 1) / 33);
        lo = new_lo;
    }
    int b = lo;
#pragma unroll
    for (int i = 0; i < kSlotRows; i += 32) {
        const int t = (int)t0 + i + lane;
        if (t >= a.T) return;
        if (t >= total) {
            a.slots[t] = -1;
            continue;
        }
        while (a.offsets[b + 1] <= t) ++b;
        const int first = a.offsets[b], n = a.offsets[b + 1] - first;
        if (n <= kExtDirect || t == first) continue;
        int s = -1;
        // (offsets that wrapped, from 2^31 tokens in one step, lead outside neither array)
        if ((unsigned)first < (unsigned)a.T && a.slots[first] >= 0) {
            const int pos = a.lengths_out[b] - n + (t - first), p = pos / a.ps;
            const int page = pos >= 0 && p < a.maxp ? a.table[(size_t)b * a.maxp + p] : -1;
            if (page >= 0) s = page * a.ps + (pos - p * a.ps);
        }
        a.slots[t] = s;
    }
}

// -------------------------------------------------------------------------- append
// Row r of K and V (T rows of Hkv * D elements, k_ld / v_ld apart) to slot
// slots[r] of the caches, rounded to bf16; a negative slot writes nothing.  Pure
// copy, bound by memory: 16-byte items, four in flight per thread (16384 rows of K and
// V, d' 512: 67 MB in 12.1 us, 5.6 TB/s; one item per thread: 18.6 us).  Plain loads: the
// kernels before it may still write rows and slots when it starts.
template <typename SrcT>
__device__ __forceinline__ uint4 load8_bf16(const SrcT* p) {
    if (sizeof(SrcT) == 2) return *reinterpret_cast<const uint4*>(p);
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    __nv_bfloat162 w[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                           __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
    return *reinterpret_cast<uint4*>(w);
}
constexpr int kAppendItems = 4;  // 16-byte stores per thread, their loads issued together
template <typename SrcT>
__global__ void __launch_bounds__(256)
    cache_append_kernel(const SrcT* K, long long k_ld, const SrcT* V, long long v_ld, const int* slots,
                        __nv_bfloat16* k_cache, __nv_bfloat16* v_cache, unsigned items, int Hkv, int D, int ps,
                        long long n_slots) {
    pdl_launch();
    pdl_wait();
    const SrcT* src = blockIdx.y == 0 ? K : V;
    const long long ld = blockIdx.y == 0 ? k_ld : v_ld;
    __nv_bfloat16* dst = blockIdx.y == 0 ? k_cache : v_cache;
    const unsigned vd = D / 8, per_row = Hkv * vd;
    const unsigned i0 = blockIdx.x * (256u * kAppendItems) + threadIdx.x;
    uint4 v[kAppendItems];
    int slot[kAppendItems];
    unsigned col[kAppendItems];
#pragma unroll
    for (int k = 0; k < kAppendItems; ++k) {
        const unsigned i = i0 + k * 256u;
        slot[k] = -1;
        if (i < items && i >= i0) {
            const unsigned r = i / per_row;
            col[k] = i - r * per_row;
            slot[k] = slots[r];
            v[k] = load8_bf16(src + r * ld + (long long)col[k] * 8);
        }
    }
#pragma unroll
    for (int k = 0; k < kAppendItems; ++k) {
        if (slot[k] < 0) continue;
        if (slot[k] >= n_slots) {
            record_error(kErrBadIndex);
            continue;
        }
        const unsigned h = col[k] / vd, page = (unsigned)slot[k] / ps;
        const size_t at = (((size_t)page * Hkv + h) * ps + (slot[k] - page * ps)) * D + (size_t)(col[k] - h * vd) * 8;
        *reinterpret_cast<uint4*>(dst + at) = v[k];
    }
}

}  // namespace cache
}  // namespace sru

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
// Three running sums (new tokens, released pages, needed pages) over the
// requests, then independent writes.  The call is bound by latency: one launch
// of one CTA, or of one cluster of 8 when there are many slots to write; every
// CTA computes the sums of all requests (8 bytes each), which costs less than
// passing them on, and the cluster's barrier orders pushes before pops and
// reads before in-place writes.
constexpr int kExtThreads = 1024;
constexpr int kExtDirect = 8;   // tokens that a request's own thread writes; more are shared out in segments
constexpr int kExtSeg = 256;    // tokens per segment (one warp)

struct ExtendArgs {
    const int *lengths, *add;
    int *table, *free_pages;
    const int* n_free;
    int *lengths_out, *n_free_out, *offsets, *slots, *refused;
    int B, maxp, pages, ps, T;
};

template <typename T>
__device__ __forceinline__ T warp_inclusive(T v, int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const T u = __shfl_up_sync(0xffffffffu, v, o);
        if (lane >= o) v += u;
    }
    return v;
}
// Inclusive sum over the block's threads; `total` gets the whole sum.
template <typename T>
__device__ __forceinline__ T block_inclusive(T v, T* warp_sums, T& total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    v = warp_inclusive(v, lane);
    __syncthreads();  // warp_sums may still be read from the last use
    if (lane == 31) warp_sums[warp] = v;
    __syncthreads();
    const T w = warp_inclusive(lane < kExtThreads / 32 ? warp_sums[lane] : T(0), lane);
    total = __shfl_sync(0xffffffffu, w, 31);
    const T before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return v + (warp == 0 ? T(0) : before);
}

__global__ void __launch_bounds__(kExtThreads) cache_extend_kernel(ExtendArgs a) {
    __shared__ long long sums[kExtThreads / 32];
    // this chunk's requests, for the segments
    __shared__ int s_seg[kExtThreads], s_first[kExtThreads], s_len[kExtThreads], s_held[kExtThreads],
        s_top[kExtThreads], s_add[kExtThreads];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t rank = 0, ncta = gridDim.x;
    if (ncta > 1) rank = cluster_ctarank();
    const long long width = (long long)a.maxp * a.ps;
    const int n_free = max(0, min(*a.n_free, a.pages));

    auto read = [&](int b, int& len, int& add, int& held) {
        len = b < a.B ? max(a.lengths[b], 0) : 0;
        add = b < a.B ? a.add[b] : 0;
        held = (int)min((long long)(len / a.ps) + (len % a.ps != 0), (long long)a.maxp);
    };
    // a page of the stack once the released pages lie on it
    auto stack = [&](long long i) { return i >= 0 && i < a.pages ? a.free_pages[i] : -1; };

    // ---- released pages onto the stack
    long long gone_before = 0;
    for (int b0 = 0; b0 < a.B; b0 += kExtThreads) {
        int len, add, held;
        read(b0 + tid, len, add, held);
        const int gone = add < 0 ? held : 0;
        long long total;
        const long long upto = block_inclusive<long long>(gone, sums, total);
        const long long base = n_free + gone_before + upto - gone;
        if ((uint32_t)warp % ncta == rank) {
            for (unsigned left = __ballot_sync(0xffffffffu, gone > 0); left != 0; left &= left - 1) {
                const int src = __ffs(left) - 1;
                const int n = __shfl_sync(0xffffffffu, gone, src);
                const long long at = __shfl_sync(0xffffffffu, base, src);
                const int* row = a.table + (size_t)(b0 + warp * 32 + src) * a.maxp;
                for (int i = lane; i < n; i += 32)
                    if (at + i < a.pages) a.free_pages[at + i] = row[i];
            }
        }
        gone_before += total;
    }
    if (ncta > 1) cluster_sync_all();
    else __syncthreads();
    const long long avail = min(n_free + gone_before, (long long)a.pages);

    // ---- grants, slots and lengths
    long long first_before = 0, need_before = 0, taken = 0;
    int refused = 0;
    for (int b0 = 0; b0 < a.B; b0 += kExtThreads) {
        const int b = b0 + tid;
        int len, add, held;
        read(b, len, add, held);
        const int grow = max(add, 0);
        if (ncta > 1) cluster_sync_all();  // every CTA has read this chunk: it may be written in place
        long long total;
        const long long last = first_before + block_inclusive<long long>(grow, sums, total);
        first_before += total;
        const long long first = last - grow, end = (long long)len + grow;
        const bool fits = grow > 0 && end <= width && last <= a.T;
        const int need = fits ? (int)((end + a.ps - 1) / a.ps) - held : 0;
        const long long upto = need_before + block_inclusive<long long>(need, sums, total);
        need_before += total;
        const bool ok = fits && (need == 0 || upto <= avail);
        const int take = ok ? need : 0;
        block_inclusive<long long>(take, sums, total);
        taken += total;
        refused += __syncthreads_count(grow > 0 && !ok);
        // page index i >= held of this request is stack entry top - i
        const int top = (int)(avail - 1 - (upto - need)) + held;
        const bool direct = grow <= kExtDirect;
        const int seg = direct ? 0 : (int)((min((long long)grow, max(0ll, a.T - first)) + kExtSeg - 1) / kExtSeg);
        long long segs;
        const long long seg_upto = block_inclusive<long long>(seg, sums, segs);
        s_seg[tid] = (int)seg_upto;
        s_first[tid] = (int)min(first, (long long)a.T);
        s_len[tid] = len;
        s_held[tid] = held;
        s_top[tid] = top;
        s_add[tid] = ok ? grow : -grow;  // negative: refused
        auto token = [&](int bb, int j, int len_, int held_, int top_, bool ok_, long long at) {
            int slot = -1;
            if (ok_) {
                const int pos = len_ + j, p = pos / a.ps, in = pos - p * a.ps;
                const int page = p < held_ ? a.table[(size_t)bb * a.maxp + p] : stack(top_ - p);
                if (p >= held_ && in == 0) a.table[(size_t)bb * a.maxp + p] = page;  // its first token is new
                if (page >= 0) slot = page * a.ps + in;
            }
            if (at < a.T) a.slots[at] = slot;
        };
        if (direct && (uint32_t)warp % ncta == rank)
            for (int j = 0; j < grow; ++j) token(b, j, len, held, top, ok, first + j);
        __syncthreads();
        for (long long q = (long long)rank * (kExtThreads / 32) + warp; q < segs;
             q += (long long)ncta * (kExtThreads / 32)) {
            int lo = 0, hi = kExtThreads - 1;  // the first request whose running segment count passes q
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (s_seg[mid] > q) hi = mid;
                else lo = mid + 1;
            }
            const int j0 = (int)(q - (lo == 0 ? 0 : s_seg[lo - 1])) * kExtSeg;
            const int n = abs(s_add[lo]);
#pragma unroll
            for (int k = 0; k < kExtSeg; k += 32)
                if (j0 + k + lane < n)
                    token(b0 + lo, j0 + k + lane, s_len[lo], s_held[lo], s_top[lo], s_add[lo] > 0,
                          (long long)s_first[lo] + j0 + k + lane);
        }
        if (rank == 0 && b < a.B) {
            a.lengths_out[b] = add < 0 ? 0 : (ok ? (int)end : len);
            a.offsets[b] = (int)first;
        }
        __syncthreads();
    }
    // rows behind the last token
    for (long long i = first_before + (long long)rank * kExtThreads + tid; i < a.T; i += (long long)ncta * kExtThreads)
        a.slots[i] = -1;
    if (rank == 0 && tid == 0) {
        a.offsets[a.B] = (int)first_before;
        *a.n_free_out = (int)(avail - taken);
        if (a.refused != nullptr) *a.refused = refused;
    }
}

// -------------------------------------------------------------------------- append
// Row r of K and V (T rows of Hkv * D elements, k_ld / v_ld apart) to slot
// slots[r] of the caches, rounded to bf16; a negative slot writes nothing.  Pure
// copy: 16-byte stores, one per thread and item.
template <typename SrcT>
__device__ __forceinline__ uint4 load8_bf16(const SrcT* p) {
    if (sizeof(SrcT) == 2) return __ldg(reinterpret_cast<const uint4*>(p));
    const float4 a = __ldg(reinterpret_cast<const float4*>(p)), b = __ldg(reinterpret_cast<const float4*>(p) + 1);
    __nv_bfloat162 w[4] = {__floats2bfloat162_rn(a.x, a.y), __floats2bfloat162_rn(a.z, a.w),
                           __floats2bfloat162_rn(b.x, b.y), __floats2bfloat162_rn(b.z, b.w)};
    return *reinterpret_cast<uint4*>(w);
}
template <typename SrcT>
__global__ void __launch_bounds__(256)
    cache_append_kernel(const SrcT* __restrict__ K, long long k_ld, const SrcT* __restrict__ V, long long v_ld,
                        const int* __restrict__ slots, __nv_bfloat16* __restrict__ k_cache,
                        __nv_bfloat16* __restrict__ v_cache, int T, int Hkv, int D, int ps, long long n_slots) {
    const SrcT* src = blockIdx.y == 0 ? K : V;
    const long long ld = blockIdx.y == 0 ? k_ld : v_ld;
    __nv_bfloat16* dst = blockIdx.y == 0 ? k_cache : v_cache;
    const int vd = D / 8, per_row = Hkv * vd;
    const long long n = (long long)T * per_row;
    for (long long i = blockIdx.x * 256ll + threadIdx.x; i < n; i += gridDim.x * 256ll) {
        const int r = (int)(i / per_row), c = (int)(i - (long long)r * per_row);
        const int slot = slots[r];
        if (slot < 0) continue;
        if (slot >= n_slots) {
            record_error(kErrBadIndex);
            continue;
        }
        const int h = c / vd, page = slot / ps;
        const size_t at = (((size_t)page * Hkv + h) * ps + (slot - page * ps)) * D + (size_t)(c - h * vd) * 8;
        *reinterpret_cast<uint4*>(dst + at) = load8_bf16(src + r * ld + (long long)c * 8);
    }
}

}  // namespace cache
}  // namespace sru

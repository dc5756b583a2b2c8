// kv_plan.hip -- page tables, slots and positions of a serving step, built on
// the GPU from the requests' lengths, and the release of finished requests'
// pages.
//
// A step needs two exclusive prefix sums over the requests (new rows, new
// pages); everything else follows from them per row and per new page.  The
// work is a few KB to a few hundred KB, so the time is latency: one launch
// and no exchange between workgroups.  Every workgroup computes the prefix
// sums itself, 1024 requests at a time (12 bytes each, from the L2 after the
// first reader), and then serves its own share of the rows and of the new
// pages; nothing that one workgroup writes is read by another.  8 requests 4.1
// us, 512 requests with 35k rows 8.0 us (a launch that does nothing: about 2).
#include "kv.h"

namespace ht {

namespace {

constexpr int kThreads = 256;
constexpr int kItems = 4;
constexpr int kChunk = kThreads * kItems;   // requests per pass
constexpr int32_t kRefused = INT32_MIN;

struct PlanKv {
    const int32_t *q_len, *kv_len, *owned;
    int32_t *table;
    const int32_t *free_pages, *n_free;
    int32_t *cu_q, *slots, *positions, *kv_out, *owned_out, *status;
    int64_t ldt;
    int32_t R, P, T, free_cap, rows_per_wg;
};

// Exclusive sums of (a, b) over the workgroup's threads, and their totals (64
// bits: what all requests ask for together may pass 2^31).
__device__ __forceinline__ void wg_scan(int64_t &a, int64_t &b, int64_t &ta, int64_t &tb, int64_t (*part)[2]) {
    const int lane = threadIdx.x & 63, wv = threadIdx.x >> 6;
    int64_t ia = a, ib = b;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
        const int64_t ua = __shfl_up(ia, d), ub = __shfl_up(ib, d);
        if (lane >= d) { ia += ua; ib += ub; }
    }
    if (lane == 63) { part[wv][0] = ia; part[wv][1] = ib; }
    __syncthreads();
    int64_t ba = 0, bb = 0;
    ta = 0; tb = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 64; ++w) {
        if (w < wv) { ba += part[w][0]; bb += part[w][1]; }
        ta += part[w][0];
        tb += part[w][1];
    }
    a = ba + ia - a;
    b = bb + ib - b;
}

// Largest i in [0, n) with v[i] <= x (v not decreasing, v[0] <= x).
__device__ __forceinline__ int last_le(const int32_t *v, int n, int32_t x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (v[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

__global__ __launch_bounds__(kThreads) void kv_plan_kernel(PlanKv a) {
    __shared__ int32_t cu[kChunk], kv[kChunk], own[kChunk];
    __shared__ int32_t pre[kChunk];     // new pages asked for before the request (avail + 1 at most)
    __shared__ int32_t first[kChunk];   // free-list place of its first new page; kRefused
    __shared__ int64_t part[kThreads / 64][2];
    __shared__ int32_t sum[2];
    const int tid = threadIdx.x;
    const int32_t avail = min(max(a.n_free[0], 0), a.free_cap);
    const int32_t t0 = int32_t(blockIdx.x) * a.rows_per_wg, t1 = min(t0 + a.rows_per_wg, a.T);
    int64_t rows = 0, pages = 0;   // before this pass
    int32_t used = 0, refused = 0;
    for (int32_t r0 = 0; r0 < a.R; r0 += kChunk) {
        const int n = min(kChunk, a.R - r0);
        int32_t q[kItems], need[kItems], k[kItems], o[kItems];
        bool wide[kItems];
        int64_t sq = 0, sn = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = tid * kItems + j;
            q[j] = i < n ? max(a.q_len[r0 + i], 0) : 0;
            k[j] = i < n ? max(a.kv_len[r0 + i], 0) : 0;
            o[j] = i < n ? max(a.owned[r0 + i], 0) : 0;
        }
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int64_t want = (int64_t(k[j]) + q[j] + kPage - 1) / kPage;
            wide[j] = want > a.P;
            need[j] = wide[j] ? 0 : max(0, int32_t(want) - o[j]);
            sq += q[j];
            sn += need[j];
        }
        int64_t eq = sq, en = sn, tq, tn;
        wg_scan(eq, en, tq, tn, part);
        eq += rows;
        en += pages;
        int32_t my_used = 0, my_ref = 0;
#pragma unroll
        for (int j = 0; j < kItems; ++j) {
            const int i = tid * kItems + j;
            const bool ok = !wide[j] && (need[j] == 0 || en + need[j] <= avail);
            if (i < n) {
                cu[i] = int32_t(eq);
                pre[i] = int32_t(min(en, int64_t(avail) + 1));
                kv[i] = k[j];
                own[i] = o[j];
                first[i] = ok ? avail - 1 - pre[i] : kRefused;
                if (ok) my_used += need[j]; else ++my_ref;
                if (blockIdx.x == 0) {
                    a.cu_q[r0 + i] = int32_t(eq);
                    a.kv_out[r0 + i] = ok ? k[j] + q[j] : k[j];
                    a.owned_out[r0 + i] = ok ? o[j] + need[j] : o[j];
                }
            }
            eq += q[j];
            en += need[j];
        }
        if (blockIdx.x == 0) {   // counts for the status words
            if (tid == 0) { sum[0] = 0; sum[1] = 0; }
            __syncthreads();
            if (my_used) atomicAdd(&sum[0], my_used);
            if (my_ref) atomicAdd(&sum[1], my_ref);
        }
        __syncthreads();
        if (blockIdx.x == 0) { used += sum[0]; refused += sum[1]; }
        // this workgroup's rows among the pass's requests
        for (int64_t row = max(int64_t(t0), rows) + tid; row < min(int64_t(t1), rows + tq); row += kThreads) {
            const int32_t t = int32_t(row);
            const int i = last_le(cu, n, t);
            const int32_t pos = kv[i] + (t - cu[i]), c = pos / kPage;
            int32_t slot = -1;
            if (first[i] != kRefused && pos >= 0 && c < a.P) {
                int32_t page;
                if (c < own[i]) {
                    page = a.table[int64_t(r0 + i) * a.ldt + c];
                } else {
                    const int32_t f = first[i] - (c - own[i]);
                    page = f >= 0 && f < avail ? a.free_pages[f] : -1;
                }
                if (page >= 0 && page < (INT32_MAX / kPage)) slot = page * kPage + pos % kPage;
            }
            a.slots[t] = slot;
            a.positions[t] = pos;
        }
        // its share of the pass's new pages (served requests come before any that asks past avail)
        const int64_t n_new = min(tn, avail - pages);
        for (int64_t e = int64_t(blockIdx.x) * kThreads + tid; e < n_new; e += int64_t(gridDim.x) * kThreads) {
            const int32_t at = int32_t(pages + e);
            const int i = last_le(pre, n, at);
            const int32_t j = at - pre[i], f = first[i] - j;
            const int64_t c = int64_t(own[i]) + j;
            if (first[i] != kRefused && f >= 0 && f < avail && c < a.P)
                a.table[int64_t(r0 + i) * a.ldt + c] = a.free_pages[f];
        }
        rows += tq;
        pages += tn;
        __syncthreads();   // the arrays are rewritten by the next pass
    }
    for (int64_t t = max(int64_t(t0), rows) + tid; t < t1; t += kThreads) {
        a.slots[t] = -1;
        a.positions[t] = 0;
    }
    if (blockIdx.x == 0 && tid == 0) {
        a.cu_q[a.R] = int32_t(rows);
        a.status[0] = avail - used;
        a.status[1] = refused;
    }
}

// One workgroup: a prefix sum of the released requests' pages gives each its
// place on the free list.
__global__ __launch_bounds__(kThreads) void kv_release_kernel(const uint8_t *which, int32_t R, int32_t *kv_len,
                                                              int32_t *owned, const int32_t *table, int32_t P,
                                                              int64_t ldt, int32_t *free_pages, int32_t free_cap,
                                                              int32_t *n_free) {
    __shared__ int64_t part[kThreads / 64][2];
    const int tid = threadIdx.x, lane = tid & 63;
    int32_t base = min(max(n_free[0], 0), free_cap);
    for (int32_t r0 = 0; r0 < R; r0 += kThreads) {
        const int32_t r = r0 + tid;
        const bool out = r < R && which[r] != 0;
        const int32_t n = out ? min(max(owned[r], 0), P) : 0;
        int64_t at = n, unused = 0, total, t2;
        wg_scan(at, unused, total, t2, part);
        at += base;
        if (out) { owned[r] = 0; kv_len[r] = 0; }
        // a wavefront writes one request's pages together
        for (uint64_t m = __ballot(n > 0); m; m &= m - 1) {
            const int l = __ffsll((unsigned long long)m) - 1;
            const int32_t cnt = __shfl(n, l), row = __shfl(r, l);
            const int64_t to = __shfl(at, l);
            for (int32_t i = lane; i < cnt; i += 64)
                if (to + i < free_cap) free_pages[to + i] = table[int64_t(row) * ldt + cnt - 1 - i];
        }
        base = int32_t(min(base + total, int64_t(free_cap)));
        __syncthreads();   // part is rewritten by the next pass; n_free was read by all before its write below
    }
    __syncthreads();
    if (tid == 0) n_free[0] = base;
}

}  // namespace
}  // namespace ht

using namespace ht;

extern "C" ht_status ht_kv_cache_bytes(int64_t n_pages, int32_t n_heads, int32_t head_dim, size_t *codes,
                                       size_t *scales) {
    if (!codes || !scales) return HT_EINVAL;
    ht_kv_cache c{reinterpret_cast<int8_t *>(256), reinterpret_cast<float *>(256), n_pages, n_heads, head_dim};
    const ht_status st = check_cache(&c);
    if (st != HT_OK) return st;
    *codes = size_t(n_pages) * size_t(n_heads) * 2u * size_t(kPage) * size_t(head_dim);
    *scales = size_t(n_pages) * size_t(n_heads) * 2u * sizeof(float);
    return HT_OK;
}

extern "C" ht_status ht_kv_plan(const int32_t *q_len, const int32_t *kv_len, const int32_t *owned, int64_t R,
                                int32_t *table, int64_t P, int64_t ldt, const int32_t *free_pages, int64_t free_cap,
                                const int32_t *n_free, int64_t T, int32_t *cu_q, int32_t *slots, int32_t *positions,
                                int32_t *kv_out, int32_t *owned_out, int32_t *status, ht_stream stream) {
    const void *in[] = {q_len, kv_len, owned, free_pages, n_free, table};
    const void *out[] = {cu_q, kv_out, owned_out, status, slots, positions};
    const int64_t lim = int64_t(1) << 30;
    if (R <= 0 || R > lim || T < 0 || T > lim || P <= 0 || P > (int64_t(1) << 24) || ldt < P || free_cap <= 0 ||
        free_cap > lim)
        return HT_ESHAPE;
    for (const void *p : in)
        if (!p) return HT_EINVAL;
    for (int i = 0; i < 6; ++i) {
        if (!out[i] && (i < 4 || T > 0)) return HT_EINVAL;   // no rows: slots and positions may be NULL
        for (const void *p : in)
            if (out[i] == p) return HT_EINVAL;
        for (int j = 0; j < i; ++j)
            if (out[i] && out[i] == out[j]) return HT_EINVAL;
        if (!al4(out[i]) || !al4(in[i])) return HT_EALIGN;
    }
    // 512 rows per workgroup: two rows a thread, and enough workgroups that
    // the rows' lookups overlap
    const int64_t wgs = T <= 512 ? 1 : T >= 512 * 512 ? 512 : (T + 511) / 512;
    PlanKv a{q_len, kv_len, owned, table, free_pages, n_free, cu_q, slots, positions, kv_out, owned_out, status,
             ldt, int32_t(R), int32_t(P), int32_t(T), int32_t(free_cap), int32_t((T + wgs - 1) / wgs)};
    kv_plan_kernel<<<dim3(uint32_t(wgs)), kThreads, 0, hipStream_t(stream)>>>(a);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

extern "C" ht_status ht_kv_release(const uint8_t *which, int64_t R, int32_t *kv_len, int32_t *owned,
                                   const int32_t *table, int64_t P, int64_t ldt, int32_t *free_pages,
                                   int64_t free_cap, int32_t *n_free, ht_stream stream) {
    const int64_t lim = int64_t(1) << 30;
    if (R <= 0 || R > lim || P <= 0 || P > (int64_t(1) << 24) || ldt < P || free_cap <= 0 || free_cap > lim)
        return HT_ESHAPE;
    if (!which || !kv_len || !owned || !table || !free_pages || !n_free) return HT_EINVAL;
    if (!al4(kv_len) || !al4(owned) || !al4(table) || !al4(free_pages) || !al4(n_free)) return HT_EALIGN;
    kv_release_kernel<<<1, kThreads, 0, hipStream_t(stream)>>>(which, int32_t(R), kv_len, owned, table, int32_t(P),
                                                               ldt, free_pages, int32_t(free_cap), n_free);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

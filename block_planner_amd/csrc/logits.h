// logits.h -- what the operators over rows of logits share: reading rows of any
// alignment, the statistics of a softmax in one pass, and the largest entries.
//
// A row's statistics are (mx, s, t): the largest entry, s = sum 2^d and
// t = sum d 2^d with d = (x - mx) c and c = log2(e) / temperature, all in fp32.
// The difference is taken before the product: it is exact near the maximum,
// and entries of any finite size, the type's lowest among them, give 0 or a
// finite d.  -Inf entries give 0 and join nothing; +Inf or NaN give a NaN s.
#pragma once
#include "rows.h"

namespace ht {

constexpr float kLn2 = 0.69314718055994531f, kLog2e = 1.44269504088896341f;
constexpr float kLowest = -3.402823466e+38f, kFar = -16384.0f;   // 2^kFar is 0
constexpr int64_t kMaxLogitRows = int64_t(1) << 22;

template <typename T>
struct LogitType;
template <>
struct LogitType<float> {
    static constexpr int kVec = 4;
    static __device__ __forceinline__ void unpack(u32x4 u, float *x) {
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = __uint_as_float(u[j]);
    }
    static __device__ __forceinline__ u32x4 pack(const float *x) {
        return u32x4{__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3])};
    }
    static __device__ __forceinline__ float get(const float *p) { return *p; }
    static __device__ __forceinline__ void put(float *p, float v) { *p = v; }
};
template <>
struct LogitType<uint16_t> {
    static constexpr int kVec = 8;
    static __device__ __forceinline__ void unpack(u32x4 u, float *x) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            x[2 * j] = bf_lo(u[j]);
            x[2 * j + 1] = bf_hi(u[j]);
        }
    }
    static __device__ __forceinline__ u32x4 pack(const float *x) {
        return u32x4{pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]), pack_bf16(x[6], x[7])};
    }
    static __device__ __forceinline__ float get(const uint16_t *p) { return __uint_as_float(uint32_t(*p) << 16); }
    static __device__ __forceinline__ void put(uint16_t *p, float v) { *p = f32_to_bf16_rne(v); }
};

// n elements from p on as `head` single ones, up to the next 16-byte boundary,
// `vecs` whole 16-byte pieces and a tail of single ones.
struct Span {
    int head, tail;
    int32_t vecs;
};
template <typename T>
__device__ __forceinline__ Span span_of(const T *p, int64_t n) {
    constexpr int kVec = LogitType<T>::kVec;
    Span s;
    s.head = int((16u - uint32_t(reinterpret_cast<uintptr_t>(p) & 15u)) & 15u) / int(sizeof(T));
    if (s.head > n) s.head = int(n);
    s.vecs = int32_t((n - s.head) / kVec);
    s.tail = int(n - s.head - int64_t(s.vecs) * kVec);
    return s;
}

__device__ __forceinline__ float exp2_fast(float d) { return __builtin_amdgcn_exp2f(d); }

struct RowStat {
    float mx, s, t;
};

__device__ __forceinline__ RowStat stat_none() { return RowStat{kLowest, 0.f, 0.f}; }

// Statistics of two parts as one.  fmaxf drops a NaN difference (both
// maxima +Inf): the sums are NaN by then.
__device__ __forceinline__ RowStat stat_join(RowStat a, RowStat b, float c) {
    const float m = fmaxf(a.mx, b.mx);
    const float da = fmaxf((a.mx - m) * c, kFar), db = fmaxf((b.mx - m) * c, kFar);
    const float fa = exp2_fast(da), fb = exp2_fast(db);
    return RowStat{m, fa * a.s + fb * b.s, fa * (a.t + da * a.s) + fb * (b.t + db * b.s)};
}

// N more entries of a lane.
template <int N, bool ENT>
__device__ __forceinline__ void stat_add(RowStat &r, const float *x, float top, float c) {
    const float m = fmaxf(r.mx, top);
    const float dm = fmaxf((r.mx - m) * c, kFar), f = exp2_fast(dm);
    float s = 0.f, t = 0.f;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        const float d = (x[j] - m) * c, e = exp2_fast(d);
        s += e;
        if constexpr (ENT) t += fmaxf(d, kFar) * e;
    }
    if constexpr (ENT) r.t = f * (r.t + dm * r.s) + t;
    r.s = f * r.s + s;
    r.mx = m;
}

__device__ __forceinline__ RowStat stat_wave(RowStat r, float c) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1)
        r = stat_join(r, RowStat{__shfl_xor(r.mx, d), __shfl_xor(r.s, d), __shfl_xor(r.t, d)}, c);
    return r;
}

// log2 of a sum s >= 1 (its largest entry adds 1): exact near 1, where the
// most likely entry's own log probability is all there is.
__device__ __forceinline__ float log2_sum(float s) { return log1pf(s - 1.0f) * kLog2e; }

// A row as the outputs see it.  kind: 0 ordinary, 1 nothing allowed (every
// entry -Inf), 2 holds NaN or +Inf.
struct RowOut {
    float mx, b, entropy;
    int kind;
};
__device__ __forceinline__ RowOut row_out(RowStat r) {
    RowOut o;
    o.kind = r.s == 0.f ? 1 : r.s > 0.f && r.s < __builtin_inff() ? 0 : 2;
    o.mx = r.mx;
    o.b = log2_sum(r.s);
    const float h = kLn2 * (o.b - r.t / r.s);
    o.entropy = h < 0.f ? 0.f : h;
    if (o.kind == 1) {
        o.mx = -__builtin_inff();
        o.b = o.entropy = 0.f;
    } else if (o.kind == 2) {
        o.mx = o.b = o.entropy = __builtin_nanf("");
    }
    return o;
}

// log probability (natural) of an entry.  In natural units throughout: the
// type's lowest value times log2(e) would be past its range.
__device__ __forceinline__ float logp_of(const RowOut &o, float x, float inv_t) {
    return o.kind == 0 ? (x - o.mx) * inv_t - o.b * kLn2 : o.kind == 1 ? -__builtin_inff() : __builtin_nanf("");
}

// ---------------------------------------------------------------------------
// The largest entries.  An entry is one 64-bit whole number: the float's bits in
// the order of the values, then the index's complement, so that larger means
// a larger value or, among equals, a lower index; 0 is none.
// ---------------------------------------------------------------------------
constexpr int kMaxTop = 64;   // a wavefront's list: one entry per lane, the largest in lane 0

__device__ __forceinline__ uint32_t order_key(float x) {
    const uint32_t u = __float_as_uint(x + 0.0f);             // -0 is 0
    return u ^ (uint32_t(int32_t(u) >> 31) | 0x80000000u);
}
__device__ __forceinline__ float key_value(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}
__device__ __forceinline__ uint64_t entry_of(float x, uint32_t i) { return (uint64_t(order_key(x)) << 32) | (0xFFFFFFFFu - i); }
__device__ __forceinline__ uint32_t entry_index(uint64_t e) { return 0xFFFFFFFFu - uint32_t(e); }

__device__ __forceinline__ uint64_t lane_xor(uint64_t v, int j) {
    return (uint64_t(uint32_t(__shfl_xor(int(v >> 32), j))) << 32) | uint32_t(__shfl_xor(int(v), j));
}

__device__ __forceinline__ uint64_t keep(uint64_t a, uint64_t b, bool larger) { return (a > b) == larger ? a : b; }

// One entry per lane in ascending order of lanes.
__device__ __forceinline__ uint64_t sort_up(uint64_t v, int lane) {
#pragma unroll
    for (int k = 2; k <= 64; k <<= 1)
#pragma unroll
        for (int j = k >> 1; j > 0; j >>= 1) v = keep(v, lane_xor(v, j), ((lane & j) == 0) != ((lane & k) == 0));
    return v;
}

// The 64 largest of a descending list and an ascending one, descending.
__device__ __forceinline__ uint64_t join_lists(uint64_t down, uint64_t up, int lane) {
    uint64_t v = down > up ? down : up;
#pragma unroll
    for (int j = 32; j > 0; j >>= 1) v = keep(v, lane_xor(v, j), (lane & j) == 0);
    return v;
}

// A wavefront's k largest so far.  Entries at least `thr` are collected in LDS
// and join the list 64 at a time, so that a sort and a merge serve many; a row
// in no order passes about k log(n / k) of them.  thr is the smallest value
// above the k-th of the list, whose entries all come before those still to be
// read: an equal one has a higher index and stays out.
struct TopList {
    uint64_t list;       // this lane's
    float thr;
    int pending;
    uint64_t *buf;       // [128] of the wavefront

    __device__ __forceinline__ void init(uint64_t *b) {
        list = 0;
        thr = -__builtin_inff();
        pending = 0;
        buf = b;
    }

    __device__ __forceinline__ void flush(int k, int lane) {
        asm volatile("" ::: "memory");                        // other lanes' stores come before these loads
        const uint64_t in = lane < pending ? buf[lane] : 0;
        const uint64_t rest = 64 + lane < pending ? buf[64 + lane] : 0;
        asm volatile("" ::: "memory");
        list = join_lists(list, sort_up(in, lane), lane);
        pending = pending > 64 ? pending - 64 : 0;
        if (lane < pending) buf[lane] = rest;
        const uint32_t kth = uint32_t(__shfl(int(list >> 32), k - 1));
        if (kth) thr = key_value(kth + 1);                    // the next float up (-0 for 0 above the negative ones)
    }

    // N entries of each lane, the j-th at index i0 + j; live: whether they exist.  top: their largest.
    template <int N>
    __device__ __forceinline__ void add(const float *x, float top, uint32_t i0, bool live, int k, int lane) {
        const uint64_t some = __ballot(live && top >= thr);
        if (some == 0) return;
        float t = thr;
        const bool crowded = __popcll(some) >= k;
        if (crowded) {
            // the k-th largest of the lanes' maxima, to 16 bits from below: at least k entries reach it
            const uint32_t key = live && top >= thr ? order_key(top) : 0;
            uint32_t p = 0;
#pragma unroll
            for (int bit = 31; bit >= 16; --bit) {
                const uint32_t q = p | (1u << bit);
                if (__popcll(__ballot(key >= q)) >= k) p = q;
            }
            const float raised = key_value(p);
            if (raised > t) t = raised;
        }
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const bool in = live && x[j] >= t;
            const uint64_t who = __ballot(in);
            if (who == 0) continue;
            const int at = pending + int(__builtin_amdgcn_mbcnt_hi(uint32_t(who >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(who), 0)));
            if (in) buf[at] = entry_of(x[j], i0 + uint32_t(j));
            pending += __popcll(who);
            if (pending >= 64) flush(k, lane);
        }
        if (crowded && pending >= k) flush(k, lane);
    }
};

// Host check of rows of logits.
inline ht_status check_logits(const void *p, int64_t ld, int64_t M, int64_t V, int32_t type) {
    if (!p) return HT_EINVAL;
    if (M > 1 && ld < V) return HT_ESHAPE;
    if (reinterpret_cast<uintptr_t>(p) % size_t(act_size(type))) return HT_EALIGN;
    return HT_OK;
}

// Temperatures whose inverse times log2(e) is a normal number.
inline ht_status check_logit_shape(int64_t M, int64_t V, int32_t type, float temperature) {
    if (M < 0 || M > kMaxLogitRows || V <= 0 || V >= (int64_t(1) << 31) - 64) return HT_ESHAPE;
    if (!act_size(type) || !(temperature >= 1e-30f) || !(temperature <= 1e30f)) return HT_EINVAL;
    return HT_OK;
}

}  // namespace ht

// logits.h -- what the operators over rows of logits share: reading rows of any
// alignment, the statistics of a softmax in one pass, and the largest entries.
//
// A row's statistics are (mx, s, t): the largest entry, s = sum 2^d and
// t = sum d 2^d with d = (x - mx) c and c = log2(e) / temperature, all in fp32.
// The difference is taken before the product: it is exact near the maximum,
// and entries of any finite size, the type's lowest among them, give 0 or a
// finite d.  -Inf entries give 0 and join nothing; +Inf or NaN give a NaN s.
// A thread's s is over all its entries; from the wavefront on one entry of the
// largest is left out of it (mx = -Inf where there is none), and the logarithm is
// log1p(s): of a nearly certain token the others' sum keeps its digits, which 1 + s
// has not.
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
    static __device__ __forceinline__ void put(uint16_t *p, float v) { *p = round_bf16(v); }
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

// The whole pieces of a row as a buffer: a piece takes one 32-bit offset, and
// those past the end read zeros and store nothing.  Its address is the same in
// every lane.
struct Pieces {
    __amdgpu_buffer_rsrc_t r;
    int32_t vecs;

    __device__ __forceinline__ Pieces(const void *p, int32_t n)
        : r(__builtin_amdgcn_make_buffer_rsrc(const_cast<void *>(p), 0, int(16u * uint32_t(n)), 0x00020000)), vecs(n) {}
    template <int AUX = 0>
    __device__ __forceinline__ u32x4 load(uint32_t byte) const {
        return __builtin_amdgcn_raw_buffer_load_b128(r, byte, 0, AUX);
    }
    template <int AUX = 0>
    __device__ __forceinline__ void store(uint32_t byte, u32x4 v) const {
        __builtin_amdgcn_raw_buffer_store_b128(v, r, byte, 0, AUX);
    }
};

// -Inf entries: what the pieces past a row's end stand for.
template <typename T>
__device__ __forceinline__ u32x4 no_entries() {
    return sizeof(T) == 4 ? u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}
                          : u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};
}

__device__ __forceinline__ float exp2_fast(float d) { return __builtin_amdgcn_exp2f(d); }

struct RowStat {
    float mx, s, t;
};

// A thread's without entries.
__device__ __forceinline__ RowStat stat_none() { return RowStat{kLowest, 0.f, 0.f}; }

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

// Largest over a wavefront, the same on all lanes.
__device__ __forceinline__ float wave_top(float v) {
    v = fmaxf(v, dpp_f32<kDppXor1>(v));
    v = fmaxf(v, dpp_f32<kDppXor2>(v));
    v = fmaxf(v, dpp_f32<kDppHalfMirror>(v));
    v = fmaxf(v, dpp_f32<kDppMirror>(v));
    v = fmaxf(v, row_xor16(v));
    return fmaxf(v, row_xor32(v));
}

// Statistics relative to a larger or equal maximum.
__device__ __forceinline__ RowStat stat_under(RowStat r, float m, float c) {
    const float d = fmaxf((r.mx - m) * c, kFar), f = exp2_fast(d);
    return RowStat{m, f * r.s, f * (r.t + d * r.s)};
}

// sum 2^d over the entries that thread `first` of NT has read (every NT-th piece and a
// `single` one, -Inf: none), one of the largest, m, left out; by a wavefront.
template <typename T, int NT>
__device__ __forceinline__ float tail_of(const Pieces &in, int32_t first, float single, float m, float c) {
    constexpr int kVec = LogitType<T>::kVec;
    const int32_t lane = threadIdx.x & 63;
    float s = 0.f, n = 0.f;
    const auto add = [&](float x) {
        s += x == m ? 0.f : exp2_fast((x - m) * c);
        n += x == m ? 1.f : 0.f;
    };
    for (int32_t i = first + NT * lane; i < in.vecs; i += NT * 64) {
        float x[kVec];
        LogitType<T>::unpack(in.load(16u * uint32_t(i)), x);
#pragma unroll
        for (int j = 0; j < kVec; ++j) add(x[j]);
    }
    if (lane == 0) add(single);
    return wave_sum(s) + (wave_sum(n) - 1.0f);
}

// Over a wavefront: the maximum first, then sums relative to it, one entry of the
// largest left out.  Its thread's own sum has been rounded with the 1 in it; where the
// others come to less than 2^-4 (else 2^-24 of 1 is at most 2^-20 of them) that
// thread's entries are read and added up again, a piece or a few by each lane.  In rows
// that are all that sure: the loss of 4096 x 32000 fp32 85.3 us (83.2 without), of
// 16384 x 4000 bf16 31.2 (28.0 in rows that are not), log probabilities of 4096 x 128000
// bf16 with 32 alternatives 205 (203).  Leaving the largest out entry by entry: an
// instruction or two per entry of every row.
template <typename T, int NT>
__device__ __forceinline__ RowStat stat_wave(RowStat r, float c, const Pieces &in, float single) {
    const float m = wave_top(r.mx);
    const uint64_t who = __ballot(r.mx == m && r.s != 0.f);
    if (who == 0) return RowStat{-__builtin_inff(), 0.f, 0.f};
    const int lane = threadIdx.x & 63, at = __builtin_ctzll(who);
    r = stat_under(r, m, c);
    const float others = wave_sum(lane == at ? 0.f : r.s), t = wave_sum(r.t);
    float own = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(r.s), at)) - 1.0f;
    if (__any(others + own < 0.0625f)) {
        single = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(single), at));
        own = tail_of<T, NT>(in, (threadIdx.x & ~63u) + at, single, m, c);
    }
    return RowStat{m, others + own, t};
}

// Results of wavefronts or of parts of rows, one in each of W = 16 or 64 lanes, as one.
template <int W>
__device__ __forceinline__ RowStat stat_meet(RowStat r, float c) {
    float m = r.mx;
    if constexpr (W == 64) {
        m = wave_top(m);
    } else {
        m = fmaxf(m, dpp_f32<kDppXor1>(m));
        m = fmaxf(m, dpp_f32<kDppXor2>(m));
        m = fmaxf(m, dpp_f32<kDppHalfMirror>(m));
        m = fmaxf(m, dpp_f32<kDppMirror>(m));
    }
    const int lane = threadIdx.x & (W - 1);
    const uint64_t who = __ballot(r.mx == m) >> (threadIdx.x & 63 & ~(W - 1));
    if (lane != __builtin_ctzll(who)) {              // the first of the largest stays left out
        const float all = r.mx > -__builtin_inff() ? 1.0f + r.s : 0.f;
        r = stat_under(RowStat{r.mx, all, r.t}, fmaxf(m, kLowest), c);
    }
    if constexpr (W == 64) return RowStat{m, wave_sum(r.s), wave_sum(r.t)};
    else return RowStat{m, group_sum<16>(r.s), group_sum<16>(r.t)};
}

// Over the NW <= 16 wavefronts' results in LDS, lane by lane of 16.
template <int NW>
__device__ __forceinline__ RowStat stat_group(const RowStat *stats, float c) {
    RowStat r{-__builtin_inff(), 0.f, 0.f};
    if (int(threadIdx.x & 15) < NW) r = stats[threadIdx.x & 15];
    return stat_meet<16>(r, c);
}

// log2(1 + x), x >= 0, to 8 units of 2^-24 however small x is: below 1/4 by
// log((1 + s) / (1 - s)) = 2 (s + s^3 / 3 + s^5 / 5 + ...) with s = x / (2 + x) <= 1/9.
__device__ __forceinline__ float log2_1p(float x) {
    const float s = x * __builtin_amdgcn_rcpf(2.0f + x), z = s * s;
    const float p = 1.0f + z * (1.0f / 3 + z * (1.0f / 5 + z * (1.0f / 7 + z * (1.0f / 9))));
    return x < 0.25f ? 2.0f * kLog2e * s * p : __builtin_amdgcn_logf(1.0f + x);
}

// 1 - 2^l, l <= 0, q = 2^l: from -1 on by the series of the exponential, which
// keeps its digits where q is nearly 1.
__device__ __forceinline__ float one_minus(float l, float q) {
    const float y = l * kLn2;
    float p = 1.0f;
#pragma unroll
    for (int i = 10; i >= 2; --i) p = 1.0f + y * (1.0f / i) * p;
    return l > -1.0f ? -y * p : 1.0f - q;
}

// A row as the outputs see it.  kind: 0 ordinary, 1 nothing allowed (every
// entry -Inf), 2 holds NaN or +Inf.
struct RowOut {
    float mx, b, entropy;
    int kind;
};
__device__ __forceinline__ RowOut row_out(RowStat r) {
    RowOut o;
    o.kind = !(r.s < __builtin_inff()) ? 2 : r.mx == -__builtin_inff() ? 1 : 0;
    o.mx = r.mx;
    o.b = log2_1p(r.s);
    const float h = kLn2 * (o.b - r.t / (1.0f + r.s));
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

// The value of lane ^ J.  Within 16 lanes by lane permutations of one or two
// moves, across them by the swaps of halves and of rows of 16.
template <int J>
__device__ __forceinline__ uint32_t lane_xor32(uint32_t v) {
    if constexpr (J == 1) return dpp_u32<kDppXor1>(v);
    else if constexpr (J == 2) return dpp_u32<kDppXor2>(v);
    else if constexpr (J == 4) return dpp_u32<0x1B>(dpp_u32<kDppHalfMirror>(v));   // ^ 7, then ^ 3
    else if constexpr (J == 8) return dpp_u32<0x128>(v);                             // rotated by 8 of 16
    else if constexpr (J == 16) {
        const auto r = __builtin_amdgcn_permlane16_swap(v, v, false, false);
        return threadIdx.x & 16 ? r[0] : r[1];
    } else {
        const auto r = __builtin_amdgcn_permlane32_swap(v, v, false, false);
        return threadIdx.x & 32 ? r[0] : r[1];
    }
}

template <int J>
__device__ __forceinline__ uint64_t lane_xor(uint64_t v) {
    return (uint64_t(lane_xor32<J>(uint32_t(v >> 32))) << 32) | lane_xor32<J>(uint32_t(v));
}

__device__ __forceinline__ uint64_t keep(uint64_t a, uint64_t b, bool larger) { return (a > b) == larger ? a : b; }

// One step of a merge within groups of 2 J lanes: K is the direction's bit.
template <int K, int J>
__device__ __forceinline__ uint64_t sort_steps(uint64_t v, int lane) {
    v = keep(v, lane_xor<J>(v), ((lane & J) == 0) != ((lane & K) == 0));
    if constexpr (J > 1) return sort_steps<K, J / 2>(v, lane);
    else return v;
}

// One entry per lane in ascending order of lanes.
__device__ __forceinline__ uint64_t sort_up(uint64_t v, int lane) {
    v = sort_steps<2, 1>(v, lane);
    v = sort_steps<4, 2>(v, lane);
    v = sort_steps<8, 4>(v, lane);
    v = sort_steps<16, 8>(v, lane);
    v = sort_steps<32, 16>(v, lane);
    return sort_steps<64, 32>(v, lane);
}

// The 64 largest of a descending list and an ascending one, descending: K = 0
// keeps the larger in the lower lane everywhere.
__device__ __forceinline__ uint64_t join_lists(uint64_t down, uint64_t up, int lane) {
    return sort_steps<128, 32>(down > up ? down : up, lane ^ 63);
}

// The k largest of what a workgroup of NW wavefronts reads.  Where a lane's entries
// reach `thr`, its two 16-byte pieces are put aside in LDS, which costs the pass over
// the row a vote and a few stores.  thr is never past the k-th largest (and at
// least the lowest finite value: entries of -Inf are not collected; the first of them
// fill a row that allows fewer than k, at the end).  It comes from the least, over
// the wavefronts, of the ceil(k / NW)-th largest of their lanes' maxima: k entries of the
// row reach that.  A wavefront's costs 24 votes (0.4 us) and no sort, so it is renewed
// after 1, 2, 4, 8 ... steps (every half as often again: the same times): a row of n
// entries in no order puts about k log2(n / 4096) pairs of pieces aside.  The wavefronts
// publish theirs without waiting: an older one is a lower bound, and what is put
// aside in vain changes nothing in the result.
// At the end what reaches the last bound, 1.5 to 2 k entries, goes into one array,
// and each entry's rank there is counted (1.3 us; 4 x 128000 with 20: 13.8 us a call,
// with a list per wavefront, sorted and merged, 14.9).  Places in that array depend on who comes first;
// ranks do not.  A wavefront that has put too much aside meanwhile moves 64 pairs into
// a list of its own, sorted; so does one at the end where the array is too small (rows
// of equal entries).  Rows in ascending order cost that all the time: 4096 x 128000
// bf16, k = 20, 1.5 ms.
template <typename T, int NW>
struct TopShared {
    static constexpr int kMost = NW > 4 ? 128 : 160, kCands = NW == 1 ? 64 : 256;
    struct Aside {
        u32x4 piece[2][kMost];
        int32_t first[kMost];    // the first one's number in the row; the second's is `apart` further
    };
    union {
        Aside aside[NW];
        uint64_t lists[NW * 64]; // once nothing is put aside any more
    };
    uint64_t cand[kCands], best[64];
    float bounds[NW];
    int rank[kCands], count;

    __device__ __forceinline__ void init() {
        if (threadIdx.x < NW) bounds[threadIdx.x] = -__builtin_inff();
        for (int i = threadIdx.x; i < kCands; i += 64 * NW) rank[i] = 0;
        if (threadIdx.x == 0) count = 0;
    }
};

template <typename T, int NW>
struct TopList {
    using Shared = TopShared<T, NW>;
    static constexpr int kVec = LogitType<T>::kVec, kFew = 8;
    uint64_t list, kth;  // this lane's entry; the k-th, 0: none yet
    float thr;           // never NaN
    float lane_top;      // the lane's largest entry, -Inf without one
    int pending, k, lane, wave;
    int part;            // ceil(k / NW)
    Shared *sh;          // the workgroup's, in LDS
    typename Shared::Aside *aside;

    __device__ __forceinline__ void init(Shared *s, int top) {
        list = kth = 0;
        thr = kLowest;
        lane_top = -__builtin_inff();
        pending = 0;
        k = top;
        lane = threadIdx.x & 63;
        wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
        part = (k + NW - 1) / NW;
        sh = s;
        aside = s->aside + wave;
    }

    // Publishes the wavefront's bound.
    __device__ __forceinline__ void raise() {
        // to 16 bits, two at a time, from below; -Inf's are those of no number
        const uint32_t key = order_key(lane_top);
        uint32_t p = 0;
#pragma unroll
        for (int bit = 30; bit >= 16; bit -= 2) {
            const uint32_t q1 = p | (1u << bit), q2 = p | (2u << bit), q3 = p | (3u << bit);
            const int n1 = __popcll(__ballot(key >= q1)), n2 = __popcll(__ballot(key >= q2)), n3 = __popcll(__ballot(key >= q3));
            p = n3 >= part ? q3 : n2 >= part ? q2 : n1 >= part ? q1 : p;
        }
        const float v = key_value(p);
        if (lane == 0 && v > -__builtin_inff())
            __hip_atomic_store(&sh->bounds[wave], v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }

    // The workgroup's bound, which thr takes over.
    __device__ __forceinline__ float refresh() {
        static_assert(NW <= 16 && (NW & (NW - 1)) == 0, "");
        float least = __hip_atomic_load(&sh->bounds[lane & (NW - 1)], __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
        if constexpr (NW > 1) least = fminf(least, dpp_f32<kDppXor1>(least));
        if constexpr (NW > 2) least = fminf(least, dpp_f32<kDppXor2>(least));
        if constexpr (NW > 4) least = fminf(least, dpp_f32<kDppHalfMirror>(least));
        if constexpr (NW > 8) least = fminf(least, dpp_f32<kDppMirror>(least));
        least = __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(least)));
        thr = fmaxf(thr, least);
        return least;
    }

    // The entries of the lanes in `who` join the list: few one by one, each moving
    // those below it one lane on, many by a sort and a merge.
    __device__ __forceinline__ void take(uint64_t e, uint64_t who) {
        if (__popcll(who) <= kFew) {
            for (; who; who &= who - 1) {
                const int from = __builtin_ctzll(who);
                const uint64_t v = (uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(e >> 32), from))) << 32) |
                                   uint32_t(__builtin_amdgcn_readlane(uint32_t(e), from));
                const int at = __popcll(__ballot(list > v));
                const uint64_t up = (uint64_t(dpp_u32<0x138>(uint32_t(list >> 32))) << 32) | dpp_u32<0x138>(uint32_t(list));
                list = lane < at ? list : lane == at ? v : up;
            }
        } else {
            list = join_lists(list, sort_up((who >> lane) & 1 ? e : 0, lane), lane);
        }
        kth = (uint64_t(uint32_t(__builtin_amdgcn_readlane(uint32_t(list >> 32), k - 1))) << 32) |
              uint32_t(__builtin_amdgcn_readlane(uint32_t(list), k - 1));
    }

    // Puts the lane's two pieces aside where their largest entry reaches thr.
    __device__ __forceinline__ void put(float top, u32x4 a, u32x4 b, int32_t first) {
        const bool in = top >= thr;
        const uint64_t who = __ballot(in);
        if (who == 0) return;
        const int at = pending + int(__builtin_amdgcn_mbcnt_hi(uint32_t(who >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(who), 0)));
        if (in) {
            aside->piece[0][at] = a;
            aside->piece[1][at] = b;
            aside->first[at] = first;
        }
        pending += __popcll(who);
    }

    // Up to 64 pairs put aside join the list; vecs: pieces of the row, i0: index of the first one's first entry.
    __device__ __forceinline__ void flush(int32_t apart, int32_t vecs, uint32_t i0) {
        asm volatile("" ::: "memory");                        // other lanes' stores come before these loads
        const bool mine = lane < pending;
        const u32x4 a = aside->piece[0][lane], b = aside->piece[1][lane];
        const int32_t first = mine ? aside->first[lane] : vecs;
        const int32_t left = pending - 64;
        for (int i = lane; i < left; i += 64) {
            aside->piece[0][i] = aside->piece[0][64 + i];
            aside->piece[1][i] = aside->piece[1][64 + i];
            aside->first[i] = aside->first[64 + i];
        }
        asm volatile("" ::: "memory");
        pending = left > 0 ? left : 0;
        float x[2 * kVec];
        uint32_t key[2 * kVec];
        LogitType<T>::unpack(a, x);
        LogitType<T>::unpack(b, x + kVec);
#pragma unroll
        for (int j = 0; j < 2 * kVec; ++j) key[j] = x[j] >= kLowest && first + j / kVec * apart < vecs ? order_key(x[j]) : 0;
        // each lane's largest in turn, while any belongs to the k
        for (;;) {
            uint32_t top = key[0];
#pragma unroll
            for (int j = 1; j < 2 * kVec; ++j) top = max(top, key[j]);
            int which = 0;
#pragma unroll
            for (int j = 2 * kVec - 1; j >= 0; --j) which = key[j] == top ? j : which;
            const uint32_t i = i0 + uint32_t(first + (which >= kVec ? apart : 0)) * kVec + uint32_t(which & (kVec - 1));
            const uint64_t e = top ? (uint64_t(top) << 32) | (0xFFFFFFFFu - i) : 0;
            const uint64_t who = __ballot(e > kth);
            if (who == 0) break;
            take(e, who);
#pragma unroll
            for (int j = 0; j < 2 * kVec; ++j) key[j] = j == which ? 0 : key[j];
        }
        if (kth) thr = fmaxf(thr, key_value(uint32_t(kth >> 32) + 1));   // the next float up (-0 for 0 above the negative ones)
    }

    // All that reach the last bound, of the whole workgroup, into sh->cand; between
    // two barriers.  Their number, sh->count, may be more than it holds.  thr, past the
    // k-th of the wavefront's list, is for pieces that are read after those in it: what
    // is still put aside may hold the k-th's value at a lower index, so it goes by the
    // larger of that value and the workgroup's bound, either included.
    __device__ __forceinline__ void gather(int32_t apart, int32_t vecs, uint32_t i0) {
        const float least = refresh();
        const float bound = fmaxf(least, kth ? key_value(uint32_t(kth >> 32)) : kLowest);
        bool old = lane < k && list != 0 && uint32_t(list >> 32) >= order_key(least);
        for (int from = 0; from == 0 || from < pending; from += 64) {
            const int i = from + lane;
            const u32x4 a = aside->piece[0][i], b = aside->piece[1][i];
            const int32_t first = i < pending ? aside->first[i] : vecs;
            float x[2 * kVec];
            LogitType<T>::unpack(a, x);
            LogitType<T>::unpack(b, x + kVec);
            if (first >= vecs) {
#pragma unroll
                for (int j = 0; j < kVec; ++j) x[j] = __builtin_nanf("");
            }
            if (first + apart >= vecs) {
#pragma unroll
                for (int j = kVec; j < 2 * kVec; ++j) x[j] = __builtin_nanf("");
            }
            uint32_t n = old ? 1 : 0;
#pragma unroll
            for (int j = 0; j < 2 * kVec; ++j) n += x[j] >= bound ? 1 : 0;
            // places: the lanes' counts bit by bit
            uint32_t at = 0, all = 0;
#pragma unroll
            for (int bit = 0; bit < 5; ++bit) {
                const uint64_t who = __ballot((n >> bit) & 1);
                at += uint32_t(__builtin_amdgcn_mbcnt_hi(uint32_t(who >> 32), __builtin_amdgcn_mbcnt_lo(uint32_t(who), 0))) << bit;
                all += uint32_t(__popcll(who)) << bit;
            }
            if (all == 0) continue;
            uint32_t base = 0;
            if (lane == 0) base = uint32_t(atomicAdd(&sh->count, int(all)));
            base = uint32_t(__builtin_amdgcn_readfirstlane(int(base)));
            if (base + all > uint32_t(Shared::kCands)) return;      // too many: the count says so
            at += base;
            if (old) sh->cand[at++] = list;
            old = false;
#pragma unroll
            for (int j = 0; j < 2 * kVec; ++j)
                if (x[j] >= bound)
                    sh->cand[at++] = entry_of(x[j], i0 + uint32_t(first + (j >= kVec ? apart : 0)) * kVec + uint32_t(j & (kVec - 1)));
        }
    }

    // The 64 largest candidates in order, in the first wavefront: each goes to the
    // place that the number of larger ones gives it, counted by as many threads per
    // candidate as there are.
    __device__ __forceinline__ void order() {
        constexpr int NT = 64 * NW;
        const int n = sh->count, t = threadIdx.x;
        int wide = 32;                               // candidates' places: a power of two
        while (wide < n) wide *= 2;
        const int c = t & (wide - 1), slice = t / wide, slices = NT / wide < 16 ? NT / wide : 16;
        if (c < n && slice < slices) {
            const uint64_t mine = sh->cand[c];
            int rank = 0;
#pragma unroll 4
            for (int i = slice; i < n; i += slices) rank += sh->cand[i] > mine ? 1 : 0;
            if (rank) atomicAdd(&sh->rank[c], rank);
        }
        __syncthreads();
        if (t < n && sh->rank[t] < 64) sh->best[sh->rank[t]] = sh->cand[t];
        __syncthreads();
        list = wave == 0 && lane < n ? sh->best[lane] : 0;
    }
};

// Statistics and largest entries of n entries from p on, whose first has index
// i0; every wavefront's result in its lanes.
template <typename T, int NT, bool ENT, bool TOP>
__device__ __forceinline__ RowStat scan_row(const T *p, int64_t n, uint32_t i0, float c, TopList<T, NT / 64> &list) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec, U = 16 / kVec;     // 16 entries per thread and step
    const Span sp = span_of(p, n);
    const int32_t t = threadIdx.x;
    RowStat r = stat_none();
    const Pieces in(p + sp.head, sp.vecs);
    u32x4 next[U];
    const auto load = [&](int32_t at) {
#pragma unroll
        for (int u = 0; u < U; ++u) next[u] = in.load<2>(16u * uint32_t(at + u * NT + t));   // not kept in the caches
    };
    load(0);
    int step = 0, renew = 1;                         // bounds are published after steps 1, 2, 4, 8, ...
    for (int32_t at = 0; at < sp.vecs; at += U * NT) {
        u32x4 cur[U];
        float x[U * kVec], top[U / 2];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            cur[u] = at + (u + 1) * NT <= sp.vecs || at + u * NT + t < sp.vecs ? next[u] : no_entries<T>();
            L::unpack(cur[u], x + u * kVec);
        }
        load(at + U * NT);
#pragma unroll
        for (int h = 0; h < U / 2; ++h) {
            top[h] = x[2 * h * kVec];
#pragma unroll
            for (int j = 1; j < 2 * kVec; ++j) top[h] = fmaxf(top[h], x[2 * h * kVec + j]);
        }
        const float most = U > 2 ? fmaxf(top[0], top[U / 2 - 1]) : top[0];
        stat_add<U * kVec, ENT>(r, x, most, c);
        if constexpr (TOP) {
            list.lane_top = fmaxf(list.lane_top, most);
            if (++step == renew && (step == 1 || at + U * NT < sp.vecs)) {   // the last bound comes after the row
                list.raise();
                if (step == 1) __syncthreads();      // no wavefront collects without a bound
                list.refresh();
                renew = 2 * step;
            }
#pragma unroll
            for (int h = 0; h < U / 2; ++h) {
                list.put(top[h], cur[2 * h], cur[2 * h + 1], at + 2 * h * NT + t);
                if (list.pending > TopShared<T, NT / 64>::kMost - 64) list.flush(NT, sp.vecs, i0 + uint32_t(sp.head));
            }
        }
    }
    float single = -__builtin_inff();
    if (t < 64 && sp.head + sp.tail) {               // the single ones before and after, by the first wavefront
        const bool live = t < sp.head + sp.tail;
        const int64_t i = t < sp.head ? int64_t(t) : n - sp.tail + (t - sp.head);
        if (live) single = L::get(p + i);
        stat_add<1, ENT>(r, &single, single, c);
        if constexpr (TOP) list.take(entry_of(single, i0 + uint32_t(i)), __ballot(live && single >= kLowest));
    }
    return stat_wave<T, NT>(r, c, in, single);
}

// Host check of rows of logits.
inline ht_status check_logits(const void *p, int64_t ld, int64_t M, int64_t V, int32_t type) {
    if (!p) return HT_EINVAL;
    if (M > 1 && ld < V) return HT_ESHAPE;
    if (reinterpret_cast<uintptr_t>(p) % size_t(act_size(type))) return HT_EALIGN;
    return HT_OK;
}

// Temperatures whose inverse times log2(e) is a normal number.
inline ht_status check_logit_shape(int64_t M, int64_t V, int32_t type, float temperature) {
    if (M < 0 || M > kMaxLogitRows || V <= 0 || V > (int64_t(1) << 29)) return HT_ESHAPE;   // a row's bytes as 32-bit offsets
    if (!act_size(type) || !(temperature >= 1e-30f) || !(temperature <= 1e30f)) return HT_EINVAL;
    return HT_OK;
}

}  // namespace ht

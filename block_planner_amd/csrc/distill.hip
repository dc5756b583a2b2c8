// distill.hip -- the loss of a student's logits against a teacher's top logits,
// the gradients of logits, and both in one pass.
//
//   p = softmax over a row's kept entries of t / temperature,
//   q = softmax over the vocabulary of x / temperature,
//   loss = sum_j p_j (log p_j - log q[id_j]);
//   d loss / d x_v = 1 / temperature (q_v - sum_{j: id_j = v} p_j).
//
// Every gradient here is  scale sum_{j: id_j = v} g_j + q_v (f + e log2 q_v)  with
// few g_j: of log probabilities of given tokens, f = -scale (sum g + h H) and
// e = -scale h log 2 with h the entropy's gradient; of distillation, g_j = p_j,
// f = -scale and e = 0.  The dense part is written for every entry, then the few given
// ones are written again, whole.
//
// Bound by HBM: logits once and the gradient once.  The step holds a row in the
// registers of a workgroup between its sum and its gradient, up to 20 pieces of
// 16 bytes per thread, and reads what lies behind them a second time, which the
// Infinity Cache serves: the rows in work are fewer than it holds.
// Measured with 20 entries per row, 2 bytes moved per byte of logits:
//   4096 x 32000 fp32: 180 us, 5.8 TB/s;  4096 x 128000 bf16: 390 us, 5.4 TB/s;
//   512 x 32000 fp32: 28 us;  two rows on a compute unit at a time and the next
//   row's loads behind the stores of this one's were slower (190 and 214 against
//   180 us, 434 and 462 against 390): one workgroup's phases are covered by the others'.
#include <type_traits>

#include "logits.h"

namespace ht {

namespace {

constexpr int kMaxEntries = 1024;   // teacher's entries or given tokens of a row

struct GradArgs {
    const void *x;
    void *dx;
    int64_t ld, ldd, V;
    float c, inv_t;
    // distillation
    const int32_t *ids;
    const float *teacher, *weight;   // weight: per row, or null (1)
    float *loss, *stats;
    int32_t k;
    // log probabilities
    const float *g, *g_entropy, *row_stats, *entropy;
    int64_t part;                    // columns per workgroup
    int32_t S, same;                 // same: dx's rows share x's alignment
};

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------
// The dense part's coefficients of a row: dx_v = f q_v, with the entropy's
// gradient dx_v = (f + e log2 q_v) q_v.
struct Dense {
    float mx, b, c, f, e;
    float scale, own;    // of the given entries: f = own - scale sum g
    bool zero;           // the row's gradient is zero whatever its logits are
};

template <bool ENT>
__device__ __forceinline__ float dense_of(const Dense &d, float x) {
    const float l = (x - d.mx) * d.c - d.b, q = exp2_fast(l);
    if constexpr (ENT) return q * (d.f + d.e * fmaxf(l, kFar));
    else return q * d.f;
}

template <typename T, bool ENT>
__device__ __forceinline__ u32x4 dense_piece(const Dense &d, u32x4 u) {
    using L = LogitType<T>;
    float x[L::kVec];
    L::unpack(u, x);
#pragma unroll
    for (int j = 0; j < L::kVec; ++j) x[j] = dense_of<ENT>(d, x[j]);
    return L::pack(x);
}

// A piece entry by entry, where dx's rows lie otherwise than x's.
template <typename T>
__device__ __forceinline__ void put_piece(T *y, u32x4 u) {
    using L = LogitType<T>;
    float x[L::kVec];
    L::unpack(u, x);
#pragma unroll
    for (int j = 0; j < L::kVec; ++j) L::put(y + j, x[j]);
}

// Entry j's place written whole: the dense part and every g of that place, in
// order.  The first entry of a place writes it: two threads' equal sums may still be
// rounded otherwise, by where the compiler fuses a product in each wavefront's code.
// scale (sum g at the place) - q scale (sum of all g) is taken as
// scale (sum at the place (1 - q) - q sum of the others): with a nearly certain token
// both terms are small and keep their digits.
template <typename T, bool ENT>
__device__ __forceinline__ void put_given(T *dx, const Dense &d, float x, int j, const int32_t *id, const float *g, int k) {
    const int32_t v = id[j];
    float sum = 0.f, rest = 0.f;
    bool first = true;
#pragma unroll 8
    for (int i = 0; i < k; ++i) {
        const int32_t w = id[i];
        const float gi = g[i];                       // read in any case: 64 entries 2.3 us less than under the condition
        sum += w == v ? gi : 0.f;
        rest += w == v ? 0.f : gi;
        first = first && (w != v || i >= j);
    }
    if (!first) return;
    const float l = (x - d.mx) * d.c - d.b, q = exp2_fast(l);
    float y = d.scale * (sum * one_minus(l, q) - q * rest);
    if constexpr (ENT) y += q * (d.own + d.e * fmaxf(l, kFar));
    LogitType<T>::put(dx + v, y);
}

// The teacher's distribution of a row by one wavefront: ids (-1: not kept), p, log2 p
// and the student's logits of its k entries (those in [lo, hi)) into LDS;
// returns whether any has weight.
template <typename T>
__device__ __forceinline__ bool teacher_wave(const int32_t *ids, const float *t, const T *row, int64_t lo, int64_t hi, int k,
                                             int64_t V, float c, int32_t *id, float *p, float *logs, float *given) {
    const int lane = threadIdx.x & 63;
    float most = -__builtin_inff();
    int at = -1;                                     // the lane's first of its largest
    for (int j = lane; j < k; j += 64) {
        const int32_t v = ids[j];
        const bool in = v >= 0 && v < V;
        const float z = in ? t[j] : -__builtin_inff();
        id[j] = in ? v : -1;
        given[j] = v >= lo && v < hi ? LogitType<T>::get(row + v) : 0.f;
        logs[j] = z;
        at = z > most ? j : at;
        most = fmaxf(most, z);
    }
    const float top = fmaxf(wave_top(most), kLowest);
    const uint64_t who = __ballot(at >= 0 && most == top);
    if (who == 0 || lane != __builtin_ctzll(who)) at = -1;
    float tail = 0.f;                                // as the student's: one entry of the largest left out
    for (int j = lane; j < k; j += 64) {
        const float d = (logs[j] - top) * c, e = exp2_fast(d);
        logs[j] = d;
        p[j] = e;
        tail += j == at ? 0.f : e;
    }
    tail = wave_sum(tail);
    const bool any = who != 0 || tail != 0.f;        // NaN too
    const float inv = 1.0f / (1.0f + tail), b = log2_1p(tail);
    for (int j = lane; j < k; j += 64) {
        p[j] = any ? p[j] * inv : 0.f;
        logs[j] -= b;
    }
    return any;
}

// A row's loss, by one wavefront after the statistics and the teacher's.
__device__ __forceinline__ void put_loss(const GradArgs &a, int64_t m, const RowOut &o, bool any, const int32_t *id,
                                         const float *p, const float *logs, const float *given) {
    const int lane = threadIdx.x & 63;
    float loss = 0.f;
    for (int j = lane; j < a.k; j += 64)
        // an entry without weight adds nothing, whatever the student says of it
        if (id[j] >= 0 && p[j] != 0.f) loss += p[j] * (logs[j] * kLn2 - logp_of(o, given[j], a.inv_t));
    loss = wave_sum(loss);
    if (lane == 0) {
        a.loss[m] = any ? loss : 0.f;
        if (a.stats) {
            a.stats[2 * m] = o.mx;
            a.stats[2 * m + 1] = o.b;
        }
    }
}

// Loss alone: the logits are read once, 2048 x 32000 fp32 in 44 us, 6.0 TB/s.  A
// workgroup of 1024 threads for each of few long rows: 11 us for one of 128000,
// 256 threads 15; of 64 for each of many short ones: 16384 x 1000 fp32 20 us (256
// threads 37), 16384 x 4000 bf16 32 (39), but 2000 x 12001 fp32 19.3 (18.8).
template <typename T, int NT>
__global__ __launch_bounds__(NT, 8) void distill_loss_kernel(GradArgs a) {
    extern __shared__ float lds[];                   // ids, p, log p, logits of the ids
    __shared__ RowStat stats[NT / 64];
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *p = lds + a.k, *logs = lds + 2 * a.k, *given = lds + 3 * a.k;
    const int64_t m = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    TopList<T, NT / 64> none;
    const RowStat r = scan_row<T, NT, false, false>(row, a.V, 0, a.c, none);
    if (lane == 0) stats[wave] = r;
    bool any = false;
    if (wave == 0) any = teacher_wave<T>(a.ids + m * a.k, a.teacher + m * a.k, row, 0, a.V, a.k, a.V, a.c, id, p, logs, given);
    __syncthreads();
    if (wave == 0) put_loss(a, m, row_out(stat_group<NT / 64>(stats, a.c)), any, id, p, logs, given);
}

// Loss and gradient of a row held in NV pieces per thread; FAR: there are more,
// read twice.  The first wavefront deals with the teacher while the others are at
// their sums.  SAME: dx's rows lie as x's do within 16 bytes, so its pieces are
// whole too.  ONCE: a gradient of more than the 256 MB Infinity Cache is neither
// read nor written with a view to the caches (524 MB: 196 -> 180 us); a smaller
// one stays for who reads it next (65 MB: 45 us with a sum over it, 56 with the
// hints).
template <typename T, int NT, int NV, bool SAME, bool ONCE, bool FAR>
__global__ __launch_bounds__(NT, NV == 4 ? 6 : 4) void distill_step_kernel(GradArgs a) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec, NW = NT / 64, kGroup = 16 / kVec < NV ? 16 / kVec : NV;
    extern __shared__ float lds[];                   // ids, p, log p, logits of the ids
    __shared__ RowStat stats[NW];
    __shared__ int some;
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *p = lds + a.k, *logs = lds + 2 * a.k, *given = lds + 3 * a.k;
    const int32_t t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const int64_t m = blockIdx.x;
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    T *dx = static_cast<T *>(a.dx) + m * a.ldd;
    const Span sp = span_of(row, a.V);
    const float w = a.weight ? a.weight[m] : 1.0f;
    // the single entries before and after the whole pieces: at most one per thread
    const bool single = t < sp.head + sp.tail;
    const int64_t at1 = t < sp.head ? int64_t(t) : a.V - sp.tail + (t - sp.head);
    Dense d{};
    d.zero = true;
    float x1 = 0.f;
    u32x4 held[NV];
    const Pieces in(row + sp.head, sp.vecs);
    if (w != 0.f) {                                  // one value per row: every thread takes the same way
#pragma unroll
        for (int i = 0; i < NV; ++i) held[i] = in.load<ONCE ? 2 : 0>(16u * uint32_t(t + i * NT));
        RowStat r = stat_none();
        if (wave == 0) {
            const bool any = teacher_wave<T>(a.ids + m * a.k, a.teacher + m * a.k, row, 0, a.V, a.k, a.V, a.c, id, p, logs, given);
            if (lane == 0) some = any;
        }
        if (single) {
            x1 = L::get(row + at1);
            stat_add<1, false>(r, &x1, x1, a.c);
        }
#pragma unroll
        for (int i = 0; i < NV; i += kGroup) {
            constexpr int N = kGroup * kVec;
            float x[N];
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                u32x4 u = held[i + g];
                if ((i + g + 1) * NT > sp.vecs && t + (i + g) * NT >= sp.vecs) u = no_entries<T>();
                L::unpack(u, x + g * kVec);
            }
            float most = x[0];
#pragma unroll
            for (int j = 1; j < N; ++j) most = fmaxf(most, x[j]);
            stat_add<N, false>(r, x, most, a.c);
            __builtin_amdgcn_sched_barrier(0);       // group by group: several at once spill
        }
        if constexpr (FAR) {
            for (int32_t at = NV * NT; at < sp.vecs; at += kGroup * NT) {
                float x[kGroup * kVec];
                u32x4 u[kGroup];
#pragma unroll
                for (int g = 0; g < kGroup; ++g) u[g] = in.load(16u * uint32_t(at + t + g * NT));
#pragma unroll
                for (int g = 0; g < kGroup; ++g) L::unpack(at + t + g * NT < sp.vecs ? u[g] : no_entries<T>(), x + g * kVec);
                float most = x[0];
#pragma unroll
                for (int j = 1; j < kGroup * kVec; ++j) most = fmaxf(most, x[j]);
                stat_add<kGroup * kVec, false>(r, x, most, a.c);
            }
        }
        r = stat_wave<T, NT>(r, a.c, in, single ? x1 : -__builtin_inff());
        if (lane == 0) stats[wave] = r;
        __syncthreads();
        const RowOut o = row_out(stat_group<NW>(stats, a.c));
        const bool any = some != 0;
        if (wave == 0) put_loss(a, m, o, any, id, p, logs, given);
        d.mx = o.mx;
        d.b = o.b;
        d.c = a.c;
        d.f = w * a.inv_t;
        d.scale = -d.f;
        d.zero = !any || o.kind == 1;
    } else {
        if (t == 0) {
            a.loss[m] = 0.f;
            if (a.stats) a.stats[2 * m] = a.stats[2 * m + 1] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) held[i] = u32x4{0, 0, 0, 0};
    }
    // the row's logits are in registers or read by now: dx may be the logits
    if (single) L::put(dx + at1, d.zero ? 0.f : dense_of<false>(d, x1));
    const Pieces out(dx + sp.head, sp.vecs);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
        u32x4 u = dense_piece<T, false>(d, held[i]);
        if (d.zero) u = u32x4{0, 0, 0, 0};
        if constexpr (SAME) {
            out.store<ONCE ? 2 : 0>(16u * uint32_t(t + i * NT), u);
        } else {
            if (t + i * NT < sp.vecs) put_piece<T>(dx + sp.head + (t + i * NT) * kVec, u);
        }
        __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (FAR) {
        for (int32_t at = NV * NT; at < sp.vecs; at += kGroup * NT) {
            u32x4 u[kGroup];
#pragma unroll
            for (int g = 0; g < kGroup; ++g) u[g] = d.zero ? u32x4{0, 0, 0, 0} : in.load(16u * uint32_t(at + t + g * NT));
#pragma unroll
            for (int g = 0; g < kGroup; ++g) {
                if (!d.zero) u[g] = dense_piece<T, false>(d, u[g]);
                if constexpr (SAME) {
                    out.store<ONCE ? 2 : 0>(16u * uint32_t(at + t + g * NT), u[g]);
                } else {
                    if (at + t + g * NT < sp.vecs) put_piece<T>(dx + sp.head + int64_t(at + t + g * NT) * kVec, u[g]);
                }
            }
        }
    }
    if (d.zero) return;
    __syncthreads();                                 // the given entries after the dense ones
    for (int j = t; j < a.k; j += NT)
        if (id[j] >= 0) put_given<T, false>(dx, d, given[j], j, id, p, a.k);
}

// Gradient from kept statistics: of the distillation's loss (DIST: weight is the
// loss's gradient) or of log probabilities and entropy.  A workgroup takes a
// part of a row of up to NV pieces per thread, all loaded before it looks at the
// given entries.  2000 x 50001 fp32: 143 us, 5.6 TB/s.
template <typename T, int NT, int NV, bool DIST, bool SAME, bool ONCE>
__global__ __launch_bounds__(NT) void logits_grad_kernel(GradArgs a) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec;
    extern __shared__ float lds[];                   // ids, g, logits of the ids, (DIST) log p
    __shared__ int some;
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *g = lds + a.k, *given = lds + 2 * a.k;
    const int64_t m = int64_t(blockIdx.x) / a.S, c0 = (int64_t(blockIdx.x) - m * a.S) * a.part;
    const int64_t n = min(a.V - c0, a.part);
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    T *dx = static_cast<T *>(a.dx) + m * a.ldd;
    const int32_t t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
    const Span sp = span_of(row + c0, n);
    const bool single = t < sp.head + sp.tail;
    const int64_t at1 = c0 + (t < sp.head ? int64_t(t) : n - sp.tail + (t - sp.head));
    const Pieces in(row + c0 + sp.head, sp.vecs), out(dx + c0 + sp.head, sp.vecs);
    Dense d{};
    d.mx = a.row_stats[2 * m];
    d.b = a.row_stats[2 * m + 1];
    d.c = a.c;
    const float w = DIST ? a.weight[m] : 0.f, e = !DIST && a.g_entropy ? a.g_entropy[m] : 0.f;
    bool any = DIST ? w != 0.f : e != 0.f;
    if constexpr (!DIST)
        for (int j = 0; j < a.k && !any; ++j) {
            const int32_t v = a.ids[m * a.k + j];
            any = v >= 0 && v < a.V && a.g[m * a.k + j] != 0.f;
        }
    d.zero = !any || d.mx == -__builtin_inff();      // no gradient, or a row that allows nothing: not read
    u32x4 held[NV];
    float x1 = 0.f;
    if (!d.zero) {
#pragma unroll
        for (int i = 0; i < NV; ++i) held[i] = in.load<ONCE ? 2 : 0>(16u * uint32_t(t + i * NT));
        if (single) x1 = L::get(row + at1);
        if constexpr (DIST) {
            if (wave == 0) {
                const bool kept = teacher_wave<T>(a.ids + m * a.k, a.teacher + m * a.k, row, c0, c0 + n, a.k, a.V, a.c, id, g,
                                                  lds + 3 * a.k, given);
                if (lane == 0) some = kept;
            }
            d.f = w * a.inv_t;
            d.scale = -d.f;
        } else {
            float sum = 0.f;                         // every wavefront its own, in the same order
            for (int j = lane; j < a.k; j += 64) {
                const int32_t v = a.ids[m * a.k + j];
                const float gj = v >= 0 && v < a.V ? a.g[m * a.k + j] : 0.f;
                sum += gj;
                if (wave == 0) {
                    id[j] = v >= 0 && v < a.V ? v : -1;
                    g[j] = gj;
                    given[j] = v >= c0 && v < c0 + n ? L::get(row + v) : 0.f;
                }
            }
            sum = wave_sum(sum);
            d.own = -a.inv_t * (e != 0.f ? e * a.entropy[m] : 0.f);
            d.f = d.own - a.inv_t * sum;
            d.e = -a.inv_t * e * kLn2;
            d.scale = a.inv_t;
        }
    } else {
#pragma unroll
        for (int i = 0; i < NV; ++i) held[i] = u32x4{0, 0, 0, 0};
    }
    __syncthreads();                                 // the given logits are read: dx may be the logits
    if (DIST && !d.zero) d.zero = some == 0;
    const auto put = [&](auto entropy) {
        constexpr bool kEnt = decltype(entropy)::value;
        if (single) L::put(dx + at1, d.zero ? 0.f : dense_of<kEnt>(d, x1));
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            u32x4 u = dense_piece<T, kEnt>(d, held[i]);
            if (d.zero) u = u32x4{0, 0, 0, 0};
            if constexpr (SAME) {
                out.store<ONCE ? 2 : 0>(16u * uint32_t(t + i * NT), u);
            } else {
                if (t + i * NT < sp.vecs) put_piece<T>(dx + c0 + sp.head + (t + i * NT) * kVec, u);
            }
            __builtin_amdgcn_sched_barrier(0);       // piece by piece: several at once spill
        }
        if (d.zero) return;
        __syncthreads();                             // the given entries after the dense ones
        for (int j = t; j < a.k; j += NT)
            if (id[j] >= c0 && id[j] < c0 + n) put_given<T, kEnt>(dx, d, given[j], j, id, g, a.k);
    };
    if (!DIST && e != 0.f) put(std::true_type{});
    else put(std::false_type{});
}

// dx's rows lie as x's do within 16 bytes: whole pieces of one are whole pieces of the other.
bool same_alignment(const void *x, int64_t ld, const void *dx, int64_t ldd, int64_t M, int size) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == (reinterpret_cast<uintptr_t>(dx) & 15) &&
           (M <= 1 || ((ld - ldd) * size) % 16 == 0);
}

bool once(const GradArgs &a, int64_t M, int size) { return M * a.V * size > (int64_t(256) << 20); }

template <typename T, int NT>
void loss_kernel(const GradArgs &a, int64_t M, hipStream_t s) {
    distill_loss_kernel<T, NT><<<uint32_t(M), NT, size_t(4) * size_t(a.k) * 4, s>>>(a);
}

template <typename T, int NT, int NV, bool FAR = false>
void step_kernel(const GradArgs &a, int64_t M, hipStream_t s) {
    const uint32_t grid = uint32_t(M);
    const size_t lds = size_t(4) * size_t(a.k) * 4;
    if (!a.same) distill_step_kernel<T, NT, NV, false, false, FAR><<<grid, NT, lds, s>>>(a);
    else if (once(a, M, int(sizeof(T)))) distill_step_kernel<T, NT, NV, true, true, FAR><<<grid, NT, lds, s>>>(a);
    else distill_step_kernel<T, NT, NV, true, false, FAR><<<grid, NT, lds, s>>>(a);
}

// Short rows by a wavefront where there are many: with 8 entries, 16384 x 1000 fp32 28
// us (256 threads 39), bf16 28 (44), 16384 x 4000 bf16 52 (79), but in 16 pieces per
// thread 108 against 103 for 16384 x 4000 fp32, and 5.4 against 4.9 for 33 x 1003 bf16.
template <typename T>
ht_status launch_step(const GradArgs &a, int64_t M, hipStream_t s) {
    const int64_t pieces = a.V / LogitType<T>::kVec;   // at most: the head takes some
    const bool many = M > 1024;
    if (pieces <= 64) step_kernel<T, 64, 1>(a, M, s);
    else if (many && pieces <= 256) step_kernel<T, 64, 4>(a, M, s);
    else if (many && pieces <= 512) step_kernel<T, 64, 8>(a, M, s);
    else if (pieces <= 256) step_kernel<T, 256, 1>(a, M, s);
    else if (pieces <= 1024) step_kernel<T, 256, 4>(a, M, s);
    else if (pieces <= 4096) step_kernel<T, 1024, 4>(a, M, s);
    else if (pieces <= 8192) step_kernel<T, 1024, 8>(a, M, s);
    else if (pieces <= 16384) step_kernel<T, 1024, 16>(a, M, s);
    else if (pieces <= 20480) step_kernel<T, 1024, 20>(a, M, s);
    else step_kernel<T, 1024, 20, true>(a, M, s);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

template <typename T, int NV, bool DIST>
void grad_kernel(const GradArgs &a, int64_t M, hipStream_t s) {
    const uint32_t grid = uint32_t(M * a.S);
    const size_t lds = size_t(4) * size_t(a.k) * 4;
    if (!a.same) logits_grad_kernel<T, 256, NV, DIST, false, false><<<grid, 256, lds, s>>>(a);
    else if (once(a, M, int(sizeof(T)))) logits_grad_kernel<T, 256, NV, DIST, true, true><<<grid, 256, lds, s>>>(a);
    else logits_grad_kernel<T, 256, NV, DIST, true, false><<<grid, 256, lds, s>>>(a);
}

// dx times *g, unless that is 1.
template <typename T>
__global__ __launch_bounds__(256) void scale_kernel(T *dx, int64_t ld, int64_t V, int32_t S, const float *g) {
    using L = LogitType<T>;
    const float f = *g;
    if (f == 1.0f) return;
    const int64_t m = int64_t(blockIdx.x) / S, part = (V + S - 1) / S, c0 = (int64_t(blockIdx.x) - m * S) * part;
    const int64_t n = min(V - c0, part);
    if (n <= 0) return;
    T *p = dx + m * ld + c0;
    const Span sp = span_of(p, n);
    const int32_t t = threadIdx.x;
    if (t < sp.head + sp.tail) {
        const int64_t i = t < sp.head ? int64_t(t) : n - sp.tail + (t - sp.head);
        L::put(p + i, L::get(p + i) * f);
    }
    u32x4 *v = reinterpret_cast<u32x4 *>(p + sp.head);
    for (int32_t i = t; i < sp.vecs; i += 256) {
        float x[L::kVec];
        L::unpack(v[i], x);
#pragma unroll
        for (int j = 0; j < L::kVec; ++j) x[j] *= f;
        v[i] = L::pack(x);
    }
}

// Equal parts of a row of at most 16 pieces per thread, or of 4 where those
// give too few workgroups to fill the card.
template <typename T, bool DIST>
ht_status launch_grad(GradArgs &a, int64_t M, hipStream_t s) {
    const int64_t piece = LogitType<T>::kVec, pieces = (a.V + piece - 1) / piece;
    int nv = 16;
    if (M * ((pieces + 4095) / 4096) < 1024 || pieces <= 1024) nv = 4;
    const int64_t S = (pieces + 256 * nv - 1) / (256 * nv);
    if (M * S >= (int64_t(1) << 24)) return HT_ESHAPE;    // the launch's limit on threads
    a.part = ((pieces + S - 1) / S) * piece;
    a.S = int32_t((a.V + a.part - 1) / a.part);
    if (nv == 16) grad_kernel<T, 16, DIST>(a, M, s);
    else grad_kernel<T, 4, DIST>(a, M, s);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

}  // namespace
}  // namespace ht

using namespace ht;

#define HT_TRY(e)                       \
    do {                                \
        const ht_status st_ = (e);      \
        if (st_ != HT_OK) return st_;   \
    } while (0)

namespace {

ht_status grad_args(GradArgs &a, const void *logits, int64_t ld, int32_t type, int64_t M, int64_t V, const int32_t *ids,
                    int32_t k, float temperature, void *dx, int64_t ldd, bool grad) {
    HT_TRY(check_logits(logits, ld, M, V, type));
    if (grad) HT_TRY(check_logits(dx, ldd, M, V, type));
    if (k > 0 && !ids) return HT_EINVAL;
    if (!al4(ids)) return HT_EALIGN;
    a.x = logits;
    a.dx = dx;
    a.ld = ld;
    a.ldd = ldd;
    a.V = V;
    a.c = kLog2e / temperature;
    a.inv_t = 1.0f / temperature;
    a.ids = ids;
    a.k = k;
    a.same = grad && same_alignment(logits, ld, dx, ldd, M, act_size(type));
    return HT_OK;
}

ht_status check_entries(int32_t k, int32_t least) { return k < least || k > kMaxEntries ? HT_ESHAPE : HT_OK; }

}  // namespace

extern "C" ht_status ht_token_logprobs_backward(const float *d_logp, const float *d_entropy, const void *logits,
                                                int64_t ld, int32_t type, int64_t M, int64_t V, const int32_t *tokens,
                                                int32_t n_tok, const float *stats, const float *entropy,
                                                float temperature, void *dx, int64_t ldd, ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, temperature));
    HT_TRY(check_entries(n_tok, 0));
    if (M == 0) return HT_OK;
    GradArgs a{};
    HT_TRY(grad_args(a, logits, ld, type, M, V, tokens, n_tok, temperature, dx, ldd, true));
    if ((n_tok > 0 && !d_logp) || !stats || (d_entropy && !entropy)) return HT_EINVAL;
    if (!al4(d_logp) || !al4(d_entropy) || !al4(stats) || !al4(entropy)) return HT_EALIGN;
    a.g = d_logp;
    a.g_entropy = d_entropy;
    a.row_stats = stats;
    a.entropy = entropy;
    return type == HT_BF16 ? launch_grad<uint16_t, false>(a, M, hipStream_t(stream))
                           : launch_grad<float, false>(a, M, hipStream_t(stream));
}

extern "C" ht_status ht_distill_loss(const void *logits, int64_t ld, int32_t type, int64_t M, int64_t V,
                                     const int32_t *ids, const float *teacher, int32_t k, float temperature, float *loss,
                                     float *stats, ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, temperature));
    HT_TRY(check_entries(k, 1));
    if (M == 0) return HT_OK;
    GradArgs a{};
    HT_TRY(grad_args(a, logits, ld, type, M, V, ids, k, temperature, nullptr, 0, false));
    if (!teacher || !loss) return HT_EINVAL;
    if (!al4(teacher) || !al4(loss) || !al4(stats)) return HT_EALIGN;
    a.teacher = teacher;
    a.loss = loss;
    a.stats = stats;
    const hipStream_t s = hipStream_t(stream);
    // a long row by a whole compute unit where there are few, a short one by a
    // wavefront where there are many
    if (type == HT_BF16) {
        if (M <= 256 && V > 16384) loss_kernel<uint16_t, 1024>(a, M, s);
        else if (M > 1024 && V <= 8192) loss_kernel<uint16_t, 64>(a, M, s);
        else loss_kernel<uint16_t, 256>(a, M, s);
    } else {
        if (M <= 256 && V > 16384) loss_kernel<float, 1024>(a, M, s);
        else if (M > 1024 && V <= 8192) loss_kernel<float, 64>(a, M, s);
        else loss_kernel<float, 256>(a, M, s);
    }
    HT_LAUNCH_CHECK();
    return HT_OK;
}

extern "C" ht_status ht_distill_backward(const float *d_loss, const void *logits, int64_t ld, int32_t type, int64_t M,
                                         int64_t V, const int32_t *ids, const float *teacher, int32_t k,
                                         const float *stats, float temperature, void *dx, int64_t ldd,
                                         ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, temperature));
    HT_TRY(check_entries(k, 1));
    if (M == 0) return HT_OK;
    GradArgs a{};
    HT_TRY(grad_args(a, logits, ld, type, M, V, ids, k, temperature, dx, ldd, true));
    if (!d_loss || !teacher || !stats) return HT_EINVAL;
    if (!al4(d_loss) || !al4(teacher) || !al4(stats)) return HT_EALIGN;
    a.teacher = teacher;
    a.weight = d_loss;
    a.row_stats = stats;
    return type == HT_BF16 ? launch_grad<uint16_t, true>(a, M, hipStream_t(stream))
                           : launch_grad<float, true>(a, M, hipStream_t(stream));
}

extern "C" ht_status ht_distill_step(const void *logits, int64_t ld, int32_t type, int64_t M, int64_t V,
                                     const int32_t *ids, const float *teacher, int32_t k, const float *weight,
                                     float temperature, float *loss, float *stats, void *dx, int64_t ldd,
                                     ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, temperature));
    HT_TRY(check_entries(k, 1));
    if (M == 0) return HT_OK;
    GradArgs a{};
    HT_TRY(grad_args(a, logits, ld, type, M, V, ids, k, temperature, dx, ldd, true));
    if (!teacher || !loss) return HT_EINVAL;
    if (!al4(teacher) || !al4(loss) || !al4(stats) || !al4(weight)) return HT_EALIGN;
    a.teacher = teacher;
    a.weight = weight;
    a.loss = loss;
    a.stats = stats;
    if (M >= (int64_t(1) << 22)) return HT_ESHAPE;   // the launch's limit on threads (1024 a row)
    return type == HT_BF16 ? launch_step<uint16_t>(a, M, hipStream_t(stream))
                           : launch_step<float>(a, M, hipStream_t(stream));
}

extern "C" ht_status ht_scale_rows(void *dx, int64_t ldd, int32_t type, int64_t M, int64_t V, const float *g,
                                   ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, 1.0f));
    if (M == 0) return HT_OK;
    HT_TRY(check_logits(dx, ldd, M, V, type));
    if (!g) return HT_EINVAL;
    if (!al4(g)) return HT_EALIGN;
    int64_t S = (V + 16383) / 16384;
    if (M * S >= (int64_t(1) << 24)) return HT_ESHAPE;    // the launch's limit on threads
    const hipStream_t s = hipStream_t(stream);
    if (type == HT_BF16) scale_kernel<<<uint32_t(M * S), 256, 0, s>>>(static_cast<uint16_t *>(dx), ldd, V, int32_t(S), g);
    else scale_kernel<<<uint32_t(M * S), 256, 0, s>>>(static_cast<float *>(dx), ldd, V, int32_t(S), g);
    HT_LAUNCH_CHECK();
    return HT_OK;
}

// distill.hip -- the loss of a student's logits against a teacher's top logits,
// the gradients of logits, and both in one pass.
//
//   p = softmax over a row's kept entries of t / temperature,
//   q = softmax over the vocabulary of x / temperature,
//   loss = sum_j p_j (log p_j - log q[id_j]);
//   d loss / d x_v = 1 / temperature (q_v - sum_{j: id_j = v} p_j).
//
// Every gradient here is  scale (sum_{j: id_j = v} g_j - q_v (G + E (log q_v + H)))
// with few g_j: log probabilities of given tokens have G = sum g and E the
// entropy's gradient, distillation g_j = p_j, G = 1, E = 0 and a scale of the
// other sign.  The dense part is written for every entry, then the few given
// ones are written again, whole.
//
// Bound by HBM: logits once and the gradient once.  The step holds a row in the
// registers of 1024 threads between its sum and its gradient where it fits
// (16-byte pieces per thread: up to 16), else it reads the row a second time,
// which the Infinity Cache serves: the rows in work are fewer than it holds.
#include "logits.h"

namespace ht {

namespace {

constexpr int kMaxEntries = 1024;   // teacher's entries or given tokens of a row

// Sum or maximum over a workgroup of NT threads; the same on all.
template <int NT>
__device__ __forceinline__ float group_total(float v, float *part) {
    v = wave_sum(v);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = 0.f;
#pragma unroll
    for (int i = 0; i < NT / 64; ++i) v += part[i];
    return v;
}
template <int NT>
__device__ __forceinline__ float group_top(float v, float *part) {
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) v = fmaxf(v, __shfl_xor(v, d));
    __syncthreads();
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = v;
    __syncthreads();
    v = part[0];
#pragma unroll
    for (int i = 1; i < NT / 64; ++i) v = fmaxf(v, part[i]);
    return v;
}

// The teacher's distribution of a row: ids (-1: not kept) and p of its k
// entries into LDS; returns whether any entry is kept.  logs: log2 p too.
template <int NT>
__device__ __forceinline__ bool teacher_row(const int32_t *ids, const float *t, int k, int64_t V, float c, int32_t *id,
                                            float *p, float *logs, float *part) {
    float top = kLowest;
    for (int j = threadIdx.x; j < k; j += NT) {
        const int32_t v = ids[j];
        const bool in = v >= 0 && v < V;
        id[j] = in ? v : -1;
        p[j] = in ? t[j] : -__builtin_inff();
        top = fmaxf(top, p[j]);
    }
    top = group_top<NT>(top, part);
    float sum = 0.f;
    for (int j = threadIdx.x; j < k; j += NT) {
        const float d = (p[j] - top) * c;
        if (logs) logs[j] = d;
        p[j] = exp2_fast(d);
        sum += p[j];
    }
    sum = group_total<NT>(sum, part);
    const float inv = 1.0f / sum, b = log2f(sum);
    for (int j = threadIdx.x; j < k; j += NT) {
        p[j] = sum == 0.f ? 0.f : p[j] * inv;
        if (logs) logs[j] -= b;
    }
    __syncthreads();
    return sum != 0.f;
}

// sum p (log p - log q), given each entry's logit.
template <typename T, int NT>
__device__ __forceinline__ float teacher_loss(const T *row, int k, const int32_t *id, const float *p, const float *logs,
                                              const RowOut &o, float inv_t, float *part) {
    float loss = 0.f;
    for (int j = threadIdx.x; j < k; j += NT) {
        // an entry without weight adds nothing, whatever the student says of it
        if (id[j] >= 0 && p[j] != 0.f) loss += p[j] * (logs[j] * kLn2 - logp_of(o, LogitType<T>::get(row + id[j]), inv_t));
    }
    return group_total<NT>(loss, part);
}

template <int NT>
__device__ __forceinline__ RowStat group_stat(RowStat r, float c, RowStat *stats) {
    r = stat_wave(r, c);
    __syncthreads();
    if ((threadIdx.x & 63) == 0) stats[threadIdx.x >> 6] = r;
    __syncthreads();
    r = stats[0];
#pragma unroll
    for (int w = 1; w < NT / 64; ++w) r = stat_join(r, stats[w], c);
    return r;
}

template <typename T>
__device__ __forceinline__ u32x4 no_entries() {
    return sizeof(T) == 4 ? u32x4{0xFF800000u, 0xFF800000u, 0xFF800000u, 0xFF800000u}
                          : u32x4{0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u};   // -Inf
}

// Statistics of a row (without entropy), read once by a workgroup.
template <typename T, int NT, int U>
__device__ __forceinline__ RowStat read_row(const T *p, int64_t n, float c) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec;
    const Span sp = span_of(p, n);
    RowStat r = stat_none();
    const u32x4 *v = reinterpret_cast<const u32x4 *>(p + sp.head);
    if (int(threadIdx.x) < sp.head + sp.tail) {
        const int64_t i = int(threadIdx.x) < sp.head ? int64_t(threadIdx.x) : n - sp.tail + (int(threadIdx.x) - sp.head);
        const float x = L::get(p + i);
        stat_add<1, false>(r, &x, x, c);
    }
    u32x4 next[U];
    const auto load = [&](int32_t at) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const int32_t i = at + u * NT + int32_t(threadIdx.x);
            next[u] = i < sp.vecs ? v[i] : no_entries<T>();
        }
    };
    load(0);
    for (int32_t at = 0; at < sp.vecs; at += U * NT) {
        float x[U * kVec];
#pragma unroll
        for (int u = 0; u < U; ++u) L::unpack(next[u], x + u * kVec);
        if (at + U * NT < sp.vecs) load(at + U * NT);
        float most = x[0];
#pragma unroll
        for (int j = 1; j < U * kVec; ++j) most = fmaxf(most, x[j]);
        stat_add<U * kVec, false>(r, x, most, c);
    }
    return r;
}

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
// Loss alone
// ---------------------------------------------------------------------------
template <typename T, int NT>
__global__ __launch_bounds__(NT) void distill_loss_kernel(GradArgs a) {
    extern __shared__ float lds[];                   // ids, p, log p
    __shared__ float part[NT / 64];
    __shared__ RowStat stats[NT / 64];
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *p = lds + a.k, *logs = lds + 2 * a.k;
    const int64_t m = blockIdx.x;
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    RowStat r = read_row<T, NT, 16 / LogitType<T>::kVec>(row, a.V, a.c);
    const bool any = teacher_row<NT>(a.ids + m * a.k, a.teacher + m * a.k, a.k, a.V, a.c, id, p, logs, part);
    const RowOut o = row_out(group_stat<NT>(r, a.c, stats));
    const float loss = teacher_loss<T, NT>(row, a.k, id, p, logs, o, a.inv_t, part);
    if (threadIdx.x == 0) {
        a.loss[m] = any ? loss : 0.f;
        if (a.stats) {
            a.stats[2 * m] = o.mx;
            a.stats[2 * m + 1] = o.b;
        }
    }
}

// ---------------------------------------------------------------------------
// Gradients
// ---------------------------------------------------------------------------
// The dense part's coefficients of a row.
struct Dense {
    float mx, b, c, G, E, H, scale;
    bool zero;           // the row's gradient is zero whatever its logits are
};

__device__ __forceinline__ float dense_of(const Dense &d, float x, bool ent) {
    const float l = (x - d.mx) * d.c - d.b;
    const float q = exp2_fast(l);
    float w = d.G;
    if (ent) w += d.E * (fmaxf(l, kFar) * kLn2 + d.H);
    return -d.scale * (q * w);
}

// Whole pieces and single entries of [c0, c0 + n) of a row; HELD 16-byte pieces
// per thread are in registers already.
template <typename T, int NT, bool ENT>
__device__ __forceinline__ u32x4 dense_piece(const Dense &d, u32x4 u) {
    using L = LogitType<T>;
    float x[L::kVec];
    L::unpack(u, x);
#pragma unroll
    for (int j = 0; j < L::kVec; ++j) x[j] = d.zero ? 0.f : dense_of(d, x[j], ENT);
    return L::pack(x);
}

template <typename T>
__device__ __forceinline__ void put_piece(T *y, u32x4 u, bool whole) {
    using L = LogitType<T>;
    if (whole) {
        *reinterpret_cast<u32x4 *>(y) = u;
        return;
    }
    float x[L::kVec];
    L::unpack(u, x);
#pragma unroll
    for (int j = 0; j < L::kVec; ++j) L::put(y + j, x[j]);
}

// Entry j's place written whole: the dense part and every g of that place, in
// order, so that equal places write equal values.
template <typename T>
__device__ __forceinline__ void put_given(T *dx, const Dense &d, float x, int32_t v, const int32_t *id, const float *g, int k,
                                          bool ent) {
    float sum = 0.f;
    for (int i = 0; i < k; ++i) sum += id[i] == v ? g[i] : 0.f;
    LogitType<T>::put(dx + v, d.zero ? 0.f : d.scale * sum + dense_of(d, x, ent));
}

// Loss and gradient; a row is held in NV pieces per thread (0: read twice).
template <typename T, int NT, int NV>
__global__ __launch_bounds__(NT) void distill_step_kernel(GradArgs a) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec;
    extern __shared__ float lds[];                   // ids, p, log p, logits of the ids
    __shared__ float part[NT / 64];
    __shared__ RowStat stats[NT / 64];
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *p = lds + a.k, *logs = lds + 2 * a.k, *given = lds + 3 * a.k;
    const int64_t m = blockIdx.x, V = a.V;
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    T *dx = static_cast<T *>(a.dx) + m * a.ldd;
    const Span sp = span_of(row, V);
    const u32x4 *v = reinterpret_cast<const u32x4 *>(row + sp.head);
    const float w = a.weight ? a.weight[m] : 1.0f;
    const int32_t t = threadIdx.x;
    // the single entries before and after the whole pieces: at most one per thread
    const bool single = t < sp.head + sp.tail;
    const int64_t at1 = t < sp.head ? int64_t(t) : V - sp.tail + (t - sp.head);
    Dense d{};
    d.zero = true;
    float x1 = 0.f;
    u32x4 held[NV > 0 ? NV : 1];
    if (w != 0.f) {                                  // one value per row: every thread takes the same way
        RowStat r = stat_none();
        if constexpr (NV > 0) {
#pragma unroll
            for (int i = 0; i < NV; ++i) held[i] = t + i * NT < sp.vecs ? v[t + i * NT] : no_entries<T>();
        } else {
            r = read_row<T, NT, 16 / kVec>(row, V, a.c);
        }
        const bool any = teacher_row<NT>(a.ids + m * a.k, a.teacher + m * a.k, a.k, V, a.c, id, p, logs, part);
        for (int j = t; j < a.k; j += NT) given[j] = id[j] >= 0 ? L::get(row + id[j]) : 0.f;
        if (single) x1 = L::get(row + at1);
        if constexpr (NV > 0) {
            if (single) stat_add<1, false>(r, &x1, x1, a.c);
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                float x[kVec], most;
                L::unpack(held[i], x);
                most = x[0];
#pragma unroll
                for (int j = 1; j < kVec; ++j) most = fmaxf(most, x[j]);
                stat_add<kVec, false>(r, x, most, a.c);
            }
        }
        const RowOut o = row_out(group_stat<NT>(r, a.c, stats));
        const float loss = teacher_loss<T, NT>(row, a.k, id, p, logs, o, a.inv_t, part);
        if (t == 0) a.loss[m] = any ? loss : 0.f;
        if (t == 0 && a.stats) {
            a.stats[2 * m] = o.mx;
            a.stats[2 * m + 1] = o.b;
        }
        d.mx = o.mx;
        d.b = o.b;
        d.c = a.c;
        d.G = 1.f;
        d.scale = -w * a.inv_t;
        d.zero = !any || o.kind == 1;
    } else if (t == 0) {
        a.loss[m] = 0.f;
        if (a.stats) a.stats[2 * m] = a.stats[2 * m + 1] = 0.f;
    }
    // the row's logits are in registers, or are read before they are written: dx may be the logits
    const bool whole = a.same != 0;
    if (single) L::put(dx + at1, d.zero ? 0.f : dense_of(d, x1, false));
    if constexpr (NV > 0) {
        if (d.zero) {
#pragma unroll
            for (int i = 0; i < NV; ++i)
                if (t + i * NT < sp.vecs) put_piece<T>(dx + sp.head + int64_t(t + i * NT) * kVec, u32x4{0, 0, 0, 0}, whole);
            return;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i)
            if (t + i * NT < sp.vecs)
                put_piece<T>(dx + sp.head + int64_t(t + i * NT) * kVec, dense_piece<T, NT, false>(d, held[i]), whole);
    } else {
        for (int32_t i = t; i < sp.vecs; i += NT) {
            const u32x4 u = d.zero ? u32x4{0, 0, 0, 0} : dense_piece<T, NT, false>(d, v[i]);
            put_piece<T>(dx + sp.head + int64_t(i) * kVec, u, whole);
        }
        if (d.zero) return;
    }
    __syncthreads();                                 // the given entries after the dense ones
    for (int j = t; j < a.k; j += NT)
        if (id[j] >= 0) put_given<T>(dx, d, given[j], id[j], id, p, a.k, false);
}

// Gradient from kept statistics: of the distillation's loss (DIST: weight is the
// loss's gradient) or of log probabilities and entropy.  A workgroup takes a
// part of a row.
template <typename T, int NT, bool DIST>
__global__ __launch_bounds__(NT) void logits_grad_kernel(GradArgs a) {
    using L = LogitType<T>;
    constexpr int kVec = L::kVec, U = 16 / kVec;
    extern __shared__ float lds[];                   // ids, g, logits of the ids
    __shared__ float part[NT / 64];
    int32_t *id = reinterpret_cast<int32_t *>(lds);
    float *g = lds + a.k, *given = lds + 2 * a.k;
    const int64_t m = int64_t(blockIdx.x) / a.S, c0 = (int64_t(blockIdx.x) - m * a.S) * a.part;
    const int64_t n = min(a.V - c0, a.part);
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    T *dx = static_cast<T *>(a.dx) + m * a.ldd;
    const int32_t t = threadIdx.x;
    Dense d{};
    d.mx = a.row_stats[2 * m];
    d.b = a.row_stats[2 * m + 1];
    d.c = a.c;
    d.zero = d.mx == -__builtin_inff();              // a row that allows nothing
    if constexpr (DIST) {
        const float w = a.weight[m];
        if (w == 0.f) d.zero = true;
        if (!d.zero) d.zero = !teacher_row<NT>(a.ids + m * a.k, a.teacher + m * a.k, a.k, a.V, a.c, id, g, nullptr, part);
        d.G = 1.f;
        d.scale = -w * a.inv_t;
    } else {
        float sum = 0.f, some = 0.f;
        for (int j = t; j < a.k; j += NT) {
            const int32_t v = a.ids[m * a.k + j];
            const bool in = v >= 0 && v < a.V;
            id[j] = in ? v : -1;
            g[j] = in ? a.g[m * a.k + j] : 0.f;
            sum += g[j];
            some += g[j] != 0.f ? 1.f : 0.f;
        }
        d.G = group_total<NT>(sum, part);
        some = group_total<NT>(some, part);
        d.E = a.g_entropy ? a.g_entropy[m] : 0.f;
        d.H = a.g_entropy ? a.entropy[m] : 0.f;
        d.scale = a.inv_t;
        if (some == 0.f && d.E == 0.f) d.zero = true;
    }
    if (!d.zero) {
        for (int j = t; j < a.k; j += NT) given[j] = id[j] >= c0 && id[j] < c0 + n ? L::get(row + id[j]) : 0.f;
    }
    const Span sp = span_of(row + c0, n);
    const bool ent = !DIST && d.E != 0.f;
    const bool whole = a.same != 0, single = t < sp.head + sp.tail;
    const int64_t at1 = c0 + (t < sp.head ? int64_t(t) : n - sp.tail + (t - sp.head));
    __syncthreads();                                 // the given logits are read: dx may be the logits
    if (single) L::put(dx + at1, d.zero ? 0.f : dense_of(d, L::get(row + at1), ent));
    const u32x4 *v = reinterpret_cast<const u32x4 *>(row + c0 + sp.head);
    T *y = dx + c0 + sp.head;
    if (d.zero) {
        for (int32_t i = t; i < sp.vecs; i += NT) put_piece<T>(y + int64_t(i) * kVec, u32x4{0, 0, 0, 0}, whole);
        return;
    }
    for (int32_t at = 0; at < sp.vecs; at += U * NT) {
        u32x4 u[U];
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int32_t i = at + j * NT + t;
            if (i < sp.vecs) u[j] = __builtin_nontemporal_load(v + i);
        }
#pragma unroll
        for (int j = 0; j < U; ++j) {
            const int32_t i = at + j * NT + t;
            if (i < sp.vecs) {
                const u32x4 o = ent ? dense_piece<T, NT, true>(d, u[j]) : dense_piece<T, NT, false>(d, u[j]);
                put_piece<T>(y + int64_t(i) * kVec, o, whole);
            }
        }
    }
    __syncthreads();                                 // the given entries after the dense ones
    for (int j = t; j < a.k; j += NT)
        if (id[j] >= c0 && id[j] < c0 + n) put_given<T>(dx, d, given[j], id[j], id, g, a.k, ent);
}

// dx's rows lie as x's do within 16 bytes: whole pieces of one are whole pieces of the other.
bool same_alignment(const void *x, int64_t ld, const void *dx, int64_t ldd, int64_t M, int size) {
    return (reinterpret_cast<uintptr_t>(x) & 15) == (reinterpret_cast<uintptr_t>(dx) & 15) &&
           (M <= 1 || ((ld - ldd) * size) % 16 == 0);
}

template <typename T>
ht_status launch_step(const GradArgs &a, int64_t M, hipStream_t s) {
    constexpr int kVec = LogitType<T>::kVec;
    const uint32_t grid = uint32_t(M);
    const size_t lds = size_t(4) * size_t(a.k) * 4;
    const int64_t pieces = a.V / kVec;               // at most: the head takes some
#define HT_STEP(NT, NV) distill_step_kernel<T, NT, NV><<<grid, NT, lds, s>>>(a)
    if (pieces <= 256) HT_STEP(256, 1);
    else if (pieces <= 1024) HT_STEP(256, 4);
    else if (pieces <= 4096) HT_STEP(1024, 4);
    else if (pieces <= 8192) HT_STEP(1024, 8);
    else if (pieces <= 16384) HT_STEP(1024, 16);
    else HT_STEP(1024, 0);
#undef HT_STEP
    HT_LAUNCH_CHECK();
    return HT_OK;
}

// Parts of a row in the gradient kernel: pieces of about 16384 entries, so
// that the teacher's distribution is computed a few times per row.
void grad_shape(GradArgs &a, int64_t M) {
    int64_t S = (a.V + 16383) / 16384;
    if (M * S < 512) {
        S = (512 + M - 1) / M;
        const int64_t most = (a.V + 4095) / 4096;
        if (S > most) S = most;
    }
    while (M * S >= (int64_t(1) << 23)) S = (S + 1) / 2;   // the launch's limit on threads
    a.part = ((a.V + S - 1) / S + 7) / 8 * 8;
    a.S = int32_t((a.V + a.part - 1) / a.part);
}

template <bool DIST>
ht_status launch_grad(GradArgs &a, int64_t M, int32_t type, hipStream_t s) {
    grad_shape(a, M);
    const uint32_t grid = uint32_t(M * a.S);
    const size_t lds = size_t(3) * size_t(a.k) * 4;
    if (type == HT_BF16) logits_grad_kernel<uint16_t, 256, DIST><<<grid, 256, lds, s>>>(a);
    else logits_grad_kernel<float, 256, DIST><<<grid, 256, lds, s>>>(a);
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
    return launch_grad<false>(a, M, type, hipStream_t(stream));
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
    const size_t lds = size_t(3) * size_t(k) * 4;
    const hipStream_t s = hipStream_t(stream);
    if (type == HT_BF16) distill_loss_kernel<uint16_t, 256><<<uint32_t(M), 256, lds, s>>>(a);
    else distill_loss_kernel<float, 256><<<uint32_t(M), 256, lds, s>>>(a);
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
    return launch_grad<true>(a, M, type, hipStream_t(stream));
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

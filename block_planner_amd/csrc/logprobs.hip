// logprobs.hip -- log probabilities of given tokens, the entropy and the most
// likely alternatives of every row of logits, in one pass over them.
//
//   z = x / temperature;  lse = log sum exp z;  logp(v) = z_v - lse;
//   H = lse - sum_v p_v z_v;  alternatives: the k largest z, ties by lower index.
//
// Bound by HBM: every logit is read once.  A workgroup takes a row, or one of
// S parts of it where rows are few; each lane keeps (mx, s, t) of its entries,
// its wavefronts put aside what may be among the k largest; they meet in LDS,
// and for parts in a second kernel over the workspace.  4096 x 128000 bf16: 174 us without
// alternatives, 6.0 TB/s, 191 with 20 and 219 with 64; a row of 32000 fp32 4.6 us, 9.3
// with 20.
#include <type_traits>

#include "logits.h"

namespace ht {

namespace {

struct LogprobArgs {
    const void *x;
    int64_t ld, V, part;        // part: columns per workgroup
    int32_t S, k, n_tok;
    float c, inv_t;             // log2(e) / temperature, 1 / temperature
    const int32_t *tokens;
    float *logp, *entropy, *top, *stats;
    int32_t *top_tokens;
    RowStat *ws_stats;          // [M][S], then
    uint64_t *ws_top;           // [M][S][k]
};

// The wavefronts' lists as one, in the first wavefront.
template <int NW>
__device__ __forceinline__ void meet_lists(uint64_t &list, uint64_t *lists) {
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    __syncthreads();
    lists[wave * 64 + lane] = list;
    __syncthreads();
    for (int w = NW / 2; w > 0; w >>= 1) {
        if (wave < w) {
            list = join_lists(list, lists[(wave + w) * 64 + 63 - lane], lane);
            lists[wave * 64 + lane] = list;
        }
        __syncthreads();
    }
}

template <typename T>
__device__ __forceinline__ void write_row(const LogprobArgs &a, int64_t m, RowStat r, uint64_t list, bool tops) {
    const RowOut o = row_out(r);
    const T *row = static_cast<const T *>(a.x) + m * a.ld;
    for (int j = threadIdx.x; j < a.n_tok; j += blockDim.x) {
        const int32_t v = a.tokens[m * a.n_tok + j];
        a.logp[m * a.n_tok + j] = v >= 0 && v < a.V ? logp_of(o, LogitType<T>::get(row + v), a.inv_t) : 0.f;
    }
    if (threadIdx.x == 0) {
        if (a.entropy) a.entropy[m] = o.entropy;
        if (a.stats) {
            a.stats[2 * m] = o.mx;
            a.stats[2 * m + 1] = o.b;
        }
    }
    if (!tops || threadIdx.x >= 64) return;
    const int lane = threadIdx.x;
    int32_t token = int32_t(entry_index(list));
    float logp = logp_of(o, key_value(uint32_t(list >> 32)), a.inv_t);
    const int found = __popcll(__ballot(list != 0));
    if (found < a.k) {
        // fewer than k are allowed: the first of the others (the rest is -Inf: 128 entries hold 64 of them)
        if (list == 0) logp = o.kind == 2 ? __builtin_nanf("") : -__builtin_inff();
        int have = found;
        for (int64_t i0 = 0; i0 < a.V && have < a.k && o.kind != 2; i0 += 64) {
            const bool in = i0 + lane < a.V && LogitType<T>::get(row + i0 + lane) == -__builtin_inff();
            uint64_t who = __ballot(in);
            for (; who && have < a.k; ++have, who &= who - 1)
                if (lane == have) token = int32_t(i0) + __builtin_ctzll(who);
        }
    }
    if (lane < a.k) {
        a.top[m * a.k + lane] = logp;
        a.top_tokens[m * a.k + lane] = o.kind == 2 ? -1 : token;
    }
}

template <typename T, int NT, bool TOP, bool PARTS>
__global__ __launch_bounds__(NT, TOP ? 6 : 8) void logprob_kernel(LogprobArgs a) {
    constexpr int NW = NT / 64;
    __shared__ std::conditional_t<TOP, TopShared<T, NW>, int> sh;
    __shared__ RowStat stats[NW];
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    if constexpr (TOP) {
        sh.init();
        __syncthreads();
    }
    const int64_t m = PARTS ? int64_t(blockIdx.x) / a.S : int64_t(blockIdx.x);
    const int64_t sl = PARTS ? int64_t(blockIdx.x) - m * a.S : 0;
    const int64_t c0 = sl * a.part, n = min(a.V - c0, a.part);
    const T *p = static_cast<const T *>(a.x) + m * a.ld + c0;
    TopList<T, NW> list;
    if constexpr (TOP) list.init(&sh, a.k);
    RowStat r = scan_row<T, NT, true, TOP>(p, n, uint32_t(c0), a.c, list);
    if (lane == 0) stats[wave] = r;
    if constexpr (TOP) list.raise();
    __syncthreads();
    r = stat_group<NW>(stats, a.c);
    if constexpr (TOP) {
        const Span sp = span_of(p, n);
        const uint32_t i0 = uint32_t(c0) + uint32_t(sp.head);
        list.gather(NT, sp.vecs, i0);
        __syncthreads();
        if (sh.count <= TopShared<T, NW>::kCands) {
            list.order();
        } else {                                     // many equal ones
            while (list.pending > 0) list.flush(NT, sp.vecs, i0);
            meet_lists<NW>(list.list, sh.lists);
        }
    }
    if constexpr (PARTS) {
        const int64_t rec = m * a.S + sl;
        if (threadIdx.x == 0) a.ws_stats[rec] = r;
        if (TOP && wave == 0 && lane < a.k) a.ws_top[rec * a.k + lane] = list.list;
    } else {
        write_row<T>(a, m, r, TOP ? list.list : 0, TOP);
    }
}

// A row's parts as one: the wavefronts take them in turn.
template <typename T, bool TOP>
__global__ __launch_bounds__(256) void logprob_join_kernel(LogprobArgs a) {
    __shared__ uint64_t lists[TOP ? 256 : 1];
    __shared__ RowStat stats[4];
    const int64_t m = blockIdx.x;
    const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
    RowStat r{-__builtin_inff(), 0.f, 0.f};
    if (int(threadIdx.x) < a.S) r = a.ws_stats[m * a.S + threadIdx.x];   // at most 256 parts
    r = stat_meet<64>(r, a.c);
    if (lane == 0) stats[wave] = r;
    uint64_t list = 0;
    if constexpr (TOP) {
        for (int i = wave; i < a.S; i += 4) {
            const int from = 63 - lane;
            const uint64_t up = from < a.k ? a.ws_top[(m * a.S + i) * a.k + from] : 0;
            list = join_lists(list, up, lane);
        }
    }
    if constexpr (TOP) meet_lists<4>(list, lists);
    else __syncthreads();
    r = stat_group<4>(stats, a.c);
    write_row<T>(a, m, r, list, TOP);
}

struct LogprobShape {
    int32_t S;
    int64_t part;
};

// Parts of a row: two workgroups for each compute unit, of at least 16384 entries
// each: parts cost a second launch and its joins.  With 20 alternatives, fp32,
// without the host's part of a call, in parts of at least 8192, 16384 and 32768:
// 1 x 128000 11.8, 12.1 and 14.4 us, 1 x 32000 10.3, 9.4 and 9.2, 64 x 32000 11.6,
// 10.2 and 10.2, 64 x 128000 14.9, 16.1 and 16.7.
LogprobShape logprob_shape(int64_t M, int64_t V) {
    LogprobShape s{1, V};
    int64_t S = (512 + M - 1) / M;
    const int64_t most = V / 16384;
    if (S > most) S = most;
    if (S > 256) S = 256;
    if (S <= 1) return s;
    s.part = ((V + S - 1) / S + 7) / 8 * 8;    // whole 16-byte pieces
    s.S = int32_t((V + s.part - 1) / s.part);
    return s;
}

template <typename T, int NT>
void launch_rows(const LogprobArgs &a, uint32_t grid, bool top, hipStream_t s) {
    if (a.S == 1) {
        if (top) logprob_kernel<T, NT, true, false><<<grid, NT, 0, s>>>(a);
        else logprob_kernel<T, NT, false, false><<<grid, NT, 0, s>>>(a);
    } else {
        if (top) logprob_kernel<T, NT, true, true><<<grid, NT, 0, s>>>(a);
        else logprob_kernel<T, NT, false, true><<<grid, NT, 0, s>>>(a);
    }
}

// 512 threads where workgroups are few, or the list is long: without the host's
// part of a call, with 20 alternatives, 10.2 us for 64 x 32000 fp32 (256 threads
// 12.3, 1024 12.0), 11.3 for 256 x 32000 (13.3, 14.2); with 64, 18.8 for 512 x 32000
// (256 threads 20.7), but 58 against 55 for 2048 x 32000.  A wavefront of its own for
// each of many short rows, which shares the list's work with no other: with 20, bf16, 44
// us for 16384 x 4000 (256 threads 84), 60 for 4096 x 32000 (65), fp32 47.5 for
// 2048 x 32000 (50), but 189 against 186 for 4096 x 128000 bf16.
template <typename T>
ht_status launch_logprobs(LogprobArgs &a, int64_t M, hipStream_t s) {
    const bool top = a.k > 0;
    const uint32_t grid = uint32_t(M * a.S);
    if (grid <= 256 || (a.k > 32 && grid <= 1024)) launch_rows<T, 512>(a, grid, top, s);
    else if (grid > 1024 && a.k <= 32 && a.V <= 32768) launch_rows<T, 64>(a, grid, top, s);
    else launch_rows<T, 256>(a, grid, top, s);
    if (a.S > 1) {
        HT_LAUNCH_CHECK();
        if (top) logprob_join_kernel<T, true><<<uint32_t(M), 256, 0, s>>>(a);
        else logprob_join_kernel<T, false><<<uint32_t(M), 256, 0, s>>>(a);
    }
    HT_LAUNCH_CHECK();
    return HT_OK;
}

ht_status check_top(int64_t V, int32_t k, int32_t n_tok) {
    return k < 0 || k > kMaxTop || k > V || n_tok < 0 || n_tok > 1024 ? HT_ESHAPE : HT_OK;
}

}  // namespace
}  // namespace ht

using namespace ht;

#define HT_TRY(e)                       \
    do {                                \
        const ht_status st_ = (e);      \
        if (st_ != HT_OK) return st_;   \
    } while (0)

extern "C" ht_status ht_token_logprobs_workspace(int64_t M, int64_t V, int32_t k, size_t *bytes) {
    if (!bytes) return HT_EINVAL;
    HT_TRY(check_logit_shape(M, V, HT_FP32, 1.0f));
    HT_TRY(check_top(V, k, 0));
    *bytes = 0;
    if (M == 0) return HT_OK;
    const LogprobShape sh = logprob_shape(M, V);
    if (sh.S > 1) *bytes = align256(size_t(M) * size_t(sh.S) * sizeof(RowStat)) + size_t(M) * size_t(sh.S) * size_t(k) * 8;
    return HT_OK;
}

extern "C" ht_status ht_token_logprobs(const void *logits, int64_t ld, int32_t type, int64_t M, int64_t V,
                                       const int32_t *tokens, int32_t n_tok, int32_t k, float temperature, float *logp,
                                       float *entropy, float *top, int32_t *top_tokens, float *stats, void *ws,
                                       size_t ws_bytes, ht_stream stream) {
    HT_TRY(check_logit_shape(M, V, type, temperature));
    HT_TRY(check_top(V, k, n_tok));
    if (M == 0) return HT_OK;
    HT_TRY(check_logits(logits, ld, M, V, type));
    if ((n_tok > 0 && (!tokens || !logp)) || (k > 0 && (!top || !top_tokens))) return HT_EINVAL;
    if (!al4(tokens) || !al4(logp) || !al4(entropy) || !al4(top) || !al4(top_tokens) || !al4(stats) || !al16p(ws))
        return HT_EALIGN;
    size_t need = 0;
    HT_TRY(ht_token_logprobs_workspace(M, V, k, &need));
    if (need && (!ws || ws_bytes < need)) return HT_ESMALL;
    const LogprobShape sh = logprob_shape(M, V);
    LogprobArgs a{};
    a.x = logits;
    a.ld = ld;
    a.V = V;
    a.part = sh.part;
    a.S = sh.S;
    a.k = k;
    a.n_tok = n_tok;
    a.c = kLog2e / temperature;
    a.inv_t = 1.0f / temperature;
    a.tokens = tokens;
    a.logp = logp;
    a.entropy = entropy;
    a.top = top;
    a.top_tokens = top_tokens;
    a.stats = stats;
    a.ws_stats = static_cast<RowStat *>(ws);
    if (sh.S > 1) a.ws_top = reinterpret_cast<uint64_t *>(static_cast<uint8_t *>(ws) + align256(size_t(M) * size_t(sh.S) * sizeof(RowStat)));
    return type == HT_BF16 ? launch_logprobs<uint16_t>(a, M, hipStream_t(stream))
                           : launch_logprobs<float>(a, M, hipStream_t(stream));
}
